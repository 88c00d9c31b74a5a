// Dropout of a tensor, with the residual it is added to.  No mask is kept: a
// thread draws its elements' numbers (philox.cuh).  67 M bf16 elements with a residual
// take 72 us, 0.84 of a plain copy's rate, and 64 % of the multiplier pipe.
#include <cuda_bf16.h>

#include "philox.cuh"

namespace {

using amsim::Drop;

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float v, float *o) { *o = v; }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(v); }

// Pieces of 16 bytes a thread: 1, 2, 4, 8 take 84, 76, 72, 80 us for that.
constexpr int kThreads = 256, kPer = 4;

template <typename T>
union Piece {
    uint4 u;
    T e[16 / sizeof(T)];
    __device__ Piece() {}
};

template <typename T, bool VEC, bool RESIDUAL>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const T *x, const T *residual, T *y, int64_t n, const Drop d)
{
    constexpr int E = 16 / sizeof(T);
    const uint64_t call = amsim::drop_call(d);
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kPer) + threadIdx.x;
    Piece<T> in[kPer], res[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t at = (first + i * kThreads) * E;
        if (VEC && at + E <= n) {
            in[i].u = *reinterpret_cast<const uint4 *>(x + at);
            if (RESIDUAL) res[i].u = *reinterpret_cast<const uint4 *>(residual + at);
        } else {
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (at + k < n) {
                    in[i].e[k] = x[at + k];
                    if (RESIDUAL) res[i].e[k] = residual[at + k];
                }
        }
    }
    // the numbers' upper halves are the same for all of a thread's quads but where they pass 2^32
    uint32_t upper = (uint32_t)((uint64_t)(first * E) >> 34);
    amsim::QuadStream stream = amsim::quad_stream(upper, call, d);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t at = (first + i * kThreads) * E;
        if (at >= n) return;
        if ((uint32_t)((uint64_t)at >> 34) != upper) {
            upper = (uint32_t)((uint64_t)at >> 34);
            stream = amsim::quad_stream(upper, call, d);
        }
        Piece<T> out;
#pragma unroll
        for (int q = 0; q < E; q += 4) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = widen(in[i].e[q + k]);
            if (d.border) {
                const uint4 u = amsim::quad_words((uint32_t)((uint64_t)(at + q) >> 2), stream, d);
                v[0] = u.x >= d.border ? v[0] * d.scale : 0.0f;
                v[1] = u.y >= d.border ? v[1] * d.scale : 0.0f;
                v[2] = u.z >= d.border ? v[2] * d.scale : 0.0f;
                v[3] = u.w >= d.border ? v[3] * d.scale : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) narrow(RESIDUAL ? v[k] + widen(res[i].e[q + k]) : v[k], &out.e[q + k]);
        }
        if (VEC && at + E <= n) {
            *reinterpret_cast<uint4 *>(y + at) = out.u;
        } else {
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (at + k < n) y[at + k] = out.e[k];
        }
    }
}

template <typename T>
int run(const void *x, const void *residual, void *y, int64_t n, const Drop &d, cudaStream_t st)
{
    const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                          reinterpret_cast<uintptr_t>(y);
    if (all & (sizeof(T) - 1)) return AMSIM_EINVAL;
    const int64_t block = (int64_t)kThreads * kPer * (16 / (int64_t)sizeof(T)), grid = (n + block - 1) / block;
    if (grid > 0x7FFFFFFF) return AMSIM_EINVAL;
    const bool vec = !(all & 15);
    auto *kernel = residual ? (vec ? dropout_kernel<T, true, true> : dropout_kernel<T, false, true>)
                            : (vec ? dropout_kernel<T, true, false> : dropout_kernel<T, false, false>);
    kernel<<<(unsigned)grid, kThreads, 0, st>>>(static_cast<const T *>(x), static_cast<const T *>(residual),
                                                static_cast<T *>(y), n, d);
    const int rc = amsim::cuda_status(cudaGetLastError());
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}

}  // namespace

extern "C" int amsim_dropout(const amsim_dropout_desc *desc, int type, int64_t n, const void *x, const void *residual,
                             void *y, amsim_stream_t stream)
{
    Drop d;
    if (!desc || !amsim::make_drop(*desc, &d) || n < 0 || (type != AMSIM_F32 && type != AMSIM_BF16)) return AMSIM_EINVAL;
    if (n == 0) return AMSIM_OK;
    if (!x || !y) return AMSIM_EINVAL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return type == AMSIM_F32 ? run<float>(x, residual, y, n, d, st) : run<__nv_bfloat16>(x, residual, y, n, d, st);
}
