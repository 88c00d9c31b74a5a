// The block norm's kernels: RMS norms before and after a block, fused with the
// block's gate and the residual scale.
//
// HBM-bound: the forward pass reads x and y and writes r and n, the backward
// pass reads y, r, dr, dn and writes dx, dy, each once.  A row is held in the
// registers of the threads that share it (8 channels per thread and step), so
// both norms of a row and everything between them take one pass over memory.
#pragma once

#include <cuda_bf16.h>

#include "amsim_internal.h"

namespace amsim {
namespace bn {

using bf16 = __nv_bfloat16;

struct Params {
    const void *x, *y, *dr, *dn, *rin;
    void *r, *n, *dx, *dy;
    const float *gate, *w_post, *w_pre;
    float *rstd_post, *rstd_pre;           // written by the forward pass, read by the backward
    float *dgate, *dw_post, *dw_pre;
    float *part_gate, *part_post, *part_pre;   // backward: row sums per share, [share][cols]
    long long rows, gate_rows;
    long long ldx, ldy, ldr, ldn, lddr, lddn, lddx, lddy;
    long long item_rows, items;            // backward: rows per share, shares
    int splits;                            // backward: shares per row of the gate
    int cols;
    int tpr, rpb;                          // threads per row, rows per thread block
    float alpha, eps;
};

// Eight channels of a row, in fp32.
struct Eight {
    float v[8];
};

template <typename T>
__device__ __forceinline__ float get(const T *p);
template <>
__device__ __forceinline__ float get<float>(const float *p) { return *p; }
template <>
__device__ __forceinline__ float get<bf16>(const bf16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16 *p, float v) { *p = __float2bfloat16_rn(v); }

// What a thread keeps of a row between its load and its use: the raw words.
template <typename T>
struct Raw {
    uint4 q[sizeof(T) == 2 ? 1 : 2];
};

// Channel of element e (0..7) of step k: vector steps take 8 neighbours per
// thread, scalar ones stride by the threads of the row.
template <bool VEC>
__device__ __forceinline__ int channel(int k, int e, int t, int tpr)
{
    return VEC ? (k * tpr + t) * 8 + e : (k * 8 + e) * tpr + t;
}

template <bool VEC, typename T>
__device__ __forceinline__ void load_raw(Raw<T> &d, const T *row, int k, int t, int tpr, int cols)
{
    if constexpr (VEC) {
        const int c = channel<true>(k, 0, t, tpr);
        if (c < cols) {
            const uint4 *p = reinterpret_cast<const uint4 *>(row + c);
            d.q[0] = p[0];
            if constexpr (sizeof(T) == 4) d.q[1] = p[1];
        } else {
            d.q[0] = make_uint4(0, 0, 0, 0);
            if constexpr (sizeof(T) == 4) d.q[1] = make_uint4(0, 0, 0, 0);
        }
    } else {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = channel<false>(k, e, t, tpr);
            if constexpr (sizeof(T) == 4) w[e] = c < cols ? reinterpret_cast<const uint32_t *>(row)[c] : 0u;
            else w[e] = c < cols ? reinterpret_cast<const uint16_t *>(row)[c] : 0u;
        }
        if constexpr (sizeof(T) == 4) {
            d.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
            d.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            d.q[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        }
    }
}

template <typename T>
__device__ __forceinline__ Eight widen(const Raw<T> &d)
{
    Eight r;
    if constexpr (sizeof(T) == 4) {
        const uint32_t w[8] = {d.q[0].x, d.q[0].y, d.q[0].z, d.q[0].w, d.q[1].x, d.q[1].y, d.q[1].z, d.q[1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = __uint_as_float(w[e]);
    } else {
        const uint32_t w[4] = {d.q[0].x, d.q[0].y, d.q[0].z, d.q[0].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r.v[2 * e] = __uint_as_float(w[e] << 16);
            r.v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
    return r;
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T *row, int k, int t, int tpr, int cols, const Eight &r)
{
    if constexpr (VEC) {
        const int c = channel<true>(k, 0, t, tpr);
        if (c >= cols) return;
        uint4 *p = reinterpret_cast<uint4 *>(row + c);
        if constexpr (sizeof(T) == 4) {
            p[0] = make_uint4(__float_as_uint(r.v[0]), __float_as_uint(r.v[1]), __float_as_uint(r.v[2]),
                              __float_as_uint(r.v[3]));
            p[1] = make_uint4(__float_as_uint(r.v[4]), __float_as_uint(r.v[5]), __float_as_uint(r.v[6]),
                              __float_as_uint(r.v[7]));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(r.v[2 * e], r.v[2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t *>(&b);
            }
            p[0] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = channel<false>(k, e, t, tpr);
            if (c < cols) put(row + c, r.v[e]);
        }
    }
}

// Eight fp32 weights (ones where there are none).
template <bool VEC>
__device__ __forceinline__ Eight weights(const float *w, int k, int t, int tpr, int cols)
{
    Eight r;
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = 1.0f;
        return r;
    }
    Raw<float> d;
    load_raw<VEC, float>(d, w, k, t, tpr, cols);
    return widen(d);
}

// Sum of `x` over the threads of a row (its warps are neighbours in the
// block).  `which` alternates between two buffers, so that one barrier per sum
// is enough.
__device__ __forceinline__ float row_sum(float x, int warps, float (*red)[32], int &which)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    if (warps == 1) return x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *buf = red[which];
    which ^= 1;
    if (lane == 0) buf[warp] = x;
    __syncthreads();
    const int first = warp / warps * warps;
    x = lane < warps ? buf[first + lane] : 0.0f;
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    return x;
}

template <int NV, int THREADS, bool VEC, typename X, typename Y, typename N>
__global__ void __launch_bounds__(THREADS) fwd_kernel(const Params p)
{
    __shared__ float red[2][32];
    int which = 0;
    const int t = threadIdx.x % p.tpr, warps = p.tpr >> 5;
    const long long row = (long long)blockIdx.x * p.rpb + threadIdx.x / p.tpr;
    const bool on = row < p.rows;
    const int cols = on ? p.cols : 0;
    const X *x = static_cast<const X *>(p.x) + row * p.ldx;
    const Y *y = static_cast<const Y *>(p.y) + row * p.ldy;
    Raw<X> xr[NV];
    Raw<Y> yr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) load_raw<VEC, X>(xr[k], x, k, t, p.tpr, cols);
    if (p.y) {
#pragma unroll
        for (int k = 0; k < NV; ++k) load_raw<VEC, Y>(yr[k], y, k, t, p.tpr, cols);
    }
    const float inv = 1.0f / (float)p.cols;
    float post = 1.0f;
    if (p.y && p.w_post) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Eight a = widen(yr[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(a.v[e], a.v[e], s);
        }
        post = 1.0f / sqrtf(fmaf(row_sum(s, warps, red, which), inv, p.eps));
        if (on && t == 0 && p.rstd_post) p.rstd_post[row] = post;
    }
    const float *gate = p.gate ? p.gate + row / p.gate_rows * p.cols : nullptr;
    Eight r[NV];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        r[k] = widen(xr[k]);
        if (p.y) {
            const Eight a = widen(yr[k]);
            const Eight w = weights<VEC>(p.w_post, k, t, p.tpr, cols), g = weights<VEC>(gate, k, t, p.tpr, cols);
            const float c = p.alpha * post;
#pragma unroll
            for (int e = 0; e < 8; ++e) r[k].v[e] = fmaf(c * a.v[e], w.v[e] * g.v[e], r[k].v[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(r[k].v[e], r[k].v[e], s);
        if (p.r) store8<VEC, X>(static_cast<X *>(p.r) + row * p.ldr, k, t, p.tpr, cols, r[k]);
    }
    if (!p.n) return;
    const float pre = 1.0f / sqrtf(fmaf(row_sum(s, warps, red, which), inv, p.eps));
    if (on && t == 0 && p.rstd_pre) p.rstd_pre[row] = pre;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const Eight w = weights<VEC>(p.w_pre, k, t, p.tpr, cols);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[k].v[e] = r[k].v[e] * pre * w.v[e];
        store8<VEC, N>(static_cast<N *>(p.n) + row * p.ldn, k, t, p.tpr, cols, r[k]);
    }
}

// Adds the row groups' sums of a block (in group order) and leaves group 0
// with the total.  `buf`: one float per thread.
__device__ __forceinline__ float group_sum(float x, int tpr, int rpb, float *buf)
{
    if (rpb == 1) return x;
    __syncthreads();
    buf[threadIdx.x] = x;
    __syncthreads();
    if ((int)threadIdx.x < tpr) {
        x = 0.0f;
        for (int g = 0; g < rpb; ++g) x += buf[g * tpr + threadIdx.x];
    }
    return x;
}

// A block takes shares (items) of item_rows rows; the rows of a share have the
// same gate.  Column sums stay in registers over a share's rows:
//   a = sum dx * yh  (per gate row: dgate = alpha w_post a, dw_post = alpha sum gate a)
//   b = sum dn * rh  (dw_pre).
// `a` leaves at the end of each share, `b` at the end of the block.
template <int NV, int THREADS, bool VEC, typename X, typename Y, typename N>
__global__ void __launch_bounds__(THREADS) bwd_kernel(const Params p)
{
    __shared__ float red[2][32];
    __shared__ float buf[THREADS];
    int which = 0;
    const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, warps = p.tpr >> 5;
    const float inv = 1.0f / (float)p.cols;
    const bool want_y = p.y != nullptr, want_n = p.dn != nullptr;
    const bool sums_a = want_y && (p.dgate || p.dw_post), sums_b = want_n && p.dw_pre;
    float b[NV * 8];
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) b[i] = 0.0f;
    bool fresh = true;                       // no share has left its sums in part_post yet
    for (long long item = blockIdx.x; item < p.items; item += gridDim.x) {
        const long long gi = item / p.splits;
        const long long g0 = gi * p.gate_rows, g1 = min(g0 + p.gate_rows, p.rows);
        const long long r0 = g0 + (item - gi * p.splits) * p.item_rows, r1 = min(r0 + p.item_rows, g1);
        const float *gate = p.gate ? p.gate + gi * p.cols : nullptr;
        float a[NV * 8];
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) a[i] = 0.0f;
        for (long long rb = r0; rb < r1; rb += p.rpb) {
            const long long row = rb + group;
            const bool on = row < r1;
            const int cols = on ? p.cols : 0;
            Eight dx[NV], rr[NV];
            Raw<Y> yr[NV];
            Raw<N> nr[NV];
            float s = 0.0f;
            if (want_y) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    load_raw<VEC, Y>(yr[k], static_cast<const Y *>(p.y) + row * p.ldy, k, t, p.tpr, cols);
            }
            if (p.dr) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    Raw<X> d;
                    load_raw<VEC, X>(d, static_cast<const X *>(p.dr) + row * p.lddr, k, t, p.tpr, cols);
                    dx[k] = widen(d);
                }
            } else {
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) dx[k].v[e] = 0.0f;
            }
            if (want_n) {
                const float pre = on ? p.rstd_pre[row] : 0.0f;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    Raw<X> d;
                    load_raw<VEC, X>(d, static_cast<const X *>(p.rin) + row * p.ldr, k, t, p.tpr, cols);
                    rr[k] = widen(d);
                    load_raw<VEC, N>(nr[k], static_cast<const N *>(p.dn) + row * p.lddn, k, t, p.tpr, cols);
                }
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const Eight n = widen(nr[k]), w = weights<VEC>(p.w_pre, k, t, p.tpr, cols);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        rr[k].v[e] *= pre;
                        s = fmaf(n.v[e] * w.v[e], rr[k].v[e], s);
                        b[k * 8 + e] = fmaf(n.v[e], rr[k].v[e], b[k * 8 + e]);
                    }
                }
                s = row_sum(s, warps, red, which) * inv;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const Eight n = widen(nr[k]), w = weights<VEC>(p.w_pre, k, t, p.tpr, cols);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dx[k].v[e] = fmaf(pre, fmaf(-rr[k].v[e], s, n.v[e] * w.v[e]), dx[k].v[e]);
                }
            }
            if (p.dx) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    store8<VEC, X>(static_cast<X *>(p.dx) + row * p.lddx, k, t, p.tpr, cols, dx[k]);
            }
            if (!want_y) continue;
            const float post = p.w_post ? (on ? p.rstd_post[row] : 0.0f) : 1.0f;
            s = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const Eight y = widen(yr[k]);
                const Eight w = weights<VEC>(p.w_post, k, t, p.tpr, cols), g = weights<VEC>(gate, k, t, p.tpr, cols);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float yh = y.v[e] * post;
                    a[k * 8 + e] = fmaf(dx[k].v[e], yh, a[k * 8 + e]);
                    dx[k].v[e] *= p.alpha * g.v[e] * w.v[e];           // s of the formulas
                    s = fmaf(dx[k].v[e], yh, s);
                }
            }
            if (!p.dy) continue;
            if (p.w_post) s = row_sum(s, warps, red, which) * inv;
            else s = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const Eight y = widen(yr[k]);
                Eight o;
#pragma unroll
                for (int e = 0; e < 8; ++e) o.v[e] = post * fmaf(-y.v[e] * post, s, dx[k].v[e]);
                store8<VEC, Y>(static_cast<Y *>(p.dy) + row * p.lddy, k, t, p.tpr, cols, o);
            }
        }
        if (!sums_a) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = group_sum(a[k * 8 + e], p.tpr, p.rpb, buf);
                const int c = channel<VEC>(k, e, t, p.tpr);
                if (group == 0 && c < p.cols) {
                    if (p.splits > 1) {
                        p.part_gate[item * p.cols + c] = v;
                    } else {
                        const float g = gate ? gate[c] : 1.0f;
                        if (p.dgate) p.dgate[gi * p.cols + c] = p.alpha * (p.w_post ? p.w_post[c] : 1.0f) * v;
                        if (p.dw_post) {
                            float *slot = p.part_post + (long long)blockIdx.x * p.cols + c;
                            *slot = fmaf(p.alpha * g, v, fresh ? 0.0f : *slot);
                        }
                    }
                }
            }
        fresh = false;
    }
    if (!sums_b) return;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = group_sum(b[k * 8 + e], p.tpr, p.rpb, buf);
            const int c = channel<VEC>(k, e, t, p.tpr);
            if (group == 0 && c < p.cols) p.part_pre[(long long)blockIdx.x * p.cols + c] = v;
        }
}

// One translation unit per type of the residual stream builds its instances.
int launch_f32(bool bwd, int nv, bool vec, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st);
int launch_bf16(bool bwd, int nv, bool vec, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st);

template <int NV, int THREADS, bool VEC, typename X, typename Y, typename N>
int launch_one(bool bwd, const Params &p, unsigned grid, cudaStream_t st)
{
    const unsigned threads = (unsigned)(p.tpr * p.rpb);
    if (bwd) bwd_kernel<NV, THREADS, VEC, X, Y, N><<<grid, threads, 0, st>>>(p);
    else fwd_kernel<NV, THREADS, VEC, X, Y, N><<<grid, threads, 0, st>>>(p);
    const int rc = cuda_status(cudaGetLastError());
    if (rc == AMSIM_OK) count_launch();
    return rc;
}

template <typename X, typename Y, typename N>
int launch_types(bool bwd, int nv, bool vec, const Params &p, unsigned grid, cudaStream_t st)
{
    const bool wide = p.tpr * p.rpb > 512;
    if (vec) {
        if (nv == 1) return launch_one<1, 512, true, X, Y, N>(bwd, p, grid, st);
        if (!wide) return launch_one<2, 512, true, X, Y, N>(bwd, p, grid, st);
        return launch_one<2, 1024, true, X, Y, N>(bwd, p, grid, st);
    }
    if (nv == 1) return launch_one<1, 512, false, X, Y, N>(bwd, p, grid, st);
    if (!wide) return launch_one<2, 512, false, X, Y, N>(bwd, p, grid, st);
    return launch_one<2, 1024, false, X, Y, N>(bwd, p, grid, st);
}

template <typename X>
int launch_stream(bool bwd, int nv, bool vec, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st)
{
    if (y_type == AMSIM_F32)
        return n_type == AMSIM_F32 ? launch_types<X, float, float>(bwd, nv, vec, p, grid, st)
                                   : launch_types<X, float, bf16>(bwd, nv, vec, p, grid, st);
    return n_type == AMSIM_F32 ? launch_types<X, bf16, float>(bwd, nv, vec, p, grid, st)
                               : launch_types<X, bf16, bf16>(bwd, nv, vec, p, grid, st);
}

}  // namespace bn
}  // namespace amsim
