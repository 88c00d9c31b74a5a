// One AdamW step over many tensors, moments in fp32 or in 8-bit blocks, and the
// values of 8-bit moments.
//
// Elementwise and HBM-bound: 28 bytes per element with fp32 moments and
// gradients (p, m, v read and written, g read), 12 plus the gradient's with
// 8-bit ones, plus 2 for a bf16 copy.  The tensors' pointers travel in the
// kernel's parameters (up to 32,764 bytes), so a step is one launch with no
// table to copy or keep; a block finds its tensor by bisection over the first
// chunks.
//
// Every operation is its correctly rounded fp32 one, in the documented order
// and with no contraction into fused multiply-adds: the step is then the same
// bit for bit as the elementwise formula, and an 8-bit code never depends on
// how the compiler grouped a product and a sum.
#include <cmath>

#include <cuda_bf16.h>

#include "amsim_internal.h"

namespace {

constexpr int kThreads = 256;
constexpr int kBlock = AMSIM_ADAMW_BLOCK;
constexpr int kChunk = 4096;                       // elements of one thread block
static_assert(kChunk % (kThreads * 8) == 0 && kBlock == 32 * 8, "one 8-bit block per warp pass");

struct Tensor {
    float *p;
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    __nv_bfloat16 *copy;
    long long n;
    float keep;        // 1 - lr wd
    float rate;        // lr / (1 - beta1^step)
    int first;         // first chunk of the launch that is this tensor's
    int flags;         // kBf16Grad, kVector
};
constexpr int kBf16Grad = 1, kVector = 2;

struct Hyper {
    float beta1, one_minus_beta1, beta2, one_minus_beta2, root, eps;   // root: 1 / sqrt(1 - beta2^step)
    const float *grad_scale;
};

template <int CAP>
struct Launch {
    Hyper h;
    int count;
    Tensor t[CAP];
};
// Capacities: a launch's parameters are copied whole, so a few tensors take a
// small struct.
constexpr int kCapacity[] = {8, 64, 400};
static_assert(sizeof(Launch<400>) <= 32764, "kernel parameters");

__device__ __forceinline__ float bf16_bits(uint32_t half) { return __uint_as_float(half << 16); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The step of one element; m, v become the new moments and s = sqrt(v).
__device__ __forceinline__ float step1(float p, float g, float &m, float &v, float &s, const Hyper &h,
                                       const Tensor &t)
{
    m = __fadd_rn(__fmul_rn(m, h.beta1), __fmul_rn(g, h.one_minus_beta1));
    v = __fadd_rn(__fmul_rn(v, h.beta2), __fmul_rn(__fmul_rn(g, g), h.one_minus_beta2));
    s = __fsqrt_rn(v);
    const float u = __fdiv_rn(m, __fadd_rn(__fmul_rn(s, h.root), h.eps));
    return __fsub_rn(__fmul_rn(p, t.keep), __fmul_rn(u, t.rate));
}

template <int CAP>
__device__ __forceinline__ const Tensor &find(const Launch<CAP> &L, int chunk)
{
    int lo = 0, hi = L.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (L.t[mid].first <= chunk) lo = mid;
        else hi = mid;
    }
    return L.t[lo];
}

// Eight elements of a tensor from element i (i % 8 == 0 within the tensor).
struct Eight {
    float x[8];
};
__device__ __forceinline__ Eight load8(const float *a, long long i)
{
    Eight r;
    *reinterpret_cast<float4 *>(r.x) = *reinterpret_cast<const float4 *>(a + i);
    *reinterpret_cast<float4 *>(r.x + 4) = *reinterpret_cast<const float4 *>(a + i + 4);
    return r;
}
__device__ __forceinline__ void store8(float *a, long long i, const Eight &r)
{
    *reinterpret_cast<float4 *>(a + i) = *reinterpret_cast<const float4 *>(r.x);
    *reinterpret_cast<float4 *>(a + i + 4) = *reinterpret_cast<const float4 *>(r.x + 4);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *a, long long i, const Eight &r)
{
    *reinterpret_cast<uint4 *>(a + i) =
        make_uint4(pack_bf16(r.x[0], r.x[1]), pack_bf16(r.x[2], r.x[3]), pack_bf16(r.x[4], r.x[5]),
                   pack_bf16(r.x[6], r.x[7]));
}
__device__ __forceinline__ Eight load8_grad(const Tensor &t, long long i)
{
    if (!(t.flags & kBf16Grad)) return load8(static_cast<const float *>(t.g), i);
    const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(t.g) + i);
    Eight r;
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r.x[2 * j] = bf16_bits(w[j] & 0xFFFFu);
        r.x[2 * j + 1] = bf16_bits(w[j] >> 16);
    }
    return r;
}
__device__ __forceinline__ float load_grad(const Tensor &t, long long i)
{
    return t.flags & kBf16Grad ? __bfloat162float(static_cast<const __nv_bfloat16 *>(t.g)[i])
                               : static_cast<const float *>(t.g)[i];
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Launch<CAP> L)
{
    const Tensor &t = find(L, (int)blockIdx.x);
    const Hyper &h = L.h;
    const float gs = h.grad_scale ? *h.grad_scale : 1.0f;
    const bool scaled = h.grad_scale != nullptr;
    const long long i0 = (long long)((int)blockIdx.x - t.first) * kChunk;
    float *m = static_cast<float *>(t.m), *v = static_cast<float *>(t.v);
    if (t.flags & kVector) {
#pragma unroll
        for (int k = 0; k < kChunk / (kThreads * 8); ++k) {
            const long long i = i0 + (k * kThreads + threadIdx.x) * 8;
            if (i + 8 <= t.n) {
                Eight p = load8(t.p, i), g = load8_grad(t, i), mm = load8(m, i), vv = load8(v, i);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float s;
                    p.x[j] = step1(p.x[j], scaled ? __fmul_rn(g.x[j], gs) : g.x[j], mm.x[j], vv.x[j], s, h, t);
                }
                store8(t.p, i, p);
                store8(m, i, mm);
                store8(v, i, vv);
                if (t.copy) store8(t.copy, i, p);
            } else {
                for (long long e = i; e < t.n; ++e) {
                    float s, g = load_grad(t, e);
                    const float p = step1(t.p[e], scaled ? __fmul_rn(g, gs) : g, m[e], v[e], s, h, t);
                    t.p[e] = p;
                    if (t.copy) t.copy[e] = __float2bfloat16_rn(p);
                }
            }
        }
        return;
    }
    const long long end = i0 + kChunk < t.n ? i0 + kChunk : t.n;
    for (long long e = i0 + threadIdx.x; e < end; e += kThreads) {
        float s, g = load_grad(t, e);
        const float p = step1(t.p[e], scaled ? __fmul_rn(g, gs) : g, m[e], v[e], s, h, t);
        t.p[e] = p;
        if (t.copy) t.copy[e] = __float2bfloat16_rn(p);
    }
}

// ------------------------------------------------------------------ 8-bit moments
// Values of the codes: the square (first moment) or the fourth power (second)
// of code / top, times the block's scale.  A power of two in the exponent of
// the map buys range: the smallest second moment a block tells from zero is
// 255^-4 of its largest.
__device__ __forceinline__ float value_m(int q, float scale)
{
    const float t = __fmul_rn((float)q, 1.0f / 127.0f);
    return __fmul_rn(__fmul_rn(t, fabsf(t)), scale);
}
__device__ __forceinline__ float value_v(unsigned q, float scale)
{
    const float t = __fmul_rn((float)q, 1.0f / 255.0f);
    const float t2 = __fmul_rn(t, t);
    return __fmul_rn(__fmul_rn(t2, t2), scale);
}

// Largest value of the warp's lanes; values are magnitudes or NaN (as bits,
// magnitudes order like integers and every NaN is above infinity).
__device__ __forceinline__ float warp_top(float x)
{
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x) & 0x7FFFFFFFu));
}
__device__ __forceinline__ float top(float a, float b)
{
    const uint32_t x = __float_as_uint(a) & 0x7FFFFFFFu, y = __float_as_uint(b) & 0x7FFFFFFFu;
    return __uint_as_float(x > y ? x : y);
}
__device__ __forceinline__ float finite_or_nan(float x) { return x <= 3.402823466e38f ? x : __uint_as_float(0x7FC00000u); }

template <int CAP>
__global__ void __launch_bounds__(kThreads) adamw8_kernel(const __grid_constant__ Launch<CAP> L)
{
    const Tensor &t = find(L, (int)blockIdx.x);
    const Hyper &h = L.h;
    const float gs = h.grad_scale ? *h.grad_scale : 1.0f;
    const bool scaled = h.grad_scale != nullptr;
    const long long i0 = (long long)((int)blockIdx.x - t.first) * kChunk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int8_t *mq = static_cast<int8_t *>(t.m);
    uint8_t *vq = static_cast<uint8_t *>(t.v);
#pragma unroll
    for (int k = 0; k < kChunk / (kThreads * 8); ++k) {
        const long long b0 = i0 + (k * (kThreads / 32) + warp) * kBlock;     // the warp's block
        if (b0 >= t.n) return;
        const long long i = b0 + lane * 8;
        const bool vec = (t.flags & kVector) && b0 + kBlock <= t.n;
        const float ms = t.m_scale[b0 / kBlock], vs = t.v_scale[b0 / kBlock];
        Eight p, g, mm, vv;
        if (vec) {
            p = load8(t.p, i);
            g = load8_grad(t, i);
            const uint2 a = *reinterpret_cast<const uint2 *>(mq + i), b = *reinterpret_cast<const uint2 *>(vq + i);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t wa = j < 4 ? a.x : a.y, wb = j < 4 ? b.x : b.y;
                mm.x[j] = value_m((int8_t)(wa >> (8 * (j & 3)) & 0xFFu), ms);
                vv.x[j] = value_v(wb >> (8 * (j & 3)) & 0xFFu, vs);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = i + j < t.n;
                p.x[j] = in ? t.p[i + j] : 0.0f;
                g.x[j] = in ? load_grad(t, i + j) : 0.0f;
                mm.x[j] = in ? value_m(mq[i + j], ms) : 0.0f;
                vv.x[j] = in ? value_v(vq[i + j], vs) : 0.0f;
            }
        }
        Eight root;
        float mt = 0.0f, vt = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float s;
            p.x[j] = step1(p.x[j], scaled ? __fmul_rn(g.x[j], gs) : g.x[j], mm.x[j], vv.x[j], s, h, t);
            root.x[j] = s;
            mt = top(mt, mm.x[j]);
            vt = top(vt, vv.x[j]);
        }
        mt = warp_top(mt);
        vt = warp_top(vt);
        const float mr = __fsqrt_rn(mt), vr = __fsqrt_rn(__fsqrt_rn(vt));
        const float mk = mr > 0.0f ? __fdiv_rn(127.0f, mr) : 0.0f, vk = vr > 0.0f ? __fdiv_rn(255.0f, vr) : 0.0f;
        uint32_t ma[2] = {0, 0}, va[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int qm = (int)fminf(rintf(__fmul_rn(__fsqrt_rn(fabsf(mm.x[j])), mk)), 127.0f);
            const int sm = mm.x[j] < 0.0f ? -qm : qm;
            int qv = (int)fminf(rintf(__fmul_rn(__fsqrt_rn(root.x[j]), vk)), 255.0f);
            if (vv.x[j] > 0.0f && qv < 1) qv = 1;
            ma[j >> 2] |= (uint32_t)(sm & 0xFF) << (8 * (j & 3));
            va[j >> 2] |= (uint32_t)(qv & 0xFF) << (8 * (j & 3));
        }
        if (vec) {
            store8(t.p, i, p);
            if (t.copy) store8(t.copy, i, p);
            *reinterpret_cast<uint2 *>(mq + i) = make_uint2(ma[0], ma[1]);
            *reinterpret_cast<uint2 *>(vq + i) = make_uint2(va[0], va[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i + j < t.n) {
                    t.p[i + j] = p.x[j];
                    if (t.copy) t.copy[i + j] = __float2bfloat16_rn(p.x[j]);
                    mq[i + j] = (int8_t)(ma[j >> 2] >> (8 * (j & 3)) & 0xFFu);
                    vq[i + j] = (uint8_t)(va[j >> 2] >> (8 * (j & 3)) & 0xFFu);
                }
        }
        if (lane == 0) {
            t.m_scale[b0 / kBlock] = finite_or_nan(mt);
            t.v_scale[b0 / kBlock] = finite_or_nan(vt);
        }
    }
}

__global__ void __launch_bounds__(kThreads) moment_values_kernel(const void *codes, const float *scales, int second,
                                                                 long long n, float *out, int vec)
{
    const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * 8;
    if (i >= n) return;
    const float s = scales[i / kBlock];
    if (vec && i + 8 <= n) {
        const uint2 a = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(codes) + i);
        Eight r;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t q = (j < 4 ? a.x : a.y) >> (8 * (j & 3)) & 0xFFu;
            r.x[j] = second ? value_v(q, s) : value_m((int8_t)q, s);
        }
        store8(out, i, r);
        return;
    }
    for (long long e = i; e < n && e < i + 8; ++e)
        out[e] = second ? value_v(static_cast<const uint8_t *>(codes)[e], s)
                        : value_m(static_cast<const int8_t *>(codes)[e], s);
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int CAP>
int launch(const Hyper &h, const Tensor *t, int count, int chunks, bool eight, cudaStream_t st)
{
    Launch<CAP> L;
    L.h = h;
    L.count = count;
    for (int i = 0; i < count; ++i) L.t[i] = t[i];
    if (eight) adamw8_kernel<CAP><<<(unsigned)chunks, kThreads, 0, st>>>(L);
    else adamw_kernel<CAP><<<(unsigned)chunks, kThreads, 0, st>>>(L);
    const int rc = amsim::cuda_status(cudaGetLastError());
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}

}  // namespace

extern "C" int amsim_adamw_step(int count, const amsim_adamw_tensor *tensors, const amsim_adamw_hyper *hyper,
                                amsim_stream_t stream)
{
    if (count < 0 || count > (1 << 20) || !hyper || (count > 0 && !tensors)) return AMSIM_EINVAL;
    const amsim_adamw_hyper &y = *hyper;
    if (!std::isfinite(y.lr) || !(y.beta1 >= 0.0 && y.beta1 < 1.0) || !(y.beta2 >= 0.0 && y.beta2 < 1.0) ||
        !(y.eps >= 0.0) || !std::isfinite(y.eps) || y.step < 1 || !aligned(y.grad_scale, 4))
        return AMSIM_EINVAL;
    bool any = false, eight = false;
    for (int i = 0; i < count; ++i) {
        const amsim_adamw_tensor &a = tensors[i];
        if (a.n < 0 || (a.g_type != AMSIM_F32 && a.g_type != AMSIM_BF16) || a.reserved != 0 ||
            !std::isfinite(a.lr_scale) || !std::isfinite(a.weight_decay) || !a.m_scale != !a.v_scale)
            return AMSIM_EINVAL;
        if (a.n == 0) continue;
        if (!a.p || !a.g || !a.m || !a.v || !aligned(a.p, 4) || !aligned(a.g, a.g_type == AMSIM_BF16 ? 2 : 4) ||
            !aligned(a.copy, 2) || !aligned(a.m_scale, 4) || !aligned(a.v_scale, 4))
            return AMSIM_EINVAL;
        const bool e = a.m_scale != nullptr;
        if (!e && (!aligned(a.m, 4) || !aligned(a.v, 4))) return AMSIM_EINVAL;
        if (any && e != eight) return AMSIM_EINVAL;
        any = true;
        eight = e;
        if ((a.n + kChunk - 1) / kChunk > 0x3FFFFFFF) return AMSIM_EINVAL;
    }
    Hyper h;
    h.beta1 = (float)y.beta1;
    h.one_minus_beta1 = (float)(1.0 - y.beta1);
    h.beta2 = (float)y.beta2;
    h.one_minus_beta2 = (float)(1.0 - y.beta2);
    h.root = (float)(1.0 / std::sqrt(1.0 - std::pow(y.beta2, (double)y.step)));
    h.eps = (float)y.eps;
    h.grad_scale = y.grad_scale;
    const double correct = 1.0 - std::pow(y.beta1, (double)y.step);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    constexpr int kMost = kCapacity[2];
    Tensor t[kMost];
    int used = 0, chunks = 0;
    for (int i = 0; i <= count; ++i) {
        long long add = 0;
        if (i < count) {
            add = (tensors[i].n + kChunk - 1) / kChunk;
            if (add == 0) continue;
        }
        if (used && (i == count || used == kMost || chunks + add > 0x7FFFFFFFLL)) {
            const int rc = used <= kCapacity[0]   ? launch<kCapacity[0]>(h, t, used, chunks, eight, st)
                           : used <= kCapacity[1] ? launch<kCapacity[1]>(h, t, used, chunks, eight, st)
                                                  : launch<kMost>(h, t, used, chunks, eight, st);
            if (rc) return rc;
            used = 0;
            chunks = 0;
        }
        if (i == count) break;
        const amsim_adamw_tensor &a = tensors[i];
        Tensor &d = t[used++];
        const double lr = y.lr * (double)a.lr_scale;
        d.p = a.p;
        d.g = a.g;
        d.m = a.m;
        d.v = a.v;
        d.m_scale = a.m_scale;
        d.v_scale = a.v_scale;
        d.copy = static_cast<__nv_bfloat16 *>(a.copy);
        d.n = a.n;
        d.keep = (float)(1.0 - lr * (double)a.weight_decay);
        d.rate = (float)(lr / correct);
        d.first = chunks;
        const size_t am = eight ? 8 : 16;
        const bool vec = aligned(a.p, 16) && aligned(a.g, 16) && aligned(a.m, am) && aligned(a.v, am) &&
                         aligned(a.copy, 16);
        d.flags = (a.g_type == AMSIM_BF16 ? kBf16Grad : 0) | (vec ? kVector : 0);
        chunks += (int)add;
    }
    return AMSIM_OK;
}

extern "C" int amsim_adamw_moment_values(const void *codes, const float *scales, int second, int64_t n, float *out,
                                         amsim_stream_t stream)
{
    if (n < 0) return AMSIM_EINVAL;
    if (n == 0) return AMSIM_OK;
    if (!codes || !scales || !out || !aligned(scales, 4) || !aligned(out, 4)) return AMSIM_EINVAL;
    const long long blocks = (n + kThreads * 8 - 1) / (kThreads * 8);
    if (blocks > 0x7FFFFFFFLL) return AMSIM_EINVAL;
    moment_values_kernel<<<(unsigned)blocks, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        codes, scales, second, n, out, aligned(codes, 8) && aligned(out, 16));
    const int rc = amsim::cuda_status(cudaGetLastError());
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}
