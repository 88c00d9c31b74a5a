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
// Measured: 256 million parameters in 200 tensors, fp32 moments and a bf16
// copy, 1.08 ms (7.1 TB/s, a little over a plain copy's rate).  With 8-bit
// moments and bf16 gradients the same step takes 829 us of the bytes' 608: some
// 100 instructions an element (decode, two roundings to codes, the block's
// maximum) fill 0.72 of the issue slots.
//
// Every operation is its correctly rounded fp32 one, in the documented order
// and with no contraction into fused multiply-adds: the step is then the same
// bit for bit as the elementwise formula, and an 8-bit code never depends on
// how the compiler grouped a product and a sum.
#include <cmath>

#include <cuda_bf16.h>

#include "amsim_internal.h"
#include "pairs.cuh"

namespace {

using amsim::both;
using amsim::mul2;

constexpr int kThreads = 256;
constexpr int kBlock = AMSIM_ADAMW_BLOCK;
constexpr int kPass = kThreads * 8;                // elements a thread block takes at once
static_assert(kBlock == 32 * 8, "one 8-bit block per warp and pass");

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
constexpr int kCapacity[] = {8, 128, 400};
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

// The tensor of a block's chunk: one thread looks, so that the others' issue
// slots are not spent on it.
template <int CAP>
__device__ __forceinline__ const Tensor &find(const Launch<CAP> &L, int chunk)
{
    __shared__ int found;
    if (threadIdx.x == 0) {
        int lo = 0, hi = L.count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (L.t[mid].first <= chunk) lo = mid;
            else hi = mid;
        }
        found = lo;
    }
    __syncthreads();
    return L.t[found];
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
    const long long i0 = (long long)((int)blockIdx.x - t.first) * kPass;
    float *m = static_cast<float *>(t.m), *v = static_cast<float *>(t.v);
    const long long i = i0 + threadIdx.x * 8;
    if ((t.flags & kVector) && i + 8 <= t.n) {
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
        return;
    }
    // a tensor's last elements by the thread they fall to, unaligned ones neighbour by neighbour
    const bool vec = t.flags & kVector;
    const long long end = min(vec ? i + 8 : i0 + kPass, t.n);
    for (long long e = vec ? i : i0 + threadIdx.x; e < end; e += vec ? 1 : kThreads) {
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
//
// Codes and floats are converted through the mantissa of 2^23 (or 1.5 * 2^23):
// the conversion and rounding instructions share the unit of the roots, which
// at a quarter of the rate would alone take 0.9 of the time of the bytes.
constexpr uint32_t kOneUlp = 0x4B000000u;          // 2^23: its ulp is 1
constexpr float kRounder = 12582912.0f;            // 1.5 * 2^23: x + kRounder rounds x to an integer

// Byte `j` of `w` as a float (signed: as int8).
template <bool SIGNED>
__device__ __forceinline__ float byte_float(uint32_t w, int j)
{
    const uint32_t bits = __byte_perm(SIGNED ? w ^ 0x80808080u : w, kOneUlp, 0x7540 + j);
    return __fsub_rn(__uint_as_float(bits), SIGNED ? 8388608.0f + 128.0f : 8388608.0f);
}

__device__ __forceinline__ float2 values_m(float2 q, float scale)
{
    const float2 t = mul2(q, both(1.0f / 127.0f));
    return mul2(mul2(t, make_float2(fabsf(t.x), fabsf(t.y))), both(scale));
}
__device__ __forceinline__ float2 values_v(float2 q, float scale)
{
    const float2 t = mul2(q, both(1.0f / 255.0f)), t2 = mul2(t, t);
    return mul2(mul2(t2, t2), both(scale));
}

// Codes round(sqrt(x) * k) of eight values as correctly rounded operations give
// them, at least `least`, with the sign of `sign`'s top bit; one per byte.  The
// approximate root (2^-23) moves root * k by less than 7e-5: only when one of
// the eight is nearer than 1e-4 to a half (or `precise`: the block's moments are
// so small that it takes some of them for zero) are the roots taken again,
// rounded.
__device__ __forceinline__ float sqrt_fast(float x)
{
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __noinline__ float root_times(float x, float k) { return __fmul_rn(__fsqrt_rn(x), k); }
template <typename X, typename LEAST, typename SIGN>
__device__ __forceinline__ uint2 codes8(float k, bool precise, X x, LEAST least, SIGN sign)
{
    float y[8], far = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = fmaxf(__fmul_rn(sqrt_fast(x(j)), k), least(j));
        far = fmaxf(far, fabsf(__fsub_rn(y[j], __fsub_rn(__fadd_rn(y[j], kRounder), kRounder))));
    }
    if (far > 0.4999f || precise) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fmaxf(root_times(x(j), k), least(j));
    }
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        c[j] = __float_as_uint(__fadd_rn(__uint_as_float(__float_as_uint(y[j]) | sign(j)), kRounder));
    auto word = [&](int j) {
        return __byte_perm(__byte_perm(c[j], c[j + 1], 0x0040), __byte_perm(c[j + 2], c[j + 3], 0x0040), 0x5410);
    };
    return make_uint2(word(0), word(4));
}

// Largest value of the warp's lanes; values are magnitudes or NaN (as bits,
// magnitudes order like integers and every NaN is above infinity).
__device__ __forceinline__ float warp_top(uint32_t x) { return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, x)); }
__device__ __forceinline__ float finite_or_nan(float x) { return x <= 3.402823466e38f ? x : __uint_as_float(0x7FC00000u); }

// The steps of two elements, as step1: products in pairs, sums one by one (a
// packed product and sum come out contracted).
__device__ __forceinline__ float2 sum2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }
__device__ __forceinline__ float2 step2(float2 p, float2 g, float2 &m, float2 &v, float2 &s, const Hyper &h,
                                        const Tensor &t)
{
    m = sum2(mul2(m, both(h.beta1)), mul2(g, both(h.one_minus_beta1)));
    v = sum2(mul2(v, both(h.beta2)), mul2(mul2(g, g), both(h.one_minus_beta2)));
    s = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
    const float2 d = sum2(mul2(s, both(h.root)), both(h.eps));
    const float2 u = make_float2(__fdiv_rn(m.x, d.x), __fdiv_rn(m.y, d.y));
    return sum2(mul2(p, both(t.keep)), mul2(u, both(-t.rate)));
}

// One warp per block of 256 elements, of which a lane holds elements 4 lane ..
// and 128 + 4 lane .., so that each load of the warp is of whole neighbouring
// sectors.  A thread block takes one pass, and the blocks of an SM cover one
// another's loads.  (Eight passes a block, with the next two's words copied
// ahead to shared memory: 256 M elements in 200 tensors with bf16 gradients and
// copies 792 us instead of 823, with fp32 ones 856 instead of 833, 300 M in one
// tensor 860 instead of 820, 12 M in 100 tensors 51 instead of 44.)
template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) adamw8_kernel(const __grid_constant__ Launch<CAP> L)
{
    const Tensor &t = find(L, (int)blockIdx.x);
    const Hyper &h = L.h;
    const float gs = h.grad_scale ? *h.grad_scale : 1.0f;
    const bool scaled = h.grad_scale != nullptr, half = t.flags & kBf16Grad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long b0 = (long long)((int)blockIdx.x - t.first) * kPass + warp * kBlock;
    if (b0 >= t.n) return;
    uint8_t *mq = static_cast<uint8_t *>(t.m), *vq = static_cast<uint8_t *>(t.v);
    const bool vec = (t.flags & kVector) && b0 + kBlock <= t.n;
    const float ms = t.m_scale[b0 / kBlock], vs = t.v_scale[b0 / kBlock];
    float p[8], g[8];
    uint32_t a[2], b[2];
    if (vec) {
        uint2 gh[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const long long i = b0 + q * 128 + lane * 4;
            *reinterpret_cast<float4 *>(p + q * 4) = *reinterpret_cast<const float4 *>(t.p + i);
            if (half) gh[q] = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(t.g) + i);
            else *reinterpret_cast<float4 *>(g + q * 4) = *reinterpret_cast<const float4 *>(static_cast<const float *>(t.g) + i);
            a[q] = *reinterpret_cast<const uint32_t *>(mq + i);
            b[q] = *reinterpret_cast<const uint32_t *>(vq + i);
        }
        if (half)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                g[q * 4] = bf16_bits(gh[q].x);
                g[q * 4 + 1] = __uint_as_float(gh[q].x & 0xFFFF0000u);
                g[q * 4 + 2] = bf16_bits(gh[q].y);
                g[q * 4 + 3] = __uint_as_float(gh[q].y & 0xFFFF0000u);
            }
    } else {
        a[0] = a[1] = b[0] = b[1] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const long long e = b0 + (j >> 2) * 128 + lane * 4 + (j & 3);
            const bool in = e < t.n;
            p[j] = in ? t.p[e] : 0.0f;
            g[j] = in ? load_grad(t, e) : 0.0f;
            a[j >> 2] |= (in ? (uint32_t)mq[e] : 0u) << (8 * (j & 3));
            b[j >> 2] |= (in ? (uint32_t)vq[e] : 0u) << (8 * (j & 3));
        }
    }
    float2 mm[4], vv[4], root[4];
    uint32_t mt = 0, vt = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t x = a[j >> 1], y = b[j >> 1];
        const int o = 2 * (j & 1);
        mm[j] = values_m(make_float2(byte_float<true>(x, o), byte_float<true>(x, o + 1)), ms);
        vv[j] = values_v(make_float2(byte_float<false>(y, o), byte_float<false>(y, o + 1)), vs);
        float2 gg = make_float2(g[2 * j], g[2 * j + 1]);
        if (scaled) gg = mul2(gg, both(gs));
        const float2 q = step2(make_float2(p[2 * j], p[2 * j + 1]), gg, mm[j], vv[j], root[j], h, t);
        p[2 * j] = q.x;
        p[2 * j + 1] = q.y;
        mt = max(mt, max(__float_as_uint(mm[j].x) & 0x7FFFFFFFu, __float_as_uint(mm[j].y) & 0x7FFFFFFFu));
        vt = max(vt, max(__float_as_uint(vv[j].x) & 0x7FFFFFFFu, __float_as_uint(vv[j].y) & 0x7FFFFFFFu));
    }
    if (vec) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const long long i = b0 + q * 128 + lane * 4;
            *reinterpret_cast<float4 *>(t.p + i) = *reinterpret_cast<const float4 *>(p + q * 4);
            if (t.copy)
                *reinterpret_cast<uint2 *>(t.copy + i) =
                    make_uint2(pack_bf16(p[q * 4], p[q * 4 + 1]), pack_bf16(p[q * 4 + 2], p[q * 4 + 3]));
        }
    }
    const float mtop = warp_top(mt), vtop = warp_top(vt);
    const float mr = __fsqrt_rn(mtop), vr = __fsqrt_rn(__fsqrt_rn(vtop));
    const float mk = mr > 0.0f ? __fdiv_rn(127.0f, mr) : 0.0f, vk = vr > 0.0f ? __fdiv_rn(255.0f, vr) : 0.0f;
    auto at = [](const float2 (&x)[4], int j) { return j & 1 ? x[j >> 1].y : x[j >> 1].x; };
    const uint2 ma = codes8(mk, mtop < 1e-30f, [&](int j) { return fabsf(at(mm, j)); }, [](int) { return 0.0f; },
                            [&](int j) { return __float_as_uint(at(mm, j)) & 0x80000000u; });
    // a second moment above zero keeps a code above zero
    const uint2 va = codes8(vk, vtop < 1e-26f, [&](int j) { return at(root, j); },
                            [&](int j) { return at(vv, j) > 0.0f ? 1.0f : 0.0f; }, [](int) { return 0u; });
    if (vec) {
        *reinterpret_cast<uint32_t *>(mq + b0 + lane * 4) = ma.x;
        *reinterpret_cast<uint32_t *>(mq + b0 + 128 + lane * 4) = ma.y;
        *reinterpret_cast<uint32_t *>(vq + b0 + lane * 4) = va.x;
        *reinterpret_cast<uint32_t *>(vq + b0 + 128 + lane * 4) = va.y;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const long long e = b0 + (j >> 2) * 128 + lane * 4 + (j & 3);
            if (e < t.n) {
                t.p[e] = p[j];
                if (t.copy) t.copy[e] = __float2bfloat16_rn(p[j]);
                mq[e] = (uint8_t)((j < 4 ? ma.x : ma.y) >> (8 * (j & 3)) & 0xFFu);
                vq[e] = (uint8_t)((j < 4 ? va.x : va.y) >> (8 * (j & 3)) & 0xFFu);
            }
        }
    }
    if (lane == 0) {
        t.m_scale[b0 / kBlock] = finite_or_nan(mtop);
        t.v_scale[b0 / kBlock] = finite_or_nan(vtop);
    }
}

// Four codes per thread and step: whole sectors of both codes and values.
constexpr int kValueSteps = 4;
template <bool SECOND>
__global__ void __launch_bounds__(kThreads) moment_values_kernel(const uint8_t *codes, const float *scales, long long n,
                                                                 float *out, int vec)
{
#pragma unroll
    for (int k = 0; k < kValueSteps; ++k) {
        const long long i = (((long long)blockIdx.x * kValueSteps + k) * kThreads + threadIdx.x) * 4;
        if (i >= n) return;
        const float s = scales[i / kBlock];
        uint32_t w = 0;
        const bool whole = vec && i + 4 <= n;
        if (whole) w = *reinterpret_cast<const uint32_t *>(codes + i);
        else
            for (int j = 0; j < 4 && i + j < n; ++j) w |= (uint32_t)codes[i + j] << (8 * j);
        const float2 a = make_float2(byte_float<!SECOND>(w, 0), byte_float<!SECOND>(w, 1));
        const float2 b = make_float2(byte_float<!SECOND>(w, 2), byte_float<!SECOND>(w, 3));
        const float2 x = SECOND ? values_v(a, s) : values_m(a, s), y = SECOND ? values_v(b, s) : values_m(b, s);
        if (whole) {
            *reinterpret_cast<float4 *>(out + i) = make_float4(x.x, x.y, y.x, y.y);
        } else {
            const float r[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < n) out[i + j] = r[j];
        }
    }
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
        if ((a.n + kPass - 1) / kPass > 0x3FFFFFFF) return AMSIM_EINVAL;
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
            add = (tensors[i].n + kPass - 1) / kPass;
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
    constexpr int kPerBlock = kThreads * 4 * kValueSteps;
    const long long blocks = (n + kPerBlock - 1) / kPerBlock;
    if (blocks > 0x7FFFFFFFLL) return AMSIM_EINVAL;
    const uint8_t *q = static_cast<const uint8_t *>(codes);
    const int vec = aligned(codes, 4) && aligned(out, 16);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (second) moment_values_kernel<true><<<(unsigned)blocks, kThreads, 0, st>>>(q, scales, n, out, vec);
    else moment_values_kernel<false><<<(unsigned)blocks, kThreads, 0, st>>>(q, scales, n, out, vec);
    const int rc = amsim::cuda_status(cudaGetLastError());
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}
