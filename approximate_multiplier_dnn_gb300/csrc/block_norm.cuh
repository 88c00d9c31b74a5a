// The block norm's kernels: RMS norms before and after a block, fused with the
// block's gate and the residual scale.
//
// HBM-bound: the forward pass reads x and y and writes r and n, the backward
// pass reads y, r, dr, dn and writes dx, dy, each once.  The threads of a row
// hold 16 channels each (fewer for narrow rows), and both norms of a row and
// everything between them happen in one pass over memory.  With 44 bytes per
// nanosecond and SM the bound leaves about 20 issue slots per channel, so the
// arithmetic goes through the packed fp32 instructions, two channels each, and
// what a row costs besides its channels (sums across warps, addresses, roots)
// is spread over many channels per thread.
//
// Measured, of 6768 GB/s for a plain copy: forward 5.3 TB/s at 16384 x 4096
// bf16 (102 us) and 5.5 at 16384 x 2048 with an fp32 stream, backward 5.3
// (152 us) and 5.6 (108 us).  Backward at 8192 x 8192 bf16 (173 to 178 us, 4.6 TB/s)
// has room in shared memory for two rows, and at 16384 columns for none.
#pragma once

#include <atomic>

#include <cuda_bf16.h>

#include "bounded_wait.cuh"
#include "chained.cuh"
#include "pairs.cuh"
#include "row_pieces.cuh"

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
    long long block_rows;                  // ring forward: rows of a thread block
    int splits;                            // backward: shares per row of the gate
    int cols;
    int tpr, rpb;                          // threads per row, rows per thread block
    int slots, slot_bytes;                 // ring kernels: rows ahead in shared memory, bytes of one
    float alpha, eps;
};

// Channels a thread takes at a step: 16 bytes of fp32, 8 of bf16, so that a
// warp's loads and stores are whole neighbouring sectors whichever the type.
constexpr int kE = 4, kP = 2;
struct Four {
    float2 p[kP];
};

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16 *p, float v) { *p = __float2bfloat16_rn(v); }

// What a thread keeps of a row between its load and its use: the raw words.
template <typename T>
struct Raw {
    uint32_t w[sizeof(T)];                 // kE elements
};

// Channel of element e (0..3) of step k: vector steps take 4 neighbours per
// thread, scalar ones stride by the threads of the row.
template <bool VEC>
__device__ __forceinline__ int channel(int k, int e, int t, int tpr)
{
    return VEC ? (k * tpr + t) * kE + e : (k * kE + e) * tpr + t;
}

template <bool VEC, typename T>
__device__ __forceinline__ void load_raw(Raw<T> &d, const T *row, int k, int t, int tpr, int cols)
{
    if constexpr (VEC) {
        const int c = channel<true>(k, 0, t, tpr);
        if constexpr (sizeof(T) == 4) {
            uint4 q = make_uint4(0, 0, 0, 0);
            if (c < cols) q = *reinterpret_cast<const uint4 *>(row + c);
            d.w[0] = q.x; d.w[1] = q.y; d.w[2] = q.z; d.w[3] = q.w;
        } else {
            uint2 q = make_uint2(0, 0);
            if (c < cols) q = *reinterpret_cast<const uint2 *>(row + c);
            d.w[0] = q.x; d.w[1] = q.y;
        }
    } else {
        uint32_t w[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int c = channel<false>(k, e, t, tpr);
            if constexpr (sizeof(T) == 4) w[e] = c < cols ? reinterpret_cast<const uint32_t *>(row)[c] : 0u;
            else w[e] = c < cols ? reinterpret_cast<const uint16_t *>(row)[c] : 0u;
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < kE; ++e) d.w[e] = w[e];
        } else {
            d.w[0] = w[0] | w[1] << 16;
            d.w[1] = w[2] | w[3] << 16;
        }
    }
}

template <typename T>
__device__ __forceinline__ Four widen(const Raw<T> &d)
{
    Four r;
    if constexpr (sizeof(T) == 4) {
        r.p[0] = make_float2(__uint_as_float(d.w[0]), __uint_as_float(d.w[1]));
        r.p[1] = make_float2(__uint_as_float(d.w[2]), __uint_as_float(d.w[3]));
    } else {
#pragma unroll
        for (int e = 0; e < kP; ++e)
            r.p[e] = make_float2(__uint_as_float(d.w[e] << 16), __uint_as_float(d.w[e] & 0xFFFF0000u));
    }
    return r;
}

template <bool VEC, typename T>
__device__ __forceinline__ void store4(T *row, int k, int t, int tpr, int cols, const Four &r)
{
    if constexpr (VEC) {
        const int c = channel<true>(k, 0, t, tpr);
        if (c >= cols) return;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(row + c) = make_float4(r.p[0].x, r.p[0].y, r.p[1].x, r.p[1].y);
        } else {
            const __nv_bfloat162 a = __float22bfloat162_rn(r.p[0]), b = __float22bfloat162_rn(r.p[1]);
            *reinterpret_cast<uint2 *>(row + c) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        }
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int c = channel<false>(k, e, t, tpr);
            if (c < cols) put(row + c, e & 1 ? r.p[e >> 1].y : r.p[e >> 1].x);
        }
    }
}

// Four fp32 weights (ones where there are none).
template <bool VEC>
__device__ __forceinline__ Four weights(const float *w, int k, int t, int tpr, int cols)
{
    if (!w) return Four{{both(1.0f), both(1.0f)}};
    Raw<float> d;
    load_raw<VEC, float>(d, w, k, t, tpr, cols);
    return widen(d);
}

// alpha gate w_post
template <bool VEC>
__device__ __forceinline__ Four weights_u(const Params &p, const float *gate, int k, int t, int cols)
{
    Four w = weights<VEC>(p.w_post, k, t, p.tpr, cols);
    const Four g = weights<VEC>(gate, k, t, p.tpr, cols);
#pragma unroll
    for (int e = 0; e < kP; ++e) w.p[e] = mul2(w.p[e], mul2(both(p.alpha), g.p[e]));
    return w;
}

// Sums of S values over the threads of a row (its warps are neighbours in the
// block), all behind one barrier of at least those threads, `sync`.  `which` alternates between two
// buffers, so that a barrier per call is enough.
template <int S>
struct Sums {
    float v[S];
};
template <int S, typename SYNC>
__device__ __forceinline__ void row_sums(Sums<S> &x, int warps, float (*red)[S][32], int &which, SYNC sync)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < S; ++i) x.v[i] += __shfl_xor_sync(0xFFFFFFFFu, x.v[i], d);
    if (warps == 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float (*buf)[32] = red[which];
    which ^= 1;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < S; ++i) buf[i][warp] = x.v[i];
    sync();
    const int first = warp / warps * warps;
    if (warps <= 8) {
        const int j = lane & 7;
#pragma unroll
        for (int i = 0; i < S; ++i) x.v[i] = j < warps ? buf[i][first + j] : 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < S; ++i) x.v[i] = lane < warps ? buf[i][first + lane] : 0.0f;
#pragma unroll
        for (int d = 16; d > 4; d >>= 1)
#pragma unroll
            for (int i = 0; i < S; ++i) x.v[i] += __shfl_xor_sync(0xFFFFFFFFu, x.v[i], d);
    }
#pragma unroll
    for (int d = 4; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < S; ++i) x.v[i] += __shfl_xor_sync(0xFFFFFFFFu, x.v[i], d);
}

// The parts of a call.  Kernels built for calls with every part (kAll), or with
// every part but dr (kNoDr: the last norm of a model, whose r is not used), test
// none of them.  (Backward without dr: 5395 x 3047 bf16 78 us with zeros in its
// place, 96 with the tests, 62 so; 16384 x 4096 190, 168, 115.)
enum Has { kSome, kAll, kNoDr };
template <int HAS>
struct Parts {
    const Params &p;
    __device__ __forceinline__ bool y() const { return HAS || p.y; }
    __device__ __forceinline__ bool post() const { return HAS || p.w_post; }
    __device__ __forceinline__ bool r() const { return HAS || p.r; }
    __device__ __forceinline__ bool n() const { return HAS || p.n; }
    __device__ __forceinline__ bool dr() const { return HAS == kAll || (HAS == kSome && p.dr); }
    __device__ __forceinline__ bool dn() const { return HAS || p.dn; }
    __device__ __forceinline__ bool dx() const { return HAS || p.dx; }
    __device__ __forceinline__ bool dy() const { return HAS || p.dy; }
};

// ------------------------------------------------------------------ one row
// Forward.  `xr`, `yr`: the thread's words of the row; `wu(k)`: alpha gate
// w_post, `wq(k)`: w_pre; `met(barrier)` runs after the first sum (or where it
// would be), `barrier` telling whether every thread was waited for there.
template <int NV, bool VEC, int HAS, typename X, typename Y, typename N, typename WU, typename WQ, typename F>
__device__ __forceinline__ void fwd_row(const Params &p, const Raw<X> (&xr)[NV], const Raw<Y> (&yr)[NV], X *ro, N *no,
                                        long long row, bool on, int t, int cols, int warps, float (*red)[1][32],
                                        int &which, WU wu, WQ wq, F met)
{
    const Parts<HAS> has{p};
    const float inv = 1.0f / (float)p.cols;
    float post = 1.0f;
    if (has.post()) {
        float2 s2 = both(0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const Four a = widen(yr[k]);
#pragma unroll
            for (int e = 0; e < kP; ++e) s2 = fma2(a.p[e], a.p[e], s2);
        }
        Sums<1> s{{s2.x + s2.y}};
        row_sums(s, warps, red, which, [] { __syncthreads(); });
        post = rsqrtf(fmaf(s.v[0], inv, p.eps));
        if (on && t == 0 && (HAS || p.rstd_post)) p.rstd_post[row] = post;
    }
    met(has.post() && warps > 1);
    Four r[NV];
    float2 s2 = both(0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        r[k] = widen(xr[k]);
        if (has.y()) {
            const Four a = widen(yr[k]), w = wu(k);
#pragma unroll
            for (int e = 0; e < kP; ++e) r[k].p[e] = fma2(mul2(both(post), a.p[e]), w.p[e], r[k].p[e]);
        }
#pragma unroll
        for (int e = 0; e < kP; ++e) s2 = fma2(r[k].p[e], r[k].p[e], s2);
        if (has.r()) store4<VEC, X>(ro, k, t, p.tpr, cols, r[k]);
    }
    if (!has.n()) return;
    Sums<1> s{{s2.x + s2.y}};
    row_sums(s, warps, red, which, [] { __syncthreads(); });
    const float pre = rsqrtf(fmaf(s.v[0], inv, p.eps));
    if (on && t == 0 && (HAS || p.rstd_pre)) p.rstd_pre[row] = pre;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const Four w = wq(k);
#pragma unroll
        for (int e = 0; e < kP; ++e) r[k].p[e] = mul2(mul2(r[k].p[e], both(pre)), w.p[e]);
        store4<VEC, N>(no, k, t, p.tpr, cols, r[k]);
    }
}

// A thread's words of one step of a row in the backward pass.
template <typename X, typename Y, typename N>
struct Step {
    Raw<X> dr, r;
    Raw<Y> y;
    Raw<N> dn;
};

// Backward.  The second norm's mean is wanted of s = wu dx, which itself
// contains the first norm's mean m = mean(t rh); as
//   dx = q - pre m rh,  q = dr + pre t,
//   mean(s yh) = mean(wu yh q) - pre m mean(wu yh rh),
// all three means come from one pass over the row and one barrier.  Between the
// passes a thread keeps q, and loads r and y again (from shared memory or the
// L1 cache; with KEEP, narrow or unaligned rows, it keeps them too): the rest of
// its registers are the column sums', two per channel.  Keeping bf16 rows in
// the streaming kernel freed their slot a row earlier and was 8 % slower.
template <int NV, bool VEC, int HAS, bool KEEP, typename X, typename Y, typename N, typename LOAD, typename WQ,
          typename WU, typename SYNC, typename F>
__device__ __forceinline__ void bwd_row(const Params &p, float pre, float post, X *dxo, Y *dyo, int t, int cols,
                                        int warps, float (*red)[3][32], int &which, float2 (&a)[NV * kP],
                                        float2 (&b)[NV * kP], LOAD load, WQ wq, WU wu, SYNC sync, F met)
{
    const Parts<HAS> has{p};
    const float inv = 1.0f / (float)p.cols;
    Four q[NV];
    Step<X, Y, N> in[KEEP ? NV : 1];
    float2 s2[3] = {both(0.0f), both(0.0f), both(0.0f)};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        Step<X, Y, N> &w = in[KEEP ? k : 0];
        w = load(k, true);
        if (has.dr()) q[k] = widen(w.dr);
        else q[k] = Four{{both(0.0f), both(0.0f)}};
        Four rh;
        if (has.dn()) {
            rh = widen(w.r);
            const Four n = widen(w.dn), v = wq(k);
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                rh.p[e] = mul2(rh.p[e], both(pre));
                const float2 t = mul2(n.p[e], v.p[e]);
                s2[0] = fma2(t, rh.p[e], s2[0]);
                b[k * kP + e] = fma2(n.p[e], rh.p[e], b[k * kP + e]);
                q[k].p[e] = fma2(both(pre), t, q[k].p[e]);
            }
        }
        if (has.y()) {
            const Four y = widen(w.y), v = wu(k);
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                const float2 u = mul2(v.p[e], mul2(y.p[e], both(post)));
                s2[1] = fma2(u, q[k].p[e], s2[1]);
                if (has.dn()) s2[2] = fma2(u, rh.p[e], s2[2]);
            }
        }
    }
    Sums<3> sum{{s2[0].x + s2[0].y, s2[1].x + s2[1].y, s2[2].x + s2[2].y}};
    const bool means = has.dn() || (has.y() && has.post());
    if (means) row_sums(sum, warps, red, which, sync);
    met(means && warps > 1);
    const float m = pre * (sum.v[0] * inv), mr = -m * pre;
    const float s = !has.post() ? 0.0f : (has.dn() ? fmaf(-m, sum.v[2], sum.v[1]) : sum.v[1]) * inv;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        Step<X, Y, N> &w = in[KEEP ? k : 0];
        if (!KEEP) w = load(k, false);
        if (has.dn()) {
            const Four r = widen(w.r);
#pragma unroll
            for (int e = 0; e < kP; ++e) q[k].p[e] = fma2(both(mr), r.p[e], q[k].p[e]);
        }
        if (has.dx()) store4<VEC, X>(dxo, k, t, p.tpr, cols, q[k]);
        if (!has.y()) continue;
        const Four y = widen(w.y), v = wu(k);
        Four o;
#pragma unroll
        for (int e = 0; e < kP; ++e) {
            const float2 yh = mul2(y.p[e], both(post));
            a[k * kP + e] = fma2(q[k].p[e], yh, a[k * kP + e]);
            o.p[e] = mul2(both(post), fma2(yh, both(-s), mul2(q[k].p[e], v.p[e])));
        }
        if (has.dy()) store4<VEC, Y>(dyo, k, t, p.tpr, cols, o);
    }
}

// A channel's sum over a share's rows leaves: to the share's slot when several
// make up a row of the gate, else to dgate and the block's slot of dw_post.
__device__ __forceinline__ void leave_a(const Params &p, float v, int c, long long item, long long gi,
                                        const float *gate, bool fresh)
{
    if (c >= p.cols) return;
    if (p.splits > 1) {
        p.part_gate[item * p.cols + c] = v;
        return;
    }
    if (p.dgate) p.dgate[gi * p.cols + c] = p.alpha * (p.w_post ? p.w_post[c] : 1.0f) * v;
    if (p.dw_post) {
        float *slot = p.part_post + (long long)blockIdx.x * p.cols + c;
        *slot = fmaf(p.alpha * (gate ? gate[c] : 1.0f), v, fresh ? 0.0f : *slot);
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

__device__ __forceinline__ float element(const float2 &v, int e) { return e & 1 ? v.y : v.x; }

// ------------------------------------------------------------------ direct loads
template <int NV, int THREADS, bool VEC, typename X, typename Y, typename N>
__global__ void __launch_bounds__(THREADS) fwd_kernel(const Params p)
{
    __shared__ float red[2][1][32];
    int which = 0;
    const int t = threadIdx.x % p.tpr, warps = p.tpr >> 5;
    const long long row = (long long)blockIdx.x * p.rpb + threadIdx.x / p.tpr;
    const bool on = row < p.rows;
    const int cols = on ? p.cols : 0;
    Raw<X> xr[NV];
    Raw<Y> yr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) load_raw<VEC, X>(xr[k], static_cast<const X *>(p.x) + row * p.ldx, k, t, p.tpr, cols);
    if (p.y)
#pragma unroll
        for (int k = 0; k < NV; ++k)
            load_raw<VEC, Y>(yr[k], static_cast<const Y *>(p.y) + row * p.ldy, k, t, p.tpr, cols);
    const float *gate = p.gate && on ? p.gate + row / p.gate_rows * p.cols : nullptr;
    fwd_row<NV, VEC, kSome, X, Y, N>(
        p, xr, yr, static_cast<X *>(p.r) + row * p.ldr, static_cast<N *>(p.n) + row * p.ldn, row, on, t, cols, warps,
        red, which, [&](int k) { return weights_u<VEC>(p, gate, k, t, cols); },
        [&](int k) { return weights<VEC>(p.w_pre, k, t, p.tpr, cols); }, [](bool) {});
}

// A block takes shares (items) of item_rows rows; the rows of a share have the
// same gate.  Column sums stay in registers over a share's rows:
//   a = sum dx * yh  (per gate row: dgate = alpha w_post a, dw_post = alpha sum gate a)
//   b = sum dn * rh  (dw_pre).
// `a` leaves at the end of each share, `b` at the end of the block.
template <int NV, int THREADS, bool VEC, typename X, typename Y, typename N>
__global__ void __launch_bounds__(THREADS) bwd_kernel(const Params p)
{
    __shared__ float red[2][3][32];
    __shared__ float buf[THREADS];
    int which = 0;
    const int t = threadIdx.x % p.tpr, group = threadIdx.x / p.tpr, warps = p.tpr >> 5;
    const bool want_y = p.y != nullptr, want_n = p.dn != nullptr;
    const bool sums_a = want_y && (p.dgate || p.dw_post), sums_b = want_n && p.dw_pre;
    float2 b[NV * kP];
#pragma unroll
    for (int i = 0; i < NV * kP; ++i) b[i] = both(0.0f);
    bool fresh = true;                       // no share has left its sums in part_post yet
    for (long long item = blockIdx.x; item < p.items; item += gridDim.x) {
        const long long gi = item / p.splits;
        const long long g0 = gi * p.gate_rows, g1 = min(g0 + p.gate_rows, p.rows);
        const long long r0 = g0 + (item - gi * p.splits) * p.item_rows, r1 = min(r0 + p.item_rows, g1);
        const float *gate = p.gate ? p.gate + gi * p.cols : nullptr;
        float2 a[NV * kP];
#pragma unroll
        for (int i = 0; i < NV * kP; ++i) a[i] = both(0.0f);
        for (long long rb = r0; rb < r1; rb += p.rpb) {
            const long long row = rb + group;
            const bool on = row < r1;
            const int cols = on ? p.cols : 0;
            const float pre = want_n && on ? p.rstd_pre[row] : 0.0f;
            const float post = !want_y || !p.w_post ? 1.0f : on ? p.rstd_post[row] : 0.0f;
            bwd_row<NV, VEC, kSome, NV <= 2 || !VEC, X, Y, N>(
                p, pre, post, static_cast<X *>(p.dx) + row * p.lddx, static_cast<Y *>(p.dy) + row * p.lddy, t, cols,
                warps, red, which, a, b,
                [&](int k, bool first) {
                    Step<X, Y, N> in;
                    if (p.dr && first) load_raw<VEC, X>(in.dr, static_cast<const X *>(p.dr) + row * p.lddr, k, t, p.tpr, cols);
                    if (want_n) {
                        load_raw<VEC, X>(in.r, static_cast<const X *>(p.rin) + row * p.ldr, k, t, p.tpr, cols);
                        if (first)
                            load_raw<VEC, N>(in.dn, static_cast<const N *>(p.dn) + row * p.lddn, k, t, p.tpr, cols);
                    }
                    if (want_y) load_raw<VEC, Y>(in.y, static_cast<const Y *>(p.y) + row * p.ldy, k, t, p.tpr, cols);
                    return in;
                },
                [&](int k) { return weights<VEC>(p.w_pre, k, t, p.tpr, cols); },
                [&](int k) { return weights_u<VEC>(p, gate, k, t, cols); }, [] { __syncthreads(); }, [](bool) {});
        }
        if (!sums_a) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float v = group_sum(element(a[k * kP + (e >> 1)], e), p.tpr, p.rpb, buf);
                if (group == 0) leave_a(p, v, channel<VEC>(k, e, t, p.tpr), item, gi, gate, fresh);
            }
        fresh = false;
    }
    if (!sums_b) return;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const float v = group_sum(element(b[k * kP + (e >> 1)], e), p.tpr, p.rpb, buf);
            const int c = channel<VEC>(k, e, t, p.tpr);
            if (group == 0 && c < p.cols) p.part_pre[(long long)blockIdx.x * p.cols + c] = v;
        }
}

// ------------------------------------------------------------------ rows by bulk copies
// The kernels above keep one row's bytes in flight per block, and none while
// they reduce it: 40 % of the copy bandwidth at 16384 x 4096.  Where there are
// many rows, a block streams them through a ring in shared memory instead: one
// thread issues whole-row bulk copies, and refills a slot once every thread is
// past it.  Channels are dealt to threads, and sums taken, as above, so a row's
// results do not depend on how many rows come with it.
//
// Rows that do not start and end on 16 bytes (WHOLE false) come as the aligned
// pieces of 16 that hold them (row_pieces.cuh), and start inside their slot.
// Backward, 5395 x 3047 bf16: 341 us by direct loads, 73 so; 16384 x 1013
// fp32/bf16: 166, 68.  Whole rows have kernels of their own, as the four rows'
// ends cost 3 to 7 % of 16384 x 4096 and 8192 x 8192 bf16.

// Waits, up to the limit once more, for the copies into a ring whose next slot is `at`.
static __device__ __noinline__ void settle_copies(uint64_t *full, int parts, int slots, int at, uint32_t phase)
{
    const unsigned long long t0 = tc::now_ns();
    for (int i = 0; i < parts * slots; ++i) {
        const int slot = i % slots;
        while (!tc::bar_try(full + i, slot < at ? phase ^ 1 : phase) && tc::now_ns() - t0 <= tc::kWaitLimitNs) {}
    }
}

// PARTS: a slot's parts arrive, and are refilled, each by itself.
template <int PARTS>
struct Ring {
    uint8_t *slot0;
    uint64_t *full;                        // [part][slot]
    int slots, bytes;
    int at = 0;
    uint32_t phase = 0;
    bool aborted = false;

    // A thread whose wait gives up waits for nothing from then on, and issues
    // nothing, so that no copy is on its way when the block ends.
    __device__ __forceinline__ uint8_t *wait()
    {
        if (!aborted) {
#pragma unroll
            for (int i = 0; i < PARTS; ++i) tc::bar_wait(full + i * slots + at, phase, aborted);
            if (aborted) settle_copies(full, PARTS, slots, at, phase);
        }
        return slot0 + at * bytes;
    }
    // On to the next slot; the number of the one left.
    __device__ __forceinline__ int next()
    {
        const int s = at;
        if (++at == slots) { at = 0; phase ^= 1; }
        return s;
    }
};

constexpr int kRingNV = 4;                 // steps per thread of the ring kernels
constexpr int kRingBarBytes = 128;         // of a ring: 2 parts of 8 slots
constexpr int kRingAlign = 128, kRingSlack = 30;   // of a slot; of a row's ends that are off 16 bytes
// Threads per SM that the kernels' registers allow (up to 128 each): forward as
// blocks of up to 256 or 512, backward as the teams of one block.
constexpr int kRingThreads = 512, kTeamThreads = 512;
__host__ __device__ inline int ring_bytes(int cols, int size, int slack)
{
    return (cols * size + slack + kRingAlign - 1) / kRingAlign * kRingAlign;
}
// Weights that wait in shared memory: a row of fp32.
__host__ __device__ inline int kept_floats(int cols) { return (cols + 3) / 4 * 4; }

template <int PARTS>
__device__ __forceinline__ Ring<PARTS> make_ring(const Params &p, uint8_t *smem, int teams, int team, int t)
{
    Ring<PARTS> r;
    r.full = reinterpret_cast<uint64_t *>(smem + team * kRingBarBytes);
    r.slot0 = smem + teams * kRingBarBytes + team * p.slots * p.slot_bytes;
    r.slots = p.slots;
    r.bytes = p.slot_bytes;
    if (t == 0) {
        for (int i = 0; i < p.slots * PARTS; ++i) tc::bar_init(r.full + i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    return r;
}

template <int SIZE> struct Bits;
template <> struct Bits<2> { using type = uint16_t; };
template <> struct Bits<4> { using type = uint32_t; };

// A row's way to a slot: the row itself, or its pieces, after the elements that
// they leave out have been copied.  The thread that issues the copy calls it
// before it arrives on the slot's barrier.
template <bool WHOLE, typename T>
__device__ __forceinline__ Pieces row_to(uint8_t *slot, const void *base, long long ld, long long row, long long rows, int bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(static_cast<const T *>(base) + row * ld);
    if constexpr (WHOLE) {
        return Pieces{a, 0, bytes};
    } else {
        using W = typename Bits<sizeof(T)>::type;
        const bool first = row == 0, last = row == rows - 1;
        if (first || last) {
            copy_ends<W>(slot, a, bytes, first, last);
            tc::fence_staged();
        }
        return row_pieces(a, bytes, first, last);
    }
}

__device__ __forceinline__ void copy_pieces(uint8_t *slot, const Pieces &r, uint64_t *bar)
{
    tc::copy_bytes(slot + r.at, reinterpret_cast<const void *>(r.from), r.bytes, bar);
}

// Where the row starts in a slot that was filled so.
template <bool WHOLE, typename T>
__device__ __forceinline__ const T *in_slot(const uint8_t *slot, const void *base, long long ld, long long row)
{
    if constexpr (WHOLE) return reinterpret_cast<const T *>(slot);
    else return reinterpret_cast<const T *>(slot + (reinterpret_cast<uintptr_t>(static_cast<const T *>(base) + row * ld) & 15));
}

// Four weights that wait in shared memory.
template <bool VEC>
__device__ __forceinline__ Four kept(const float *w, int k, int t, int tpr, int cols)
{
    Raw<float> d;
    load_raw<VEC, float>(d, w, k, t, tpr, cols);
    return widen(d);
}

template <int THREADS, bool VEC, bool WHOLE, int HAS, typename X, typename Y, typename N>
__global__ void __launch_bounds__(THREADS, kRingThreads / THREADS) fwd_ring_kernel(const Params p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][1][32];
    constexpr int NV = kRingNV;
    const Parts<HAS> has{p};
    int which = 0;
    const int t = threadIdx.x, warps = p.tpr >> 5, cols = p.cols;
    const int bytes_x = cols * (int)sizeof(X), bytes_y = cols * (int)sizeof(Y);
    const int yoff = ring_bytes(cols, sizeof(X), WHOLE ? 0 : kRingSlack);
    const long long r0 = blockIdx.x * p.block_rows, r1 = min(r0 + p.block_rows, p.rows);
    Ring<1> ring = make_ring<1>(p, smem, 1, 0, t);
    auto issue = [&](long long row, int slot) {
        uint8_t *s = ring.slot0 + slot * ring.bytes;
        uint64_t *full = ring.full + slot;
        const Pieces x = row_to<WHOLE, X>(s, p.x, p.ldx, row, p.rows, bytes_x);
        Pieces y{};
        if (has.y()) y = row_to<WHOLE, Y>(s + yoff, p.y, p.ldy, row, p.rows, bytes_y);
        tc::bar_expect(full, x.bytes + y.bytes);
        copy_pieces(s, x, full);
        if (has.y()) copy_pieces(s + yoff, y, full);
    };
    if (t == 0)
        for (int i = 0; i < p.slots && r0 + i < r1; ++i) issue(r0 + i, i);
    Four wq[NV], wu[NV];                   // w_pre, and alpha gate w_post of the rows' gate
    if (has.n())
#pragma unroll
        for (int k = 0; k < NV; ++k) wq[k] = weights<VEC>(p.w_pre, k, t, p.tpr, cols);
    X *ro = static_cast<X *>(p.r) + r0 * p.ldr;
    N *no = static_cast<N *>(p.n) + r0 * p.ldn;
    long long gate_end = r0;               // first row with another gate
    for (long long row = r0; row < r1; ++row, ro += p.ldr, no += p.ldn) {
        if (has.y() && row == gate_end) {
            const long long g = row / p.gate_rows;
            const float *gate = p.gate ? p.gate + g * cols : nullptr;
            gate_end = (g + 1) * p.gate_rows;
#pragma unroll
            for (int k = 0; k < NV; ++k) wu[k] = weights_u<VEC>(p, gate, k, t, cols);
        }
        const uint8_t *slot = ring.wait();
        Raw<X> xr[NV];
        Raw<Y> yr[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) load_raw<VEC, X>(xr[k], in_slot<WHOLE, X>(slot, p.x, p.ldx, row), k, t, p.tpr, cols);
        if (has.y())
#pragma unroll
            for (int k = 0; k < NV; ++k)
                load_raw<VEC, Y>(yr[k], in_slot<WHOLE, Y>(slot + yoff, p.y, p.ldy, row), k, t, p.tpr, cols);
        fwd_row<NV, VEC, HAS, X, Y, N>(
            p, xr, yr, ro, no, row, true, t, cols, warps, red, which,
            [&](int k) { return wu[k]; }, [&](int k) { return wq[k]; },
            [&](bool barrier) {
                if (!barrier) __syncthreads();             // the row is in registers
                const int freed = ring.next();
                if (t == 0 && row + p.slots < r1 && !ring.aborted) issue(row + p.slots, freed);
            });
    }
}

// As bwd_kernel, with the SM's threads as teams of the threads of a row, each
// with a ring of its own.  They share the weights, which wait in shared memory
// (w_pre, then alpha gate w_post of the share's gate): a block per row would
// hold a copy each, and leave room for one row ahead where teams have two.
template <bool VEC, bool WHOLE, int HAS, typename X, typename Y, typename N>
__global__ void __launch_bounds__(kTeamThreads, 1) bwd_ring_kernel(const Params p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][3][32];
    constexpr int NV = kRingNV;
    const Parts<HAS> has{p};
    int which = 0;
    const int teams = p.rpb, team = threadIdx.x / p.tpr, t = threadIdx.x - team * p.tpr;
    const int warps = p.tpr >> 5, cols = p.cols;
    const bool sums_a = has.y() && (p.dgate || p.dw_post), sums_b = has.dn() && p.dw_pre;
    const int bytes_x = cols * (int)sizeof(X), bytes_y = cols * (int)sizeof(Y), bytes_n = cols * (int)sizeof(N);
    const int rxb = ring_bytes(cols, sizeof(X), WHOLE ? 0 : kRingSlack), rnb = ring_bytes(cols, sizeof(N), WHOLE ? 0 : kRingSlack);
    const int off_n = has.dr() ? rxb : 0, off_r = off_n + (has.dn() ? rnb : 0), off_y = off_r + (has.dn() ? rxb : 0);
    float *wq = reinterpret_cast<float *>(smem + teams * (kRingBarBytes + p.slots * p.slot_bytes));
    const int row_floats = VEC ? cols : kept_floats(cols);
    float *wu = wq + row_floats;
    float4 *buf = reinterpret_cast<float4 *>(wu + row_floats);     // one per thread, with several teams
    Ring<2> ring = make_ring<2>(p, smem, teams, team, t);
    auto sync = [&] {
        if (warps == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(p.tpr) : "memory");
    };
    // a team's rows in order: every teams-th of shares blockIdx.x, + gridDim.x, ...
    struct Place {
        long long item, row, end;
    };
    auto settle = [&](Place &q) {            // to the share's first row of this team, or on to the next share's
        for (; q.item < p.items; q.item += gridDim.x) {
            const long long gi = q.item / p.splits, g0 = gi * p.gate_rows, r0 = g0 + (q.item - gi * p.splits) * p.item_rows;
            q.row = r0 + team;
            q.end = min(min(r0 + p.item_rows, g0 + p.gate_rows), p.rows);
            if (q.row < q.end) return;
        }
    };
    // A slot's first part, dr and dn, is read by a row's first pass alone, and
    // refilled half a row before the second part, r and y, is free.  (8192 x
    // 8192 bf16, room for two rows: 203 us with whole slots, 173 so; 16384 x
    // 4096: 159, 152; 8192 x 4096 fp32, room for three: 146, 152, as the one
    // thread issues twice a row.  A second warp's thread for the second part
    // made the first 183.)
    auto issue_first = [&](long long row, int slot) {
        uint8_t *s = ring.slot0 + slot * ring.bytes;
        uint64_t *full = ring.full + slot;
        Pieces dr{}, dn{};
        if (has.dr()) dr = row_to<WHOLE, X>(s, p.dr, p.lddr, row, p.rows, bytes_x);
        if (has.dn()) dn = row_to<WHOLE, N>(s + off_n, p.dn, p.lddn, row, p.rows, bytes_n);
        tc::bar_expect(full, dr.bytes + dn.bytes);
        if (has.dr()) copy_pieces(s, dr, full);
        if (has.dn()) copy_pieces(s + off_n, dn, full);
    };
    auto issue_second = [&](long long row, int slot) {
        uint8_t *s = ring.slot0 + slot * ring.bytes;
        uint64_t *full = ring.full + ring.slots + slot;
        Pieces r{}, y{};
        if (has.dn()) r = row_to<WHOLE, X>(s + off_r, p.rin, p.ldr, row, p.rows, bytes_x);
        if (has.y()) y = row_to<WHOLE, Y>(s + off_y, p.y, p.ldy, row, p.rows, bytes_y);
        tc::bar_expect(full, r.bytes + y.bytes);
        if (has.dn()) copy_pieces(s + off_r, r, full);
        if (has.y()) copy_pieces(s + off_y, y, full);
    };
    auto advance = [&](Place &q) {
        if ((q.row += teams) < q.end) return;
        q.item += gridDim.x;
        settle(q);
    };
    Place ahead{(long long)blockIdx.x, 0, 0};
    settle(ahead);
    if (t == 0)
        for (int i = 0; i < p.slots && ahead.item < p.items; ++i) {
            issue_first(ahead.row, i);
            issue_second(ahead.row, i);
            advance(ahead);
        }
    if (has.dn())
        for (int c = threadIdx.x; c < cols; c += blockDim.x) wq[c] = p.w_pre ? p.w_pre[c] : 1.0f;
    // the teams' sums of four channels, in team order, in team 0's hands
    auto joined = [&](float2 x, float2 y) {
        float4 v = make_float4(x.x, x.y, y.x, y.y);
        if (teams == 1) return v;
        __syncthreads();
        buf[threadIdx.x] = v;
        __syncthreads();
        if (team == 0)
            for (int g = 1; g < teams; ++g) {
                const float4 w = buf[g * p.tpr + t];
                v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
            }
        return v;
    };
    float2 b[NV * kP];
#pragma unroll
    for (int i = 0; i < NV * kP; ++i) b[i] = both(0.0f);
    bool fresh = true;                       // no share has left its sums in part_post yet
    int last = -1;                           // the slot of the row before, not yet refilled,
    long long refill = -1;                   // and the row whose first part it already has
    for (long long item = blockIdx.x; item < p.items; item += gridDim.x) {
        const long long gi = item / p.splits, g0 = gi * p.gate_rows, r0 = g0 + (item - gi * p.splits) * p.item_rows;
        const long long end = min(min(r0 + p.item_rows, g0 + p.gate_rows), p.rows), first = r0 + team;
        const float *gate = p.gate ? p.gate + gi * cols : nullptr;
        if (has.y() && (fresh || gate)) {
            __syncthreads();                 // the last share's weights are no longer read
            for (int c = threadIdx.x; c < cols; c += blockDim.x)
                wu[c] = (p.w_post ? p.w_post[c] : 1.0f) * (p.alpha * (gate ? gate[c] : 1.0f));
        }
        if (fresh || gate) __syncthreads();
        float2 a[NV * kP];
#pragma unroll
        for (int i = 0; i < NV * kP; ++i) a[i] = both(0.0f);
        // a row's own numbers are fetched a row ahead of its work
        auto pre_of = [&](long long row) { return has.dn() && row < end ? p.rstd_pre[row] : 0.0f; };
        auto post_of = [&](long long row) { return has.y() && has.post() && row < end ? p.rstd_post[row] : 1.0f; };
        float next_pre = pre_of(first), next_post = post_of(first);
        X *dxo = static_cast<X *>(p.dx) + first * p.lddx;
        Y *dyo = static_cast<Y *>(p.dy) + first * p.lddy;
        for (long long row = first; row < end; row += teams, dxo += teams * p.lddx, dyo += teams * p.lddy) {
            const float pre = next_pre, post = next_post;
            next_pre = pre_of(row + teams);
            next_post = post_of(row + teams);
            const uint8_t *slot = ring.wait();
            bwd_row<NV, VEC, HAS, false, X, Y, N>(
                p, pre, post, dxo, dyo, t, cols, warps, red, which, a, b,
                [&](int k, bool first) {
                    Step<X, Y, N> in;
                    if (has.dr() && first) load_raw<VEC, X>(in.dr, in_slot<WHOLE, X>(slot, p.dr, p.lddr, row), k, t, p.tpr, cols);
                    if (has.dn()) {
                        load_raw<VEC, X>(in.r, in_slot<WHOLE, X>(slot + off_r, p.rin, p.ldr, row), k, t, p.tpr, cols);
                        if (first) load_raw<VEC, N>(in.dn, in_slot<WHOLE, N>(slot + off_n, p.dn, p.lddn, row), k, t, p.tpr, cols);
                    }
                    if (has.y()) load_raw<VEC, Y>(in.y, in_slot<WHOLE, Y>(slot + off_y, p.y, p.ldy, row), k, t, p.tpr, cols);
                    return in;
                },
                [&](int k) { return kept<VEC>(wq, k, t, p.tpr, cols); },
                [&](int k) { return kept<VEC>(wu, k, t, p.tpr, cols); },
                sync,
                [&](bool barrier) {
                    // every thread of the team is past the last row, and this one's first pass
                    if (!barrier) sync();
                    if (t == 0 && !ring.aborted) {
                        if (refill >= 0) issue_second(refill, last);
                        refill = -1;
                        if (ahead.item < p.items) {
                            issue_first(refill = ahead.row, ring.at);
                            advance(ahead);
                        }
                    }
                    last = ring.next();
                });
        }
        if (sums_a) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const float4 v = joined(a[k * kP], a[k * kP + 1]);
                if (team > 0) continue;
                leave_a(p, v.x, channel<VEC>(k, 0, t, p.tpr), item, gi, gate, fresh);
                leave_a(p, v.y, channel<VEC>(k, 1, t, p.tpr), item, gi, gate, fresh);
                leave_a(p, v.z, channel<VEC>(k, 2, t, p.tpr), item, gi, gate, fresh);
                leave_a(p, v.w, channel<VEC>(k, 3, t, p.tpr), item, gi, gate, fresh);
            }
        }
        fresh = false;
    }
    if (!sums_b) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const float4 v = joined(b[k * kP], b[k * kP + 1]);
        if (team > 0) continue;
        auto leave = [&](int e, float x) {
            const int c = channel<VEC>(k, e, t, p.tpr);
            if (c < cols) p.part_pre[(long long)blockIdx.x * cols + c] = x;
        };
        leave(0, v.x);
        leave(1, v.y);
        leave(2, v.z);
        leave(3, v.w);
    }
}

// ------------------------------------------------------------------ launches
// How a call runs: single loads for unaligned rows or vector loads, directly or
// through the ring, where rows off 16 bytes come in pieces.
enum Loads { kScalar, kVector, kRing, kPieceRing, kScalarRing };

// One translation unit per direction and type of the residual stream builds
// its instances.
int launch_fwd_f32(int nv, Loads loads, Has has, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st);
int launch_fwd_bf16(int nv, Loads loads, Has has, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st);
int launch_bwd_f32(int nv, Loads loads, Has has, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st);
int launch_bwd_bf16(int nv, Loads loads, Has has, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st);

// The kernel is a template argument, so that `allowed` is its own: the devices
// on which it may have all the shared memory there is.  (A limit set to each
// call's own size would be lowered by a call from another thread between here
// and the launch.)
template <auto KERNEL>
int launch_kernel(const Params &p, unsigned grid, size_t smem, cudaStream_t st)
{
    static std::atomic<uint64_t> allowed{0};
    if (smem > 40 * 1024) {                // with the static shared memory, 48 KB go without asking
        int sms = 0;
        const int dev = current_device(&sms);
        const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
        if (!bit || !(allowed.load(std::memory_order_relaxed) & bit)) {
            cudaFuncAttributes a;
            cudaError_t e = cudaFuncGetAttributes(&a, KERNEL);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMaxSmemPerCta - (int)a.sharedSizeBytes);
            if (e != cudaSuccess) return cuda_status(e);
            allowed.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    KERNEL<<<grid, (unsigned)(p.tpr * p.rpb), smem, st>>>(p);
    const int rc = cuda_status(cudaGetLastError());
    if (rc == AMSIM_OK) count_launch();
    return rc;
}

template <bool BWD, typename X, typename Y, typename N>
int launch_types(int nv, Loads loads, Has has, const Params &p, unsigned grid, cudaStream_t st)
{
    const int threads = p.tpr * p.rpb;
#define AMSIM_BN(...)                                                                             \
    do {                                                                                          \
        if constexpr (BWD) return launch_kernel<bwd_kernel<__VA_ARGS__, X, Y, N>>(p, grid, 0, st); \
        else return launch_kernel<fwd_kernel<__VA_ARGS__, X, Y, N>>(p, grid, 0, st);               \
    } while (0)
    const size_t rows_smem = (size_t)(BWD ? p.rpb : 1) * (kRingBarBytes + p.slots * p.slot_bytes);
    if constexpr (BWD) {
        const size_t smem = rows_smem + 8 * (size_t)kept_floats(p.cols) + (p.rpb > 1 ? kTeamThreads * sizeof(float4) : 0);
#define AMSIM_RING(...)                                                                                  \
    return has == kAll    ? launch_kernel<bwd_ring_kernel<__VA_ARGS__, kAll, X, Y, N>>(p, grid, smem, st)  \
           : has == kNoDr ? launch_kernel<bwd_ring_kernel<__VA_ARGS__, kNoDr, X, Y, N>>(p, grid, smem, st) \
                          : launch_kernel<bwd_ring_kernel<__VA_ARGS__, kSome, X, Y, N>>(p, grid, smem, st)
        if (loads == kScalarRing) AMSIM_RING(false, false);
        if (loads == kPieceRing) AMSIM_RING(true, false);
        if (loads == kRing) AMSIM_RING(true, true);
#undef AMSIM_RING
    } else {
        const size_t smem = rows_smem;
#define AMSIM_RING(...)                                                                                        \
    return threads > 256 ? launch_kernel<fwd_ring_kernel<512, __VA_ARGS__, kAll, X, Y, N>>(p, grid, smem, st)  \
                         : launch_kernel<fwd_ring_kernel<256, __VA_ARGS__, kAll, X, Y, N>>(p, grid, smem, st)
        if (loads == kScalarRing) AMSIM_RING(false, false);
        if (loads == kPieceRing) AMSIM_RING(true, false);
        if (loads == kRing && has == kAll) AMSIM_RING(true, true);
        if (loads == kRing) return launch_kernel<fwd_ring_kernel<256, true, true, kSome, X, Y, N>>(p, grid, smem, st);
#undef AMSIM_RING
    }
    if (loads == kVector) {
        if (nv == 1) AMSIM_BN(1, 128, true);
        if (nv == 2) AMSIM_BN(2, 128, true);
        if (threads <= 256) AMSIM_BN(4, 256, true);
        AMSIM_BN(4, 1024, true);
    }
    if (nv <= 2) AMSIM_BN(2, 128, false);
    if (threads <= 256) AMSIM_BN(4, 256, false);
    AMSIM_BN(4, 1024, false);
#undef AMSIM_BN
}

template <bool BWD, typename X>
int launch_stream(int nv, Loads loads, Has has, int y_type, int n_type, const Params &p, unsigned grid,
                  cudaStream_t st)
{
    if (y_type == AMSIM_F32)
        return n_type == AMSIM_F32 ? launch_types<BWD, X, float, float>(nv, loads, has, p, grid, st)
                                   : launch_types<BWD, X, float, bf16>(nv, loads, has, p, grid, st);
    return n_type == AMSIM_F32 ? launch_types<BWD, X, bf16, float>(nv, loads, has, p, grid, st)
                               : launch_types<BWD, X, bf16, bf16>(nv, loads, has, p, grid, st);
}

}  // namespace bn
}  // namespace amsim
