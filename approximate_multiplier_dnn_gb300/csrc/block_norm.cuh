// The block norm's kernels: RMS norms before and after a block, fused with the
// block's gate and the residual scale.
//
// HBM-bound: the forward pass reads x and y and writes r and n, the backward
// pass reads y, r, dr, dn and writes dx, dy, each once.  A row is held in the
// registers of the threads that share it (8 channels per thread and step), so
// both norms of a row and everything between them take one pass over memory.
#pragma once

#include <cuda_bf16.h>

#include "bounded_wait.cuh"

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
    int slots, slot_bytes;                 // ring kernels: rows ahead in shared memory, bytes of one
    long long block_rows;                  // ring forward: rows of a thread block
    float alpha, eps;
};

// Channels a thread takes at a step: 16 bytes of fp32, 8 of bf16, so that a
// warp's loads and stores are whole neighbouring sectors whichever the type.
constexpr int kE = 4;
struct Four {
    float v[kE];
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
#pragma unroll
        for (int e = 0; e < kE; ++e) r.v[e] = __uint_as_float(d.w[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            r.v[2 * e] = __uint_as_float(d.w[e] << 16);
            r.v[2 * e + 1] = __uint_as_float(d.w[e] & 0xFFFF0000u);
        }
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
            *reinterpret_cast<float4 *>(row + c) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(r.v[0], r.v[1]), b = __floats2bfloat162_rn(r.v[2], r.v[3]);
            *reinterpret_cast<uint2 *>(row + c) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        }
    } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int c = channel<false>(k, e, t, tpr);
            if (c < cols) put(row + c, r.v[e]);
        }
    }
}

// Four fp32 weights (ones where there are none).
template <bool VEC>
__device__ __forceinline__ Four weights(const float *w, int k, int t, int tpr, int cols)
{
    Four r;
    if (!w) {
#pragma unroll
        for (int e = 0; e < kE; ++e) r.v[e] = 1.0f;
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

// Three such sums behind one barrier.
struct Three {
    float v[3];
};
__device__ __forceinline__ Three row_sums(Three x, int warps, float (*red)[3][32], int &which)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) x.v[i] += __shfl_xor_sync(0xFFFFFFFFu, x.v[i], d);
    if (warps == 1) return x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float (*buf)[32] = red[which];
    which ^= 1;
    if (lane < 3) buf[lane][warp] = lane == 0 ? x.v[0] : lane == 1 ? x.v[1] : x.v[2];
    __syncthreads();
    const int first = warp / warps * warps;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        float v = lane < warps ? buf[i][first + lane] : 0.0f;
#pragma unroll
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        x.v[i] = v;
    }
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
            const Four a = widen(yr[k]);
#pragma unroll
            for (int e = 0; e < kE; ++e) s = fmaf(a.v[e], a.v[e], s);
        }
        post = 1.0f / sqrtf(fmaf(row_sum(s, warps, red, which), inv, p.eps));
        if (on && t == 0 && p.rstd_post) p.rstd_post[row] = post;
    }
    const float *gate = p.gate ? p.gate + row / p.gate_rows * p.cols : nullptr;
    Four r[NV];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        r[k] = widen(xr[k]);
        if (p.y) {
            const Four a = widen(yr[k]);
            const Four w = weights<VEC>(p.w_post, k, t, p.tpr, cols), g = weights<VEC>(gate, k, t, p.tpr, cols);
#pragma unroll
            for (int e = 0; e < kE; ++e) r[k].v[e] = fmaf(post * a.v[e], w.v[e] * (p.alpha * g.v[e]), r[k].v[e]);
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) s = fmaf(r[k].v[e], r[k].v[e], s);
        if (p.r) store4<VEC, X>(static_cast<X *>(p.r) + row * p.ldr, k, t, p.tpr, cols, r[k]);
    }
    if (!p.n) return;
    const float pre = 1.0f / sqrtf(fmaf(row_sum(s, warps, red, which), inv, p.eps));
    if (on && t == 0 && p.rstd_pre) p.rstd_pre[row] = pre;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const Four w = weights<VEC>(p.w_pre, k, t, p.tpr, cols);
#pragma unroll
        for (int e = 0; e < kE; ++e) r[k].v[e] = r[k].v[e] * pre * w.v[e];
        store4<VEC, N>(static_cast<N *>(p.n) + row * p.ldn, k, t, p.tpr, cols, r[k]);
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

// A channel's sum over a share's rows leaves: to the share's slot when several
// make up a row of the gate, else to dgate and the block's slot of dw_post.
template <bool VEC>
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

// A thread's words of one step of a row in the backward pass.
template <typename X, typename Y, typename N>
struct Step {
    Raw<X> dr, r;
    Raw<Y> y;
    Raw<N> dn;
};

// The gradients of one row.  The second norm's mean is wanted of s = wu dx,
// which itself contains the first norm's mean m = mean(t rh); as
//   dx = q - pre m rh,  q = dr + pre t,
//   mean(s yh) = mean(wu yh q) - pre m mean(wu yh rh),
// all three means come from one pass over the row and one barrier.
// `load(k)`: the thread's words of step k; `wq(k)`: w_pre; `wu(k)`: alpha gate
// w_post.  Rows of up to two steps per thread stay in registers between the
// two passes; wider ones are loaded again (from shared memory or the L1 cache),
// which leaves the registers to the column sums.  `met(barrier)` runs between
// the passes, `barrier` telling whether every thread was waited for there.
template <int NV, bool VEC, typename X, typename Y, typename N, typename LOAD, typename WQ, typename WU, typename F>
__device__ __forceinline__ void bwd_row(const Params &p, float pre, float post, long long row, int t, int cols,
                                        int warps, float (*red)[3][32], int &which, float (&a)[NV * kE],
                                        float (&b)[NV * kE], LOAD load, WQ wq, WU wu, F met)
{
    const bool want_y = p.y != nullptr, want_n = p.dn != nullptr;
    const float inv = 1.0f / (float)p.cols;
    constexpr bool keep = NV <= 2;
    Four qs[keep ? NV : 1], rhs[keep ? NV : 1], yhs[keep ? NV : 1];
    auto widened = [&](const Step<X, Y, N> &in, int k, Four &q, Four &rh, Four &yh, Four &t) {
        if (p.dr) {
            q = widen(in.dr);
        } else {
#pragma unroll
            for (int e = 0; e < kE; ++e) q.v[e] = 0.0f;
        }
        if (want_n) {
            rh = widen(in.r);
            const Four n = widen(in.dn), w = wq(k);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                rh.v[e] *= pre;
                t.v[e] = n.v[e] * w.v[e];
                q.v[e] = fmaf(pre, t.v[e], q.v[e]);
            }
        }
        if (want_y) {
            yh = widen(in.y);
#pragma unroll
            for (int e = 0; e < kE; ++e) yh.v[e] *= post;
        }
    };
    Three sum = {{0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const Step<X, Y, N> in = load(k);
        Four t, &q = qs[keep ? k : 0], &rh = rhs[keep ? k : 0], &yh = yhs[keep ? k : 0];
        widened(in, k, q, rh, yh, t);
        if (want_n) {
            const Four n = widen(in.dn);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                sum.v[0] = fmaf(t.v[e], rh.v[e], sum.v[0]);
                b[k * kE + e] = fmaf(n.v[e], rh.v[e], b[k * kE + e]);
            }
        }
        if (want_y) {
            const Four w = wu(k);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float u = w.v[e] * yh.v[e];
                sum.v[1] = fmaf(u, q.v[e], sum.v[1]);
                if (want_n) sum.v[2] = fmaf(u, rh.v[e], sum.v[2]);
            }
        }
    }
    const bool means = want_n || (want_y && p.w_post);
    if (means) sum = row_sums(sum, warps, red, which);
    met(means && warps > 1);
    const float m = pre * (sum.v[0] * inv);
    const float s = !p.w_post ? 0.0f : (want_n ? fmaf(-m, sum.v[2], sum.v[1]) : sum.v[1]) * inv;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        Four &q = qs[keep ? k : 0], &rh = rhs[keep ? k : 0], &yh = yhs[keep ? k : 0];
        if (!keep) {
            Four none;
            widened(load(k), k, q, rh, yh, none);
        }
        if (want_n)
#pragma unroll
            for (int e = 0; e < kE; ++e) q.v[e] = fmaf(-m, rh.v[e], q.v[e]);
        if (p.dx) store4<VEC, X>(static_cast<X *>(p.dx) + row * p.lddx, k, t, p.tpr, cols, q);
        if (!want_y) continue;
        const Four w = wu(k);
        Four o;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            a[k * kE + e] = fmaf(q.v[e], yh.v[e], a[k * kE + e]);
            o.v[e] = post * fmaf(-yh.v[e], s, q.v[e] * w.v[e]);
        }
        if (p.dy) store4<VEC, Y>(static_cast<Y *>(p.dy) + row * p.lddy, k, t, p.tpr, cols, o);
    }
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
    float b[NV * kE];
#pragma unroll
    for (int i = 0; i < NV * kE; ++i) b[i] = 0.0f;
    bool fresh = true;                       // no share has left its sums in part_post yet
    for (long long item = blockIdx.x; item < p.items; item += gridDim.x) {
        const long long gi = item / p.splits;
        const long long g0 = gi * p.gate_rows, g1 = min(g0 + p.gate_rows, p.rows);
        const long long r0 = g0 + (item - gi * p.splits) * p.item_rows, r1 = min(r0 + p.item_rows, g1);
        const float *gate = p.gate ? p.gate + gi * p.cols : nullptr;
        float a[NV * kE];
#pragma unroll
        for (int i = 0; i < NV * kE; ++i) a[i] = 0.0f;
        for (long long rb = r0; rb < r1; rb += p.rpb) {
            const long long row = rb + group;
            const bool on = row < r1;
            const int cols = on ? p.cols : 0;
            const float pre = want_n && on ? p.rstd_pre[row] : 0.0f;
            const float post = !want_y || !p.w_post ? 1.0f : on ? p.rstd_post[row] : 0.0f;
            bwd_row<NV, VEC, X, Y, N>(
                p, pre, post, row, t, cols, warps, red, which, a, b,
                [&](int k) {
                    Step<X, Y, N> in;
                    if (p.dr) load_raw<VEC, X>(in.dr, static_cast<const X *>(p.dr) + row * p.lddr, k, t, p.tpr, cols);
                    if (want_n) {
                        load_raw<VEC, X>(in.r, static_cast<const X *>(p.rin) + row * p.ldr, k, t, p.tpr, cols);
                        load_raw<VEC, N>(in.dn, static_cast<const N *>(p.dn) + row * p.lddn, k, t, p.tpr, cols);
                    }
                    if (want_y) load_raw<VEC, Y>(in.y, static_cast<const Y *>(p.y) + row * p.ldy, k, t, p.tpr, cols);
                    return in;
                },
                [&](int k) { return weights<VEC>(p.w_pre, k, t, p.tpr, cols); },
                [&](int k) {
                    Four w = weights<VEC>(p.w_post, k, t, p.tpr, cols);
                    const Four g = weights<VEC>(gate, k, t, p.tpr, cols);
#pragma unroll
                    for (int e = 0; e < kE; ++e) w.v[e] *= p.alpha * g.v[e];
                    return w;
                },
                [](bool) {});
        }
        if (!sums_a) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float v = group_sum(a[k * kE + e], p.tpr, p.rpb, buf);
                if (group == 0) leave_a<VEC>(p, v, channel<VEC>(k, e, t, p.tpr), item, gi, gate, fresh);
            }
        fresh = false;
    }
    if (!sums_b) return;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const float v = group_sum(b[k * kE + e], p.tpr, p.rpb, buf);
            const int c = channel<VEC>(k, e, t, p.tpr);
            if (group == 0 && c < p.cols) p.part_pre[(long long)blockIdx.x * p.cols + c] = v;
        }
}

// ------------------------------------------------------------------ rows by bulk copies
// The kernels above keep one row's bytes in flight per block, and none while
// they reduce it: 40 % of the copy bandwidth at 16384 x 4096.  Where rows are
// vectors of 16 bytes and there are many, a block streams its rows through a
// ring in shared memory instead: one thread issues whole-row bulk copies, and
// refills a slot as soon as every thread has its words of it in registers.
// Channels are dealt to threads, and sums taken, as above, so a row's results
// do not depend on how many rows come with it.
struct Ring {
    uint8_t *slot0;
    uint64_t *full;
    int slots, bytes;
    int at = 0;
    uint32_t phase = 0;
    bool aborted = false;

    __device__ __forceinline__ uint8_t *wait()
    {
        tc::bar_wait(full + at, phase, aborted);
        return slot0 + (size_t)at * bytes;
    }
    // The slot just read is free: `at` moves on.
    __device__ __forceinline__ int next()
    {
        const int s = at;
        if (++at == slots) { at = 0; phase ^= 1; }
        return s;
    }
};

constexpr int kRingBarBytes = 128;         // up to 16 slots
// Resident blocks of 256 threads per SM, by direction and steps per thread.
#ifndef RBF2
#define RBF2 3
#endif
#ifndef RBF4
#define RBF4 2
#endif
#ifndef RBB2
#define RBB2 2
#endif
#ifndef RBB4
#define RBB4 2
#endif
__host__ __device__ constexpr int ring_blocks(bool bwd, int nv) { return bwd ? (nv == 2 ? RBB2 : RBB4) : (nv == 2 ? RBF2 : RBF4); }
constexpr int kRingAlign = 128;
__host__ __device__ inline int ring_bytes(int cols, int size) { return (cols * size + kRingAlign - 1) / kRingAlign * kRingAlign; }

__device__ __forceinline__ Ring make_ring(const Params &p, uint8_t *smem)
{
    Ring r;
    r.full = reinterpret_cast<uint64_t *>(smem);
    r.slot0 = smem + kRingBarBytes;
    r.slots = p.slots;
    r.bytes = p.slot_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.slots; ++i) tc::bar_init(r.full + i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    return r;
}

// The thread's words of step k of a row in shared memory.
template <typename T>
__device__ __forceinline__ void take(Raw<T> &d, const uint8_t *row, int k, int t, int tpr, int cols)
{
    load_raw<true, T>(d, reinterpret_cast<const T *>(row), k, t, tpr, cols);
}

template <int NV, int THREADS, typename X, typename Y, typename N>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? ring_blocks(false, NV) : 1) fwd_ring_kernel(const Params p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][32];
    int which = 0;
    const int t = threadIdx.x, warps = p.tpr >> 5, cols = p.cols;
    const int xb = cols * (int)sizeof(X), yb = cols * (int)sizeof(Y), yoff = ring_bytes(cols, sizeof(X));
    const long long r0 = blockIdx.x * p.block_rows, r1 = min(r0 + p.block_rows, p.rows);
    Ring ring = make_ring(p, smem);
    auto issue = [&](long long row, int slot) {
        uint8_t *s = ring.slot0 + (size_t)slot * ring.bytes;
        tc::bar_expect(ring.full + slot, xb + (p.y ? yb : 0));
        tc::copy_bytes(s, static_cast<const X *>(p.x) + row * p.ldx, xb, ring.full + slot);
        if (p.y) tc::copy_bytes(s + yoff, static_cast<const Y *>(p.y) + row * p.ldy, yb, ring.full + slot);
    };
    if (t == 0)
        for (int i = 0; i < p.slots && r0 + i < r1; ++i) issue(r0 + i, i);
    const float inv = 1.0f / (float)cols;
    Four wq[NV], wu[NV];                  // w_pre, and alpha gate w_post of the rows' gate
    if (p.n)
#pragma unroll
        for (int k = 0; k < NV; ++k) wq[k] = weights<true>(p.w_pre, k, t, p.tpr, cols);
    long long gate_end = r0;               // first row with another gate
    for (long long row = r0; row < r1; ++row) {
        if (p.y && row == gate_end) {
            const long long g = row / p.gate_rows;
            gate_end = (g + 1) * p.gate_rows;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                wu[k] = weights<true>(p.w_post, k, t, p.tpr, cols);
                const Four a = weights<true>(p.gate ? p.gate + g * cols : nullptr, k, t, p.tpr, cols);
#pragma unroll
                for (int e = 0; e < kE; ++e) wu[k].v[e] *= p.alpha * a.v[e];
            }
        }
        const uint8_t *slot = ring.wait();
        Raw<X> xr[NV];
        Raw<Y> yr[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) take<X>(xr[k], slot, k, t, p.tpr, cols);
        if (p.y)
#pragma unroll
            for (int k = 0; k < NV; ++k) take<Y>(yr[k], slot + yoff, k, t, p.tpr, cols);
        float post = 1.0f;
        if (p.w_post) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const Four a = widen(yr[k]);
#pragma unroll
                for (int e = 0; e < kE; ++e) s = fmaf(a.v[e], a.v[e], s);
            }
            post = 1.0f / sqrtf(fmaf(row_sum(s, warps, red, which), inv, p.eps));
            if (t == 0 && p.rstd_post) p.rstd_post[row] = post;
        }
        if (!p.w_post || warps == 1) __syncthreads();      // else row_sum's barrier: the slot has been read
        const int freed = ring.next();
        if (t == 0 && row + p.slots < r1) issue(row + p.slots, freed);
        Four r[NV];
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            r[k] = widen(xr[k]);
            if (p.y) {
                const Four a = widen(yr[k]);
#pragma unroll
                for (int e = 0; e < kE; ++e) r[k].v[e] = fmaf(post * a.v[e], wu[k].v[e], r[k].v[e]);
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) s = fmaf(r[k].v[e], r[k].v[e], s);
            if (p.r) store4<true, X>(static_cast<X *>(p.r) + row * p.ldr, k, t, p.tpr, cols, r[k]);
        }
        if (!p.n) continue;
        const float pre = 1.0f / sqrtf(fmaf(row_sum(s, warps, red, which), inv, p.eps));
        if (t == 0 && p.rstd_pre) p.rstd_pre[row] = pre;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int e = 0; e < kE; ++e) r[k].v[e] = r[k].v[e] * pre * wq[k].v[e];
            store4<true, N>(static_cast<N *>(p.n) + row * p.ldn, k, t, p.tpr, cols, r[k]);
        }
    }
}

// As bwd_kernel, one row at a time per block.  The weights wait in shared
// memory after the ring (w_pre, then alpha gate w_post of the share's gate).
template <int NV, int THREADS, typename X, typename Y, typename N>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? ring_blocks(true, NV) : 1) bwd_ring_kernel(const Params p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[2][3][32];
    int which = 0;
    const int t = threadIdx.x, warps = p.tpr >> 5, cols = p.cols;
    const bool want_y = p.y != nullptr, want_n = p.dn != nullptr;
    const bool sums_a = want_y && (p.dgate || p.dw_post), sums_b = want_n && p.dw_pre;
    const int xb = cols * (int)sizeof(X), yb = cols * (int)sizeof(Y), nb = cols * (int)sizeof(N);
    const int rxb = ring_bytes(cols, sizeof(X)), rnb = ring_bytes(cols, sizeof(N));
    const int off_r = p.dr ? rxb : 0, off_n = off_r + (want_n ? rxb : 0), off_y = off_n + (want_n ? rnb : 0);
    float *wq = reinterpret_cast<float *>(smem + kRingBarBytes + (size_t)p.slots * p.slot_bytes);
    float *wu = wq + cols;
    Ring ring = make_ring(p, smem);
    // the rows of this block in order: shares blockIdx.x, + gridDim.x, ...
    struct Place {
        long long item, row, end;
    };
    auto bounds = [&](Place &q) {
        if (q.item >= p.items) { q.row = q.end = 0; return; }
        const long long gi = q.item / p.splits, g0 = gi * p.gate_rows;
        q.row = g0 + (q.item - gi * p.splits) * p.item_rows;
        q.end = min(min(q.row + p.item_rows, g0 + p.gate_rows), p.rows);
    };
    auto issue = [&](const Place &q, int slot) {
        uint8_t *s = ring.slot0 + (size_t)slot * ring.bytes;
        tc::bar_expect(ring.full + slot, (p.dr ? xb : 0) + (want_n ? xb + nb : 0) + (want_y ? yb : 0));
        if (p.dr) tc::copy_bytes(s, static_cast<const X *>(p.dr) + q.row * p.lddr, xb, ring.full + slot);
        if (want_n) {
            tc::copy_bytes(s + off_r, static_cast<const X *>(p.rin) + q.row * p.ldr, xb, ring.full + slot);
            tc::copy_bytes(s + off_n, static_cast<const N *>(p.dn) + q.row * p.lddn, nb, ring.full + slot);
        }
        if (want_y) tc::copy_bytes(s + off_y, static_cast<const Y *>(p.y) + q.row * p.ldy, yb, ring.full + slot);
    };
    auto advance = [&](Place &q) {
        if (++q.row < q.end) return;
        q.item += gridDim.x;
        bounds(q);
    };
    Place ahead{(long long)blockIdx.x, 0, 0};
    bounds(ahead);
    if (t == 0)
        for (int i = 0; i < p.slots && ahead.item < p.items; ++i) {
            issue(ahead, i);
            advance(ahead);
        }
    auto kept = [&](const float *w, int k) {
        Raw<float> d;
        load_raw<true, float>(d, w, k, t, p.tpr, cols);
        return widen(d);
    };
    if (want_n)
        for (int c = t; c < cols; c += p.tpr) wq[c] = p.w_pre ? p.w_pre[c] : 1.0f;
    float b[NV * kE];
#pragma unroll
    for (int i = 0; i < NV * kE; ++i) b[i] = 0.0f;
    bool fresh = true;                       // no share has left its sums in part_post yet
    int last = -1;                           // the slot of the row before, not yet refilled
    for (long long item = blockIdx.x; item < p.items; item += gridDim.x) {
        Place q{item, 0, 0};
        bounds(q);
        const long long gi = item / p.splits;
        const float *gate = p.gate ? p.gate + gi * cols : nullptr;
        if (want_y && (fresh || gate)) {
            __syncthreads();                 // the last share's weights are no longer read
            for (int c = t; c < cols; c += p.tpr)
                wu[c] = (p.w_post ? p.w_post[c] : 1.0f) * (p.alpha * (gate ? gate[c] : 1.0f));
        }
        if (fresh || gate) __syncthreads();
        float a[NV * kE];
#pragma unroll
        for (int i = 0; i < NV * kE; ++i) a[i] = 0.0f;
        // a row's own numbers are fetched a row ahead: their latency is longer than the row's work
        auto pre_of = [&](long long row) { return want_n && row < q.end ? p.rstd_pre[row] : 0.0f; };
        auto post_of = [&](long long row) { return want_y && p.w_post && row < q.end ? p.rstd_post[row] : 1.0f; };
        float next_pre = pre_of(q.row), next_post = post_of(q.row);
        for (long long row = q.row; row < q.end; ++row) {
            const float pre = next_pre, post = next_post;
            next_pre = pre_of(row + 1);
            next_post = post_of(row + 1);
            const uint8_t *slot = ring.wait();
            bwd_row<NV, true, X, Y, N>(
                p, pre, post, row, t, cols, warps, red, which, a, b,
                [&](int k) {
                    Step<X, Y, N> in;
                    if (p.dr) take<X>(in.dr, slot, k, t, p.tpr, cols);
                    if (want_n) {
                        take<X>(in.r, slot + off_r, k, t, p.tpr, cols);
                        take<N>(in.dn, slot + off_n, k, t, p.tpr, cols);
                    }
                    if (want_y) take<Y>(in.y, slot + off_y, k, t, p.tpr, cols);
                    return in;
                },
                [&](int k) { return kept(wq, k); }, [&](int k) { return kept(wu, k); },
                [&](bool barrier) {
                    // free now: this row's slot if it stays in registers, else the last row's
                    if (!barrier) __syncthreads();
                    const int freed = NV <= 2 ? ring.next() : last;
                    if (NV > 2) last = ring.next();
                    if (t == 0 && freed >= 0 && ahead.item < p.items) {
                        issue(ahead, freed);
                        advance(ahead);
                    }
                });
        }
        if (sums_a) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < kE; ++e)
                    leave_a<true>(p, a[k * kE + e], channel<true>(k, e, t, p.tpr), item, gi, gate, fresh);
        }
        fresh = false;
    }
    if (!sums_b) return;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const int c = channel<true>(k, e, t, p.tpr);
            if (c < cols) p.part_pre[(long long)blockIdx.x * cols + c] = b[k * kE + e];
        }
}

// How a call runs: single loads for unaligned rows, vector loads, or the ring.
enum Loads { kScalar = 0, kVector = 1, kRing = 2 };

// One translation unit per type of the residual stream builds its instances.
int launch_f32(bool bwd, int nv, Loads loads, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st);
int launch_bf16(bool bwd, int nv, Loads loads, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st);

template <typename K>
int launch_kernel(K kernel, const Params &p, unsigned grid, size_t smem, cudaStream_t st)
{
    if (smem > 40 * 1024) {                // with the static shared memory, 48 KB go without asking
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return cuda_status(e);
    }
    kernel<<<grid, (unsigned)(p.tpr * p.rpb), smem, st>>>(p);
    const int rc = cuda_status(cudaGetLastError());
    if (rc == AMSIM_OK) count_launch();
    return rc;
}

template <typename X, typename Y, typename N>
int launch_types(bool bwd, int nv, Loads loads, const Params &p, unsigned grid, cudaStream_t st)
{
    const int threads = p.tpr * p.rpb;
#define AMSIM_BN(KERNEL, ...) \
    launch_kernel(bwd ? bwd_##KERNEL<__VA_ARGS__, X, Y, N> : fwd_##KERNEL<__VA_ARGS__, X, Y, N>, p, grid, smem, st)
    size_t smem = 0;
    if (loads == kRing) {
        smem = kRingBarBytes + (size_t)p.slots * p.slot_bytes + (bwd ? 8 * (size_t)p.cols : 0);
        if (nv == 2) return AMSIM_BN(ring_kernel, 2, 256);
        if (threads <= 256) return AMSIM_BN(ring_kernel, 4, 256);
        return AMSIM_BN(ring_kernel, 4, 512);
    }
    if (loads == kVector) {
        if (nv == 1) return AMSIM_BN(kernel, 1, 128, true);
        if (nv == 2) return AMSIM_BN(kernel, 2, 256, true);
        if (threads <= 512) return AMSIM_BN(kernel, 4, 512, true);
        return AMSIM_BN(kernel, 4, 1024, true);
    }
    if (nv <= 2) return AMSIM_BN(kernel, 2, 256, false);
    return AMSIM_BN(kernel, 4, 1024, false);
#undef AMSIM_BN
}

template <typename X>
int launch_stream(bool bwd, int nv, Loads loads, int y_type, int n_type, const Params &p, unsigned grid, cudaStream_t st)
{
    if (y_type == AMSIM_F32)
        return n_type == AMSIM_F32 ? launch_types<X, float, float>(bwd, nv, loads, p, grid, st)
                                   : launch_types<X, float, bf16>(bwd, nv, loads, p, grid, st);
    return n_type == AMSIM_F32 ? launch_types<X, bf16, float>(bwd, nv, loads, p, grid, st)
                               : launch_types<X, bf16, bf16>(bwd, nv, loads, p, grid, st);
}

}  // namespace bn
}  // namespace amsim
