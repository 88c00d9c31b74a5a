// The group norm with its activation, channels last, and its gradients.
//
// Two ways.  Where a slab (a sample's pixels over some whole groups, at least
// 128 bytes of a pixel) fits the shared memory of a cluster, its blocks keep it
// there: x (backward: x and dy) is read once and the result written, which is
// all that has to move.  Each thread copies, sums and finishes pieces of its
// own, so the copies need no barrier between threads; the blocks of a cluster
// exchange the groups' sums through distributed shared memory.  Larger slabs go
// through three launches that read x (and dy) twice.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "amsim_internal.h"
#include "chained.cuh"
#include "pairs.cuh"

namespace {

struct Params {
    const void *x, *dy;
    const float *w, *b;
    void *y, *dx;
    float *mean, *rstd, *dw, *db;
    float2 *part, *sums, *means;             // scratch: [batch][chunks][channels], [batch][channels], [batch][groups]
    int64_t pixels, ldx, ldy, lddx, chunk;   // chunk: pixels of a share
    int batch, chunks, channels, groups, size;   // size: channels of a group
    int act, tx, tiles;                      // tx: threads side by side over channels
    int slab, slab_groups, slabs, cluster;   // resident: channels and groups of a slab; blocks of a cluster,
    int rows, step, steps;                   // pixels of a block, of its threads at once, of a thread
    float eps;
};

constexpr int kThreads = 256;

template <typename T, int E>
struct alignas(sizeof(T) * E) Vec {
    T e[E];
};
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float v, float *o) { *o = v; }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(v); }

template <int E, typename T>
__device__ __forceinline__ void load(const T *at, float (&v)[E])
{
    const Vec<T, E> r = *reinterpret_cast<const Vec<T, E> *>(at);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = widen(r.e[e]);
}
template <int E, typename T>
__device__ __forceinline__ void store(T *at, const float (&v)[E])
{
    Vec<T, E> r;
#pragma unroll
    for (int e = 0; e < E; ++e) narrow(v[e], &r.e[e]);
    *reinterpret_cast<Vec<T, E> *>(at) = r;
}

// n values with their mean and their sum of squares about it; two sets joined.
struct Moments {
    float n, mean, m2;
};
__device__ __forceinline__ Moments join(const Moments &a, const Moments &b)
{
    if (b.n == 0.0f) return a;
    if (a.n == 0.0f) return b;
    const float n = a.n + b.n;
    const float d = b.mean - a.mean, f = __fdividef(b.n, n);
    return Moments{n, a.mean + d * f, a.m2 + b.m2 + d * d * (a.n * f)};
}

// 1 / (1 + exp(-z)), from t = -z log2(e).  The approximate instructions' errors
// are a rounding of t and some 2^-22, no more than z's own rounding leaves; expf
// and an exact quotient take three times the instructions, and the kernels are
// near the issue limit.
constexpr float kMinusLog2E = -1.44269504088896341f;
__device__ __forceinline__ float power_of_2(float t)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return e;
}
__device__ __forceinline__ float reciprocal(float d)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}
__device__ __forceinline__ float sigmoid(float z) { return reciprocal(1.0f + power_of_2(z * kMinusLog2E)); }
template <int ACT>
__device__ __forceinline__ float activate(float z)
{
    if (ACT == AMSIM_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if (ACT == AMSIM_ACT_SILU) return z * sigmoid(z);
    return z;
}

// The activation as a constant of the loop that `use` holds.
template <int ACT>
struct Act {
    static constexpr int value = ACT;
};
template <typename F>
__device__ __forceinline__ void with_activation(int act, F use)
{
    if (act == AMSIM_ACT_RELU)
        use(Act<AMSIM_ACT_RELU>{});
    else if (act == AMSIM_ACT_SILU)
        use(Act<AMSIM_ACT_SILU>{});
    else
        use(Act<AMSIM_ACT_NONE>{});
}

// dy act'(z).  relu's gradient jumps where z = 0: a z that its own roundings
// (three of xh w, one of the sum: at most 2^-22 of the terms) could carry
// across is computed again in 64 bits.
template <int ACT>
__device__ __forceinline__ float before_activation(float dy, float x, float xh, float mean, float rstd, float w, float b)
{
    if (ACT == AMSIM_ACT_NONE) return dy;
    const float z = fmaf(xh, w, b);
    if (ACT == AMSIM_ACT_RELU) {
        bool on = z > 0.0f;
        if (fabsf(z) <= 0x1p-21f * (fabsf(xh * w) + fabsf(b)))
            on = ((double)x - (double)mean) * (double)rstd * (double)w + (double)b > 0.0;
        return on ? dy : 0.0f;
    }
    const float s = sigmoid(z);
    return dy * (s * fmaf(z, 1.0f - s, 1.0f));
}

// A thread's place: its first channel and its first pixel, by blocks of
// (chunk of pixels, tile of channels, sample).
struct Place {
    int n, chunk, c, y, ty;
    int64_t first, last;
    bool on;
};
template <int E>
__device__ __forceinline__ Place place(const Params &p)
{
    Place t;
    const int tile = (int)(blockIdx.x / (unsigned)p.chunks) % p.tiles;
    t.n = (int)(blockIdx.x / (unsigned)p.chunks) / p.tiles;
    t.chunk = (int)(blockIdx.x % (unsigned)p.chunks);
    t.ty = kThreads / p.tx;
    t.y = threadIdx.x / p.tx;
    t.c = (tile * p.tx + (int)threadIdx.x % p.tx) * E;
    t.on = t.c < p.channels;
    t.first = t.chunk * p.chunk;
    t.last = min(t.first + p.chunk, p.pixels);
    return t;
}

// Each channel's moments over a chunk of pixels.  A thread sums about its first
// value, so what cancels is no larger than the values' own spread.
template <typename TX, int E>
__global__ void __launch_bounds__(kThreads) moments_kernel(const Params p)
{
    __shared__ Moments all[E][kThreads];
    const Place t = place<E>(p);
    float s1[E] = {}, s2[E] = {}, about[E] = {};
    int count = 0;
    if (t.on) {
        const TX *x = static_cast<const TX *>(p.x) + t.n * p.pixels * p.ldx + t.c;
#pragma unroll 4
        for (int64_t i = t.first + t.y; i < t.last; i += t.ty) {
            float v[E];
            load<E>(x + i * p.ldx, v);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (count == 0) about[e] = v[e];
                const float d = v[e] - about[e];
                s1[e] += d;
                s2[e] = fmaf(d, d, s2[e]);
            }
            ++count;
        }
    }
    const float n = (float)count, inv = count ? 1.0f / n : 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float m = s1[e] * inv;
        all[e][threadIdx.x] = Moments{n, about[e] + m, fmaxf(s2[e] - s1[e] * m, 0.0f)};
    }
    for (int half = t.ty >> 1; half; half >>= 1) {
        __syncthreads();
        if (t.y < half)
#pragma unroll
            for (int e = 0; e < E; ++e)
                all[e][threadIdx.x] = join(all[e][threadIdx.x], all[e][threadIdx.x + half * p.tx]);
    }
    if (t.on && t.y == 0)
#pragma unroll
        for (int e = 0; e < E; ++e)
            p.part[((int64_t)t.n * p.chunks + t.chunk) * p.channels + t.c + e] =
                make_float2(all[e][threadIdx.x].mean, all[e][threadIdx.x].m2);
}

// A group's moments from its channels' over all chunks: a block per (n, g).
__global__ void __launch_bounds__(kThreads) join_kernel(const Params p)
{
    __shared__ Moments all[kThreads];
    amsim::chain_wait();
    const int n = blockIdx.x / p.groups, g = blockIdx.x % p.groups;
    Moments m{0.0f, 0.0f, 0.0f};
    for (int64_t i = threadIdx.x; i < (int64_t)p.chunks * p.size; i += kThreads) {
        const int64_t chunk = i / p.size;
        const float2 v = p.part[((int64_t)n * p.chunks + chunk) * p.channels + g * p.size + i % p.size];
        m = join(m, Moments{(float)(min((chunk + 1) * p.chunk, p.pixels) - chunk * p.chunk), v.x, v.y});
    }
    all[threadIdx.x] = m;
    for (int half = kThreads / 2; half; half >>= 1) {
        __syncthreads();
        if (threadIdx.x < half) all[threadIdx.x] = join(all[threadIdx.x], all[threadIdx.x + half]);
    }
    if (threadIdx.x == 0) {
        p.mean[blockIdx.x] = all[0].mean;
        p.rstd[blockIdx.x] = 1.0f / sqrtf((all[0].n > 0.0f ? all[0].m2 / all[0].n : 0.0f) + p.eps);
    }
}

template <int E>
struct Channels {
    float mean[E], rstd[E], w[E], b[E];
};
template <int E>
__device__ __forceinline__ Channels<E> channels(const Params &p, int n, int c)
{
    Channels<E> k;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int g = (c + e) / p.size;
        k.mean[e] = p.mean[(int64_t)n * p.groups + g];
        k.rstd[e] = p.rstd[(int64_t)n * p.groups + g];
        k.w[e] = p.w ? p.w[c + e] : 1.0f;
        k.b[e] = p.b ? p.b[c + e] : 0.0f;
    }
    return k;
}

template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(kThreads) apply_kernel(const Params p)
{
    amsim::chain_wait();
    const Place t = place<E>(p);
    if (!t.on) return;
    const TX *x = static_cast<const TX *>(p.x) + t.n * p.pixels * p.ldx + t.c;
    TY *y = static_cast<TY *>(p.y) + t.n * p.pixels * p.ldy + t.c;
    const Channels<E> k = channels<E>(p, t.n, t.c);
    with_activation(p.act, [&](auto act) {
#pragma unroll 4
        for (int64_t i = t.first + t.y; i < t.last; i += t.ty) {
            float v[E];
            load<E>(x + i * p.ldx, v);
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] = activate<act.value>(fmaf((v[e] - k.mean[e]) * k.rstd[e], k.w[e], k.b[e]));
            store<E>(y + i * p.ldy, v);
        }
    });
}

// Each channel's sums of dz and dz xh over a chunk of pixels.
template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(kThreads) sums_kernel(const Params p)
{
    __shared__ float2 all[E][kThreads];
    const Place t = place<E>(p);
    float2 s[E] = {};
    if (t.on) {
        const TX *x = static_cast<const TX *>(p.x) + t.n * p.pixels * p.ldx + t.c;
        const TY *dy = static_cast<const TY *>(p.dy) + t.n * p.pixels * p.ldy + t.c;
        const Channels<E> k = channels<E>(p, t.n, t.c);
        with_activation(p.act, [&](auto act) {
#pragma unroll 2
            for (int64_t i = t.first + t.y; i < t.last; i += t.ty) {
                float v[E], d[E];
                load<E>(x + i * p.ldx, v);
                load<E>(dy + i * p.ldy, d);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float xh = (v[e] - k.mean[e]) * k.rstd[e];
                    const float dz = before_activation<act.value>(d[e], v[e], xh, k.mean[e], k.rstd[e], k.w[e], k.b[e]);
                    s[e].x += dz;
                    s[e].y = fmaf(dz, xh, s[e].y);
                }
            }
        });
    }
#pragma unroll
    for (int e = 0; e < E; ++e) all[e][threadIdx.x] = s[e];
    for (int half = t.ty >> 1; half; half >>= 1) {
        __syncthreads();
        if (t.y < half)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                all[e][threadIdx.x].x += all[e][threadIdx.x + half * p.tx].x;
                all[e][threadIdx.x].y += all[e][threadIdx.x + half * p.tx].y;
            }
    }
    if (t.on && t.y == 0)
#pragma unroll
        for (int e = 0; e < E; ++e)
            p.part[((int64_t)t.n * p.chunks + t.chunk) * p.channels + t.c + e] = all[e][threadIdx.x];
}

// A sample's sums by channel over its chunks, and a group's means of t and t xh: a block per (n, g).
__global__ void __launch_bounds__(kThreads) means_kernel(const Params p)
{
    __shared__ float2 all[kThreads];
    amsim::chain_wait();
    const int n = blockIdx.x / p.groups, g = blockIdx.x % p.groups;
    float2 m = make_float2(0.0f, 0.0f);
    for (int i = threadIdx.x; i < p.size; i += kThreads) {
        const int c = g * p.size + i;
        float2 s = make_float2(0.0f, 0.0f);
        for (int k = 0; k < p.chunks; ++k) {
            const float2 v = p.part[((int64_t)n * p.chunks + k) * p.channels + c];
            s.x += v.x;
            s.y += v.y;
        }
        p.sums[(int64_t)n * p.channels + c] = s;
        const float w = p.w ? p.w[c] : 1.0f;
        m.x = fmaf(w, s.x, m.x);
        m.y = fmaf(w, s.y, m.y);
    }
    all[threadIdx.x] = m;
    for (int half = kThreads / 2; half; half >>= 1) {
        __syncthreads();
        if (threadIdx.x < half) {
            all[threadIdx.x].x += all[threadIdx.x + half].x;
            all[threadIdx.x].y += all[threadIdx.x + half].y;
        }
    }
    if (threadIdx.x == 0) {
        const float count = (float)p.size * (float)p.pixels;
        p.means[blockIdx.x] = make_float2(all[0].x / count, all[0].y / count);
    }
}

// dw and db from the samples' sums: a block takes 32 channels, its 32 warps every 32nd sample.
__global__ void __launch_bounds__(1024) weights_kernel(const Params p)
{
    __shared__ float2 part[32][33];
    amsim::chain_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + lane;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < p.channels)
        for (int n = warp; n < p.batch; n += 32) {
            const float2 v = p.sums[(int64_t)n * p.channels + c];
            s.x += v.x;
            s.y += v.y;
        }
    part[warp][lane] = s;
    __syncthreads();
    s = part[lane][warp];
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, d);
        s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, d);
    }
    const int mine = (int)blockIdx.x * 32 + warp;
    if (lane || mine >= p.channels) return;
    if (p.db) p.db[mine] = s.x;
    if (p.dw) p.dw[mine] = s.y;
}

template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(kThreads) gradient_kernel(const Params p)
{
    amsim::chain_wait();
    const Place t = place<E>(p);
    if (!t.on) return;
    const TX *x = static_cast<const TX *>(p.x) + t.n * p.pixels * p.ldx + t.c;
    const TY *dy = static_cast<const TY *>(p.dy) + t.n * p.pixels * p.ldy + t.c;
    TX *dx = static_cast<TX *>(p.dx) + t.n * p.pixels * p.lddx + t.c;
    const Channels<E> k = channels<E>(p, t.n, t.c);
    float2 m[E];
#pragma unroll
    for (int e = 0; e < E; ++e) m[e] = p.means[(int64_t)t.n * p.groups + (t.c + e) / p.size];
    with_activation(p.act, [&](auto act) {
#pragma unroll 2
        for (int64_t i = t.first + t.y; i < t.last; i += t.ty) {
            float v[E], d[E];
            load<E>(x + i * p.ldx, v);
            load<E>(dy + i * p.ldy, d);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float xh = (v[e] - k.mean[e]) * k.rstd[e];
                const float dz = before_activation<act.value>(d[e], v[e], xh, k.mean[e], k.rstd[e], k.w[e], k.b[e]);
                v[e] = k.rstd[e] * (fmaf(dz, k.w[e], -m[e].x) - xh * m[e].y);
            }
            store<E>(dx + i * p.lddx, v);
        }
    });
}

// ------------------------------------------------------------------ resident slabs
constexpr int kSlabThreads = 256, kSlabBlocks = 2;       // blocks: of an SM
constexpr int kSlabGroups = 64;              // at most: 128 bytes of bf16 channels, a group each

__device__ __forceinline__ uint32_t shared_address(const void *q)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(q));
}
// BYTES from global to this thread's own slot; done after copies_wait.
template <int BYTES>
__device__ __forceinline__ void copy_in(uint8_t *to, const void *from)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared_address(to)), "l"(from) : "memory");
    else if constexpr (BYTES >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(shared_address(to)), "l"(from), "n"(BYTES)
                     : "memory");
    else
        *reinterpret_cast<uint16_t *>(to) = *static_cast<const uint16_t *>(from);
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// No block leaves while another reads its sums: it says that it has read, and
// waits at its end for all to have said so.  Nothing it wrote is handed over,
// so its stores are not waited for.
__device__ __forceinline__ void cluster_has_read() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_leave() { asm volatile("barrier.cluster.wait;" ::: "memory"); }
// A float2 of block `rank` of the cluster at the place of this block's `q`.
__device__ __forceinline__ float2 of_rank(const float2 *q, int rank)
{
    uint32_t at;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(shared_address(q)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

// A thread's part of a slab: the channels of one piece, every `step`-th pixel
// of the block's from `first` on.
struct Part {
    int n, c0, channels, groups;             // sample, first channel, channels and groups of the slab
    int rank, wide, piece, row, step;        // wide: pieces of a pixel
    int64_t first;                           // the block's first pixel
    int rows, count;                         // the block's pixels, this thread's
};
template <int E>
__device__ __forceinline__ Part part_of(const Params &p)
{
    Part t;
    unsigned unit;
    asm("mov.u32 %0, %%clusterid.x;" : "=r"(unit));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(t.rank));
    t.n = (int)(unit / (unsigned)p.slabs);
    t.c0 = (int)(unit - (unsigned)t.n * (unsigned)p.slabs) * p.slab;
    t.channels = p.slab;
    t.groups = p.slab_groups;
    t.step = p.step;
    if (t.c0 + p.slab > p.channels) {        // the last slab is narrower
        t.channels = p.channels - t.c0;
        t.groups = t.channels / p.size;
        t.step = kSlabThreads / (t.channels / E);
    }
    t.wide = t.channels / E;
    t.row = (int)(threadIdx.x / (unsigned)t.wide);
    t.piece = (int)threadIdx.x - t.row * t.wide;
    t.first = (int64_t)t.rank * p.rows;
    t.rows = (int)max((int64_t)0, min((int64_t)p.rows, p.pixels - t.first));
    t.count = t.row < t.step ? (int)((unsigned)max(0, t.rows - t.row + t.step - 1) / (unsigned)t.step) : 0;
    return t;
}

// Packed arithmetic on a piece's values, two an instruction.
template <int E>
struct Values {
    float2 v[(E + 1) / 2];
};
template <int E, typename F>
__device__ __forceinline__ void each_pair(F use)
{
#pragma unroll
    for (int i = 0; i < (E + 1) / 2; ++i) use(i);
}
template <int E, typename T>
__device__ __forceinline__ Values<E> take(const void *slot)
{
    float f[E];
    load<E>(static_cast<const T *>(slot), f);
    Values<E> r;
    each_pair<E>([&](int i) { r.v[i] = make_float2(f[2 * i], 2 * i + 1 < E ? f[2 * i + 1 < E ? 2 * i + 1 : 0] : 0.0f); });
    return r;
}
template <int E, typename T>
__device__ __forceinline__ void put(T *at, const Values<E> &r)
{
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = e & 1 ? r.v[e >> 1].y : r.v[e >> 1].x;
    store<E>(at, f);
}

using amsim::add2;
using amsim::both;
using amsim::fma2;
using amsim::mul2;

__device__ __forceinline__ float2 sigmoid2(float2 z)
{
    const float2 t = mul2(z, both(kMinusLog2E));
    const float2 d = add2(make_float2(power_of_2(t.x), power_of_2(t.y)), both(1.0f));
    return make_float2(reciprocal(d.x), reciprocal(d.y));
}
template <int ACT>
__device__ __forceinline__ float2 activate2(float2 z)
{
    if (ACT == AMSIM_ACT_SILU) return mul2(z, sigmoid2(z));
    return make_float2(activate<ACT>(z.x), activate<ACT>(z.y));
}
// before_activation of a pair.
template <int ACT>
__device__ __forceinline__ float2 before2(float2 dy, float2 x, float2 xh, float mean, float rstd, float2 w, float2 b)
{
    if (ACT == AMSIM_ACT_NONE) return dy;
    if (ACT == AMSIM_ACT_RELU)
        return make_float2(before_activation<ACT>(dy.x, x.x, xh.x, mean, rstd, w.x, b.x),
                           before_activation<ACT>(dy.y, x.y, xh.y, mean, rstd, w.y, b.y));
    const float2 z = fma2(xh, w, b), s = sigmoid2(z);
    return mul2(mul2(dy, s), fma2(z, fma2(s, both(-1.0f), both(1.0f)), both(1.0f)));
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// The copies are told apart in two halves, so that a thread sums what has
// arrived while the rest is on its way.
template <typename F>
__device__ __forceinline__ void in_halves(int count, F use)
{
    const int half = (count + 1) >> 1;
    copies_wait<1>();
#pragma unroll 4
    for (int i = 0; i < half; ++i) use(i);
    copies_wait<0>();
#pragma unroll 4
    for (int i = half; i < count; ++i) use(i);
}

// Dynamic shared memory: the slots [steps][threads] of x (then of dy), then
// (backward) sums by channel.  A piece lies within one group.
template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(kSlabThreads, kSlabBlocks) slab_forward_kernel(const Params p)
{
    extern __shared__ __align__(16) uint8_t slots[];
    __shared__ Moments all[kSlabThreads];
    __shared__ float2 found[kSlabGroups], stats[kSlabGroups];
    constexpr int bytes = E * (int)sizeof(TX);
    const Part t = part_of<E>(p);
    const int c = t.c0 + t.piece * E, mine = t.piece * E / p.size, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t pixel = t.n * p.pixels + t.first + t.row;
    uint8_t *slot = slots + threadIdx.x * bytes;
    {
        const TX *x = static_cast<const TX *>(p.x) + pixel * p.ldx + c;
        const int64_t far = (int64_t)t.step * p.ldx;
        const int half = (t.count + 1) >> 1;
#pragma unroll 4
        for (int i = 0; i < half; ++i) copy_in<bytes>(slot + i * (kSlabThreads * bytes), x + i * far);
        copies_commit();
#pragma unroll 4
        for (int i = half; i < t.count; ++i) copy_in<bytes>(slot + i * (kSlabThreads * bytes), x + i * far);
        copies_commit();
    }
    // Sums about the thread's first value: what cancels is no larger than the
    // values' own spread.
    float2 s1 = both(0.0f), s2 = both(0.0f);
    float about = 0.0f;
    in_halves(t.count, [&](int i) {
        const Values<E> r = take<E, TX>(slot + i * (kSlabThreads * bytes));
        if (i == 0) about = r.v[0].x;
        each_pair<E>([&](int j) {
            float2 d = add2(r.v[j], both(-about));
            if (E == 1) d.y = 0.0f;
            s1 = add2(s1, d);
            s2 = fma2(d, d, s2);
        });
    });
    {
        const float n = (float)(t.count * E), sum = s1.x + s1.y, m = t.count ? sum / n : 0.0f;
        all[threadIdx.x] = Moments{n, about + m, fmaxf((s2.x + s2.y) - sum * m, 0.0f)};
    }
    __syncthreads();
    // a warp per group joins its threads: pieces side by side, then rows
    const int wide = p.size / E, threads = wide * t.step;
    for (int g = warp; g < t.groups; g += kSlabThreads / 32) {
        Moments m{0.0f, 0.0f, 0.0f};
        for (int i = lane; i < threads; i += 32) {
            const int row = (int)((unsigned)i / (unsigned)wide);
            m = join(m, all[row * t.wide + g * wide + (i - row * wide)]);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1)
            m = join(m, Moments{__shfl_down_sync(0xFFFFFFFFu, m.n, d), __shfl_down_sync(0xFFFFFFFFu, m.mean, d),
                                __shfl_down_sync(0xFFFFFFFFu, m.m2, d)});
        if (lane == 0) found[g] = make_float2(m.mean, m.m2);
    }
    if (p.cluster > 1)
        cluster_barrier();
    else
        __syncthreads();
    for (int g = threadIdx.x; g < t.groups; g += kSlabThreads) {
        Moments m{0.0f, 0.0f, 0.0f};
        for (int r = 0; r < p.cluster; ++r) {
            const float2 f = p.cluster > 1 ? of_rank(&found[g], r) : found[g];
            const int64_t rows = max((int64_t)0, min((int64_t)p.rows, p.pixels - (int64_t)r * p.rows));
            m = join(m, Moments{(float)rows * (float)p.size, f.x, f.y});
        }
        const float2 f = make_float2(m.mean, 1.0f / sqrtf(m.m2 / m.n + p.eps));
        stats[g] = f;
        if (t.rank == 0) {
            const int64_t at = (int64_t)t.n * p.groups + t.c0 / p.size + g;
            p.mean[at] = f.x;
            p.rstd[at] = f.y;
        }
    }
    __syncthreads();
    if (p.cluster > 1) cluster_has_read();
    const float2 f = stats[mine];
    float2 w[(E + 1) / 2], b[(E + 1) / 2];
    each_pair<E>([&](int j) {
        const bool two = 2 * j + 1 < E;
        w[j] = p.w ? make_float2(p.w[c + 2 * j], two ? p.w[c + 2 * j + two] : 0.0f) : both(1.0f);
        b[j] = p.b ? make_float2(p.b[c + 2 * j], two ? p.b[c + 2 * j + two] : 0.0f) : both(0.0f);
        // z = x (rstd w) + (b - mean rstd w): what this rounds is of the size of what the mean's rounding leaves
        w[j] = mul2(w[j], both(f.y));
        b[j] = fma2(w[j], both(-f.x), b[j]);
    });
    TY *y = static_cast<TY *>(p.y) + pixel * p.ldy + c;
    const int64_t far = (int64_t)t.step * p.ldy;
    with_activation(p.act, [&](auto act) {
#pragma unroll 4
        for (int i = 0; i < t.count; ++i) {
            Values<E> r = take<E, TX>(slot + i * (kSlabThreads * bytes));
            each_pair<E>([&](int j) { r.v[j] = activate2<act.value>(fma2(r.v[j], w[j], b[j])); });
            put<E>(y + i * far, r);
        }
    });
    if (p.cluster > 1) cluster_leave();
}

template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(kSlabThreads, kSlabBlocks) slab_backward_kernel(const Params p)
{
    extern __shared__ __align__(16) uint8_t slots[];
    __shared__ float2 sums[E][kSlabThreads], means[kSlabGroups];
    constexpr int xb = E * (int)sizeof(TX), yb = E * (int)sizeof(TY);
    // fp32 slots of x and dy give their places to xh and dz, so that these are computed once
    constexpr bool kKeepY = sizeof(TY) == 4, kKeepX = kKeepY && sizeof(TX) == 4;
    const Part t = part_of<E>(p);
    const int c = t.c0 + t.piece * E, mine = t.piece * E / p.size, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t pixel = t.n * p.pixels + t.first + t.row;
    uint8_t *sx = slots + threadIdx.x * xb, *sy = slots + p.steps * (kSlabThreads * xb) + threadIdx.x * yb;
    float2 *by_channel = reinterpret_cast<float2 *>(slots + p.steps * (kSlabThreads * (xb + yb)));
    {
        const TX *x = static_cast<const TX *>(p.x) + pixel * p.ldx + c;
        const TY *dy = static_cast<const TY *>(p.dy) + pixel * p.ldy + c;
        const int64_t xfar = (int64_t)t.step * p.ldx, yfar = (int64_t)t.step * p.ldy;
        auto copy = [&](int from, int to) {
#pragma unroll 4
            for (int i = from; i < to; ++i) {
                copy_in<xb>(sx + i * (kSlabThreads * xb), x + i * xfar);
                copy_in<yb>(sy + i * (kSlabThreads * yb), dy + i * yfar);
            }
            copies_commit();
        };
        copy(0, (t.count + 1) >> 1);
        copy((t.count + 1) >> 1, t.count);
    }
    const int64_t group = (int64_t)t.n * p.groups + t.c0 / p.size + mine;
    const float mean = p.mean[group], rstd = p.rstd[group];
    float2 w[(E + 1) / 2], b[(E + 1) / 2];
    each_pair<E>([&](int j) {
        const bool two = 2 * j + 1 < E;
        w[j] = p.w ? make_float2(p.w[c + 2 * j], two ? p.w[c + 2 * j + two] : 0.0f) : both(1.0f);
        b[j] = p.b ? make_float2(p.b[c + 2 * j], two ? p.b[c + 2 * j + two] : 0.0f) : both(0.0f);
    });
    auto values = [&](auto act, int i, Values<E> &xh, Values<E> &dz) {
        const Values<E> x = take<E, TX>(sx + i * (kSlabThreads * xb));
        dz = take<E, TY>(sy + i * (kSlabThreads * yb));
        each_pair<E>([&](int j) {
            xh.v[j] = mul2(add2(x.v[j], both(-mean)), both(rstd));
            dz.v[j] = before2<act.value>(dz.v[j], x.v[j], xh.v[j], mean, rstd, w[j], b[j]);
        });
    };
    float2 s[(E + 1) / 2], q[(E + 1) / 2];
    each_pair<E>([&](int j) { s[j] = q[j] = both(0.0f); });
    with_activation(p.act, [&](auto act) {
        in_halves(t.count, [&](int i) {
            Values<E> xh, dz;
            values(act, i, xh, dz);
            if (kKeepX) put<E>(reinterpret_cast<TX *>(sx + i * (kSlabThreads * xb)), xh);
            if (kKeepY) put<E>(reinterpret_cast<TY *>(sy + i * (kSlabThreads * yb)), dz);
            each_pair<E>([&](int j) {
                s[j] = add2(s[j], dz.v[j]);
                q[j] = fma2(dz.v[j], xh.v[j], q[j]);
            });
        });
    });
    // over the rows of threads, in a fixed order: where a warp holds whole rows
    // across its lanes first, then rows (or warps) across shared memory
    int rows = t.step, row = t.row, apart = t.wide;
    if (32 % t.wide == 0) {
        for (int d = t.wide; d < 32; d <<= 1)
            each_pair<E>([&](int j) {
                s[j] = add2(s[j], make_float2(__shfl_xor_sync(0xFFFFFFFFu, s[j].x, d),
                                              __shfl_xor_sync(0xFFFFFFFFu, s[j].y, d)));
                q[j] = add2(q[j], make_float2(__shfl_xor_sync(0xFFFFFFFFu, q[j].x, d),
                                              __shfl_xor_sync(0xFFFFFFFFu, q[j].y, d)));
            });
        rows = kSlabThreads / 32;
        row = lane < t.wide ? warp : rows;
        apart = 32;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        sums[e][threadIdx.x] = e & 1 ? make_float2(s[e >> 1].y, q[e >> 1].y) : make_float2(s[e >> 1].x, q[e >> 1].x);
    while (rows > 1) {
        const int half = (rows + 1) >> 1;
        __syncthreads();
        if (row + half < rows)
#pragma unroll
            for (int e = 0; e < E; ++e)
                sums[e][threadIdx.x] = add2(sums[e][threadIdx.x], sums[e][threadIdx.x + half * apart]);
        rows = half;
    }
    if (row == 0)
#pragma unroll
        for (int e = 0; e < E; ++e) by_channel[t.piece * E + e] = sums[e][threadIdx.x];
    if (p.cluster > 1)
        cluster_barrier();
    else
        __syncthreads();
    // the slab's sums by channel, over its blocks in their order; the group's means from them
    for (int g = warp; g < t.groups; g += kSlabThreads / 32) {
        float2 m = both(0.0f);
        for (int i = lane; i < p.size; i += 32) {
            const int at = g * p.size + i;
            float2 v = both(0.0f);
            if (p.cluster > 1)
                for (int r = 0; r < p.cluster; ++r) v = add2(v, of_rank(&by_channel[at], r));
            else
                v = by_channel[at];
            if (t.rank == 0) p.sums[(int64_t)t.n * p.channels + t.c0 + at] = v;
            m = fma2(v, both(p.w ? p.w[t.c0 + at] : 1.0f), m);
        }
        m.x = warp_sum(m.x);
        m.y = warp_sum(m.y);
        const float count = (float)p.size * (float)p.pixels;
        if (lane == 0) means[g] = make_float2(m.x / count, m.y / count);
    }
    __syncthreads();
    if (p.cluster > 1) cluster_has_read();
    // dx = dz (w rstd) - mean(t) rstd - xh (mean(t xh) rstd)
    const float2 m = mul2(means[mine], both(-rstd));
    each_pair<E>([&](int j) { s[j] = mul2(w[j], both(rstd)); });
    TX *dx = static_cast<TX *>(p.dx) + pixel * p.lddx + c;
    const int64_t far = (int64_t)t.step * p.lddx;
    auto finish = [&](auto act) {
#pragma unroll 4
        for (int i = 0; i < t.count; ++i) {
            Values<E> xh, dz;
            if (kKeepY) {
                xh = take<E, TX>(sx + i * (kSlabThreads * xb));
                dz = take<E, TY>(sy + i * (kSlabThreads * yb));
                if (!kKeepX) each_pair<E>([&](int j) { xh.v[j] = mul2(add2(xh.v[j], both(-mean)), both(rstd)); });
            } else {
                values(act, i, xh, dz);
            }
            each_pair<E>([&](int j) { dz.v[j] = fma2(xh.v[j], both(m.y), fma2(dz.v[j], s[j], both(m.x))); });
            put<E>(dx + i * far, dz);
        }
    };
    if (kKeepY)
        finish(Act<AMSIM_ACT_NONE>{});
    else
        with_activation(p.act, finish);
    if (p.cluster > 1) cluster_leave();
}

size_t type_size(int t) { return t == AMSIM_BF16 ? 2 : 4; }
bool aligned(const void *q, size_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }

int check(const amsim_group_norm_desc *d)
{
    if (!d || d->batch < 0 || d->pixels < 0 || d->channels < 1 || d->groups < 1 || d->channels % d->groups)
        return AMSIM_EINVAL;
    // a block for each sample and tile of at least 32 channels, or group, fits a grid
    if (d->batch > 0x7FFFFFFF || d->pixels > (int64_t)1 << 40 || d->channels > 1 << 24 ||
        d->batch * std::max<int64_t>(d->groups, (d->channels + 31) / 32) > 0x7FFFFFFF)
        return AMSIM_EINVAL;
    for (int t : {d->x_type, d->y_type})
        if (t != AMSIM_F32 && t != AMSIM_BF16) return AMSIM_EINVAL;
    for (int64_t ld : {d->ldx, d->ldy, d->lddx})
        if (ld != 0 && (ld < d->channels || ld > (int64_t)1 << 40)) return AMSIM_EINVAL;
    if (d->activation < AMSIM_ACT_NONE || d->activation > AMSIM_ACT_SILU) return AMSIM_EINVAL;
    return std::isfinite(d->eps) && d->eps >= 0.0f ? AMSIM_OK : AMSIM_EINVAL;
}

int device_sms()
{
    int sms = 0;
    return amsim::current_device(&sms) < 0 ? 0 : sms;
}

// Elements of a thread's piece: 16 bytes of the wider type, where every row of them is on its size.
int piece(const amsim_group_norm_desc *d)
{
    return d->x_type == AMSIM_BF16 && d->y_type == AMSIM_BF16 ? 8 : 4;
}
bool whole(const void *q, int64_t ld, size_t size, int E) { return aligned(q, E * size) && ld % E == 0; }

// Chunks of pixels: about eight blocks an SM, no chunk below 64 pixels.
void split(Params &p, int E, int sms)
{
    p.tx = 1;
    while (p.tx < 32 && p.tx * E < p.channels) p.tx *= 2;
    p.tiles = (p.channels + p.tx * E - 1) / (p.tx * E);
    int64_t chunks = std::max<int64_t>(1, (int64_t)sms * 8 / ((int64_t)p.tiles * std::max(1, p.batch)));
    chunks = std::min(chunks, std::max<int64_t>(1, p.pixels / 64));
    p.chunk = std::max<int64_t>(1, (p.pixels + chunks - 1) / chunks);
    p.chunks = (int)std::max<int64_t>(1, (p.pixels + p.chunk - 1) / p.chunk);
}

// The resident way's shape, or false.  A slab is some 128 bytes of a pixel, in
// whole groups; its cluster has as many blocks as hold it, and more where the
// machine is not full and threads keep four pixels.  A slab that is too large
// for eight blocks of which an SM takes two is taken narrower, or in larger blocks.
constexpr int kHalfSm = 96 * 1024, kWholeSm = 200 * 1024;
constexpr int kMaxCluster = 8;
constexpr int kSums = 8;                     // bytes of a channel's sums, backward
// E: of a piece; bytes: of an element on chip (x; backward x and dy); chan: of a channel's sums there
bool resident(Params &p, int E, int bytes, int chan, int sms)
{
    struct Try {
        int width, room;
    };
    for (const Try t : {Try{128, kHalfSm}, Try{64, kHalfSm}, Try{64, kWholeSm}, Try{32, kWholeSm}}) {
        p.slab = std::min(p.channels, std::max(1, t.width / (bytes * p.size)) * p.size);
        if (p.slab / E > kSlabThreads || p.slab / p.size > kSlabGroups) continue;
        p.slab_groups = p.slab / p.size;
        p.slabs = (p.channels + p.slab - 1) / p.slab;
        const int step = p.step = kSlabThreads / (p.slab / E), most = (t.room - p.slab * chan) / (kSlabThreads * E * bytes);
        if (most < 1) continue;
        const int64_t need = (p.pixels + (int64_t)step * most - 1) / ((int64_t)step * most);
        if (need > kMaxCluster) continue;
        const int64_t units = (int64_t)p.batch * p.slabs;
        const int64_t fill = std::min((2 * (int64_t)sms + units - 1) / units, p.pixels / (4 * step));
        p.cluster = (int)std::max<int64_t>(need, std::min<int64_t>(kMaxCluster, fill));
        while (p.cluster > need && (p.cluster & (p.cluster - 1))) --p.cluster;
        p.rows = (int)((p.pixels + p.cluster - 1) / p.cluster);
        p.steps = (p.rows + step - 1) / step;
        if (units * p.cluster <= 0x7FFFFFFF) return true;
    }
    return false;
}

Params params(const amsim_group_norm_desc *d)
{
    Params p{};
    p.pixels = d->pixels;
    p.batch = (int)d->batch;
    p.channels = d->channels;
    p.groups = d->groups;
    p.size = d->channels / d->groups;
    p.ldx = d->ldx ? d->ldx : d->channels;
    p.ldy = d->ldy ? d->ldy : d->channels;
    p.lddx = d->lddx ? d->lddx : d->channels;
    p.act = d->activation;
    p.eps = d->eps;
    return p;
}

dim3 grid(const Params &p) { return dim3((unsigned)((int64_t)p.batch * p.tiles * p.chunks)); }

int start(bool chained, void (*kernel)(Params), dim3 grid, int threads, const Params &p, cudaStream_t st)
{
    const int rc = amsim::cuda_status(amsim::chain_launch(chained, kernel, grid, dim3((unsigned)threads), 0, st, p));
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}

int start_slabs(void (*kernel)(Params), const Params &p, int bytes, int chan, cudaStream_t st)
{
    int rc = amsim::cuda_status(
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWholeSm));
    if (!rc && p.cluster > 8)
        rc = amsim::cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    if (rc) return rc;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)((int64_t)p.batch * p.slabs * p.cluster));
    c.blockDim = dim3(kSlabThreads);
    c.dynamicSmemBytes = (size_t)p.steps * kSlabThreads * bytes + (size_t)p.slab * chan;
    c.stream = st;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = (unsigned)p.cluster;
    a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
    c.attrs = a;
    c.numAttrs = p.cluster > 1 ? 1 : 0;
    rc = amsim::cuda_status(cudaLaunchKernelEx(&c, kernel, p));
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}

template <typename TX, typename TY, int E>
int slab_pass(bool fwd, const Params &p, cudaStream_t st)
{
    if (fwd) return start_slabs(slab_forward_kernel<TX, TY, E>, p, E * (int)sizeof(TX), 0, st);
    const int rc = start_slabs(slab_backward_kernel<TX, TY, E>, p, E * (int)(sizeof(TX) + sizeof(TY)), kSums, st);
    if (rc || (!p.dw && !p.db)) return rc;
    return start(true, weights_kernel, dim3((unsigned)((p.channels + 31) / 32)), 1024, p, st);
}

template <typename TX, typename TY, int E>
int wide_pass(bool fwd, const Params &p, cudaStream_t st)
{
    if (fwd) {
        if (int rc = start(false, moments_kernel<TX, E>, grid(p), kThreads, p, st)) return rc;
        if (int rc = start(true, join_kernel, dim3((unsigned)(p.batch * p.groups)), kThreads, p, st)) return rc;
        return start(true, apply_kernel<TX, TY, E>, grid(p), kThreads, p, st);
    }
    if (int rc = start(false, sums_kernel<TX, TY, E>, grid(p), kThreads, p, st)) return rc;
    if (int rc = start(true, means_kernel, dim3((unsigned)(p.batch * p.groups)), kThreads, p, st)) return rc;
    if (int rc = start(true, gradient_kernel<TX, TY, E>, grid(p), kThreads, p, st)) return rc;
    if (!p.dw && !p.db) return AMSIM_OK;
    return start(false, weights_kernel, dim3((unsigned)((p.channels + 31) / 32)), 1024, p, st);
}

template <typename TX, typename TY>
int pass(bool fwd, int E, const Params &p, cudaStream_t st)
{
    constexpr int most = sizeof(TX) + sizeof(TY) == 4 ? 8 : 4;   // 16 bytes of the wider type
    if (p.cluster)
        return E == 4   ? slab_pass<TX, TY, 4>(fwd, p, st)
               : E == 2 ? slab_pass<TX, TY, 2>(fwd, p, st)
                        : slab_pass<TX, TY, 1>(fwd, p, st);
    return E == most ? wide_pass<TX, TY, most>(fwd, p, st) : wide_pass<TX, TY, 1>(fwd, p, st);
}

// The way a call goes: slabs in pieces of up to four channels that lie within
// one group, else whole pieces of 16 bytes, or single channels.  `fits(E)`: the
// call's rows are on E elements.
template <typename F>
int plan(const amsim_group_norm_desc *d, bool fwd, int sms, Params &p, F fits)
{
    const int bytes = (int)(type_size(d->x_type) + (fwd ? 0 : type_size(d->y_type)));
    int E = 4;
    while (E > 1 && (p.size % E || !fits(E))) E /= 2;
    if (resident(p, E, bytes, fwd ? 0 : kSums, sms)) return E;
    p.cluster = 0;
    E = piece(d);
    if (d->channels % E || !fits(E)) E = 1;
    split(p, E, sms);
    return E;
}

int run(const amsim_group_norm_desc *d, bool fwd, int E, const Params &p, cudaStream_t st)
{
    using B = __nv_bfloat16;
    if (d->x_type == AMSIM_F32)
        return d->y_type == AMSIM_F32 ? pass<float, float>(fwd, E, p, st) : pass<float, B>(fwd, E, p, st);
    return d->y_type == AMSIM_F32 ? pass<B, float>(fwd, E, p, st) : pass<B, B>(fwd, E, p, st);
}
}  // namespace

extern "C" size_t amsim_group_norm_workspace_size(const amsim_group_norm_desc *d, int which)
{
    if (check(d) || which < 0 || which > 1 || !d->batch || !d->pixels) return 0;
    const int sms = device_sms();
    Params p = params(d);
    size_t most = 0;
    for (int on : {1, 2, 4, 8}) {                // the calls' pointers and strides decide which
        plan(d, !which, sms ? sms : 1, p, [&](int E) { return E <= on; });
        if (!p.cluster) most = std::max(most, (size_t)p.batch * p.chunks * p.channels);
    }
    return (most + (which ? (size_t)p.batch * (p.channels + p.groups) : 0)) * sizeof(float2);
}

extern "C" int amsim_group_norm_fwd(const amsim_group_norm_desc *d, const void *x, const float *w, const float *b,
                                    void *y, float *mean, float *rstd, void *ws, size_t ws_bytes,
                                    amsim_stream_t stream)
{
    if (const int rc = check(d)) return rc;
    if (!d->batch) return AMSIM_OK;
    if (!mean || !rstd || (d->pixels && (!x || !y))) return AMSIM_EINVAL;
    const size_t xs = type_size(d->x_type), ys = type_size(d->y_type);
    if (!aligned(x, xs) || !aligned(y, ys) || !aligned(ws, 8)) return AMSIM_EINVAL;
    for (const float *f : {w, b, (const float *)mean, (const float *)rstd})
        if (!aligned(f, 4)) return AMSIM_EINVAL;
    const size_t need = d->pixels ? amsim_group_norm_workspace_size(d, 0) : 0;
    if (need && (!ws || ws_bytes < need)) return AMSIM_EINVAL;
    Params p = params(d);
    p.x = x;
    p.y = y;
    p.w = w;
    p.b = b;
    p.mean = mean;
    p.rstd = rstd;
    p.part = static_cast<float2 *>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    if (!d->pixels) return start(false, join_kernel, dim3((unsigned)(p.batch * p.groups)), kThreads, p, st);
    const int E = plan(d, true, sms, p, [&](int n) { return whole(x, p.ldx, xs, n) && whole(y, p.ldy, ys, n); });
    return run(d, true, E, p, st);
}

extern "C" int amsim_group_norm_bwd(const amsim_group_norm_desc *d, const void *dy, const void *x, const float *w,
                                    const float *b, const float *mean, const float *rstd, void *dx, float *dw,
                                    float *db, void *ws, size_t ws_bytes, amsim_stream_t stream)
{
    if (const int rc = check(d)) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t xs = type_size(d->x_type), ys = type_size(d->y_type);
    if (!aligned(x, xs) || !aligned(dx, xs) || !aligned(dy, ys) || !aligned(ws, 8)) return AMSIM_EINVAL;
    for (const float *f : {w, b, mean, rstd, (const float *)dw, (const float *)db})
        if (!aligned(f, 4)) return AMSIM_EINVAL;
    if (!d->batch || !d->pixels) {
        for (float *f : {dw, db})
            if (f && cudaMemsetAsync(f, 0, (size_t)d->channels * 4, st) != cudaSuccess) {
                cudaGetLastError();
                return AMSIM_ECUDA;
            }
        return AMSIM_OK;
    }
    if (!x || !dy || !dx || !mean || !rstd || !ws || ws_bytes < amsim_group_norm_workspace_size(d, 1))
        return AMSIM_EINVAL;
    Params p = params(d);
    p.x = x;
    p.dy = dy;
    p.dx = dx;
    p.w = w;
    p.b = b;
    p.mean = const_cast<float *>(mean);
    p.rstd = const_cast<float *>(rstd);
    p.dw = dw;
    p.db = db;
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    const int E = plan(d, false, sms, p, [&](int n) {
        return whole(x, p.ldx, xs, n) && whole(dx, p.lddx, xs, n) && whole(dy, p.ldy, ys, n);
    });
    p.sums = static_cast<float2 *>(ws);
    p.means = p.sums + (size_t)p.batch * p.channels;
    p.part = p.means + (size_t)p.batch * p.groups;
    return run(d, false, E, p, st);
}
