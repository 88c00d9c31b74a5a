// The group norm with its activation, channels last, and its gradients.
//
// x is needed twice, for the statistics and for the result; what has to move is
// one reading.  So the results of a tile follow its statistics some 32 MB behind,
// and find x (and dy) in the L2 cache.  Both are blocks of one launch, whose order
// is that in which they start: a block takes the next number, the even ones of a
// pair work out results, the odd ones the statistics that come 32 MB later.  A
// block of results waits until all of its tile's statistics are there, which
// blocks that started before it work on; these wait for nothing.  Statistics are
// joined by whoever needs them, in a fixed order.  64 x 56 x 56 x 256 fp32
// backward takes 142 us, 0.65 of a plain copy's rate, and reads 421 of 411 MB; with a launch
// for each wave it took 159 us, with slabs kept in a cluster's shared memory 154 us.  Neither
// memory (55 %) nor the issue slots (36 %) are full, with 22 warps an SM.  8 x 128 x 128 x 512 bf16
// forward takes 74 us, 0.54.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>

#include "amsim_internal.h"
#include "chained.cuh"
#include "pairs.cuh"

namespace {

using amsim::add2;
using amsim::both;
using amsim::fma2;
using amsim::mul2;

// Quotients by a number that the host knows: a product's upper half (exact for
// dividends below 2^31: the multiplier is the next whole number above 2^(32 + shift) / d).
struct Divisor {
    unsigned d, mul, shift;
    __device__ __forceinline__ unsigned operator()(unsigned n) const
    {
        return d == 1 ? n : __umulhi(n, mul) >> shift;
    }
};
Divisor divisor(unsigned d)
{
    Divisor r{d, 0, 0};
    if (d == 1) return r;
    while ((1ull << (r.shift + 1)) < d) ++r.shift;
    r.mul = (unsigned)(((1ull << (32 + r.shift)) + d - 1) / d);
    return r;
}

// The waits that gave up, and after how long.
__device__ unsigned int g_wait_timeouts;
__device__ long long g_wait_limit_ns = 2000000000LL;
int wait_status(unsigned int *bits, int clear)
{
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) return AMSIM_ECUDA;
    *bits |= v;
    if (clear && v) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(zero)) != cudaSuccess) return AMSIM_ECUDA;
    }
    return AMSIM_OK;
}
int wait_limit(long long ns)
{
    return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns)) == cudaSuccess ? AMSIM_OK : AMSIM_ECUDA;
}
[[maybe_unused]] const bool g_wait_words = amsim::register_wait_words(&wait_status, &wait_limit);

struct Params {
    const void *x, *dy;
    const float *w, *b;
    void *y, *dx;
    float *mean, *rstd, *dw, *db;
    // scratch: of each sample's chunk of pixels, per part of a group (mean, sum of
    // squares about it; backward the sums of dz w and dz w xh), per channel (dz, dz xh)
    float2 *by_part, *by_channel;
    int64_t pixels, ldx, ldy, lddx, samples_chunks;
    int channels, groups, size;              // size: channels of a group
    int act;
    float eps;
    // A tile is some channels of a sample: whole groups, or (splits > 1) a part of one.
    int tile, tiles, splits, chunks, rows;   // tile: channels; rows: pixels of a chunk
    int step, vec;                           // pixels of a block at once; w and b on 16 bytes
    int whole;                               // a block has all of its tile's pixels, and does both parts
    Divisor by_tiles, by_splits, by_chunks, by_wide, by_step, by_group_wide, by_size;
    Divisor by_pair;                         // of 2 chunks
    unsigned units, lag;                     // tiles of all samples; how many the results are behind
    unsigned *next, *ready;                  // the next block's number; statistics of a tile (or group) that are there
};

constexpr int kThreads = 256;
constexpr int kTileGroups = 128;             // at most

template <typename T, int E>
struct alignas(sizeof(T) * E) Vec {
    T e[E];
};
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float v, float *o) { *o = v; }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(v); }

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

// Whether z > 0, in 64 bits.  Not inlined: the few calls that need it branch to
// it, and no other pays for 64-bit arithmetic, which this machine does slowly.
__device__ __noinline__ bool above_zero(float x, float mean, float rstd, float w, float b)
{
    return ((double)x - (double)mean) * (double)rstd * (double)w + (double)b > 0.0;
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
        if (fabsf(z) <= 0x1p-21f * (fabsf(xh * w) + fabsf(b))) on = above_zero(x, mean, rstd, w, b);
        return on ? dy : 0.0f;
    }
    const float s = sigmoid(z);
    return dy * (s * fmaf(z, 1.0f - s, 1.0f));
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
__device__ __forceinline__ void put(T *at, const Values<E> &r)
{
    if constexpr (sizeof(T) == 2 && E > 1) {     // a pair's rounding is one instruction
        Vec<__nv_bfloat162, E / 2> v;
        each_pair<E>([&](int j) { v.e[j] = __float22bfloat162_rn(r.v[j]); });
        *reinterpret_cast<Vec<__nv_bfloat162, E / 2> *>(at) = v;
    } else {
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = e & 1 ? r.v[e >> 1].y : r.v[e >> 1].x;
        store<E>(at, f);
    }
}

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

// A block's part: a role, a tile of a sample, a chunk of its pixels; a thread's
// part of that: the channels of one piece, which lies within one group, and
// every step-th pixel.
struct Part {
    bool stats;
    unsigned unit;
    int n, chunk, c0, channels, groups;      // the tile's first channel, channels, groups (1: a part of one)
    int group, split;                        // its first group, and which part of it
    int wide, piece, row, step, count;       // pieces of a pixel; this thread's, its first pixel, how many
    int mine;                                // its piece's group in the tile
    int64_t first;                           // the chunk's first pixel in the sample
    int rows;                                // and its pixels
};
template <int E, bool WHOLE>
__device__ __forceinline__ Part part_of(const Params &p, unsigned number)
{
    Part t;
    unsigned unit = blockIdx.x;
    t.stats = true;
    t.chunk = 0;
    if (!WHOLE) {
        // the first `lag` tiles' statistics, then pairs of results and statistics, then the last results
        const unsigned chunks = (unsigned)p.chunks, b = number, lead = p.lag * chunks, pairs = 2 * (p.units - p.lag) * chunks;
        if (b < lead || b >= lead + pairs) {
            t.stats = b < lead;
            const unsigned m = t.stats ? b : b - lead - pairs;
            unit = p.by_chunks(m);
            t.chunk = (int)(m - unit * chunks);
            if (!t.stats) unit += p.units - p.lag;
        } else {
            const unsigned m = b - lead, pair = p.by_pair(m), r = m - pair * 2 * chunks;
            t.stats = r & 1;
            t.chunk = (int)(r >> 1);
            unit = t.stats ? pair + p.lag : pair;
        }
    }
    t.unit = unit;
    t.n = (int)p.by_tiles(unit);
    const int tile = (int)(unit - (unsigned)t.n * (unsigned)p.tiles);
    t.wide = p.tile / E;
    t.step = p.step;
    bool odd;                                // a tile that is narrower than the others
    if (p.splits > 1) {
        t.group = (int)p.by_splits((unsigned)tile);
        t.split = tile - t.group * p.splits;
        t.c0 = t.group * p.size + t.split * p.tile;
        t.channels = min(p.tile, p.size - t.split * p.tile);
        t.groups = 1;
        odd = t.channels < p.tile;
    } else {
        t.c0 = tile * p.tile;
        t.channels = min(p.tile, p.channels - t.c0);
        t.group = (int)p.by_size((unsigned)t.c0);
        t.split = 0;
        t.groups = (int)p.by_size((unsigned)t.channels);
        odd = t.channels < p.tile;
    }
    if (odd) {
        t.wide = t.channels / E;
        t.step = kThreads / t.wide;
        t.row = (int)(threadIdx.x / (unsigned)t.wide);
    } else {
        t.row = (int)p.by_wide(threadIdx.x);
    }
    t.piece = (int)threadIdx.x - t.row * t.wide;
    t.mine = p.splits > 1 ? 0 : (int)p.by_group_wide((unsigned)t.piece);
    t.first = (int64_t)t.chunk * p.rows;
    t.rows = (int)min((int64_t)p.rows, p.pixels - t.first);
    const unsigned more = (unsigned)max(0, t.rows - t.row + t.step - 1);
    t.count = t.row >= t.step ? 0 : (int)(odd ? more / (unsigned)t.step : p.by_step(more));
    return t;
}
// The block's number in the order in which blocks start.
__device__ __forceinline__ unsigned take_number(const Params &p)
{
    __shared__ unsigned number;
    if (threadIdx.x == 0) number = atomicAdd(p.next, 1u);
    __syncthreads();
    return number;
}
__device__ __forceinline__ unsigned *ready_of(const Params &p, const Part &t)
{
    return p.ready + (p.splits > 1 ? (unsigned)t.n * (unsigned)p.groups + (unsigned)t.group : t.unit);
}
// A block's statistics are written.
__device__ __forceinline__ void announce(const Params &p, const Part &t)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(ready_of(p, t), 1u);
    }
}
// Until all statistics that the block's results need are there, or the limit has
// passed: then it says so, and its results are wrong.
__device__ __forceinline__ void await(const Params &p, const Part &t)
{
    if (threadIdx.x == 0) {
        const unsigned all = (unsigned)p.chunks * (unsigned)p.splits, *flag = ready_of(p, t);
        long long since = 0;
        for (unsigned i = 0;; ++i) {
            unsigned there;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(there) : "l"(flag) : "memory");
            if (there >= all) break;
            if (i & 63) continue;            // the timer once in 64 polls
            long long now;
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
            if (!since) since = now;
            if (now - since >= g_wait_limit_ns) {
                atomicOr(&g_wait_timeouts, (unsigned)AMSIM_WAIT_PARTIAL);
                break;
            }
        }
    }
    __syncthreads();
}

// Where the parts of a sample's chunk lie: one for each group, or for each split of it.
__device__ __forceinline__ int64_t parts_at(const Params &p, int n, int chunk)
{
    return ((int64_t)n * p.chunks + chunk) * ((int64_t)p.groups * p.splits);
}
// How many values a part holds.
__device__ __forceinline__ float values_of(const Params &p, int chunk, int split)
{
    const int64_t rows = min((int64_t)p.rows, p.pixels - (int64_t)chunk * p.rows);
    const int channels = p.splits > 1 ? min(p.tile, p.size - split * p.tile) : p.size;
    return (float)rows * (float)channels;
}

// The weights of a piece's channels.
template <int E>
__device__ __forceinline__ Values<E> weights_of(const Params &p, const float *w, int c, float otherwise)
{
    Values<E> r;
    if (E >= 4 && w && p.vec) {
#pragma unroll
        for (int j = 0; j < (E + 3) / 4; ++j) {
            const float4 f = *reinterpret_cast<const float4 *>(w + c + 4 * j);
            r.v[2 * j < (E + 1) / 2 ? 2 * j : 0] = make_float2(f.x, f.y);
            r.v[2 * j + 1 < (E + 1) / 2 ? 2 * j + 1 : 0] = make_float2(f.z, f.w);
        }
        return r;
    }
    each_pair<E>([&](int j) {
        const bool two = 2 * j + 1 < E;
        r.v[j] = w ? make_float2(w[c + 2 * j], two ? w[c + 2 * j + two] : 0.0f) : both(otherwise);
    });
    return r;
}

// A piece as it is in memory, to be widened where it is used.  What is read for
// the last time, and what is written, leaves the cache first: its room is for the
// tiles that are read again.
template <typename T, int E>
struct Raw {
    static constexpr int bytes = E * (int)sizeof(T);
    using Word = std::conditional_t<bytes == 16, uint4,
                                    std::conditional_t<bytes == 8, uint2, std::conditional_t<bytes == 4, uint32_t, uint16_t>>>;
    Word w;
    __device__ __forceinline__ Values<E> values() const
    {
        union {
            Word w;
            Vec<T, E> v;
        } u{w};
        Values<E> r;
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = widen(u.v.e[e]);
        each_pair<E>([&](int i) { r.v[i] = make_float2(f[2 * i], 2 * i + 1 < E ? f[2 * i + 1 < E ? 2 * i + 1 : 0] : 0.0f); });
        return r;
    }
};
template <int E, typename T>
__device__ __forceinline__ Raw<T, E> read(const T *at)
{
    return Raw<T, E>{*reinterpret_cast<const typename Raw<T, E>::Word *>(at)};
}
template <int E, typename T>
__device__ __forceinline__ Raw<T, E> read_last(const T *at)
{
    return Raw<T, E>{__ldcs(reinterpret_cast<const typename Raw<T, E>::Word *>(at))};
}
template <int E, typename T>
__device__ __forceinline__ void put_last(T *at, const Values<E> &r)
{
    alignas(16) T out[E];
    put<E>(out, r);
    __stcs(reinterpret_cast<typename Raw<T, E>::Word *>(at), *reinterpret_cast<const typename Raw<T, E>::Word *>(out));
}

// Runs over a thread's pieces: `load(i, k)` A at a time into places k, `use(i, k)`
// of A while the next are under way.
template <int A, typename L, typename U>
__device__ __forceinline__ void over_pieces(int count, L load, U use)
{
    auto load_all = [&](int i, int place) {
#pragma unroll
        for (int k = 0; k < A; ++k) load(i + k, place + k);
    };
    auto use_all = [&](int i, int place) {
#pragma unroll
        for (int k = 0; k < A; ++k) use(i + k, place + k);
    };
    int i = 0;
    if (A <= count) load_all(0, 0);
#pragma unroll 1
    while (i + A <= count) {
        if (i + 2 * A <= count) load_all(i + A, A);
        use_all(i, 0);
        i += A;
        if (i + A > count) break;
        if (i + 2 * A <= count) load_all(i + A, 0);
        use_all(i, A);
        i += A;
    }
#pragma unroll 1
    for (; i < count; ++i) {
        load(i, 0);
        use(i, 0);
    }
}
constexpr int kForwardAhead = 4, kBackwardAhead = 2;

// Forward, statistics: a chunk's moments by part.  A thread sums about its first
// value, so that what cancels is of the size of the values' spread, not of their
// mean.  Where the first is far from all the others, its square is summed for each
// of the n that a thread has: 5e-5 of the thread's sum of squares is lost at n = 96
// (24 pieces of four), 1e-3 at n = 1024, which samples of millions of pixels give.
// They go to `found` where the block itself works out the results.
template <typename TX, int E, bool WHOLE>
__device__ __forceinline__ void moments(const Params &p, const Part &t, float2 *found)
{
    __shared__ Moments all[kThreads];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const TX *x = static_cast<const TX *>(p.x) + (t.n * p.pixels + t.first + t.row) * p.ldx + t.c0 + t.piece * E;
    const int64_t far = (int64_t)t.step * p.ldx;
    float2 s1 = both(0.0f), s2 = both(0.0f);
    float about = 0.0f;
    if (t.count) about = read<E>(x).values().v[0].x;
    Raw<TX, E> r[2 * kForwardAhead];
    over_pieces<kForwardAhead>(
        t.count, [&](int i, int k) { r[k] = read<E>(x + i * far); },
        [&](int, int k) {
            const Values<E> v = r[k].values();
            each_pair<E>([&](int j) {
                float2 d = add2(v.v[j], both(-about));
                if (E == 1) d.y = 0.0f;
                s1 = add2(s1, d);
                s2 = fma2(d, d, s2);
            });
        });
    const float n = (float)(t.count * E), sum = s1.x + s1.y, m = t.count ? __fdividef(sum, n) : 0.0f;
    const float m2 = (s2.x + s2.y) - sum * m;
    all[threadIdx.x] = Moments{n, about + m, m2 < 0.0f ? 0.0f : m2};     // NaN stays
    __syncthreads();
    // a warp per group joins its threads: pieces side by side, then rows
    const int wide = p.splits > 1 ? t.wide : p.size / E, threads = wide * t.step;
    for (int g = warp; g < t.groups; g += kThreads / 32) {
        Moments m{0.0f, 0.0f, 0.0f};
        for (int i = lane; i < threads; i += 32) {
            const int row = p.splits > 1 ? i / wide : (int)p.by_group_wide((unsigned)i);
            m = join(m, all[row * t.wide + g * wide + (i - row * wide)]);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1)
            m = join(m, Moments{__shfl_down_sync(0xFFFFFFFFu, m.n, d), __shfl_down_sync(0xFFFFFFFFu, m.mean, d),
                                __shfl_down_sync(0xFFFFFFFFu, m.m2, d)});
        if (lane == 0)
            *(WHOLE ? found + g : p.by_part + parts_at(p, t.n, t.chunk) + (int64_t)(t.group + g) * p.splits + t.split) =
                make_float2(m.mean, m.m2);
    }
}

// bf16 results of groups whose mean is at most so many deviations from zero are x (rstd w) + (b - mean rstd w):
// what the second factor's rounding loses, u (|b| + 4 |w|), a value four deviations out loses of itself.  Further
// away it would not (a constant group of 3000 gave -0.025 for b = 0): there the mean is taken off first
// (8 x 128 x 128 x 512, silu: 75 and 78 us; 64 x 56 x 56 x 256, relu: 62 and 65), by all of a warp's lanes,
// which else would run through both forms (every second group far from zero: 108 and 91 us).
constexpr float kFoldedMean = 4.0f;

// Forward, results.
template <typename TX, typename TY, int E, bool WHOLE>
__device__ __forceinline__ void normalise(const Params &p, const Part &t, float2 *stats)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = warp; g < t.groups; g += kThreads / 32) {
        Moments m{0.0f, 0.0f, 0.0f};
        if (WHOLE) m = Moments{values_of(p, 0, 0), stats[g].x, stats[g].y};
        for (int i = lane; !WHOLE && i < p.chunks * p.splits; i += 32) {
            const int chunk = (int)p.by_splits((unsigned)i), split = i - chunk * p.splits;
            const float2 f = __ldcg(&p.by_part[parts_at(p, t.n, chunk) + (int64_t)(t.group + g) * p.splits + split]);
            m = join(m, Moments{values_of(p, chunk, split), f.x, f.y});
        }
#pragma unroll
        for (int d = 16; d && !WHOLE; d >>= 1)
            m = join(m, Moments{__shfl_down_sync(0xFFFFFFFFu, m.n, d), __shfl_down_sync(0xFFFFFFFFu, m.mean, d),
                                __shfl_down_sync(0xFFFFFFFFu, m.m2, d)});
        __syncwarp();                        // every lane has read stats[g]
        if (lane == 0) {
            const float2 f = make_float2(m.mean, __frsqrt_rn(m.m2 / m.n + p.eps));
            stats[g] = f;
            if (t.chunk == 0 && t.split == 0) {
                p.mean[(int64_t)t.n * p.groups + t.group + g] = f.x;
                p.rstd[(int64_t)t.n * p.groups + t.group + g] = f.y;
            }
        }
    }
    const int c = t.c0 + t.piece * E;
    Values<E> w = weights_of<E>(p, p.w, c, 1.0f), b = weights_of<E>(p, p.b, c, 0.0f);
    __syncthreads();
    const float2 f = stats[t.mine];
    const int64_t pixel = t.n * p.pixels + t.first + t.row;
    const TX *x = static_cast<const TX *>(p.x) + pixel * p.ldx + c;
    TY *y = static_cast<TY *>(p.y) + pixel * p.ldy + c;
    const int64_t far_x = (int64_t)t.step * p.ldx, far_y = (int64_t)t.step * p.ldy;
    auto results = [&](auto z) {
        with_activation(p.act, [&](auto act) {
            Raw<TX, E> r[2 * kForwardAhead];
            over_pieces<kForwardAhead>(
                t.count, [&](int i, int k) { r[k] = read_last<E>(x + i * far_x); },
                [&](int i, int k) {
                    Values<E> v = r[k].values();
                    each_pair<E>([&](int j) { v.v[j] = activate2<act.value>(z(v.v[j], j)); });
                    put_last<E>(y + i * far_y, v);
                });
        });
    };
    if constexpr (sizeof(TY) == 4) {
        results([&](float2 v, int j) { return fma2(mul2(add2(v, both(-f.x)), both(f.y)), w.v[j], b.v[j]); });
    } else {
        // one factor rstd w, a product an element less
        each_pair<E>([&](int j) { w.v[j] = mul2(w.v[j], both(f.y)); });
        if (!__any_sync(0xFFFFFFFFu, fabsf(f.x) * f.y > kFoldedMean)) {
            each_pair<E>([&](int j) { b.v[j] = fma2(w.v[j], both(-f.x), b.v[j]); });
            results([&](float2 v, int j) { return fma2(v, w.v[j], b.v[j]); });
        } else {
            results([&](float2 v, int j) { return fma2(add2(v, both(-f.x)), w.v[j], b.v[j]); });
        }
    }
}

// WHOLE: a block has all of its tile's pixels, and does both parts.
template <typename TX, typename TY, int E, bool WHOLE>
__global__ void __launch_bounds__(kThreads, WHOLE ? 3 : 4) forward_kernel(const Params p)
{
    __shared__ float2 stats[kTileGroups];
    const Part t = part_of<E, WHOLE>(p, WHOLE ? 0 : take_number(p));
    if (WHOLE) {
        moments<TX, E, WHOLE>(p, t, stats);
        __syncthreads();
        normalise<TX, TY, E, WHOLE>(p, t, stats);
    } else if (t.stats) {
        moments<TX, E, WHOLE>(p, t, stats);
        announce(p, t);
    } else {
        await(p, t);
        normalise<TX, TY, E, WHOLE>(p, t, stats);
    }
}

// What backward knows of a thread's group and channels.
template <int E>
struct Known {
    float mean, rstd;
    Values<E> w, b;
};
template <int E>
__device__ __forceinline__ Known<E> known(const Params &p, const Part &t)
{
    Known<E> k;
    const int c = t.c0 + t.piece * E;
    const int64_t group = (int64_t)t.n * p.groups + t.group + t.mine;
    k.mean = p.mean[group];
    k.rstd = p.rstd[group];
    k.w = weights_of<E>(p, p.w, c, 1.0f);
    k.b = weights_of<E>(p, p.b, c, 0.0f);
    return k;
}
template <int ACT, int E>
__device__ __forceinline__ void derive(const Known<E> &k, const Values<E> &x, Values<E> &xh, Values<E> &dz)
{
    each_pair<E>([&](int j) {
        xh.v[j] = mul2(add2(x.v[j], both(-k.mean)), both(k.rstd));
        dz.v[j] = before2<ACT>(dz.v[j], x.v[j], xh.v[j], k.mean, k.rstd, k.w.v[j], k.b.v[j]);
    });
}

// Backward, statistics: a chunk's sums of dz and dz xh by channel, and of these times w by part.
template <typename TX, typename TY, int E>
__device__ __forceinline__ void channel_sums(const Params &p, const Part &t)
{
    __shared__ float2 sums[E][kThreads];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = t.c0 + t.piece * E;
    const int64_t pixel = t.n * p.pixels + t.first + t.row;
    const TX *x = static_cast<const TX *>(p.x) + pixel * p.ldx + c;
    const TY *dy = static_cast<const TY *>(p.dy) + pixel * p.ldy + c;
    const int64_t far_x = (int64_t)t.step * p.ldx, far_y = (int64_t)t.step * p.ldy;
    const Known<E> k = known<E>(p, t);
    float2 s[(E + 1) / 2], q[(E + 1) / 2];
    each_pair<E>([&](int j) { s[j] = q[j] = both(0.0f); });
    with_activation(p.act, [&](auto act) {
        Raw<TX, E> r[2 * kBackwardAhead];
        Raw<TY, E> d[2 * kBackwardAhead];
        over_pieces<kBackwardAhead>(
            t.count,
            [&](int i, int k) {
                r[k] = read<E>(x + i * far_x);
                d[k] = read<E>(dy + i * far_y);
            },
            [&](int, int n) {
                Values<E> xh, dz = d[n].values();
                derive<act.value>(k, r[n].values(), xh, dz);
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
        rows = kThreads / 32;
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
    __syncthreads();
    // channel i of the tile is now sums[i % E][i / E]
    float2 *out = p.by_channel + ((int64_t)t.n * p.chunks + t.chunk) * p.channels + t.c0;
    const int size = p.splits > 1 ? t.channels : p.size;
    for (int g = warp; g < t.groups; g += kThreads / 32) {
        float2 m = both(0.0f);
        for (int i = g * size + lane; i < (g + 1) * size; i += 32) {
            const float2 v = sums[i % E][i / E];
            out[i] = v;
            m = fma2(v, both(p.w ? p.w[t.c0 + i] : 1.0f), m);
        }
        m = make_float2(warp_sum(m.x), warp_sum(m.y));
        if (lane == 0) p.by_part[parts_at(p, t.n, t.chunk) + (int64_t)(t.group + g) * p.splits + t.split] = m;
    }
}

// Backward, results: dx = dz (w rstd) - mean(t) rstd - xh (mean(t xh) rstd).
template <typename TX, typename TY, int E, bool WHOLE>
__device__ __forceinline__ void gradients(const Params &p, const Part &t)
{
    __shared__ float2 means[kTileGroups];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = t.c0 + t.piece * E;
    const Known<E> k = known<E>(p, t);
    if (!WHOLE) await(p, t);
    for (int g = warp; g < t.groups; g += kThreads / 32) {
        float2 m = both(0.0f);
        for (int i = lane; i < p.chunks * p.splits; i += 32) {
            const int chunk = (int)p.by_splits((unsigned)i), split = i - chunk * p.splits;
            m = add2(m, __ldcg(&p.by_part[parts_at(p, t.n, chunk) + (int64_t)(t.group + g) * p.splits + split]));
        }
        m = make_float2(warp_sum(m.x), warp_sum(m.y));
        const float count = (float)p.size * (float)p.pixels;
        if (lane == 0) means[g] = make_float2(m.x / count, m.y / count);
    }
    __syncthreads();
    const float2 m = mul2(means[t.mine], both(-k.rstd));
    Values<E> scale;
    each_pair<E>([&](int j) { scale.v[j] = mul2(k.w.v[j], both(k.rstd)); });
    const int64_t pixel = t.n * p.pixels + t.first + t.row;
    const TX *x = static_cast<const TX *>(p.x) + pixel * p.ldx + c;
    const TY *dy = static_cast<const TY *>(p.dy) + pixel * p.ldy + c;
    TX *dx = static_cast<TX *>(p.dx) + pixel * p.lddx + c;
    const int64_t far_x = (int64_t)t.step * p.ldx, far_y = (int64_t)t.step * p.ldy, far = (int64_t)t.step * p.lddx;
    with_activation(p.act, [&](auto act) {
        Raw<TX, E> r[2 * kBackwardAhead];
        Raw<TY, E> d[2 * kBackwardAhead];
        over_pieces<kBackwardAhead>(
            t.count,
            [&](int i, int n) {
                r[n] = read_last<E>(x + i * far_x);
                d[n] = read_last<E>(dy + i * far_y);
            },
            [&](int i, int n) {
                Values<E> xh, dz = d[n].values();
                derive<act.value>(k, r[n].values(), xh, dz);
                each_pair<E>([&](int j) { dz.v[j] = fma2(xh.v[j], both(m.y), fma2(dz.v[j], scale.v[j], both(m.x))); });
                put_last<E>(dx + i * far, dz);
            });
    });
}

template <typename TX, typename TY, int E, bool WHOLE>
__global__ void __launch_bounds__(kThreads, WHOLE || E == 8 ? 2 : 3) backward_kernel(const Params p)
{
    amsim::chain_start();
    const Part t = part_of<E, WHOLE>(p, WHOLE ? 0 : take_number(p));
    if (WHOLE) {
        channel_sums<TX, TY, E>(p, t);
        __syncthreads();
        gradients<TX, TY, E, WHOLE>(p, t);
    } else if (t.stats) {
        channel_sums<TX, TY, E>(p, t);
        announce(p, t);
    } else {
        gradients<TX, TY, E, WHOLE>(p, t);
    }
}

// Without pixels: mean 0, rstd 1 / sqrt(eps).
__global__ void __launch_bounds__(kThreads) empty_kernel(const Params p, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    p.mean[i] = 0.0f;
    p.rstd[i] = 1.0f / sqrtf(p.eps);
}

// dw and db from the sums by channel: a block takes 32 channels, its 32 warps
// every 32nd chunk, eight loads at a time.
__global__ void __launch_bounds__(1024) weights_kernel(const Params p)
{
    __shared__ float2 part[32][33];
    amsim::chain_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + lane;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < p.channels) {
#pragma unroll 8
        for (int64_t n = warp; n < p.samples_chunks; n += 32) s = add2(s, p.by_channel[n * p.channels + c]);
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

size_t type_size(int t) { return t == AMSIM_BF16 ? 2 : 4; }
bool aligned(const void *q, size_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }
bool whole(const void *q, int64_t ld, size_t size, int E) { return aligned(q, E * size) && ld % E == 0; }

int check(const amsim_group_norm_desc *d)
{
    if (!d || d->batch < 0 || d->pixels < 0 || d->channels < 1 || d->groups < 1 || d->channels % d->groups)
        return AMSIM_EINVAL;
    if (d->batch > 0x7FFFFFFF || d->pixels > (int64_t)1 << 40 || d->channels > 1 << 24) return AMSIM_EINVAL;
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

Params params(const amsim_group_norm_desc *d)
{
    Params p{};
    p.pixels = d->pixels;
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

// Channels of a piece, and scratch of a call: values by part and by channel, flags.
struct Plan {
    int E;
    size_t parts, sums, flags;
    size_t bytes() const { return (parts + sums) * sizeof(float2) + flags * sizeof(unsigned); }
};
constexpr int kTileBytes = 256;              // of a pixel, about
// Of a thread: a block's own costs are spread over them (16, 24, 32: 94, 89, 87 us for 64 x 56 x 56 x 256 fp32
// forward, 144, 142, 149 us backward), and of one whose block has all of its tile's pixels.
constexpr int kPieces = 24, kWholePieces = 32;
constexpr int64_t kBehind = 32 << 20;        // bytes of what is read twice between a tile's statistics and results

// `fits(E)`: the call's rows are on E elements.  false: too many blocks.
template <typename F>
bool plan(const amsim_group_norm_desc *d, bool fwd, int sms, Params &p, Plan *out, F fits)
{
    const int xs = (int)type_size(d->x_type), ys = (int)type_size(d->y_type), bytes = xs + (fwd ? 0 : ys);
    int E = xs + ys == 4 ? 8 : 4;                // 16 bytes of the wider type
    while (E > 1 && (p.size % E || !fits(E))) E /= 2;
    // tiles of about kTileBytes of a pixel, or of half of it where one block then has all of a tile's pixels
    // (128 x 32 x 32 x 64 fp32 backward 41 and 32 us)
    for (int width : {kTileBytes, kTileBytes / 2}) {
        const int widest = std::min(kThreads * E, std::max(E, width / std::max(xs, ys)));
        Params q = p;
        if (q.size > widest) {                   // parts of one group, alike up to a piece
            q.splits = (q.size + widest - 1) / widest;
            q.tile = ((q.size / E + q.splits - 1) / q.splits) * E;
            q.splits = (q.size + q.tile - 1) / q.tile;
            q.tiles = q.groups * q.splits;
        } else {
            q.splits = 1;
            q.tile = std::min({widest / q.size, q.groups, kTileGroups}) * q.size;
            q.tiles = (q.channels + q.tile - 1) / q.tile;
        }
        q.whole = q.splits == 1 && d->pixels <= (int64_t)(kThreads / (q.tile / E)) * kWholePieces;
        if (width == kTileBytes || q.whole) {
            p = q;
            if (q.whole) break;
        }
    }
    const int64_t units = d->batch * p.tiles;
    const int step = kThreads / (p.tile / E);
    // chunks of kPieces a thread, smaller where these do not give every SM four blocks
    int64_t chunks = (d->pixels + (int64_t)step * kPieces - 1) / ((int64_t)step * kPieces);
    const int64_t enough = (4 * (int64_t)sms + units - 1) / units, most = (d->pixels + 2 * step - 1) / (2 * step);
    chunks = std::max<int64_t>(1, std::min<int64_t>(std::max(chunks, std::min(enough, most)), 1024));
    if (p.whole) chunks = 1;
    const int64_t rows = (d->pixels + chunks - 1) / chunks;
    if (rows > 0x7FFFFFFF - kThreads) return false;
    p.rows = (int)rows;
    p.chunks = (int)((d->pixels + rows - 1) / rows);
    p.samples_chunks = d->batch * p.chunks;
    p.step = step;
    p.by_tiles = divisor((unsigned)p.tiles);
    p.by_splits = divisor((unsigned)p.splits);
    p.by_chunks = divisor((unsigned)p.chunks);
    p.by_wide = divisor((unsigned)(p.tile / E));
    p.by_step = divisor((unsigned)step);
    p.by_group_wide = divisor((unsigned)std::max(1, p.size / E));
    p.by_size = divisor((unsigned)p.size);
    p.vec = aligned(p.w, 16) && aligned(p.b, 16);
    p.by_pair = divisor(2u * (unsigned)p.chunks);
    const int64_t unit_bytes = std::max<int64_t>(1, d->pixels * p.tile * bytes);
    if (units > 0x7FFFFFFF || 2 * units * p.chunks > 0x7FFFFFFF) return false;
    p.units = (unsigned)units;
    p.lag = (unsigned)std::min(units, std::max<int64_t>(p.splits, (kBehind + unit_bytes - 1) / unit_bytes));
    out->E = E;
    out->parts = fwd && p.whole ? 0 : (size_t)p.samples_chunks * p.groups * p.splits;
    out->sums = fwd ? 0 : (size_t)p.samples_chunks * p.channels;
    out->flags = p.whole ? 0 : 1 + (size_t)(p.splits > 1 ? d->batch * p.groups : units);
    return true;
}

void scratch(Params &p, const Plan &q, void *ws)
{
    p.by_part = static_cast<float2 *>(ws);
    p.by_channel = p.by_part + q.parts;
    p.next = reinterpret_cast<unsigned *>(p.by_channel + q.sums);
    p.ready = p.next + 1;
}

int start(bool chained, void (*kernel)(Params), int64_t blocks, int threads, const Params &p, cudaStream_t st)
{
    const int rc = amsim::cuda_status(
        amsim::chain_launch(chained, kernel, dim3((unsigned)blocks), dim3((unsigned)threads), 0, st, p));
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}

template <typename TX, typename TY, int E>
int pass(bool fwd, const Params &p, const Plan &plan, cudaStream_t st)
{
    int rc;
    if (p.whole) {
        rc = start(false, fwd ? forward_kernel<TX, TY, E, true> : backward_kernel<TX, TY, E, true>, p.units, kThreads, p, st);
    } else {
        rc = amsim::cuda_status(cudaMemsetAsync(p.next, 0, plan.flags * sizeof(unsigned), st));
        if (rc) return rc;
        rc = start(false, fwd ? forward_kernel<TX, TY, E, false> : backward_kernel<TX, TY, E, false>,
                   2 * (int64_t)p.units * p.chunks, kThreads, p, st);
    }
    if (rc || fwd || (!p.dw && !p.db)) return rc;
    return start(true, weights_kernel, (p.channels + 31) / 32, 1024, p, st);
}
template <typename TX, typename TY>
int pass(bool fwd, const Params &p, const Plan &plan, cudaStream_t st)
{
    if constexpr (sizeof(TX) + sizeof(TY) == 4)
        if (plan.E == 8) return pass<TX, TY, 8>(fwd, p, plan, st);
    return plan.E == 4   ? pass<TX, TY, 4>(fwd, p, plan, st)
           : plan.E == 2 ? pass<TX, TY, 2>(fwd, p, plan, st)
                         : pass<TX, TY, 1>(fwd, p, plan, st);
}
int run(const amsim_group_norm_desc *d, bool fwd, const Params &p, const Plan &plan, cudaStream_t st)
{
    using B = __nv_bfloat16;
    if (d->x_type == AMSIM_F32)
        return d->y_type == AMSIM_F32 ? pass<float, float>(fwd, p, plan, st) : pass<float, B>(fwd, p, plan, st);
    return d->y_type == AMSIM_F32 ? pass<B, float>(fwd, p, plan, st) : pass<B, B>(fwd, p, plan, st);
}

}  // namespace

extern "C" size_t amsim_group_norm_workspace_size(const amsim_group_norm_desc *d, int which)
{
    if (check(d) || which < 0 || which > 1 || !d->batch || !d->pixels) return 0;
    const int sms = device_sms();
    size_t most = 0;
    for (int on : {1, 2, 4, 8}) {                // the calls' pointers and strides decide which
        Params p = params(d);
        Plan q;
        if (!plan(d, !which, sms ? sms : 1, p, &q, [&](int E) { return E <= on; })) return 0;
        most = std::max(most, q.bytes());
    }
    return most;
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
    const int sms = device_sms();
    Params p = params(d);
    p.x = x;
    p.y = y;
    p.w = w;
    p.b = b;
    p.mean = mean;
    p.rstd = rstd;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!d->pixels) {
        const int64_t n = d->batch * d->groups, blocks = (n + kThreads - 1) / kThreads;
        if (blocks > 0x7FFFFFFF) return AMSIM_EINVAL;
        empty_kernel<<<(unsigned)blocks, kThreads, 0, st>>>(p, n);
        const int rc = amsim::cuda_status(cudaGetLastError());
        if (rc == AMSIM_OK) amsim::count_launch();
        return rc;
    }
    Plan q;
    if (!plan(d, true, sms ? sms : 1, p, &q,
              [&](int n) { return whole(x, p.ldx, xs, n) && whole(y, p.ldy, ys, n); }))
        return AMSIM_EINVAL;
    if (q.bytes() && (!ws || ws_bytes < q.bytes())) return AMSIM_EINVAL;
    if (!sms) return AMSIM_ECUDA;
    scratch(p, q, ws);
    return run(d, true, p, q, st);
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
    if (!x || !dy || !dx || !mean || !rstd) return AMSIM_EINVAL;
    const int sms = device_sms();
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
    Plan q;
    if (!plan(d, false, sms ? sms : 1, p, &q, [&](int n) {
            return whole(x, p.ldx, xs, n) && whole(dx, p.lddx, xs, n) && whole(dy, p.ldy, ys, n);
        }))
        return AMSIM_EINVAL;
    if (!ws || ws_bytes < q.bytes()) return AMSIM_EINVAL;
    if (!sms) return AMSIM_ECUDA;
    scratch(p, q, ws);
    return run(d, false, p, q, st);
}
