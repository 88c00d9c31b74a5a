// The softmax between attention's contractions, with a relative position bias,
// lengths, a causal mask and dropout, and its gradient with the bias table's.
//
// A row is read once and kept in registers, so the traffic is the compulsory
// one.  It is taken in chunks of 128 columns, a chunk by a warp: up to 512
// columns one warp has the whole row, longer rows are shared by the warps of a
// block and then by the blocks of a cluster, whose maxima and sums are joined
// once per row (each warp's exponentials are relative to its own maximum until
// then).  Longer rows are read twice (shape() below).
//
// Memory bounds both where rows are on 16 bytes: 32 x 16 x 512 x 512 with bias and
// dropout takes 174 us forward, 0.92 of a plain copy's rate (the generator's products keep
// the multiplier pipe 66 % busy meanwhile), and 254 us backward, 0.95.  Rows off 16 bytes
// are nearer the issue slots: 7 x 12 x 333 x 1531 with lengths 53 us forward, 0.82.
//
// Within a chunk a lane has four columns: neighbours where rows are on 16 bytes
// (one load of 16 bytes), else every 32nd (four coalesced loads).
//
// Blocks belong to one head and keep its bias by distance in shared memory.
// dtable wants the sum of dS along each diagonal of the scores (one distance,
// all of a head's rows).  Within a row every distance inside (-D, D) occurs at
// one column, so a warp adds its row to an array by distance in shared memory
// without conflicts; columns further away go to two registers.  The arrays are
// added in a fixed order, then by bucket.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "chained.cuh"
#include "pairs.cuh"
#include "philox.cuh"

namespace {

using amsim::add2;
using amsim::both;
using amsim::Drop;
using amsim::fma2;
using amsim::mul2;

struct Params {
    const float *scores, *probs, *dprobs, *stats, *table;   // inputs
    const int32_t *buckets, *lengths, *offsets;
    float *out, *out_stats, *dtable, *part;
    int64_t ld_in, ld_g, ld_out, offset;     // ld_in: of scores or probs
    int queries, keys, quads, chunks, heads;
    int groups, row_groups, shares;          // groups of rows of one head, of one sequence and head
    int ahead_b, ahead_i;                    // shares, in sequences and groups
    int cluster, causal, num_buckets, D;
    Drop drop;
};

constexpr int kWarpRows = 8;                 // warps of a block that each take a row
constexpr int kFewThreads = 768;             // of a block that keeps four chunks of two tensors a warp
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kLog2E = 1.44269504088896341f;

// Four values of a lane.
struct Four {
    float2 a, b;
};
__device__ __forceinline__ Four four(float v) { return Four{both(v), both(v)}; }
template <typename F>
__device__ __forceinline__ void each(Four &v, F use)
{
    use(v.a.x, 0);
    use(v.a.y, 1);
    use(v.b.x, 2);
    use(v.b.y, 3);
}
__device__ __forceinline__ Four add(const Four &x, const Four &y) { return Four{add2(x.a, y.a), add2(x.b, y.b)}; }
__device__ __forceinline__ Four mul(const Four &x, const Four &y) { return Four{mul2(x.a, y.a), mul2(x.b, y.b)}; }
__device__ __forceinline__ float sum(const Four &v)
{
    const float2 s = add2(v.a, v.b);
    return s.x + s.y;
}

// Column k of a lane's four in a chunk.
template <bool VEC>
__device__ __forceinline__ int column(int chunk, int lane, int k)
{
    return chunk * 128 + (VEC ? 4 * lane + k : 32 * k + lane);
}

// A chunk as it is loaded: nothing waits for it here, so that a row's loads are
// all under way before the first is used.  Pieces that begin at a visible key are whole.
template <bool VEC, bool FULL = false>
__device__ __forceinline__ Four load_chunk(const float *row, int chunk, int lane, int visible, float fill)
{
    Four v = four(fill);
    const int c = column<VEC>(chunk, lane, 0);
    if (VEC) {
        float4 f = make_float4(fill, fill, fill, fill);
        if (FULL || c < visible) f = *reinterpret_cast<const float4 *>(row + c);
        v = Four{make_float2(f.x, f.y), make_float2(f.z, f.w)};
    } else if (FULL || (chunk + 1) * 128 <= visible) {
        each(v, [&](float &x, int k) { x = row[c + 32 * k]; });
    } else {
        each(v, [&](float &x, int k) { if (c + 32 * k < visible) x = row[c + 32 * k]; });
    }
    return v;
}
// `fill` behind the last visible key of a whole piece; of any piece where something was added to it (ADDED).
template <bool VEC, bool FULL = false, bool ADDED = false>
__device__ __forceinline__ void fill_chunk(Four &v, int chunk, int lane, int visible, float fill)
{
    if ((VEC || ADDED) && !FULL && (chunk + 1) * 128 > visible)
        each(v, [&](float &x, int k) { if (column<VEC>(chunk, lane, k) >= visible) x = fill; });
}
// Zeros where no key is visible.
template <bool VEC, bool FULL = false>
__device__ __forceinline__ void hide(Four &v, int chunk, int lane, int visible)
{
    if (!FULL && (chunk + 1) * 128 > visible) each(v, [&](float &x, int k) { if (column<VEC>(chunk, lane, k) >= visible) x = 0.0f; });
}
template <bool VEC, bool FULL = false>
__device__ __forceinline__ void store_chunk(float *row, int chunk, int lane, int keys, Four v)
{
    const int c = column<VEC>(chunk, lane, 0);
    if (VEC) {
        if (FULL || c < keys) *reinterpret_cast<float4 *>(row + c) = make_float4(v.a.x, v.a.y, v.b.x, v.b.y);
    } else if (FULL || (chunk + 1) * 128 <= keys) {
        each(v, [&](float &x, int k) { row[c + 32 * k] = x; });
    } else {
        each(v, [&](float &x, int k) { if (c + 32 * k < keys) row[c + 32 * k] = x; });
    }
}

// exp((a - base)): the difference first, so that rows of the type's lowest value
// stay finite; two roundings of the difference and some 2^-22 of the instruction.
__device__ __forceinline__ float power_of_2(float t)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return e;
}
__device__ __forceinline__ Four exponentials(Four v, float base)
{
    v = Four{mul2(add2(v.a, both(-base)), both(kLog2E)), mul2(add2(v.b, both(-base)), both(kLog2E))};
    each(v, [](float &x, int) { x = power_of_2(x); });
    return v;
}
__device__ __forceinline__ float finite_base(float top) { return top == -INFINITY ? 0.0f : top; }

// The quads of a row: their numbers' lower halves from `lower` on.  (A row whose
// numbers pass 2^32 has `split`, and each lane takes the upper half of its own.)
struct RowDraws {
    amsim::QuadStream stream;
    uint32_t lower, upper;
    bool split;
};
__device__ __forceinline__ RowDraws row_draws(int64_t row, const Params &p, uint64_t call)
{
    const uint64_t first = (uint64_t)row * (unsigned)p.quads;
    RowDraws r;
    r.lower = (uint32_t)first;
    r.upper = (uint32_t)(first >> 32);
    r.split = r.lower + (unsigned)p.chunks * 32u < r.lower;
    r.stream = amsim::quad_stream(r.upper, call, p.drop);
    return r;
}
__device__ __noinline__ amsim::QuadStream next_stream(uint32_t upper, uint64_t call, const Drop &d)
{
    return amsim::quad_stream(upper + 1, call, d);
}
// Dropout of a chunk's values, which stay times `scale`.  A lane draws the quad
// of columns 4 lane ..; where it has other columns the lanes exchange one bit a column.
template <bool VEC>
__device__ __forceinline__ void drop_chunk(Four &v, const RowDraws &r, int chunk, int lane, const Params &p,
                                           uint64_t call, float scale)
{
    const uint32_t quad = r.lower + (uint32_t)(chunk * 32 + lane);
    amsim::QuadStream stream = r.stream;
    if (r.split && quad < r.lower) stream = next_stream(r.upper, call, p.drop);
    const uint4 w = amsim::quad_words(quad, stream, p.drop);
    const uint32_t border = p.drop.border;
    v = mul(v, four(scale));
    if (VEC) {
        v.a.x = w.x >= border ? v.a.x : 0.0f;
        v.a.y = w.y >= border ? v.a.y : 0.0f;
        v.b.x = w.z >= border ? v.b.x : 0.0f;
        v.b.y = w.w >= border ? v.b.y : 0.0f;
    } else {
        const unsigned m0 = __ballot_sync(kAll, w.x >= border), m1 = __ballot_sync(kAll, w.y >= border),
                       m2 = __ballot_sync(kAll, w.z >= border), m3 = __ballot_sync(kAll, w.w >= border);
        const unsigned mine = (lane & 2 ? (lane & 1 ? m3 : m2) : (lane & 1 ? m1 : m0)) >> (lane >> 2);
        each(v, [&](float &x, int k) { x = mine >> (8 * k) & 1 ? x : 0.0f; });
    }
}

// Arrays by distance hold four entries more at each end, where distances beyond
// D act as D: entry i is distance i - D - 4.  A lane's four neighbours then take
// one access of 16 bytes, whose place is off by `i & 3`: the bias is kept in four
// copies, copy k from entry k on.
__host__ __device__ __forceinline__ int entries(int D) { return (2 * D + 15) & ~3; }

// The head's bias by distance, into shared memory.
__device__ __forceinline__ void load_bias(const Params &p, int head, float *bias)
{
    const int n = entries(p.D);
    for (int i = threadIdx.x; i < n + 3; i += blockDim.x) {
        const int k = p.buckets[min(max(i - 4, 0), 2 * p.D)];
        const float v = (unsigned)k < (unsigned)p.num_buckets ? p.table[(int64_t)k * p.heads + head] : 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (i >= c && i - c < n) bias[c * n + i - c] = v;
    }
}
template <bool VEC>
__device__ __forceinline__ void add_bias(Four &v, const float *bias, int chunk, int lane, int pos, const Params &p)
{
    const int first = column<VEC>(chunk, lane, 0) - pos + p.D + 4;
    if (VEC) {
        const int i = min(max(first, 0), 2 * p.D + 5), k = i & 3;
        const float4 f = *reinterpret_cast<const float4 *>(bias + k * entries(p.D) + (i - k));
        v = add(v, Four{make_float2(f.x, f.y), make_float2(f.z, f.w)});
    } else {
        each(v, [&](float &x, int k) { x += bias[min(max(first + 32 * k, 0), 2 * p.D + 8)]; });
    }
}

// One row: where it is, what it sees, and its query's place.  Warps that take rows of their own take them by the place modulo
// eight, so that a warp's sums by distance keep their place modulo four.
struct Row {
    int64_t row;
    int visible, pos;
    bool on;
};
template <bool BLOCK>
__device__ __forceinline__ Row row_of(const Params &p, int head, int b, int i)
{
    const int64_t first = p.offsets ? (int64_t)p.offsets[b] : p.offset;
    if (!BLOCK) i = kWarpRows * i + (((int)(threadIdx.x >> 5) - (int)first) & (kWarpRows - 1));
    Row w;
    w.on = i < p.queries;
    w.row = ((int64_t)b * p.heads + head) * p.queries + i;
    int end = p.keys;
    if (p.lengths) end = min(end, max(p.lengths[b], 0));
    // brought near enough for 32 bits; every column of the row's chunks then stays further than D
    const int64_t pos = max(min(first + i, (int64_t)p.chunks * 128 + p.D + 8), -(int64_t)p.D - 8);
    w.pos = (int)pos;
    if (p.causal) end = min(end, max(w.pos + 1, 0));
    w.visible = end;
    return w;
}
// A head's groups of rows in turn, from the share's first on: sequence and place in it.
struct Place {
    int b, i;
};
__device__ __forceinline__ Place first_place(const Params &p, int share)
{
    Place t;
    t.b = (int)((unsigned)share / (unsigned)p.row_groups);
    t.i = share - t.b * p.row_groups;
    return t;
}
__device__ __forceinline__ void advance(const Params &p, Place &t)
{
    t.i += p.ahead_i;
    t.b += p.ahead_b;
    if (t.i >= p.row_groups) {
        t.i -= p.row_groups;
        ++t.b;
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// A cluster's blocks.
__device__ __forceinline__ int cluster_rank()
{
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float2 of_rank(const float2 *q, int rank)
{
    uint32_t at;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(q)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

// exp(mine - top), 0 for a part that sees nothing.
__device__ __forceinline__ float part_factor(float mine, float top)
{
    return mine == -INFINITY ? 0.0f : power_of_2((mine - top) * kLog2E);
}

// What the warps (and blocks) that share a row exchange, once per row; two sets
// in turn, so that one barrier a row is enough: a set is written again only
// after the barrier that follows its last reader.
struct Exchange {
    float2 warps[2][32], blocks[2];
};

// The row's maximum, and 1 / sum, from each warp's (maximum, sum).
template <bool BLOCK>
__device__ __forceinline__ float2 join_rows(const Params &p, float top, float total, Exchange &x, int turn)
{
    if (BLOCK) {
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) x.warps[turn][threadIdx.x >> 5] = make_float2(top, total);
        __syncthreads();
        const float2 v = lane < warps ? x.warps[turn][lane] : make_float2(-INFINITY, 0.0f);
        top = warp_max(v.x);
        total = warp_sum(v.y == 0.0f ? 0.0f : v.y * part_factor(v.x, top));
        if (p.cluster > 1) {
            if (threadIdx.x == 0) x.blocks[turn] = make_float2(top, total);
            cluster_barrier();
            const float2 b = lane < p.cluster ? of_rank(&x.blocks[turn], lane) : make_float2(-INFINITY, 0.0f);
            top = warp_max(b.x);
            total = warp_sum(b.y == 0.0f ? 0.0f : b.y * part_factor(b.x, top));
        }
    }
    return make_float2(top, total == 0.0f ? 0.0f : 1.0f / total);
}
template <bool BLOCK>
__device__ __forceinline__ float join_sums(const Params &p, float v, Exchange &x, int turn)
{
    if (BLOCK) {
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) x.warps[turn][threadIdx.x >> 5].x = v;
        __syncthreads();
        v = warp_sum(lane < warps ? x.warps[turn][lane].x : 0.0f);
        if (p.cluster > 1) {
            if (threadIdx.x == 0) x.blocks[turn].x = v;
            cluster_barrier();
            v = warp_sum(lane < p.cluster ? of_rank(&x.blocks[turn], lane).x : 0.0f);
        }
    }
    return v;
}

// A block's part of the work: a head, and which of its groups of rows.
struct Part {
    int head, share, rank;
    int first_chunk, step;                   // this warp's chunks
};
template <bool BLOCK>
__device__ __forceinline__ Part part_of(const Params &p)
{
    Part t;
    unsigned unit = blockIdx.x;
    t.rank = 0;
    if (BLOCK && p.cluster > 1) {
        t.rank = cluster_rank();
        unit /= (unsigned)p.cluster;
    }
    t.head = (int)(unit / (unsigned)p.shares);
    t.share = (int)(unit - (unsigned)t.head * (unsigned)p.shares);
    const int warps = BLOCK ? (int)(blockDim.x >> 5) : 1;
    t.first_chunk = BLOCK ? t.rank * warps + (int)(threadIdx.x >> 5) : 0;
    t.step = BLOCK ? warps * p.cluster : 1;
    return t;
}

// The rows of a block.  NV > 0: a warp's part of the row is NV chunks, kept in
// registers; NV == 0: a row of any length, read twice.
template <int NV, bool VEC, bool BLOCK, bool BIAS, bool DROP>
__device__ __forceinline__ void forward_rows(const Params &p, const Part &t, const float *bias, Exchange &exchange)
{
    const int lane = threadIdx.x & 31;
    const uint64_t call = DROP ? amsim::drop_call(p.drop) : 0;
    int turn = 0;
    Place at = first_place(p, t.share);
    for (int g = t.share; g < p.groups; g += p.shares, turn ^= 1, advance(p, at)) {
        const Row w = row_of<BLOCK>(p, t.head, at.b, at.i);
        if (!BLOCK && !w.on) continue;
        const float *in = p.scores + w.row * p.ld_in;
        float *out = p.out + w.row * p.ld_out;
        RowDraws draws{};
        if (DROP) draws = row_draws(w.row, p, call);
        auto logits = [&](auto full, Four a, int chunk) {
            constexpr bool FULL = decltype(full)::value;
            if (FULL || chunk * 128 < w.visible) {
                if (BIAS) add_bias<VEC>(a, bias, chunk, lane, w.pos, p);
                fill_chunk<VEC, FULL, BIAS>(a, chunk, lane, w.visible, -INFINITY);   // whatever hidden keys' biases are
            }
            return a;
        };
        auto finish = [&](auto full, Four e, int chunk, float factor) {
            constexpr bool FULL = decltype(full)::value;
            if (!FULL && chunk * 128 >= w.visible)
                e = four(0.0f);
            else if (DROP)
                drop_chunk<VEC>(e, draws, chunk, lane, p, call, factor * p.drop.scale);
            else
                e = mul(e, four(factor));
            hide<VEC, FULL>(e, chunk, lane, w.visible);
            store_chunk<VEC, FULL>(out, chunk, lane, p.keys, e);
        };
        float mine = -INFINITY, total = 0.0f;
        float2 joined;
        if (NV) {
            Four a[NV ? NV : 1];
            // `full`: every key of this warp's chunks is visible, and nothing has to be checked
            auto begin = [&](auto full) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    a[v] = load_chunk<VEC, decltype(full)::value>(in, t.first_chunk + v * t.step, lane, w.visible, -INFINITY);
#pragma unroll
                for (int v = 0; v < NV; ++v) a[v] = logits(full, a[v], t.first_chunk + v * t.step);
            };
            const bool all = (t.first_chunk + (NV - 1) * t.step + 1) * 128 <= w.visible;
            if (all)
                begin(std::true_type{});
            else
                begin(std::false_type{});
#pragma unroll
            for (int v = 0; v < NV; ++v)
                mine = fmaxf(fmaxf(mine, fmaxf(a[v].a.x, a[v].a.y)), fmaxf(a[v].b.x, a[v].b.y));
            mine = warp_max(mine);
            const float base = finite_base(mine);
            Four sums = four(0.0f);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                a[v] = exponentials(a[v], base);
                sums = add(sums, a[v]);
            }
            total = warp_sum(sum(sums));
            joined = join_rows<BLOCK>(p, mine, total, exchange, turn);
            const float factor = BLOCK ? joined.y * part_factor(mine, joined.x) : joined.y;
            auto end = [&](auto full) {
#pragma unroll
                for (int v = 0; v < NV; ++v) finish(full, a[v], t.first_chunk + v * t.step, factor);
            };
            if (all)
                end(std::true_type{});
            else
                end(std::false_type{});
        } else {
            // four chunks at a time, whose loads are under way together
            std::false_type some;
            auto logits_of = [&](int chunk, Four (&a)[4]) {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    a[v] = load_chunk<VEC>(in, chunk + v * t.step, lane, w.visible, -INFINITY);
#pragma unroll
                for (int v = 0; v < 4; ++v) a[v] = logits(some, a[v], chunk + v * t.step);
            };
            Four a[4];
            for (int chunk = t.first_chunk; chunk * 128 < w.visible; chunk += 4 * t.step) {
                logits_of(chunk, a);
                float most = -INFINITY;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    most = fmaxf(fmaxf(most, fmaxf(a[v].a.x, a[v].a.y)), fmaxf(a[v].b.x, a[v].b.y));
                if (most > mine) {
                    total *= part_factor(mine, most);
                    mine = most;
                }
                const float base = finite_base(mine);
                Four sums = exponentials(a[0], base);
#pragma unroll
                for (int v = 1; v < 4; ++v) sums = add(sums, exponentials(a[v], base));
                total += sum(sums);
            }
            const float top = warp_max(mine);
            total = warp_sum(mine == -INFINITY ? total : total * part_factor(mine, top));
            joined = join_rows<BLOCK>(p, top, total, exchange, turn);
            const float base = finite_base(joined.x);
            for (int chunk = t.first_chunk; chunk < p.chunks; chunk += 4 * t.step) {
                logits_of(chunk, a);
#pragma unroll
                for (int v = 0; v < 4; ++v) finish(some, exponentials(a[v], base), chunk + v * t.step, joined.y);
            }
        }
        if (p.out_stats && lane == 0 && (!BLOCK || (threadIdx.x == 0 && t.rank == 0)))
            *reinterpret_cast<float2 *>(p.out_stats + 2 * w.row) = joined;
    }
}

template <int NV, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kWarpRows) forward_kernel(const Params p)
{
    extern __shared__ __align__(16) float bias[];
    __shared__ Exchange exchange;
    const Part t = part_of<BLOCK>(p);
    if (p.table) {
        load_bias(p, t.head, bias);
        __syncthreads();
        if (p.drop.border)
            forward_rows<NV, VEC, BLOCK, true, true>(p, t, bias, exchange);
        else
            forward_rows<NV, VEC, BLOCK, true, false>(p, t, bias, exchange);
    } else if (p.drop.border) {
        forward_rows<NV, VEC, BLOCK, false, true>(p, t, bias, exchange);
    } else {
        forward_rows<NV, VEC, BLOCK, false, false>(p, t, bias, exchange);
    }
    if (BLOCK && p.cluster > 1) cluster_barrier();       // no block leaves while another reads from it
}

// dtable of a head from its sums by distance; each warp takes buckets of its own.
__device__ __forceinline__ void by_bucket(const Params &p, int head, const float *total)
{
    const int lane = threadIdx.x & 31;
    for (int k = threadIdx.x >> 5; k < p.num_buckets; k += blockDim.x >> 5) {
        float s = 0.0f;
        for (int i = lane; i <= 2 * p.D; i += 32)
            if (p.buckets[i] == k) s += total[i];
        s = warp_sum(s);
        if (lane == 0) p.dtable[(int64_t)k * p.heads + head] = s;
    }
}

// The sums by distance of a block: arrays in shared memory, and what lies further away.
struct Distances {
    float *diagonals;
    int size, shift;
    float2 before, behind;                   // columns at distances up to -D, from D on
};

// The rows of a block.  PROBS: the probabilities are given; else they come from
// the scores and statistics, DROP with the forward pass's mask.
template <int NV, bool VEC, bool BLOCK, bool PROBS, bool DROP>
__device__ __forceinline__ void backward_rows(const Params &p, const Part &t, const float *bias, Distances &d,
                                              Exchange &exchange)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t call = DROP ? amsim::drop_call(p.drop) : 0;
    constexpr float kHidden = PROBS ? 0.0f : -INFINITY;
    int turn = 0;
    Place at = first_place(p, t.share);
    for (int g = t.share; g < p.groups; g += p.shares, turn ^= 1, advance(p, at)) {
        const Row w = row_of<BLOCK>(p, t.head, at.b, at.i);
        if (!BLOCK && !w.on) continue;
        const float *in = (PROBS ? p.probs : p.scores) + w.row * p.ld_in, *up = p.dprobs + w.row * p.ld_g;
        float *out = p.out + w.row * p.ld_out;
        float base = 0.0f, inv = 1.0f;
        if (!PROBS) {
            const float2 f = *reinterpret_cast<const float2 *>(p.stats + 2 * w.row);
            base = finite_base(f.x);
            inv = f.y;
        }
        const int origin = p.D + 4 - w.pos;              // entry of column 0
        RowDraws draws{};
        if (DROP) draws = row_draws(w.row, p, call);
        auto values = [&](auto full, int chunk, Four &a, Four &g) {
            constexpr bool FULL = decltype(full)::value;
            fill_chunk<VEC, FULL>(a, chunk, lane, w.visible, kHidden);
            fill_chunk<VEC, FULL>(g, chunk, lane, w.visible, 0.0f);
            if (PROBS || (!FULL && chunk * 128 >= w.visible)) return;
            if (p.table) add_bias<VEC>(a, bias, chunk, lane, w.pos, p);
            a = mul(exponentials(a, base), four(inv));
            hide<VEC, FULL>(a, chunk, lane, w.visible);
            if (DROP) drop_chunk<VEC>(g, draws, chunk, lane, p, call, p.drop.scale);
        };
        auto finish = [&](auto full, int chunk, float dot, Four a, const Four &g) {
            constexpr bool FULL = decltype(full)::value;
            const bool seen = FULL || chunk * 128 < w.visible;
            a = seen ? mul(a, add(g, four(-dot))) : four(0.0f);
            hide<VEC, FULL>(a, chunk, lane, w.visible);
            if (p.dtable && seen) {
                const int first = column<VEC>(chunk, lane, 0) + origin;
                if (VEC) {
                    if ((unsigned)first <= (unsigned)(2 * p.D + 5)) {
                        const int k = first & 3;
                        float4 *to = reinterpret_cast<float4 *>(BLOCK ? d.diagonals + k * d.size + (first - k)
                                                                      : d.diagonals + warp * d.size + (first + d.shift));
                        const float4 s = *to;
                        const Four v = add(a, Four{make_float2(s.x, s.y), make_float2(s.z, s.w)});
                        *to = make_float4(v.a.x, v.a.y, v.b.x, v.b.y);
                    } else if (first < 0) {
                        d.before = add2(d.before, add2(a.a, a.b));
                    } else {
                        d.behind = add2(d.behind, add2(a.a, a.b));
                    }
                } else {
                    const int low = chunk * 128 + origin;        // the chunk's first entry
                    if (low + 127 < 0) {                         // all of it far away
                        d.before = add2(d.before, add2(a.a, a.b));
                    } else if (low > 2 * p.D + 8) {
                        d.behind = add2(d.behind, add2(a.a, a.b));
                    } else {
                        float *to = d.diagonals + (BLOCK ? 0 : warp * d.size);
                        each(a, [&](float &x, int k) {
                            const int i = first + 32 * k;
                            if ((unsigned)i <= (unsigned)(2 * p.D + 8))
                                to[i] += x;
                            else if (i < 0)
                                d.before.x += x;
                            else
                                d.behind.x += x;
                        });
                    }
                }
            }
            store_chunk<VEC, FULL>(out, chunk, lane, p.keys, a);
        };
        Four part = four(0.0f);
        if (NV) {
            Four a[NV ? NV : 1], g[NV ? NV : 1];
            // `full`: every key of this warp's chunks is visible, and nothing has to be checked
            auto begin = [&](auto full) {
                constexpr bool FULL = decltype(full)::value;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int chunk = t.first_chunk + v * t.step;
                    a[v] = load_chunk<VEC, FULL>(in, chunk, lane, w.visible, kHidden);
                    g[v] = load_chunk<VEC, FULL>(up, chunk, lane, w.visible, 0.0f);
                }
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int chunk = t.first_chunk + v * t.step;
                    values(full, chunk, a[v], g[v]);
                    if (FULL || chunk * 128 < w.visible)
                        part = Four{fma2(a[v].a, g[v].a, part.a), fma2(a[v].b, g[v].b, part.b)};
                }
            };
            const bool all = (t.first_chunk + (NV - 1) * t.step + 1) * 128 <= w.visible;
            if (all)
                begin(std::true_type{});
            else
                begin(std::false_type{});
            const float dot = join_sums<BLOCK>(p, warp_sum(sum(part)), exchange, turn);
            auto end = [&](auto full) {
#pragma unroll
                for (int v = 0; v < NV; ++v) finish(full, t.first_chunk + v * t.step, dot, a[v], g[v]);
            };
            if (all)
                end(std::true_type{});
            else
                end(std::false_type{});
        } else {
            // two chunks at a time, whose loads are under way together
            std::false_type some;
            auto both_of = [&](int chunk, Four (&a)[2], Four (&g)[2]) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    a[v] = load_chunk<VEC>(in, chunk + v * t.step, lane, w.visible, kHidden);
                    g[v] = load_chunk<VEC>(up, chunk + v * t.step, lane, w.visible, 0.0f);
                }
#pragma unroll
                for (int v = 0; v < 2; ++v) values(some, chunk + v * t.step, a[v], g[v]);
            };
            Four a[2], g[2];
            for (int chunk = t.first_chunk; chunk * 128 < w.visible; chunk += 2 * t.step) {
                both_of(chunk, a, g);
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    if ((chunk + v * t.step) * 128 < w.visible)
                        part = Four{fma2(a[v].a, g[v].a, part.a), fma2(a[v].b, g[v].b, part.b)};
            }
            const float dot = join_sums<BLOCK>(p, warp_sum(sum(part)), exchange, turn);
            for (int chunk = t.first_chunk; chunk < p.chunks; chunk += 2 * t.step) {
                both_of(chunk, a, g);
#pragma unroll
                for (int v = 0; v < 2; ++v) finish(some, chunk + v * t.step, dot, a[v], g[v]);
            }
        }
        if (!BLOCK) __syncwarp();            // other lanes add to the same distances for the next row
    }
}

template <int NV, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(!BLOCK ? 32 * kWarpRows : NV == 4 ? kFewThreads : 1024, BLOCK ? 1 : 3) backward_kernel(const Params p)
{
    extern __shared__ __align__(16) float shared[];
    __shared__ Exchange exchange;
    __shared__ float ends[2][32];
    const Part t = part_of<BLOCK>(p);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // sums by distance: an array a warp, shifted by its rows' place modulo four
    // (BLOCK: four copies, as the bias has, since a block takes rows of every place)
    const int n = entries(p.D), arrays = BLOCK ? 4 : kWarpRows, size = n + 4;
    float *bias = shared, *diagonals = shared + (p.table ? 4 * n : 0);
    if (p.dtable)
        for (int i = threadIdx.x; i < arrays * size; i += blockDim.x) diagonals[i] = 0.0f;
    if (p.table) load_bias(p, t.head, bias);
    __syncthreads();
    Distances d{diagonals, size, VEC && !BLOCK ? (warp - p.D) & 3 : 0, both(0.0f), both(0.0f)};
    if (p.probs)
        backward_rows<NV, VEC, BLOCK, true, false>(p, t, bias, d, exchange);
    else if (p.drop.border)
        backward_rows<NV, VEC, BLOCK, false, true>(p, t, bias, d, exchange);
    else
        backward_rows<NV, VEC, BLOCK, false, false>(p, t, bias, d, exchange);
    if (BLOCK && p.cluster > 1) cluster_barrier();       // no block leaves while another reads from it
    if (!p.dtable) return;
    amsim::chain_start();
    const float low = warp_sum(d.before.x + d.before.y), high = warp_sum(d.behind.x + d.behind.y);
    if (lane == 0) {
        ends[0][warp] = low;
        ends[1][warp] = high;
    }
    __syncthreads();
    // the block's sum of an entry, in a fixed order
    auto entry = [&](int i) {
        float s = 0.0f;
        for (int k = 0; k < (BLOCK ? (VEC ? 4 : 1) : kWarpRows); ++k) {
            const int at = BLOCK ? i - k : VEC ? i + ((k - p.D) & 3) : i;
            if (at >= 0) s += diagonals[k * size + at];
        }
        return s;
    };
    float *total = p.shares * p.cluster > 1 ? p.part + (int64_t)blockIdx.x * (2 * p.D + 1) : bias;
    if (p.shares * p.cluster == 1 && !p.table) total = diagonals + arrays * size;
    for (int i = threadIdx.x; i <= 2 * p.D; i += blockDim.x) {
        float s = entry(i + 4);
        if (i == 0) {
            for (int j = 0; j < 4; ++j) s += entry(j);
            for (int k = 0; k < (int)(blockDim.x >> 5); ++k) s += ends[0][k];
        }
        if (i == 2 * p.D) {
            for (int j = 5; j <= 8; ++j) s += entry(2 * p.D + j);
            for (int k = 0; k < (int)(blockDim.x >> 5); ++k) s += ends[1][k];
        }
        total[i] = s;
    }
    if (p.shares * p.cluster > 1) return;
    __syncthreads();
    by_bucket(p, t.head, total);
}

// dtable from the blocks' sums by distance: a block per head and bucket, whose
// threads go through the bucket's distances in every block's sums.
constexpr int kTableThreads = 1024;
__global__ void __launch_bounds__(kTableThreads) table_kernel(const Params p)
{
    extern __shared__ __align__(16) int list[];          // the bucket's distances
    __shared__ int count;
    __shared__ float sums[32];
    const int n = 2 * p.D + 1, blocks = p.shares * p.cluster, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = (int)(blockIdx.x / (unsigned)p.num_buckets), k = (int)blockIdx.x - head * p.num_buckets;
    if (warp == 0) {
        int found = 0;
#pragma unroll 4
        for (int i = lane; i < n + lane; i += 32) {
            const bool mine = i < n && p.buckets[min(i, n - 1)] == k;
            const unsigned all = __ballot_sync(kAll, mine);
            if (mine) list[found + __popc(all & ((1u << lane) - 1))] = i;
            found += __popc(all);
        }
        if (lane == 0) count = found;
    }
    amsim::chain_wait();
    __syncthreads();
    const int each = count;
    const int64_t pairs = (int64_t)each * blocks;
    const float *part = p.part + (int64_t)head * blocks * n;
    // pair i is distance i % each of block i / each
    int t = each ? (int)threadIdx.x / each : 0, j = each ? (int)threadIdx.x % each : 0;
    const int dt = each ? kTableThreads / each : 0, dj = each ? kTableThreads % each : 0;
    float s = 0.0f;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < pairs; i += kTableThreads) {
        s += part[(int64_t)t * n + list[j]];
        t += dt;
        j += dj;
        if (j >= each) {
            j -= each;
            ++t;
        }
    }
    s = warp_sum(s);
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    if (warp) return;
    s = warp_sum(sums[lane]);
    if (lane == 0) p.dtable[(int64_t)k * p.heads + head] = s;
}

bool aligned(const void *q, size_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }
int64_t stride(int64_t ld, int64_t keys) { return ld ? ld : keys; }

int check(const amsim_attention_softmax_desc *d, Drop *drop)
{
    if (!d || d->batch < 0 || d->heads < 0 || d->queries < 0 || d->keys < 0 || d->reserved) return AMSIM_EINVAL;
    constexpr int64_t most = 0x7FFFFFFF - (1 << 20);         // indexes of rows stay in 32 bits a step behind the last
    for (int64_t n : {d->batch, d->heads, d->queries, d->keys})
        if (n > most) return AMSIM_EINVAL;
    if (d->keys > (int64_t)1 << 30) return AMSIM_EINVAL;             // columns of chunks behind the last fit 32 bits
    if (d->batch * d->queries > most || d->batch * d->queries * d->heads > (int64_t)1 << 40) return AMSIM_EINVAL;
    for (int64_t ld : {d->ld_scores, d->ld_probs, d->ld_dprobs, d->ld_dscores})
        if (ld != 0 && (ld < d->keys || ld > (int64_t)1 << 31)) return AMSIM_EINVAL;
    if (d->offset > (int64_t)1 << 40 || d->offset < -((int64_t)1 << 40)) return AMSIM_EINVAL;
    if ((d->causal != 0 && d->causal != 1) || !aligned(d->lengths, 4) || !aligned(d->offsets, 4)) return AMSIM_EINVAL;
    return amsim::make_drop(d->dropout, drop) ? AMSIM_OK : AMSIM_EINVAL;
}

// How rows are shared: up to four chunks by a warp, then by a block, four chunks a
// warp (what a row costs each warp is spread over 16 columns a lane), then by a
// cluster of blocks.  Backward keeps two tensors, and beyond 768 threads of them
// two chunks a warp.
// Rows that two blocks of 1024 threads do not hold are read twice where there are
// many (the second time from the cache) by clusters of eight small blocks, four or more an SM, whose
// loads, exchanges and stores overlap: 300 rows of 131072 keys 77 us, of blocks
// that fill an SM each and hold the row 133 us.  Few rows get those: one alone is
// done sooner the more threads it has.  The border is where the large blocks no longer
// fit the machine at once, some rows from where both are alike: of 131072 keys (eight
// blocks a row) 8 rows take 11.2 us in small and 7.4 in large blocks, 16 rows 12.4 and
// 13.8, 20 rows 12.8 and 14.4, 32 rows 13.7 and 21; of 40000 keys (three) 32 rows 8.2
// and 6.8, 38 rows 8.8 and 11.4, 64 rows 10.4 and 12.6.
constexpr int kMaxCluster = 8;
struct Shape {
    int nv, threads, cluster;
    bool block;
};
Shape shape(const amsim_attention_softmax_desc *d, bool fwd, int sms)
{
    const int64_t chunks = (d->keys + 127) / 128;
    Shape s{1, 32 * kWarpRows, 1, false};
    if (chunks <= 4) {
        while (s.nv < chunks) s.nv *= 2;
        return s;
    }
    s.block = true;
    s.nv = fwd || chunks <= 4 * kFewThreads / 32 ? 4 : 2;
    const int64_t blocks = (chunks + 32 * s.nv - 1) / (32 * s.nv), rows = d->batch * d->heads * d->queries;
    const bool many = rows * std::min<int64_t>(blocks, kMaxCluster) > (int64_t)sms;
    if (blocks > kMaxCluster || (blocks > 2 && many)) return Shape{0, many ? 256 : 1024, kMaxCluster, true};
    while (s.cluster < blocks) s.cluster *= 2;
    s.threads = 32 * (int)((chunks + s.nv * s.cluster - 1) / (s.nv * s.cluster));
    return s;
}

int64_t row_groups(const amsim_attention_softmax_desc *d, const Shape &s)
{
    return s.block ? d->queries : (d->queries + kWarpRows - 1) / kWarpRows;
}

template <bool VEC>
auto *forward_of(const Shape &s)
{
    if (!s.block)
        return s.nv == 1 ? forward_kernel<1, VEC, false> : s.nv == 2 ? forward_kernel<2, VEC, false>
                                                                     : forward_kernel<4, VEC, false>;
    return s.nv ? forward_kernel<4, VEC, true> : forward_kernel<0, VEC, true>;
}
template <bool VEC>
auto *backward_of(const Shape &s)
{
    if (!s.block)
        return s.nv == 1 ? backward_kernel<1, VEC, false> : s.nv == 2 ? backward_kernel<2, VEC, false>
                                                                      : backward_kernel<4, VEC, false>;
    return s.nv == 4   ? backward_kernel<4, VEC, true>
           : s.nv == 2 ? backward_kernel<2, VEC, true>
                       : backward_kernel<0, VEC, true>;
}

// Shared memory of the bias and of the sums by distance, and the most of it;
// every call that needs it sets this same limit, so that host threads do not lower one another's.
constexpr int entries_at(int D) { return (2 * D + 15) & ~3; }
constexpr int shared_bytes(int D, bool table, bool dtable, int arrays)
{
    return 4 * ((table ? 4 * entries_at(D) : 0) + (dtable ? arrays * (entries_at(D) + 4) + (table ? 0 : 2 * D + 1) : 0));
}
constexpr int kMaxShared = shared_bytes(AMSIM_MAX_DISTANCE, true, true, kWarpRows);

// How many of a kernel's blocks an SM holds; asked once for each kernel and shape.
int resident_blocks(void (*kernel)(Params), int threads, int bytes)
{
    struct Known {
        void (*kernel)(Params);
        int threads, bytes, count;
    };
    constexpr int kMost = 64;
    static std::mutex mutex;
    static Known known[kMost];
    static int held, next;
    std::lock_guard<std::mutex> lock(mutex);
    for (int i = 0; i < held; ++i)
        if (known[i].kernel == kernel && known[i].threads == threads && known[i].bytes == bytes) return known[i].count;
    int count = 0;
    if (bytes > 48 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&count, kernel, threads, (size_t)bytes) != cudaSuccess || count < 1) {
        cudaGetLastError();
        return std::max(1, 1024 / threads);              // no device here
    }
    known[next] = Known{kernel, threads, bytes, count};
    held = std::max(held, next + 1);
    next = (next + 1) % kMost;
    return count;
}

// Shares of a head's groups of rows: as many blocks as the SMs hold at once, no more than groups.
int share_count(const amsim_attention_softmax_desc *d, const Shape &s, void (*kernel)(Params), int bytes, int sms)
{
    const int64_t groups = d->batch * row_groups(d, s);
    const int64_t blocks = (int64_t)sms * resident_blocks(kernel, s.threads, bytes) / s.cluster;
    return (int)std::max<int64_t>(1, std::min(blocks / std::max<int64_t>(1, d->heads), groups));
}

int launch(void (*kernel)(Params), const Params &p, const Shape &s, int bytes, cudaStream_t st)
{
    if (bytes > 48 * 1024) {
        const int rc = amsim::cuda_status(
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared));
        if (rc) return rc;
    }
    const int64_t grid = (int64_t)p.heads * p.shares * p.cluster;
    if (grid > 0x7FFFFFFF) return AMSIM_EINVAL;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = dim3((unsigned)s.threads);
    c.dynamicSmemBytes = (size_t)bytes;
    c.stream = st;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = (unsigned)p.cluster;
    a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
    c.attrs = a;
    c.numAttrs = p.cluster > 1 ? 1 : 0;
    const int rc = amsim::cuda_status(cudaLaunchKernelEx(&c, kernel, p));
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}

void fill(Params &p, const amsim_attention_softmax_desc *d, const Shape &s, int shares)
{
    p.lengths = d->lengths;
    p.offsets = d->offsets;
    p.offset = d->offset;
    p.queries = (int)d->queries;
    p.keys = (int)d->keys;
    p.quads = (int)((d->keys + 3) / 4);
    p.chunks = (int)((d->keys + 127) / 128);
    p.heads = (int)d->heads;
    p.row_groups = (int)row_groups(d, s);
    p.groups = (int)(d->batch * p.row_groups);
    p.shares = shares;
    p.ahead_b = shares / p.row_groups;
    p.ahead_i = shares % p.row_groups;
    p.cluster = s.cluster;
    p.causal = d->causal;
}

int check_bias(const amsim_attention_softmax_desc *d, Params &p)
{
    if (!aligned(p.table, 4) || !aligned(p.buckets, 4) || d->num_buckets < 1 || d->max_distance < 0) return AMSIM_EINVAL;
    if ((int64_t)d->num_buckets * d->heads > 0x7FFFFFFF) return AMSIM_EINVAL;
    if (d->max_distance > AMSIM_MAX_DISTANCE) return AMSIM_EUNSUPPORTED;
    p.num_buckets = d->num_buckets;
    p.D = d->max_distance;
    return AMSIM_OK;
}

int device_sms()
{
    int sms = 0;
    return amsim::current_device(&sms) < 0 ? 0 : sms;
}

}  // namespace

extern "C" int amsim_attention_softmax_fwd(const amsim_attention_softmax_desc *d, const float *scores,
                                           const float *table, const int32_t *buckets, float *probs, float *stats,
                                           amsim_stream_t stream)
{
    Params p{};
    int rc = check(d, &p.drop);
    if (rc) return rc;
    if (!table != !buckets) return AMSIM_EINVAL;
    p.table = table;
    p.buckets = buckets;
    if (table && (rc = check_bias(d, p))) return rc;
    if (!d->batch || !d->heads || !d->queries || !d->keys) return AMSIM_OK;
    if (!scores || !probs || !aligned(scores, 4) || !aligned(probs, 4) || !aligned(stats, 8)) return AMSIM_EINVAL;
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    const Shape s = shape(d, true, sms);
    const bool vec = aligned(scores, 16) && aligned(probs, 16) && !((d->keys | stride(d->ld_scores, d->keys) |
                                                                     stride(d->ld_probs, d->keys)) & 3);
    auto *kernel = vec ? forward_of<true>(s) : forward_of<false>(s);
    const int bytes = shared_bytes(p.D, table, false, 0);
    fill(p, d, s, share_count(d, s, kernel, bytes, sms));
    p.scores = scores;
    p.out = probs;
    p.out_stats = stats;
    p.ld_in = stride(d->ld_scores, d->keys);
    p.ld_out = stride(d->ld_probs, d->keys);
    return launch(kernel, p, s, bytes, static_cast<cudaStream_t>(stream));
}

extern "C" size_t amsim_attention_softmax_workspace_size(const amsim_attention_softmax_desc *d)
{
    Drop drop;
    if (check(d, &drop) || d->num_buckets < 0 || d->max_distance < 0 || d->max_distance > AMSIM_MAX_DISTANCE) return 0;
    if (!d->batch || !d->heads || !d->queries || !d->keys) return 0;
    const int sms = device_sms();
    const Shape s = shape(d, false, sms ? sms : 1);
    int shares = 0;
    for (const bool vec : {false, true})         // the calls' pointers and arguments decide which
        for (const bool table : {false, true})
            shares = std::max(shares, share_count(d, s, vec ? backward_of<true>(s) : backward_of<false>(s),
                                                  shared_bytes(d->max_distance, table, true, s.block ? 4 : kWarpRows),
                                                  sms ? sms : 1));
    const int64_t blocks = (int64_t)shares * s.cluster;
    return blocks > 1 ? (size_t)d->heads * blocks * (2 * d->max_distance + 1) * 4 : 0;
}

extern "C" int amsim_attention_softmax_bwd(const amsim_attention_softmax_desc *d, const float *dprobs,
                                           const float *scores, const float *stats, const float *probs,
                                           const float *table, const int32_t *buckets, float *dscores, float *dtable,
                                           void *ws, size_t ws_bytes, amsim_stream_t stream)
{
    Params p{};
    int rc = check(d, &p.drop);
    if (rc) return rc;
    if ((table || dtable) && !buckets) return AMSIM_EINVAL;
    if (probs && (p.drop.border || scores || table)) return AMSIM_EINVAL;
    p.table = table;
    p.buckets = buckets;
    p.dtable = dtable;
    if ((table || dtable) && (rc = check_bias(d, p))) return rc;
    if (!aligned(dtable, 4) || !aligned(ws, 4)) return AMSIM_EINVAL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!d->batch || !d->heads || !d->queries || !d->keys) {
        if (dtable && d->heads)
            return amsim::cuda_status(cudaMemsetAsync(dtable, 0, (size_t)p.num_buckets * (size_t)d->heads * 4, st));
        return AMSIM_OK;
    }
    if (!dprobs || !dscores || (!scores && !probs) || (scores && !stats)) return AMSIM_EINVAL;
    for (const float *f : {dprobs, scores, probs, (const float *)dscores})
        if (!aligned(f, 4)) return AMSIM_EINVAL;
    if (!aligned(stats, 8)) return AMSIM_EINVAL;
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    const bool vec = aligned(scores, 16) && aligned(probs, 16) && aligned(dprobs, 16) && aligned(dscores, 16) &&
                     !((d->keys | stride(scores ? d->ld_scores : d->ld_probs, d->keys) |
                        stride(d->ld_dprobs, d->keys) | stride(d->ld_dscores, d->keys)) & 3);
    Shape s = shape(d, false, sms);
    const size_t one = (size_t)d->heads * (2 * p.D + 1) * 4, room = ws ? ws_bytes / one : 0;
    if (dtable && s.cluster > 1 && room < (size_t)s.cluster)
        s = Shape{0, 1024, 1, true};             // no room for a cluster's sums: one block, rows read twice
    auto *kernel = vec ? backward_of<true>(s) : backward_of<false>(s);
    const int bytes = shared_bytes(p.D, table, dtable, s.block ? 4 : kWarpRows);
    int shares = share_count(d, s, kernel, bytes, sms);
    if (dtable) shares = (int)std::max<size_t>(1, std::min<size_t>(shares, room / s.cluster));
    fill(p, d, s, shares);
    p.dprobs = dprobs;
    p.scores = scores;
    p.stats = stats;
    p.probs = probs;
    p.out = dscores;
    p.part = static_cast<float *>(ws);
    p.ld_in = stride(scores ? d->ld_scores : d->ld_probs, d->keys);
    p.ld_g = stride(d->ld_dprobs, d->keys);
    p.ld_out = stride(d->ld_dscores, d->keys);
    rc = launch(kernel, p, s, bytes, st);
    if (rc || !dtable || p.shares * p.cluster == 1) return rc;
    rc = amsim::cuda_status(amsim::chain_launch(true, table_kernel, dim3((unsigned)(p.heads * p.num_buckets)),
                                                kTableThreads, 4 * (2 * p.D + 1), st, p));
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}
