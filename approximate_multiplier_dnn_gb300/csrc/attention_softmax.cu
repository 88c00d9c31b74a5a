// The softmax between attention's contractions, with a relative position bias,
// lengths, a causal mask and dropout, and its gradient with the bias table's.
//
// A row is read once and kept in registers, a quad of columns at a time per
// thread, so the traffic is the compulsory one: scores in, probabilities out.
// Blocks belong to one head and keep its bias by distance in shared memory.
// dtable wants the sum of dS along each diagonal of the scores (one distance,
// all of a head's rows): within a row every distance inside (-D, D) occurs at
// one column, so a warp (or the block that shares a row) adds its row to an
// array by distance in shared memory without conflicts; columns further away
// go to two registers.  The arrays are added in a fixed order, then by bucket.
#include <algorithm>

#include "chained.cuh"
#include "philox.cuh"

namespace {

using amsim::Drop;

struct Params {
    const float *scores, *probs, *dprobs, *stats, *table;   // inputs
    const int32_t *buckets, *lengths, *offsets;
    float *out, *out_stats, *dtable, *part;
    int64_t queries, ld_in, ld_g, ld_out, offset;            // ld_in: of scores or probs
    int keys, heads, rows, share_rows, shares;               // rows: of one head
    int causal, num_buckets, D;
    Drop drop;
};

constexpr int kWarpRows = 8;                 // warps of a block that each take a row
constexpr unsigned kAll = 0xFFFFFFFFu;

// Arrays by distance: lanes read and write every fourth entry at a time, and a
// word more every 32 lets those fall into 32 banks.
__host__ __device__ __forceinline__ int place(int i) { return i + (i >> 5); }
__host__ __device__ __forceinline__ int places(int D) { return place(2 * D) + 1; }

// One row: where it is, what it sees, and its query's place, brought near enough for 32 bits.
struct Row {
    int64_t row;
    int visible, pos;
};
__device__ __forceinline__ Row row_of(const Params &p, int head, int r)
{
    const int b = (int)((unsigned)r / (unsigned)p.queries), i = r - b * (int)p.queries;
    Row w;
    w.row = ((int64_t)b * p.heads + head) * p.queries + i;
    const int64_t pos = (p.offsets ? (int64_t)p.offsets[b] : p.offset) + i;
    int64_t end = p.keys;
    if (p.lengths) end = min(end, (int64_t)max(p.lengths[b], 0));
    if (p.causal) end = min(end, max(pos + 1, (int64_t)0));
    w.visible = (int)end;
    w.pos = (int)max(min(pos, (int64_t)p.keys + p.D), -(int64_t)p.D - 1);
    return w;
}

template <bool VEC>
__device__ __forceinline__ void load_quad(const float *row, int col, int limit, float fill, float (&v)[4])
{
    if (VEC) {
        float4 f = make_float4(fill, fill, fill, fill);
        if (col < limit) f = *reinterpret_cast<const float4 *>(row + col);
        v[0] = f.x;
        v[1] = col + 1 < limit ? f.y : fill;
        v[2] = col + 2 < limit ? f.z : fill;
        v[3] = col + 3 < limit ? f.w : fill;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = col + k < limit ? row[col + k] : fill;
    }
}

template <bool VEC>
__device__ __forceinline__ void store_quad(float *row, int col, int keys, const float (&v)[4])
{
    if (VEC) {
        if (col < keys) *reinterpret_cast<float4 *>(row + col) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (col + k < keys) row[col + k] = v[k];
    }
}

// The head's bias by distance, into shared memory.
__device__ __forceinline__ void load_bias(const Params &p, int head, float *bias)
{
    for (int i = threadIdx.x; i <= 2 * p.D; i += blockDim.x) {
        const int k = p.buckets[i];
        bias[place(i)] = (unsigned)k < (unsigned)p.num_buckets ? p.table[(int64_t)k * p.heads + head] : 0.0f;
    }
    __syncthreads();
}
__device__ __forceinline__ void add_bias(const Params &p, const float *bias, int col, int pos, float (&v)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += bias[place(min(max(col + k - pos + p.D, 0), 2 * p.D))];
}

// Maximum or sum over the threads of a row: a warp's, or (BLOCK) the block's.
template <bool BLOCK, bool MAX>
__device__ __forceinline__ float reduce(float v, float *shared)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float o = __shfl_xor_sync(kAll, v, d);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    if (BLOCK) {
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();                     // the values of the reduction before have been read
        if (lane == 0) shared[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? shared[lane] : MAX ? -INFINITY : 0.0f;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const float o = __shfl_xor_sync(kAll, v, d);
            v = MAX ? fmaxf(v, o) : v + o;
        }
    }
    return v;
}

__device__ __forceinline__ float finite_base(float top) { return top == -INFINITY ? 0.0f : top; }

// Probabilities of a quad from its exponentials: dropout, zeros where no key is visible.
__device__ __forceinline__ void finish_probs(const Params &p, const Row &w, int col, uint64_t call, float inv, float (&v)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = col + k < w.visible ? v[k] * inv : 0.0f;
    if (p.drop.border && col < w.visible)
        amsim::drop_quad(v, (uint64_t)w.row * (unsigned)((p.keys + 3) >> 2) + (unsigned)(col >> 2), p.drop, call);
}

// NV > 0: the row's quads stay in NV x 4 registers a thread; NV == 0: a row of
// any length, read twice.
template <int NV, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kWarpRows) forward_kernel(const Params p)
{
    extern __shared__ float shared[];
    __shared__ float sums[32];
    const int head = blockIdx.x / p.shares, share = blockIdx.x % p.shares;
    const int width = BLOCK ? blockDim.x : 32, lane = BLOCK ? threadIdx.x : threadIdx.x & 31;
    if (p.table) load_bias(p, head, shared);
    const uint64_t call = amsim::drop_call(p.drop);
    const int last = min(p.rows, (share + 1) * p.share_rows);
    for (int r = share * p.share_rows + (BLOCK ? 0 : threadIdx.x >> 5); r < last; r += BLOCK ? 1 : kWarpRows) {
        const Row w = row_of(p, head, r);
        const float *in = p.scores + w.row * p.ld_in;
        float *out = p.out + w.row * p.ld_out;
        float top = -INFINITY, sum = 0.0f, base, inv;
        auto quad = [&](int col, float (&v)[4]) {
            load_quad<VEC>(in, col, w.visible, -INFINITY, v);
            if (p.table) add_bias(p, shared, col, w.pos, v);
        };
        if (NV) {
            float a[NV ? NV : 1][4];
#pragma unroll
            for (int v = 0; v < NV; ++v) quad(4 * (lane + v * width), a[v]);
#pragma unroll
            for (int v = 0; v < NV; ++v) top = fmaxf(fmaxf(fmaxf(top, a[v][0]), fmaxf(a[v][1], a[v][2])), a[v][3]);
            top = reduce<BLOCK, true>(top, sums);
            base = finite_base(top);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int k = 0; k < 4; ++k) sum += a[v][k] = expf(a[v][k] - base);
            sum = reduce<BLOCK, false>(sum, sums);
            inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int col = 4 * (lane + v * width);
                finish_probs(p, w, col, call, inv, a[v]);
                store_quad<VEC>(out, col, p.keys, a[v]);
            }
        } else {
            for (int col = 4 * lane; col < w.visible; col += 4 * width) {
                float a[4];
                quad(col, a);
                const float most = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                if (most > top) {
                    sum *= expf(top - most);             // exp(-infinity) = 0 the first time
                    top = most;
                }
                base = finite_base(top);
#pragma unroll
                for (int k = 0; k < 4; ++k) sum += expf(a[k] - base);
            }
            const float mine = top;
            top = reduce<BLOCK, true>(top, sums);
            base = finite_base(top);
            sum = reduce<BLOCK, false>(mine == -INFINITY ? sum : sum * expf(mine - base), sums);
            inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            for (int col = 4 * lane; col < p.keys; col += 4 * width) {
                float a[4];
                quad(col, a);
#pragma unroll
                for (int k = 0; k < 4; ++k) a[k] = expf(a[k] - base);
                finish_probs(p, w, col, call, inv, a);
                store_quad<VEC>(out, col, p.keys, a);
            }
        }
        if (p.out_stats && lane == 0) {
            p.out_stats[2 * w.row] = top;
            p.out_stats[2 * w.row + 1] = inv;
        }
    }
}

// dtable of a head from its sums by distance; each warp takes buckets of its own.
__device__ __forceinline__ void by_bucket(const Params &p, int head, const float *total)
{
    const int lane = threadIdx.x & 31;
    for (int k = threadIdx.x >> 5; k < p.num_buckets; k += blockDim.x >> 5) {
        float s = 0.0f;
        for (int i = lane; i <= 2 * p.D; i += 32)
            if (p.buckets[i] == k) s += total[place(i)];
        s = reduce<false, false>(s, nullptr);
        if (lane == 0) p.dtable[(int64_t)k * p.heads + head] = s;
    }
}

template <int NV, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kWarpRows) backward_kernel(const Params p)
{
    extern __shared__ float shared[];
    __shared__ float sums[32];
    const int head = blockIdx.x / p.shares, share = blockIdx.x % p.shares;
    const int width = BLOCK ? blockDim.x : 32, lane = BLOCK ? threadIdx.x : threadIdx.x & 31;
    const int size = places(p.D), teams = BLOCK ? 1 : kWarpRows;
    float *bias = shared, *diagonals = shared + (p.table ? size : 0);
    float *mine = diagonals + (BLOCK ? 0 : (threadIdx.x >> 5) * size);
    if (p.dtable)
        for (int i = threadIdx.x; i < teams * size; i += blockDim.x) diagonals[i] = 0.0f;
    if (p.table)
        load_bias(p, head, bias);
    else
        __syncthreads();
    const uint64_t call = amsim::drop_call(p.drop);
    float before = 0.0f, behind = 0.0f;      // columns at distances up to -D, from D on
    const int last = min(p.rows, (share + 1) * p.share_rows);
    for (int r = share * p.share_rows + (BLOCK ? 0 : threadIdx.x >> 5); r < last; r += BLOCK ? 1 : kWarpRows) {
        const Row w = row_of(p, head, r);
        const float *in = (p.probs ? p.probs : p.scores) + w.row * p.ld_in, *up = p.dprobs + w.row * p.ld_g;
        float *out = p.out + w.row * p.ld_out;
        float base = 0.0f, inv = 1.0f;
        if (!p.probs) {
            base = finite_base(p.stats[2 * w.row]);
            inv = p.stats[2 * w.row + 1];
        }
        auto load = [&](int col, float (&a)[4], float (&g)[4]) {
            load_quad<VEC>(in, col, w.visible, p.probs ? 0.0f : -INFINITY, a);
            load_quad<VEC>(up, col, w.visible, 0.0f, g);
        };
        auto values = [&](int col, float (&a)[4], float (&g)[4]) {
            if (!p.probs) {
                if (p.table) add_bias(p, bias, col, w.pos, a);
#pragma unroll
                for (int k = 0; k < 4; ++k) a[k] = col + k < w.visible ? expf(a[k] - base) * inv : 0.0f;
                if (p.drop.border && col < w.visible)
                    amsim::drop_quad(g, (uint64_t)w.row * (unsigned)((p.keys + 3) >> 2) + (unsigned)(col >> 2), p.drop,
                                     call);
            }
        };
        auto finish = [&](int col, float dot, float (&a)[4], const float (&g)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = col + k < w.visible ? a[k] * (g[k] - dot) : 0.0f;
            if (p.dtable) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = col + k - w.pos + p.D;
                    if (i <= 0)
                        before += a[k];
                    else if (i >= 2 * p.D)
                        behind += a[k];
                    else if (col + k < w.visible)
                        mine[place(i)] += a[k];
                }
            }
            store_quad<VEC>(out, col, p.keys, a);
        };
        float dot = 0.0f;
        if (NV) {
            float a[NV ? NV : 1][4], g[NV ? NV : 1][4];
#pragma unroll
            for (int v = 0; v < NV; ++v) load(4 * (lane + v * width), a[v], g[v]);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                values(4 * (lane + v * width), a[v], g[v]);
#pragma unroll
                for (int k = 0; k < 4; ++k) dot = fmaf(a[v][k], g[v][k], dot);
            }
            dot = reduce<BLOCK, false>(dot, sums);
#pragma unroll
            for (int v = 0; v < NV; ++v) finish(4 * (lane + v * width), dot, a[v], g[v]);
        } else {
            float a[4], g[4];
            for (int col = 4 * lane; col < w.visible; col += 4 * width) {
                load(col, a, g);
                values(col, a, g);
#pragma unroll
                for (int k = 0; k < 4; ++k) dot = fmaf(a[k], g[k], dot);
            }
            dot = reduce<BLOCK, false>(dot, sums);
            for (int col = 4 * lane; col < p.keys; col += 4 * width) {
                load(col, a, g);
                values(col, a, g);
                finish(col, dot, a, g);
            }
        }
        if (!BLOCK) __syncwarp();            // other lanes add to the same distances for the next row
    }
    if (!p.dtable) return;
    amsim::chain_start();
    before = reduce<BLOCK, false>(before, sums);
    behind = reduce<BLOCK, false>(behind, sums);
    __syncthreads();
    if (lane == 0) {
        mine[place(0)] += before;
        mine[place(2 * p.D)] += behind;
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= 2 * p.D; i += blockDim.x) {
        float s = diagonals[place(i)];
        for (int t = 1; t < teams; ++t) s += diagonals[t * size + place(i)];
        if (p.shares > 1)
            p.part[(int64_t)blockIdx.x * (2 * p.D + 1) + i] = s;
        else
            diagonals[place(i)] = s;         // read by this thread alone so far
    }
    if (p.shares > 1) return;
    __syncthreads();
    by_bucket(p, head, diagonals);
}

// dtable from the shares' sums by distance: a block per head.
constexpr int kTableThreads = 1024;
__global__ void __launch_bounds__(kTableThreads) table_kernel(const Params p)
{
    extern __shared__ float shared[];
    amsim::chain_wait();
    const int n = 2 * p.D + 1;
    const float *part = p.part + (int64_t)blockIdx.x * p.shares * n;
    for (int i = threadIdx.x; i < n; i += kTableThreads) {
        float s = 0.0f;
#pragma unroll 8
        for (int t = 0; t < p.shares; ++t) s += part[(int64_t)t * n + i];
        shared[place(i)] = s;
    }
    __syncthreads();
    by_bucket(p, (int)blockIdx.x, shared);
}

bool aligned(const void *q, size_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }
int64_t stride(int64_t ld, int64_t keys) { return ld ? ld : keys; }

int check(const amsim_attention_softmax_desc *d, Drop *drop)
{
    if (!d || d->batch < 0 || d->heads < 0 || d->queries < 0 || d->keys < 0 || d->reserved) return AMSIM_EINVAL;
    constexpr int64_t most = 0x7FFFFFFF - 4096;
    for (int64_t n : {d->batch, d->heads, d->queries, d->keys})
        if (n > most) return AMSIM_EINVAL;
    if (d->batch * d->queries > most || d->batch * d->queries * d->heads > (int64_t)1 << 40) return AMSIM_EINVAL;
    for (int64_t ld : {d->ld_scores, d->ld_probs, d->ld_dprobs, d->ld_dscores})
        if (ld != 0 && (ld < d->keys || ld > (int64_t)1 << 31)) return AMSIM_EINVAL;
    if (d->offset > (int64_t)1 << 40 || d->offset < -((int64_t)1 << 40)) return AMSIM_EINVAL;
    if ((d->causal != 0 && d->causal != 1) || !aligned(d->lengths, 4) || !aligned(d->offsets, 4)) return AMSIM_EINVAL;
    if (d->num_buckets < 0 || d->max_distance < 0) return AMSIM_EINVAL;
    return amsim::make_drop(d->dropout, drop) ? AMSIM_OK : AMSIM_EINVAL;
}

// Threads of a row and quads a thread: a warp up to 1024 columns, then a block
// of up to 1024 threads; longer rows are read twice.
struct Shape {
    int nv, threads;
    bool block;
};
Shape shape(int64_t keys)
{
    const int64_t quads = (keys + 3) / 4;
    Shape s{1, 32 * kWarpRows, false};
    if (quads <= 256) {
        while (32 * s.nv < quads) s.nv *= 2;
        return s;
    }
    s.block = true;
    s.nv = quads <= 4096 ? 4 : 0;
    s.threads = s.nv ? (int)((quads + s.nv * 32 - 1) / (s.nv * 32)) * 32 : 1024;
    return s;
}

// Shares of a head's rows: as many blocks as fill the SMs, no more than rows.
int share_count(const amsim_attention_softmax_desc *d, const Shape &s, int sms)
{
    const int64_t rows = d->batch * d->queries, at_once = s.block ? 1 : kWarpRows;
    const int64_t want = std::max<int64_t>(1, (int64_t)sms * std::max(1, 2048 / s.threads) / std::max<int64_t>(1, d->heads));
    return (int)std::min(want, (rows + at_once - 1) / at_once);
}

template <bool VEC>
auto *forward_of(const Shape &s)
{
    if (!s.block)
        return s.nv == 1 ? forward_kernel<1, VEC, false> : s.nv == 2 ? forward_kernel<2, VEC, false>
               : s.nv == 4 ? forward_kernel<4, VEC, false> : forward_kernel<8, VEC, false>;
    return s.nv ? forward_kernel<4, VEC, true> : forward_kernel<0, VEC, true>;
}
template <bool VEC>
auto *backward_of(const Shape &s)
{
    if (!s.block)
        return s.nv == 1 ? backward_kernel<1, VEC, false> : s.nv == 2 ? backward_kernel<2, VEC, false>
               : s.nv == 4 ? backward_kernel<4, VEC, false> : backward_kernel<8, VEC, false>;
    return s.nv ? backward_kernel<4, VEC, true> : backward_kernel<0, VEC, true>;
}

// The most shared memory a kernel here takes; every call sets this same limit,
// so that host threads do not lower one another's.
constexpr int kMaxShared = (kWarpRows + 1) * (2 * AMSIM_MAX_DISTANCE + 2 * AMSIM_MAX_DISTANCE / 32 + 1) * 4;

int launch(void (*kernel)(Params), const Params &p, const Shape &s, int bytes, cudaStream_t st)
{
    if (bytes > 48 * 1024) {
        const int rc = amsim::cuda_status(
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared));
        if (rc) return rc;
    }
    const int64_t grid = (int64_t)p.heads * p.shares;
    if (grid > 0x7FFFFFFF) return AMSIM_EINVAL;
    kernel<<<(unsigned)grid, s.threads, bytes, st>>>(p);
    const int rc = amsim::cuda_status(cudaGetLastError());
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}

void fill(Params &p, const amsim_attention_softmax_desc *d)
{
    p.lengths = d->lengths;
    p.offsets = d->offsets;
    p.offset = d->offset;
    p.queries = d->queries;
    p.keys = (int)d->keys;
    p.heads = (int)d->heads;
    p.rows = (int)(d->batch * d->queries);
    p.causal = d->causal;
}

void share_rows(Params &p, int shares)
{
    p.share_rows = (p.rows + shares - 1) / shares;
    p.shares = (p.rows + p.share_rows - 1) / p.share_rows;
}

int check_bias(const amsim_attention_softmax_desc *d, Params &p)
{
    if (!aligned(p.table, 4) || !aligned(p.buckets, 4) || d->num_buckets < 1) return AMSIM_EINVAL;
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
    if (!scores || !probs || !aligned(scores, 4) || !aligned(probs, 4) || !aligned(stats, 4)) return AMSIM_EINVAL;
    fill(p, d);
    p.scores = scores;
    p.out = probs;
    p.out_stats = stats;
    p.ld_in = stride(d->ld_scores, d->keys);
    p.ld_out = stride(d->ld_probs, d->keys);
    const bool vec = aligned(scores, 16) && aligned(probs, 16) && !((d->keys | p.ld_in | p.ld_out) & 3);
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    const Shape s = shape(d->keys);
    share_rows(p, share_count(d, s, sms));
    return launch(vec ? forward_of<true>(s) : forward_of<false>(s), p, s, table ? 4 * places(p.D) : 0,
                  static_cast<cudaStream_t>(stream));
}

extern "C" size_t amsim_attention_softmax_workspace_size(const amsim_attention_softmax_desc *d)
{
    Drop drop;
    if (check(d, &drop) || d->max_distance > AMSIM_MAX_DISTANCE) return 0;
    if (!d->batch || !d->heads || !d->queries || !d->keys) return 0;
    const int sms = device_sms();
    const int shares = share_count(d, shape(d->keys), sms ? sms : 1);
    return shares > 1 ? (size_t)d->heads * shares * (2 * d->max_distance + 1) * 4 : 0;
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
    for (const float *f : {dprobs, scores, stats, probs, (const float *)dscores})
        if (!aligned(f, 4)) return AMSIM_EINVAL;
    fill(p, d);
    p.dprobs = dprobs;
    p.scores = scores;
    p.stats = stats;
    p.probs = probs;
    p.out = dscores;
    p.ld_in = stride(scores ? d->ld_scores : d->ld_probs, d->keys);
    p.ld_g = stride(d->ld_dprobs, d->keys);
    p.ld_out = stride(d->ld_dscores, d->keys);
    const bool vec = aligned(scores, 16) && aligned(probs, 16) && aligned(dprobs, 16) && aligned(dscores, 16) &&
                     !((d->keys | p.ld_in | p.ld_g | p.ld_out) & 3);
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    const Shape s = shape(d->keys);
    int shares = share_count(d, s, sms);
    if (dtable) {
        const size_t one = (size_t)d->heads * (2 * p.D + 1) * 4;
        shares = (int)std::max<size_t>(1, std::min<size_t>(shares, ws ? ws_bytes / one : 1));
    }
    share_rows(p, shares);
    p.part = static_cast<float *>(ws);
    const int arrays = (table ? 1 : 0) + (dtable ? (s.block ? 1 : kWarpRows) : 0);
    rc = launch(vec ? backward_of<true>(s) : backward_of<false>(s), p, s, arrays * 4 * places(p.D), st);
    if (rc || !dtable || p.shares == 1) return rc;
    rc = amsim::cuda_status(amsim::chain_launch(true, table_kernel, dim3((unsigned)p.heads), kTableThreads,
                                                4 * places(p.D), st, p));
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}
