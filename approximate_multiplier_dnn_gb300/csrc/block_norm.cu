// The block norm's entry points: argument checks, launch shapes, and the
// kernel that adds the backward pass's column sums.
#include <algorithm>
#include <cmath>

#include "block_norm.cuh"

namespace {

using amsim::bn::Params;

// dgate, dw_post and dw_pre from the shares' sums, in a fixed order: a block
// takes 32 channels, its 32 warps every 32nd share, eight loads at a time.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) sums_kernel(const Params p, int blocks)
{
    __shared__ float part[kSumWarps][33];
    amsim::chain_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (int)blockIdx.x * 32 + lane;
    const bool on = c < p.cols;
    auto total = [&](const float *src, long long n) {
        float s = 0.0f;
        if (on) {
#pragma unroll 8
            for (long long i = warp; i < n; i += kSumWarps) s += src[i * p.cols + c];
        }
        __syncthreads();
        part[warp][lane] = s;
        __syncthreads();
        s = part[lane][warp];                  // channel `warp` of the block: its shares across the lanes
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        return s;                              // every lane of warp i: channel i
    };
    const int mine = (int)blockIdx.x * 32 + warp;
    const bool out = lane == 0 && mine < p.cols;
    if (blockIdx.y == 0) {
        if (!p.dw_pre || !p.part_pre) return;
        const float s = total(p.part_pre, blocks);
        if (out) p.dw_pre[mine] = s;
        return;
    }
    if (p.splits == 1) {
        if (!p.dw_post || !p.part_post) return;
        const float s = total(p.part_post, blocks);
        if (out) p.dw_post[mine] = s;
        return;
    }
    if (!p.part_gate) return;
    // as many rows of the gate at once as the warps make, `per` warps each (8 of
    // them at 16384 x 4096, one after the other with all warps: 18 us)
    const long long groups = p.items / p.splits;
    int per = kSumWarps;
    while (per > 1 && kSumWarps / per < groups) per >>= 1;
    const float w = mine < p.cols && p.w_post ? p.w_post[mine] : 1.0f;
    float dw = 0.0f;
    for (long long g0 = 0; g0 < groups; g0 += kSumWarps / per) {
        const long long from = g0 + warp / per;
        float s = 0.0f;
        if (on && from < groups) {
            const float *src = p.part_gate + from * p.splits * p.cols + c;
#pragma unroll 8
            for (int i = warp % per; i < p.splits; i += per) s += src[(long long)i * p.cols];
        }
        __syncthreads();
        part[warp][lane] = s;
        __syncthreads();
        s = part[lane][warp];                  // channel `warp` of the block: the gate's rows across the lanes
        for (int d = 1; d < per; d <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        const long long g = g0 + lane / per;
        float add = 0.0f;
        if (lane % per == 0 && mine < p.cols && g < groups) {
            if (p.dgate) p.dgate[g * p.cols + mine] = p.alpha * w * s;
            add = p.alpha * (p.gate ? p.gate[g * p.cols + mine] : 1.0f) * s;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) add += __shfl_xor_sync(0xFFFFFFFFu, add, d);
        dw += add;
    }
    if (out && p.dw_post) p.dw_post[mine] = dw;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// Rows that take a thread's four channels as one load, and rows that start and end on 16 bytes.
bool vector_rows(const void *p, int64_t ld, size_t size)
{
    return !p || (aligned(p, 4 * size) && ld % 4 == 0);
}
bool bulk_rows(const void *p, int64_t ld, size_t size, int cols)
{
    return !p || (aligned(p, 16) && ld * (int64_t)size % 16 == 0 && cols * size % 16 == 0);
}
size_t type_size(int t) { return t == AMSIM_BF16 ? 2 : 4; }
int64_t stride(int64_t ld, int cols) { return ld ? ld : cols; }

int device_sms()
{
    int sms = 0;
    return amsim::current_device(&sms) < 0 ? 0 : sms;
}

int check(const amsim_block_norm_desc *d)
{
    if (!d || d->rows < 0 || d->cols < 1) return AMSIM_EINVAL;
    if (d->cols > AMSIM_BLOCK_NORM_MAX_COLS) return AMSIM_EUNSUPPORTED;
    if (d->gate_rows < 0 || (d->gate_rows > 0 && d->rows % d->gate_rows)) return AMSIM_EINVAL;
    for (int t : {d->x_type, d->y_type, d->n_type})
        if (t != AMSIM_F32 && t != AMSIM_BF16) return AMSIM_EINVAL;
    for (int64_t ld : {d->ldx, d->ldy, d->ldr, d->ldn, d->lddr, d->lddn, d->lddx, d->lddy})
        if (ld != 0 && (ld < d->cols || ld > (int64_t)1 << 40)) return AMSIM_EINVAL;
    if (!std::isfinite(d->alpha) || !std::isfinite(d->eps) || d->eps < 0.0f) return AMSIM_EINVAL;
    return AMSIM_OK;
}

// Steps of 4 channels per thread, threads per row and rows per block: four
// steps, so that what a row costs per thread is spread over 16 channels, fewer
// where that would not fill a warp; narrow rows share blocks of 128 threads.
struct Shape {
    int nv, tpr, rpb;
};
Shape shape(int cols, bool vec)
{
    Shape s;
    const int steps = (cols + amsim::bn::kE - 1) / amsim::bn::kE;
    s.nv = steps <= 32 && vec ? 1 : steps <= 96 ? 2 : 4;
    s.tpr = ((steps + s.nv - 1) / s.nv + 31) / 32 * 32;
    s.rpb = std::max(1, 128 / s.tpr);
    return s;
}

// The ring's shape: rows at work on an SM, in blocks of their own (forward) or
// in teams of one block (backward), and as many rows ahead of each as there is
// room for.  slots < 2: the row is too wide (or too narrow).
struct RingShape {
    int tpr, at_work, slots, slot_bytes;
};
RingShape ring_shape(int cols, int slot_bytes, bool bwd)
{
    RingShape s{};
    const Shape d = shape(cols, true);
    if (d.nv != amsim::bn::kRingNV || d.tpr > 512) return s;
    s.tpr = d.tpr;
    s.at_work = (bwd ? amsim::bn::kTeamThreads : amsim::bn::kRingThreads) / s.tpr;
    s.slot_bytes = slot_bytes;
    for (;; --s.at_work) {
        // what is not for rows: barriers, sums, a block's own kilobyte, backward the weights and the teams' sums
        const int joined = s.at_work > 1 ? amsim::bn::kTeamThreads * 16 : 0;
        const int room = bwd ? (amsim::kMaxSmemPerCta - 2048 - 8 * cols - joined) / s.at_work - amsim::bn::kRingBarBytes
                             : amsim::kMaxSmemPerCta / s.at_work - 2048 - amsim::bn::kRingBarBytes;
        s.slots = std::min(8, room / slot_bytes);
        if (s.slots >= 2 || s.at_work == 1) return s;
    }
}

// The ring from half a row for each at work on.  By kernels alone, bf16: 608 x
// 1024 forward 3.9 us by direct loads, 3.2 so, backward 17.3 and 13.8; 152 x
// 4096 3.9, 3.2 and 16.0, 15.9; 304 x 2048 backward 14.7, 14.3.  With half of
// that backward is no faster, and a small call's time is the host's.
bool ring_pays(int64_t rows, const RingShape &r, int sms)
{
    return r.slots >= 2 && 2 * rows >= (int64_t)sms * r.at_work;
}

// Resident blocks per SM of the kernels that load directly: about 1024 threads.
int direct_blocks(const Shape &s) { return std::max(1, 1024 / (s.tpr * s.rpb)); }

// The backward pass's shares: `splits` per row of the gate, `blocks` thread
// blocks that take them.  `slots`: how many [cols] sums the scratch holds.
struct Shares {
    int splits;
    int64_t item_rows, items;
    int blocks;
};
Shares shares(const amsim_block_norm_desc *d, int per_sm, int rpb, int sms, int64_t slots)
{
    const int64_t gate_rows = d->gate_rows ? d->gate_rows : d->rows;
    const int64_t groups = d->rows / gate_rows;
    // every SM full, at least 2 passes of a block over its rows
    int64_t want = std::max<int64_t>(1, (int64_t)sms * per_sm);
    want = std::min(want, std::max<int64_t>(1, d->rows / (2 * rpb)));
    Shares r;
    for (;;) {
        int64_t splits = std::max<int64_t>(1, want / groups);
        r.item_rows = (gate_rows + splits - 1) / splits;
        splits = (gate_rows + r.item_rows - 1) / r.item_rows;
        r.splits = (int)splits;
        r.items = groups * splits;
        r.blocks = (int)std::min<int64_t>(r.items, std::max<int64_t>(want, 1));
        // part_gate or part_post, and part_pre
        const int64_t need = (splits > 1 ? r.items : r.blocks) + r.blocks;
        if (need <= slots || want == 1) return r;
        want = std::max<int64_t>(1, want / 2);
    }
}

}  // namespace

extern "C" int amsim_block_norm_fwd(const amsim_block_norm_desc *d, const void *x, const void *y, const float *gate,
                                    const float *w_post, const float *w_pre, void *r, void *n, float *rstd_post,
                                    float *rstd_pre, amsim_stream_t stream)
{
    const int rc = check(d);
    if (rc) return rc;
    if (d->rows == 0) return AMSIM_OK;
    if (!x || (!r && !n) || (!y && (gate || w_post))) return AMSIM_EINVAL;
    const size_t xs = type_size(d->x_type), ys = type_size(d->y_type), ns = type_size(d->n_type);
    if (!aligned(x, xs) || !aligned(r, xs) || !aligned(y, ys) || !aligned(n, ns)) return AMSIM_EINVAL;
    for (const float *f : {gate, w_post, w_pre, (const float *)rstd_post, (const float *)rstd_pre})
        if (!aligned(f, 4)) return AMSIM_EINVAL;
    Params p{};
    p.x = x;
    p.y = y;
    p.r = r;
    p.n = n;
    p.gate = gate;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.rstd_post = rstd_post;
    p.rstd_pre = rstd_pre;
    p.rows = d->rows;
    p.gate_rows = d->gate_rows ? d->gate_rows : d->rows;
    p.cols = d->cols;
    p.ldx = stride(d->ldx, d->cols);
    p.ldy = stride(d->ldy, d->cols);
    p.ldr = stride(d->ldr, d->cols);
    p.ldn = stride(d->ldn, d->cols);
    p.alpha = d->alpha;
    p.eps = d->eps;
    bool vec = d->cols % amsim::bn::kE == 0;
    for (const void *q : {(const void *)gate, (const void *)w_post, (const void *)w_pre}) vec = vec && aligned(q, 16);
    vec = vec && vector_rows(x, p.ldx, xs) && vector_rows(y, p.ldy, ys) && vector_rows(r, p.ldr, xs) &&
          vector_rows(n, p.ldn, ns);
    const bool whole = vec && bulk_rows(x, p.ldx, xs, d->cols) && bulk_rows(y, p.ldy, ys, d->cols);
    const int slack = whole ? 0 : amsim::bn::kRingSlack;
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    const Shape s = shape(d->cols, vec);
    const RingShape ring = ring_shape(
        d->cols, amsim::bn::ring_bytes(d->cols, (int)xs, slack) + (y ? amsim::bn::ring_bytes(d->cols, (int)ys, slack) : 0), false);
    const amsim::bn::Has has = y && w_post && r && n && rstd_post && rstd_pre ? amsim::bn::kAll : amsim::bn::kSome;
    int64_t grid;
    amsim::bn::Loads loads = vec ? amsim::bn::kVector : amsim::bn::kScalar;
    if (ring_pays(d->rows, ring, sms) && (has == amsim::bn::kAll || (whole && ring.tpr <= 256))) {
        loads = whole ? amsim::bn::kRing : vec ? amsim::bn::kPieceRing : amsim::bn::kScalarRing;
        p.tpr = ring.tpr;
        p.rpb = 1;
        p.slots = ring.slots;
        p.slot_bytes = ring.slot_bytes;
        p.block_rows = (d->rows + (int64_t)sms * ring.at_work - 1) / ((int64_t)sms * ring.at_work);
        grid = (d->rows + p.block_rows - 1) / p.block_rows;
    } else {
        p.tpr = s.tpr;
        p.rpb = s.rpb;
        grid = (d->rows + s.rpb - 1) / s.rpb;
    }
    if (grid > 0x7FFFFFFF) return AMSIM_EINVAL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return d->x_type == AMSIM_F32
               ? amsim::bn::launch_fwd_f32(s.nv, loads, has, d->y_type, d->n_type, p, (unsigned)grid, st)
               : amsim::bn::launch_fwd_bf16(s.nv, loads, has, d->y_type, d->n_type, p, (unsigned)grid, st);
}

extern "C" size_t amsim_block_norm_workspace_size(const amsim_block_norm_desc *d)
{
    if (check(d) || d->rows == 0) return 0;
    const int sms = device_sms();
    const Shape s = shape(d->cols, true);
    const Shares h = shares(d, direct_blocks(s), s.rpb, sms ? sms : 1,
                            INT64_MAX);
    if (h.blocks == 1 && h.splits == 1) return 0;
    const int64_t n = (h.splits > 1 ? h.items : h.blocks) + h.blocks;
    return (size_t)n * (size_t)d->cols * 4;
}

extern "C" int amsim_block_norm_bwd(const amsim_block_norm_desc *d, const void *dr, const void *dn, const void *r,
                                    const void *y, const float *gate, const float *w_post, const float *w_pre,
                                    const float *rstd_post, const float *rstd_pre, void *dx, void *dy, float *dgate,
                                    float *dw_post, float *dw_pre, void *ws, size_t ws_bytes, amsim_stream_t stream)
{
    int rc = check(d);
    if (rc) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d->rows == 0) {                      // sums over no rows; gate_rows 0: the gate has a row all the same
        for (float *f : {d->gate_rows ? nullptr : dgate, dw_post, dw_pre})
            if (f && cudaMemsetAsync(f, 0, (size_t)d->cols * 4, st) != cudaSuccess) {
                cudaGetLastError();
                return AMSIM_ECUDA;
            }
        return AMSIM_OK;
    }
    if (!y && (gate || w_post || dy || dgate || dw_post)) return AMSIM_EINVAL;
    if ((dgate && !gate) || (dw_post && !w_post) || (dw_pre && !dn)) return AMSIM_EINVAL;
    if (!dx && !dy && !dgate && !dw_post && !dw_pre) return AMSIM_EINVAL;
    if ((!dr && !dn) || (dn && (!r || !rstd_pre)) || (w_post && !rstd_post)) return AMSIM_EINVAL;
    const size_t xs = type_size(d->x_type), ys = type_size(d->y_type), ns = type_size(d->n_type);
    if (!aligned(dr, xs) || !aligned(r, xs) || !aligned(dx, xs) || !aligned(y, ys) || !aligned(dy, ys) ||
        !aligned(dn, ns))
        return AMSIM_EINVAL;
    for (const float *f : {gate, w_post, w_pre, rstd_post, rstd_pre, (const float *)dgate, (const float *)dw_post,
                           (const float *)dw_pre, (const float *)ws})
        if (!aligned(f, 4)) return AMSIM_EINVAL;
    Params p{};
    p.y = y;
    p.dr = dr;
    p.dn = dn;
    p.rin = r;
    p.dx = dx;
    p.dy = dy;
    p.gate = gate;
    p.w_post = w_post;
    p.w_pre = w_pre;
    p.rstd_post = const_cast<float *>(rstd_post);
    p.rstd_pre = const_cast<float *>(rstd_pre);
    p.dgate = dgate;
    p.dw_post = dw_post;
    p.dw_pre = dw_pre;
    p.rows = d->rows;
    p.gate_rows = d->gate_rows ? d->gate_rows : d->rows;
    p.cols = d->cols;
    p.ldy = stride(d->ldy, d->cols);
    p.ldr = stride(d->ldr, d->cols);
    p.lddr = stride(d->lddr, d->cols);
    p.lddn = stride(d->lddn, d->cols);
    p.lddx = stride(d->lddx, d->cols);
    p.lddy = stride(d->lddy, d->cols);
    p.alpha = d->alpha;
    p.eps = d->eps;
    bool vec = d->cols % amsim::bn::kE == 0;
    for (const void *q : {(const void *)gate, (const void *)w_post, (const void *)w_pre}) vec = vec && aligned(q, 16);
    vec = vec && vector_rows(r, p.ldr, xs) && vector_rows(dr, p.lddr, xs) && vector_rows(dx, p.lddx, xs) &&
          vector_rows(y, p.ldy, ys) && vector_rows(dy, p.lddy, ys) && vector_rows(dn, p.lddn, ns);
    const bool whole = vec && bulk_rows(r, p.ldr, xs, d->cols) && bulk_rows(dr, p.lddr, xs, d->cols) &&
                       bulk_rows(y, p.ldy, ys, d->cols) && bulk_rows(dn, p.lddn, ns, d->cols);
    const int slack = whole ? 0 : amsim::bn::kRingSlack;
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    const Shape s = shape(d->cols, vec);
    const int rx = amsim::bn::ring_bytes(d->cols, (int)xs, slack);
    const RingShape ring =
        ring_shape(d->cols, (dr ? rx : 0) + (dn ? rx + amsim::bn::ring_bytes(d->cols, (int)ns, slack) : 0) +
                                (y ? amsim::bn::ring_bytes(d->cols, (int)ys, slack) : 0), true);
    const bool rest = dn && y && w_post && dx && dy;
    const amsim::bn::Has has = !rest ? amsim::bn::kSome : dr ? amsim::bn::kAll : amsim::bn::kNoDr;
    int per_sm = direct_blocks(s);
    amsim::bn::Loads loads = vec ? amsim::bn::kVector : amsim::bn::kScalar;
    p.tpr = s.tpr;
    p.rpb = s.rpb;
    if (ring_pays(d->rows, ring, sms)) {
        loads = whole ? amsim::bn::kRing : vec ? amsim::bn::kPieceRing : amsim::bn::kScalarRing;
        p.tpr = ring.tpr;
        p.rpb = ring.at_work;
        p.slots = ring.slots;
        p.slot_bytes = ring.slot_bytes;
        per_sm = 1;
    }
    const bool sums = dgate || dw_post || dw_pre;
    const int64_t slots = sums ? (ws ? (int64_t)(ws_bytes / ((size_t)d->cols * 4)) : 0) : INT64_MAX;
    const Shares h = shares(d, per_sm, p.rpb, sms, slots);
    p.splits = h.splits;
    p.item_rows = h.item_rows;
    p.items = h.items;
    // one block: its sums go straight to the outputs
    const bool direct = h.blocks == 1 && h.splits == 1;
    if (sums && !direct) {
        float *base = static_cast<float *>(ws);
        const int64_t first = h.splits > 1 ? h.items : h.blocks;
        (h.splits > 1 ? p.part_gate : p.part_post) = base;
        p.part_pre = base + first * d->cols;
    } else {
        p.part_post = dw_post;
        p.part_pre = dw_pre;
    }
    rc = d->x_type == AMSIM_F32
             ? amsim::bn::launch_bwd_f32(s.nv, loads, has, d->y_type, d->n_type, p, (unsigned)h.blocks, st)
             : amsim::bn::launch_bwd_bf16(s.nv, loads, has, d->y_type, d->n_type, p, (unsigned)h.blocks, st);
    if (rc || !sums || direct) return rc;
    rc = amsim::cuda_status(amsim::chain_launch(true, sums_kernel, dim3((unsigned)((d->cols + 31) / 32), 2),
                                                kSumWarps * 32, 0, st, p, h.blocks));
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}
