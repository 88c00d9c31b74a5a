// The block norm's entry points: argument checks, launch shapes, and the
// kernel that adds the backward pass's column sums.
#include <algorithm>
#include <cmath>

#include "block_norm.cuh"

namespace {

using amsim::bn::Params;

// dgate, dw_post and dw_pre from the shares' sums, in share order.  A block
// takes 32 channels; its warps take the shares in turn and add up at the end.
__global__ void __launch_bounds__(512) sums_kernel(const Params p, int blocks)
{
    __shared__ float part[16][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (int)blockIdx.x * 32 + lane;
    const bool on = c < p.cols;
    auto total = [&](const float *src, long long n) {
        float s = 0.0f;
        if (on)
            for (long long i = warp; i < n; i += 16) s += src[i * p.cols + c];
        __syncthreads();
        part[warp][lane] = s;
        __syncthreads();
        s = 0.0f;
        if (warp == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) s += part[i][lane];
        return s;                              // warp 0 holds the sum
    };
    if (blockIdx.y == 0) {
        if (!p.dw_pre || !p.part_pre) return;
        const float s = total(p.part_pre, blocks);
        if (warp == 0 && on) p.dw_pre[c] = s;
        return;
    }
    if (p.splits == 1) {
        if (!p.dw_post || !p.part_post) return;
        const float s = total(p.part_post, blocks);
        if (warp == 0 && on) p.dw_post[c] = s;
        return;
    }
    if (!p.part_gate) return;
    const long long groups = p.items / p.splits;
    const float w = on && p.w_post ? p.w_post[c] : 1.0f;
    float dw = 0.0f;
    for (long long g = 0; g < groups; ++g) {
        const float s = total(p.part_gate + g * p.splits * p.cols, p.splits);
        if (p.dgate && warp == 0 && on) p.dgate[g * p.cols + c] = p.alpha * w * s;
        dw = fmaf(p.alpha * (on && p.gate ? p.gate[g * p.cols + c] : 1.0f), s, dw);
    }
    if (p.dw_post && warp == 0 && on) p.dw_post[c] = dw;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
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

// Steps of 8 channels per thread, threads per row and rows per block: one step
// while a row fits 512 threads, so that a row's loads are spread over as many
// threads as possible; narrow rows share blocks of 128 threads.
struct Shape {
    int nv, tpr, rpb;
};
Shape shape(int cols)
{
    Shape s;
    const int steps = (cols + 7) / 8;
    s.nv = steps <= 512 ? 1 : 2;
    s.tpr = ((steps + s.nv - 1) / s.nv + 31) / 32 * 32;
    s.rpb = std::max(1, 128 / s.tpr);
    return s;
}

// The backward pass's shares: `splits` per row of the gate, `blocks` thread
// blocks that take them.  `slots`: how many [cols] sums the scratch holds.
struct Shares {
    int splits;
    int64_t item_rows, items;
    int blocks;
};
Shares shares(const amsim_block_norm_desc *d, const Shape &s, int sms, int64_t slots)
{
    const int64_t gate_rows = d->gate_rows ? d->gate_rows : d->rows;
    const int64_t groups = d->rows / gate_rows;
    // about 1024 threads per SM, at least 4 passes of a block over its rows
    int64_t want = std::max<int64_t>(1, (int64_t)sms * std::max(1, 1024 / (s.tpr * s.rpb)));
    want = std::min(want, std::max<int64_t>(1, d->rows / (4 * s.rpb)));
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
    bool vec = d->cols % 8 == 0;
    for (const void *q : {x, y, (const void *)r, (const void *)n, (const void *)gate, (const void *)w_post,
                          (const void *)w_pre})
        vec = vec && aligned(q, 16);
    vec = vec && p.ldx * xs % 16 == 0 && p.ldr * xs % 16 == 0 && p.ldy * ys % 16 == 0 && p.ldn * ns % 16 == 0;
    const Shape s = shape(d->cols);
    p.tpr = s.tpr;
    p.rpb = s.rpb;
    const int64_t grid = (d->rows + s.rpb - 1) / s.rpb;
    if (grid > 0x7FFFFFFF) return AMSIM_EINVAL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return d->x_type == AMSIM_F32
               ? amsim::bn::launch_f32(false, s.nv, vec, d->y_type, d->n_type, p, (unsigned)grid, st)
               : amsim::bn::launch_bf16(false, s.nv, vec, d->y_type, d->n_type, p, (unsigned)grid, st);
}

extern "C" size_t amsim_block_norm_workspace_size(const amsim_block_norm_desc *d)
{
    if (check(d) || d->rows == 0) return 0;
    const int sms = device_sms();
    const Shares h = shares(d, shape(d->cols), sms ? sms : 1, INT64_MAX);
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
    if (d->rows == 0) {                      // sums over no rows
        for (float *f : {dw_post, dw_pre})
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
    bool vec = d->cols % 8 == 0;
    for (const void *q : {dr, dn, r, y, (const void *)dx, (const void *)dy, (const void *)gate, (const void *)w_post,
                          (const void *)w_pre})
        vec = vec && aligned(q, 16);
    vec = vec && p.ldr * xs % 16 == 0 && p.lddr * xs % 16 == 0 && p.lddx * xs % 16 == 0 && p.ldy * ys % 16 == 0 &&
          p.lddy * ys % 16 == 0 && p.lddn * ns % 16 == 0;
    const Shape s = shape(d->cols);
    p.tpr = s.tpr;
    p.rpb = s.rpb;
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    const bool sums = dgate || dw_post || dw_pre;
    const int64_t slots = sums ? (ws ? (int64_t)(ws_bytes / ((size_t)d->cols * 4)) : 0) : INT64_MAX;
    const Shares h = shares(d, s, sms, slots);
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
             ? amsim::bn::launch_f32(true, s.nv, vec, d->y_type, d->n_type, p, (unsigned)h.blocks, st)
             : amsim::bn::launch_bf16(true, s.nv, vec, d->y_type, d->n_type, p, (unsigned)h.blocks, st);
    if (rc || !sums || direct) return rc;
    sums_kernel<<<dim3((unsigned)((d->cols + 31) / 32), 2), 512, 0, st>>>(p, h.blocks);
    rc = amsim::cuda_status(cudaGetLastError());
    if (rc == AMSIM_OK) amsim::count_launch();
    return rc;
}
