// The group norm with its activation, channels last, and its gradients.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "amsim_internal.h"
#include "chained.cuh"

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
    const float n = a.n + b.n;
    if (n == 0.0f) return a;
    const float d = b.mean - a.mean, f = b.n / n;
    return Moments{n, a.mean + d * f, a.m2 + b.m2 + d * d * (a.n * f)};
}

__device__ __forceinline__ float activate(float z, int act)
{
    if (act == AMSIM_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if (act == AMSIM_ACT_SILU) return z / (1.0f + expf(-z));
    return z;
}

// dy act'(z).  relu's gradient jumps where z = 0: a z that its own roundings
// (three of xh w, one of the sum: at most 2^-22 of the terms) could carry
// across is computed again in 64 bits.
__device__ __forceinline__ float before_activation(float dy, float x, float xh, float mean, float rstd, float w, float b,
                                                   int act)
{
    if (act == AMSIM_ACT_NONE) return dy;
    const float z = fmaf(xh, w, b);
    if (act == AMSIM_ACT_RELU) {
        bool on = z > 0.0f;
        if (fabsf(z) <= 0x1p-21f * (fabsf(xh * w) + fabsf(b)))
            on = ((double)x - (double)mean) * (double)rstd * (double)w + (double)b > 0.0;
        return on ? dy : 0.0f;
    }
    const float s = 1.0f / (1.0f + expf(-z));
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
#pragma unroll 4
    for (int64_t i = t.first + t.y; i < t.last; i += t.ty) {
        float v[E];
        load<E>(x + i * p.ldx, v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = activate(fmaf((v[e] - k.mean[e]) * k.rstd[e], k.w[e], k.b[e]), p.act);
        store<E>(y + i * p.ldy, v);
    }
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
#pragma unroll 2
        for (int64_t i = t.first + t.y; i < t.last; i += t.ty) {
            float v[E], d[E];
            load<E>(x + i * p.ldx, v);
            load<E>(dy + i * p.ldy, d);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float xh = (v[e] - k.mean[e]) * k.rstd[e];
                const float dz = before_activation(d[e], v[e], xh, k.mean[e], k.rstd[e], k.w[e], k.b[e], p.act);
                s[e].x += dz;
                s[e].y = fmaf(dz, xh, s[e].y);
            }
        }
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
#pragma unroll 2
    for (int64_t i = t.first + t.y; i < t.last; i += t.ty) {
        float v[E], d[E];
        load<E>(x + i * p.ldx, v);
        load<E>(dy + i * p.ldy, d);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float xh = (v[e] - k.mean[e]) * k.rstd[e];
            const float dz = before_activation(d[e], v[e], xh, k.mean[e], k.rstd[e], k.w[e], k.b[e], p.act);
            v[e] = k.rstd[e] * (fmaf(dz, k.w[e], -m[e].x) - xh * m[e].y);
        }
        store<E>(dx + i * p.lddx, v);
    }
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

template <typename TX, typename TY, int E>
int forward(const Params &p, cudaStream_t st)
{
    if (int rc = start(false, moments_kernel<TX, E>, grid(p), kThreads, p, st)) return rc;
    if (int rc = start(true, join_kernel, dim3((unsigned)(p.batch * p.groups)), kThreads, p, st)) return rc;
    return start(true, apply_kernel<TX, TY, E>, grid(p), kThreads, p, st);
}

template <typename TX, typename TY, int E>
int backward(const Params &p, cudaStream_t st)
{
    if (int rc = start(false, sums_kernel<TX, TY, E>, grid(p), kThreads, p, st)) return rc;
    if (int rc = start(true, means_kernel, dim3((unsigned)(p.batch * p.groups)), kThreads, p, st)) return rc;
    if (int rc = start(true, gradient_kernel<TX, TY, E>, grid(p), kThreads, p, st)) return rc;
    if (!p.dw && !p.db) return AMSIM_OK;
    return start(false, weights_kernel, dim3((unsigned)((p.channels + 31) / 32)), 1024, p, st);
}

template <int EB, int EF>
int run(bool fwd, const amsim_group_norm_desc *d, const Params &p, cudaStream_t st)
{
    using B = __nv_bfloat16;
    if (d->x_type == AMSIM_F32)
        return d->y_type == AMSIM_F32 ? (fwd ? forward<float, float, EF>(p, st) : backward<float, float, EF>(p, st))
                                      : (fwd ? forward<float, B, EF>(p, st) : backward<float, B, EF>(p, st));
    return d->y_type == AMSIM_F32 ? (fwd ? forward<B, float, EF>(p, st) : backward<B, float, EF>(p, st))
                                  : (fwd ? forward<B, B, EB>(p, st) : backward<B, B, EB>(p, st));
}

}  // namespace

extern "C" size_t amsim_group_norm_workspace_size(const amsim_group_norm_desc *d, int which)
{
    if (check(d) || which < 0 || which > 1 || !d->batch || !d->pixels) return 0;
    const int sms = device_sms();
    Params p = params(d);
    size_t most = 0;
    for (int E : {1, piece(d)}) {                // the calls' pointers decide which
        split(p, E, sms ? sms : 1);
        most = std::max(most, (size_t)p.batch * p.chunks * p.channels);
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
    if (d->pixels && (!ws || ws_bytes < amsim_group_norm_workspace_size(d, 0))) return AMSIM_EINVAL;
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
    const int E = piece(d);
    const bool vec = d->channels % E == 0 && whole(x, p.ldx, xs, E) && whole(y, p.ldy, ys, E);
    split(p, vec ? E : 1, sms);
    return vec ? run<8, 4>(true, d, p, st) : run<1, 1>(true, d, p, st);
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
    const int E = piece(d);
    const bool vec = d->channels % E == 0 && whole(x, p.ldx, xs, E) && whole(dx, p.lddx, xs, E) &&
                     whole(dy, p.ldy, ys, E);
    split(p, vec ? E : 1, sms);
    p.sums = static_cast<float2 *>(ws);
    p.means = p.sums + (size_t)p.batch * p.channels;
    p.part = p.means + (size_t)p.batch * p.groups;
    return vec ? run<8, 4>(false, d, p, st) : run<1, 1>(false, d, p, st);
}
