// Softmax cross entropy over a large vocabulary without keeping the logits,
// with the gradients of the hidden states and of the vocabulary weights.
//
// z = h W^T (tokens x vocab) is computed tile by tile on the tensor cores and
// reduced where it is computed: each row of a 128-column piece leaves its
// maximum and its sum of exponentials, from which a merge makes lse and the
// loss.  For the gradients the piece also leaves 16 bits per logit, the
// distance to the piece's maximum in steps of 2^-11 (a relative error of the
// probability of at most 2^-12, a sixteenth of a bf16 rounding): half the traffic of fp32
// logits, and no second h W^T product.  A pass over them writes
// G = exp(z - lse) - onehot in bf16 in place, and two more products give
// dh = G W and dW = G^T h.
//
// All three products run in one kernel: pairs of CTAs that share tiles of
// 256 x 256, bf16 operands copied by TMA into 128-byte swizzled tiles of 64
// steps of the reduction, six deep, tcgen05 matrix instructions of 256 x 256 x
// 16 issued for both CTAs by one thread, and two fp32 accumulators in tensor
// memory, so that eight warps reduce or write one tile while the next is being
// computed.  (A CTA alone would read each operand byte from shared memory for
// half as many products, and a pair holds half of B: 641 -> 462 us at 1531
// tokens x 50021 x 1000, with gradients, when pairs and whole-box stores came
// in.)  dh and dW read G, W and h as they lie in memory: an operand whose rows
// run along M or N instead of K only changes its descriptor.
//
// Bound by the matrix pipe where the sizes are large: 4096 tokens x 32768 x
// 1024 takes 148 to 158 us a product (1.8e15 operations/s; the pipe 87 to 96 %
// active) and 81 us for G, whose 4 bytes per logit run at the memory's rate;
// 8192 x 65536 x 4096 takes 8.0 ms (1.64e15/s), at the power limit.  With few
// tokens it reads W twice and writes dW, and a tile of 256 rows is mostly
// padding: 19 x 46024 x 2048 takes 55, 38 and 50 us for its products, the
// first two for 189 MB (28 us) each.  The smallest calls cost their chain of
// six launches, which start while the one before ends: 24 x 8192 x 256 takes
// 37 us.
#include <algorithm>
#include <atomic>

#include "chained.cuh"
#include "tensor_core.cuh"

namespace {

using namespace amsim;
using bf16 = __nv_bfloat16;

constexpr int kTileM = 256, kTileN = 256, kTileK = 64;   // of a CTA pair
constexpr int kHalfM = kTileM / 2, kHalfN = kTileN / 2;   // what each CTA holds of A and of B
constexpr int kPiece = 128;                        // columns that share a maximum
constexpr int kStages = 6;
constexpr int kStageA = kHalfM * kTileK * 2, kStageB = kHalfN * kTileK * 2;
constexpr int kStage = kStageA + kStageB;          // 32 KB
constexpr int kBox = 64;                           // elements of a 128-byte row
constexpr int kFirstEpilogueWarp = 2;              // after the copy and the matrix warp
constexpr int kThreads = (kFirstEpilogueWarp + 8) * 32;
constexpr int kBuffer = 32 * 128;                  // of a warp: 32 rows of 128 bytes on their way out
constexpr int kSmem = kStages * kStage + 8 * kBuffer + 1024 + 256;
static_assert(kSmem <= amsim::kMaxSmemPerCta, "shared memory of a CTA");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSteps = 2048.0f;                  // code steps per unit of the logit

enum Product { kLogits = 0, kDh = 1, kDw = 2 };

// Steps of the reduction that one accumulator takes before it is handed over.
// The tensor cores add with truncation: each of the additions of 16 products
// pulls a sum towards zero, and over 4096 products a logit came out 2e-6 low
// (relative), which lse and the loss inherit.  So logits are handed over every
// 1024 products and added with rounding in registers (3e-7, as at a width of
// 1024); dh and dw, rounded to bf16, take their whole reduction in one.
template <int PRODUCT>
constexpr int kSegment = PRODUCT == kLogits ? 16 : 0x7FFFFFFF;

struct ProductParams {
    int m, n, kblocks;              // rows, columns, steps of 64 of the reduction
    int mt, nt, splits, per_split;  // tiles, parts of the reduction and their steps
    int group;                      // row tiles visited together
    // kLogits
    const int64_t *targets;         // of the chunk's rows
    float *target_logit;
    float2 *stats;                  // [piece][rows]: maximum, sum of exponentials
    unsigned int *done;             // the merge's count of blocks, zeroed here
    const uint16_t *codes;          // null: not wanted; else the output map is over them
    // kDh, kDw
    bf16 *out;
    long long ld_out;
    int boxes, pairs;               // out goes through the tensor map; its rows are 4-byte aligned
    const float *scale;             // 1 / A
    float *acc;                     // fp32 sums of earlier chunks (kDw) or the splits' sums (kDh)
    long long ld_acc, split_rows;   // its row stride and rows per split
    int acc_read, acc_write;
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// a = b where i == j.  A chain of these picks one of many registers; written
// in C, the compiler indexes a copy of them in local memory instead.
__device__ __forceinline__ void select_if(float &a, float b, int i, int j)
{
    asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %2, %3;\n\tselp.f32 %0, %1, %0, p;\n\t}" : "+f"(a) : "f"(b), "r"(i), "r"(j));
}

struct Tile {
    int m, n, split;
};
// Tiles in the order they are taken: `group` row tiles by every column tile,
// so that a wave of CTAs reads few distinct operand tiles.
__device__ __forceinline__ Tile tile_at(const ProductParams &p, int i)
{
    Tile t;
    const int per = p.mt * p.nt;
    t.split = i / per;
    i -= t.split * per;
    const int full = p.group * p.nt, g = i / full, m0 = g * p.group;
    const int rows = min(p.group, p.mt - m0);
    i -= g * full;
    t.n = i / rows;
    t.m = m0 + i - t.n * rows;
    return t;
}

// What leaves a tile goes through a warp's buffer of 32 rows by 128 bytes,
// swizzled like the operand tiles (a row's 16-byte words exchanged by the row
// number modulo 8: no bank conflicts), and out by a box copy.  Stores straight
// from the registers, a row per lane, touch 32 lines per instruction: they held
// the logits' epilogue at 12.7 us a tile where the products took 4.3.
struct Out {
    uint8_t *buffer;
    const CUtensorMap *map;
    int lane;

    // begin, the eight 16-byte words of every lane's row, end: the warp's rows
    // from `y`, 128 bytes from column `x` (in elements of the map's type), if any
    // of them is inside.
    __device__ __forceinline__ void begin() const
    {
        if (lane == 0) tc::stores_read();
        __syncwarp();
    }
    __device__ __forceinline__ void word(int j, uint32_t a, uint32_t b, uint32_t c, uint32_t d) const
    {
        reinterpret_cast<uint4 *>(buffer + lane * 128)[j ^ (lane & 7)] = make_uint4(a, b, c, d);
    }
    // the same, by the warp's own coalesced stores, for rows that box copies
    // cannot write: `rows` x `cols` elements of 16 bits to `dst`, two at a time
    // where they are 4-byte aligned (496 tokens x 68330 x 3356, forward and
    // gradients: 807 us with single elements, 768 with pairs)
    __device__ __forceinline__ void end_rows(bf16 *dst, long long ld, int rows, int cols, bool pairs) const
    {
        __syncwarp();
        if (pairs) {
#pragma unroll 8
            for (int r = 0; r < 32; ++r) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(
                    buffer + r * 128 + ((lane >> 2) ^ (r & 7)) * 16 + (lane & 3) * 4);
                if (r < rows && 2 * lane + 1 < cols) *reinterpret_cast<uint32_t *>(dst + r * ld + 2 * lane) = w;
                else if (r < rows && 2 * lane < cols) reinterpret_cast<uint16_t *>(dst)[r * ld + 2 * lane] = (uint16_t)w;
            }
        } else {
#pragma unroll 4
            for (int r = 0; r < 32; ++r) {
                const uint16_t *row = reinterpret_cast<const uint16_t *>(buffer + r * 128);
#pragma unroll
                for (int e = lane; e < 64; e += 32)
                    if (r < rows && e < cols)
                        reinterpret_cast<uint16_t *>(dst)[r * ld + e] = row[((e >> 3) ^ (r & 7)) * 8 + (e & 7)];
            }
        }
        __syncwarp();
    }
    __device__ __forceinline__ void end(int x, int y, bool inside) const
    {
        tc::fence_staged();
        __syncwarp();
        if (lane == 0 && inside) {
            tc::store_box(map, x, y, buffer);
            tc::stores_commit();
        }
    }
};

// One 128-column piece of a row of logits, in the registers of its thread.
// fmaxf skips NaN; the sum does not, so a NaN logit makes the row's lse NaN.
// The code of a logit is the rounding of a sum with 2^23: its low 16 bits.
template <bool MASKED>
__device__ __forceinline__ void reduce_piece(const ProductParams &p, const float (&z)[kPiece], int row, int col0,
                                             const Out &out)
{
    float tops[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) tops[j] = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPiece; ++j)
        if (!MASKED || col0 + j < p.n) tops[j & 7] = fmaxf(tops[j & 7], z[j]);
    const float top = fmaxf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])),
                            fmaxf(fmaxf(tops[4], tops[5]), fmaxf(tops[6], tops[7])));
    if (row < p.m) {
        const long long d = p.targets[row] - col0;
        if (d >= 0 && d < kPiece && col0 + d < p.n) {
            float pick = 0.0f;
#pragma unroll
            for (int j = 0; j < kPiece; ++j) select_if(pick, z[j], (int)d, j);
            p.target_logit[row] = pick;
        }
    }
    const float shift = top == -INFINITY ? 0.0f : top * kLog2e;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kPiece; ++j)
        if (!MASKED || col0 + j < p.n) sum[j & 3] += exp2_fast(fmaf(z[j], kLog2e, -shift));
    if (row < p.m) p.stats[(long long)(col0 / kPiece) * p.m + row] = make_float2(top, (sum[0] + sum[1]) + (sum[2] + sum[3]));
    if (p.codes) {
        constexpr float kBase = 8388608.0f, kLast = kBase + 65535.0f;
        auto code = [&](int j) {
            const float a = fminf(fmaf(top - z[2 * j], kSteps, kBase), kLast);
            const float b = fminf(fmaf(top - z[2 * j + 1], kSteps, kBase), kLast);
            return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
        };
#pragma unroll
        for (int c = 0; c < kPiece / kBox; ++c) {
            out.begin();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = c * 32 + j * 4;
                out.word(j, code(i), code(i + 1), code(i + 2), code(i + 3));
            }
            out.end(col0 + c * kBox, row - out.lane, (!MASKED || col0 + c * kBox < p.n) && row - out.lane < p.m);
        }
    }
}

// A 128-column piece of a row of dh or dw: added to the fp32 sums, or scaled,
// rounded and written; `release` is called when tensor memory has been read.
template <typename F>
__device__ __forceinline__ void store_piece(const ProductParams &p, uint32_t tmem, int row, int col0, int split,
                                            const Out &out, F release)
{
    const bool on = row < p.m, warp_on = row - out.lane < p.m && col0 < p.n;
    const float scale = p.out ? *p.scale : 1.0f;
    float *acc = p.acc ? p.acc + (split * p.split_rows + row) * p.ld_acc + col0 : nullptr;
    if (p.acc_write) {
#pragma unroll
        for (int c = 0; c < kPiece / 32; ++c) {
            uint32_t r[32];
            tc::tmem_load32(tmem + c * 32, r);
            tc::tmem_load_wait(r);
            if (c == kPiece / 32 - 1) release();
            const int left = on ? p.n - (col0 + c * 32) : 0;
            if (p.acc_read) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j < left) r[j] = __float_as_uint(__uint_as_float(r[j]) + acc[c * 32 + j]);
            }
            out.begin();
#pragma unroll
            for (int j = 0; j < 8; ++j) out.word(j, r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
            out.end(col0 + c * 32, (int)(split * p.split_rows) + row - out.lane, warp_on && col0 + c * 32 < p.n);
        }
        return;
    }
    uint32_t w[kPiece / 2];
#pragma unroll
    for (int c = 0; c < kPiece / 32; ++c) {
        uint32_t r[32];
        tc::tmem_load32(tmem + c * 32, r);
        tc::tmem_load_wait(r);
        const int left = on ? p.n - (col0 + c * 32) : 0;
        if (p.acc_read) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < left) r[j] = __float_as_uint(__uint_as_float(r[j]) + acc[c * 32 + j]);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
            w[c * 16 + j] = pack2(__uint_as_float(r[2 * j]) * scale, __uint_as_float(r[2 * j + 1]) * scale);
    }
    release();
#pragma unroll
    for (int c = 0; c < kPiece / kBox; ++c) {
        out.begin();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = c * 32 + j * 4;
            out.word(j, w[i], w[i + 1], w[i + 2], w[i + 3]);
        }
        const int row0 = row - out.lane, col = col0 + c * kBox;
        if (p.boxes) out.end(col, row0, warp_on && col < p.n);
        else out.end_rows(p.out + row0 * p.ld_out + col, p.ld_out, warp_on ? p.m - row0 : 0, p.n - col, p.pairs);
    }
}

template <int PRODUCT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const ProductParams p, const __grid_constant__ CUtensorMap amap,
                   const __grid_constant__ CUtensorMap bmap, const __grid_constant__ CUtensorMap omap)
{
    constexpr bool a_mn = PRODUCT == kDw, b_mn = PRODUCT != kLogits;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *buffers = ring + kStages * kStage;
    uint64_t *full = reinterpret_cast<uint64_t *>(buffers + 8 * kBuffer);
    uint64_t *empty = full + kStages, *ready = empty + kStages, *taken = ready + 2, *drained = taken + 2;
    uint32_t *slot = reinterpret_cast<uint32_t *>(drained + 1);
    // the roles' loops are uniform over a warp (one lane issues): the copies and
    // matrix instructions take their operands from uniform registers
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)tc::pair_rank(), pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
    if (warp == 0 && lane == 0) {
        tc::prefetch_map(&amap);
        tc::prefetch_map(&bmap);
        for (int i = 0; i < kStages; ++i) {
            tc::bar_init(full + i, 1);
            tc::bar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(ready + i, 1);
            tc::bar_init(taken + i, 2 * 8);            // a lane of each epilogue warp of the pair
        }
        tc::bar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::tmem_alloc<512>(slot);
    chain_start();
    tc::fence_before();
    tc::pair_sync();
    tc::fence_after();
    const uint32_t tmem = *slot;
    chain_wait();
    if (PRODUCT == kLogits && blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
    const int tiles = p.mt * p.nt * p.splits;
    bool aborted = false;
    if (warp == 0) {
        // both CTAs copy their halves; the bytes of both are counted on the leader's barrier
        const bool one = tc::elect_one();
        const uint32_t full_at = tc::leader_addr(full);
        int s = 0;
        uint32_t phase = 0;
        long long issued = 0;
        for (int i = pair; i < tiles && !aborted; i += pairs) {
            const Tile t = tile_at(p, i);
            const int m0 = t.m * kTileM + rank * kHalfM, n0 = t.n * kTileN + rank * kHalfN;
            const int k1 = min(p.kblocks, (t.split + 1) * p.per_split);
            for (int k = t.split * p.per_split; k < k1; ++k) {
                if (!tc::warp_wait(empty + s, phase ^ 1, aborted)) break;
                uint8_t *a = ring + s * kStage, *b = a + kStageA;
                const uint32_t bar = full_at + s * 8;
                if (one) {
                    if (rank == 0) tc::bar_expect(full + s, 2 * kStage);
                    if constexpr (a_mn) {
#pragma unroll
                        for (int j = 0; j < kHalfM / kBox; ++j)
                            tc::load_box(a + j * kBox * kTileK * 2, &amap, m0 + j * kBox, k * kTileK, bar);
                    } else {
                        tc::load_box(a, &amap, k * kTileK, m0, bar);
                    }
                    if constexpr (b_mn) {
#pragma unroll
                        for (int j = 0; j < kHalfN / kBox; ++j)
                            tc::load_box(b + j * kBox * kTileK * 2, &bmap, n0 + j * kBox, k * kTileK, bar);
                    } else {
                        tc::load_box(b, &bmap, k * kTileK, n0, bar);
                    }
                }
                ++issued;
                if (++s == kStages) { s = 0; phase ^= 1; }
            }
        }
        // Every copy has landed and every release has arrived before the CTA's
        // memory goes away: a released stage's copies were read.
        bool gave_up = false;
        for (long long j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
            tc::warp_wait(empty + j % kStages, (uint32_t)(j / kStages & 1), gave_up);
    } else if (warp == 1) {
        if (rank == 0) {
            // One lane feeds both SMs' tensor cores 512 cycles of work per step
            // of 64: what is computed per step is kept to an add per operand.
            const bool one = tc::elect_one();
            constexpr uint32_t idesc = tc::instr_desc(kTileM, kTileN, a_mn, b_mn);
            constexpr uint32_t high = tc::desc_high(1024);
            constexpr uint32_t lead_a = a_mn ? kBox * kTileK * 2 : 16, lead_b = b_mn ? kBox * kTileK * 2 : 16;
            constexpr uint32_t step_a = (a_mn ? 2048 : 32) / 16, step_b = (b_mn ? 2048 : 32) / 16;
            const uint32_t a0 = tc::desc_low(tc::smem_addr(ring), lead_a);
            const uint32_t b0 = tc::desc_low(tc::smem_addr(ring) + kStageA, lead_b);
            int s = 0;
            uint32_t phase = 0, count = 0;
            for (int i = pair; i < tiles && !aborted; i += pairs) {
                const Tile t = tile_at(p, i);
                int left = min(p.kblocks, (t.split + 1) * p.per_split) - t.split * p.per_split;
                while (left > 0 && !aborted) {
                    const int n = min(left, kSegment<PRODUCT>);
                    const uint32_t half = count & 1, d = tmem + half * kTileN;
                    if (!tc::warp_wait(taken + half, (count >> 1 & 1) ^ 1, aborted)) break;
                    tc::fence_after();
                    for (int k = 0; k < n; ++k) {
                        if (!tc::warp_wait(full + s, phase, aborted)) break;
                        tc::fence_after();
                        const uint32_t a = a0 + s * (kStage / 16), b = b0 + s * (kStage / 16);
                        if (one) {
#pragma unroll
                            for (int j = 0; j < kTileK / 16; ++j)
                                tc::mma(d, a + j * step_a, high, b + j * step_b, high, idesc, j > 0 || k > 0);
                            tc::mma_commit(empty + s);
                            if (k + 1 == n) tc::mma_commit(ready + half);
                        }
                        if (++s == kStages) { s = 0; phase ^= 1; }
                    }
                    ++count;
                    left -= n;
                }
            }
            if (aborted) {      // instructions still running finish before the memory goes away
                bool gave_up = false;
                if (one) tc::mma_commit(drained);
                tc::warp_wait(drained, 0, gave_up);
            }
        }
    } else {
        // the first four of these warps take columns [0, 128) of a tile, the
        // others the rest; a warp reads the 32 rows of tensor memory that its
        // number modulo 4 allows
        const int part = (warp - kFirstEpilogueWarp) >> 2, quarter = warp & 3;
        const Out out{buffers + (warp - kFirstEpilogueWarp) * kBuffer, &omap, lane};
        uint32_t count = 0;
        // the next accumulator is complete
        auto next = [&](uint32_t &addr, uint32_t &half) {
            half = count & 1;
            const bool ok = tc::warp_wait(ready + half, count >> 1 & 1, aborted);
            ++count;
            tc::fence_after();
            addr = tmem + half * kTileN + part * kPiece + ((uint32_t)quarter * 32 << 16);
            return ok;
        };
        const uint32_t taken_at[2] = {tc::leader_addr(taken), tc::leader_addr(taken + 1)};
        // the accumulator has been read: one arrival per warp, on the leader's barrier
        auto release = [&](uint32_t half) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive_at(taken_at[half]);
        };
        for (int i = pair; i < tiles; i += pairs) {
            const Tile t = tile_at(p, i);
            const int row = t.m * kTileM + rank * kHalfM + quarter * 32 + lane, col0 = t.n * kTileN + part * kPiece;
            uint32_t addr, half;
            if constexpr (PRODUCT == kLogits) {
                float z[kPiece];
                bool ok = true;
                for (int k = 0; k < p.kblocks; k += kSegment<PRODUCT>) {
                    if (!(ok = next(addr, half))) break;
#pragma unroll
                    for (int c = 0; c < kPiece / 32; ++c) {
                        uint32_t r[32];
                        tc::tmem_load32(addr + c * 32, r);
                        tc::tmem_load_wait(r);
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float x = __uint_as_float(r[j]);
                            z[c * 32 + j] = k ? z[c * 32 + j] + x : x;
                        }
                    }
                    release(half);
                }
                if (!ok) break;
                if (col0 + kPiece <= p.n) reduce_piece<false>(p, z, row, col0, out);
                else if (col0 < p.n) reduce_piece<true>(p, z, row, col0, out);
            } else {
                if (!next(addr, half)) break;
                store_piece(p, addr, row, col0, t.split, out, [&] { release(half); });
            }
        }
        if (lane == 0) tc::stores_done();
    }
    __syncwarp();
    tc::fence_before();
    tc::pair_sync();
    tc::fence_after();
    if (warp == 1) tc::tmem_free<512>(tmem);
}

// ------------------------------------------------------------------ losses
// What the row kernels share over a call.
struct Totals {
    unsigned int done;       // blocks of the merge that have finished
    float scale;             // 1 / A
    float loss;              // sum of weight * row loss of the chunks so far
};

struct MergeParams {
    const float2 *stats;
    const float *target_logit;
    const int64_t *targets;       // of the chunk
    const int64_t *all_targets;
    const float *row_weight;      // of all tokens, or null
    float *row_loss, *lse;        // of the chunk (scratch when the caller wants none)
    float *weight;                // of the chunk: the weight of a token that counts and has a valid target, else 0
    float *loss;
    Totals *totals;
    long long tokens, first, ignore;   // all tokens, the chunk's first
    int rows, pieces, vocab, mean;
    int first_chunk, last_chunk;
    int blocks;                   // that merge; those behind them copy h
    const uint16_t *h;            // of the chunk, rows on 16 bytes
    uint16_t *kept;
    long long ld_h, ld_kept;
    int dim, copy_rows;           // of h; rows of it that a block copies
};

// Weight of a row in the gradients: 0 for a token that does not count or whose target is no entry.
__device__ __forceinline__ float row_weight(const MergeParams &p, int row)
{
    const long long target = p.targets[row];
    return target == p.ignore || target < 0 || target >= p.vocab ? 0.0f : p.row_weight ? p.row_weight[p.first + row] : 1.0f;
}

// A running sum with the rounding errors carried along (compensated
// summation): thousands of terms per thread stay at one rounding, without fp64,
// whose units are few here (32 warps adding doubles took 20 us).
struct Sum {
    float s = 0.0f, lost = 0.0f;
    __device__ __forceinline__ void add(float x)
    {
        const float y = __fsub_rn(x, lost), t = __fadd_rn(s, y);
        const float l = __fsub_rn(__fsub_rn(t, s), y);
        lost = l == l ? l : 0.0f;          // an infinite sum stays infinite
        s = t;
    }
};

// The block's total in a fixed order, in every thread of warp 0.
__device__ __forceinline__ float block_total(float x, float *red)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = threadIdx.x < blockDim.x >> 5 ? red[threadIdx.x] : 0.0f;
    if (threadIdx.x < 32)
#pragma unroll
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    return x;
}

// Adds a piece's exponentials: (maximum, sum) pairs.  Where both maxima are
// -inf (or only NaN was seen), the sums are 0 or NaN and stay so.
__device__ __forceinline__ void add_piece(float &top, float &sum, float2 s)
{
    const float t = fmaxf(top, s.x);
    if (t == -INFINITY) {
        sum += s.y;
    } else {
        sum = sum * exp2_fast((top - t) * kLog2e) + s.y * exp2_fast((s.x - t) * kLog2e);
        top = t;
    }
}

// lse and loss of each row from its pieces (lane by lane over the rows, so
// that a warp reads neighbouring rows); the last block adds the losses.
//
// With gradients, more blocks copy the hidden states for dW = G^T h, with zeros
// where a row's weight is zero: a row of G that is zero would still make NaN of
// a masked token's infinities.  (4 bytes per element of h, on SMs that the merge
// leaves idle: 4096 x 32768 x 1024 with gradients 560 us, 555 without.  In the
// pass that forms G, which has no registers to spare, it took 569, and 596 in
// blocks of its own there.)
constexpr int kMergeThreads = 1024, kMergeRows = 32, kCopyWords = 4 * kMergeThreads;
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const MergeParams p)
{
    __shared__ float2 part[kMergeThreads / 32][kMergeRows];
    __shared__ float red[kMergeThreads / 32];
    __shared__ bool last;
    chain_start();
    chain_wait();
    if ((int)blockIdx.x >= p.blocks) {
        const int r0 = ((int)blockIdx.x - p.blocks) * p.copy_rows, words = (p.dim + 7) / 8;
        const int n = min(p.copy_rows, p.rows - r0) * words;
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += kMergeThreads) {
            const int r = i / words, c = (i - r * words) * 8;
            const uint16_t *from = p.h + (r0 + r) * p.ld_h + c;
            uint16_t *to = p.kept + (r0 + r) * p.ld_kept + c;
            const bool zero = row_weight(p, r0 + r) == 0.0f;
            if (c + 8 <= p.dim) {
                const uint4 v = *reinterpret_cast<const uint4 *>(from);
                *reinterpret_cast<uint4 *>(to) = zero ? make_uint4(0, 0, 0, 0) : v;
            } else {
                for (int j = 0; c + j < p.dim; ++j) to[j] = zero ? (uint16_t)0 : from[j];
            }
        }
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x * kMergeRows + lane;
    float top = -INFINITY, sum = 0.0f;
    if (row < p.rows) {
#pragma unroll 4
        for (int i = warp; i < p.pieces; i += kMergeThreads / 32) add_piece(top, sum, p.stats[(long long)i * p.rows + row]);
    }
    part[warp][lane] = make_float2(top, sum);
    __syncthreads();
    if (warp == 0 && row < p.rows) {
#pragma unroll 8
        for (int i = 1; i < kMergeThreads / 32; ++i) add_piece(top, sum, part[i][lane]);
        const float lse = top + logf(sum);
        const long long target = p.targets[row];
        const bool counts = target != p.ignore, valid = target >= 0 && target < p.vocab;
        p.lse[row] = lse;
        p.row_loss[row] = !counts ? 0.0f : valid ? lse - p.target_logit[row] : __uint_as_float(0x7FC00000u);
        p.weight[row] = row_weight(p, row);
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&p.totals->done, 1u) == (unsigned)p.blocks - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    Sum losses, weights;
    for (int i = threadIdx.x; i < p.rows; i += kMergeThreads)
        if (p.targets[i] != p.ignore)
            losses.add((p.row_weight ? p.row_weight[p.first + i] : 1.0f) * __ldcg(p.row_loss + i));
    float loss = block_total(losses.s, red), weight = 0.0f;
    if (p.mean && p.first_chunk) {
        for (long long i = threadIdx.x; i < p.tokens; i += kMergeThreads)
            if (p.all_targets[i] != p.ignore) weights.add(p.row_weight ? p.row_weight[i] : 1.0f);
        weight = block_total(weights.s, red);
    }
    if (threadIdx.x == 0) {
        Totals *t = p.totals;
        if (p.first_chunk) t->scale = !p.mean ? 1.0f : weight != 0.0f ? 1.0f / weight : 0.0f;
        else loss += t->loss;
        t->loss = loss;
        if (p.last_chunk) *p.loss = loss * t->scale;
    }
}

// Codes to G, in place: G = weight (exp(top - lse - code / 2048) - [col == target]).
// 4 bytes of traffic per element; the conversion of a code goes through the
// mantissa of 2^23 + code, since the conversion instructions share the
// exponential's unit, which alone needs 0.4 of the time of the bytes.
struct GradParams {
    uint16_t *codes;
    const float2 *stats;
    const float *lse, *weight;
    const int64_t *targets;
    long long ld;
    int rows, vocab;
};
constexpr int kGradThreads = 256, kGradSteps = 4;
constexpr int kGradCols = kGradThreads * 8 * kGradSteps;      // of a block
__global__ void __launch_bounds__(kGradThreads) grad_kernel(const GradParams p)
{
    chain_start();
    chain_wait();
    const int row = blockIdx.y;
    const int col0 = (int)blockIdx.x * kGradCols + (int)threadIdx.x * 8;
    uint16_t *codes = p.codes + row * p.ld;
    const float w = p.weight[row];
    if (w == 0.0f) {
#pragma unroll
        for (int k = 0; k < kGradSteps; ++k)
            if (col0 + k * kGradThreads * 8 < p.vocab)
                *reinterpret_cast<uint4 *>(codes + col0 + k * kGradThreads * 8) = make_uint4(0, 0, 0, 0);
        return;
    }
    uint4 q[kGradSteps];
    float base[kGradSteps];
    const float lse = p.lse[row], none = lse - lse;   // 0; NaN in a row of NaN logits, whose codes tell nothing
#pragma unroll
    for (int k = 0; k < kGradSteps; ++k) {
        const int col = col0 + k * kGradThreads * 8;
        if (col < p.vocab) {
            q[k] = *reinterpret_cast<const uint4 *>(codes + col);
            base[k] = p.stats[(long long)(col / kPiece) * p.rows + row].x;
        }
    }
    const long long target = p.targets[row];
#pragma unroll
    for (int k = 0; k < kGradSteps; ++k) {
        const int col = col0 + k * kGradThreads * 8;
        if (col >= p.vocab) break;
        const float shift = (base[k] - lse) * kLog2e;
        const uint32_t c[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t bits = __byte_perm(c[j >> 1], 0x4B00u, j & 1 ? 0x5432 : 0x5410);
            const float code = __uint_as_float(bits) - 8388608.0f;
            // the last code stands for everything from 32 below the maximum on
            g[j] = code == 65535.0f ? none : exp2_fast(fmaf(code, -kLog2e / kSteps, shift));
        }
        const long long d = target - col;
        if (d >= 0 && d < 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j == (int)d) g[j] -= 1.0f;
        }
        *reinterpret_cast<uint4 *>(codes + col) = make_uint4(pack2(g[0] * w, g[1] * w), pack2(g[2] * w, g[3] * w),
                                                             pack2(g[4] * w, g[5] * w), pack2(g[6] * w, g[7] * w));
    }
}

// dh of a row range from the splits' sums, in split order.
__global__ void __launch_bounds__(256) join_kernel(const float *acc, int splits, long long split_rows, long long ld_acc,
                                                   int cols, const float *scale, bf16 *out, long long ld)
{
    chain_start();
    chain_wait();
    const long long row = blockIdx.y;
    const int col = (int)(blockIdx.x * 256 + threadIdx.x);
    if (col >= cols) return;
    const float *src = acc + row * ld_acc + col;
    float s = 0.0f;
    for (int k = 0; k < splits; ++k) s += src[k * split_rows * ld_acc];
    out[row * ld + col] = __float2bfloat16_rn(s * *scale);
}

// Copies an operand into rows of whole 128-byte lines.  Eight elements per
// thread, read as 32-bit words even where the rows are only 2-byte aligned;
// single elements at the tensor's start and at the rows' ends, so that nothing
// outside the rows' span is read.
constexpr int kPackThreads = 256;
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const uint16_t *src, long long ld, uint16_t *dst,
                                                            long long ld_dst, long long rows, int cols, int block_rows)
{
    chain_start();
    chain_wait();
    const int chunks = (cols + 7) / 8;
    const long long r0 = (long long)blockIdx.x * block_rows;
    const int n = (int)min((long long)block_rows, rows - r0) * chunks;
    for (int i = threadIdx.x; i < n; i += kPackThreads) {
        const int r = i / chunks, c = (i - r * chunks) * 8;
        const uint16_t *from = src + (r0 + r) * ld + c;
        uint16_t *to = dst + (r0 + r) * ld_dst + c;
        const uint32_t odd = (uint32_t)(reinterpret_cast<uintptr_t>(from) & 2);
        if (c + 8 < cols && (!odd || r0 + r + c > 0)) {
            const uint32_t *word = reinterpret_cast<const uint32_t *>(reinterpret_cast<uintptr_t>(from) & ~(uintptr_t)3);
            uint32_t w[5];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = word[j];
            w[4] = odd ? word[4] : 0u;
            *reinterpret_cast<uint4 *>(to) =
                make_uint4(__funnelshift_r(w[0], w[1], odd * 8), __funnelshift_r(w[1], w[2], odd * 8),
                           __funnelshift_r(w[2], w[3], odd * 8), __funnelshift_r(w[3], w[4], odd * 8));
        } else {
            for (int j = 0; j < 8 && c + j < cols; ++j) to[j] = from[j];
        }
    }
}

__global__ void zero_loss_kernel(float *loss) { *loss = 0.0f; }

// ------------------------------------------------------------------ host
bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

int launched(cudaError_t e)
{
    const int rc = cuda_status(e);
    if (rc == AMSIM_OK) count_launch();
    return rc;
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Map of a bf16 (or fp32) matrix, `inner` contiguous elements by `outer` rows of
// stride `ld`; boxes of 128 bytes by `box` rows, zeros outside.
int matrix_map(CUtensorMap *map, const void *base, long long inner, long long outer, long long ld, int box,
               bool fp32 = false)
{
    static const EncodeTiled encode = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
    if (!encode) return AMSIM_EUNSUPPORTED;
    const int size = fp32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * size};
    const cuuint32_t boxes[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box}, ones[2] = {1, 1};
    return encode(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void *>(base), dims, strides, boxes, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? AMSIM_OK
               : AMSIM_EUNSUPPORTED;
}

struct Matrix {
    const bf16 *p;
    long long ld;
};

int check(const amsim_vocab_loss_desc *d)
{
    if (!d || d->tokens < 0 || d->tokens > (int64_t)1 << 40 || d->vocab < 1 || d->vocab > 0x7FFFFF00 || d->dim < 1 ||
        d->dim > 0x7FFFFF00)
        return AMSIM_EINVAL;
    for (int64_t ld : {d->ld_h, d->ld_w, d->ld_dh, d->ld_dw})
        if (ld != 0 && (ld < d->dim || ld > (int64_t)1 << 38)) return AMSIM_EINVAL;
    if (d->reduction != AMSIM_REDUCE_MEAN && d->reduction != AMSIM_REDUCE_SUM) return AMSIM_EINVAL;
    return AMSIM_OK;
}

int device_sms()
{
    int sms = 0;
    return current_device(&sms) < 0 ? 0 : sms;
}

// Scratch of a call over chunks of `rows` tokens.
struct Layout {
    size_t totals, row_loss, lse, weight, target_logit, stats, codes, kept, dw_acc, dh_acc, pack_h, pack_w, bytes;
    long long ld_codes, ld_pack, ld_acc, split_rows;
    int dh_splits;
};

constexpr size_t kCodesCap = (size_t)4 << 30;
constexpr long long kMostRows = 32768;         // of a chunk

// Parts of dh's reduction over the vocabulary when its tiles do not fill the
// GPU: each part's fp32 sums go to scratch and a join adds them.
int dh_splits(long long rows, const amsim_vocab_loss_desc *d, int sms)
{
    const long long tiles = ((rows + kTileM - 1) / kTileM) * ((d->dim + kTileN - 1) / kTileN);
    const int kblocks = (d->vocab + kTileK - 1) / kTileK, pairs = sms / 2;
    if (tiles * 2 > pairs) return 1;
    return (int)std::max<long long>(1, std::min<long long>(pairs / tiles, kblocks / 8));
}

Layout layout(const amsim_vocab_loss_desc *d, bool grad, long long rows, bool pack_h, bool pack_w, int sms)
{
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t r = at;
        at += up256(n);
        return r;
    };
    const long long pieces = (d->vocab + kPiece - 1) / kPiece;
    l.totals = take(sizeof(Totals));
    l.row_loss = take((size_t)rows * 4);
    l.lse = take((size_t)rows * 4);
    l.weight = take((size_t)rows * 4);
    l.target_logit = take((size_t)rows * 4);
    l.stats = take((size_t)pieces * rows * 8);
    l.ld_codes = (d->vocab + 63) & ~63LL;       // rows of whole 128-byte lines
    l.ld_pack = (d->dim + 63) & ~63LL;
    l.ld_acc = (d->dim + 3) & ~3LL;
    l.split_rows = (rows + kTileM - 1) / kTileM * kTileM;   // whole tiles: a box never reaches the next split
    l.dh_splits = 1;
    if (grad) {
        l.codes = take((size_t)rows * l.ld_codes * 2);
        l.kept = take((size_t)rows * l.ld_pack * 2);
        if (rows < d->tokens) l.dw_acc = take((size_t)d->vocab * l.ld_acc * 4);
        l.dh_splits = dh_splits(rows, d, sms);
        if (l.dh_splits > 1) l.dh_acc = take((size_t)l.dh_splits * l.split_rows * l.ld_acc * 4);
    }
    if (pack_h) l.pack_h = take((size_t)d->tokens * l.ld_pack * 2);
    if (pack_w) l.pack_w = take((size_t)d->vocab * l.ld_pack * 2);
    l.bytes = at;
    return l;
}

bool tma_rows(const void *p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

// An operand is copied into aligned rows when TMA cannot take its own (base or
// stride off 16 bytes).  h is copied also when its rows are not whole 128-byte
// lines, so that each 128-byte row of a tile straddles two, and there are
// enough tokens: 1024 x 50021 x 1000 with gradients takes 298 us without the
// copy and 273 with it, 512 tokens 186 and 183, 128 tokens 123 and 128.  W is
// not: the copy gained 1 % at 4096 tokens and lost 5 % at 1531.
constexpr int64_t kPackTokens = 1024;
bool pack_h(const void *h, int64_t ld, int64_t tokens)
{
    return !tma_rows(h, ld) || (tokens >= kPackTokens && (ld % 64 != 0 || !aligned(h, 128)));
}

long long full_rows(const amsim_vocab_loss_desc *d)
{
    long long rows = std::min<long long>(d->tokens, kMostRows);
    const long long cap = (long long)(kCodesCap / ((size_t)((d->vocab + 63) & ~63LL) * 2));
    if (rows > cap) rows = std::max<long long>(kTileM, cap / kTileM * kTileM);
    return std::min<long long>(rows, d->tokens);
}

template <int PRODUCT>
int launch_product(bool chained, const ProductParams &p, const CUtensorMap &a, const CUtensorMap &b,
                   const CUtensorMap &o, int sms, cudaStream_t st)
{
    static std::atomic<uint64_t> allowed{0};          // devices on which the kernel may have its shared memory
    int n = 0;
    const int dev = current_device(&n);
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (!bit || !(allowed.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(product_kernel<PRODUCT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return cuda_status(e);
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    const long long tiles = (long long)p.mt * p.nt * p.splits;
    if (tiles > 0x7FFFFFFFLL - sms) return AMSIM_EUNSUPPORTED;
    const int grid = 2 * (int)std::min<long long>(tiles, std::max(1, sms / 2));
    return launched(chain_launch(chained, product_kernel<PRODUCT>, grid, kThreads, kSmem, st, p, a, b, o));
}

ProductParams product(long long m, long long n, long long k, int splits)
{
    ProductParams p{};
    p.m = (int)m;
    p.n = (int)n;
    p.kblocks = (int)((k + kTileK - 1) / kTileK);
    p.mt = (int)((m + kTileM - 1) / kTileM);
    p.nt = (int)((n + kTileN - 1) / kTileN);
    p.per_split = (p.kblocks + splits - 1) / splits;
    p.splits = (p.kblocks + p.per_split - 1) / p.per_split;
    p.group = 8;
    return p;
}

int run(const amsim_vocab_loss_desc *d, bool grad, const void *h, const void *w, const int64_t *targets,
        const float *row_weight, float *loss, float *row_loss, float *lse, void *dh, void *dw, void *ws,
        size_t ws_bytes, cudaStream_t st)
{
    int rc = check(d);
    if (rc) return rc;
    if (!loss || !w || !aligned(w, 2) || !aligned(loss, 4) || (grad && (!dw || !aligned(dw, 2)))) return AMSIM_EINVAL;
    const long long ld_h = d->ld_h ? d->ld_h : d->dim, ld_w = d->ld_w ? d->ld_w : d->dim;
    const long long ld_dh = d->ld_dh ? d->ld_dh : d->dim, ld_dw = d->ld_dw ? d->ld_dw : d->dim;
    if (d->tokens == 0) {
        if (grad && cudaMemset2DAsync(dw, (size_t)ld_dw * 2, 0, (size_t)d->dim * 2, (size_t)d->vocab, st) !=
                        cudaSuccess) {
            cudaGetLastError();
            return AMSIM_ECUDA;
        }
        zero_loss_kernel<<<1, 1, 0, st>>>(loss);
        return launched(cudaGetLastError());
    }
    if (!h || !targets || !ws || !aligned(h, 2) || !aligned(targets, 8) || !aligned(row_weight, 4) ||
        !aligned(row_loss, 4) || !aligned(lse, 4) || !aligned(ws, 256) || (grad && (!dh || !aligned(dh, 2))))
        return AMSIM_EINVAL;
    const int sms = device_sms();
    if (!sms) return AMSIM_ECUDA;
    const bool copy_h = pack_h(h, ld_h, d->tokens), copy_w = !tma_rows(w, ld_w);
    long long rows = full_rows(d);
    Layout l = layout(d, grad, rows, copy_h, copy_w, sms);
    while (l.bytes > ws_bytes) {              // smaller chunks: whole row tiles, down to one
        if (rows <= kTileM) return AMSIM_EINVAL;
        rows = std::max<long long>(kTileM, (rows / 2 + kTileM - 1) / kTileM * kTileM);
        l = layout(d, grad, rows, copy_h, copy_w, sms);
    }
    uint8_t *base = static_cast<uint8_t *>(ws);
    Totals *totals = reinterpret_cast<Totals *>(base + l.totals);
    bool chained = false;                     // the first kernel follows whatever the stream holds
    Matrix H{static_cast<const bf16 *>(h), ld_h}, W{static_cast<const bf16 *>(w), ld_w};
    auto pack = [&](Matrix &m, size_t off, long long n) {
        bf16 *dst = reinterpret_cast<bf16 *>(base + off);
        const int block_rows = std::max(1, 2048 / ((d->dim + 7) / 8));
        const int r = launched(chain_launch(chained, pack_kernel, (unsigned)((n + block_rows - 1) / block_rows),
                                            kPackThreads, 0, st, reinterpret_cast<const uint16_t *>(m.p), m.ld,
                                            reinterpret_cast<uint16_t *>(dst), l.ld_pack, n, d->dim, block_rows));
        m = Matrix{dst, l.ld_pack};
        chained = true;
        return r;
    };
    if (copy_h && (rc = pack(H, l.pack_h, d->tokens))) return rc;
    if (copy_w && (rc = pack(W, l.pack_w, d->vocab))) return rc;

    uint16_t *codes = grad ? reinterpret_cast<uint16_t *>(base + l.codes) : nullptr;
    const bf16 *g = reinterpret_cast<const bf16 *>(codes);
    float2 *stats = reinterpret_cast<float2 *>(base + l.stats);
    float *target_logit = reinterpret_cast<float *>(base + l.target_logit);
    float *weight = reinterpret_cast<float *>(base + l.weight);
    float *dw_acc = reinterpret_cast<float *>(base + l.dw_acc);
    for (long long t0 = 0; t0 < d->tokens; t0 += rows) {
        const long long n = std::min(rows, d->tokens - t0);
        const bool first = t0 == 0, last = t0 + n == d->tokens;
        CUtensorMap am, bm, om;
        ProductParams p = product(n, d->vocab, d->dim, 1);
        p.targets = targets + t0;
        p.target_logit = target_logit;
        p.stats = stats;
        p.done = &totals->done;
        p.codes = codes;
        if ((rc = matrix_map(&am, H.p + t0 * H.ld, d->dim, n, H.ld, kHalfM)) ||
            (rc = matrix_map(&bm, W.p, d->dim, d->vocab, W.ld, kHalfN)) ||
            (grad && (rc = matrix_map(&om, codes, d->vocab, n, l.ld_codes, 32))) ||
            (rc = launch_product<kLogits>(chained, p, am, bm, grad ? om : am, sms, st)))
            return rc;
        MergeParams q{};
        q.stats = stats;
        q.target_logit = target_logit;
        q.targets = targets + t0;
        q.all_targets = targets;
        q.row_weight = row_weight;
        q.row_loss = row_loss ? row_loss + t0 : reinterpret_cast<float *>(base + l.row_loss);
        q.lse = lse ? lse + t0 : reinterpret_cast<float *>(base + l.lse);
        q.weight = weight;
        q.loss = loss;
        q.totals = totals;
        q.tokens = d->tokens;
        q.first = t0;
        q.ignore = d->ignore_index;
        q.rows = (int)n;
        q.pieces = (d->vocab + kPiece - 1) / kPiece;
        q.vocab = d->vocab;
        q.mean = d->reduction == AMSIM_REDUCE_MEAN;
        q.first_chunk = first;
        q.last_chunk = last;
        chained = true;
        q.blocks = (int)((n + kMergeRows - 1) / kMergeRows);
        int copies = 0;
        bf16 *kept = reinterpret_cast<bf16 *>(base + l.kept);
        if (grad) {
            q.h = reinterpret_cast<const uint16_t *>(H.p + t0 * H.ld);
            q.kept = reinterpret_cast<uint16_t *>(kept);
            q.ld_h = H.ld;
            q.ld_kept = l.ld_pack;
            q.dim = d->dim;
            q.copy_rows = std::max(1, kCopyWords / ((d->dim + 7) / 8));
            copies = (int)((n + q.copy_rows - 1) / q.copy_rows);
        }
        rc = launched(chain_launch(true, merge_kernel, (unsigned)(q.blocks + copies), kMergeThreads, 0, st, q));
        if (rc) return rc;
        if (!grad) continue;
        GradParams e{codes, stats, q.lse, weight, targets + t0, l.ld_codes, (int)n, d->vocab};
        rc = launched(chain_launch(true, grad_kernel, dim3((unsigned)((d->vocab + kGradCols - 1) / kGradCols), (unsigned)n),
                                   kGradThreads, 0, st, e));
        if (rc) return rc;
        // dh = G W
        p = product(n, d->dim, d->vocab, l.dh_splits);
        bf16 *dh_out = static_cast<bf16 *>(dh) + t0 * ld_dh;
        p.scale = &totals->scale;
        if (p.splits > 1) {
            p.acc = reinterpret_cast<float *>(base + l.dh_acc);
            p.ld_acc = l.ld_acc;
            p.split_rows = l.split_rows;
            p.acc_write = 1;
            rc = matrix_map(&om, p.acc, d->dim, p.splits * l.split_rows, l.ld_acc, 32, true);
        } else {
            p.out = dh_out;
            p.ld_out = ld_dh;
            p.boxes = tma_rows(dh_out, ld_dh);
            p.pairs = aligned(dh_out, 4) && ld_dh % 2 == 0;
            om = am;
            if (p.boxes) rc = matrix_map(&om, dh_out, d->dim, n, ld_dh, 32);
        }
        if (rc || (rc = matrix_map(&am, g, d->vocab, n, l.ld_codes, kHalfM)) ||
            (rc = matrix_map(&bm, W.p, d->dim, d->vocab, W.ld, kTileK)) ||
            (rc = launch_product<kDh>(true, p, am, bm, om, sms, st)))
            return rc;
        if (p.splits > 1) {
            rc = launched(chain_launch(true, join_kernel, dim3((unsigned)((d->dim + 255) / 256), (unsigned)n), 256, 0, st,
                                       (const float *)p.acc, p.splits, l.split_rows, l.ld_acc, d->dim,
                                       (const float *)&totals->scale, dh_out, ld_dh));
            if (rc) return rc;
        }
        // dW = G^T h, over the chunks so far
        p = product(d->vocab, d->dim, n, 1);
        p.scale = &totals->scale;
        if (!(first && last)) {
            p.acc = dw_acc;
            p.ld_acc = l.ld_acc;
            p.acc_read = !first;
            p.acc_write = !last;
        }
        om = am;
        if (last) {
            p.out = static_cast<bf16 *>(dw);
            p.ld_out = ld_dw;
            p.boxes = tma_rows(dw, ld_dw);
            p.pairs = aligned(dw, 4) && ld_dw % 2 == 0;
            if (p.boxes) rc = matrix_map(&om, dw, d->dim, d->vocab, ld_dw, 32);
        } else {
            rc = matrix_map(&om, dw_acc, d->dim, d->vocab, l.ld_acc, 32, true);
        }
        if (rc || (rc = matrix_map(&am, g, d->vocab, n, l.ld_codes, kTileK)) ||
            (rc = matrix_map(&bm, kept, d->dim, n, l.ld_pack, kTileK)) ||
            (rc = launch_product<kDw>(true, p, am, bm, om, sms, st)))
            return rc;
    }
    return AMSIM_OK;
}

}  // namespace

extern "C" int amsim_vocab_loss(const amsim_vocab_loss_desc *desc, const void *h, const void *w,
                                const int64_t *targets, const float *row_weight, float *loss, float *row_loss,
                                float *lse, void *ws, size_t ws_bytes, amsim_stream_t stream)
{
    return run(desc, false, h, w, targets, row_weight, loss, row_loss, lse, nullptr, nullptr, ws, ws_bytes,
               static_cast<cudaStream_t>(stream));
}

extern "C" int amsim_vocab_loss_grad(const amsim_vocab_loss_desc *desc, const void *h, const void *w,
                                     const int64_t *targets, const float *row_weight, float *loss, float *row_loss,
                                     float *lse, void *dh, void *dw, void *ws, size_t ws_bytes, amsim_stream_t stream)
{
    return run(desc, true, h, w, targets, row_weight, loss, row_loss, lse, dh, dw, ws, ws_bytes,
               static_cast<cudaStream_t>(stream));
}

// The sizes by the descriptor alone leave room for packed copies of h and w,
// whose base addresses may be off 16 bytes.
extern "C" size_t amsim_vocab_loss_workspace_size(const amsim_vocab_loss_desc *desc, int which)
{
    if (check(desc) || (which != 0 && which != 1) || desc->tokens == 0) return 0;
    const int sms = device_sms();
    return layout(desc, which == 1, full_rows(desc), true, true, sms ? sms : 1).bytes;
}

extern "C" size_t amsim_vocab_loss_workspace_size_at(const amsim_vocab_loss_desc *desc, int which, const void *h,
                                                     const void *w)
{
    if (check(desc) || (which != 0 && which != 1) || desc->tokens == 0) return 0;
    const int sms = device_sms();
    return layout(desc, which == 1, full_rows(desc), pack_h(h, desc->ld_h ? desc->ld_h : desc->dim, desc->tokens),
                  !tma_rows(w, desc->ld_w ? desc->ld_w : desc->dim), sms ? sms : 1).bytes;
}

extern "C" size_t amsim_vocab_loss_workspace_min(const amsim_vocab_loss_desc *desc, int which)
{
    if (check(desc) || (which != 0 && which != 1) || desc->tokens == 0) return 0;
    const int sms = device_sms();
    // one chunk needs no sums of dw between chunks, and may need less than several
    return std::min(layout(desc, which == 1, std::min<long long>(desc->tokens, kTileM), true, true, sms ? sms : 1).bytes,
                    amsim_vocab_loss_workspace_size(desc, which));
}
