// Random numbers of dropout: the counter-based generator Philox4x32 with ten
// rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011).  A quad of elements takes the four words of one counter,
// so any thread draws any element's number by itself, and the backward pass
// draws the forward pass's again.
#pragma once

#include <cmath>

#include "amsim_internal.h"

namespace amsim {

constexpr uint32_t kPhiloxA = 0xD2511F53u, kPhiloxB = 0xCD9E8D57u;      // multipliers
constexpr uint32_t kPhiloxStepA = 0x9E3779B9u, kPhiloxStepB = 0xBB67AE85u;  // of the key, a round
constexpr int kPhiloxRounds = 10;

// A dropout as kernels take it.  border 0: everything stays.  The rounds' keys
// come with it, so that they are operands of the rounds and take no instructions.
struct Drop {
    uint32_t border;
    float scale;
    uint64_t call;
    const int64_t *step;
    uint32_t key[2 * kPhiloxRounds];
};

// false: p is outside [0, 1), or so near 1 that its border is 2^32, or step is off its alignment.
inline bool make_drop(const amsim_dropout_desc &d, Drop *out)
{
    if (!(d.p >= 0.0 && d.p < 1.0)) return false;
    const double border = std::nearbyint(d.p * 4294967296.0);
    if (border > 4294967295.0 || (reinterpret_cast<uintptr_t>(d.step) & 7)) return false;
    out->border = (uint32_t)border;
    out->scale = (float)(1.0 / (1.0 - d.p));
    out->call = d.call;
    out->step = d.step;
    uint32_t a = (uint32_t)d.seed, b = (uint32_t)(d.seed >> 32);
    for (int r = 0; r < kPhiloxRounds; ++r, a += kPhiloxStepA, b += kPhiloxStepB) {
        out->key[2 * r] = a;
        out->key[2 * r + 1] = b;
    }
    return true;
}

// The call's number with the device's part; once per thread.
__device__ __forceinline__ uint64_t drop_call(const Drop &d)
{
    return d.call + (d.border && d.step ? (uint64_t)*d.step : 0);
}

struct Product {
    uint32_t hi, lo;
};
__device__ __forceinline__ Product product(uint32_t x, uint32_t m)
{
    const uint64_t v = (uint64_t)x * m;
    return Product{(uint32_t)(v >> 32), (uint32_t)v};
}

// What the quads whose number has one upper half share: the first round's second
// product, and the second round's first, which do not depend on the lower half.
struct QuadStream {
    uint32_t c1, c3, a_hi, a_lo;
};
__device__ __forceinline__ QuadStream quad_stream(uint32_t upper, uint64_t call, const Drop &d)
{
    const Product b = product((uint32_t)call, kPhiloxB), a = product(b.hi ^ upper ^ d.key[0], kPhiloxA);
    return QuadStream{b.lo ^ d.key[2], (uint32_t)(call >> 32) ^ d.key[1], a.hi ^ d.key[3], a.lo};
}
// The four words of a quad.
__device__ __forceinline__ uint4 quad_words(uint32_t lower, const QuadStream &s, const Drop &d)
{
    Product a = product(lower, kPhiloxA), b = product(a.hi ^ s.c3, kPhiloxB);
    uint32_t c0 = b.hi ^ s.c1, c1 = b.lo, c2 = s.a_hi ^ a.lo, c3 = s.a_lo;      // after two rounds
#pragma unroll
    for (int r = 2; r < kPhiloxRounds; ++r) {
        a = product(c0, kPhiloxA);
        b = product(c2, kPhiloxB);
        c0 = b.hi ^ c1 ^ d.key[2 * r];
        c1 = b.lo;
        c2 = a.hi ^ c3 ^ d.key[2 * r + 1];
        c3 = a.lo;
    }
    return make_uint4(c0, c1, c2, c3);
}

}  // namespace amsim
