// Random numbers of dropout: the counter-based generator Philox4x32 with ten
// rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011).  A quad of elements takes the four words of one counter,
// so any thread draws any element's number by itself, and the backward pass
// draws the forward pass's again.
#pragma once

#include <cmath>

#include "amsim_internal.h"

namespace amsim {

// A dropout as kernels take it.  border 0: everything stays.
struct Drop {
    uint32_t border;
    float scale;
    uint64_t seed, call;
    const int64_t *step;
};

// false: p is outside [0, 1), or so near 1 that its border is 2^32, or step is off its alignment.
inline bool make_drop(const amsim_dropout_desc &d, Drop *out)
{
    if (!(d.p >= 0.0 && d.p < 1.0)) return false;
    const double border = std::nearbyint(d.p * 4294967296.0);
    if (border > 4294967295.0 || (reinterpret_cast<uintptr_t>(d.step) & 7)) return false;
    *out = Drop{(uint32_t)border, (float)(1.0 / (1.0 - d.p)), d.seed, d.call, d.step};
    return true;
}

// The call's number with the device's part; once per thread.
__device__ __forceinline__ uint64_t drop_call(const Drop &d)
{
    return d.call + (d.border && d.step ? (uint64_t)*d.step : 0);
}

// The four words of a quad.
__device__ __forceinline__ uint4 philox(uint64_t quad, uint64_t call, uint64_t seed)
{
    uint32_t c0 = (uint32_t)quad, c1 = (uint32_t)(quad >> 32), c2 = (uint32_t)call, c3 = (uint32_t)(call >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Dropout of a quad's four values.
__device__ __forceinline__ void drop_quad(float (&v)[4], uint64_t quad, const Drop &d, uint64_t call)
{
    const uint4 w = philox(quad, call, d.seed);
    v[0] = w.x >= d.border ? v[0] * d.scale : 0.0f;
    v[1] = w.y >= d.border ? v[1] * d.scale : 0.0f;
    v[2] = w.z >= d.border ? v[2] * d.scale : 0.0f;
    v[3] = w.w >= d.border ? v[3] * d.scale : 0.0f;
}

}  // namespace amsim
