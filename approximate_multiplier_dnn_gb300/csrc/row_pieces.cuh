// Which bytes a bulk copy takes of a row that does not start and end on 16
// bytes: the aligned pieces of 16 that hold it.  Between two rows of a tensor
// such a piece holds bytes of its neighbours or of the gap between them, which
// are not used.  The piece that holds the tensor's first element, or its last
// one, would reach outside the tensor: it is left out, and its elements of the
// row are copied one by one.
#pragma once

#include <cstdint>

namespace amsim {
namespace bn {

// From address `from` to offset `at` of the row's slot, both on 16 bytes.
struct Pieces {
    uintptr_t from;
    int at, bytes;
};

// The pieces of a row of `bytes` (at least 32) at address `a`; `first`, `last`:
// it is the tensor's first or last row.
__host__ __device__ __forceinline__ Pieces row_pieces(uintptr_t a, int bytes, bool first, bool last)
{
    const int head = (int)(a & 15), end = head + bytes;
    const int lo = first && head ? 16 : 0, hi = last ? end & ~15 : (end + 15) & ~15;
    return Pieces{a - head + lo, lo, hi - lo};
}

// Copies the row's elements that row_pieces leaves out to their places.
template <typename W>
__host__ __device__ __forceinline__ void copy_ends(uint8_t *slot, uintptr_t a, int bytes, bool first, bool last)
{
    const int head = (int)(a & 15), end = head + bytes;
    const W *row = reinterpret_cast<const W *>(a - head);
    W *to = reinterpret_cast<W *>(slot);
    if (first && head)
        for (int i = head / (int)sizeof(W); i < 16 / (int)sizeof(W); ++i) to[i] = row[i];
    if (last)
        for (int i = (end & ~15) / (int)sizeof(W); i < end / (int)sizeof(W); ++i) to[i] = row[i];
}

}  // namespace bn
}  // namespace amsim
