"""The pieces in which rows off 16 bytes are copied, compiled for the host: on
16 bytes, inside the tensor, and with the elements copied one by one the whole
row and nothing else of it."""
import os
import subprocess

import approximate_multiplier_dnn_gb300 as am

CSRC = os.path.join(os.path.dirname(os.path.abspath(am.__file__)), "csrc")

PROGRAM = r"""
#define __host__
#define __device__
#define __forceinline__ inline
#include <cstdio>
#include <cstring>
#include <vector>
#include "row_pieces.cuh"
using namespace amsim::bn;

static int bad(const char *what, int head, int bytes, long row)
{
    std::printf("%s: base + %d, rows of %d bytes, row %ld\n", what, head, bytes, row);
    return 1;
}

template <typename W>
static int check(int cols, int ld, int head)
{
    const int size = (int)sizeof(W), bytes = cols * size;
    const long rows = 4, span = ((rows - 1) * ld + cols) * size;
    // a tensor between guards, its base `head` bytes past a multiple of 16
    std::vector<uint8_t> mem(span + 128);
    uint8_t *base = mem.data() + (16 - (reinterpret_cast<uintptr_t>(mem.data()) & 15)) % 16 + 32 + head;
    for (long i = 0; i < span; ++i) base[i] = (uint8_t)(i * 7 + 1);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base), hi = lo + span;
    for (long row = 0; row < rows; ++row) {
        const uintptr_t a = lo + row * ld * size;
        const bool first = row == 0, last = row == rows - 1;
        const Pieces p = row_pieces(a, bytes, first, last);
        if (p.from % 16 || p.at % 16 || p.bytes % 16 || p.bytes <= 0) return bad("alignment", head, bytes, row);
        if (p.from < lo || p.from + p.bytes > hi) return bad("outside the tensor", head, bytes, row);
        const int slot_bytes = (bytes + 30 + 127) / 128 * 128;
        if (p.at + p.bytes > slot_bytes) return bad("outside the slot", head, bytes, row);
        alignas(16) uint8_t slot[4096];
        std::memset(slot, 0xEE, sizeof(slot));
        std::memcpy(slot + p.at, reinterpret_cast<const void *>(p.from), p.bytes);
        copy_ends<W>(slot, a, bytes, first, last);
        if (std::memcmp(slot + a % 16, reinterpret_cast<const void *>(a), bytes)) return bad("bytes", head, bytes, row);
        for (int i = slot_bytes; i < (int)sizeof(slot); ++i)
            if (slot[i] != 0xEE) return bad("behind the slot", head, bytes, row);
    }
    return 0;
}

int main()
{
    for (int cols = 389; cols < 389 + 24; ++cols)
        for (int gap = 0; gap < 9; ++gap)
            for (int off = 0; off < 8; ++off) {
                if (check<uint16_t>(cols, cols + gap, 2 * off)) return 1;
                if (off < 4 && check<uint32_t>(cols, cols + gap, 4 * off)) return 1;
            }
    return 0;
}
"""


def test_pieces_stay_inside_the_tensor(tmp_path):
    src, exe = tmp_path / "pieces.cpp", tmp_path / "pieces"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
