"""The reference generator of the dropout tests against its published known answers."""
import numpy as np
import pytest

from philox_reference import quad_words, words


@pytest.mark.parametrize("counter,key,out", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])])
def test_known_answers(counter, key, out):
    assert words(counter, key) == out


def test_arrays_agree():
    quads, call, seed = [0, 1, 2 ** 32 + 5, 2 ** 40], 2 ** 33 + 7, 2 ** 50 + 3
    got = quad_words(quads, call, seed)
    for q, row in zip(quads, got):
        one = words([q % 2 ** 32, q >> 32, call % 2 ** 32, call >> 32], [seed % 2 ** 32, seed >> 32])
        assert np.array_equal(row, np.array(one, dtype=np.uint64))
