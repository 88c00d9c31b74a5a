"""Dropout's random numbers in plain integers: Philox4x32-10 as published
(Salmon et al., SC 2011), one counter at a time or over an array of them."""
import numpy as np

M0, M1, W0, W1, LOW = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF


def words(counter, key):
    """The four output words of one counter (four words) under a key (two)."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * M0, c[2] * M1
        c = [(b >> 32) ^ c[1] ^ k[0], b & LOW, (a >> 32) ^ c[3] ^ k[1], a & LOW]
        k = [(k[0] + W0) & LOW, (k[1] + W1) & LOW]
    return c


def quad_words(quads, call, seed):
    """[n, 4] words of the quads' numbers (uint64 array)."""
    q = np.asarray(quads, dtype=np.uint64)
    low = np.uint64(LOW)
    call, seed = call % 2 ** 64, seed % 2 ** 64
    c0, c1 = q & low, q >> np.uint64(32)
    c2, c3 = np.full_like(q, call & LOW), np.full_like(q, call >> 32)
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        a, b = c0 * np.uint64(M0), c2 * np.uint64(M1)
        c0, c1, c2, c3 = ((b >> np.uint64(32)) ^ c1 ^ np.uint64(k0), b & low, (a >> np.uint64(32)) ^ c3 ^ np.uint64(k1),
                          a & low)
        k0, k1 = (k0 + W0) & LOW, (k1 + W1) & LOW
    return np.stack([c0, c1, c2, c3], -1)


def stays(rows, cols, p, call, seed):
    """Which elements of a matrix stay: every row takes ceil(cols / 4) quads."""
    quads = -(-cols // 4)
    w = quad_words(np.arange(rows * quads, dtype=np.uint64), call, seed)
    return (w >= round(p * 2 ** 32)).reshape(rows, 4 * quads)[:, :cols]
