"""Dropout from a counter-based generator, on the host in NumPy.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The mask: element i of a tensor (row-major index) belongs to piece i / 8; the
piece's 128 bits are Philox4x32 with 7 rounds (Salmon, Moraes, Dror, Shaw,
"Parallel random numbers: as easy as 1, 2, 3", SC11) of the counter (piece
low, piece high, offset low, offset high) under the key (seed low, seed high);
element i takes 16-bit half i % 8 and is kept when it is at least t.
"""
import numpy as np

ROUNDS = 7


def philox4x32(counter, key, rounds=ROUNDS):
    """counter: four uint64 arrays of 32-bit values, key: two ints."""
    m32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [np.asarray(v, np.uint64) for v in counter]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(rounds):
        lo = c[0] * np.uint64(0xD2511F53)
        hi = c[2] * np.uint64(0xCD9E8D57)
        c = [(hi >> sh) ^ c[1] ^ np.uint64(k0), hi & m32,
             (lo >> sh) ^ c[3] ^ np.uint64(k1), lo & m32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def threshold(p):
    """p is a float32 in the interface."""
    return int(min(65535, np.floor(np.float64(np.float32(p)) * 65536.0 + 0.5)))


def scale(p):
    return 65536.0 / (65536 - threshold(p))


def halves(n, seed, offset, first=0):
    """The 16-bit values of elements first .. first + n - 1."""
    p0, p1 = first // 8, (first + n + 7) // 8
    piece = np.arange(p0, p1, dtype=np.uint64)
    z = np.zeros_like(piece)
    words = philox4x32([piece & np.uint64(0xFFFFFFFF), piece >> np.uint64(32),
                        z + np.uint64(offset & 0xFFFFFFFF), z + np.uint64(offset >> 32)],
                       (seed & 0xFFFFFFFF, seed >> 32))
    h = np.stack([v for w in words for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], axis=1)
    return h.reshape(-1)[first - 8 * p0:first - 8 * p0 + n].astype(np.int64)


def keep(shape, p, seed, offset):
    """Boolean mask of a tensor of this shape."""
    return (halves(int(np.prod(shape)), seed, offset) >= threshold(p)).reshape(shape)
