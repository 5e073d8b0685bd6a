"""The 8-bit checkpoint of activations, on the host in NumPy.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Blocks of 64 values along a row: c = fl32(amax / 127), code = rint(fl32(x / c))
(ties to even, 0 where c = 0), value = bf16(fl32(code c)); a block with a NaN
or an infinity has c = NaN and codes 0.  fl32 of a quotient or product of two
fp32 values is taken from float64: 53 bits are more than twice 24 and two, so
the second rounding changes nothing.
"""
import numpy as np

from .nf4 import bf16_bits_to_f64, bf16_rne_bits

BLOCK = 64


def pack(bits):
    """codes int8 [M, K] and constants float32 [M, K / 64] of bf16 bit patterns."""
    M, K = bits.shape
    x = bf16_bits_to_f64(bits).reshape(M, K // BLOCK, BLOCK)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        amax = np.abs(x).max(axis=2)
        good = np.isfinite(x).all(axis=2)
        c = np.where(good, amax / 127.0, np.nan).astype(np.float32)
        cd = c.astype(np.float64)[:, :, None]
        q = np.where(cd > 0, x / np.where(cd > 0, cd, 1), 0.0).astype(np.float32)
    codes = np.where(good[:, :, None], np.rint(np.where(good[:, :, None], q, 0)), 0)
    assert np.abs(codes).max(initial=0) <= 127
    return codes.astype(np.int8).reshape(M, K), c


def value_bits(codes, c):
    """bf16 bit patterns of the values."""
    M, K = codes.shape
    with np.errstate(over="ignore", invalid="ignore"):
        v = (codes.reshape(M, -1, BLOCK).astype(np.float64)
             * c.astype(np.float64)[:, :, None]).astype(np.float32)
    return bf16_rne_bits(v).reshape(M, K)
