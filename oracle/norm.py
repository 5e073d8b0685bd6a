"""The root-mean-square norm in front of a layer, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

    h = bf16(x + residual),  rstd = (mean_k h^2 + eps)^-1/2,  y = h rstd g
    n = h rstd,  c = mean_k(dy g n),  dx = dres + rstd (dy g - n c),
    dg = sum over rows of dy n

The bounds are those of an evaluation in fp32 with sums in any order and one
rounding of each output: a sum of n terms is off by at most n U times the sum
of their magnitudes, and every other operation by half a step.
"""
import numpy as np

from .nf4 import bf16_bits_to_f64, bf16_rne_bits

U = 2.0 ** -24         # half a step of fp32
HALF_BF16 = 2.0 ** -8  # half a step of bf16


def stream(x, residual=None):
    """h of bf16-valued float64 arrays: the sum rounded to bf16 once."""
    if residual is None:
        return x
    # (a sum of two bf16 values fits float32 or rounds there without harm: 24
    # bits are more than twice 8 and two)
    return bf16_bits_to_f64(bf16_rne_bits((x + residual).astype(np.float32)))


def fwd(h, g, eps):
    rstd = 1 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * g, rstd


def fwd_bounds(h, g, eps):
    """Of y (rounded to bf16) and rstd."""
    y, rstd = fwd(h, g, eps)
    # the mean: K terms, all positive, a division and the addition of eps; the
    # root halves its error; root and quotient round once each
    rel = (h.shape[1] + 3) * U / 2 + 2 * U
    return np.abs(y) * (HALF_BF16 + 1.01 * (rel + 2 * U)) + 1e-40, rstd * rel * 1.01


def bwd(dy, h, rstd, g, dres=None):
    n = h * rstd[:, None]
    d = dy * g
    c = (d * n).mean(axis=1, keepdims=True)
    dx = rstd[:, None] * (d - n * c) + (0 if dres is None else dres)
    return dx, (dy * n).sum(axis=0)


def bwd_bounds(dy, h, rstd, g, dres=None, half_dg=U):
    """Of dx (rounded to bf16) and dg (rounded by half_dg); rstd is an input."""
    dx, dg = bwd(dy, h, rstd, g, dres)
    M, K = h.shape
    n, d = np.abs(h * rstd[:, None]), np.abs(dy * g)
    mag = (d * n).mean(axis=1, keepdims=True)
    ec = (K + 4) * U * mag          # the sum, its factors d and n, the division
    inner = 3 * U * (d + n * mag) + n * ec
    b = rstd[:, None] * (inner + U * (d + n * mag)) + U * np.abs(dx)
    return (HALF_BF16 * np.abs(dx) + 1.01 * b + 1e-40,
            half_dg * np.abs(dg) + 1.01 * (M + 2) * U * (np.abs(dy) * n).sum(axis=0) + 1e-40)
