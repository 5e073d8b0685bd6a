"""Pins of the oracle of the norm, the 8-bit checkpoints and the router, against
something other than itself (CPU)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import act8, bf16_bits_to_f64, bf16_rne_bits, norm, router


def test_act8_against_exact_rationals():
    """Every constant, code and value against fractions: c is the float32 next to
    amax / 127, the code the integer next to the float32 quotient."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 192)).astype(np.float32)
    x[0, :64] *= 1e-39                       # constants below the normal range
    x[1, 64:128] = 0
    bits = bf16_rne_bits(x)
    codes, c = act8.pack(bits)
    v = bf16_bits_to_f64(bits)
    for m in range(3):
        for b in range(3):
            blk = [Fraction(t) for t in v[m, 64 * b:64 * b + 64]]
            ratio = max(map(abs, blk)) / 127
            near = np.float32(float(ratio))
            assert c[m, b] == near and all(
                abs(Fraction(float(near)) - ratio) <= abs(Fraction(float(o)) - ratio)
                for o in (np.nextafter(near, np.float32(9)), np.nextafter(near, np.float32(-9))))
            for i, t in enumerate(blk):
                k = int(codes[m, 64 * b + i])
                if c[m, b] == 0:
                    assert k == 0
                    continue
                quo = np.float32(float(t / Fraction(float(c[m, b]))))
                assert abs(Fraction(float(quo)) - k) <= Fraction(1, 2)
                if abs(Fraction(float(quo)) - k) == Fraction(1, 2):
                    assert k % 2 == 0
    got = bf16_bits_to_f64(act8.value_bits(codes, c))
    # half a step of the block, and the value's rounding to bf16
    amax = np.abs(v).reshape(3, 3, 64).max(2, keepdims=True)
    err = np.abs(got - v).reshape(3, 3, 64)
    bound = amax / 254 * (1 + 2.0 ** -8) + 2.0 ** -8 * amax
    assert (err[1:] <= bound[1:]).all() and (err[0, 1:] <= bound[0, 1:]).all()


def test_act8_non_finite_blocks():
    x = np.ones((2, 128), np.float32)
    x[0, 5], x[1, 70] = np.inf, np.nan
    codes, c = act8.pack(bf16_rne_bits(x))
    assert np.isnan(c[0, 0]) and np.isnan(c[1, 1]) and not codes[0, :64].any()
    assert c[0, 1] == c[1, 0] == np.float32(1 / 127) and (codes[0, 64:] == 127).all()
    v = bf16_bits_to_f64(act8.value_bits(codes, c))
    assert np.isnan(v[0, :64]).all() and (v[0, 64:] == 1).all()


def test_norm_against_torch_and_differences():
    rng = np.random.default_rng(1)
    h, g, dy = rng.standard_normal((4, 24)), rng.standard_normal(24), rng.standard_normal((4, 24))
    dres = rng.standard_normal((4, 24))
    eps = 1e-3
    y, rstd = norm.fwd(h, g, eps)
    want = torch.nn.functional.rms_norm(torch.from_numpy(h), (24,), torch.from_numpy(g), eps)
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-13)
    dx, dg = norm.bwd(dy, h, rstd, g, dres)
    loss = lambda h, g: (norm.fwd(h, g, eps)[0] * dy).sum() + (h * dres).sum()
    d = 1e-6
    for i, k in [(0, 0), (1, 7), (3, 23)]:
        e = np.zeros_like(h)
        e[i, k] = d
        assert abs((loss(h + e, g) - loss(h - e, g)) / (2 * d) - dx[i, k]) < 1e-7
    for k in (0, 11):
        e = np.zeros_like(g)
        e[k] = d
        assert abs((loss(h, g + e) - loss(h, g - e)) / (2 * d) - dg[k]) < 1e-7


def test_norm_stream_rounds_once():
    rng = np.random.default_rng(2)
    a = bf16_bits_to_f64(bf16_rne_bits((rng.standard_normal(4000) * 10.0 ** rng.uniform(
        -4, 4, 4000)).astype(np.float32)))
    b = a[::-1].copy()
    got = norm.stream(a, b)
    # nearest among the neighbours, by exact float64 sums
    s, bits = a + b, bf16_rne_bits(got.astype(np.float32)).astype(np.int64)
    for step in (-1, 1):
        near = bf16_bits_to_f64((bits + step).astype(np.uint16))
        ok = np.isfinite(near) & (got != 0)
        assert (np.abs(got - s)[ok] <= np.abs(near - s)[ok]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_weights_and_gradients(score, renorm):
    """Weights against torch, gradients against differences."""
    rng = np.random.default_rng(3)
    X, dW = 2 * rng.standard_normal((5, 12)), rng.standard_normal((5, 3))
    X[2, 4:] = -np.inf
    X[3, 1:] = -np.inf                        # one expert for three slots
    ids, w = router.fwd(X, 3, score, renorm=renorm, scale=1.5)
    assert ids[3].tolist() == [0, -1, -1] and w[3, 1] == 0
    t = torch.from_numpy(X)
    p = torch.softmax(t, 1) if score == "softmax" else torch.sigmoid(t)
    for i in range(5):
        live = ids[i] >= 0
        q = p[i, ids[i][live]]
        q = 1.5 * (q / q.sum() if renorm else q)
        np.testing.assert_allclose(w[i][live], q.numpy(), rtol=1e-12)
        np.testing.assert_array_equal(ids[i][live], torch.topk(t[i], int(live.sum())).indices)
    got, mag = router.bwd(dW, X, ids, score, renorm, 1.5)
    assert (np.abs(got) <= mag + 1e-300).all()
    d = 1e-6
    for i in range(5):
        for e in range(12):
            if X[i, e] == -np.inf:
                assert got[i, e] == 0
                continue
            lo, hi = X[i].copy(), X[i].copy()
            lo[e] -= d
            hi[e] += d
            f = lambda x: router.weights(x, ids[i], score, renorm, 1.5) @ dW[i]
            assert abs((f(hi) - f(lo)) / (2 * d) - got[i, e]) < 1e-8


def test_router_choice():
    inf = np.inf
    x = np.array([1.0, 3.0, 3.0, -0.0, 0.0, -inf, 2.0, 2.0])
    c = router.choose
    assert c(x, 5) == [1, 2, 6, 7, 0]                        # ties to the lower index
    assert c(x, 8) == [1, 2, 6, 7, 0, 3, 4, -1]              # -0 ties with 0
    assert c(np.full(4, -inf), 2) == [-1, -1]
    bias = np.array([0, 0, 0, 0, 9.0, 9.0, 0, -inf])
    assert c(x, 3, bias=bias) == [4, 1, 2]                   # a masked expert stays masked
    assert 7 not in c(x, 7, bias=bias)
    # groups 0: {1, 3}, 1: {3, -0}, 2: {0, -inf}, 3: {2, 2}
    assert c(x, 2, groups=4, top_groups=1) == [1, 0]         # best member 3 in two groups
    assert c(x, 2, "sigmoid", groups=4, top_groups=1, group_top=2) == [6, 7]
    assert c(x, 4, groups=4, top_groups=2) == [1, 2, 0, 3]
    y = np.array([-inf, -inf, 1.0, -inf])
    assert c(y, 2, groups=2, top_groups=1, group_top=2) == [2, -1]
