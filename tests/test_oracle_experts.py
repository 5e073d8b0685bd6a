"""Pins of the oracle of dropout, the layer grouped by expert and the exchange
around it, against something other than itself (CPU)."""
import numpy as np
import pytest
import torch

from oracle import dropout as od
from oracle import experts as ox


def test_philox_known_answers():
    """The generator's published test vectors for a zero counter and key."""
    z = [np.zeros(1, np.uint64)] * 4
    got = [int(v[0]) for v in od.philox4x32(z, (0, 0), 10)]
    assert got == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    got = [int(v[0]) for v in od.philox4x32(z, (0, 0), 7)]
    assert got == [0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48]


def test_mask_depends_on_position_seed_and_offset_only():
    a = od.halves(1000, 5, 9)
    np.testing.assert_array_equal(a[13:700], od.halves(687, 5, 9, first=13))
    # the counter's third and fourth words are the offset, the key the seed
    assert not np.array_equal(a, od.halves(1000, 5, 10))
    assert not np.array_equal(a, od.halves(1000, 5 + 2 ** 32, 9))
    assert not np.array_equal(a, od.halves(1000, 5, 9 + 2 ** 32))
    # a piece beyond 2^32 reaches the counter's second word
    far = 8 * (2 ** 32 + 3)
    z = np.zeros(1, np.uint64)
    w = od.philox4x32([z + np.uint64(3), z + np.uint64(1), z + np.uint64(9), z], (5, 0))
    assert od.halves(1, 5, 9, first=far)[0] == int(w[0][0]) & 0xFFFF


@pytest.mark.parametrize("p", [0.05, 0.3, 0.5])
def test_keep_rate_and_independence(p):
    """The share kept and the products of neighbours' masks are within five
    standard deviations of independent draws of the rounded probability."""
    n = 1 << 20
    k = od.keep((n,), p, 1234567, 42).astype(np.float64)
    q = 1 - od.threshold(p) / 65536
    assert abs(k.mean() - q) < 5 * np.sqrt(q * (1 - q) / n)
    for lag in (1, 2, 7, 8, 64):
        c = (k[:-lag] - q) * (k[lag:] - q)
        assert abs(c.mean()) < 5 * q * (1 - q) / np.sqrt(n - lag)


def test_threshold_edges():
    assert od.threshold(0.0) == 0 and od.scale(0.0) == 1.0
    assert od.threshold(0.5) == 32768 and od.scale(0.5) == 2.0
    assert od.threshold(np.nextafter(np.float32(1), np.float32(0))) == 65535
    assert od.threshold(2.0 ** -18) == 0


def _case(seed, sizes, N, K, r, p):
    rng = np.random.default_rng(seed)
    E, M = len(sizes), sum(sizes)
    X, dY = rng.standard_normal((M, K)), rng.standard_normal((M, N))
    Ws = [rng.standard_normal((N, K)) * 0.1 for _ in range(E)]
    As = [rng.standard_normal((K, r)) for _ in range(E)]
    Bs = [rng.standard_normal((r, N)) for _ in range(E)]
    off = np.concatenate([[0], np.cumsum(sizes)])
    D = od.keep((M, K), p, 3, 4) if p else None
    return X, dY, off, Ws, As, Bs, D, od.scale(p) if p else 1.0


@pytest.mark.parametrize("p", [0.0, 0.25])
def test_grouped_matches_autograd(p):
    """A loop over the rows, each through its own expert, in torch's float64
    autograd."""
    sizes, s = [3, 0, 1, 4], 0.5
    X, dY, off, Ws, As, Bs, D, c = _case(1, sizes, 6, 8, 2, p)
    t = lambda a: torch.tensor(np.asarray(a), dtype=torch.float64, requires_grad=True)
    tX, tA, tB = t(X), t(np.stack(As)), t(np.stack(Bs))
    owner = np.repeat(np.arange(len(sizes)), sizes)
    rows = []
    for m, e in enumerate(owner):
        x = tX[m]
        xd = x * torch.tensor(D[m] * c) if D is not None else x
        rows.append(torch.tensor(Ws[e]) @ x + s * ((xd @ tA[e]) @ tB[e]))
    Y = torch.stack(rows)
    (Y * torch.tensor(dY)).sum().backward()
    Yr, _ = ox.grouped_fwd(X, off, Ws, As, Bs, s, D, c)
    dX, dA, dB = ox.grouped_bwd(dY, X, off, Ws, As, Bs, s, D, c)
    for got, ref in ((Yr, Y.detach()), (dX, tX.grad), (dA, tA.grad), (dB, tB.grad)):
        np.testing.assert_allclose(got, ref.numpy(), rtol=1e-12, atol=1e-12)
    assert not dA[1].any() and not dB[1].any()


def test_grouped_gradients_by_differences():
    """The loss is linear in X and in each adapter factor alone, so central
    differences are exact up to rounding."""
    sizes, s, p = [2, 3], 0.5, 0.25
    X, dY, off, Ws, As, Bs, D, c = _case(2, sizes, 4, 8, 2, p)
    loss = lambda X, As, Bs: (ox.grouped_fwd(X, off, Ws, As, Bs, s, D, c)[0] * dY).sum()
    dX, dA, dB = ox.grouped_bwd(dY, X, off, Ws, As, Bs, s, D, c)
    rng = np.random.default_rng(0)
    v = rng.standard_normal(X.shape)
    assert (loss(X + v, As, Bs) - loss(X - v, As, Bs)) / 2 == pytest.approx((dX * v).sum())
    v = [rng.standard_normal(a.shape) for a in As]
    d = loss(X, [a + u for a, u in zip(As, v)], Bs) - loss(X, [a - u for a, u in zip(As, v)], Bs)
    assert d / 2 == pytest.approx(sum((g * u).sum() for g, u in zip(dA, v)))
    v = [rng.standard_normal(b.shape) for b in Bs]
    d = loss(X, As, [b + u for b, u in zip(Bs, v)]) - loss(X, As, [b - u for b, u in zip(Bs, v)])
    assert d / 2 == pytest.approx(sum((g * u).sum() for g, u in zip(dB, v)))


def test_one_expert_without_dropout_is_the_layer():
    from oracle import linear
    X, dY, off, Ws, As, Bs, _, _ = _case(3, [5], 6, 8, 2, 0.0)
    Y, T = ox.grouped_fwd(X, off, Ws, As, Bs, 0.5)
    Yr, Tr = linear.linear_fwd_f64(X, Ws[0], As[0], Bs[0], 0.5)
    np.testing.assert_allclose(Y, Yr, rtol=1e-13)
    np.testing.assert_allclose(T, Tr, rtol=1e-13)
    for g, r in zip(ox.grouped_bwd(dY, X, off, Ws, As, Bs, 0.5),
                    linear.linear_bwd_f64(dY, X, Ws[0], As[0], Bs[0], 0.5)):
        np.testing.assert_allclose(g.reshape(r.shape), r, rtol=1e-13, atol=1e-13)


def test_bounds_hold_for_a_float32_evaluation():
    """A float32 evaluation with bf16 outputs stays inside the stated bounds,
    and a planted mistake of two bf16 steps does not."""
    X, dY, off, Ws, As, Bs, D, c = _case(4, [7, 9], 16, 64, 8, 0.25)
    bf = lambda a: torch.tensor(np.asarray(a)).bfloat16().double().numpy()
    X, dY, Ws, As, Bs = bf(X), bf(dY), [bf(w) for w in Ws], [bf(a) for a in As], [bf(b) for b in Bs]
    bound = ox.grouped_bounds(dY, X, off, Ws, As, Bs, 0.5, D, c)
    ref = dict(zip(("Y", "T"), ox.grouped_fwd(X, off, Ws, As, Bs, 0.5, D, c)))
    ref.update(zip(("dX", "dA", "dB"), ox.grouped_bwd(dY, X, off, Ws, As, Bs, 0.5, D, c)))
    f = lambda a: np.asarray(a, np.float32)
    Y32, _ = ox.grouped_fwd(f(X), off, [f(w) for w in Ws], [f(a) for a in As], [f(b) for b in Bs],
                            np.float32(0.5), D, np.float32(c))
    assert (np.abs(bf(Y32) - ref["Y"]) <= bound["Y"]).all()
    assert (np.abs(ref["Y"] * (1 + 2.0 ** -6) - ref["Y"]) > bound["Y"]).mean() > 0.9


def test_plan_is_the_stable_sort():
    rng = np.random.default_rng(5)
    ids = rng.integers(-1, 8, (50, 3))       # -1 and 7 get no row
    off, order, inv = ox.plan(ids, 7)
    flat = ids.reshape(-1)
    good = (flat >= 0) & (flat < 7)
    key = np.where(good, flat, 7)
    ref = np.argsort(key, kind="stable")
    kept = int(good.sum())
    np.testing.assert_array_equal(order[:kept], ref[:kept])
    assert (order[kept:] == -1).all() and off[-1] == kept
    np.testing.assert_array_equal(np.diff(off), np.bincount(flat[good], minlength=7))
    np.testing.assert_array_equal(inv.reshape(-1)[order[:kept]], np.arange(kept))
    assert (inv.reshape(-1)[~good] == -1).all()


def test_combine_matches_autograd():
    rng = np.random.default_rng(6)
    ids = rng.integers(-1, 4, (9, 2))
    _, _, inv = ox.plan(ids, 4)
    Y, w, dOut = rng.standard_normal((18, 8)), rng.random((9, 2)), rng.standard_normal((9, 8))
    tY, tw = (torch.tensor(a, requires_grad=True) for a in (Y, w))
    out = torch.stack([sum((tw[t, j] * tY[inv[t, j]] for j in range(2) if inv[t, j] >= 0),
                           torch.zeros(8, dtype=torch.float64)) for t in range(9)])
    (out * torch.tensor(dOut)).sum().backward()
    np.testing.assert_allclose(ox.combine(Y, inv, w)[0], out.detach().numpy(), atol=1e-14)
    dY, dw, _ = ox.combine_bwd(dOut, Y, inv, w)
    np.testing.assert_allclose(dY, tY.grad.numpy(), atol=1e-14)
    np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-13)
