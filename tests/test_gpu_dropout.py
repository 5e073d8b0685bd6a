"""GPU parity of dropout: the standalone call bit for bit against the oracle's
mask and roundings, the layer with adapter dropout within the bounds derived in
oracle/experts.py (one expert that has all rows)."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import OFFSET, SEED, Grouped, state, within
from gpu_util import bf16, bits, dev, need_gpu, say, torch
from oracle import bf16_bits_to_f64, bf16_rne_bits
from oracle import dropout as od

pytestmark = pytest.mark.gpu


def _ref(xb, p):
    """bf16 bits of bf16_rne(fl32(x c)) where kept, 0 where dropped."""
    x = bf16_bits_to_f64(xb).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        y = bf16_rne_bits(x * np.float32(od.scale(p)))
    return np.where(od.keep(xb.shape, p, SEED, OFFSET), y, np.uint16(0))


@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 1000, 8191, 8192, 8193, 100003])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.99999])
def test_dropout_bit_exact(n, p):
    need_gpu()
    say(f"dropout n={n} p={p}")
    rng = np.random.default_rng(n)
    xb = bf16_rne_bits(rng.standard_normal(n).astype(np.float32))
    x = bf16(xb)
    y = q.qlora_dropout(x, p, state())
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(y), _ref(xb, p))
    # in place, and nothing behind the tensor
    buf = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device=dev())
    buf[:n] = x
    q.qlora_dropout(buf[:n], p, state(), out=buf[:n])
    torch.cuda.synchronize()
    assert torch.equal(buf[:n], y) and (buf[n:] == 7).all()


def test_dropped_infinities_and_nans_are_zero():
    need_gpu()
    say("dropout of inf and nan")
    n, p = 4096, 0.5
    xb = np.resize(np.array([0x7F80, 0xFF80, 0x7FC0, 0x7F7F, 0x0001, 0x8000], np.uint16), n)
    y = bits(q.qlora_dropout(bf16(xb), p, state()))
    keep = od.keep((n,), p, SEED, OFFSET)
    assert (y[~keep] == 0).all()
    f = bf16_bits_to_f64(y)
    assert np.isnan(f[keep & (xb == 0x7FC0)]).all()
    assert np.isposinf(f[keep & (xb == 0x7F80)]).all() and np.isposinf(f[keep & (xb == 0x7F7F)]).all()
    assert (f[keep & (xb == 0x0001)] > 0).all()


def test_p_zero_needs_no_state_and_empty_tensors_pass():
    need_gpu()
    say("dropout p=0, n=0")
    x = torch.randn(33, device=dev()).bfloat16()
    assert torch.equal(q.qlora_dropout(x, 0.0, None), x)
    assert q.qlora_dropout(x[:0], 0.5, state()).numel() == 0


def test_positions_past_32_bits():
    """Element 2^32 + i of a tensor takes its mask from piece 2^29 + i / 8 (an
    8 GiB tensor; its tail against the oracle)."""
    need_gpu()
    n = 2 ** 32 + 1003
    say(f"dropout n={n}")
    x = torch.ones(n, dtype=torch.bfloat16, device=dev())
    q.qlora_dropout(x, 0.5, state(), out=x)
    torch.cuda.synchronize()
    for first in (2 ** 32 - 50, 2 ** 31 + 5):
        m = min(1003, n - first)
        keep = od.halves(m, SEED, OFFSET, first) >= od.threshold(0.5)
        np.testing.assert_array_equal(x[first:first + m].cpu().float().numpy(), 2.0 * keep)


LAYERS = [
    # M, N, K, r, p, book, dq
    (1, 64, 64, 8, 0.1, "nf4", True),
    (16, 1024, 1024, 16, 0.1, "nf4", True),
    (5, 200, 320, 40, 0.5, "nf4", False),
    (17, 264, 64 * 33, 64, 0.05, "nf4", True),
    (300, 520, 448, 72, 0.3, "nf4", True),
    (600, 136, 1024, 256, 0.1, "fp4", True),
    (129, 136, 64, 8, 0.2, "int4", False),
    (260, 512, 256, 64, 0.99999, "nf4", True),
    (40, 520, 64, 0, 0.5, "nf4", True),
]


@pytest.mark.parametrize("M,N,K,r,p,book,dq", LAYERS)
def test_layer_with_dropout(M, N, K, r, p, book, dq):
    need_gpu()
    say(f"layer with dropout M={M} N={N} K={K} r={r} p={p} {book} dq={dq}")
    g = Grouped([M], N, K, r, p=p, book=book, dq=dq, seed=M + N + K + r)
    ab = (g.A[0], g.B[0]) if r else (None, None)
    Y, T = q.qlora_linear_dropout_fwd(g.X, g.w, *ab, g.s, p, g.state)
    outs = [q.qlora_linear_dropout_bwd(g.dY, g.X, g.w, *ab, g.s, p, g.state, T=t)
            for t in (T, None)]
    torch.cuda.synchronize()
    within("Y", Y, g.Y, g.bound["Y"])
    if r:
        within("T", T, g.T, g.bound["T"])
    for dX, dA, dB in outs:
        within("dX", dX, g.dX, g.bound["dX"])
        if r:
            within("dA", dA, g.dA[0], g.bound["dA"][0])
            within("dB", dB, g.dB[0], g.bound["dB"][0])


@pytest.mark.parametrize("M", [3, 16, 70])
def test_p_zero_is_the_plain_layer_bit_for_bit(M):
    need_gpu()
    say(f"layer with p=0, M={M}")
    g = Grouped([M], 256, 512, 16, seed=M)
    w = q.NF4Weight(*g.w[:5])
    Y, T = q.qlora_linear_dropout_fwd(g.X, w, g.A[0], g.B[0], g.s)
    Y1, T1 = q.qlora_linear_fwd(g.X, w, g.A[0], g.B[0], g.s)
    a = q.qlora_linear_dropout_bwd(g.dY, g.X, w, g.A[0], g.B[0], g.s, 0.0, g.state, T=T)
    b = q.qlora_linear_bwd(g.dY, g.X, w, g.A[0], g.B[0], g.s, T=T1)
    torch.cuda.synchronize()
    for u, v in zip((Y, T, *a), (Y1, T1, *b)):
        assert torch.equal(u, v)


def test_nan_in_a_dropped_activation_does_not_reach_the_adapter():
    """A NaN of X whose element is dropped reaches Y through the base product
    only: T and the adapters' gradients stay finite."""
    need_gpu()
    say("NaN at a dropped place")
    M, K, p = 40, 128, 0.5
    g = Grouped([M], 128, K, 16, p=p, seed=1)
    m, k = np.argwhere(~g.D)[5]
    g.X[m, k] = float("nan")
    Y, T = q.qlora_linear_dropout_fwd(g.X, g.w, g.A[0], g.B[0], g.s, p, g.state)
    _, dA, dB = q.qlora_linear_dropout_bwd(g.dY, g.X, g.w, g.A[0], g.B[0], g.s, p, g.state)
    torch.cuda.synchronize()
    within("T", T, g.T, g.bound["T"])
    within("dA", dA, g.dA[0], g.bound["dA"][0])
    within("dB", dB, g.dB[0], g.bound["dB"][0])
    assert torch.isnan(Y[m]).all() and not torch.isnan(Y[m - 1]).any()


def test_gradients_by_differences():
    """dA and dX of the layer with dropout against differences of its own
    forward along random directions.  Y is rounded to bf16, 2^-8 of its
    magnitude at worst and independently per element, so the difference of two
    sums over n outputs is off by at most about 2^-8 sqrt(n) of the outputs'
    size; a step h as large as the input itself keeps the difference (linear in
    h) far above that."""
    need_gpu()
    say("layer with dropout, differences")
    M, N, K, r, p = 64, 256, 256, 16, 0.25
    g = Grouped([M], N, K, r, p=p, seed=4)
    A, B = g.A[0], g.B[0]
    dX, dA, dB = q.qlora_linear_dropout_bwd(g.dY, g.X, g.w, A, B, g.s, p, g.state)
    def loss(X, A, B):
        Y, _ = q.qlora_linear_dropout_fwd(X, g.w, A, B, g.s, p, g.state)
        return Y.double(), float((Y.double() * g.dY.double()).sum())
    gen = torch.Generator(device=dev())
    gen.manual_seed(1)
    for which, grad, base in (("X", dX, g.X), ("A", dA, A), ("B", dB, B)):
        # a direction along the gradient's signs, so the change is not lost
        v = (grad.float().sign() * base.float().abs().mean()).bfloat16()
        lo, hi = (base.float() - v.float()).bfloat16(), (base.float() + v.float()).bfloat16()
        step = hi.double() - lo.double()
        args = lambda t: {"X": (t, A, B), "A": (g.X, t, B), "B": (g.X, A, t)}[which]
        Yh, lh = loss(*args(hi))
        Yl, ll = loss(*args(lo))
        want = float((grad.double() * step).sum())
        # worst case: every output's rounding with its dY, and dX/dA/dB's own
        tol = 2.0 ** -8 * float(((Yh.abs() + Yl.abs()) * g.dY.double().abs()).pow(2).sum().sqrt() * 6
                                + (grad.double() * step).abs().sum())
        say(f"  {which}: {lh - ll:.4f} against {want:.4f}, tolerance {tol:.4f}")
        assert abs((lh - ll) - want) <= tol and abs(want) > 4 * tol


def test_graph_draws_another_mask_per_replay():
    need_gpu()
    say("dropout in a graph")
    x = torch.randn(5000, device=dev()).bfloat16()
    st = state()
    y = torch.empty_like(x)
    q.qlora_dropout(x, 0.5, st, out=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qlora_dropout(x, 0.5, st, out=y)
        st[1] += 1
    seen = []
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = od.keep((5000,), 0.5, SEED, (OFFSET + i) % 2 ** 64)
        np.testing.assert_array_equal((y != 0).cpu().numpy() | (x == 0).cpu().numpy(),
                                      want | (x == 0).cpu().numpy())
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])
