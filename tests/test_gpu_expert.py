"""GPU parity of the exchange around the grouped layer (qlora_expert_*): the
plan's integers exactly, the rows bit for bit or within bounds counted from
their roundings."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import within
from gpu_util import bf16, bits, dev, need_gpu, say, torch
from oracle import bf16_bits_to_f64, bf16_rne_bits
from oracle import experts as ox

pytestmark = pytest.mark.gpu


def _np(t):
    return t.cpu().numpy().astype(np.int64)


PLANS = [
    # tokens, topk, E, how the ids are drawn
    (0, 2, 4, "even"), (1, 1, 1, "even"), (1, 2, 3, "even"), (8, 2, 8, "even"),
    (33, 3, 5, "lost"), (64, 1, 1, "even"), (512, 2, 64, "even"), (513, 2, 65, "lost"),
    (1024, 1, 1024, "even"), (1025, 1, 1000, "lost"), (2000, 4, 7, "one"), (4096, 8, 128, "skew"),
    (70001, 2, 33, "lost"), (300, 6, 6, "none"), (20000, 8, 256, "skew"),
]


@pytest.mark.parametrize("tokens,topk,E,how", PLANS)
def test_plan(tokens, topk, E, how):
    need_gpu()
    say(f"plan tokens={tokens} topk={topk} E={E} {how}")
    rng = np.random.default_rng(tokens + topk + E)
    ids = rng.integers(0, E, (tokens, topk))
    if how == "lost":      # ids outside 0..E-1, on both sides
        ids = rng.integers(-3, E + 3, (tokens, topk))
        ids.reshape(-1)[::17] = rng.choice([-2 ** 31, 2 ** 31 - 1, E], ids.reshape(-1)[::17].size)
    elif how == "one":
        ids[:] = E - 1
    elif how == "none":
        ids[:] = -1
    elif how == "skew":
        ids = np.minimum(rng.geometric(0.2, (tokens, topk)) - 1, E - 1)
    t = torch.from_numpy(ids.astype(np.int32)).to(dev())
    off, order, inv = q.qlora_expert_plan(t, E)
    torch.cuda.synchronize()
    o, s, i = ox.plan(ids, E)
    np.testing.assert_array_equal(_np(off), o)
    np.testing.assert_array_equal(_np(order), s)
    np.testing.assert_array_equal(_np(inv), i)


ROWS = [
    # tokens, topk, E, K
    (1, 1, 1, 8), (1, 2, 4, 64), (5, 3, 4, 72), (40, 2, 8, 2048), (9, 2, 3, 2056), (7, 4, 9, 8192),
    (33, 64, 70, 16), (300, 6, 16, 264),
]


@pytest.mark.parametrize("tokens,topk,E,K", ROWS)
def test_rows(tokens, topk, E, K):
    need_gpu()
    say(f"rows tokens={tokens} topk={topk} E={E} K={K}")
    rng = np.random.default_rng(tokens + K)
    ids = rng.integers(-1, E, (tokens, topk)).astype(np.int32)
    _, _, inv = ox.plan(ids, E)
    kept, n = int((inv >= 0).sum()), tokens * topk
    draw = lambda *s: bf16_rne_bits(rng.standard_normal(s).astype(np.float32))
    Xb, Yb, gb = draw(tokens, K), draw(n, K), draw(tokens, K)
    w = (rng.random((tokens, topk)) - 0.3).astype(np.float32)
    Yb[kept:] = 0x7FC0                       # rows no slot has
    w[inv < 0] = np.nan                      # weights of slots without a row
    X, Y, g, ti = bf16(Xb), bf16(Yb), bf16(gb), torch.from_numpy(inv.astype(np.int32)).to(dev())
    tw = torch.from_numpy(w).to(dev())
    full = lambda: torch.full((n, K), 7.0, dtype=torch.bfloat16, device=dev())

    Xs = q.qlora_expert_gather(X, ti, out=full())
    out = q.qlora_expert_combine(Y, ti, tw)
    ones = q.qlora_expert_combine(Y, ti)
    dY, dw = q.qlora_expert_combine_bwd(g, Y, ti, tw, dY=full())
    torch.cuda.synchronize()
    want = np.full((n, K), 0x40E0, np.uint16)          # 7.0
    for t in range(tokens):
        for j in range(topk):
            if inv[t, j] >= 0:
                want[inv[t, j]] = Xb[t]
    np.testing.assert_array_equal(bits(Xs), want)

    Yf, wf, gf = bf16_bits_to_f64(Yb), np.where(inv < 0, 0, w).astype(np.float64), bf16_bits_to_f64(gb)
    # topk fused multiply-adds of half a step each, one rounding to bf16
    for name, got, ww in (("combine", out, wf), ("combine, weights 1", ones, np.ones_like(wf))):
        ref, mag = ox.combine(Yf, inv, ww)
        within(name, got, ref, 2.0 ** -8 * np.abs(ref) + 1.01 * topk * 2.0 ** -24 * mag)
    dYr, dwr, mag = ox.combine_bwd(gf, Yf, inv, wf)
    # one product in fp32, one rounding to bf16
    within("dY", dY[:kept], dYr[:kept], (2.0 ** -8 + 2.0 ** -23) * np.abs(dYr[:kept]))
    assert (dY[kept:] == 7).all()
    within("dw", dw, dwr, 1.01 * (K + 16) * 2.0 ** -24 * mag)


def test_rows_refuse_to_leave_the_buffers():
    """Rows named outside [0, n) count as none."""
    need_gpu()
    say("wrong rows")
    inv = torch.tensor([[0, 4], [-7, 2 ** 31 - 1]], dtype=torch.int32, device=dev())
    X = torch.ones((2, 64), dtype=torch.bfloat16, device=dev())
    guard = torch.full((12, 64), 7.0, dtype=torch.bfloat16, device=dev())
    Xs = q.qlora_expert_gather(X, inv, out=guard[4:8])
    out = q.qlora_expert_combine(Xs, inv)
    dY, dw = q.qlora_expert_combine_bwd(X, Xs, inv, torch.ones((2, 2), device=dev()),
                                        dY=torch.zeros_like(Xs))
    torch.cuda.synchronize()
    assert (guard[:4] == 7).all() and (guard[5:] == 7).all() and (guard[4] == 1).all()
    assert (out[0] == 1).all() and (out[1] == 0).all()
    assert dw.cpu().tolist() == [[64.0, 0.0], [0.0, 0.0]] and (dY[1:] == 0).all()


def test_repeats_are_bit_equal_and_graphs_follow_their_buffers():
    need_gpu()
    say("exchange in a graph")
    rng = np.random.default_rng(1)
    tokens, topk, E, K = 900, 3, 12, 128
    ids = torch.zeros((tokens, topk), dtype=torch.int32, device=dev())
    X = torch.randn((tokens, K), device=dev()).bfloat16()
    w = torch.rand((tokens, topk), device=dev())
    def step():
        off, order, inv = q.qlora_expert_plan(ids, E)
        Xs = q.qlora_expert_gather(X, inv)
        out = q.qlora_expert_combine(Xs, inv, w)
        return (off, order, inv, Xs, out) + q.qlora_expert_combine_bwd(out, Xs, inv, w)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        ids.copy_(torch.from_numpy(rng.integers(0, E, (tokens, topk)).astype(np.int32)))
        graph.replay()
        a = [t.clone() for t in got]
        b = step()
        torch.cuda.synchronize()
        for u, v in zip(a, b):
            assert torch.equal(u, v)
