"""GPU parity of the layer grouped by expert (qlora_grouped_*) against the
float64 oracle, element by element within the bounds derived in
oracle/experts.py: groups that are empty, of one row, and around the tile
sizes; rows that belong to no group; every codebook and constant format; adapter
dropout; more experts than lanes of a wave; split reductions; the largest and
smallest ranks; graph replays, side streams and dirty workspaces."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import Grouped, state, within
from gpu_util import bf16, dev, need_gpu, say, torch

pytestmark = pytest.mark.gpu

CASES = [
    # sizes, N, K, r, keywords
    ([1], 256, 64, 8, {}),
    ([0, 1, 0], 256, 64, 8, {}),
    ([0, 0], 256, 64, 8, dict(behind=3)),
    ([2, 0, 1, 3], 128, 128, 16, dict(behind=5)),
    ([5, 4, 0, 7], 128, 128, 16, dict(before=3, behind=2, p=0.1)),
    ([15, 16, 17], 64, 256, 24, dict(p=0.3)),
    ([63, 64, 65, 0, 1], 64, 256, 40, {}),
    ([31, 32, 33], 8, 2048, 8, dict(p=0.5)),             # 8 rows an expert, reduction split
    ([16, 3], 256, 2048, 64, dict(p=0.05)),              # few tokens, reduction split
    ([255, 256, 257], 128, 128, 64, dict(p=0.1)),
    ([700], 264, 1024, 64, dict(dq=False, p=0.2)),       # one expert, ragged rows and K
    ([1, 511, 0, 130], 200, 320, 72, dict(dq=False, behind=9)),
    ([129, 300], 256, 448, 256, dict(p=0.1)),            # the largest rank, K % 128 == 64
    ([40, 8, 200], 512, 96 * 64, 8, {}),                 # wide K
    ([3, 1] * 40, 64, 256, 8, {}),                       # 80 experts
    ([0] * 70 + [9] + [0] * 60 + [2], 16, 1024, 16, dict(p=0.1)),
    ([130, 20], 256, 64, 0, dict(p=0.1)),                # base only: dropout has no effect
    ([20, 300], 128, 128, 16, dict(book="int4")),
    ([20, 300], 128, 128, 16, dict(book="fp4", dq=False, p=0.25)),
    ([33, 0, 14], 24, 192, 16, dict(book="int4", dq=False)),
    ([500, 400], 128, 128, 16, dict(x_kind="shifted", p=0.9)),
]


@pytest.mark.parametrize("sizes,N,K,r,kw", CASES)
def test_grouped_parity(sizes, N, K, r, kw):
    need_gpu()
    say(f"grouped sizes={sizes if len(sizes) < 9 else len(sizes)} N={N} K={K} r={r} {kw}")
    Grouped(sizes, N, K, r, seed=len(sizes) + N + K + r, **kw).check()


@pytest.mark.parametrize("M", [1, 3, 16, 17, 60, 200])
def test_one_expert_is_the_layer(M):
    """E = 1 over all rows against the plain layer's own calls (both within
    their bounds of the same reference)."""
    need_gpu()
    say(f"grouped E=1 against the layer, M={M}")
    g = Grouped([M], 512, 512, 16, seed=M)
    Y, T, dX, dA, dB = g.check()
    Y1, T1 = q.qlora_linear_fwd(g.X, q.NF4Weight(*g.w[:5]), g.A[0], g.B[0], g.s)
    dX1, dA1, dB1 = q.qlora_linear_bwd(g.dY, g.X, q.NF4Weight(*g.w[:5]), g.A[0], g.B[0], g.s, T=T1)
    torch.cuda.synchronize()
    within("Y of the layer", Y1, g.Y, g.bound["Y"])
    within("dX of the layer", dX1, g.dX, g.bound["dX"])
    within("dA of the layer", dA1, g.dA[0], g.bound["dA"][0])
    within("dB of the layer", dB1, g.dB[0], g.bound["dB"][0])


def test_no_rows_at_all():
    """M = 0: no output rows, zero adapter gradients."""
    need_gpu()
    say("grouped M=0")
    g = Grouped([0, 0, 0], 256, 64, 8, seed=1)
    g.check()
    dA, dB = (torch.full_like(t, 3.0) for t in (g.A, g.B))
    _, dA, dB = g.bwd(None, dA=dA, dB=dB)
    torch.cuda.synchronize()
    assert not dA.any() and not dB.any()


def test_adapter_gradients_of_idle_experts_are_zero():
    need_gpu()
    say("idle experts")
    g = Grouped([0, 90, 0], 256, 64, 8, seed=2)
    dA, dB = (torch.full_like(t, float("nan")) for t in (g.A, g.B))
    _, dA, dB = g.bwd(None, dA=dA, dB=dB)
    torch.cuda.synchronize()
    assert not dA[[0, 2]].any() and not dB[[0, 2]].any()
    within("dA", dA, g.dA, g.bound["dA"])


@pytest.mark.parametrize("off", [[0, 9, 4, 40], [-5, 10, 30, 99], [40, 40, 40, 40], [50, 60, 70, 80],
                                 [30, 20, 10, 0]])
def test_wrong_offsets_stay_inside_the_buffers(off):
    """Offsets that fall, are negative or lie behind the last row: guarded
    buffers around every output keep their values."""
    need_gpu()
    say(f"offsets {off}")
    g = Grouped([20, 10, 10], 256, 64, 8, seed=3)
    g.offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    guard = torch.full((3 * g.M, g.N), 7.0, dtype=torch.bfloat16, device=dev())
    Y, T = q.qlora_grouped_fwd(g.X, g.offsets, g.w, g.E, Y=guard[g.M:2 * g.M], **g.kw())
    dX, _, _ = g.bwd(None)
    torch.cuda.synchronize()
    assert (guard[:g.M] == 7).all() and (guard[2 * g.M:] == 7).all()
    clamped = [min(max(v, 0), g.M) for v in off]
    if clamped == sorted(clamped):     # the clamped groups are the groups
        assert (Y[:clamped[0]] == 7).all() and (Y[clamped[3]:] == 7).all()


def test_repeats_and_dirty_workspace_are_bit_equal():
    need_gpu()
    say("grouped determinism")
    for sizes, N, K in (([5, 0, 9], 256, 1024), ([300, 270, 1], 256, 256)):
        g = Grouped(sizes, N, K, 24, p=0.2, seed=5)
        Y, T, dX, dA, dB = g.check()
        nb = max(q.lib().qlora_grouped_fwd_workspace_bytes(g.M, g.E, N, K, 24),
                 q.lib().qlora_grouped_bwd_workspace_bytes(g.M, g.E, N, K, 24))
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=dev())
        Y2, T2 = g.fwd(workspace=ws)
        ws.fill_(0xFF)
        out = g.bwd(T, workspace=ws)
        torch.cuda.synchronize()
        for a, b in zip((Y, T, dX, dA, dB), (Y2, T2, *out)):
            assert torch.equal(a, b)


def test_graph_replays_follow_offsets_and_state():
    """A captured forward and backward, replayed with other offsets and another
    state in the same buffers, equals the eager calls on them."""
    need_gpu()
    say("grouped graph")
    g = Grouped([40, 0, 30], 256, 128, 16, p=0.25, seed=6)
    def step():
        Y, T = q.qlora_grouped_fwd(g.X, g.offsets, g.w, g.E, **g.kw())
        return (Y, T) + q.qlora_grouped_bwd(g.dY, g.X, g.offsets, g.w, g.E, T=T, **g.kw())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i, off in enumerate(([0, 40, 40, 70], [0, 1, 69, 70], [0, 0, 70, 70], [0, 70, 70, 70])):
        g.offsets.copy_(torch.tensor(off, dtype=torch.int32))
        g.state.copy_(state(11 + i, i))
        graph.replay()
        got = [t.clone() for t in out]
        ref = step()
        torch.cuda.synchronize()
        for name, a, b in zip(("Y", "T", "dX", "dA", "dB"), got, ref):
            assert torch.equal(a, b), (name, off)


def test_other_stream():
    need_gpu()
    say("grouped on another stream")
    g = Grouped([40, 3, 30], 256, 128, 16, seed=7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Y, T = g.fwd()
        dX, dA, dB = g.bwd(T)
    side.synchronize()
    g.check_rows("Y", Y, g.Y, g.bound["Y"])
    within("dA", dA, g.dA, g.bound["dA"])


def test_training_layer_of_experts():
    """The calls of a mixture-of-experts layer as they are used together: plan,
    gather, grouped forward, combine, and all their backwards, against float64
    autograd over the same definition."""
    need_gpu()
    say("plan, gather, grouped, combine and back")
    tokens, topk, E, N, K, r, s, p = 70, 2, 5, 256, 128, 16, 0.5, 0.2
    g = Grouped([tokens * topk] + [0] * (E - 1), N, K, r, s=s, p=p, seed=8)   # weights, adapters
    rng = np.random.default_rng(9)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(tokens)]).astype(np.int32)
    ids[3, 1] = -1                                        # a dropped slot
    X = torch.from_numpy(rng.standard_normal((tokens, K))).bfloat16().to(dev())
    wts = torch.from_numpy(rng.random((tokens, topk)).astype(np.float32)).to(dev())
    dOut = torch.from_numpy(rng.standard_normal((tokens, N))).bfloat16().to(dev())
    offsets, order, inv = q.qlora_expert_plan(torch.from_numpy(ids).to(dev()), E)
    Xs = q.qlora_expert_gather(X, inv)
    Y, T = q.qlora_grouped_fwd(Xs, offsets, g.w, E, g.A, g.B, s, p, g.state)
    out = q.qlora_expert_combine(Y, inv, wts)
    dY, dw = q.qlora_expert_combine_bwd(dOut, Y, inv, wts)
    dXs, dA, dB = q.qlora_grouped_bwd(dY, Xs, offsets, g.w, E, g.A, g.B, s, p, g.state, T=T)
    dX = q.qlora_expert_combine(dXs, inv)
    torch.cuda.synchronize()

    t64 = lambda t: t.double().cpu().requires_grad_()
    tX, tA, tB, tw = t64(X), t64(g.A), t64(g.B), t64(wts)
    W = q.qlora_q4_dequantize(g.w).double().cpu().reshape(E, N, K)
    rows = inv.cpu().numpy()
    from expert_util import OFFSET, SEED
    from oracle import dropout as od
    D = torch.from_numpy(od.keep((tokens * topk, K), p, SEED, OFFSET) * od.scale(p))
    acc = []
    for t in range(tokens):
        y = torch.zeros(N, dtype=torch.float64)
        for j in range(topk):
            if ids[t, j] >= 0:
                e = int(ids[t, j])
                xd = tX[t] * D[rows[t, j]]
                y = y + tw[t, j] * (W[e] @ tX[t] + s * ((xd @ tA[e]) @ tB[e]))
        acc.append(y)
    ref = torch.stack(acc)
    (ref * dOut.double().cpu()).sum().backward()
    # Y and dY are rounded to bf16 on the way, dXs and the outputs once more: a
    # few half steps (2^-8) of the magnitudes, which a relative Frobenius bound
    # of 3 half steps covers
    for name, a, b in (("out", out, ref.detach()), ("dX", dX, tX.grad), ("dA", dA, tA.grad),
                       ("dB", dB, tB.grad), ("dw", dw, tw.grad)):
        a = a.double().cpu()
        rel = float((a - b).norm() / b.norm())
        say(f"  {name}: relative error {rel:.2e}")
        assert rel <= 3 * 2.0 ** -8, name
