"""The grouped layer at the edges its kernels switch bodies on, and the calls a
program may make of it: group sizes one off every tile height, one kernel after
the other by token count, rank, rows and constants; NaN in one expert's rows;
tensors past 2^32 elements; several streams, captured graphs and a shared
workspace; padded batches and repeated choices through the exchange."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import OFFSET, SEED, Grouped, within
from gpu_util import bits, dev, need_gpu, say, torch
from oracle import bf16_bits_to_f64, codebooks as cb
from oracle import dropout as od
from oracle import experts as ox

pytestmark = pytest.mark.gpu

EDGES = [
    # sizes, N, K, r, keywords
    # up to 16 tokens: waves split K, 32 weight rows a workgroup
    ([16], 40, 64, 256, dict(dq=False)),
    ([0, 16, 0], 256, 1024 + 64, 248, {}),
    ([1] * 16, 64, 256, 8, dict(p=0.4)),
    ([0] * 69 + [3], 64, 256, 32, dict(book="fp4")),
    ([1, 0, 0, 1], 8, 64 * 130, 40, dict(dq=False, behind=14)),   # no more rows than the bound
    ([7, 2], 1032, 448, 0, dict(dq=False, book="int4")),
    ([4, 5, 0, 3, 2, 1], 264, 64 * 9, 24, dict(dq=False, p=0.2)),   # around four rows
    ([4], 64, 64 * 35, 8, dict(dq=False, before=1, behind=2)),
    ([3, 4, 4, 4], 128, 64 * 34, 16, {}),
    # 32 tokens a tile
    ([17], 128, 128, 16, {}),
    ([16, 17, 32, 33, 1, 15, 31, 34], 264, 192, 24, dict(dq=False)),
    ([24] * 40, 4096, 64, 8, {}),                         # 256 weight rows a workgroup
    # the same, constants in windows of 2048 columns: split inside and between them
    ([17, 3], 256, 64 * 67, 8, {}),
    ([16, 17, 0, 9], 256, 64 * 130, 16, dict(p=0.1)),
    ([20, 25], 128, 128 * 40, 8, dict(book="fp4")),
    ([20] * 200, 128, 64 * 34, 8, {}),                    # not split
    # 64 tokens a tile
    ([64, 65, 16, 17, 33, 32, 1, 48], 264, 192, 16, dict(dq=False, p=0.1)),
    ([31, 33] * 32, 2048, 128, 8, dict(p=0.1)),           # 256 weight rows a workgroup
    # 192 tokens a tile (forward), 256 (dX), with the narrower bodies of both
    ([191, 192, 193], 264, 128, 16, dict(dq=False)),
    ([64, 65, 128, 129, 63, 127], 128, 128, 72, {}),
    ([383, 385, 2, 449], 128, 320, 16, dict(dq=False, p=0.2)),
    ([255, 256, 257, 320, 321, 384, 513], 256, 64, 16, {}),
    ([60] * 70, 512, 192, 8, dict(p=0.1)),                # 256 weight rows, more than 64 experts
    ([90, 41], 128, 128 * 33, 16, {}),                    # reductions split unevenly
]


@pytest.mark.parametrize("sizes,N,K,r,kw", EDGES)
def test_edges(sizes, N, K, r, kw):
    need_gpu()
    say(f"grouped edges sizes={sizes if len(sizes) < 9 else len(sizes)} N={N} K={K} r={r} {kw}")
    Grouped(sizes, N, K, r, seed=len(sizes) + N + K + r, **kw).check()


MANY = [
    # many rows and columns: dX in tiles of 256 columns x 192 tokens
    ([300, 200, 64, 129, 65], 256, 64 * 161, 16, dict(before=3, behind=5)),
    ([193, 1, 0, 400, 128], 72, 10240, 72, dict(dq=False)),
    ([100] * 4, 8, 64 * 260, 8, dict(dq=False, book="int4")),
    ([150] * 3, 200, 64 * 257, 0, dict(dq=False)),
    ([260] * 3, 128, 16384, 256, dict(book="fp4")),
    ([1, 700, 0, 63], 192, 256 * 64, 40, dict(x_kind="shifted")),
    ([300, 200, 64, 129, 65], 256, 64 * 161, 16, dict(p=0.2)),
    ([600], 8, 16384, 8, dict(dq=False, p=0.1)),        # one expert: rounds decide
    ([700], 8, 11008, 8, dict(dq=False)),
    ([380, 1], 8, 32768, 8, dict(dq=False)),
]


@pytest.mark.parametrize("sizes,N,K,r,kw", MANY)
def test_many_rows_and_columns(sizes, N, K, r, kw):
    need_gpu()
    say(f"grouped many sizes={sizes} N={N} K={K} r={r} {kw}")
    Grouped(sizes, N, K, r, seed=len(sizes) + N + K + r, **kw).check()


def test_many_rows_with_a_poisoned_expert():
    """NaN constants, activations and gradients of one expert leave the others'
    dX as it was."""
    need_gpu()
    say("poisoned expert, many rows")
    g = Grouped([200, 150, 130, 90], 8, 64 * 260, 8, dq=False, seed=3)
    _, T, dX, dA, dB = g.check()
    own = slice(int(g.off[1]), int(g.off[2]))
    n = g.N * g.K // 64
    g.w.absmax_scale[n:2 * n] = float("nan")
    g.dY[own] = float("nan")
    g.A[1] = float("inf")
    dX2, dA2, dB2 = g.bwd(T)
    torch.cuda.synchronize()
    assert torch.equal(dX[:own.start], dX2[:own.start])
    assert torch.equal(dX[own.stop:], dX2[own.stop:]) and torch.isnan(dX2[own]).all()


@pytest.mark.parametrize("sizes", [[3, 5, 2], [20, 11, 30], [70, 100, 60]])
def test_nan_and_infinity_stay_with_their_expert(sizes):
    """NaN in one expert's activations, infinity in its gradients and NaN in its
    adapters: the other experts' results do not change by a bit."""
    need_gpu()
    say(f"poisoned expert, sizes={sizes}")
    g = Grouped(sizes, 256, 1024, 16, p=0.2, seed=3)
    Y, T, dX, dA, dB = g.check()
    own = slice(int(g.off[1]), int(g.off[2]))
    g.X[own] = float("nan")
    g.dY[own] = float("inf")
    g.A[1], g.B[1] = float("nan"), float("nan")
    Y2, T2 = g.fwd()
    dX2, dA2, dB2 = g.bwd(None)
    torch.cuda.synchronize()
    rest = torch.ones(g.M, dtype=torch.bool, device=dev())
    rest[own] = False
    for a, b in ((Y, Y2), (T, T2), (dX, dX2)):
        assert torch.equal(a[rest], b[rest]) and not torch.isfinite(b[own]).any()
    for a, b in ((dA, dA2), (dB, dB2)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_tensors_past_32_bits():
    """X and dX of more than 2^32 elements (8 GiB each), the last expert's rows
    behind the limit: its results, and the neighbour's last rows, against the
    oracle on those rows alone."""
    need_gpu()
    N, K, r, s, p, tail = 8, 8192, 8, 0.25, 0.25, 40
    M = 2 ** 32 // K + 300
    say(f"grouped M={M} K={K}")
    g = Grouped([1, 1], N, K, r, s=s, p=p, dq=False, seed=9)   # weights and adapters of two experts
    gen = torch.Generator(device=dev())
    gen.manual_seed(5)
    X = torch.empty((M, K), dtype=torch.bfloat16, device=dev())
    for i in range(0, M, 1 << 16):
        n = min(1 << 16, M - i)
        X[i:i + n] = torch.randn((n, K), generator=gen, device=dev(), dtype=torch.float32).bfloat16()
    dY = torch.randn((M, N), generator=gen, device=dev()).bfloat16()
    off = torch.tensor([0, M - tail, M], dtype=torch.int32, device=dev())
    kw = dict(A=g.A, B=g.B, s=s, p=p, state=g.state)
    Y, T = q.qlora_grouped_fwd(X, off, g.w, 2, **kw)
    dX, dA, dB = q.qlora_grouped_bwd(dY, X, off, g.w, 2, T=T, **kw)
    torch.cuda.synchronize()
    f = bf16_bits_to_f64
    W = f(cb.dequantize_q4(g.w.codes.cpu().numpy(), None, g.w.absmax_scale.cpu().numpy(), 2 * N, K,
                           "nf4", False)).reshape(2, N, K)
    for e, rows in ((1, slice(M - tail, M)), (0, slice(M - tail - 9, M - tail))):
        n = rows.stop - rows.start
        D = od.halves(n * K, SEED, OFFSET, rows.start * K).reshape(n, K) >= od.threshold(p)
        args = (f(bits(X[rows])), [0, n], [W[e]], [f(bits(g.A[e]))], [f(bits(g.B[e]))], s, D,
                od.scale(p))
        y, t = ox.grouped_fwd(*args)
        fdY = f(bits(dY[rows]))
        dx, da, db = ox.grouped_bwd(fdY, *args)
        b = ox.grouped_bounds(fdY, *args)
        within("Y", Y[rows], y, b["Y"])
        within("T", T[rows], t, b["T"])
        within("dX", dX[rows], dx, b["dX"])
        if e == 1:
            within("dA", dA[1], da[0], b["dA"][0])
            within("dB", dB[1], db[0], b["dB"][0])


def test_calls_in_flight_on_several_streams():
    """Forward and backward of three layers on three streams at once, the
    library's scratch memory being each call's own."""
    need_gpu()
    say("three streams")
    layers = [Grouped(sz, 256, 1024, 16, p=0.1, seed=i)
              for i, sz in enumerate(([3, 9], [40, 0, 30], [150, 100]))]
    want = [g.check() for g in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in layers]
    for _ in range(6):
        for i, (g, st) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(st):
                Y, T = g.fwd()
                got[i].append((Y, T, *g.bwd(T)))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for run in runs:
            for a, b in zip(w, run):
                assert torch.equal(a, b)


def test_two_graphs_share_a_workspace():
    """Nothing in a workspace outlives its call: two graphs captured on one,
    replayed in turn with eager calls between them."""
    need_gpu()
    say("two graphs, one workspace")
    layers = [Grouped([40, 0, 30], 256, 1024, 16, p=0.25, seed=1),
              Grouped([5, 1, 6], 256, 2048, 24, p=0.1, seed=2)]
    L = q.lib()
    nb = max(f(g.M, g.E, g.N, g.K, g.r) for g in layers
             for f in (L.qlora_grouped_fwd_workspace_bytes, L.qlora_grouped_bwd_workspace_bytes))
    ws = torch.empty(nb, dtype=torch.uint8, device=dev())
    def step(g):
        Y, T = g.fwd(workspace=ws)
        return (Y, T) + g.bwd(T, workspace=ws)
    want = [step(g) for g in layers]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for g in layers:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(g))
    for i in (0, 1, 1, 0, 1, 0):
        for t in outs[i]:
            t.fill_(3.0)
        graphs[i].replay()
        step(layers[1 - i])
        torch.cuda.synchronize()
        for a, b in zip(want[i], outs[i]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("sizes", [[2, 3], [20, 15], [40, 90]])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_constants_at_any_address(sizes, shift):
    """The 8-bit constants may start at any byte."""
    need_gpu()
    say(f"constants {shift} bytes off, sizes={sizes}")
    g = Grouped(sizes, 256, 64 * 35, 16, seed=6)
    want = g.check()
    buf = torch.full((g.w.absmax_q.numel() + 8,), 0xFF, dtype=torch.uint8, device=dev())
    moved = buf[shift:shift + g.w.absmax_q.numel()]
    moved.copy_(g.w.absmax_q)
    g.w = g.w._replace(absmax_q=moved)
    Y, T = g.fwd()
    out = (Y, T) + g.bwd(T)
    torch.cuda.synchronize()
    for a, b in zip(want, out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [8, 100])
def test_padded_batch_and_repeated_choices(tokens):
    """Tokens without an expert (padding) and tokens that choose one expert
    twice, through the whole layer, with every buffer full of NaN beforehand:
    padded tokens come out as zeros and get zero gradients, repeated choices as
    two rows."""
    need_gpu()
    say(f"padded batch of {tokens}")
    E, N, K, topk = 4, 256, 128, 2
    g = Grouped([1] * E, N, K, 16, seed=4)
    rng = np.random.default_rng(tokens)
    ids = rng.integers(0, E, (tokens, topk)).astype(np.int32)
    ids[1::4] = -1                           # padded
    ids[2::4, 1] = ids[2::4, 0]              # the same expert twice
    X = torch.from_numpy(rng.standard_normal((tokens, K))).bfloat16().to(dev())
    X[1::4] = float("nan")
    dOut = torch.from_numpy(rng.standard_normal((tokens, N))).bfloat16().to(dev())
    dOut[1::4] = float("nan")
    wts = torch.full((tokens, topk), 0.5, device=dev())
    wts[1::4] = float("nan")
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev())
    n = tokens * topk
    off, order, inv = q.qlora_expert_plan(torch.from_numpy(ids).to(dev()), E)
    Xs = q.qlora_expert_gather(X, inv, out=nan(n, K))
    Y, T = q.qlora_grouped_fwd(Xs, off, g.w, E, g.A, g.B, g.s, Y=nan(n, N))
    out = q.qlora_expert_combine(Y, inv, wts)
    dY, dw = q.qlora_expert_combine_bwd(dOut, Y, inv, wts, dY=nan(n, N))
    dXs, dA, dB = q.qlora_grouped_bwd(dY, Xs, off, g.w, E, g.A, g.B, g.s, T=T, dX=nan(n, K))
    dX = q.qlora_expert_combine(dXs, inv)
    torch.cuda.synchronize()
    for t in (out, dw, dX):
        assert not t[1::4].any() and torch.isfinite(t).all()
    assert torch.isfinite(dA).all() and torch.isfinite(dB).all()
    # 0.5 y + 0.5 y is y: the token's own row of its expert, bit for bit
    two = inv[2::4]
    assert torch.equal(Y[two[:, 0].long()], Y[two[:, 1].long()])
    assert torch.equal(out[2::4], Y[two[:, 0].long()])
    assert torch.equal(dw[2::4, 0], dw[2::4, 1])


@pytest.mark.parametrize("rows", [12, 600])
def test_the_most_experts(rows):
    """1024 experts, most of them without a row."""
    need_gpu()
    say(f"1024 experts, {rows} rows")
    rng = np.random.default_rng(rows)
    sizes = [0] * 1024
    for e in rng.integers(0, 1024, rows):
        sizes[e] += 1
    Grouped(sizes, 8, 128, 8, dq=False, seed=rows, behind=3).check()


@pytest.mark.parametrize("sizes", [[3, 2], [50, 40]])
def test_adapter_gradients_alone(sizes):
    """need_dx = False computes the same dA and dB; without adapters nothing is
    left to do."""
    need_gpu()
    say(f"no dX, sizes={sizes}")
    g = Grouped(sizes, 256, 256, 16, p=0.1, seed=2)
    Y, T, dX, dA, dB = g.check()
    none, dA2, dB2 = q.qlora_grouped_bwd(g.dY, g.X, g.offsets, g.w, g.E, T=T, need_dx=False,
                                         **g.kw())
    torch.cuda.synchronize()
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)
    assert q.qlora_grouped_bwd(g.dY, g.X, g.offsets, g.w, g.E, need_dx=False) == (None, None, None)


def test_probabilities_at_the_ends():
    """p below half a 65536th keeps everything; p next to 1 drops all but one
    16-bit value of 65536, whose elements are scaled by 65536."""
    need_gpu()
    say("p next to 0 and 1")
    from expert_util import state
    x = torch.ones(1 << 20, dtype=torch.bfloat16, device=dev())
    assert torch.equal(q.qlora_dropout(x, 1e-6, state()), x)
    y = q.qlora_dropout(x, 0.9999999, state())
    keep = od.halves(x.numel(), SEED, OFFSET) == 65535
    np.testing.assert_array_equal(y.float().cpu().numpy(), 65536.0 * keep)


def test_layer_with_dropout_in_a_graph():
    """Forward and backward of one layer, captured: every replay draws the mask of
    its state and equals the eager calls on it."""
    need_gpu()
    say("layer with dropout in a graph")
    from expert_util import state
    for M in (7, 90):
        g = Grouped([M], 256, 512, 16, p=0.3, seed=M)
        st = g.state
        def step():
            Y, T = q.qlora_linear_dropout_fwd(g.X, g.w, g.A[0], g.B[0], g.s, g.p, st)
            return (Y, T) + q.qlora_linear_dropout_bwd(g.dY, g.X, g.w, g.A[0], g.B[0], g.s, g.p, st,
                                                       T=T)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
            st[1] += 1
        st.copy_(state(5, 100))
        seen = []
        for i in range(4):
            graph.replay()
            got = [t.clone() for t in out]
            st.copy_(state(5, 100 + i))
            want = step()
            st.copy_(state(5, 101 + i))
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            seen.append(got[1])
        assert not torch.equal(seen[0], seen[1])


def test_exchange_past_32_bits():
    """Token rows of more than 2^32 elements (8 GiB), there and back."""
    need_gpu()
    tokens, K = 2 ** 16 + 40, 2 ** 16
    say(f"exchange tokens={tokens} K={K}")
    X = torch.empty((tokens, K), dtype=torch.bfloat16, device=dev())
    X.copy_(torch.arange(tokens, device=dev()).remainder(251).to(torch.bfloat16)[:, None])
    X[:, 3] = torch.arange(tokens, device=dev()).remainder(127).to(torch.bfloat16)
    inv = torch.arange(tokens - 1, -1, -1, dtype=torch.int32, device=dev())[:, None]
    Xs = q.qlora_expert_gather(X, inv)
    for t in (0, 1, 39, tokens // 2, tokens - 41, tokens - 1):
        assert torch.equal(Xs[tokens - 1 - t], X[t])
    w = torch.full((tokens, 1), 2.0, device=dev())
    out = q.qlora_expert_combine(Xs, inv, w)
    dY, dw = q.qlora_expert_combine_bwd(X, Xs, inv, w)
    torch.cuda.synchronize()
    for t in (0, 1, 39, tokens // 2, tokens - 41, tokens - 1):
        assert torch.equal(out[t], 2 * X[t]) and torch.equal(dY[tokens - 1 - t], 2 * X[t])
        v = float(t % 251)
        want = (K - 1) * v * v + float(t % 127) ** 2
        # sums of K products of 16 significant bits in fp32
        assert abs(float(dw[t]) - want) <= K * 2.0 ** -24 * want
