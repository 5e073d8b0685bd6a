"""GPU parity of the 8-bit checkpoints of activations and of the layer's backward
from them: codes, constants and values bit for bit, the backward bit for bit that
of the unpacked values and within the bounds of a float64 evaluation."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
import oracle
from expert_util import Grouped, state, within
from gpu_util import bf16, bits, dev, f32, need_gpu, say, torch
from oracle import act8 as oa
from oracle import experts as ox

pytestmark = pytest.mark.gpu


def _special(M, K, seed):
    """bf16 patterns whose blocks span the exponents, with zeros, subnormals,
    the largest values, infinities and NaNs among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K // 64, 64)).astype(np.float32)
    x *= (2.0 ** rng.integers(-20, 20, (M, K // 64, 1))).astype(np.float32)
    b = oracle.bf16_rne_bits(x).reshape(-1, 64)
    kinds = rng.integers(0, 12, len(b))
    b[kinds == 0] = 0x8000 * rng.integers(0, 2, (int((kinds == 0).sum()), 64))   # +0 and -0
    sub = kinds == 1
    b[sub] = rng.integers(0, 0x80, (int(sub.sum()), 64)) | (0x8000 * rng.integers(0, 2, 64))
    low = kinds == 2                                # constants from 2^-140 to 2^-90
    b[low] = rng.integers(0, 0x1400, (int(low.sum()), 64))
    big = kinds == 3
    b[big, 7] = 0x7F7F
    b[kinds == 4, 9] = 0xFF80
    b[kinds == 5, 63] = 0x7FC1
    b[kinds == 6, 1:] = 0                           # one value alone
    return b.astype(np.uint16).reshape(M, K)


def _packed(b):
    x8 = q.qlora_act8_pack(bf16(b))
    v = q.qlora_act8_unpack(x8)
    torch.cuda.synchronize()
    return x8, v


def _same(b, x8, v):
    codes, c = oa.pack(b)
    np.testing.assert_array_equal(x8.codes.cpu().numpy(), codes)
    got = x8.scales.cpu().numpy()
    nan = np.isnan(c)
    np.testing.assert_array_equal(np.isnan(got), nan)
    np.testing.assert_array_equal(got[~nan].view(np.uint32), c[~nan].view(np.uint32))
    want, gv = oa.value_bits(codes, c), bits(v)
    nv = np.repeat(nan, 64, axis=1)
    assert torch.isnan(v).cpu().numpy()[nv].all()
    np.testing.assert_array_equal(gv[~nv], want[~nv])


@pytest.mark.parametrize("M,K", [(1, 64), (3, 64), (1, 4096), (5, 192), (64, 1024), (33, 8192),
                                 (257, 448), (7, 17920)])
def test_pack_and_unpack(M, K):
    need_gpu()
    say(f"act8 {M} x {K}")
    b = _special(M, K, M + K)
    _same(b, *_packed(b))


@pytest.mark.parametrize("amax", [0x0001, 0x0042, 0x007F, 0x0080, 0x0FFF, 0x1280, 0x1301, 0x3F80,
                                  0x3FAB, 0x42FE, 0x7F00, 0x7F7F])
def test_every_value_below_a_largest(amax):
    """Every bf16 value up to each of several block maxima, both signs."""
    need_gpu()
    say(f"act8, every value up to {amax:#06x}")
    v = np.arange(amax + 1, dtype=np.uint16)
    v = np.concatenate([v, v | 0x8000])
    v = np.concatenate([v, np.zeros(-len(v) % 63, np.uint16)]).reshape(-1, 63)
    b = np.concatenate([v, np.full((len(v), 1), amax, np.uint16)], axis=1)
    _same(b, *_packed(b))


def test_codes_past_4g():
    """Offsets past 2^32 in codes and 2^33 bytes in values: the last rows."""
    need_gpu()
    M, K = (1 << 20) + 5, 4096
    say(f"act8 {M} x {K}")
    X = torch.zeros((M, K), dtype=torch.bfloat16, device=dev())
    b = _special(9, K, 1)
    X[-9:] = bf16(b)
    X[:9] = bf16(b)
    x8 = q.qlora_act8_pack(X)
    torch.cuda.synchronize()
    X.fill_(5.0)
    q.qlora_act8_unpack(x8, out=X)
    torch.cuda.synchronize()
    for rows in (slice(0, 9), slice(M - 9, M)):
        _same(b, q.Act8(x8.codes[rows], x8.scales[rows]), X[rows])
    assert not x8.codes[9:-9].any() and not X[9:-9].any()
    # dA of the layer from the last rows alone
    w = q.qlora_q4_quantize(torch.randn(8, K, device=dev()) * 0.02, "nf4", False)
    dY = torch.zeros((M, 8), dtype=torch.bfloat16, device=dev())
    dY[-9:] = 1.0
    A = torch.randn(K, 8, device=dev()).bfloat16()
    B = torch.randn(8, 8, device=dev()).bfloat16()
    T = torch.zeros((M, 8), device=dev())
    rng = np.random.default_rng(2)
    X[-9:] = bf16(oracle.bf16_rne_bits(rng.standard_normal((9, K)).astype(np.float32)))
    q.qlora_act8_pack(X, out=x8)
    _, dA, _ = q.qlora_linear_act8_bwd(dY, x8, w, A, B, 1.0, T=T, need_dx=False)
    V = q.qlora_act8_unpack(q.Act8(x8.codes[-9:].clone(), x8.scales[-9:].clone()))
    torch.cuda.synchronize()
    # a column that is NaN in one of the first rows (where dY is zero) is NaN; the
    # others are the last nine rows' products, whatever tiles those fall into
    bad = np.isnan(oracle.bf16_bits_to_f64(oa.value_bits(*oa.pack(b)))).any(axis=0)
    f = lambda t: t.double().cpu().numpy()
    args = (f(V), np.array([0, 9]), [f(q.qlora_q4_dequantize(w))], [f(A)], [f(B)], 1.0)
    _, ref, _ = ox.grouped_bwd(np.ones((9, 8)), *args)
    bound = ox.grouped_bounds(np.ones((9, 8)), *args)["dA"]
    assert torch.isnan(dA).cpu().numpy()[bad].all() and bad.any() and not bad.all()
    within("dA", dA[torch.from_numpy(~bad).to(dev())], ref[0][~bad], bound[0][~bad])


LINEAR = [
    # M, N, K, r, p, book, dq
    (1, 64, 64, 8, 0.0, "nf4", True), (5, 8, 64, 16, 0.3, "int4", False),
    (16, 256, 1024, 16, 0.0, "nf4", True), (17, 264, 320, 72, 0.0, "fp4", True),
    (130, 512, 960, 64, 0.1, "nf4", True), (300, 1024, 1024, 8, 0.0, "nf4", False),
    (700, 128, 2048, 256, 0.5, "nf4", True), (64, 256, 512, 0, 0.0, "nf4", True),
    (2048, 256, 128, 64, 0.05, "nf4", True),
]


@pytest.mark.parametrize("M,N,K,r,p,book,dq", LINEAR)
def test_linear_backward(M, N, K, r, p, book, dq):
    need_gpu()
    say(f"linear act8 bwd M={M} N={N} K={K} r={r} p={p} {book} dq={dq}")
    g = Grouped([M], N, K, r, p=p, book=book, dq=dq, seed=M + r)
    x8 = q.qlora_act8_pack(g.X)
    X = q.qlora_act8_unpack(x8)
    kw = dict(s=0.25, p=p, state=g.state)
    if r:
        kw.update(A=g.A[0], B=g.B[0])
    _, T = q.qlora_linear_dropout_fwd(X, g.w, **kw)
    want = q.qlora_linear_dropout_bwd(g.dY, X, g.w, T=T, **kw)
    got = q.qlora_linear_act8_bwd(g.dY, x8, g.w, T=T, **kw)
    again = q.qlora_linear_act8_bwd(g.dY, x8, g.w, T=None, **kw)
    wagain = q.qlora_linear_dropout_bwd(g.dY, X, g.w, T=None, **kw)
    no_dx = q.qlora_linear_act8_bwd(g.dY, x8, g.w, T=T, need_dx=False, **kw)
    torch.cuda.synchronize()
    assert no_dx[0] is None
    for a, b in zip(got[1:] + got[:1] + no_dx[1:], want[1:] + want[:1] + want[1:]):
        assert (a is None and b is None) or torch.equal(a, b)
    if r == 0:
        return
    assert torch.equal(again[0], wagain[0]) and torch.equal(again[1], wagain[1])
    if M > 16:
        assert torch.equal(again[2], wagain[2])
    # float64, on the values of the checkpoint
    f = oracle.bf16_bits_to_f64
    fX, fdY = f(bits(X)), f(bits(g.dY))
    D = g.D
    W = f(bits(q.qlora_q4_dequantize(g.w)))
    args = (fX, np.array([0, M]), [W], [f(bits(g.A[0]))], [f(bits(g.B[0]))], 0.25, D,
            1.0 if D is None else 65536 / (65536 - oracle.dropout.threshold(p)))
    dX, dA, dB = ox.grouped_bwd(fdY, *args)
    bound = ox.grouped_bounds(fdY, *args)
    for res in (got, again):
        within("dX", res[0], dX, bound["dX"])
        within("dA", res[1], dA[0], bound["dA"][0])
        within("dB", res[2], dB[0], bound["dB"][0])


GROUPED = [
    # tokens, topk, E, N, K, r, p, dropped share of the slots
    (1, 1, 1, 256, 64, 8, 0.0, 0.0), (3, 2, 4, 256, 64, 8, 0.0, 0.3),
    (40, 2, 8, 256, 320, 16, 0.0, 0.1), (9, 6, 7, 64, 1024, 72, 0.2, 0.0),
    (200, 3, 5, 512, 512, 64, 0.0, 0.2), (333, 5, 6, 128, 192, 8, 0.4, 0.0),
    (600, 1, 3, 256, 256, 16, 0.0, 0.5), (500, 4, 16, 64, 128, 0, 0.0, 0.0),
    (2000, 2, 2, 64, 256, 32, 0.1, 0.0), (50, 64, 70, 8, 64, 8, 0.0, 0.1),
]


@pytest.mark.parametrize("tokens,topk,E,N,K,r,p,lost", GROUPED)
def test_grouped_backward(tokens, topk, E, N, K, r, p, lost):
    """From the tokens' rows through the plan's order, and from the rows in expert
    order: bit for bit the bf16 call on the unpacked rows."""
    need_gpu()
    say(f"grouped act8 bwd tokens={tokens} topk={topk} E={E} N={N} K={K} r={r} p={p}")
    rng = np.random.default_rng(tokens + E)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(tokens)]).astype(np.int32)
    ids[rng.random(ids.shape) < lost] = -1
    t = torch.from_numpy(ids).to(dev())
    offsets, order, inverse = q.qlora_expert_plan(t, E)
    M = tokens * topk
    gen = torch.Generator(device=dev()).manual_seed(tokens)
    rand = lambda *s: torch.randn(s, generator=gen, device=dev())
    w = q.qlora_q4_quantize(rand(E * N, K) * 0.02, "nf4", False)
    x8 = q.qlora_act8_pack(rand(tokens, K).bfloat16())
    full = lambda: torch.full((M, K), 7.0, dtype=torch.bfloat16, device=dev())
    Xs = q.qlora_expert_gather(q.qlora_act8_unpack(x8), inverse, out=full())
    dY = rand(M, N).bfloat16()
    kw = dict(s=0.5, p=p, state=state())
    if r:
        kw.update(A=rand(E, K, r).bfloat16(), B=rand(E, r, N).bfloat16())
    _, T = q.qlora_grouped_fwd(Xs, offsets, w, E, **kw)
    for Tk in (T, None):
        want = q.qlora_grouped_bwd(dY, Xs, offsets, w, E, T=Tk, dX=full(), **kw)
        got = q.qlora_grouped_act8_bwd(dY, x8, offsets, w, E, order=order, topk=topk, T=Tk,
                                       dX=full(), **kw)
        rows = q.qlora_grouped_act8_bwd(dY, q.qlora_act8_pack(Xs), offsets, w, E, T=Tk, dX=full(),
                                        **kw)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert (a is None and b is None) or torch.equal(a, b)
        # (codes of values that are a checkpoint's already need not give them again)
        assert torch.equal(rows[0], want[0]) and (r == 0 or torch.equal(rows[2], want[2]) or Tk is None)
    if r and M <= 2000:   # float64
        f = oracle.bf16_bits_to_f64
        off = offsets.cpu().numpy()
        fX, fdY = f(bits(Xs)), f(bits(dY))
        W = f(bits(q.qlora_q4_dequantize(w))).reshape(E, N, K)
        D = oracle.dropout.keep((M, K), p, *_seed()) if p else None
        c = 65536 / (65536 - oracle.dropout.threshold(p))
        args = (fX, off, list(W), list(f(bits(kw["A"]))), list(f(bits(kw["B"]))), 0.5, D, c)
        dX, dA, dB = ox.grouped_bwd(fdY, *args)
        bound = ox.grouped_bounds(fdY, *args)
        end = int(off[-1])
        within("dX", got[0][:end], dX[:end], bound["dX"][:end])
        within("dA", got[1], dA, bound["dA"])
        within("dB", got[2], dB, bound["dB"])
        assert (got[0][end:] == 7).all()


def _seed():
    from expert_util import OFFSET, SEED
    return SEED, OFFSET


def test_orders_that_leave_the_checkpoint():
    """Slots whose token is not in the checkpoint are rows of zeros, and nothing
    outside it is read (NaN lies around it)."""
    need_gpu()
    say("wrong orders")
    tokens, topk, N, K, r = 6, 3, 64, 128, 8
    rng = np.random.default_rng(0)
    order = np.array([0, 17, 18, -1, -2 ** 31, 2 ** 31 - 1, 5, 19, 1000], np.int32)
    M = len(order)
    buf = torch.full((tokens + 8, K), 77, dtype=torch.int8, device=dev())
    sc = torch.full((tokens + 8, K // 64), float("nan"), device=dev())
    X = bf16(oracle.bf16_rne_bits(rng.standard_normal((tokens, K)).astype(np.float32)))
    x8 = q.qlora_act8_pack(X, out=q.Act8(buf[4:4 + tokens], sc[4:4 + tokens].clone()))
    sc[4:4 + tokens] = x8.scales
    sc16 = torch.full((16 + tokens * 2 + 16,), float("nan"), device=dev())
    sc16[16:16 + tokens * 2] = x8.scales.reshape(-1)
    x8 = q.Act8(buf[4:4 + tokens], sc16[16:16 + tokens * 2].view(tokens, 2))
    w = q.qlora_q4_quantize(torch.randn(N, K, device=dev()) * 0.02, "nf4", False)
    A = torch.randn(1, K, r, device=dev()).bfloat16()
    B = torch.randn(1, r, N, device=dev()).bfloat16()
    dY = torch.randn(M, N, device=dev()).bfloat16()
    off = torch.tensor([0, M], dtype=torch.int32, device=dev())
    tok = np.where((order >= 0) & (order // topk < tokens), order // topk, -1)
    Xs = torch.zeros((M, K), dtype=torch.bfloat16, device=dev())
    V = q.qlora_act8_unpack(x8)
    for i, k in enumerate(tok):
        if k >= 0:
            Xs[i] = V[k]
    for T in (None, torch.randn(M, r, device=dev())):
        want = q.qlora_grouped_bwd(dY, Xs, off, w, 1, A, B, T=T)
        got = q.qlora_grouped_act8_bwd(dY, x8, off, w, 1, A, B, order=torch.from_numpy(order).to(dev()),
                                       topk=topk, T=T)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_non_finite_blocks_reach_the_gradient():
    """A block with an infinity makes its 64 rows of dA NaN, and no others; where
    dropout takes such values out they leave nothing."""
    need_gpu()
    say("NaN blocks")
    M, N, K, r = 40, 64, 256, 8
    X = torch.randn(M, K, device=dev()).bfloat16()
    X[3, 70] = float("inf")
    x8 = q.qlora_act8_pack(X)
    w = q.qlora_q4_quantize(torch.randn(N, K, device=dev()) * 0.02, "nf4", False)
    A, B = torch.randn(K, r, device=dev()).bfloat16(), torch.randn(r, N, device=dev()).bfloat16()
    dY, T = torch.randn(M, N, device=dev()).bfloat16(), torch.randn(M, r, device=dev())
    dX, dA, dB = q.qlora_linear_act8_bwd(dY, x8, w, A, B, T=T)
    torch.cuda.synchronize()
    assert torch.isnan(dA[64:128]).all() and torch.isfinite(dA[:64]).all()
    assert torch.isfinite(dA[128:]).all() and torch.isfinite(dX).all() and torch.isfinite(dB).all()
    keep = torch.from_numpy(oracle.dropout.keep((M, K), 0.5, *_seed())).to(dev())
    _, dA, _ = q.qlora_linear_act8_bwd(dY, x8, w, A, B, p=0.5, state=state(), T=T)
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(dA).all(dim=1)[64:128], keep[3, 64:128])


def test_streams_graph_and_views():
    """On a stream of its own, in a graph whose buffers change between replays, and
    into slices of larger buffers."""
    need_gpu()
    say("act8 in a graph")
    M, N, K, r = 100, 128, 320, 16
    X = torch.randn(M, K, device=dev()).bfloat16()
    w = q.qlora_q4_quantize(torch.randn(N, K, device=dev()) * 0.02, "nf4", False)
    A, B = torch.randn(K, r, device=dev()).bfloat16(), torch.randn(r, N, device=dev()).bfloat16()
    dY = torch.randn(M, N, device=dev()).bfloat16()

    def step():
        x8 = q.qlora_act8_pack(X)
        return (*x8, q.qlora_act8_unpack(x8),
                *q.qlora_linear_act8_bwd(dY, x8, w, A, B, 0.5))
    first = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        X.copy_(torch.randn(M, K, device=dev()) * (i + 1))
        dY.copy_(torch.randn(M, N, device=dev()))
        graph.replay()
        a = [t.clone() for t in got]
        b = step()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    big = torch.full((M + 4, K), 7.0, dtype=torch.bfloat16, device=dev())
    q.qlora_act8_unpack(q.qlora_act8_pack(X), out=big[2:2 + M])
    torch.cuda.synchronize()
    assert (big[:2] == 7).all() and (big[2 + M:] == 7).all() and torch.equal(big[2:2 + M], b[2])
    # rows of a checkpoint, whose constants then start at any four bytes
    part = q.Act8(b[0][3:50], b[1][3:50])
    v = q.qlora_act8_unpack(part)
    gs = q.qlora_linear_act8_bwd(dY[3:50], part, w, A, B, 0.5)
    ws = q.qlora_linear_act8_bwd(dY[3:50].clone(), q.Act8(part.codes.clone(), part.scales.clone()), w,
                                 A, B, 0.5)
    torch.cuda.synchronize()
    assert torch.equal(v, b[2][3:50]) and all(torch.equal(s, t) for s, t in zip(gs, ws))
    empty = q.qlora_act8_pack(X[:0])
    assert q.qlora_act8_unpack(empty).shape == (0, K)
