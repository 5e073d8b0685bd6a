"""GPU parity of the root-mean-square norm with the residual's addition and the
8-bit checkpoint of its output, and of its backward, against float64 within the
bounds of an fp32 evaluation."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import within
from gpu_util import bf16, bits, dev, need_gpu, say, torch
from oracle import act8 as oa
from oracle import bf16_bits_to_f64, bf16_rne_bits
from oracle import norm as on

pytestmark = pytest.mark.gpu

EPS = 1e-5
# every number of threads a row and pieces a thread, whole and ragged, one row and several
SIZES = [(1, 8), (5, 64), (4, 504), (9, 512), (3, 520), (7, 1024), (2, 1032), (6, 2048), (3, 2056),
         (5, 4096), (2, 4160), (17, 8192), (3, 8200), (2, 16384), (3, 16392), (2, 32768),
         (2, 32832), (2, 65536), (3, 65544), (2, 70016), (1, 1 << 18)]


def _draw(rng, *shape, std=1.0):
    return bf16_rne_bits((rng.standard_normal(shape) * std).astype(np.float32))


def _inputs(M, K, seed, g32):
    rng = np.random.default_rng(seed)
    x, r = _draw(rng, M, K), _draw(rng, M, K, std=3.0)
    x[:, ::97] = bf16_rne_bits((30 * rng.standard_normal(x[:, ::97].shape)).astype(np.float32))
    g = (1 + 0.2 * rng.standard_normal(K)).astype(np.float32)
    tg = torch.from_numpy(g).to(dev())
    if not g32:
        tg = tg.bfloat16()
    return rng, x, r, tg, tg.double().cpu().numpy()


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("res,g32", [(True, True), (False, False)])
def test_forward(M, K, res, g32):
    need_gpu()
    say(f"norm fwd {M} x {K} residual={res} g32={g32}")
    _, x, r, tg, g = _inputs(M, K, M + K, g32)
    f = bf16_bits_to_f64
    want = on.stream(f(x), f(r) if res else None)
    tx, tr = bf16(x), bf16(r) if res else None
    keep = K % 64 == 0
    out = q.qlora_rms_norm_fwd(tx, tg, tr, EPS, act8=keep)
    torch.cuda.synchronize()
    h, y, rstd = out[:3]
    np.testing.assert_array_equal(f(bits(h)), want)
    assert h is tx or res
    yr, rr = on.fwd(want, g, EPS)
    by, br = on.fwd_bounds(want, g, EPS)
    within("y", y, yr, by)
    within("rstd", rstd, rr, br)
    if keep:   # the checkpoint of y as it was rounded, bit for bit
        codes, c = oa.pack(bits(y))
        np.testing.assert_array_equal(out[3].codes.cpu().numpy(), codes)
        np.testing.assert_array_equal(out[3].scales.cpu().numpy(), c)
        plain = q.qlora_rms_norm_fwd(tx, tg, tr, EPS)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(plain, out))


@pytest.mark.parametrize("M,K", SIZES + [(0, 64), (0, 17000), (300, 64), (1000, 1024), (700, 3000),
                                         (4099, 520), (300, 8192), (140, 16384), (60, 40000),
                                         (40, 66000), (300, 17000), (1100, 512), (1500, 1024),
                                         (1030, 2400), (1100, 4104), (1025, 16384), (130, 65544)])
@pytest.mark.parametrize("res,g32", [(True, False), (False, True)])
def test_backward(M, K, res, g32):
    need_gpu()
    say(f"norm bwd {M} x {K} dres={res} g32={g32}")
    rng, x, r, tg, g = _inputs(M, K, M + K + 1, g32)
    f = bf16_bits_to_f64
    dy = _draw(rng, M, K)
    _, rstd = on.fwd(f(x), g, EPS) if M else (None, np.zeros(0))
    rstd = rstd.astype(np.float32)
    trstd = torch.from_numpy(rstd).to(dev())
    tdy, th, tr = bf16(dy), bf16(x), bf16(r) if res else None
    dx, dg = q.qlora_rms_norm_bwd(tdy, th, trstd, tg, dres=tr)
    dx2, none = q.qlora_rms_norm_bwd(tdy, th, trstd, tg, dres=tr, need_dg=False)
    torch.cuda.synchronize()
    assert none is None and torch.equal(dx, dx2) and dg.dtype == tg.dtype
    if M == 0:
        assert not dg.any()
        return
    args = (f(dy), f(x), rstd.astype(np.float64), g, f(r) if res else None)
    wx, wg = on.bwd(*args)
    bx, bg = on.bwd_bounds(*args, half_dg=on.U if g32 else on.HALF_BF16)
    within("dx", dx, wx, bx)
    within("dg", dg, wg, bg)
    again = q.qlora_rms_norm_bwd(tdy, th, trstd, tg, dres=tr)
    torch.cuda.synchronize()
    assert torch.equal(dx, again[0]) and torch.equal(dg, again[1])
    if res:   # in place of dres
        q.qlora_rms_norm_bwd(tdy, th, trstd, tg, dres=tr, dx=tr)
        torch.cuda.synchronize()
        assert torch.equal(tr, dx)


@pytest.mark.parametrize("K", [64, 2048, 8192, 66048])
def test_in_place_stream(K):
    """h in the place of x or of the residual."""
    need_gpu()
    say(f"norm in place K={K}")
    _, x, r, tg, _ = _inputs(6, K, K, True)
    want = q.qlora_rms_norm_fwd(bf16(x), tg, bf16(r), EPS, act8=True)
    for which in (0, 1):
        t = [bf16(x), bf16(r)]
        got = q.qlora_rms_norm_fwd(t[0], tg, t[1], EPS, act8=True, h=t[which])
        torch.cuda.synchronize()
        assert got[0] is t[which]
        assert all(torch.equal(a, b) for a, b in zip(got[:3] + got[3], want[:3] + want[3]))


def test_rows_do_not_meet():
    """NaN and infinity in one row reach that row alone (and dg); a row of zeros
    gives zeros."""
    need_gpu()
    say("norm, NaN rows")
    for K in (64, 1024, 4096):
        _, x, r, tg, _ = _inputs(12, K, K, True)
        x[3, 5], x[7, K - 1], x[9] = 0x7FC0, 0x7F80, 0
        h, y, rstd, y8 = q.qlora_rms_norm_fwd(bf16(x), tg, eps=EPS, act8=True)
        dx, _ = q.qlora_rms_norm_bwd(bf16(r), h, rstd, tg)
        v = q.qlora_act8_unpack(y8)
        torch.cuda.synchronize()
        bad = torch.zeros(12, dtype=torch.bool, device=dev())
        bad[3] = bad[7] = True
        assert torch.isnan(y[3]).all() and torch.isnan(v[3]).all() and torch.isnan(dx[bad]).any(1).all()
        assert rstd[7] == 0 and torch.isnan(y[7, K - 1]) and torch.isnan(v[7, -64:]).all()
        assert not y[9].any() and not v[9].any()
        for t in (y, v, dx):
            assert torch.isfinite(t[~bad]).all()


def test_largest_and_smallest_rows():
    """Values at the top of the range whose squares still sum, and subnormal ones,
    where eps alone stands under the root."""
    need_gpu()
    say("norm, extreme rows")
    K = 256
    x = np.empty((3, K), np.uint16)
    rng = np.random.default_rng(3)
    x[0] = bf16_rne_bits((1e18 * rng.standard_normal(K)).astype(np.float32))
    x[1] = bf16_rne_bits((1e-39 * rng.standard_normal(K)).astype(np.float32))
    x[2] = bf16_rne_bits((1e-12 * rng.standard_normal(K)).astype(np.float32))
    g = np.ones(K)
    h, y, rstd = q.qlora_rms_norm_fwd(bf16(x), torch.ones(K, device=dev()), eps=EPS)
    torch.cuda.synchronize()
    f = bf16_bits_to_f64(x)
    yr, rr = on.fwd(f, g, float(np.float32(EPS)))
    by, br = on.fwd_bounds(f, g, float(np.float32(EPS)))
    within("y", y, yr, by)
    within("rstd", rstd, rr, br)


def test_past_4g_elements():
    """Row offsets past 2^32: the first and last rows, forward and backward."""
    need_gpu()
    M, K = (1 << 19) + 3, 8192 + 64
    say(f"norm {M} x {K}")
    _, x, r, tg, g = _inputs(4, K, 5, True)
    X = torch.zeros((M, K), dtype=torch.bfloat16, device=dev())
    X[:4], X[-4:] = bf16(x), bf16(x)
    h, y, rstd, y8 = q.qlora_rms_norm_fwd(X, tg, eps=EPS, act8=True)
    want = q.qlora_rms_norm_fwd(bf16(x), tg, eps=EPS, act8=True)
    torch.cuda.synchronize()
    for rows in (slice(0, 4), slice(M - 4, M)):
        for a, b in zip((h, y, rstd) + tuple(y8), want[:3] + tuple(want[3])):
            assert torch.equal(a[rows], b)
    assert not y[4:-4].any()
    y.zero_()
    y[-4:] = bf16(r)
    dx, dg = q.qlora_rms_norm_bwd(y, h, rstd, tg, dx=None)
    wx, wg = q.qlora_rms_norm_bwd(bf16(r), bf16(x), want[2], tg)
    torch.cuda.synchronize()
    assert torch.equal(dx[-4:], wx) and not dx[4:-4].any() and not dx[:4].any()
    # four terms each, the zeros of the other rows in any order between them
    torch.testing.assert_close(dg, wg, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("M,K", [((1 << 21) + 3, 1032), ((1 << 23) + 9, 8)])
def test_more_rows_than_one_row_of_workgroups(M, K):
    """More workgroups than a row of the grid takes: the ones past the last row of the
    matrix write nothing."""
    need_gpu()
    say(f"norm {M} x {K}")
    _, x, r, tg, g = _inputs(4, K, 7, True)
    X = torch.zeros((M, K), dtype=torch.bfloat16, device=dev())
    X[:4], X[-4:] = bf16(x), bf16(x)
    h, y, rstd = q.qlora_rms_norm_fwd(X, tg, eps=EPS)
    _, wy, wr = q.qlora_rms_norm_fwd(bf16(x), tg, eps=EPS)
    torch.cuda.synchronize()
    for rows in (slice(0, 4), slice(M - 4, M)):
        assert torch.equal(y[rows], wy) and torch.equal(rstd[rows], wr)
    y.zero_()
    y[-4:] = bf16(r)
    dx, none = q.qlora_rms_norm_bwd(y, h, rstd, tg, need_dg=False)
    dx2, dg = q.qlora_rms_norm_bwd(y, h, rstd, tg)
    wx, wg = q.qlora_rms_norm_bwd(bf16(r), bf16(x), wr, tg)
    torch.cuda.synchronize()
    assert none is None and torch.equal(dx, dx2)
    assert torch.equal(dx[-4:], wx) and not dx[4:-4].any()
    torch.testing.assert_close(dg, wg, rtol=1e-5, atol=1e-5)


def test_streams_graph_and_workspaces():
    """On another stream, and in two graphs that share no workspace with eager
    calls between their replays."""
    need_gpu()
    say("norm in graphs")
    M, K = 1200, 4096    # sums of workgroups in a workspace
    x, r = torch.randn(M, K, device=dev()).bfloat16(), torch.randn(M, K, device=dev()).bfloat16()
    dy, g = torch.randn(M, K, device=dev()).bfloat16(), torch.rand(K, device=dev()) + 0.5
    ws = torch.full((q.lib().qlora_rms_norm_bwd_workspace_bytes(M, K),), 0xFF, dtype=torch.uint8,
                    device=dev())
    assert ws.numel() > 0

    def step(workspace=None):
        h, y, rstd, y8 = q.qlora_rms_norm_fwd(x, g, r, EPS, act8=True)
        return (h, y, rstd, *y8, *q.qlora_rms_norm_bwd(dy, h, rstd, g, dres=y, workspace=workspace))
    first = step(ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step()))
    for i in range(3):
        x.copy_(torch.randn(M, K, device=dev()))
        dy.copy_(torch.randn(M, K, device=dev()))
        for graph, _ in graphs:
            graph.replay()
        a = [[t.clone() for t in got] for _, got in graphs]
        b = step(ws)
        torch.cuda.synchronize()
        for got in a:
            assert all(torch.equal(u, v) for u, v in zip(got, b))


def test_neighbours_stay():
    """Outputs in the middle of larger buffers: nothing around them changes."""
    need_gpu()
    say("norm, guards")
    for M, K in ((3, 72), (5, 2048), (2, 8200), (700, 3200)):
        _, x, r, tg, _ = _inputs(M, K, K, True)
        pad = lambda: torch.full((M + 2, K), 7.0, dtype=torch.bfloat16, device=dev())
        H, Y, DX = pad(), pad(), pad()
        dg = torch.full((K + 64,), 7.0, device=dev())
        q.qlora_rms_norm_fwd(bf16(x), tg, bf16(r), EPS, h=H[1:-1], y=Y[1:-1])
        rstd = torch.ones(M, device=dev())
        q.qlora_rms_norm_bwd(bf16(x), bf16(r), rstd, tg, dx=DX[1:-1], dg=dg[32:-32])
        torch.cuda.synchronize()
        for t in (H, Y, DX):
            assert (t[0] == 7).all() and (t[-1] == 7).all()
        assert (dg[:32] == 7).all() and (dg[-32:] == 7).all()
