"""GPU parity of the routing to experts: ids exactly those of a float64 choice,
weights and gradients within half a step of their type."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import within
from gpu_util import dev, need_gpu, say, torch
from oracle import router as orr

pytestmark = pytest.mark.gpu

# one rounding of a 64-bit value to fp32 (and to bf16 after it), 64-bit error besides
F32, BF16 = 1.001 * 2.0 ** -24, 2.0 ** -8 + 2.0 ** -23

CASES = [
    # tokens, E, topk, score, bias, groups, top_groups, group_top, renorm, fp32
    (1, 1, 1, "softmax", False, 1, 1, 1, True, True),
    (3, 8, 2, "softmax", False, 1, 1, 1, True, False),
    (5, 8, 8, "softmax", False, 1, 1, 1, False, True),
    (7, 7, 3, "sigmoid", False, 1, 1, 1, False, False),
    (33, 64, 6, "softmax", True, 1, 1, 1, True, True),
    (20, 65, 4, "sigmoid", True, 1, 1, 1, True, True),
    (64, 100, 10, "softmax", False, 4, 2, 1, False, True),
    (31, 128, 8, "softmax", False, 8, 3, 2, True, True),
    (50, 256, 8, "sigmoid", True, 8, 4, 2, True, True),
    (50, 256, 8, "sigmoid", True, 8, 4, 2, False, False),
    (9, 160, 6, "softmax", True, 8, 3, 1, False, False),
    (6, 63, 5, "sigmoid", True, 21, 5, 2, True, True),
    (6, 64, 3, "softmax", True, 64, 9, 1, True, True),
    (10, 320, 12, "softmax", True, 5, 2, 2, True, True),
    (4, 512, 64, "softmax", False, 1, 1, 1, True, True),
    (5, 1000, 64, "sigmoid", True, 10, 3, 2, True, False),
    (3, 1024, 33, "softmax", False, 32, 7, 2, False, True),
    (3, 1024, 64, "softmax", True, 1, 1, 1, False, True),
]


def _logits(rng, tokens, E, fp32, kind):
    x = 2 * rng.standard_normal((tokens, E)) + rng.standard_normal(E)
    if kind == "ties":          # few different values, both zeros
        x = rng.integers(-2, 3, (tokens, E)) * 0.5
        x[x == 0] = rng.choice([0.0, -0.0], int((x == 0).sum()))
    elif kind == "masked":
        x[rng.random(x.shape) < 0.5] = -np.inf
        x[::3] = -np.inf        # rows that the mask leaves empty
        x[1::3, : E // 2] = np.finfo(np.float32).min if fp32 else -3.3895313892515355e38
    elif kind == "wide":
        x *= 60.0
    t = torch.from_numpy(x.astype(np.float32)).to(dev())
    t = t if fp32 else t.bfloat16()
    return t, t.double().cpu().numpy()


@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "wide"])
@pytest.mark.parametrize("tokens,E,topk,score,bias,groups,tg,gt,renorm,fp32", CASES)
def test_router(tokens, E, topk, score, bias, groups, tg, gt, renorm, fp32, kind):
    need_gpu()
    say(f"router tokens={tokens} E={E} topk={topk} {score} bias={bias} groups={groups}/{tg}/{gt} "
        f"renorm={renorm} fp32={fp32} {kind}")
    if kind in ("ties", "wide") and tg < groups and gt == 2:
        # sums of two scores: equal ones are rounded apart, or not, as they are formed
        kind = "normal"
    rng = np.random.default_rng(E + topk)
    t, x = _logits(rng, tokens, E, fp32, kind)
    b = None
    if bias:
        b = torch.from_numpy((0.05 * rng.standard_normal(E)).astype(np.float32)).to(dev())
        if kind == "ties":
            b = torch.zeros_like(b)     # equal logits stay equal
    kw = dict(score=score, renorm=renorm, scale=2.5)
    ids, w = q.qlora_router_fwd(t, topk, bias=b, groups=groups, top_groups=tg, group_top=gt, **kw)
    dw = torch.from_numpy(rng.standard_normal((tokens, topk)).astype(np.float32)).to(dev())
    dl = q.qlora_router_bwd(dw, t, ids, **kw)
    torch.cuda.synchronize()
    wid, ww = orr.fwd(x, topk, score, None if b is None else b.double().cpu().numpy(), groups, tg,
                      gt, renorm, 2.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), wid)
    within("weights", w, ww, F32 * np.abs(ww) + 2.0 ** -149)
    assert dl.dtype == t.dtype
    want, mag = orr.bwd(dw.double().cpu().numpy(), x, wid, score, renorm, 2.5)
    bound = (F32 if fp32 else BF16) * np.abs(want) + 1e-13 * mag + (2.0 ** -149 if fp32 else 2.0 ** -133)
    if score == "softmax" and not renorm:
        # p_e (dw_e - sum_j p_j dw_j) in 64 bits, here and in the reference: p is off by
        # (E / 64 + 8 for the sum's additions) 2^-53, at most 24 2^-53, of itself, the sum over
        # j by topk 2^-53 more, each times |dw|; where p_e is next to 1 this is what is left
        bound += 2.5 * 2 * (topk + 24) * 2.0 ** -53 * np.abs(dw.double().cpu().numpy()).max(
            axis=1, keepdims=True)
    within("dlogits", dl, want, bound)


def test_many_tokens():
    """A batch of 8192 tokens and 256 experts: every id, in the order of 64 bits."""
    need_gpu()
    say("router, 8192 x 256")
    g = torch.Generator(device=dev()).manual_seed(0)
    x = 2 * torch.randn(8192, 256, generator=g, device=dev())
    b = 0.05 * torch.randn(256, generator=g, device=dev())
    ids, w = q.qlora_router_fwd(x, 8, "sigmoid", b, groups=8, top_groups=4, group_top=2)
    torch.cuda.synchronize()
    rank = 1 / (1 + np.exp(-x.double().cpu().numpy())) + b.double().cpu().numpy()
    two = np.sort(rank.reshape(8192, 8, 32), axis=2)[:, :, -2:].sum(axis=2)
    stay = np.argsort(-two, axis=1, kind="stable")[:, :4]
    keep = np.zeros((8192, 8), bool)
    np.put_along_axis(keep, stay, True, 1)
    rank[~np.repeat(keep, 32, axis=1)] = -np.inf
    np.testing.assert_array_equal(ids.cpu().numpy(),
                                  np.argsort(-rank, axis=1, kind="stable")[:, :8])
    np.testing.assert_allclose(w.sum(dim=1).cpu().numpy(), 1, rtol=8 * 2.0 ** -24)


@pytest.mark.parametrize("E,groups,tg,gt", [(8, 1, 1, 1), (64, 8, 3, 2), (128, 16, 5, 1),
                                            (256, 8, 4, 2), (256, 16, 4, 2), (252, 4, 2, 2),
                                            (512, 8, 2, 1), (1024, 4, 1, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choices_next_to_each_other(E, groups, tg, gt, score):
    """Ranks that 32 bits cannot tell apart, or tell apart wrongly: logits next to each
    other with biases that make up for them, equal ones, ones that mask and force."""
    need_gpu()
    say(f"router, close ranks E={E} groups={groups}/{tg}/{gt} {score}")
    rng = np.random.default_rng(E)
    T, k = 40, min(8, E // groups * tg)
    x = rng.standard_normal((T, E)).astype(np.float32)
    p = np.stack([orr.scores(r.astype(np.float64), score) for r in x])
    b = (0.5 - p.mean(axis=0)).astype(np.float32)
    x[10:20] = x[0]                      # a token whose biases level all its ranks
    b2 = (0.5 - p[0]).astype(np.float32)
    x[20:24, 3] = -np.inf
    x[24:28] = np.round(x[24:28])        # few different values
    special = b.copy()
    special[[0, E // 2, E - 1]] = [np.inf, -np.inf, np.nan]
    special[1] = np.inf
    t = torch.from_numpy(x).to(dev())
    for bias in (b, b2, np.zeros(E, np.float32), special):
        ids, _ = q.qlora_router_fwd(t, k, score, torch.from_numpy(bias).to(dev()), groups, tg, gt)
        torch.cuda.synchronize()
        got = ids.cpu().numpy()
        for i in range(T):
            r = orr.scores(x[i].astype(np.float64), score) + bias.astype(np.float64)
            want = orr.choose(x[i].astype(np.float64), k, score, bias.astype(np.float64), groups, tg,
                              gt)
            if got[i].tolist() != want:
                # 64-bit ranks may be rounded apart: the same ranks to 2^-50, expert for expert,
                # and where groups are chosen, a border that close
                a_, w_ = r[got[i]], r[np.array(want)]
                close = np.abs(a_ - w_) <= 2.0 ** -50
                assert (close | (groups > tg)).all() and (np.sort(got[i]) >= 0).all(), (i, got[i], want)
                if groups > tg:
                    two = -np.sort(-np.where(np.isnan(r) | (x[i] == -np.inf), -np.inf, r).reshape(
                        groups, -1), axis=1)[:, :gt]
                    s = np.sort(np.where(np.isfinite(two), two, 0).sum(axis=1))[::-1]
                    assert close.all() or abs(s[tg - 1] - s[tg]) <= 2.0 ** -49, (i, got[i], want)


@pytest.mark.parametrize("E,topk,groups,tg,gt,fp32", [
    (256, 8, 8, 4, 2, False), (256, 8, 8, 4, 2, True), (256, 32, 4, 2, 1, True), (250, 7, 1, 1, 1, True),
    (128, 6, 16, 5, 2, True), (128, 1, 4, 2, 1, False), (100, 6, 1, 1, 1, False), (64, 6, 8, 3, 2, True),
    (64, 6, 32, 9, 2, True), (33, 5, 1, 1, 1, True), (4, 4, 1, 1, 1, False), (1, 1, 1, 1, 1, True)])
@pytest.mark.parametrize("renorm", [True, False])
def test_many_tokens_as_few(E, topk, groups, tg, gt, fp32, renorm):
    """Two tokens share a wave in a large batch: every token gets the bits that it gets in
    a small one, with ranks next to each other and equal, masked, NaN and tiny scores."""
    need_gpu()
    say(f"router, 2051 tokens as few E={E} topk={topk} groups={groups}/{tg}/{gt} fp32={fp32}")
    rng = np.random.default_rng(E + topk)
    T = 2051
    x = rng.standard_normal((T, E)).astype(np.float32)
    x[100:200] = x[100]
    x[200:300] = np.round(x[200:300])
    x[300:400] = x[300] + 1e-6 * rng.standard_normal((100, E))
    x[400:500][rng.random((100, E)) < 0.7] = -np.inf
    x[500:502] = -np.inf
    x[502:504] = -700 + x[502:504]           # sigmoids that hardly are numbers
    x[504:506, 0] = np.nan
    x[507, E - 1] = np.inf
    t = torch.from_numpy(x).to(dev())
    t = t if fp32 else t.bfloat16()
    xs = t.double().cpu().numpy()
    levels = [np.zeros(E), 0.05 * rng.standard_normal(E), 0.5 - orr.scores(xs[100], "sigmoid"),
              0.5 - orr.scores(xs[300], "sigmoid")]
    special = levels[1].copy()
    special[0], special[E // 2], special[E - 1] = np.inf, -np.inf, np.nan
    for i, level in enumerate(levels + [special]):
        b = torch.from_numpy(level.astype(np.float32)).to(dev())
        args = (topk, "sigmoid", b, groups, tg, gt, renorm, 2.5)
        I = torch.full((T + 2, topk), 77, dtype=torch.int32, device=dev())
        W = torch.full((T + 2, topk), 77.0, device=dev())
        q.qlora_router_fwd(t, *args, ids=I[1:-1], weights=W[1:-1])
        few = [q.qlora_router_fwd(t[j:j + 293], *args) for j in range(0, T, 293)]
        torch.cuda.synchronize()
        ids, w = torch.cat([f[0] for f in few]), torch.cat([f[1] for f in few])
        assert (I[0] == 77).all() and (I[-1] == 77).all() and (W[0] == 77).all() and (W[-1] == 77).all()
        np.testing.assert_array_equal(I[1:-1].cpu().numpy(), ids.cpu().numpy())
        np.testing.assert_array_equal(W[1:-1].cpu().numpy(), w.cpu().numpy())
        if i == 1:   # ranks that lie apart
            some = np.r_[0:20, 400:420, 500:504, 2040:2051]
            wid, ww = orr.fwd(xs[some], topk, "sigmoid", b.double().cpu().numpy(), groups, tg, gt, renorm, 2.5)
            np.testing.assert_array_equal(ids.cpu().numpy()[some], wid)
            within("weights", w[torch.from_numpy(some).to(dev())], ww, F32 * np.abs(ww) + 2.0 ** -149)


@pytest.mark.parametrize("E,topk", [(256, 8), (256, 32), (250, 7), (128, 8), (100, 6), (64, 6), (64, 32),
                                    (33, 5), (8, 2), (2, 2), (1, 1)])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", True), ("sigmoid", False),
                                          ("softmax", False)])
def test_many_tokens_by_logit_as_few(E, topk, fp32, score, renorm):
    """The same without a bias: logits equal within a lane and across, zeros of both
    signs, masked, extreme, NaN, and sigmoids that hardly are numbers."""
    need_gpu()
    say(f"router by logit, 2051 tokens as few E={E} topk={topk} fp32={fp32} {score} renorm={renorm}")
    rng = np.random.default_rng(E + topk)
    T = 2051
    x = rng.standard_normal((T, E)).astype(np.float32)
    x[100:200] = np.round(2 * x[100:200]) / 2
    x[200:300] = np.where(rng.random((100, E)) < 0.5, 0.0, -0.0)
    x[300:400][rng.random((100, E)) < 0.7] = -np.inf
    x[400:402] = -np.inf
    x[402:405] = -700 + x[402:405]
    x[405] = np.where(rng.random(E) < 0.5, 3.3e38, -3.3e38)
    x[406, 0] = np.nan
    x[407, E - 1] = np.inf
    x[409], x[411] = np.nan, 1e-40 * x[411]
    t = torch.from_numpy(x).to(dev())
    t = t if fp32 else t.bfloat16()
    args = (topk, score, None, 1, 1, 1, renorm, 2.5)
    I = torch.full((T + 2, topk), 77, dtype=torch.int32, device=dev())
    W = torch.full((T + 2, topk), 77.0, device=dev())
    q.qlora_router_fwd(t, *args, ids=I[1:-1], weights=W[1:-1])
    few = [q.qlora_router_fwd(t[j:j + 293], *args) for j in range(0, T, 293)]
    torch.cuda.synchronize()
    ids, w = torch.cat([f[0] for f in few]), torch.cat([f[1] for f in few])
    assert (I[0] == 77).all() and (I[-1] == 77).all() and (W[0] == 77).all() and (W[-1] == 77).all()
    np.testing.assert_array_equal(I[1:-1].cpu().numpy(), ids.cpu().numpy())
    np.testing.assert_array_equal(W[1:-1].cpu().numpy(), w.cpu().numpy())
    some = np.r_[0:20, 100:120, 200:210, 300:330, 400:406, 411, T - 11:T]
    wid, ww = orr.fwd(t.double().cpu().numpy()[some], topk, score, None, 1, 1, 1, renorm, 2.5)
    np.testing.assert_array_equal(I[1:-1].cpu().numpy()[some], wid)
    within("weights", w[torch.from_numpy(some).to(dev())], ww, F32 * np.abs(ww) + 2.0 ** -149)


@pytest.mark.parametrize("E,topk,fp32", [(256, 8, False), (256, 32, True), (250, 7, False), (100, 6, True),
                                         (64, 6, False), (33, 9, True), (8, 2, False), (1, 1, True)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", True), ("sigmoid", False),
                                          ("softmax", False)])
def test_many_gradients_as_few(E, topk, fp32, score, renorm):
    """The same of the backward, with ids that are missing, outside and named twice."""
    need_gpu()
    say(f"router backward, 4099 tokens as few E={E} topk={topk} {score} renorm={renorm}")
    rng = np.random.default_rng(E + topk)
    T = 4099
    x = 2 * rng.standard_normal((T, E)).astype(np.float32)
    x[100:300][rng.random((200, E)) < 0.5] = -np.inf
    x[300:302] = -np.inf
    x[302:304] = -700 + x[302:304]
    x[305, 0], x[306, E - 1] = np.nan, np.inf
    t = torch.from_numpy(x).to(dev())
    t = t if fp32 else t.bfloat16()
    ids = rng.integers(-2, E + 2, (T, topk)).astype(np.int32)       # any, some twice
    ids[::2] = np.argsort(rng.random((len(ids[::2]), E)), axis=1)[:, :topk]   # all apart
    ids = torch.from_numpy(ids).to(dev())
    dw = torch.from_numpy(rng.standard_normal((T, topk)).astype(np.float32)).to(dev())
    D = torch.full((T + 2, E), 77.0, device=dev(), dtype=t.dtype)
    q.qlora_router_bwd(dw, t, ids, score, renorm, 2.5, dlogits=D[1:-1])
    few = torch.cat([q.qlora_router_bwd(dw[j:j + 293], t[j:j + 293], ids[j:j + 293], score, renorm, 2.5)
                     for j in range(0, T, 293)])
    torch.cuda.synchronize()
    assert (D[0] == 77).all() and (D[-1] == 77).all()
    assert torch.equal(D[1:-1].nan_to_num(5e4), few.nan_to_num(5e4))
    bad = torch.isnan(few).any(dim=1)
    assert bad[305] and bad[306] and bad.sum() == 2 and torch.isnan(few[bad]).all()
    some = np.r_[0:30, 100:130, 300:304, T - 20:T]
    xs, n = t.double().cpu().numpy()[some], ids.cpu().numpy()[some]
    n = np.where((n < 0) | (n >= E), -1, n)
    n = np.where((n >= 0) & (np.take_along_axis(xs, np.maximum(n, 0), 1) == -np.inf), -1, n)
    want, mag = orr.bwd(dw.double().cpu().numpy()[some], xs, n, score, renorm, 2.5)
    got = few[torch.from_numpy(some).to(dev())]
    within("dlogits", got, want, (F32 if fp32 else BF16) * np.abs(want) + 1e-13 * mag + 2.0 ** -149)


def test_gradient_of_a_sure_choice():
    """Where one expert takes all but 1e-6, the gradient keeps its digits."""
    need_gpu()
    say("router, sure choices")
    x = np.zeros((4, 8), np.float32)
    x[:, 0] = [14.0, 20.0, 40.0, 80.0]
    t = torch.from_numpy(x).to(dev())
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, _ = q.qlora_router_fwd(t, 2, score, renorm=renorm)
            dw = torch.tensor([[1.0, -0.5]] * 4, device=dev())
            dl = q.qlora_router_bwd(dw, t, ids, score, renorm)
            torch.cuda.synchronize()
            want, mag = orr.bwd(dw.double().cpu().numpy(), x.astype(np.float64), ids.cpu().numpy(), score,
                                renorm)
            # 1 - p to 2^-53, where p is within 1e-6 of 1
            within("dlogits", dl, want, F32 * np.abs(want) + 4e-16 + 2.0 ** -149)


def test_bad_logits_show():
    """NaN and +inf make a token's weights and gradients NaN; its ids stay within
    the experts and apart, and other tokens are as without them."""
    need_gpu()
    say("router, NaN logits")
    for E, groups in ((8, 1), (96, 4), (512, 8)):
        t = torch.randn(9, E, device=dev())
        clean = t.clone()
        t[2, 3], t[5, 0], t[7] = float("nan"), float("inf"), float("nan")
        for score in ("softmax", "sigmoid"):
            for bias in (None, torch.randn(E, device=dev())):
                for renorm in (True, False):
                    cfg = dict(score=score, renorm=renorm)
                    kw = dict(bias=bias, groups=groups, top_groups=max(1, groups // 2), **cfg)
                    ids, w = q.qlora_router_fwd(t, 3, **kw)
                    ids0, w0 = q.qlora_router_fwd(clean, 3, **kw)
                    dw = torch.ones_like(w)
                    dl = q.qlora_router_bwd(dw, t, ids, **cfg)
                    dl0 = q.qlora_router_bwd(dw, clean, ids0, **cfg)
                    torch.cuda.synchronize()
                    bad = torch.tensor([2, 5, 7], device=dev())
                    good = torch.tensor([0, 1, 3, 4, 6, 8], device=dev())
                    assert torch.equal(ids[good], ids0[good]) and torch.equal(w[good], w0[good])
                    assert torch.equal(dl[good], dl0[good])
                    assert (ids >= -1).all() and (ids < E).all() and (ids[7] == -1).all()
                    for row in (2, 5):
                        assert len(set(ids[row].tolist())) == 3 and 3 not in ids[2].tolist()
                        assert torch.isnan(w[row][ids[row] >= 0]).all()
                    assert torch.isnan(dl[bad]).all() and not w[7].any()


def test_ids_of_the_callers_own():
    """Backward: ids outside the experts are slots not taken, the same expert twice
    adds up, and a masked expert named by an id has no gradient."""
    need_gpu()
    say("router, ids of the caller's own")
    x = torch.randn(5, 12, device=dev())
    x[4, 2] = -float("inf")
    ids = torch.tensor([[3, 3, 1], [-1, 5, 12], [-2 ** 31, 2 ** 31 - 1, -1], [0, 11, 0], [2, 1, 4]],
                       dtype=torch.int32, device=dev())
    dw = torch.randn(5, 3, device=dev())
    norm = np.where((ids.cpu().numpy() < 0) | (ids.cpu().numpy() >= 12), -1, ids.cpu().numpy())
    norm[4, 0] = -1
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            dl = q.qlora_router_bwd(dw, x, ids, score, renorm)
            torch.cuda.synchronize()
            want, mag = orr.bwd(dw.double().cpu().numpy(), x.double().cpu().numpy(), norm, score,
                                renorm)
            within("dlogits", dl, want, F32 * np.abs(want) + 1e-13 * mag + 2.0 ** -149)


def test_guards_streams_and_graph():
    """Nothing around the outputs changes; another stream and replays of a graph
    give the same bits as eager calls."""
    need_gpu()
    say("router in a graph")
    T, E, k = 301, 72, 5
    x, b = torch.randn(T, E, device=dev()), 0.1 * torch.randn(E, device=dev())
    dw = torch.randn(T, k, device=dev())
    I = torch.full((T + 2, k), 7, dtype=torch.int32, device=dev())
    W, D = torch.full((T + 2, k), 7.0, device=dev()), torch.full((T + 4, E), 7.0, device=dev())
    q.qlora_router_fwd(x, k, bias=b, groups=9, top_groups=4, ids=I[1:-1], weights=W[1:-1])
    q.qlora_router_bwd(dw, x, I[1:-1], dlogits=D[2:-2])
    torch.cuda.synchronize()
    assert (I[0] == 7).all() and (I[-1] == 7).all() and (W[0] == 7).all() and (W[-1] == 7).all()
    assert (D[:2] == 7).all() and (D[-2:] == 7).all()

    def step():
        ids, w = q.qlora_router_fwd(x, k, bias=b, groups=9, top_groups=4)
        return ids, w, q.qlora_router_bwd(dw, x, ids)
    first = step()
    torch.cuda.synchronize()
    assert torch.equal(first[0], I[1:-1]) and torch.equal(first[2], D[2:-2])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        x.copy_(torch.randn(T, E, device=dev()))
        graph.replay()
        a = [t.clone() for t in got]
        e = step()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(a, e))
    # rows of larger logits, which start at any element
    for E2, dt in ((65, torch.bfloat16), (130, torch.bfloat16), (7, torch.bfloat16), (66, torch.float32),
                   (3, torch.float32)):
        big = torch.randn(T * E2 + 1, device=dev()).to(dt)[1:].view(T, E2)
        bias = torch.randn(E2 + 1, device=dev())[1:]
        for lo in (1, 2, 3):
            for s in ("softmax", "sigmoid"):
                i1, w1 = q.qlora_router_fwd(big[lo:lo + 40], 3, s, bias)
                i2, w2 = q.qlora_router_fwd(big[lo:lo + 40].clone(), 3, s, bias.clone())
                d1 = q.qlora_router_bwd(w1, big[lo:lo + 40], i1, s)
                d2 = q.qlora_router_bwd(w2, big[lo:lo + 40].clone(), i2, s)
                torch.cuda.synchronize()
                assert torch.equal(i1, i2) and torch.equal(w1, w2) and torch.equal(d1, d2)
    ids, w = q.qlora_router_fwd(x[:0], k)
    assert ids.shape == (0, k) and q.qlora_router_bwd(dw[:0], x[:0], ids).shape == (0, E)


def test_many_tokens_in_a_graph():
    """The batches whose tokens share waves, captured once and replayed on new inputs
    with eager calls on another stream between the replays."""
    need_gpu()
    say("router, many tokens in a graph")
    T, E, k = 4099, 96, 6
    x, b = torch.randn(T, E, device=dev()), 0.1 * torch.randn(E, device=dev())
    dw = torch.randn(T, k, device=dev())

    def step():
        a = q.qlora_router_fwd(x, k, "sigmoid", b, groups=3, top_groups=2, group_top=2)
        c = q.qlora_router_fwd(x, k)
        return (*a, *c, q.qlora_router_bwd(dw, x, a[0], "sigmoid"), q.qlora_router_bwd(dw, x, c[0]))
    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        x.copy_(torch.randn(T, E, device=dev()))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            other = step()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        for a, c, e in zip(got, other, eager):
            assert torch.equal(a, c) and torch.equal(a, e)
