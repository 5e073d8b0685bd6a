"""The router's choice where ranks and sums of two are equal to the last bit, and large
batches against a float64 choice of every token."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import within
from gpu_util import dev, need_gpu, say, torch
from oracle import router as orr

pytestmark = pytest.mark.gpu

F32, BF16 = 1.001 * 2.0 ** -24, 2.0 ** -8 + 2.0 ** -23

GROUPS = [
    # tokens, E, topk, groups, top_groups; groups within lanes, across them, of few tokens and many
    (40, 256, 8, 8, 4), (2100, 256, 8, 8, 4), (2053, 64, 6, 8, 3), (30, 128, 8, 8, 3),
    (2049, 128, 12, 16, 5), (25, 63, 5, 21, 5), (20, 320, 12, 5, 2), (2060, 96, 7, 6, 4),
    (12, 1000, 30, 10, 3), (12, 1024, 33, 32, 7), (2051, 160, 6, 8, 3),
]


@pytest.mark.parametrize("tokens,E,topk,groups,tg", GROUPS)
@pytest.mark.parametrize("score,bias", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                        ("sigmoid", True)])
@pytest.mark.parametrize("fp32", [True, False])
def test_groups_of_equal_sums(tokens, E, topk, groups, tg, score, bias, fp32):
    """Every group is a copy of one of three, its members in another order: sums of two
    that are equal however they are formed, the lower group first, and equal experts in
    several groups, the lower index first."""
    need_gpu()
    say(f"router, equal groups tokens={tokens} E={E} topk={topk} groups={groups}/{tg} {score} bias={bias}")
    rng = np.random.default_rng(E + topk)
    size = E // groups
    # values apart by 2^-6 at least, so that only equal ranks are close (bf16 holds them: 3 size <= 300)
    base = rng.permuted(np.tile(np.arange(3 * size) / 64.0 - 1.0, (tokens, 1)), axis=1).reshape(
        tokens, 3, size)
    kind = rng.integers(0, 3, (tokens, groups))
    x = np.take_along_axis(base, kind[:, :, None], axis=1)
    x = rng.permuted(x, axis=2).reshape(tokens, E)
    b = np.zeros(E) if bias else None
    t = torch.from_numpy(x.astype(np.float32)).to(dev())
    t = t if fp32 else t.bfloat16()
    xs = t.double().cpu().numpy()
    some = np.arange(tokens) if tokens < 100 else rng.choice(tokens, 60, replace=False)
    kw = dict(score=score, groups=groups, top_groups=tg, group_top=2)
    ids, w = q.qlora_router_fwd(t, topk, bias=None if b is None else torch.zeros(E, device=dev()),
                                scale=2.5, **kw)
    torch.cuda.synchronize()
    want, ww = orr.fwd(xs[some], topk, score, b, groups, tg, 2, True, 2.5)
    np.testing.assert_array_equal(ids.cpu().numpy()[some], want)
    within("weights", w[torch.from_numpy(some).to(dev())], ww, F32 * np.abs(ww) + 2.0 ** -149)
    # the rule itself: among groups of one kind, no later one without the earlier ones
    staying = np.zeros((tokens, groups), bool)
    for g in range(groups):
        staying[:, g] = ((ids.cpu().numpy() // size) == g).any(axis=1)
    for k in range(3):
        of = kind == k
        earlier = np.cumsum(of & ~staying, axis=1) - (of & ~staying)   # ones left out before
        assert not (of & staying & (earlier > 0)).any()


def _is_clear(x, score, b, topk, groups, tg):
    """Whether what decides a token's choice is equal to the last bit or well apart."""
    size = len(x) // groups
    p = orr.scores(x, score)
    rank = p if b is None else p + b
    far = lambda v: all(a == c or a - c > 1e-12 * max(abs(a), abs(c)) + 1e-300 for a, c in zip(v, v[1:]))
    sums = sorted((sum(sorted(rank[g * size:(g + 1) * size], reverse=True)[:2]) for g in range(groups)),
                  reverse=True)
    best = orr.choose(x, min(topk + 1, size * tg), score, b, groups, tg, 2)
    return far(sums[:tg + 1]) and (b is None or far([rank[e] for e in best]))


@pytest.mark.parametrize("tokens,E,topk,groups,tg", GROUPS)
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True),
                                        ("softmax", True)])
def test_groups_of_saturated_scores(tokens, E, topk, groups, tg, score, bias):
    """Logits so wide that scores round to one and to zero: the sums of two of many groups
    are equal.  Tokens whose border two evaluations of 64 bits could see differently are
    left out (at most half, by the reference alone)."""
    need_gpu()
    say(f"router, saturated groups tokens={tokens} E={E} groups={groups}/{tg} {score} bias={bias}")
    rng = np.random.default_rng(E + topk + 1)
    x = (300.0 * rng.standard_normal((tokens, E))).astype(np.float32)
    # away from where 1 + exp(-x) rounds to one or not, and from subnormal scores
    x = np.where((np.abs(x) > 20) & (np.abs(x) < 39), 20 * np.sign(x), x)
    x = np.where((x < -660) & (x > -760), -600 + rng.random(x.shape), x).astype(np.float32)
    b = (rng.integers(-8, 9, E) / 64.0) if bias else None
    t = torch.from_numpy(x).to(dev())
    ids, w = q.qlora_router_fwd(t, topk, score, None if b is None else torch.from_numpy(
        b.astype(np.float32)).to(dev()), groups, tg, 2, True, 2.5)
    torch.cuda.synchronize()
    some = np.arange(min(tokens, 40))
    xs = x[some].astype(np.float64)
    clear = np.array([_is_clear(r, score, b, topk, groups, tg) for r in xs])
    assert clear.mean() >= 0.5, clear.mean()
    want, ww = orr.fwd(xs[clear], topk, score, b, groups, tg, 2, True, 2.5)
    np.testing.assert_array_equal(ids.cpu().numpy()[some][clear], want)
    within("weights", w[torch.from_numpy(some[clear]).to(dev())], ww, F32 * np.abs(ww) + 2.0 ** -149)


def _whole(x, topk, score, renorm, dw=None):
    """Choice by the logit, weights (times 2.5), and with dw the gradient and its
    magnitudes, of all tokens at once in float64 (finite or -inf logits)."""
    x = x.double().cpu()
    at = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :topk]
    lx = x.gather(1, at)
    live = lx > -np.inf
    if score == "sigmoid":
        t = torch.exp(-x.abs())
        p = torch.where(x > 0, torch.ones_like(t), t) / (1 + t)
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    u = torch.where(live, p.gather(1, at), torch.zeros_like(lx))
    w = u / u.sum(1, keepdim=True) if renorm else u
    ids = torch.where(live, at, torch.full_like(at, -1))
    if dw is None:
        return ids, 2.5 * w
    d = torch.where(live, 2.5 * dw.double().cpu(), torch.zeros_like(w))
    out, mag = torch.zeros_like(x), torch.zeros_like(x)
    slope = 1 / (1 + torch.exp(lx)) if score == "sigmoid" else 1.0
    if renorm:
        g = w * (d * w.sum(1, keepdim=True) - (w * d).sum(1, keepdim=True)) * slope
        m = w * (d.abs() + (w * d).abs().sum(1, keepdim=True)) * slope
    else:
        g = m = w * d * slope
    out.scatter_add_(1, at, g)
    mag.scatter_add_(1, at, m.abs())
    if not renorm and score == "softmax":
        s = (w * d)
        out -= p * s.sum(1, keepdim=True)
        mag += p * s.abs().sum(1, keepdim=True)
    return ids, out, mag


@pytest.mark.parametrize("tokens,E,topk", [(8192, 64, 6), (8192, 256, 8), (3000, 100, 6), (4099, 128, 32),
                                           (2500, 300, 10), (2100, 1024, 40), (16001, 8, 2)])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_every_token_by_logit(tokens, E, topk, fp32, score, renorm):
    """Ids, weights and gradients of every token of a large batch, equal logits (bf16 has
    many) and masked ones among them."""
    need_gpu()
    say(f"router by logit, every token of {tokens} x {E} topk={topk} fp32={fp32} {score} renorm={renorm}")
    g = torch.Generator(device=dev()).manual_seed(tokens + E)
    x = 2 * torch.randn(tokens, E, generator=g, device=dev())
    x[100:600] = torch.round(x[100:600])
    x[600:1000][torch.rand((400, E), generator=g, device=dev()) < 0.4] = -float("inf")
    x[600:1000, 0] = 0.5     # (one expert at least)
    x = x if fp32 else x.bfloat16()
    dw = torch.randn(tokens, topk, generator=g, device=dev())
    ids, w = q.qlora_router_fwd(x, topk, score, renorm=renorm, scale=2.5)
    dl = q.qlora_router_bwd(dw, x, ids, score, renorm, 2.5)
    torch.cuda.synchronize()
    want, ww = _whole(x, topk, score, renorm)
    assert torch.equal(ids.long().cpu(), want)
    within("weights", w, ww.numpy(), F32 * ww.abs().numpy() + 2.0 ** -149)
    _, out, mag = _whole(x, topk, score, renorm, dw)
    least = 2.0 ** -149 if fp32 else 2.0 ** -133
    within("dlogits", dl, out.numpy(), ((F32 if fp32 else BF16) * out.abs() + 1e-13 * mag + least).numpy())
