"""The router's gradients where one expert takes nearly all: what is left of 1 - p
keeps its digits, so the bounds are relative to the value, with nothing absolute
beside the last place of the type."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from gpu_util import dev, need_gpu, say, torch
from oracle import router as orr

pytestmark = pytest.mark.gpu

# one rounding of a 64-bit value to fp32 (and to bf16 after it); 64-bit arithmetic is off by
# (E / 64 + topk + 20) 2^-53 of the magnitudes added at most, under 1e-13 of them
F32, BF16, F64 = 1.001 * 2.0 ** -24, 2.0 ** -8 + 2.0 ** -23, 1e-13


def within(name, got, ref, bound):
    """Element by element, down to the smallest numbers."""
    err = np.abs(got.double().cpu().numpy() - ref)
    say(f"  {name}: worst error {(err / bound).max():.3f} of its bound")
    assert (err <= bound).all(), name   # (false for NaN)


def _check(x, ids, dw, score, renorm, fp32):
    t = torch.from_numpy(x.astype(np.float32)).to(dev())
    t = t if fp32 else t.bfloat16()
    xs = t.double().cpu().numpy()
    dl = q.qlora_router_bwd(torch.from_numpy(dw.astype(np.float32)).to(dev()), t,
                            torch.from_numpy(ids.astype(np.int32)).to(dev()), score, renorm, 2.5)
    torch.cuda.synchronize()
    want, mag = orr.bwd(dw.astype(np.float32).astype(np.float64), xs, ids, score, renorm, 2.5)
    least = 2.0 ** -149 if fp32 else 2.0 ** -133
    within(f"dlogits {score} renorm={renorm}", dl, want,
           (F32 if fp32 else BF16) * np.abs(want) + F64 * mag + least)
    return dl, want


@pytest.mark.parametrize("E,topk", [(8, 2), (8, 1), (1, 1), (2, 2), (7, 7), (64, 6), (100, 4), (250, 12),
                                    (512, 8), (1024, 64)])
@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                          ("sigmoid", True)])
def test_digits_of_a_sure_choice(E, topk, fp32, score, renorm):
    """Winners ahead by 5 to 90, the others near each other; all experts chosen, one, or
    some; masked experts among them."""
    need_gpu()
    say(f"router, sure choices E={E} topk={topk} {score} renorm={renorm} fp32={fp32}")
    rng = np.random.default_rng(E + topk)
    gaps = np.array([5.0, 14.0, 20.0, 30.0, 36.0, 40.0, 60.0, 80.0, 90.0] * 2)
    x = 0.5 * rng.standard_normal((len(gaps), E))
    first = rng.integers(0, E, len(gaps))
    x[np.arange(len(gaps)), first] = gaps
    x[9:][rng.random((9, E)) < 0.3] = -np.inf
    ids = np.argsort(-x, axis=1, kind="stable")[:, :topk]
    ids = np.where(np.take_along_axis(x, ids, 1) == -np.inf, -1, ids)
    dw = rng.standard_normal((len(gaps), topk))
    _, want = _check(x, ids, dw, score, renorm, fp32)
    if E > 1 and not renorm:   # the winners' gradients are there to be checked
        sure = np.abs(want[np.arange(7), first[:7]])
        assert (sure > 1e-37).all() and (sure[5:] < 1e-12).all()


def _any_ids(rng, E, topk, T=60):
    """A winner ahead by 0 to 85; experts named twice or more, missing, outside, masked."""
    x = 0.5 * rng.standard_normal((T, E))
    x[:, 1] = np.linspace(0, 85, T)
    x[rng.random((T, E)) < 0.1] = -np.inf
    ids = rng.integers(-1, min(E, 6) + 1, (T, topk))
    ids[::3, 0], ids[::3, -1] = 1, 1
    ids[T // 2:, topk // 2] = E + 3
    live = (ids >= 0) & (ids < E)
    live &= np.take_along_axis(x, np.where(live, ids, 0), 1) > -np.inf
    return x, ids, live, rng.standard_normal((T, topk))


@pytest.mark.parametrize("E,topk", [(8, 3), (96, 6), (300, 20)])
def test_ids_of_the_callers_own(E, topk):
    """Softmax, not renormalised: an expert's slots add up."""
    need_gpu()
    say(f"router, sure choices, any ids E={E} topk={topk}")
    x, ids, live, dw = _any_ids(np.random.default_rng(E), E, topk)
    t = torch.from_numpy(x.astype(np.float32)).to(dev())
    dwt = torch.from_numpy(dw.astype(np.float32)).to(dev())
    dl = q.qlora_router_bwd(dwt, t, torch.from_numpy(ids.astype(np.int32)).to(dev()), "softmax", False, 2.5)
    torch.cuda.synchronize()
    want, mag = orr.bwd(dwt.double().cpu().numpy(), t.double().cpu().numpy(), np.where(live, ids, -1),
                        "softmax", False, 2.5)
    within("dlogits", dl, want, F32 * np.abs(want) + F64 * mag + 2.0 ** -149)


@pytest.mark.parametrize("E,topk,copies", [(8, 3, 1), (96, 6, 1), (300, 20, 1), (64, 6, 80)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalised_ids_of_the_callers_own(E, topk, copies, score):
    """Renormalised weights: with q_i the slots' shares, expert e gets the sum over its
    slots i and the others' slots j of q_i q_j (dw_i - dw_j); two slots of one expert
    have nothing to give each other.  (With copies, enough tokens to share waves.)"""
    need_gpu()
    say(f"router, sure choices, any ids E={E} topk={topk} {score} renormalised")
    x, ids, live, dw = _any_ids(np.random.default_rng(E), E, topk)
    t = torch.from_numpy(x.astype(np.float32)).to(dev())
    dwt = torch.from_numpy(dw.astype(np.float32)).to(dev())
    idt = torch.from_numpy(ids.astype(np.int32)).to(dev())
    dl = q.qlora_router_bwd(dwt.repeat(copies, 1), t.repeat(copies, 1), idt.repeat(copies, 1), score, True,
                            2.5).view(copies, *t.shape)
    torch.cuda.synchronize()
    assert (dl == dl[:1]).all()
    xs, d = t.double().cpu().numpy(), dwt.double().cpu().numpy()
    want, mag = np.zeros(xs.shape), np.zeros(xs.shape)
    for i, row in enumerate(xs):
        n = np.flatnonzero(live[i])
        e, v = ids[i, n], row[ids[i, n]]
        low = np.minimum(v, 0) if score == "sigmoid" else v
        u = np.exp(low - low.max(initial=-np.inf)) / (1 + np.exp(-np.abs(v)) if score == "sigmoid" else 1)
        u = u / u.sum()
        slope = 1 / (1 + np.exp(v)) if score == "sigmoid" else np.ones(len(v))
        for a in range(len(n)):
            for b in range(len(n)):
                if e[a] != e[b]:
                    term = 2.5 * slope[a] * u[a] * u[b] * (d[i, n[a]] - d[i, n[b]])
                    want[i, e[a]] += term
                    mag[i, e[a]] += abs(term)
    within("dlogits", dl[0], want, F32 * np.abs(want) + F64 * mag + 2.0 ** -149)


def test_against_differences():
    """The softmax that is not renormalised: the gradient of sum_i dw_i w_i by differences
    of 64-bit weights."""
    need_gpu()
    say("router, gradient by differences")
    rng = np.random.default_rng(11)
    x = rng.standard_normal((6, 20))
    x[3:, 4] = [4.0, 8.0, 11.0]
    x = x.astype(np.float32).astype(np.float64)
    ids, _ = orr.fwd(x, 5, "softmax", renorm=False)
    dw = rng.standard_normal((6, 5)).astype(np.float32)
    dl, _ = _check(x, ids, dw, "softmax", False, True)
    step = 1e-4
    for e in range(20):
        up, down = x.copy(), x.copy()
        up[:, e] += step
        down[:, e] -= step
        w = [np.array([orr.weights(r, i, "softmax", False, 2.5) for r, i in zip(v, ids)])
             for v in (up, down)]
        diff = ((w[0] - w[1]) * dw).sum(axis=1) / (2 * step)
        # a weight's third derivative is at most 2.5 / 8, times step^2 / 6: 5.3e-10; 24 roundings of
        # two weights to 2^-53 over twice the step: 6.7e-11; and the gradient's own rounding
        bound = 1e-9 * np.abs(dw).sum(axis=1) + 2.0 ** -24 * np.abs(diff)
        assert (np.abs(dl[:, e].double().cpu().numpy() - diff) <= bound).all()
