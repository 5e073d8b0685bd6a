"""Sigmoid and bias: the choice that 32 bits make and 64 prove is the one that is made
wholly in 64 bits, to the last id.  A token with a NaN logit is chosen wholly in 64 bits,
and NaN is passed over as a masked logit is: so a token with one expert masked, and the
same token with that expert at NaN, have to get the same ids."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from gpu_util import dev, need_gpu, say, torch

pytestmark = pytest.mark.gpu


def _inputs(kind, T, E, rng):
    x, b = rng.standard_normal((T, E)), 0.05 * rng.standard_normal(E)
    if kind == "level":       # biases that make up for a row's scores, logits next to that row
        noise = x
        x = x[:1] + 1e-7 * 10.0 ** rng.integers(0, 4, (T, 1)) * noise
        b = 0.5 - 1 / (1 + np.exp(-x[0]))
    elif kind == "near":      # a token's logits and the biases next to each other
        x = x[:, :1] + 1e-6 * 10.0 ** rng.integers(0, 4, (T, 1)) * x
        b = 1e-6 * b
    elif kind == "few":       # few different values: equal ranks and sums
        x, b = np.round(2 * x) / 2, np.round(40 * b) / 8
    elif kind == "wide":
        x, b = 100 * x, b * 10.0 ** rng.integers(-8, 3)
    else:                     # biases that force and forbid
        b[rng.integers(0, E, 4)] = [np.inf, 3e38, -np.inf, np.nan]
    x = torch.from_numpy(x.astype(np.float32)).to(dev())
    x[torch.from_numpy(rng.random((T, E)) < 0.2).to(dev())[: T // 4].nonzero(as_tuple=True)] = -float("inf")
    return x, torch.from_numpy(b.astype(np.float32)).to(dev())


@pytest.mark.parametrize("kind", ["level", "near", "few", "wide", "special"])
@pytest.mark.parametrize("E,topk,groups,tg,gt", [
    (256, 8, 8, 4, 2), (256, 8, 8, 4, 1), (256, 32, 4, 2, 2), (250, 7, 1, 1, 1), (128, 6, 16, 5, 2),
    (64, 6, 8, 3, 2), (64, 6, 32, 9, 2), (64, 3, 64, 9, 1), (32, 4, 8, 5, 2), (512, 12, 8, 2, 2),
    (1024, 40, 16, 4, 2), (8, 2, 4, 2, 2)])
@pytest.mark.parametrize("T", [500, 2500])
def test_choice_of_32_bits_is_that_of_64(kind, E, topk, groups, tg, gt, T):
    need_gpu()
    say(f"router, close ranks {kind} T={T} E={E} topk={topk} groups={groups}/{tg}/{gt}")
    rng = np.random.default_rng(E + topk + T)
    x, b = _inputs(kind, T, E, rng)
    one = torch.from_numpy(rng.integers(0, E, (T, 1))).to(dev())
    for t in (x, x.bfloat16()):
        args = (topk, "sigmoid", b, groups, tg, gt)
        ids, w = q.qlora_router_fwd(t.scatter(1, one, -float("inf")), *args)
        wide, bad = q.qlora_router_fwd(t.scatter(1, one, float("nan")), *args)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(ids.cpu().numpy(), wide.cpu().numpy())
        assert torch.isnan(bad[wide >= 0]).all() and torch.isfinite(w).all()
        assert not (ids == one).any()
