"""Tokens that share a wave do not show in each other: whatever a neighbour's gradients,
ids and logits are, a token gets the same bits."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from gpu_util import dev, need_gpu, say, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,topk", [(64, 6), (256, 8), (8, 2), (250, 32)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_gradients_beside_any_neighbour(E, topk, score, renorm):
    """Even tokens are the same in both calls, with infinite and NaN gradients among
    them; odd ones name experts twice, hold NaN, or are ordinary."""
    need_gpu()
    say(f"router backward, neighbours E={E} topk={topk} {score} renorm={renorm}")
    g = torch.Generator(device=dev()).manual_seed(E)
    T = 4100
    x = 2 * torch.randn(T, E, generator=g, device=dev())
    ids = torch.rand((T, E), generator=g, device=dev()).argsort(dim=1)[:, :topk].int().contiguous()
    dw = torch.randn(T, topk, generator=g, device=dev())
    dw[::6, 0], dw[2::12, topk - 1] = float("inf"), float("nan")
    first = q.qlora_router_bwd(dw, x, ids, score, renorm, 2.5)
    ids[1::4, -1] = ids[1::4, 0]
    x[3::8, 0] = float("nan")
    dw[7::8] = float("inf")
    again = q.qlora_router_bwd(dw, x, ids, score, renorm, 2.5)
    torch.cuda.synchronize()
    even = slice(0, None, 2)
    np.testing.assert_array_equal(first[even].cpu().numpy(), again[even].cpu().numpy())
    assert torch.isfinite(first[4::12]).all() and torch.isnan(again[3::8]).all()
