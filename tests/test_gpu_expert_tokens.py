"""The exchange over more tokens than one launch has workgroups for."""
import pytest

import bit_quantized_fine_amd as q
from gpu_util import dev, need_gpu, say, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,topk", [(2 ** 24 + 3, 1), (2 ** 23 + 1, 2)])
def test_many_tokens(tokens, topk):
    """Rows of eight values there and back, a sixth of the slots without a row;
    moved bits are equal, sums within their roundings."""
    need_gpu()
    say(f"exchange tokens={tokens} topk={topk}")
    K, E, n = 8, 5, tokens * topk
    gen = torch.Generator(device=dev())
    gen.manual_seed(tokens)
    draw = lambda *s: torch.randn(s, generator=gen, device=dev()).bfloat16()
    ids = torch.randint(-1, E, (tokens, topk), generator=gen, device=dev(), dtype=torch.int32)
    X, Y, dOut = draw(tokens, K), draw(n, K), draw(tokens, K)
    w = torch.rand((tokens, topk), generator=gen, device=dev())
    off, order, inv = q.qlora_expert_plan(ids, E)
    Xs = q.qlora_expert_gather(X, inv, out=torch.full((n, K), 7.0, dtype=torch.bfloat16,
                                                      device=dev()))
    out = q.qlora_expert_combine(Y, inv, w)
    dY, dw = q.qlora_expert_combine_bwd(dOut, Y, inv, w,
                                        dY=torch.full_like(Y, 7.0))
    torch.cuda.synchronize()

    flat = torch.where(ids < 0, E, ids).reshape(-1)
    key, slot = torch.sort(flat, stable=True)
    kept = int((key < E).sum())
    assert int(off[E]) == kept and 0 < kept < n
    assert torch.equal(order[:kept].long(), slot[:kept]) and (order[kept:] == -1).all()
    token = slot[:kept] // topk
    assert torch.equal(Xs[:kept], X[token]) and (Xs[kept:] == 7).all()
    live = inv >= 0
    rows = inv.clamp(min=0).long()
    ww = torch.where(live, w, torch.zeros_like(w))
    ref = sum(ww[:, j, None].double() * Y[rows[:, j]].double() for j in range(topk))
    mag = sum((ww[:, j, None] * Y[rows[:, j]]).abs().double() for j in range(topk))
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1.01 * topk * 2.0 ** -24 * mag).all()
    want = w.reshape(-1)[slot[:kept], None].double() * dOut[token].double()
    assert ((dY[:kept].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs()).all()
    assert (dY[kept:] == 7).all()
    for j in range(topk):
        prod = dOut.double() * Y[rows[:, j]].double()
        ref = torch.where(live[:, j], prod.sum(1), torch.zeros((), device=dev(), dtype=torch.float64))
        err = (dw[:, j].double() - ref).abs()
        assert (err <= 1.01 * (K + 16) * 2.0 ** -24 * prod.abs().sum(1)).all()
        assert (dw[:, j][~live[:, j]] == 0).all()
