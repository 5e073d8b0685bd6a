"""dX of few tokens runs in tiles of 64 or 128 tokens where more take 256: the same
sums in the same order, so a token's row is bit for bit that of a larger call."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import state
from gpu_util import dev, need_gpu, say, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,r", [(1000, 1088, 16), (1024, 1024, 64), (64, 4096, 8), (4096, 320, 0)])
@pytest.mark.parametrize("book,dq", [("nf4", True), ("int4", False)])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_rows_of_a_larger_call(N, K, r, book, dq, p):
    """200 rows (one tile of 256), and the first 1, 64, 65 and 128 of them.  dY and B are
    small integers, so that G = dY B^T is exact however its sum is split."""
    need_gpu()
    if r == 0 and p > 0:
        pytest.skip("dropout needs an adapter")
    say(f"dX of few rows N={N} K={K} r={r} {book} dq={dq} p={p}")
    g = torch.Generator(device=dev()).manual_seed(N + K)
    ints = lambda *shape: torch.randint(-2, 3, shape, generator=g, device=dev()).bfloat16()
    w = q.qlora_q4_quantize(torch.randn(N, K, generator=g, device=dev()) / K ** 0.5, book, dq)
    A = (torch.randn(K, r, generator=g, device=dev()) / 8).bfloat16() if r else None
    B = ints(r, N) if r else None
    dY, X = ints(200, N), ints(200, K)
    T = torch.zeros(200, r, device=dev()) if r else None
    kw = dict(p=p, state=state(7, 11) if p else None)

    def dx(m, act8=False):
        t = T[:m] if r else None
        if act8:
            return q.qlora_linear_act8_bwd(dY[:m], q.qlora_act8_pack(X[:m]), w, A, B, 0.25, T=t, **kw)[0]
        return q.qlora_linear_dropout_bwd(dY[:m], X[:m], w, A, B, 0.25, T=t, **kw)[0]
    whole = dx(200)
    for m in (1, 63, 64, 65, 100, 128, 129):
        for act8 in (False, True):
            got = dx(m, act8)
            torch.cuda.synchronize()
            np.testing.assert_array_equal(got.view(torch.int16).cpu().numpy(),
                                          whole[:m].view(torch.int16).cpu().numpy())


@pytest.mark.parametrize("N,K,r", [(1000, 1088, 16), (64, 4096, 8)])
def test_rows_of_a_larger_call_16_bit(N, K, r):
    """The same over a bf16 weight."""
    need_gpu()
    say(f"dX of few rows, bf16 weight N={N} K={K} r={r}")
    g = torch.Generator(device=dev()).manual_seed(N + K)
    ints = lambda *shape: torch.randint(-2, 3, shape, generator=g, device=dev()).bfloat16()
    W = (torch.randn(N, K, generator=g, device=dev()) / K ** 0.5).bfloat16()
    A, B = (torch.randn(K, r, generator=g, device=dev()) / 8).bfloat16(), ints(r, N)
    dY, X, T = ints(200, N), ints(200, K), torch.zeros(200, r, device=dev())
    whole = q.qlora_lora16_bwd(dY, X, W, A, B, 0.25, T=T)[0]
    for m in (1, 64, 65, 128, 129):
        got = q.qlora_lora16_bwd(dY[:m], X[:m], W, A, B, 0.25, T=T[:m])[0]
        torch.cuda.synchronize()
        np.testing.assert_array_equal(got.view(torch.int16).cpu().numpy(),
                                      whole[:m].view(torch.int16).cpu().numpy())
