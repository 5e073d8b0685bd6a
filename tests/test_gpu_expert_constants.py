"""Block constants of one expert that are not finite (or too large for bf16) and
the other experts' results: no kernel behind the grouped calls may let them
through, whichever the sizes choose.  An expert whose rows are no multiple of
64 shares its last chunk of weight rows with its neighbour in the kernels of few
tiles, with and without a split reduction."""
import pytest

from expert_util import Grouped
from gpu_util import need_gpu, say, torch

pytestmark = pytest.mark.gpu

CASES = [
    # sizes, N, K, r, keywords
    ([20, 11, 30], 72, 1024, 16, dict(dq=False)),
    ([20, 11, 30], 200, 320, 16, dict(dq=False, p=0.2)),
    ([3, 5, 2], 72, 2048, 8, {}),                          # 8-bit constants
    ([70, 100, 60], 72, 2048, 8, dict(p=0.3)),
    ([300, 140, 129], 40, 256, 24, dict(dq=False)),        # all token heights
    ([9, 30, 20], 1000, 256, 16, dict(dq=False)),          # split reduction
    ([130, 30, 260], 1032, 320, 0, dict(dq=False)),
    ([40, 8, 66], 1096, 2048, 8, dict(p=0.1)),
]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3.4e38])
@pytest.mark.parametrize("sizes,N,K,r,kw", CASES)
def test_constants_stay_with_their_expert(sizes, N, K, r, kw, bad):
    need_gpu()
    say(f"constants {bad}: sizes={sizes} N={N} K={K} r={r} {kw}")
    g = Grouped(sizes, N, K, r, seed=N + K, **kw)
    want = g.check()
    per = N * K // (64 * 256 if g.w.double_quant else 64)
    g.w.absmax_scale[per:2 * per] = bad
    Y, T = g.fwd()
    got = (Y, T) + g.bwd(want[1])
    torch.cuda.synchronize()
    own = slice(int(g.off[1]), int(g.off[2]))
    for name, a, b in zip(("Y", "T", "dX"), want, got):
        if a is not None:
            assert torch.equal(a[:own.start], b[:own.start]), name
            assert torch.equal(a[own.stop:], b[own.stop:]), name
    for name, a, b in zip(("dA", "dB"), want[3:], got[3:]):   # no weight in them
        assert a is None or torch.equal(a, b), name
    if bad != bad:
        assert torch.isnan(Y[own]).all() and torch.isnan(got[2][own]).all()
