"""The grouped calls under wrong offsets, on every path that the sizes choose (few
tokens, each tile height, split and whole reductions, both dX kernels): all outputs
and the workspace lie between guards that keep their bytes, and offsets that ascend
but leave [0, M] give the clamped offsets' results bit for bit."""
import pytest

import bit_quantized_fine_amd as q
from expert_util import Grouped
from gpu_util import dev, need_gpu, say, torch

pytestmark = pytest.mark.gpu

SHAPES = [
    # sizes, N, K, r, keywords
    ([5, 6, 4], 256, 1024, 16, {}),                        # up to 16 rows, T folded in
    ([20, 10, 10], 1024, 2048, 16, dict(p=0.2)),           # both reductions split
    ([20, 10, 10], 264, 320, 0, dict(dq=False)),
    ([300, 100, 140], 256, 1024, 72, {}),                  # 192 and 256 tokens a tile
    ([600, 500, 520], 64, 256, 8, dict(p=0.1)),            # adapter gradients split
    ([200, 150, 130], 8, 64 * 260, 8, dict(dq=False)),     # dX of many tiles
    ([200, 150, 130], 8, 64 * 260, 8, dict(dq=False, p=0.3)),
]
LOW, HIGH = -2 ** 31, 2 ** 31 - 1
OFFSETS = {   # of M rows
    "falling inside": lambda M: [0, M // 4, M // 10, M],
    "starting late": lambda M: [M // 2, M // 5, M // 5, M],
    "ending early": lambda M: [0, M, M // 3, M // 2],
    "out of range": lambda M: [-5, M // 4, 3 * M // 4, 5 * M],
    "all behind": lambda M: [M + 1, M + 9, 2 * M, HIGH],
    "all at the end": lambda M: [M, M, M, M],
    "falling": lambda M: [3 * M // 4, M // 2, M // 4, 0],
    "extreme": lambda M: [LOW, HIGH, LOW, HIGH],
    "extreme, rising": lambda M: [LOW, LOW, HIGH, HIGH],
}


class Guarded:
    """A tensor between two runs of bytes that must not change."""

    def __init__(self, shape, dtype):
        n = dtype.itemsize
        for s in shape:
            n *= s
        self.pad = max(1 << 16, (n + 255) // 256 * 256)
        self.end = self.pad + n
        self.buf = torch.full((self.end + self.pad,), 0x5A, dtype=torch.uint8, device=dev())
        self.t = self.buf[self.pad:self.end].view(dtype).view(shape)

    def intact(self):
        return bool((self.buf[:self.pad] == 0x5A).all() and (self.buf[self.end:] == 0x5A).all())


def _run(g, offsets):
    """Forward and backward between guards: the five outputs, and whether all
    guards kept their bytes."""
    off = torch.tensor(offsets, dtype=torch.int32, device=dev())
    bf, L = torch.bfloat16, q.lib()
    G = dict(Y=Guarded((g.M, g.N), bf), dX=Guarded((g.M, g.K), bf))
    if g.r:
        G.update(T=Guarded((g.M, g.r), torch.float32), dA=Guarded((g.E, g.K, g.r), bf),
                 dB=Guarded((g.E, g.r, g.N), bf))
    args = (g.M, g.E, g.N, g.K, g.r)
    for name, fn in (("wf", L.qlora_grouped_fwd_workspace_bytes),
                     ("wb", L.qlora_grouped_bwd_workspace_bytes)):
        G[name] = Guarded((fn(*args),), torch.uint8)
    t = {k: v.t for k, v in G.items()}
    q.qlora_grouped_fwd(g.X, off, g.w, g.E, Y=t["Y"], T=t.get("T"), workspace=t["wf"], **g.kw())
    q.qlora_grouped_bwd(g.dY, g.X, off, g.w, g.E, T=t.get("T"), dX=t["dX"], dA=t.get("dA"),
                        dB=t.get("dB"), workspace=t["wb"], **g.kw())
    torch.cuda.synchronize()
    broken = [k for k, v in G.items() if not v.intact()]
    return [t[k] for k in ("Y", "T", "dX", "dA", "dB") if k in t], broken


@pytest.mark.parametrize("kind", sorted(OFFSETS))
@pytest.mark.parametrize("sizes,N,K,r,kw", SHAPES)
def test_offsets(sizes, N, K, r, kw, kind):
    need_gpu()
    g = Grouped(sizes, N, K, r, seed=N + K + r, **kw)
    off = OFFSETS[kind](g.M)
    say(f"offsets {off}: sizes={sizes} N={N} K={K} r={r} {kw}")
    got, broken = _run(g, off)
    assert broken == []
    clamped = [min(max(v, 0), g.M) for v in off]
    if clamped == sorted(clamped):
        want, _ = _run(g, clamped)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
