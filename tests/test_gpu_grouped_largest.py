"""The grouped calls on the largest weight that the interface takes, 2^32 weights (2 GB
of codes, so that buffer offsets reach 2^31): sampled output columns of the first and
the last expert against the dequantized rows in 64 bits, on every path."""
import pytest

import bit_quantized_fine_amd as q
from gpu_util import dev, need_gpu, say, torch

pytestmark = pytest.mark.gpu

E, N, K, R, S = 4, 32768, 32768, 16, 0.25
U, HALF, SPLIT = 2.0 ** -24, 2.0 ** -8, 2.0 ** -16   # fp32, bf16, two bf16 halves


@pytest.fixture(scope="module")
def model():
    need_gpu()
    gen = torch.Generator(device=dev())
    gen.manual_seed(11)
    nb = E * N * K // 64
    codes = torch.randint(0, 256, (E * N * K // 2,), generator=gen, device=dev(), dtype=torch.uint8)
    absmax_q = torch.randint(100, 256, (nb,), generator=gen, device=dev(), dtype=torch.uint8)
    scale = 0.065 / 255 * (0.9 + 0.2 * torch.rand(nb // 256, generator=gen, device=dev()))
    w = q.Q4Weight(codes, absmax_q, scale, E * N, K, "nf4", True)
    A = (torch.randn((E, K, R), generator=gen, device=dev()) / R).bfloat16()
    B = (torch.randn((E, R, N), generator=gen, device=dev()) * 0.1).bfloat16()
    yield gen, w, A, B
    del codes, absmax_q, scale, w, A, B
    torch.cuda.empty_cache()


def _rows64(w, rows):
    """Rows of the stacked weight in 64 bits (values rounded to bf16 as defined)."""
    c = w.codes.view(E * N, K // 2)[rows].int()
    lv = torch.as_tensor(q.qlora_nf4_levels(), dtype=torch.float32, device=dev())
    v = torch.stack([lv[(c & 15).long()], lv[(c >> 4).long()]], dim=2).reshape(len(rows), K)
    blocks = rows[:, None] * (K // 64) + torch.arange(K // 64, device=dev())
    ch = w.absmax_q[blocks].float() * w.absmax_scale[blocks // 256]
    return (v * ch.repeat_interleave(64, dim=1)).bfloat16().double()


# one row: dX by the kernel of few tiles; from two rows on by that of many
@pytest.mark.parametrize("sizes", [[0, 0, 0, 1], [3, 0, 0, 5], [20, 0, 0, 30], [40, 0, 0, 90],
                                   [200, 1, 0, 260]])
def test_largest_weight(model, sizes):
    say(f"2^32 weights, sizes={sizes}")
    gen, w, A, B = model
    M = sum(sizes)
    ends = [0]
    for m in sizes:
        ends.append(ends[-1] + m)
    off = torch.tensor(ends, dtype=torch.int32, device=dev())
    X = torch.randn((M, K), generator=gen, device=dev()).bfloat16()
    cols = torch.cat([torch.arange(4), torch.randint(0, N, (24,)), torch.arange(N - 4, N)]).to(dev())
    cols = cols.unique()
    dY = torch.zeros((M, N), dtype=torch.bfloat16, device=dev())
    dY[:, cols] = torch.randn((M, len(cols)), generator=gen, device=dev()).bfloat16()
    Y, T = q.qlora_grouped_fwd(X, off, w, E, A, B, S)
    dX, dA, dB = q.qlora_grouped_bwd(dY, X, off, w, E, A, B, S, T=T)
    torch.cuda.synchronize()
    n = lambda k: (k + 8) * U
    for e in (0, E - 1):
        rows = slice(ends[e], ends[e + 1])
        if sizes[e] == 0:
            assert not dA[e].any() and not dB[e].any()
            continue
        W, x = _rows64(w, e * N + cols), X[rows].double()
        a, b, g = A[e].double(), B[e][:, cols].double(), dY[rows][:, cols].double()
        t, mT = x @ a, x.abs() @ a.abs()
        eT = n(K) * mT
        assert ((T[rows].double() - t).abs() <= eT).all()
        y = x @ W.T + S * (t @ b)
        bound = (HALF * y.abs() + (1 + HALF) * (n(K + 2 * R) * (x.abs() @ W.abs().T + S * (mT @ b.abs()))
                                                + S * ((eT + SPLIT * t.abs()) @ b.abs())))
        assert ((Y[rows][:, cols].double() - y).abs() <= bound).all()
        G, mG = g @ b.T, g.abs() @ b.abs().T
        eG = n(N) * mG + SPLIT * G.abs()
        dx = g @ W + S * (G @ a.T)
        bound = (HALF * dx.abs() + (1 + HALF) * (n(N + 2 * R) * (g.abs() @ W.abs() + S * (mG @ a.abs().T))
                                                 + S * (eG @ a.abs().T)))
        assert ((dX[rows].double() - dx).abs() <= bound).all()
        m = sizes[e]
        da, db = S * (x.T @ G), S * (t.T @ g)
        bound = HALF * da.abs() + (1 + HALF) * S * (n(2 * m) * (x.abs().T @ mG) + x.abs().T @ eG)
        assert ((dA[e].double() - da).abs() <= bound).all()
        bound = HALF * db.abs() + (1 + HALF) * S * (n(2 * m) * (mT.T @ g.abs())
                                                    + (eT + SPLIT * t.abs()).T @ g.abs())
        assert ((dB[e][:, cols].double() - db).abs() <= bound).all()
        rest = torch.ones(N, dtype=torch.bool, device=dev())
        rest[cols] = False
        assert not dB[e][:, rest].any()
