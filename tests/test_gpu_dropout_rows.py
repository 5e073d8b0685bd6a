"""The layer with adapter dropout over more rows than 65536 tiles of 128 tokens."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
from expert_util import OFFSET, SEED, Grouped, within
from gpu_util import bits, dev, need_gpu, say, torch
from oracle import bf16_bits_to_f64, codebooks as cb
from oracle import dropout as od
from oracle import experts as ox

pytestmark = pytest.mark.gpu


def test_more_than_2_to_the_23_rows():
    """2^23 + 200 rows; the rows around the 65536th tile and the last ones against
    the oracle on those rows alone.  The gradient rows are zero elsewhere, so that dA
    and dB depend on those alone as well."""
    need_gpu()
    M, N, K, r, s, p = 2 ** 23 + 200, 8, 64, 8, 0.25, 0.25
    say(f"layer with dropout M={M}")
    g = Grouped([1], N, K, r, s=s, p=p, dq=False, seed=4)   # weight and adapters
    gen = torch.Generator(device=dev())
    gen.manual_seed(6)
    X = torch.randn((M, K), generator=gen, device=dev()).bfloat16()
    rows = slice(2 ** 23 - 60, M)
    dY = torch.zeros((M, N), dtype=torch.bfloat16, device=dev())
    dY[rows] = torch.randn((M - rows.start, N), generator=gen, device=dev()).bfloat16()
    A, B = g.A[0], g.B[0]
    Y, T = q.qlora_linear_dropout_fwd(X, g.w, A, B, s, p, g.state)
    dX, dA, dB = q.qlora_linear_dropout_bwd(dY, X, g.w, A, B, s, p, g.state, T=T)
    torch.cuda.synchronize()
    f = bf16_bits_to_f64
    W = f(cb.dequantize_q4(g.w.codes.cpu().numpy(), None, g.w.absmax_scale.cpu().numpy(), N, K,
                           "nf4", False)).reshape(N, K)
    n = M - rows.start
    D = od.halves(n * K, SEED, OFFSET, rows.start * K).reshape(n, K) >= od.threshold(p)
    args = (f(bits(X[rows])), [0, n], [W], [f(bits(A))], [f(bits(B))], s, D, od.scale(p))
    y, t = ox.grouped_fwd(*args)
    fdY = f(bits(dY[rows]))
    dx, da, db = ox.grouped_bwd(fdY, *args)
    b = ox.grouped_bounds(fdY, *args)
    within("Y", Y[rows], y, b["Y"])
    within("T", T[rows], t, b["T"])
    within("dX", dX[rows], dx, b["dX"])
    within("dA", dA, da[0], b["dA"][0])
    within("dB", dB, db[0], b["dB"][0])
    assert not dX[:rows.start].any()
    # rows in front, by the formula in 64 bits on the first thousand
    m = 1000
    D0 = od.halves(m * K, SEED, OFFSET, 0).reshape(m, K) >= od.threshold(p)
    a0 = (f(bits(X[:m])), [0, m], [W], [f(bits(A))], [f(bits(B))], s, D0, od.scale(p))
    y0, t0 = ox.grouped_fwd(*a0)
    b0 = ox.grouped_bounds(np.zeros((m, N)), *a0)
    within("Y, first rows", Y[:m], y0, b0["Y"])
    within("T, first rows", T[:m], t0, b0["T"])
