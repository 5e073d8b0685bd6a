"""The grouped backward from a checkpoint of rows that lie in expert order already (no
order given): dX, dA and dB bit for bit those of the bf16 call on the unpacked rows,
and within the bounds of a float64 evaluation."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
import oracle
from expert_util import OFFSET, SEED, state, within
from gpu_util import bits, dev, need_gpu, say, torch
from oracle import experts as ox

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,N,K,r,p,before,behind", [
    ([1], 64, 64, 8, 0.0, 0, 0), ([5, 0, 3], 256, 320, 16, 0.0, 2, 1), ([0, 0, 70], 64, 1024, 72, 0.2, 3, 9),
    ([200, 1, 64, 63, 65], 128, 512, 64, 0.0, 1, 40), ([0, 0], 256, 192, 8, 0.0, 0, 20),
    ([700, 300], 64, 256, 256, 0.5, 65, 7), ([17] * 30, 8, 64, 8, 0.0, 0, 3),
    ([900, 0, 1100], 256, 2048, 32, 0.0, 5, 0), ([33, 90], 512, 128, 0, 0.0, 4, 4)])
def test_rows_in_expert_order(sizes, N, K, r, p, before, behind):
    need_gpu()
    E = len(sizes)
    say(f"grouped act8 bwd, no order: E={E} rows={sum(sizes)} N={N} K={K} r={r} p={p}")
    g = torch.Generator(device=dev()).manual_seed(sum(sizes) + K)
    rand = lambda *s: torch.randn(s, generator=g, device=dev())
    M = before + sum(sizes) + behind
    ends = before + np.concatenate([[0], np.cumsum(sizes)])
    rows = slice(before, before + sum(sizes))
    offsets = torch.tensor(ends, dtype=torch.int32, device=dev())
    w = q.qlora_q4_quantize(rand(E * N, K) * 0.02, "nf4", False)
    # rows of many magnitudes, so that another row's constant shows
    X = (rand(M, K) * torch.exp2(torch.randint(-6, 7, (M, 1), generator=g, device=dev()))).bfloat16()
    X[:before], X[rows.stop:] = float("nan"), float("nan")     # where nobody may look
    x8 = q.qlora_act8_pack(X)
    Xr = q.qlora_act8_unpack(x8)
    dY = rand(M, N).bfloat16()
    kw = dict(s=0.5, p=p, state=state())
    if r:
        kw.update(A=rand(E, K, r).bfloat16(), B=rand(E, r, N).bfloat16())
    full = lambda: torch.full((M, K), 7.0, dtype=torch.bfloat16, device=dev())
    Ts = [None]
    if r:
        Ts.append(q.qlora_grouped_fwd(Xr, offsets, w, E, **kw)[1])
    for T in Ts:
        want = q.qlora_grouped_bwd(dY, Xr, offsets, w, E, T=T, dX=full(), **kw)
        got = q.qlora_grouped_act8_bwd(dY, x8, offsets, w, E, T=T, dX=full(), **kw)
        again = q.qlora_grouped_act8_bwd(dY, x8, offsets, w, E, T=T, dX=full(), **kw)
        torch.cuda.synchronize()
        for name, a, b, c in zip(("dX", "dA", "dB"), got, want, again):
            assert (a is None and b is None) or (torch.equal(a, b) and torch.equal(a, c)), name
        assert (got[0][:before] == 7).all() and (got[0][rows.stop:] == 7).all()
        f = oracle.bf16_bits_to_f64
        fX, fdY = f(bits(Xr)), f(bits(dY))
        fX[:before], fX[rows.stop:] = 0, 0
        W = f(bits(q.qlora_q4_dequantize(w))).reshape(E, N, K)
        D = oracle.dropout.keep((M, K), p, SEED, OFFSET) if p else None
        A, B = (f(bits(kw["A"])), f(bits(kw["B"]))) if r else (np.zeros((E, K, 0)), np.zeros((E, 0, N)))
        args = (fX, ends, list(W), list(A), list(B), 0.5, D,
                65536 / (65536 - oracle.dropout.threshold(p)))
        dX, dA, dB = ox.grouped_bwd(fdY, *args)
        bound = ox.grouped_bounds(fdY, *args)
        within("dX", got[0][rows], dX[rows], bound["dX"][rows])
        if r:
            within("dA", got[1], dA, bound["dA"])
            within("dB", got[2], dB, bound["dB"])


def test_constants_and_codes_change_the_gradient():
    """One row's constant or code changed: dA changes in that row's columns, on its expert
    alone, and nothing else does."""
    need_gpu()
    say("grouped act8 bwd, no order: one block at a time")
    E, N, K, r = 3, 64, 192, 8
    g = torch.Generator(device=dev()).manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g, device=dev())
    offsets = torch.tensor([2, 72, 72, 140], dtype=torch.int32, device=dev())
    w = q.qlora_q4_quantize(rand(E * N, K) * 0.02, "nf4", False)
    x8, dY, T = q.qlora_act8_pack(rand(150, K).bfloat16()), rand(150, N).bfloat16(), rand(150, r)
    A, B = rand(E, K, r).bfloat16(), rand(E, r, N).bfloat16()
    call = lambda x: q.qlora_grouped_act8_bwd(dY, x, offsets, w, E, A, B, T=T)[1]
    first = call(x8)
    for row, block, e in ((2, 0, 0), (71, 2, 0), (72, 1, 2), (139, 2, 2), (1, 1, None), (140, 0, None)):
        more = q.Act8(x8.codes.clone(), x8.scales.clone())
        more.scales[row, block] *= 32
        dA = call(more)
        torch.cuda.synchronize()
        same = dA == first
        if e is not None:
            inside = same[e, 64 * block:64 * block + 64]
            assert inside.float().mean() < 0.2
            same[e, 64 * block:64 * block + 64] = True
        assert same.all(), (row, block)
