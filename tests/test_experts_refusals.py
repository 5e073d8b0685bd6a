"""Refusals of the dropout, grouped and exchange calls: the C entry points'
argument checks (nothing is launched) and the binding's tensor checks (CPU)."""
import ctypes
import os

import pytest
import torch

import bit_quantized_fine_amd as q

pytestmark = pytest.mark.skipif(not os.path.exists(q.LIB_PATH),
                                reason="libqlora_nf4.so not built (run __graft_entry__.build())")

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)       # 8-byte, not 16-byte aligned
NULL, SHAPE, RANK, ALIGN, WORKSPACE, FORMAT, EXPERT, DROPOUT = 1, 2, 3, 4, 6, 8, 9, 10
BIG = 1 << 40


def drop(p, state=4096):
    return ctypes.byref(q._Dropout(state, p))


def weight(N=256, K=64, book=0, dq=1, codes=4096, aq=4096, sc=4096):
    return ctypes.byref(q._Q4Weight(codes, aq, sc, N, K, book, dq))


def test_dropout_apply():
    f = q.lib().qlora_dropout_apply
    assert f(P, 8, None, P, None) == NULL
    for p in (-0.1, 1.0, 1.5, float("nan"), float("inf")):
        assert f(P, 8, drop(p), P, None) == DROPOUT
    assert f(P, 8, drop(0.5, None), P, None) == NULL
    assert f(P, 8, drop(0.5, 4100), P, None) == ALIGN
    assert f(P, -1, drop(0.5), P, None) == SHAPE
    assert f(None, 8, drop(0.5), P, None) == NULL
    assert f(P, 8, drop(0.5), ODD, None) == ALIGN
    assert f(None, 0, drop(0.5), None, None) == 0


def fwd(X=P, M=16, w=None, A=P, B=P, r=8, d=None, Y=P, T=P, ws=P, wsb=BIG):
    return q.lib().qlora_linear_dropout_fwd(X, M, w or weight(), A, B, r, 1.0, d, Y, T, ws, wsb,
                                            None)


def bwd(dY=P, X=P, M=16, w=None, A=P, B=P, r=8, d=None, T=P, dX=P, dA=P, dB=P, ws=P, wsb=BIG):
    return q.lib().qlora_linear_dropout_bwd(dY, X, M, w or weight(), A, B, r, 1.0, d, T, dX, dA,
                                            dB, ws, wsb, None)


def test_linear_dropout():
    assert fwd(d=drop(1.0)) == DROPOUT and bwd(d=drop(-1.0)) == DROPOUT
    assert fwd(d=drop(0.5, None)) == NULL and bwd(d=drop(0.5, None)) == NULL
    assert fwd(X=None) == NULL and fwd(T=None) == NULL and bwd(dA=None) == NULL
    assert fwd(M=0) == SHAPE and fwd(w=weight(N=12)) == SHAPE and fwd(r=12) == RANK
    assert fwd(w=weight(book=3)) == FORMAT and bwd(w=weight(book=3)) == FORMAT
    assert fwd(A=ODD) == ALIGN and bwd(dX=ODD) == ALIGN
    need = q.lib().qlora_linear_dropout_fwd_workspace_bytes(16, 256, 64, 8)
    assert need > 0 and fwd(d=drop(0.5), wsb=need - 1) == WORKSPACE and fwd(ws=None) == WORKSPACE
    need = q.lib().qlora_linear_dropout_bwd_workspace_bytes(16, 256, 64, 8)
    assert need > 0 and bwd(d=drop(0.5), wsb=need - 1) == WORKSPACE


def gfwd(X=P, M=16, off=P, E=2, w=None, A=P, B=P, r=8, d=None, Y=P, T=P, ws=P, wsb=BIG):
    return q.lib().qlora_grouped_fwd(X, M, off, E, w or weight(512), A, B, r, 1.0, d, Y, T, ws,
                                     wsb, None)


def gbwd(dY=P, X=P, M=16, off=P, E=2, w=None, A=P, B=P, r=8, d=None, T=P, dX=P, dA=P, dB=P, ws=P,
         wsb=BIG):
    return q.lib().qlora_grouped_bwd(dY, X, M, off, E, w or weight(512), A, B, r, 1.0, d, T, dX,
                                     dA, dB, ws, wsb, None)


@pytest.mark.parametrize("call", [gfwd, gbwd])
def test_grouped(call):
    assert call(E=0) == EXPERT and call(E=1025, w=weight(256 * 1025)) == EXPERT
    assert call(E=3) == EXPERT                                  # 512 rows over 3
    assert call(E=2, w=weight(2 * 128)) == EXPERT               # half a group each
    assert call(E=2, w=weight(2 * 12, K=64, dq=0)) == SHAPE     # N % 8
    assert call(M=-1) == SHAPE and call(M=1 << 31) == SHAPE
    assert call(off=None) == NULL and call(X=None) == NULL and call(A=None) == NULL
    assert call(off=ctypes.c_void_p(4098)) == ALIGN and call(X=ODD) == ALIGN
    assert call(T=ODD) == ALIGN
    assert call(r=4) == RANK and call(r=264) == RANK
    assert call(d=drop(2.0)) == DROPOUT and call(d=drop(0.5, None)) == NULL
    assert call(w=weight(512, book=9)) == FORMAT and call(w=weight(512, K=100)) == SHAPE


def test_grouped_workspace_and_empty():
    L = q.lib()
    need = L.qlora_grouped_bwd_workspace_bytes(16, 2, 256, 64, 8)
    assert need >= 2 * 16 * 8 * 4 and gbwd(wsb=need - 1) == WORKSPACE
    assert gbwd(ws=None) == WORKSPACE
    need = L.qlora_grouped_fwd_workspace_bytes(16, 2, 256, 8192, 8)   # split reductions
    assert need > 0 and gfwd(w=weight(512, K=8192), wsb=need - 1) == WORKSPACE
    assert L.qlora_grouped_fwd_workspace_bytes(0, 2, 256, 64, 8) == 0
    assert L.qlora_grouped_fwd_workspace_bytes(16, 0, 256, 64, 8) == 0
    # no rows: nothing to do, and no buffers needed
    assert gfwd(X=None, M=0, Y=None, T=None, ws=None, wsb=0) == 0
    # grids past what a launch takes
    assert gfwd(M=(1 << 31) - 1, w=weight(1 << 22, K=64, dq=0), E=1) == SHAPE


def test_expert_plan():
    f, L = q.lib().qlora_expert_plan, q.lib()
    assert f(P, 8, 0, P, P, P, P, BIG, None) == EXPERT
    assert f(P, 8, 1025, P, P, P, P, BIG, None) == EXPERT
    assert f(P, -1, 4, P, P, P, P, BIG, None) == SHAPE
    assert f(P, (1 << 30) + 1, 4, P, P, P, P, BIG, None) == SHAPE
    assert f(None, 8, 4, P, P, P, P, BIG, None) == NULL
    assert f(P, 8, 4, None, P, P, P, BIG, None) == NULL
    assert f(P, 8, 4, ctypes.c_void_p(4097), P, P, P, BIG, None) == ALIGN
    need = L.qlora_expert_plan_workspace_bytes(1 << 20, 64)
    assert need > 0 and f(P, 1 << 20, 64, P, P, P, P, need - 1, None) == WORKSPACE
    assert L.qlora_expert_plan_workspace_bytes(16, 64) == 0


def test_expert_rows():
    L = q.lib()
    calls = [lambda **k: L.qlora_expert_gather(k.get("X", P), k.get("t", 4), k.get("j", 2),
                                               k.get("K", 64), k.get("i", P), P, None),
             lambda **k: L.qlora_expert_combine(k.get("X", P), k.get("t", 4), k.get("j", 2),
                                                k.get("K", 64), k.get("i", P), None, P, None),
             lambda **k: L.qlora_expert_combine_bwd(P, k.get("X", P), k.get("t", 4),
                                                    k.get("j", 2), k.get("K", 64), k.get("i", P),
                                                    P, P, P, None)]
    for f in calls:
        assert f(j=0) == EXPERT and f(j=65) == EXPERT
        assert f(K=12) == SHAPE and f(K=0) == SHAPE and f(t=-1) == SHAPE and f(t=1 << 30) == SHAPE
        assert f(X=None) == NULL and f(i=None) == NULL
        assert f(X=ODD) == ALIGN and f(i=ctypes.c_void_p(4098)) == ALIGN
        assert f(t=0, X=None, i=None) == 0
    assert L.qlora_expert_combine_bwd(P, P, 4, 2, 64, P, None, P, P, None) == NULL


def test_status_strings():
    for s in (EXPERT, DROPOUT):
        assert q.status_string(s) != "unknown status"
    assert q.status_string(11) == "unknown status"


def _w(N=256, K=64):
    return q.NF4Weight(torch.zeros(N * K // 2, dtype=torch.uint8),
                       torch.zeros(N * K // 64, dtype=torch.uint8),
                       torch.zeros((N * K // 64 + 255) // 256), N, K)


def test_binding_refusals():
    bf = dict(dtype=torch.bfloat16)
    X, A, B = torch.zeros(4, 64, **bf), torch.zeros(64, 8, **bf), torch.zeros(8, 256, **bf)
    st, off = torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="state is required"):
        q.qlora_dropout(X, 0.5, None)
    with pytest.raises(TypeError, match="int64"):
        q.qlora_dropout(X, 0.5, torch.zeros(2))
    with pytest.raises(ValueError, match="contiguous"):
        q.qlora_dropout(X.t(), 0.5, st)
    with pytest.raises(ValueError, match="GPU tensor"):
        q.qlora_dropout(X, 0.5, st)
    with pytest.raises(ValueError, match="B must have shape"):
        q.qlora_linear_dropout_fwd(X, _w(), A, torch.zeros(8, 248, **bf), 1.0, 0.5, st)
    with pytest.raises(ValueError, match="GPU tensor"):
        q.qlora_linear_dropout_bwd(torch.zeros(4, 256, **bf), X, _w(), A, B, 1.0, 0.5, st)
    with pytest.raises(ValueError, match="multiple of E"):
        q.qlora_grouped_fwd(X, off, _w(), 3)
    with pytest.raises(ValueError, match="offsets"):
        q.qlora_grouped_fwd(X, off, _w(512), 2)
    with pytest.raises(TypeError, match="int32"):
        q.qlora_grouped_fwd(X, off.long(), _w(), 1)
    with pytest.raises(ValueError, match="A must be"):
        q.qlora_grouped_fwd(X, off, _w(), 1, A, B)
    with pytest.raises(ValueError, match="together"):
        q.qlora_grouped_bwd(torch.zeros(4, 256, **bf), X, off, _w(), 1, A[None], None)
    with pytest.raises(ValueError, match="dY"):
        q.qlora_grouped_bwd(torch.zeros(4, 248, **bf), X, off, _w(), 1)
    with pytest.raises(TypeError, match="int32"):
        q.qlora_expert_plan(torch.zeros(4, 2, dtype=torch.int64), 4)
    inv = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="tokens, topk"):
        q.qlora_expert_gather(X, inv.reshape(-1))
    with pytest.raises(ValueError, match="X must have shape"):
        q.qlora_expert_gather(torch.zeros(5, 64, **bf), inv)
    with pytest.raises(ValueError, match="Y must have shape"):
        q.qlora_expert_combine(X, inv)
    with pytest.raises(ValueError, match="weights is required"):
        q.qlora_expert_combine_bwd(X, torch.zeros(8, 64, **bf), inv, None)
