"""Refusals of the norm, the 8-bit checkpoints, the backward passes from them and
the router: the C entry points' argument checks (nothing is launched) and the
binding's tensor checks (CPU)."""
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


def x8(codes=4096, scales=4096):
    return ctypes.byref(q._Act8(codes, scales))


def weight(N=256, K=64, book=0, dq=1):
    return ctypes.byref(q._Q4Weight(4096, 4096, 4096, N, K, book, dq))


def drop(p, state=4096):
    return ctypes.byref(q._Dropout(state, p))


def test_act8():
    L = q.lib()
    pack = lambda X=P, M=4, K=64, c=None: L.qlora_act8_pack(X, M, K, c or x8(), None)
    unpack = lambda X=P, M=4, K=64, c=None: L.qlora_act8_unpack(c or x8(), M, K, X, None)
    for f in (pack, unpack):
        assert f(K=32) == SHAPE and f(K=96) == SHAPE and f(K=0) == SHAPE and f(M=-1) == SHAPE
        assert f(K=(1 << 22) + 64) == SHAPE and f(M=(1 << 34) + 1) == SHAPE
        assert f(X=None) == NULL and f(c=x8(None)) == NULL and f(c=x8(4096, None)) == NULL
        assert f(X=ODD) == ALIGN and f(c=x8(4104)) == ALIGN and f(c=x8(4096, 4098)) == ALIGN
        assert f(M=0, X=None, c=x8(None, None)) == 0
    assert L.qlora_act8_pack(P, 4, 64, None, None) == NULL
    assert L.qlora_act8_unpack(None, 4, 64, P, None) == NULL


def lin(dY=P, c=None, M=16, w=None, A=P, B=P, r=8, d=None, T=P, dX=P, dA=P, dB=P, ws=P, wsb=BIG):
    return q.lib().qlora_linear_act8_bwd(dY, c or x8(), M, w or weight(), A, B, r, 1.0, d, T, dX,
                                         dA, dB, ws, wsb, None)


def grp(dY=P, c=None, tokens=8, order=P, topk=2, M=16, off=P, E=2, w=None, A=P, B=P, r=8, d=None,
        T=P, dX=P, dA=P, dB=P, ws=P, wsb=BIG):
    return q.lib().qlora_grouped_act8_bwd(dY, c or x8(), tokens, order, topk, M, off, E,
                                          w or weight(512), A, B, r, 1.0, d, T, dX, dA, dB, ws,
                                          wsb, None)


def test_backward_from_a_checkpoint():
    for f, n in ((lin, 256), (grp, 512)):
        assert f(c=x8(None)) == NULL and f(c=x8(4096, None)) == NULL and f(dY=None) == NULL
        assert f(c=x8(4104)) == ALIGN and f(c=x8(4096, 4098)) == ALIGN and f(dA=ODD) == ALIGN
        assert f(dA=None) == NULL and f(A=None) == NULL and f(r=12) == RANK
        assert f(w=weight(n, K=100)) == SHAPE and f(w=weight(n, book=5)) == FORMAT
        assert f(M=-1) == SHAPE and f(d=drop(1.0)) == DROPOUT and f(d=drop(0.5, None)) == NULL
    assert lin(M=0) == SHAPE
    assert q.lib().qlora_linear_act8_bwd(P, None, 16, weight(), P, P, 8, 1.0, None, P, P, P, P, P,
                                         BIG, None) == NULL
    assert grp(topk=0) == EXPERT and grp(topk=65) == EXPERT and grp(E=3) == EXPERT
    assert grp(order=ctypes.c_void_p(4098)) == ALIGN and grp(tokens=-1) == SHAPE
    assert grp(order=None, tokens=8, M=16) == SHAPE        # rows as they are: one each
    assert grp(tokens=1 << 31) == SHAPE and grp(off=None) == NULL
    L = q.lib()
    need = L.qlora_linear_act8_bwd_workspace_bytes(16, 256, 64, 8)
    assert need > 0 and lin(wsb=need - 1) == WORKSPACE and lin(ws=None) == WORKSPACE
    need = L.qlora_grouped_act8_bwd_workspace_bytes(16, 2, 256, 64, 8)
    assert need > 0 and grp(wsb=need - 1) == WORKSPACE
    # dA's launch would hold 2^32 threads: 2^16 tiles of 64 columns, 4 of ranks, 64 experts
    big = weight(64 * 8, 1 << 22, dq=0)
    assert grp(w=big, E=64, r=256) == SHAPE


def nf(x=P, res=P, g=P, g32=1, M=4, K=64, eps=1e-5, h=P, y=P, rstd=P, c=None):
    return q.lib().qlora_rms_norm_fwd(x, res, g, g32, M, K, eps, h, y, rstd, c, None)


def nb(dy=P, dres=P, h=P, rstd=P, g=P, g32=1, M=4, K=64, dx=P, dg=P, ws=P, wsb=BIG):
    return q.lib().qlora_rms_norm_bwd(dy, dres, h, rstd, g, g32, M, K, dx, dg, ws, wsb, None)


def test_norm():
    for f in (nf, nb):
        assert f(K=12) == SHAPE and f(K=0) == SHAPE and f(M=-1) == SHAPE
        assert f(K=(1 << 22) + 8) == SHAPE and f(M=(1 << 37) + 1, K=8) == SHAPE
        assert f(g=None) == NULL and f(h=None) == NULL and f(rstd=None) == NULL
        assert f(g=ODD) == ALIGN and f(h=ODD) == ALIGN and f(rstd=ctypes.c_void_p(4098)) == ALIGN
    assert nf(x=None) == NULL and nf(y=None) == NULL and nf(x=ODD) == ALIGN and nf(y=ODD) == ALIGN
    assert nf(res=ODD) == ALIGN
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert nf(eps=eps) == SHAPE
    assert nf(c=x8(), K=72) == SHAPE and nf(c=x8(None)) == NULL and nf(c=x8(4104)) == ALIGN
    assert nf(M=0, x=None, y=None, h=None, rstd=None) == 0
    assert nb(dy=None) == NULL and nb(dx=None) == NULL
    assert nb(dy=ODD) == ALIGN and nb(dres=ODD) == ALIGN and nb(dx=ODD) == ALIGN and nb(dg=ODD) == ALIGN
    assert nb(M=0, dy=None, h=None, rstd=None, dx=None, dg=None) == 0
    need = q.lib().qlora_rms_norm_bwd_workspace_bytes(4096, 8192)
    assert need > 0 and nb(M=4096, K=8192, wsb=need - 1) == WORKSPACE
    assert nb(M=4096, K=8192, ws=None) == WORKSPACE and nb(M=4096, K=8192, ws=ODD) == ALIGN
    assert q.lib().qlora_rms_norm_bwd_workspace_bytes(4, 12) == 0
    assert q.lib().qlora_rms_norm_bwd_workspace_bytes(0, 64) == 0


def cfg(score=0, topk=2, groups=1, top_groups=1, group_top=1, renorm=1, scale=1.0):
    return ctypes.byref(q._RouterConfig(score, topk, groups, top_groups, group_top, renorm, scale))


def rf(logits=P, tokens=4, E=8, bias=P, c=None, ids=P, weights=P):
    return q.lib().qlora_router_fwd(logits, 1, tokens, E, bias, c or cfg(), ids, weights, None)


def rb(logits=P, tokens=4, E=8, c=None, ids=P, weights=P, dlogits=P):
    return q.lib().qlora_router_bwd(weights, logits, 1, ids, tokens, E, c or cfg(), dlogits, None)


def test_router():
    for f in (rf, rb):
        assert f(E=0) == EXPERT and f(E=1025) == EXPERT
        for bad in (cfg(score=2), cfg(score=-1), cfg(topk=0), cfg(topk=65), cfg(topk=9),
                    cfg(groups=0), cfg(groups=3), cfg(groups=65), cfg(top_groups=0),
                    cfg(top_groups=2), cfg(group_top=0), cfg(group_top=3), cfg(renorm=2),
                    cfg(scale=float("inf")), cfg(scale=float("nan")),
                    cfg(topk=3, groups=4, top_groups=1)):
            assert f(c=bad) == EXPERT
        assert f(tokens=-1) == SHAPE and f(tokens=(1 << 29) + 1) == SHAPE
        assert f(logits=None) == NULL and f(ids=None) == NULL and f(weights=None) == NULL
        assert f(logits=ctypes.c_void_p(4098)) == ALIGN and f(ids=ctypes.c_void_p(4098)) == ALIGN
        assert f(tokens=0, logits=None, ids=None, weights=None) == 0
    assert rf(bias=ctypes.c_void_p(4098)) == ALIGN
    assert rb(dlogits=None) == NULL and rb(dlogits=ctypes.c_void_p(4098)) == ALIGN
    for f, args in ((q.lib().qlora_router_fwd, lambda p: (p, 0, 4, 8, None, cfg(), P, P, None)),
                    (q.lib().qlora_router_bwd, lambda p: (P, p, 0, P, 4, 8, cfg(), P, None))):
        assert f(*args(ctypes.c_void_p(4097))) == ALIGN
    L = q.lib()
    assert L.qlora_router_fwd(P, 1, 4, 8, None, None, P, P, None) == NULL
    assert L.qlora_router_bwd(P, P, 1, P, 4, 8, None, P, None) == NULL


def _w(N=256, K=64):
    return q.NF4Weight(torch.zeros(N * K // 2, dtype=torch.uint8),
                       torch.zeros(N * K // 64, dtype=torch.uint8),
                       torch.zeros((N * K // 64 + 255) // 256), N, K)


def test_binding_refusals():
    bf = dict(dtype=torch.bfloat16)
    X, g = torch.zeros(4, 64, **bf), torch.ones(64)
    c8 = q.Act8(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1))
    with pytest.raises(ValueError, match="multiple of 64"):
        q.qlora_act8_pack(torch.zeros(4, 72, **bf))
    with pytest.raises(TypeError, match="bfloat16"):
        q.qlora_act8_pack(X.float())
    with pytest.raises(ValueError, match="two-dimensional"):
        q.qlora_act8_pack(X[0])
    with pytest.raises(ValueError, match="contiguous"):
        q.qlora_act8_pack(torch.zeros(64, 64, **bf).t())
    with pytest.raises(ValueError, match="GPU tensor"):
        q.qlora_act8_pack(X)
    with pytest.raises(ValueError, match="out.codes must have shape"):
        q.qlora_act8_pack(torch.zeros(5, 64, **bf), c8)
    with pytest.raises(TypeError, match="x8.codes"):
        q.qlora_act8_unpack(c8._replace(codes=c8.codes.view(torch.uint8)))
    with pytest.raises(ValueError, match="x8.scales"):
        q.qlora_act8_unpack(c8._replace(scales=torch.zeros(4, 2)))
    with pytest.raises(ValueError, match="x8 is required"):
        q.qlora_act8_unpack(None)
    dY, off = torch.zeros(4, 256, **bf), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="dY must have shape"):
        q.qlora_linear_act8_bwd(dY[:3], c8, _w())
    with pytest.raises(ValueError, match="x8.codes must have shape"):
        q.qlora_linear_act8_bwd(dY, c8, _w(128, 128))
    with pytest.raises(ValueError, match="state is required"):
        q.qlora_linear_act8_bwd(dY, c8, _w(), p=0.5)
    with pytest.raises(ValueError, match="GPU tensor"):
        q.qlora_linear_act8_bwd(dY, c8, _w())
    with pytest.raises(ValueError, match="x8.codes must have shape"):
        q.qlora_grouped_act8_bwd(torch.zeros(8, 256, **bf), c8, off, _w(), 1)
    with pytest.raises(TypeError, match="order"):
        q.qlora_grouped_act8_bwd(dY, c8, off, _w(), 1, order=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="order"):
        q.qlora_grouped_act8_bwd(dY, c8, off, _w(), 1, order=torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError, match="offsets"):
        q.qlora_grouped_act8_bwd(dY, c8, off, _w(512), 2)
    with pytest.raises(TypeError, match="g must be"):
        q.qlora_rms_norm_fwd(X, g.double())
    with pytest.raises(ValueError, match="g must have shape"):
        q.qlora_rms_norm_fwd(X, g[:32])
    with pytest.raises(ValueError, match="residual"):
        q.qlora_rms_norm_fwd(X, g, X[:3])
    with pytest.raises(ValueError, match="without a residual"):
        q.qlora_rms_norm_fwd(X, g, h=torch.zeros_like(X))
    with pytest.raises(ValueError, match="multiple of 64"):
        q.qlora_rms_norm_fwd(torch.zeros(4, 72, **bf), torch.ones(72), act8=True)
    with pytest.raises(ValueError, match="act8.codes"):
        q.qlora_rms_norm_fwd(torch.zeros(5, 64, **bf), g, act8=c8)
    with pytest.raises(ValueError, match="GPU tensor"):
        q.qlora_rms_norm_fwd(X, g, X)
    with pytest.raises(TypeError, match="rstd"):
        q.qlora_rms_norm_bwd(X, X, torch.ones(4, **bf), g)
    with pytest.raises(TypeError, match="dg"):
        q.qlora_rms_norm_bwd(X, X, torch.ones(4), g, dg=torch.zeros(64, **bf))
    with pytest.raises(ValueError, match="dres"):
        q.qlora_rms_norm_bwd(X, X, torch.ones(4), g, dres=X[:2])
    lg = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="score must be"):
        q.qlora_router_fwd(lg, 2, "tanh")
    with pytest.raises(TypeError, match="logits must be"):
        q.qlora_router_fwd(lg.double(), 2)
    with pytest.raises(TypeError, match="bias must be"):
        q.qlora_router_fwd(lg, 2, bias=torch.zeros(8, **bf))
    with pytest.raises(ValueError, match="GPU tensor"):
        q.qlora_router_fwd(lg, 2)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError, match="ids must be"):
        q.qlora_router_bwd(torch.zeros(4, 2), lg, ids.long())
    with pytest.raises(ValueError, match="dweights"):
        q.qlora_router_bwd(torch.zeros(4, 3), lg, ids)
    with pytest.raises(TypeError, match="dlogits"):
        q.qlora_router_bwd(torch.zeros(4, 2), lg, ids, dlogits=torch.zeros(4, 8, **bf))
