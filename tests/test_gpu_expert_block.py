"""The norm, the router, the plan, the exchange, the grouped layer and the 8-bit
checkpoint run together, as a block of a mixture of experts trains: every stage
against float64 on the inputs that the stage before it left, and the whole in a
graph."""
import numpy as np
import pytest

import bit_quantized_fine_amd as q
import oracle
from expert_util import within
from gpu_util import bits, dev, need_gpu, say, torch
from oracle import act8 as oa
from oracle import experts as ox
from oracle import norm as on
from oracle import router as orr

pytestmark = pytest.mark.gpu

EPS = 1e-5


def f(t):
    return t.double().cpu().numpy()


class Block:
    def __init__(self, tokens, K, E, topk, r, seed):
        g = torch.Generator(device=dev()).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device=dev())
        self.tokens, self.K, self.E, self.topk = tokens, K, E, topk
        self.x, self.res = rand(tokens, K).bfloat16(), rand(tokens, K).bfloat16()
        self.g = 1 + 0.1 * rand(K)
        self.Wr = rand(K, E) / K ** 0.5                   # the router's own projection
        self.bias = 0.05 * rand(E)
        self.w = q.qlora_q4_quantize(rand(E * K, K) * 0.02, "nf4", True)
        self.A, self.B = (rand(E, K, r) / r).bfloat16(), (rand(E, r, K) * 0.1).bfloat16()
        self.dout = rand(tokens, K).bfloat16()
        self.cfg = dict(score="sigmoid", renorm=True, scale=1.5)

    def forward(self):
        h, y, rstd, y8 = q.qlora_rms_norm_fwd(self.x, self.g, self.res, EPS, act8=True)
        logits = y.float() @ self.Wr
        ids, weights = q.qlora_router_fwd(logits, self.topk, bias=self.bias, **self.cfg)
        offsets, order, inverse = q.qlora_expert_plan(ids, self.E)
        Xs = q.qlora_expert_gather(y, inverse)
        Y, T = q.qlora_grouped_fwd(Xs, offsets, self.w, self.E, self.A, self.B, 0.5)
        out = q.qlora_expert_combine(Y, inverse, weights)
        return dict(h=h, y=y, rstd=rstd, codes=y8.codes, scales=y8.scales, logits=logits, ids=ids,
                    weights=weights, offsets=offsets, order=order, inverse=inverse, Y=Y, T=T,
                    out=out)

    def backward(self, s):
        """Keeps no bf16 copy of y or of its gathered rows."""
        dY, dw = q.qlora_expert_combine_bwd(self.dout, s["Y"], s["inverse"], s["weights"])
        dXs, dA, dB = q.qlora_grouped_act8_bwd(dY, q.Act8(s["codes"], s["scales"]), s["offsets"],
                                               self.w, self.E, self.A, self.B, 0.5,
                                               order=s["order"], topk=self.topk, T=s["T"])
        dlogits = q.qlora_router_bwd(dw, s["logits"], s["ids"], **self.cfg)
        dy = q.qlora_expert_combine(dXs, s["inverse"])     # the gather's backward
        dy = (dy.float() + dlogits @ self.Wr.t()).bfloat16()
        dx, dg = q.qlora_rms_norm_bwd(dy, s["h"], s["rstd"], self.g, dres=self.dout)
        return dict(dY=dY, dw=dw, dXs=dXs, dA=dA, dB=dB, dlogits=dlogits, dy=dy, dx=dx, dg=dg)

    def step(self):
        s = self.forward()
        return {**s, **self.backward(s)}


@pytest.mark.parametrize("tokens,K,E,topk,r", [(1, 128, 4, 2, 8), (37, 256, 8, 2, 16),
                                               (300, 256, 6, 3, 32)])
def test_stages(tokens, K, E, topk, r):
    need_gpu()
    say(f"block tokens={tokens} K={K} E={E} topk={topk}")
    b = Block(tokens, K, E, topk, r, tokens)
    s = b.step()
    torch.cuda.synchronize()
    h = on.stream(f(b.x), f(b.res))
    np.testing.assert_array_equal(f(s["h"]), h)
    within("y", s["y"], on.fwd(h, f(b.g), EPS)[0], on.fwd_bounds(h, f(b.g), EPS)[0])
    codes, c = oa.pack(bits(s["y"]))
    np.testing.assert_array_equal(s["codes"].cpu().numpy(), codes)
    ids, w = orr.fwd(f(s["logits"]), topk, "sigmoid", f(b.bias), renorm=True, scale=1.5)
    np.testing.assert_array_equal(s["ids"].cpu().numpy(), ids)
    within("weights", s["weights"], w, 1.001 * 2.0 ** -24 * w)
    off, order, inv = ox.plan(ids, E)
    np.testing.assert_array_equal(s["order"].cpu().numpy(), order)
    # forward rows from y itself, gradients from its checkpoint
    rows = order // topk
    W = f(q.qlora_q4_dequantize(b.w)).reshape(E, K, K)
    args = lambda X: (X[rows], off, list(W), list(f(b.A)), list(f(b.B)), 0.5)
    Y, T = ox.grouped_fwd(*args(f(s["y"])))
    bound = ox.grouped_bounds(None, *args(f(s["y"])))
    within("Y", s["Y"], Y, bound["Y"])
    within("T", s["T"], T, bound["T"])
    out, mag = ox.combine(f(s["Y"]), inv, f(s["weights"]))
    within("out", s["out"], out, 2.0 ** -8 * np.abs(out) + 1.01 * topk * 2.0 ** -24 * mag)
    kept = oracle.bf16_bits_to_f64(oa.value_bits(codes, c))
    dX, dA, _ = ox.grouped_bwd(f(s["dY"]), *args(kept))
    bound = ox.grouped_bounds(f(s["dY"]), *args(kept))
    within("dXs", s["dXs"], dX, bound["dX"])
    within("dA", s["dA"], dA, bound["dA"])
    # dB takes the forward's T: X A of y, not of its checkpoint
    dB = np.stack([0.5 * f(s["T"])[off[e]:off[e + 1]].T @ f(s["dY"])[off[e]:off[e + 1]]
                   for e in range(E)])
    magB = np.stack([0.5 * np.abs(f(s["T"])[off[e]:off[e + 1]]).T
                     @ np.abs(f(s["dY"])[off[e]:off[e + 1]]) for e in range(E)])
    n = (off[1:] - off[:-1])[:, None, None]
    within("dB", s["dB"], dB, 2.0 ** -8 * np.abs(dB) + 1.01 * ((2 * n + 8) * 2.0 ** -24
                                                             + 2.0 ** -16) * magB)
    dl, mag = orr.bwd(f(s["dw"]), f(s["logits"]), ids, "sigmoid", True, 1.5)
    within("dlogits", s["dlogits"], dl, 1.001 * 2.0 ** -24 * np.abs(dl) + 1e-13 * mag)
    a = (f(s["dy"]), h, f(s["rstd"]), f(b.g), f(b.dout))
    dx, dg = on.bwd(*a)
    bx, bg = on.bwd_bounds(*a)
    within("dx", s["dx"], dx, bx)
    within("dg", s["dg"], dg, bg)


def test_step_in_a_graph():
    """Replays with new inputs, eager work between them: the bits of eager steps."""
    need_gpu()
    say("block in a graph")
    b = Block(200, 256, 8, 2, 16, 9)
    b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.step()
    for i in range(3):
        b.x.copy_(torch.randn_like(b.x.float()))
        b.dout.copy_(torch.randn_like(b.x.float()))
        graph.replay()
        a = {k: t.clone() for k, t in got.items()}
        e = b.step()
        torch.cuda.synchronize()
        for k in a:
            assert torch.equal(a[k], e[k]), k
