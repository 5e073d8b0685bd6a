"""The timed cases of the operators in front of and around a QLoRA layer's
projections: the root-mean-square norm with the residual's addition (with an
8-bit checkpoint of its output where asked), checkpoints of activations in 8
bits and the layer's backward pass from them, and the routing of tokens to
experts.

Each case is a dict of plain values.  `prepare` makes its inputs from a seed,
`run` makes one pass: with `own` false in elementary torch operations (32-bit
arithmetic, 64 bits in the router, rounded once at the end), with
`own` true through this repository's package.  `exact` gives the same outputs
from the definitions in 64 bits, and `work` the bytes and operations a pass
cannot do without.

Definitions (tokens or rows M, width K)
  norm      h = bf16(x + residual) (x itself without one), rstd = 1 / sqrt(mean
            of a row's h^2 + eps), y = bf16(h rstd g)
            backward: n = h rstd, c = mean of a row's dy g n,
            dx = bf16(dres + rstd (dy g - n c)), dg = sum over rows of dy n
  act8      blocks of 64 along K: c = fl32(max |x| / 127), code =
            rint(fl32(x / c)), the value bf16(fl32(code c)); a block of zeros
            has c = 0.  The norm's 8-bit output is that of its bf16 y.
  layer     with X the values of a checkpoint: G = dY B^T, dX = dY W + s G A^T,
            dA = s X^T G, dB = s T^T dY, grouped by expert on the rows of each
            expert; row i of a grouped call is token order[i] / topk
  router    p = softmax or sigmoid of a token's logits; experts are ranked by
            p + bias in 64 bits (by the logit without a bias), ties to the
            lower index; of `groups` equal groups of experts the `top_groups`
            with the largest sum of their `group_top` best ranks stay; the topk
            best experts, best first: ids; weights p, or p / sum of the chosen
            p with `renorm`, times scale.  An expert with a logit of -inf is
            never chosen, slots left over have id -1 and weight 0.
            backward: the gradient of the weights, ids held fixed
W is 4-bit codes in blocks of 64 with one constant c_b each (an 8-bit integer
times one fp32 per 256 blocks, or fp32): bf16(level[code] c_b).
"""
import math
import statistics

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5
_S = 0.25       # the adapters' scale, alpha / r of 16 / 64
_SCALE = 2.5    # the router's factor on its weights


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a 65B-shaped stack: four tokens, latency
        dict(name="norm_fwd_decode", kind="norm", back=False, M=4, K=8192, residual=True,
             act8=False, g="fp32"),
        # training forward of a 33B-shaped layer at 4096 tokens, its input kept in 8 bits
        dict(name="norm_fwd_train", kind="norm", back=False, M=4096, K=6656, residual=True,
             act8=True, g="fp32"),
        # backward of the smallest training step: 16 tokens
        dict(name="norm_bwd_1k", kind="norm", back=True, M=16, K=1024, residual=True, act8=False,
             g="bf16"),
        # backward of a 65B-shaped layer at 4096 tokens
        dict(name="norm_bwd_train", kind="norm", back=True, M=4096, K=8192, residual=True,
             act8=False, g="fp32"),
        # a checkpoint of 16 tokens, written and read back
        dict(name="act8_16x1024", kind="act8", M=16, K=1024),
        # the input of a 33B-shaped down projection at 4096 tokens, written and read back
        dict(name="act8_4096x17920", kind="act8", M=4096, K=17920),
        # the smallest training step's backward from a checkpoint
        dict(name="linear_bwd_1k", kind="linear", M=16, N=1024, K=1024, r=16, book="nf4", dq=True),
        # backward of eight experts' up projection, 4096 tokens with two experts each, from the
        # checkpoint of the tokens (each row kept once, not once for each expert)
        dict(name="grouped_bwd_train", kind="grouped", tokens=4096, topk=2, E=8, N=11008, K=4096,
             r=64, book="nf4", dq=True),
        # a decode step of eight experts: latency
        dict(name="router_fwd_decode", kind="router", back=False, tokens=8, E=8, topk=2,
             score="softmax", bias=False, groups=1, top_groups=1, group_top=1, renorm=True,
             logits="bf16", masked=0.0),
        # a training batch of fine-grained experts: sigmoid scores, a bias that balances, groups
        dict(name="router_fwd_train", kind="router", back=False, tokens=8192, E=256, topk=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2, renorm=True,
             logits="fp32", masked=0.0),
        # the gradients of the decode-sized batch (the last, small batch of an epoch)
        dict(name="router_bwd_8", kind="router", back=True, tokens=8, E=8, topk=2,
             score="softmax", bias=False, groups=1, top_groups=1, group_top=1, renorm=False,
             logits="fp32", masked=0.0),
        # and of a training batch of 64 experts
        dict(name="router_bwd_train", kind="router", back=True, tokens=8192, E=64, topk=4,
             score="softmax", bias=False, groups=1, top_groups=1, group_top=1, renorm=True,
             logits="bf16", masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_weight(rng):
    """N (a multiple of 8), K (of 64), r (of 8), the codebook and constants."""
    N = 8 * _log_int(rng, 8, 1376)
    K = 64 * _log_int(rng, 1, 172)
    r = 8 * _log_int(rng, 1, 16)
    return N, K, r, rng.choice(["nf4", "nf4", "nf4", "int4", "fp4"]), rng.random() < 0.75


def draw(rng):
    kind = rng.choice(["norm", "norm", "act8", "linear", "grouped", "router", "router"])
    if kind == "norm":
        back, act8 = rng.random() < 0.5, rng.random() < 0.4
        K = 64 * _log_int(rng, 1, 280) if act8 else 8 * _log_int(rng, 1, 2240)
        M = min(_log_int(rng, 1, 16384), 4096 * 17920 // K)
        return dict(kind=kind, back=back, M=M, K=K, residual=rng.random() < 0.7,
                    act8=act8 and not back, g=rng.choice(["fp32", "bf16"]))
    if kind == "act8":
        K = 64 * _log_int(rng, 1, 280)
        return dict(kind=kind, M=min(_log_int(rng, 1, 16384), 4096 * 17920 // K), K=K)
    if kind == "linear":
        N, K, r, book, dq = _draw_weight(rng)
        return dict(kind=kind, M=_log_int(rng, 1, 2048), N=N, K=K, r=r, book=book, dq=dq)
    if kind == "grouped":
        N, K, r, book, dq = _draw_weight(rng)
        E = _log_int(rng, 1, 48)
        while E * N * K > 8 * 11008 * 4096:
            E = (E + 1) // 2
        if dq:   # an expert's weight is whole groups of 256 blocks
            step = 16384 // math.gcd(16384, 8 * K)
            N = 8 * step * max(1, round(N / (8 * step)))
        topk = rng.randint(1, min(6, E))
        rows = max(topk, min(8192, 8192 * 4096 * 11008 // (2 * N * K)))
        return dict(kind=kind, tokens=_log_int(rng, 1, rows // topk), topk=topk, E=E, N=N, K=K,
                    r=r, book=book, dq=dq)
    score = rng.choice(["softmax", "sigmoid"])
    groups = rng.choice([1, 1, 2, 4, 8])
    E = groups * _log_int(rng, 1, 512 // groups)
    top_groups = rng.randint(1, groups)
    # (two members' sigmoids can sum to the same value in two groups; a bias sets them apart)
    bias = rng.random() < 0.5 or (score == "sigmoid" and top_groups < groups)
    return dict(kind=kind, back=rng.random() < 0.4, tokens=_log_int(rng, 1, 16384), E=E,
                topk=rng.randint(1, min(12, E // groups * top_groups)), score=score,
                bias=bias, groups=groups, top_groups=top_groups,
                group_top=rng.randint(1, min(2, E // groups)), renorm=rng.random() < 0.6,
                logits=rng.choice(["bf16", "fp32"]), masked=rng.choice([0.0, 0.0, 0.3]))


def work(case):
    kind = case["kind"]
    if kind == "norm":
        n, gb = case["M"] * case["K"], case["K"] * (4 if case["g"] == "fp32" else 2)
        if case["back"]:      # h, dy (and dres) -> dx; rstd and g in, dg out
            return {"bytes": n * (6 + 2 * case["residual"]) + 4 * case["M"] + 2 * gb,
                    "flops": 10 * n}
        b = n * (4 + 4 * case["residual"]) + 4 * case["M"] + gb
        if case["act8"]:      # codes and constants out, and read back as values
            b += int(n * (2 * (1 + 4 / 64) + 2))
        return {"bytes": b, "flops": 5 * n}
    if kind == "act8":        # x -> codes and constants -> values
        n = case["M"] * case["K"]
        return {"bytes": int(n * (4 + 2 * (1 + 4 / 64))), "flops": 6 * n}
    if kind == "router":
        n, k, eb = case["tokens"] * case["E"], case["tokens"] * case["topk"], \
            2 if case["logits"] == "bf16" else 4
        if case["back"]:      # logits, ids, dweights -> dlogits
            return {"bytes": 2 * n * eb + 8 * k, "flops": 5 * n}
        return {"bytes": n * eb + 8 * k + 4 * case["E"] * case["bias"], "flops": 10 * n}
    N, K, r = case["N"], case["K"], case["r"]
    linear = kind == "linear"
    tokens = case["M"] if linear else case["tokens"]
    E, M = (1, tokens) if linear else (case["E"], tokens * case["topk"])
    active = min(E, M)
    wbytes = N * K / 2 + (N * K / 64 * (1 + 4 / 256) if case["dq"] else N * K / 64 * 4)
    adapters = 2 * r * (N + K)
    # weights and adapters, dY -> dX, T, the checkpoint; dA and dB of every expert
    b = active * (wbytes + adapters) + 2 * M * (N + K) + 4 * M * r + tokens * K * (1 + 4 / 64) \
        + E * adapters + (0 if linear else 4 * M)
    return {"bytes": int(b), "flops": 2 * M * N * K + 4 * M * r * (N + K)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _bf16(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _activations(g, M, K):
    """A layer's activations: normal, with a few wide channels."""
    wide = 1 + 12 * (torch.rand(K, generator=g, device=DEV) < 0.01)
    return (torch.randn((M, K), generator=g, device=DEV) * wide).to(torch.bfloat16)


def _weight(g, rows, K, dq):
    """Codes and constants of a weight of standard deviation about 0.02: the
    codes are near uniform (each level of NF4 covers equal probability mass)
    and a block's largest magnitude is near 2.4 standard deviations."""
    nb = rows * K // 64
    codes = torch.randint(0, 256, (rows * K // 2,), generator=g, device=DEV, dtype=torch.uint8)
    if not dq:
        return codes, None, 0.048 * (0.7 + 0.6 * torch.rand(nb, generator=g, device=DEV))
    q = torch.randint(100, 256, (nb,), generator=g, device=DEV, dtype=torch.uint8)
    scale = 0.065 / 255 * (0.9 + 0.2 * torch.rand((nb + 255) // 256, generator=g, device=DEV))
    return codes, q, scale


def _make(case, seed):
    """The inputs of a case, the same for every form."""
    g = _gen(seed)
    kind = case["kind"]
    if kind == "act8":
        return dict(x=_activations(g, case["M"], case["K"]))
    if kind == "norm":
        M, K = case["M"], case["K"]
        w = 1 + 0.1 * torch.randn(K, generator=g, device=DEV)
        st = dict(x=_activations(g, M, K), g=w if case["g"] == "fp32" else w.to(torch.bfloat16))
        if case["back"]:
            # what the forward pass kept: the residual stream h and its rows' rstd
            st["h"] = st.pop("x")
            st["rstd"] = (st["h"].float().square().mean(1) + EPS).rsqrt()
            st["dy"] = _bf16(g, (M, K))
            st["dres"] = _bf16(g, (M, K)) if case["residual"] else None
        else:
            st["residual"] = _activations(g, M, K) if case["residual"] else None
        return st
    if kind == "router":
        T, E = case["tokens"], case["E"]
        x = 2 * torch.randn((T, E), generator=g, device=DEV)
        x += torch.randn(E, generator=g, device=DEV)        # popular experts
        x = torch.where(torch.rand((T, E), generator=g, device=DEV) < case["masked"],
                        torch.full_like(x, -math.inf), x)
        st = dict(logits=x if case["logits"] == "fp32" else x.to(torch.bfloat16), bias=None)
        if case["bias"]:
            st["bias"] = 0.05 * torch.randn(E, generator=g, device=DEV)
        if case["back"]:
            st["dweights"] = torch.randn((T, case["topk"]), generator=g, device=DEV)
            st["ids"] = _plain_route(dict(st, case=case))[0]   # the forward pass chose them
        return st
    N, K, r = case["N"], case["K"], case["r"]
    linear = kind == "linear"
    E, tokens = (1, case["M"]) if linear else (case["E"], case["tokens"])
    M = tokens if linear else tokens * case["topk"]
    st = dict(x8=_pack(_activations(g, tokens, K)), w=_weight(g, E * N, K, case["dq"]),
              A=_bf16(g, (E, K, r), 1.0 / r), B=_bf16(g, (E, r, N), 0.01), dY=_bf16(g, (M, N)),
              T=torch.randn((M, r), generator=g, device=DEV))   # kept by the forward pass
    if not linear:
        # topk different experts for every token, some experts popular; slots sorted by expert
        key = torch.rand((tokens, E), generator=g, device=DEV)
        key += 0.5 * torch.rand((1, E), generator=g, device=DEV)
        ids = key.topk(case["topk"], dim=1).indices.reshape(-1)
        ids, order = torch.sort(ids, stable=True)
        st["order"] = order.to(torch.int32)
        st["offsets"] = torch.searchsorted(ids, torch.arange(E + 1, device=DEV)).to(torch.int32)
    return st


def prepare(case, seed):
    st = _make(case, seed)
    st["case"] = case
    kind = case["kind"]
    if kind in ("linear", "grouped"):
        st["sizes"] = [case["M"]] if kind == "linear" else \
            (st["offsets"][1:] - st["offsets"][:-1]).tolist()
        if kind == "linear":
            st["A"], st["B"] = st["A"][0], st["B"][0]
        if own:
            import bit_quantized_fine_amd as q
            st["ow"] = q.Q4Weight(*st["w"], len(st["sizes"]) * case["N"], case["K"], case["book"],
                                  case["dq"])
            st["ox"] = q.Act8(*st["x8"])
    return st


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _pack(x):
    """codes int8 [M, K] and constants fp32 [M, K / 64] of bf16 x."""
    b = x.float().reshape(x.shape[0], -1, 64)
    top = b.abs().amax(2)
    c = top / torch.full_like(top, 127)   # (by a Python number torch multiplies by 1 / 127)
    codes = torch.round(torch.where(c[:, :, None] > 0, b / c[:, :, None], torch.zeros_like(b)))
    return codes.clamp(-127, 127).to(torch.int8).reshape(x.shape), c


def _unpack(codes, c):
    b = codes.float().reshape(codes.shape[0], -1, 64)
    return (b * c[:, :, None]).to(torch.bfloat16).reshape(codes.shape)


def _plain_norm(st):
    x, g = st["x"].float(), st["g"].float()
    h = x if st["residual"] is None else (x + st["residual"].float()).to(torch.bfloat16).float()
    rstd = 1 / torch.sqrt((h * h).mean(1) + EPS)
    y = (h * rstd[:, None] * g).to(torch.bfloat16)
    out = (h.to(torch.bfloat16), y, rstd)
    if not st["case"]["act8"]:
        return out
    codes, c = _pack(y)
    return out + (_unpack(codes, c),)


def _plain_norm_bwd(st):
    h, dy, rstd = st["h"].float(), st["dy"].float(), st["rstd"][:, None]
    n, d = h * rstd, dy * st["g"].float()
    dx = rstd * (d - n * (d * n).mean(1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return dx.to(torch.bfloat16), (dy * n).sum(0).to(st["g"].dtype)


def _scores(st):
    """p [T, E] and the values experts are ranked by, in 64 bits."""
    case, x = st["case"], st["logits"].double()
    if case["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
        p = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    rank = x if st["bias"] is None else \
        torch.where(x > -math.inf, p + st["bias"].double(), x)
    return p, rank


def _plain_route(st):
    case = st["case"]
    T, E, G = case["tokens"], case["E"], case["groups"]
    p, rank = _scores(st)
    if case["top_groups"] < G:
        # (a single best member without a bias: by its logit, which ranks as its p does)
        by = rank if case["bias"] or case["group_top"] == 1 else \
            torch.where(rank > -math.inf, p, rank)
        best = torch.sort(by.reshape(T, G, E // G), dim=2, descending=True).values
        best = best[:, :, :case["group_top"]]
        total = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        total = torch.where(best[:, :, 0] > -math.inf, total, best[:, :, 0])
        order = torch.sort(total, dim=1, descending=True, stable=True).indices
        keep = torch.zeros((T, G), dtype=torch.bool, device=DEV)
        keep.scatter_(1, order[:, :case["top_groups"]], True)
        keep = keep[:, :, None].expand(T, G, E // G).reshape(T, E)
        rank = torch.where(keep, rank, torch.full_like(rank, -math.inf))
    rank, ids = torch.sort(rank, dim=1, descending=True, stable=True)
    rank, ids = rank[:, :case["topk"]], ids[:, :case["topk"]]
    live = rank > -math.inf
    w = torch.where(live, p.gather(1, ids), torch.zeros_like(rank))
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(live, ids, torch.full_like(ids, -1)).to(torch.int32), \
        (_SCALE * w).float()


def _plain_route_bwd(st):
    # (in 64 bits: where one expert takes nearly all, its gradient is what is left of 1 - p)
    case, ids, x = st["case"], st["ids"].long(), st["logits"].double()
    live, at = ids >= 0, ids.clamp(min=0)
    dw = torch.where(live, _SCALE * st["dweights"].double(), torch.zeros_like(at).double())
    p = _scores(dict(st, bias=None))[0]
    q = torch.where(live, p.gather(1, at), torch.zeros_like(dw))
    out = torch.zeros_like(x)
    slope = 1.0
    if case["score"] == "sigmoid":
        slope = 1 / (1 + torch.exp(x.gather(1, at)))
    if case["renorm"]:
        q = q / q.sum(1, keepdim=True).clamp(min=1e-300)
        out.scatter_add_(1, at, q * (dw - (q * dw).sum(1, keepdim=True)) * slope)
    else:
        out.scatter_add_(1, at, q * dw * slope)
        if case["score"] == "softmax":
            out -= p * (q * dw).sum(1, keepdim=True)
    return out.to(st["logits"].dtype)


def _levels(book):
    if book == "nf4":
        pos = torch.special.ndtri(0.5 + (torch.arange(1, 9, dtype=torch.float64) - 0.5) / 16)
        neg = torch.special.ndtri(0.5 + (torch.arange(1, 8, dtype=torch.float64) - 0.5) / 14)
        lv = torch.cat([-neg.flip(0) / neg[-1], torch.zeros(1, dtype=torch.float64),
                        pos / pos[-1]])
    elif book == "int4":
        lv = (2 * torch.arange(16, dtype=torch.float64) - 15) / 15
    else:
        mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64) / 6
        lv = torch.cat([-mag.flip(0)[:7], torch.zeros(1, dtype=torch.float64), -mag[:1], mag[1:]])
    return lv.to(torch.float32).to(DEV)


def _dequant(st, e):
    """Weight of expert e, fp32 [N, K] holding bf16 values."""
    case = st["case"]
    N, K = case["N"], case["K"]
    codes, q, scale = st["w"]
    nb = N * K // 64
    c = codes[e * N * K // 2:(e + 1) * N * K // 2]
    lv = _levels(case["book"])
    w = torch.stack([lv[(c & 15).long()], lv[(c >> 4).long()]], dim=1).reshape(nb, 64)
    blocks = torch.arange(e * nb, (e + 1) * nb, device=DEV)
    ch = q[blocks].float() * scale[blocks // 256] if q is not None else scale[blocks]
    return (w * ch[:, None]).to(torch.bfloat16).float().reshape(N, K)


def _grads(st, X, dY, T, A, B, e):
    X, dY, A, B = X.float(), dY.float(), A.float(), B.float()
    G = dY @ B.t()
    dX = dY @ _dequant(st, e) + _S * (G @ A.t())
    return tuple(t.to(torch.bfloat16) for t in (dX, _S * (X.t() @ G), _S * (T.t() @ dY)))


def _plain_grouped(st):
    case = st["case"]
    X = _unpack(*st["x8"])[st["order"].long() // case["topk"]]
    dX = torch.empty_like(X)
    dA, dB = torch.empty_like(st["A"]), torch.empty_like(st["B"])
    lo = 0
    for e, m in enumerate(st["sizes"]):
        r = slice(lo, lo + m)
        dX[r], dA[e], dB[e] = _grads(st, X[r], st["dY"][r], st["T"][r], st["A"][e], st["B"][e], e)
        lo += m
    return dX, dA, dB


def _plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "norm":
        return _plain_norm_bwd(st) if case["back"] else _plain_norm(st)
    if kind == "act8":
        codes, c = _pack(st["x"])
        return _unpack(codes, c), c
    if kind == "linear":
        return _grads(st, _unpack(*st["x8"]), st["dY"], st["T"], st["A"], st["B"], 0)
    if kind == "grouped":
        return _plain_grouped(st)
    return _plain_route_bwd(st) if case["back"] else _plain_route(st)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    if not own:
        return _plain(st)
    import bit_quantized_fine_amd as q
    case = st["case"]
    kind = case["kind"]
    if kind == "norm":
        if case["back"]:
            return q.qlora_rms_norm_bwd(st["dy"], st["h"], st["rstd"], st["g"], dres=st["dres"])
        out = q.qlora_rms_norm_fwd(st["x"], st["g"], residual=st["residual"], eps=EPS,
                                   act8=case["act8"])
        return out[:3] + (q.qlora_act8_unpack(out[3]),) if case["act8"] else out
    if kind == "act8":
        x8 = q.qlora_act8_pack(st["x"])
        return q.qlora_act8_unpack(x8), x8.scales
    if kind == "linear":
        return q.qlora_linear_act8_bwd(st["dY"], st["ox"], st["ow"], st["A"], st["B"], _S,
                                       T=st["T"])
    if kind == "grouped":
        return q.qlora_grouped_act8_bwd(st["dY"], st["ox"], st["offsets"], st["ow"], case["E"],
                                        st["A"], st["B"], _S, order=st["order"],
                                        topk=case["topk"], T=st["T"])
    if case["back"]:
        return q.qlora_router_bwd(st["dweights"], st["logits"], st["ids"], score=case["score"],
                                  renorm=case["renorm"], scale=_SCALE)
    return q.qlora_router_fwd(st["logits"], case["topk"], score=case["score"], bias=st["bias"],
                              groups=case["groups"], top_groups=case["top_groups"],
                              group_top=case["group_top"], renorm=case["renorm"], scale=_SCALE)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, apart from the plain forms above
# ---------------------------------------------------------------------------

def _value64(x):
    """The values of the checkpoint of bf16-valued float64 x [M, K], and its
    constants.  The roundings to fp32 and bf16 are the format's own."""
    M, K = x.shape
    v = x.reshape(M * K // 64, 64)
    top = torch.maximum(v.max(1).values, -v.min(1).values)
    c = (top / 127.0).float().double()
    ratio = (v / torch.where(c == 0, torch.ones_like(c), c).unsqueeze(1)).float().double()
    low = torch.floor(ratio)
    frac = ratio - low
    up = (frac > 0.5) | ((frac == 0.5) & (torch.remainder(low, 2) == 1))
    code = torch.clamp(low + up.double(), -127, 127)
    val = (code * c.unsqueeze(1)).float().bfloat16().double()
    return val.reshape(M, K), c.reshape(M, K // 64)


def _codes64(x8):
    codes, c = x8
    v = codes.double() * torch.repeat_interleave(c.double(), 64, dim=1)
    return v.float().bfloat16().double()


def _levels64(book):
    """The fp32 levels of a codebook (part of the format), from the standard
    library's normal quantiles and from the E2M1 bit patterns."""
    if book == "nf4":
        z = statistics.NormalDist().inv_cdf
        pos = [z(0.5 + (j - 0.5) / 16) for j in range(1, 9)]
        neg = [z(0.5 + (j - 0.5) / 14) for j in range(1, 8)]
        lv = [-v / neg[-1] for v in reversed(neg)] + [0.0] + [v / pos[-1] for v in pos]
    elif book == "int4":
        lv = [(2 * k - 15) / 15 for k in range(16)]
    else:
        mag = [(b & 1) * 0.5 if b < 2 else math.ldexp(1 + (b & 1) / 2, (b >> 1) - 1)
               for b in range(8)]
        lv = [-v / 6 for v in reversed(mag[1:])] + [0.0, -0.0] + [v / 6 for v in mag[1:]]
    return torch.from_numpy(np.array(lv).astype(np.float32)).to(DEV)


def _w64(codes, q, scale, lv, N, K, e):
    """deq(W_e) in 64 bits: the rounding to bf16 of the exact products of the
    fp32 level and the fp32 constant is part of the format, and so is the
    constant's own rounding to fp32."""
    nb = N * K // 64
    byte = codes.reshape(-1, nb, 32)[e].int()
    idx = torch.empty((nb, 64), dtype=torch.int64, device=DEV)
    idx[:, 0::2], idx[:, 1::2] = byte % 16, byte // 16
    if q is not None:
        b = torch.arange(e * nb, e * nb + nb, device=DEV)
        c = (q.reshape(-1, nb)[e].double() * scale.double()[b // 256]).float()
    else:
        c = scale.reshape(-1, nb)[e]
    prod = (lv.double()[idx] * c.double()[:, None]).float()
    return prod.bfloat16().double().reshape(N, K)


def _route64(case, st):
    """ids [tokens, topk] on the host, by one search for the largest value
    after the other."""
    x = st["logits"].double().cpu().numpy()
    T, E, G, k = case["tokens"], case["E"], case["groups"], case["topk"]
    dead = np.isneginf(x)
    if case["score"] == "sigmoid":
        t = np.exp(-np.abs(x))
        p = np.where(x > 0, 1.0, t) / (1.0 + t)
    else:
        p = np.exp(x - np.where(dead.all(1), 0.0, x.max(1))[:, None])
        p = p / np.where(dead.all(1), 1.0, p.sum(1))[:, None]
    rank = x.copy()
    if st["bias"] is not None:
        rank = np.where(dead, -np.inf, p + st["bias"].double().cpu().numpy())
    row = np.arange(T)
    if case["top_groups"] < G:
        by = rank if case["bias"] or case["group_top"] == 1 else np.where(dead, -np.inf, p)
        left = by.reshape(T, G, E // G).copy()
        total = np.full((T, G), -np.inf)
        for i in range(case["group_top"]):
            at = left.argmax(2)[:, :, None]
            best = np.take_along_axis(left, at, 2)[:, :, 0]
            total = best if i == 0 else total + np.where(np.isneginf(best), 0.0, best)
            np.put_along_axis(left, at, -np.inf, 2)
        kept = np.zeros((T, G), bool)
        for _ in range(case["top_groups"]):
            at = total.argmax(1)
            kept[row, at] |= ~np.isneginf(total[row, at])
            total[row, at] = -np.inf
        rank[~np.repeat(kept, E // G, axis=1)] = -np.inf
    ids = np.full((T, k), -1, np.int64)
    for j in range(k):
        at = rank.argmax(1)
        ids[:, j] = np.where(np.isneginf(rank[row, at]), -1, at)
        rank[row, at] = -np.inf
    return ids


def _weights64(case, x, ids):
    """The weights [tokens, topk] of chosen experts as a function of the
    logits x (float64, differentiable), 0 for a slot without one."""
    live = ids >= 0
    at = torch.where(live, ids, torch.zeros_like(ids))
    if case["score"] == "sigmoid":
        logp = torch.nn.functional.logsigmoid(x)
    else:
        logp = x - torch.logsumexp(x, 1, keepdim=True)
    mine = torch.where(live, torch.gather(logp, 1, at), torch.full_like(at, -math.inf,
                                                                       dtype=torch.float64))
    if case["renorm"]:
        some = live.any(1, keepdim=True)
        total = torch.logsumexp(torch.where(some, mine, torch.zeros_like(mine)), 1, keepdim=True)
        mine = torch.where(live, mine, torch.zeros_like(mine)) - total
    else:
        mine = torch.where(live, mine, torch.zeros_like(mine))
    return torch.where(live, _SCALE * torch.exp(mine), torch.zeros_like(mine))


def _exact_router(case, st):
    if not case["back"]:
        ids = torch.from_numpy(_route64(case, st)).to(DEV)
        # (-inf would make 0 times infinity in what nobody reads)
        x = st["logits"].double().clamp(min=-1e30)
        return ids.to(torch.int32), _weights64(case, x, ids)
    ids = st["ids"].long()
    x = st["logits"].double().clamp(min=-1e30).requires_grad_(True)
    w = _weights64(case, x, ids)
    return torch.autograd.grad((w * st["dweights"].double()).sum(), x)[0]


def exact(case, seed):
    st = _make(case, seed)
    kind = case["kind"]
    if kind == "act8":
        return _value64(st["x"].double())
    if kind == "router":
        return _exact_router(case, st)
    if kind == "norm":
        g = st["g"].double()
        if case["back"]:
            h, dy, rstd = st["h"].double(), st["dy"].double(), st["rstd"].double().unsqueeze(1)
            inner = torch.sum(dy * h * g, 1, keepdim=True) / case["K"]
            dx = rstd * g * dy - h * (rstd ** 3 * inner)
            dx = dx if st["dres"] is None else dx + st["dres"].double()
            return dx, torch.sum(h * rstd * dy, 0)
        h = st["x"].double()
        if st["residual"] is not None:
            h = (h + st["residual"].double()).bfloat16().double()   # the stored stream
        rstd = torch.pow(torch.sum(h ** 2, 1) / case["K"] + EPS, -0.5)
        y = g * h * rstd.unsqueeze(1)
        if not case["act8"]:
            return h, y, rstd
        return h, y, rstd, _value64(y.bfloat16().double())[0]
    N, K, r = case["N"], case["K"], case["r"]
    X = _codes64(st["x8"])
    lv = _levels64(case["book"])
    if kind == "linear":
        ends = np.array([case["M"]])
    else:
        X = X[torch.div(st["order"].long(), case["topk"], rounding_mode="floor")]
        ends = st["offsets"].cpu().numpy()[1:]
    dX = torch.empty_like(X)
    dA = torch.zeros((len(ends), K, r), dtype=torch.float64, device=DEV)
    dB = torch.zeros((len(ends), r, N), dtype=torch.float64, device=DEV)
    a = 0
    for e, b in enumerate(int(v) for v in ends):
        dY, A = st["dY"][a:b].double(), st["A"][e].double()
        G = torch.mm(dY, st["B"][e].double().T) * _S
        dX[a:b] = torch.mm(dY, _w64(*st["w"], lv, N, K, e)) + torch.mm(G, A.T)
        dA[e] = torch.mm(X[a:b].T, G)
        dB[e] = torch.mm(st["T"][a:b].double().T, dY) * _S
        a = b
    return (dX, dA[0], dB[0]) if kind == "linear" else (dX, dA, dB)
