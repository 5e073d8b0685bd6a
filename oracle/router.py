"""Routing of tokens to experts, on the host in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

p = softmax or sigmoid of a token's logits; experts rank by p + bias, or by the
logit without a bias; of `groups` groups the top_groups with the largest sum of
their group_top best ranks (best p without a bias) stay; the topk best experts,
best first, ties to the lower index; weights scale p, or scale p over the sum of
the chosen p.  Experts at -inf (or NaN) are not chosen; slots left over have id
-1 and weight 0.
"""
import math

import numpy as np


def scores(x, score):
    """p of one token's logits (float64, finite or -inf)."""
    if score == "sigmoid":
        return np.array([math.exp(min(v, 0.0)) / (1 + math.exp(-abs(v))) if v > -math.inf else 0.0
                         for v in x])
    if not (x > -np.inf).any():
        return np.zeros(len(x))
    e = np.exp(x - x.max())
    return e / math.fsum(e)


def choose(x, topk, score="softmax", bias=None, groups=1, top_groups=1, group_top=1):
    """The ids of one token, best first, -1 for slots left over."""
    E = len(x)
    p = scores(x, score)
    rank = [float(v) for v in (x if bias is None else p + bias)]
    open_ = [e for e in range(E) if x[e] > -np.inf and rank[e] > -np.inf]
    if top_groups < groups:
        size = E // groups
        by = rank if bias is not None or group_top == 1 else p
        total = []
        for j in range(groups):
            best = sorted((float(by[e]) for e in open_ if e // size == j), reverse=True)
            if best:
                total.append((-sum(best[:group_top]), j))
        stay = {j for _, j in sorted(total)[:top_groups]}
        open_ = [e for e in open_ if e // size in stay]
    best = sorted(open_, key=lambda e: (-rank[e], e))[:topk]
    return best + [-1] * (topk - len(best))


def weights(x, ids, score="softmax", renorm=True, scale=1.0):
    """The weights of one token's chosen experts."""
    live = [j for j, e in enumerate(ids) if e >= 0]
    w = np.zeros(len(ids))
    if not live:
        return w
    v = np.array([x[ids[j]] for j in live])
    if renorm:   # the factor that the chosen share is taken out first
        low = np.minimum(v, 0.0) if score == "sigmoid" else v
        u = np.exp(low - low.max())
        if score == "sigmoid":
            u = u / (1 + np.exp(-np.abs(v)))
        u = u / math.fsum(u)
    else:
        u = scores(x, score)[[ids[j] for j in live]]
    w[live] = scale * u
    return w


def fwd(X, topk, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=True,
        scale=1.0):
    ids = np.array([choose(x, topk, score, bias, groups, top_groups, group_top) for x in X],
                   np.int64).reshape(len(X), topk)
    return ids, np.array([weights(x, i, score, renorm, scale)
                          for x, i in zip(X, ids)]).reshape(len(X), topk)


def bwd(dW, X, ids, score="softmax", renorm=True, scale=1.0):
    """dlogits, from the Jacobian of each token's weights, and the sums of
    magnitudes behind each.  What is left of one is a sum of the other shares,
    which keeps its digits where one expert takes nearly all."""
    out, mag = np.zeros(X.shape), np.zeros(X.shape)
    for t, (x, row) in enumerate(zip(X, ids)):
        p = scores(x, score)
        w = weights(x, row, score, renorm, 1.0)
        rest = lambda v, i: math.fsum(v[:i]) + math.fsum(v[i + 1:])
        slope = (lambda e: 1.0 / (1.0 + math.exp(x[e])) if x[e] < 700 else 0.0)
        for i, ei in enumerate(row):
            if ei < 0:
                continue
            for e in range(len(x)):
                # d w_i / d x_e
                if renorm:
                    js = [j for j, ej in enumerate(row) if ej == e]
                    d = sum(w[i] * (rest(w, i) if i == j else -w[j]) for j in js)
                    d *= slope(e) if score == "sigmoid" else 1.0
                elif score == "sigmoid":
                    d = p[e] * slope(e) if e == ei else 0.0
                else:
                    d = p[ei] * (rest(p, e) if e == ei else -p[e])
                out[t, e] += scale * dW[t, i] * d
                mag[t, e] += abs(scale * dW[t, i] * d)
    return out, mag
