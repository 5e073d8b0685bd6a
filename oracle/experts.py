"""The layer grouped by expert and the exchange around it, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Rows offsets[e] .. offsets[e+1]-1 of X belong to expert e.  With mask D (1
where an element of X is kept, 0 where it is dropped) and c its scale:

    T  = c (D X) A_e              Y  = X W_e^T + s T B_e
    G  = dY B_e^T                 dX = dY W_e + s c D (G A_e^T)
    dA_e = s c (D X)^T G          dB_e = s T^T dY

Every product is also formed from absolute values: the sums of magnitudes
that bound a finite-precision evaluation's error (see grouped_bounds).
"""
import numpy as np


def _fwd(X, Xd, W, A, B, s):
    T = Xd @ A
    return X @ W.T + s * (T @ B), T


def grouped_fwd(X, offsets, Ws, As, Bs, s, D=None, c=1.0):
    """float64 operands, lists per expert; rows outside the groups are NaN."""
    Y = np.full((X.shape[0], Ws[0].shape[0]), np.nan)
    T = np.full((X.shape[0], As[0].shape[1]), np.nan)
    Xd = X if D is None else np.where(D, X, 0.0) * c
    for e, (W, A, B) in enumerate(zip(Ws, As, Bs)):
        r = slice(offsets[e], offsets[e + 1])
        Y[r], T[r] = _fwd(X[r], Xd[r], W, A, B, s)
    return Y, T


def grouped_bwd(dY, X, offsets, Ws, As, Bs, s, D=None, c=1.0):
    dX = np.full(X.shape, np.nan)
    Xd = X if D is None else np.where(D, X, 0.0) * c
    dAs, dBs = [], []
    for e, (W, A, B) in enumerate(zip(Ws, As, Bs)):
        r = slice(offsets[e], offsets[e + 1])
        G = dY[r] @ B.T
        L = s * (G @ A.T)
        if D is not None:
            L = np.where(D[r], L, 0.0) * c
        dX[r] = dY[r] @ W + L
        dAs.append(s * (Xd[r].T @ G))
        dBs.append(s * ((Xd[r] @ A).T @ dY[r]))
    return dX, np.stack(dAs), np.stack(dBs)


U = 2.0 ** -24        # half a step of fp32
HALF_BF16 = 2.0 ** -8  # half a step of bf16
SPLIT = 2.0 ** -16    # an fp32 factor as the sum of two bf16 halves


def grouped_bounds(dY, X, offsets, Ws, As, Bs, s, D=None, c=1.0):
    """Elementwise error bounds of (Y, T, dX, dA, dB) for an evaluation with
    exact products of bf16 factors, fp32 sums in any order, fp32 T and G that
    enter their products as two bf16 halves, and one rounding to bf16.

    A sum of n terms in fp32 is off by at most n U times the sum of their
    magnitudes (first order); 8 more roundings cover the scale factors, the
    joins of split sums and the second order.  A factor's own error (T's, G's)
    goes through its product; a split loses SPLIT of the factor's magnitude.
    """
    n = lambda k: (k + 8) * U
    aX, aS = np.abs(X), abs(s)
    Xd = aX if D is None else np.where(D, aX, 0.0) * c
    M, K = X.shape
    out = {k: None for k in ("Y", "T", "dX")}
    out["Y"] = np.zeros((M, Ws[0].shape[0]))
    out["T"] = np.zeros((M, As[0].shape[1]))
    out["dX"] = np.zeros((M, K))
    dA, dB = [], []
    Yr, Tr = grouped_fwd(X, offsets, Ws, As, Bs, s, D, c)
    if dY is not None:
        dXr, dAr, dBr = grouped_bwd(dY, X, offsets, Ws, As, Bs, s, D, c)
    for e, (W, A, B) in enumerate(zip(Ws, As, Bs)):
        rows = slice(offsets[e], offsets[e + 1])
        N, r = W.shape[0], A.shape[1]
        aW, aA, aB = np.abs(W), np.abs(A), np.abs(B)
        mT = Xd[rows] @ aA                    # magnitudes behind T
        eT = n(K) * mT
        out["T"][rows] = eT
        out["Y"][rows] = (HALF_BF16 * np.abs(Yr[rows])
                          + (1 + HALF_BF16) * (n(K + 2 * r) * (aX[rows] @ aW.T + aS * (mT @ aB))
                                               + aS * ((eT + SPLIT * np.abs(Tr[rows])) @ aB)))
        if dY is None:
            continue
        adY = np.abs(dY[rows])
        mG = adY @ aB.T
        eG = n(N) * mG + SPLIT * np.abs(dY[rows] @ B.T)
        keep = 1.0 if D is None else np.where(D[rows], c, 0.0)
        out["dX"][rows] = (HALF_BF16 * np.abs(dXr[rows]) + (1 + HALF_BF16) * (
            n(N + 2 * r) * (adY @ aW + aS * keep * (mG @ aA.T)) + aS * keep * (eG @ aA.T)))
        m = adY.shape[0]
        dA.append(HALF_BF16 * np.abs(dAr[e]) + (1 + HALF_BF16) * aS * (
            n(2 * m) * (Xd[rows].T @ mG) + Xd[rows].T @ eG))
        dB.append(HALF_BF16 * np.abs(dBr[e]) + (1 + HALF_BF16) * aS * (
            n(2 * m) * (mT.T @ adY) + (eT + SPLIT * np.abs(Tr[rows])).T @ adY))
    if dY is not None:
        out["dA"], out["dB"] = np.stack(dA), np.stack(dB)
    return out


def plan(ids, E):
    """(offsets [E+1], order [n], inverse of ids' shape) by a loop over slots."""
    flat = [int(v) for v in np.asarray(ids).reshape(-1)]
    order, offsets = [], [0]
    for e in range(E):
        order += [i for i, v in enumerate(flat) if v == e]
        offsets.append(len(order))
    inverse = np.full(len(flat), -1, np.int64)
    for row, slot in enumerate(order):
        inverse[slot] = row
    order += [-1] * (len(flat) - len(order))
    return np.array(offsets), np.array(order, np.int64), inverse.reshape(np.asarray(ids).shape)


def combine(Y, inverse, w):
    """out[t] = sum_j w[t, j] Y[inverse[t, j]] and the sums of magnitudes."""
    out = np.zeros((inverse.shape[0], Y.shape[1]))
    mag = np.zeros_like(out)
    for t, rows in enumerate(inverse):
        for j, row in enumerate(rows):
            if row >= 0:
                out[t] += w[t, j] * Y[row]
                mag[t] += np.abs(w[t, j] * Y[row])
    return out, mag


def combine_bwd(dOut, Y, inverse, w):
    """dY (rows no slot has: 0), dw and the sums of magnitudes behind dw."""
    dY, dw = np.zeros(Y.shape), np.zeros(w.shape)
    mag = np.zeros(w.shape)
    for t, rows in enumerate(inverse):
        for j, row in enumerate(rows):
            if row >= 0:
                dY[row] = w[t, j] * dOut[t]
                dw[t, j] = dOut[t] @ Y[row]
                mag[t, j] = np.abs(dOut[t]) @ np.abs(Y[row])
    return dY, dw, mag
