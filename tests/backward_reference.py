"""Plain 64-bit forms (numpy) of the block's gradients, for the tests, written
from the formulas in include/moe.h, with bounds on what 32-bit sums and bf16
operands may differ by."""
from __future__ import annotations

import numpy as np

U_BF16 = 2.0 ** -8      # half a step, relative
U_FP32 = 2.0 ** -24


def combine(dout, y, inv, w):
    """(dy by row, dw, sum of |products| of dw) of moe_combine_backward; y None: dw None."""
    T, k = w.shape
    rows = inv.reshape(T, k)
    dy = {}
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = rows[t, j]
            if r >= 0:
                dy[int(r)] = w[t, j] * dout[t]
                if y is not None:
                    dw[t, j] = (dout[t] * y[r]).sum()
                    mag[t, j] = np.abs(dout[t] * y[r]).sum()
    return dy, dw, mag


def dispatch(dxs, inv, T, k, add=None):
    """(dx, sum of |terms|) of moe_dispatch_backward."""
    dx = np.zeros((T, dxs.shape[1]))
    mag = np.zeros_like(dx)
    for t in range(T):
        for r in inv.reshape(T, k)[t]:
            if r >= 0:
                dx[t] += dxs[r]
                mag[t] += np.abs(dxs[r])
    if add is not None:
        dx, mag = dx + add, mag + np.abs(add)
    return dx, mag


def norm(h, dx, w=None, eps=1e-6, unit_offset=False, add=None):
    """(dh, dw, magnitude of dh's terms, sum of dw's |terms|) of moe_norm_backward."""
    r = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    q = dx if w is None else dx * (1.0 + w if unit_offset else w)
    dh = r * (q - h * r * r * (q * h).mean(1, keepdims=True))
    mag = r * (np.abs(q) + np.abs(h) * r * r * np.abs(q * h).mean(1, keepdims=True))
    n = dx * h * r
    if add is not None:
        dh, mag = dh + add, mag + np.abs(add)
    return dh, n.sum(0), mag, np.abs(n).sum(0)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def route(logits, ids, dw, score="softmax", renormalize=True, scale=1.0):
    """(d_logits, magnitude of its terms) of moe_route_backward, row by row through the forward's own steps."""
    T, E = logits.shape
    l = np.where(np.isnan(logits) | (logits == np.inf), -np.inf, logits)
    dl, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = [(j, int(e)) for j, e in enumerate(ids[t]) if 0 <= e < E and np.isfinite(l[t, e])]
        if not on:
            continue
        j, e = np.array([a for a, _ in on]), np.array([b for _, b in on])
        g = scale * dw[t, j]
        if renormalize:
            z = l[t, e] if score == "softmax" else -np.logaddexp(0.0, -l[t, e])
            v = np.exp(z - z.max())
            v /= v.sum()
            term, m = v * (g - (g * v).sum()), v * (np.abs(g) + np.abs(g * v).sum())
            if score == "sigmoid":
                term, m = term * sigmoid(-l[t, e]), m * sigmoid(-l[t, e])
        elif score == "sigmoid":
            term = g * sigmoid(l[t, e]) * sigmoid(-l[t, e])
            m = np.abs(term)
        else:
            p = np.exp(l[t] - l[t].max())
            p /= p.sum()
            dl[t] -= p * (g * p[e]).sum()
            mag[t] += p * np.abs(g * p[e]).sum()
            term = g * p[e]
            m = np.abs(term)
        np.add.at(dl[t], e, term)
        np.add.at(mag[t], e, m)
    return dl, mag


def mma_rel(terms):
    """What an fp32 sum of `terms` products on the tensor cores, 16 at a time and truncating, may be off,
    relative to the sum of |products|."""
    return (terms / 16 + 32) * 2.0 ** -23


def experts(x, dy, W13, W2, bounds):
    """Gradients of the experts' rows and weights and, for each, a bound on the error of unrounded
    outputs computed from bf16 operands a and [dg du] with fp32 sums.

    a and [dg du] are off by half a bf16 step plus what their own fp32 products carry (mma_rel of the sums,
    through derivatives of at most 1.1 (silu'), 0.5 (silu'')). Those errors are independent from row to row and column
    to column, so a sum of c_i e_i, |e_i| <= d_i, passes 7 sqrt(sum (c_i d_i)^2) once in 2e10 elements
    (Hoeffding: 2 exp(-49/2)). The products' own sums add mma_rel of the sum of |terms|."""
    R, H = x.shape
    E, _, I = W2.shape
    out = {n: np.zeros(s) for n, s in (("dx", (R, H)), ("dW13", W13.shape), ("dW2", W2.shape))}
    tol = {n: np.zeros_like(v) for n, v in out.items()}
    for e in range(E):
        lo, hi = int(bounds[e]), int(bounds[e + 1])
        if hi <= lo:
            continue
        xe, de, w13, w2 = x[lo:hi], dy[lo:hi], W13[e], W2[e]
        gu, mgu = xe @ w13.T, mma_rel(H) * (np.abs(xe) @ np.abs(w13).T)
        d, md = de @ w2, mma_rel(H) * (np.abs(de) @ np.abs(w2))
        g, u = gu[:, :I], gu[:, I:]
        eg, eu = mgu[:, :I], mgu[:, I:]
        s = sigmoid(g)
        silu, dsilu = g * s, s * (1 + g * (1 - s))
        a = silu * u
        dgu = np.concatenate([d * u * dsilu, d * silu], 1)
        ea = U_BF16 * np.abs(a) + 2 * (1.1 * eg * np.abs(u) + np.abs(silu) * eu) + 4e-6 * np.abs(a)
        edg = np.abs(u * dsilu) * md + np.abs(d * dsilu) * eu + 0.5 * np.abs(d * u) * eg
        edu = np.abs(silu) * md + 1.1 * np.abs(d) * eg
        edgu = U_BF16 * np.abs(dgu) + 2 * np.concatenate([edg, edu], 1) + 4e-6 * np.abs(dgu)
        out["dx"][lo:hi] = dgu @ w13
        out["dW13"][e] = dgu.T @ xe
        out["dW2"][e] = de.T @ a
        n = hi - lo
        tol["dx"][lo:hi] = 7 * np.sqrt(edgu ** 2 @ w13 ** 2) + mma_rel(2 * I) * (np.abs(dgu) @ np.abs(w13))
        tol["dW13"][e] = 7 * np.sqrt((edgu ** 2).T @ xe ** 2) + mma_rel(n) * (np.abs(dgu).T @ np.abs(xe))
        tol["dW2"][e] = 7 * np.sqrt((de ** 2).T @ ea ** 2) + mma_rel(n) * (np.abs(de).T @ np.abs(a))
    return out, tol
