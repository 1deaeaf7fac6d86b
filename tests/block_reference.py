"""Plain 64-bit forms (numpy) of the block around the experts -- norms, router,
residual -- for the tests, written from the formulas in include/moe.h."""
from __future__ import annotations

import numpy as np
import torch


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def rms_scale(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps)


def norm(v, w=None, eps=1e-6, unit_offset=False):
    out = v * rms_scale(v, eps)
    if w is not None:
        out = out * (1.0 + w if unit_offset else w)
    return out


def gate_rows(gate, kind):
    """The gate broadcastable over [T, H]; kind 0 none, 1 channel, 2 token, 3 element."""
    if kind == 0:
        return 1.0
    return gate[:, None] if kind == 2 else gate


def residual(h, y, w_post=None, norm_block=False, gate=None, gate_kind=0, scale=1.0, eps=1e-6, unit_offset=False):
    n = norm(y, w_post, eps, unit_offset) if norm_block else y
    step = scale * gate_rows(gate, gate_kind) * n
    return h + step, step


def route(logits, k, score="softmax", renormalize=True, bias=None, n_group=1, topk_group=1, group_top=1, scale=1.0):
    """(ids, weights, margin): margin[t] = the smallest difference of keys that decides row t's result
    (ties that the rule decides by index count as no difference)."""
    l = np.where(np.isnan(logits) | (logits == np.inf), -np.inf, logits.astype(np.float64))
    T, E = l.shape
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if score == "softmax":
            mx = l.max(axis=1, keepdims=True)
            p = np.exp(l - np.where(np.isfinite(mx), mx, 0.0))
            s = p / p.sum(axis=1, keepdims=True)
        else:
            s = 1.0 / (1.0 + np.exp(-l))
    by_score = bias is not None or group_top > 1
    key = np.where(np.isneginf(l), -np.inf, s + (0.0 if bias is None else bias)) if by_score else l
    key = np.where(np.isnan(key), -np.inf, key)
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    margin = np.full(T, np.inf)
    gs = E // n_group
    for t in range(T):
        v = key[t].copy()
        gaps = []
        if n_group > 1:
            top = np.sort(v.reshape(n_group, gs), axis=1)[:, ::-1][:, :group_top].sum(axis=1)
            order = np.lexsort((np.arange(n_group), -top))
            gaps.append(np.abs(np.diff(top[order])[topk_group - 1: topk_group]))
            keep = np.isin(np.arange(E) // gs, order[:topk_group])
            v[~keep] = -np.inf
        order = np.lexsort((np.arange(E), -v))
        with np.errstate(invalid="ignore"):
            gaps.append(np.abs(np.diff(v[order[: k + 1]])))
        chosen = [e for e in order[:k] if v[e] > -np.inf]
        ids[t, : len(chosen)] = chosen
        if chosen:
            if renormalize:
                lg = l[t, chosen] if score == "softmax" else -np.logaddexp(0.0, -l[t, chosen])
                q = np.exp(lg - lg.max())
                w[t, : len(chosen)] = q / q.sum()
            else:
                w[t, : len(chosen)] = s[t, chosen]
        g = np.concatenate(gaps)
        g = g[np.isfinite(g) & (g > 0)]
        margin[t] = g.min() if g.size else np.inf
    return ids, w * scale, margin


def experts(v, ids, weights, W13, W2):
    """y[t] = sum_j w[t, j] * MLP_{ids[t, j]}(v[t]) on unrounded activations; ids -1 are skipped."""
    I = W2.shape[2]
    y = np.zeros_like(v)
    for e in range(W13.shape[0]):
        t, j = np.nonzero(ids == e)
        if len(t):
            gu = v[t] @ W13[e].T
            g, u = gu[:, :I], gu[:, I:]
            y[t] += weights[t, j, None] * ((g / (1.0 + np.exp(-g)) * u) @ W2[e].T)
    return y
