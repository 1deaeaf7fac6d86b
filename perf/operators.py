"""The mixture-of-experts block's operators as measured cases: the norm before
the block, the router, the norm, gate and residual scale after it, and the
whole block for a few tokens.

Each case runs in two forms. With ``own`` false, ``run`` computes the operator
with elementary torch operations in 32 bits, rounded once at the end; with
``own`` true it calls the framework's entry point as a user does, on buffers
kept between calls. ``exact`` computes the same outputs in 64 bits.

Notation: T tokens, E experts, k experts per token, H hidden size, I
intermediate size. Hidden, intermediate and expert counts are this
repository's own workload shapes (decode, prefill, large batch) or generic.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

EPS = 1e-6
_NEG = float("-inf")

# Rows of the router's input whose selection hangs on less than this (in the
# logits' unit of about one standard deviation) are drawn again: the expert
# ids are compared exactly, and two sums of the same products in another
# order differ by far less.
_MARGIN = 1e-3


# ------------------------------------------------------------------ cases

def _norm(name, T, H, h="bf16", w="bf16", unit_offset=False):
    return {"op": "norm", "name": name, "T": T, "H": H, "h": h, "w": w, "unit_offset": unit_offset}


def _norm_residual(name, T, H, h="bf16", w="bf16", post=True, gate="none", scale=1.0, nxt=True):
    return {"op": "norm_residual", "name": name, "T": T, "H": H, "h": h, "w": w, "post": post, "gate": gate,
            "scale": scale, "next": nxt}


def _route(name, T, E, k, H, score="softmax", renorm=True, bias=False, n_group=1, topk_group=1, group_top=1,
           scale=1.0, logits=False):
    return {"op": "route", "name": name, "T": T, "E": E, "k": k, "H": H, "score": score, "renorm": renorm,
            "bias": bias, "n_group": n_group, "topk_group": topk_group, "group_top": group_top, "scale": scale,
            "logits": logits}


def _layer(name, T, E, k, H, I, weights="bf16", score="softmax", bias=False, post=True, gate="none", scale=1.0,
           nxt=False):
    # the residual stream in bf16: the experts' products take bf16 activations
    return {"op": "layer", "name": name, "T": T, "E": E, "k": k, "H": H, "I": I, "weights": weights, "h": "bf16",
            "w": "bf16", "score": score, "renorm": True, "bias": bias, "n_group": 1, "topk_group": 1,
            "group_top": 1, "post": post, "gate": gate, "scale": scale, "next": nxt}


def listed():
    return [
        # one decoded token: a single row, where only latency counts
        _norm("norm_decode1", 1, 7168),
        # a large batch: bandwidth
        _norm("norm_large", 8192, 4096),
        # a few decoded tokens (an odd number), post-norm, the next block's norm in the same pass
        _norm_residual("norm_residual_decode7", 7, 7168),
        # a ragged large batch with the residual stream in fp32, a gate per channel and a residual scale
        _norm_residual("norm_residual_large_fp32", 8191, 4096, h="fp32", w="fp32", gate="channel", scale=0.5),
        # one decoded token over the decode workload's 384 experts
        _route("route_decode1", 1, 384, 6, 7168),
        # an odd few tokens, sigmoid scores with a selection bias and limited groups of experts
        _route("route_groups61", 61, 256, 8, 7168, score="sigmoid", bias=True, n_group=8, topk_group=4, group_top=2,
               scale=2.5),
        # the prefill workload's tokens and experts, scores not renormalised
        _route("route_prefill", 2048, 384, 6, 7168, renorm=False),
        # the large batch, with the logits kept (a load-balancing statistic reads them)
        _route("route_large", 8192, 128, 8, 4096, logits=True),
        # the decode workload as a whole layer: one token and eight
        _layer("layer_decode1", 1, 384, 6, 7168, 3072),
        _layer("layer_decode8", 8, 384, 6, 7168, 3072, nxt=True),
        # a wider decode batch on the large workload's experts, sigmoid scores with a bias, a gate per channel
        _layer("layer_batch64", 64, 128, 8, 4096, 1536, score="sigmoid", bias=True, gate="channel", scale=0.5),
        # a few tokens with quantized expert weights (E4M3 codes, one scale per 32)
        _layer("layer_mxfp8_13", 13, 64, 4, 2048, 1024, weights="mxfp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    v = max(lo, min(hi, _log(rng, lo, hi) // m * m))
    return v - m if v == 3 * 1024 else v    # an intermediate size of the workloads, not a hidden one


def draw(rng):
    op = rng.choice(["norm", "norm_residual", "route", "layer"])
    if op == "norm":
        return _norm(None, _log(rng, 1, 8192), _mult(rng, 256, 7168, 64), h=rng.choice(["bf16", "fp32"]),
                     w=rng.choice(["bf16", "fp32"]), unit_offset=rng.random() < 0.3)
    if op == "norm_residual":
        return _norm_residual(None, _log(rng, 1, 8192), _mult(rng, 256, 7168, 64), h=rng.choice(["bf16", "fp32"]),
                              w=rng.choice(["bf16", "fp32"]), post=rng.random() < 0.7,
                              gate=rng.choice(["none", "channel", "token", "element"]),
                              scale=rng.choice([1.0, 0.5, 0.22]), nxt=rng.random() < 0.5)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        size = _log(rng, 4, 384 // groups) if groups > 1 else _log(rng, 8, 512)
        E = groups * size
        keep = rng.randint(2, groups) if groups > 1 else 1
        score = rng.choice(["softmax", "sigmoid"])
        return _route(None, _log(rng, 1, 8192), E, rng.randint(1, min(8, keep * size)),
                      _mult(rng, 256, 4096, 64), score=score, renorm=rng.random() < 0.7,
                      bias=score == "sigmoid" and rng.random() < 0.5, n_group=groups, topk_group=keep,
                      group_top=rng.choice([1, 2]) if groups > 1 else 1, scale=rng.choice([1.0, 2.5]),
                      logits=rng.random() < 0.3)
    mx = rng.random() < 0.3
    m = 128 if mx else 64
    E = _log(rng, 8, 256)
    return _layer(None, _log(rng, 1, 64), E, rng.randint(1, min(8, E)), _mult(rng, 256, 4096, m),
                  _mult(rng, 256, 2048, m), weights="mxfp8" if mx else "bf16",
                  score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.3, post=rng.random() < 0.7,
                  gate=rng.choice(["none", "channel", "token", "element"]), scale=rng.choice([1.0, 0.5]),
                  nxt=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _randn(g, shape, dtype, std=1.0, mean=0.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(mean, std, generator=g)


def _stream_rows(g, T, H, dtype):
    """Rows of a residual stream: each row at its own level, a few channels far above the rest."""
    h = _randn(g, (T, H), torch.float32)
    h *= torch.exp(_randn(g, (T, 1), torch.float32, 0.5))
    h[:, :: 509] *= 8.0
    return h.to(dtype)


def _norm_weight(g, H, dtype, unit_offset=False):
    return _randn(g, (H,), dtype, 0.1, 0.0 if unit_offset else 1.0)


def _gate_input(g, case):
    T, H = case["T"], case["H"]
    if case["gate"] == "channel":
        return _randn(g, (H,), _DT[case["w"]], 0.2, 0.5)
    if case["gate"] == "token":
        return torch.sigmoid(_randn(g, (T,), torch.float32))
    if case["gate"] == "element":
        return torch.sigmoid(_randn(g, (T, H), torch.float32)).to(torch.bfloat16)
    return None


def _keys64(case, x, w_router, bias):
    """Selection keys in 64 bits, for the margins of the drawn inputs only."""
    l = x.double() @ w_router.double().T
    if bias is None and case["group_top"] == 1:
        return l, 1.0
    s = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
    return (s if bias is None else s + bias.double()), float(s.std()) + 1e-30


def _near_tie(case, x, w_router, bias):
    """Rows whose selection a difference of _MARGIN standard deviations could change."""
    keys, unit = _keys64(case, x, w_router, bias)
    near = torch.zeros(len(keys), dtype=torch.bool, device=keys.device)
    G, k = case["n_group"], case["k"]
    if G > 1:
        by_group = keys.view(len(keys), G, -1)
        top = by_group.sort(2, descending=True).values[:, :, : case["group_top"]].sum(2)
        order = top.sort(1, descending=True)
        if case["topk_group"] < G:
            c = case["topk_group"]
            near |= order.values[:, c - 1] - order.values[:, c] < _MARGIN * unit
        keep = torch.zeros_like(top, dtype=torch.bool).scatter_(1, order.indices[:, : case["topk_group"]], True)
        keys = by_group.masked_fill(~keep[:, :, None], _NEG).reshape(len(keys), -1)
    top = keys.sort(1, descending=True).values[:, : k + 1]
    return near | (top[:, :-1] - top[:, 1:] < _MARGIN * unit).any(1)


def _redraw_near_ties(case, g, rows, normed, w_router, bias):
    """Draw the rows again (in place) whose selection is a near tie."""
    for _ in range(40):
        bad = _near_tie(case, normed(rows), w_router, bias).nonzero()[:, 0]
        if not len(bad):
            return
        if case["op"] == "layer":
            rows[bad] = _stream_rows(g, len(bad), case["H"], rows.dtype)
        else:
            rows[bad] = _randn(g, (len(bad), case["H"]), rows.dtype)


def _mxfp8_weights(g, rows, K):
    """Random weights as E4M3 codes [rows, K] and power-of-two exponents [rows, K/32]."""
    codes = torch.empty((rows, K), dtype=torch.uint8, device="cuda")
    exps = torch.empty((rows, K // 32), dtype=torch.int32, device="cuda")
    for r in range(0, rows, 16384):    # a block of rows at a time: the 32-bit values take four times the codes
        w = _randn(g, (min(16384, rows - r), K // 32, 32), torch.float32, 0.02)
        e = torch.floor(torch.log2(w.abs().amax(2))).clamp(-110, 23) - 8
        q = (w * torch.exp2(-e)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        codes[r: r + len(w)] = q.view(torch.uint8).view(len(w), K)
        exps[r: r + len(w)] = e.to(torch.int32)
    return codes, exps


def _mxfp8_buffer(codes, e):
    """Codes, then the scale bytes by 128-row tile, 128-wide K block, row, sub-block."""
    rows, K = codes.shape
    s = (e + 127).to(torch.uint8).view(rows // 128, 128, K // 128, 4).permute(0, 2, 1, 3)
    return torch.cat([codes.reshape(-1), s.reshape(-1)])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    T, H = case["T"], case["H"]
    st = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_residual", "layer"):
        st["h"] = _stream_rows(g, T, H, _DT[case["h"]])
    if op == "norm":
        st["w"] = _norm_weight(g, H, _DT[case["w"]], case["unit_offset"])
    if op == "norm_residual":
        st["y"] = _randn(g, (T, H), torch.bfloat16, 0.3)
    if op in ("norm_residual", "layer"):
        st["w_post"] = _norm_weight(g, H, _DT[case["w"]]) if case["post"] else None
        st["gate"] = _gate_input(g, case)
        st["w_next"] = _norm_weight(g, H, _DT[case["w"]]) if case["next"] else None
    if op in ("route", "layer"):
        E = case["E"]
        st["w_router"] = _randn(g, (E, H), torch.bfloat16, 1.0 / math.sqrt(H))
        st["bias"] = _randn(g, (E,), torch.float32, 0.05) if case["bias"] else None
        if op == "route":
            st["x"] = _randn(g, (T, H), torch.bfloat16)
            _redraw_near_ties(case, g, st["x"], lambda r: r, st["w_router"], st["bias"])
        else:
            st["w_pre"] = _norm_weight(g, H, _DT[case["w"]])
            _redraw_near_ties(case, g, st["h"], lambda r: _rms64(r.double()) * st["w_pre"].double(),
                              st["w_router"], st["bias"])
    if op == "layer":
        E, I = case["E"], case["I"]
        if case["weights"] == "mxfp8":
            st["W13"] = _mxfp8_weights(g, E * 2 * I, H)
            st["W2"] = _mxfp8_weights(g, E * H, I)
        else:
            st["W13"] = _randn(g, (E, 2 * I, H), torch.bfloat16, 0.02)
            st["W2"] = _randn(g, (E, H, I), torch.bfloat16, 0.02)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """The problem descriptions, outputs and workspaces that a user's program keeps."""
    from moe_routed_expert_routing_gb300 import binding as B

    case = st["case"]
    op, T, H = case["op"], case["T"], case["H"]

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    st["B"] = B
    gates = {"none": B.MOE_GATE_NONE, "channel": B.MOE_GATE_CHANNEL, "token": B.MOE_GATE_TOKEN,
             "element": B.MOE_GATE_ELEMENT}
    if op != "route":
        st["norm"] = B.NormProblem.make(
            T, H, h_dtype=_DT[case["h"]], w_dtype=_DT[case["w"]], eps=EPS,
            unit_offset=case.get("unit_offset", False), norm_block=case.get("post", False),
            gate=gates[case.get("gate", "none")], residual_scale=case.get("scale", 1.0))
    if op == "norm":
        st["x_out"] = empty((T, H), torch.bfloat16)
    if op in ("norm_residual", "layer"):
        st["h_out"] = empty((T, H), _DT[case["h"]])
        st["x_next"] = empty((T, H), torch.bfloat16) if case["next"] else None
    if op in ("route", "layer"):
        E, k = case["E"], case["k"]
        st["router"] = B.RouterProblem.make(
            T, E, k, H, score=B.MOE_SCORE_SOFTMAX if case["score"] == "softmax" else B.MOE_SCORE_SIGMOID,
            renormalize=case["renorm"], n_group=case["n_group"], topk_group=case["topk_group"],
            group_top=case["group_top"], scale=case["scale"] if op == "route" else 1.0)
        st["ids"] = empty((T, k), torch.int32)
        st["weights"] = empty((T, k), torch.float32)
    if op == "route":
        st["logits"] = empty((T, case["E"]), torch.float32) if case["logits"] else None
        st["ws"] = torch.zeros(B.moe_route_workspace_size(st["router"]), dtype=torch.uint8, device="cuda")
    if op == "layer":
        mx = case["weights"] == "mxfp8"
        st["experts"] = B.Problem.make(T, case["E"], case["k"], H, case["I"],
                                       weight_layout=B.MOE_WEIGHTS_MXFP8 if mx else B.MOE_WEIGHTS_ROW_MAJOR)
        st["layer"] = B.LayerProblem.make(st["experts"], st["router"], st["norm"])
        if mx:
            st["W13"], st["W2"] = _mxfp8_buffer(*st["W13"]), _mxfp8_buffer(*st["W2"])
        st["expert_offsets"] = empty((case["E"] + 1,), torch.int32)
        st["perm"] = empty((T * case["k"],), torch.int32)
        st["ws"] = torch.zeros(B.moe_layer_workspace_size(st["layer"]), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------- plain forms

def _rms(v):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


def _plain_norm(h, w, unit_offset):
    w = w.float()
    return _rms(h.float()) * (w + 1.0 if unit_offset else w)


def _plain_residual(case, st, y):
    n = y if st["w_post"] is None else _rms(y) * st["w_post"].float()
    if st["gate"] is not None:
        gate = st["gate"].float()
        n = n * (gate[:, None] if case["gate"] == "token" else gate)
    h = st["h"].float() + case["scale"] * n
    nxt = None if st["w_next"] is None else (_rms(h) * st["w_next"].float()).to(torch.bfloat16)
    return h.to(st["h"].dtype), nxt


def _plain_route(case, x, w_router, bias, scale):
    logits = x @ w_router.float().T
    if case["score"] == "softmax":
        ex = torch.exp(logits - logits.amax(1, keepdim=True))
        score = ex / ex.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    # without a bias or sums over a group, the logits are in the scores' order
    key = logits if bias is None and case["group_top"] == 1 else score if bias is None else score + bias
    if case["n_group"] > 1:
        by_group = key.view(len(key), case["n_group"], -1)
        value = by_group.sort(2, descending=True).values[:, :, : case["group_top"]].sum(2)
        best = value.sort(dim=1, descending=True, stable=True).indices[:, : case["topk_group"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
        key = by_group.masked_fill(~keep[:, :, None], _NEG).reshape(len(key), -1)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, : case["k"]]
    weights = score.gather(1, ids)
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    return ids.to(torch.int32), weights * scale, logits


def _plain_weights(case, st, which, ids):
    """The weight matrices of the chosen experts (a device list), in 32 bits."""
    w = st[which]
    if case["weights"] != "mxfp8":
        return w[ids].float()
    E, K = case["E"], (case["H"] if which == "W13" else case["I"])
    codes = w[0].view(E, -1, K)[ids].view(torch.float8_e4m3fn).float()
    scale = torch.exp2(w[1].view(E, -1, K // 32)[ids].float())
    return (codes.view(len(ids), -1, K // 32, 32) * scale[..., None]).view(len(ids), -1, K)


def _plain_experts(case, st, x, ids, weights):
    T, k, I = case["T"], case["k"], case["I"]
    flat = ids.reshape(-1).long()
    rows = x[:, None, :].expand(T, k, -1).reshape(T * k, -1, 1)
    gu = (_plain_weights(case, st, "W13", flat) @ rows)[:, :, 0]
    act = gu[:, :I] / (1.0 + torch.exp(-gu[:, :I])) * gu[:, I:]
    y = (_plain_weights(case, st, "W2", flat) @ act[:, :, None])[:, :, 0]
    return (weights[:, :, None] * y.view(T, k, -1)).sum(1)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "norm":
        return _plain_norm(st["h"], st["w"], case["unit_offset"]).to(torch.bfloat16)
    if op == "norm_residual":
        h, nxt = _plain_residual(case, st, st["y"].float())
        return {"h": h} if nxt is None else {"h": h, "x_next": nxt}
    if op == "route":
        ids, weights, logits = _plain_route(case, st["x"].float(), st["w_router"], st["bias"], case["scale"])
        out = {"ids": ids, "weights": weights}
        if case["logits"]:
            out["logits"] = logits
        return out
    x = _plain_norm(st["h"], st["w_pre"], False)
    ids, weights, _ = _plain_route(case, x, st["w_router"], st["bias"], 1.0)
    h, nxt = _plain_residual(case, st, _plain_experts(case, st, x, ids, weights))
    out = {"h": h, "ids": ids, "weights": weights}
    if nxt is not None:
        out["x_next"] = nxt
    return out


# ------------------------------------------------------- the framework's calls

def _run_own(st):
    B, case = st["B"], st["case"]
    op = case["op"]
    if op == "norm":
        B.moe_norm(st["norm"], st["h"], st["w"], st["x_out"])
        return st["x_out"]
    if op == "norm_residual":
        B.moe_norm_residual(st["norm"], st["h"], st["y"], st["h_out"], w_post=st["w_post"], gate=st["gate"],
                            w_next=st["w_next"], x_next=st["x_next"])
        return {"h": st["h_out"]} if st["x_next"] is None else {"h": st["h_out"], "x_next": st["x_next"]}
    if op == "route":
        B.moe_route(st["router"], st["x"], st["w_router"], st["ids"], st["weights"], st["ws"], bias=st["bias"],
                    logits=st["logits"])
        out = {"ids": st["ids"], "weights": st["weights"]}
        if case["logits"]:
            out["logits"] = st["logits"]
        return out
    B.moe_layer(st["layer"], st["h"], st["w_pre"], st["w_router"], st["W13"], st["W2"], st["ids"], st["weights"],
                st["expert_offsets"], st["perm"], st["h_out"], st["ws"], bias=st["bias"], w_post=st["w_post"],
                gate=st["gate"], w_next=st["w_next"], x_next=st["x_next"])
    out = {"h": st["h_out"], "ids": st["ids"], "weights": st["weights"]}
    if st["x_next"] is not None:
        out["x_next"] = st["x_next"]
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work

def work(case):
    T, H = case["T"], case["H"]
    hb = 4 if case.get("h") == "fp32" else 2
    wb = 4 if case.get("w") == "fp32" else 2
    op = case["op"]
    if op == "norm":
        return {"bytes": T * H * (hb + 2) + H * wb, "flops": 4 * T * H}
    b = f = 0
    if op in ("norm_residual", "layer"):
        b += T * H * (2 * hb + (2 if case["next"] else 0)) + H * wb * (int(case["post"]) + int(case["next"]))
        b += {"none": 0, "channel": H * wb, "token": 4 * T, "element": 2 * T * H}[case["gate"]]
        f += T * H * (3 + (4 if case["post"] else 0) + (4 if case["next"] else 0))
    if op == "norm_residual":
        return {"bytes": b + 2 * T * H, "flops": f}
    E, k = case["E"], case["k"]
    b += 2 * E * H + 8 * T * k + (4 * E if case["bias"] else 0)
    f += 2 * T * H * E
    if op == "route":
        return {"bytes": b + 2 * T * H + (4 * T * E if case["logits"] else 0), "flops": f}
    # the experts that T tokens touch on average when each picks k of E at random
    touched = E * (1.0 - (1.0 - k / E) ** T)
    per = 3 * H * case["I"] * (2 if case["weights"] == "bf16" else 1 + 1 / 32)
    return {"bytes": int(b + H * wb + touched * per), "flops": int(f + 6 * T * k * H * case["I"] + 4 * T * H)}


# ---------------------------------------------------------- exact, 64 bits

def _rms64(v):
    return v / torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + EPS)


def _exact_select(case, logits, bias, scale):
    """Selection and weights of one batch of logits (numpy, 64 bits), row by row."""
    G, k = case["n_group"], case["k"]
    T, E = logits.shape
    if case["score"] == "softmax":
        p = np.exp(logits - logits.max(1, keepdims=True))
        score = p / p.sum(1, keepdims=True)
    else:
        score = 1.0 / (1.0 + np.exp(-logits))
    key = score + (0.0 if bias is None else bias)
    ids = np.empty((T, k), dtype=np.int32)
    index = np.arange(E)
    for t in range(T):
        v = key[t]
        if G > 1:
            parts = np.sort(v.reshape(G, -1), axis=1)[:, ::-1][:, : case["group_top"]].sum(1)
            kept = np.lexsort((np.arange(G), -parts))[: case["topk_group"]]
            v = np.where(np.isin(index // (E // G), kept), v, -np.inf)
        ids[t] = np.lexsort((index, -v))[:k]
    w = np.take_along_axis(score, ids.astype(np.int64), 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return ids, w * scale


def _exact_expert_weights(case, st, which, e):
    w = st[which]
    if case["weights"] != "mxfp8":
        return w[e].double()
    K = case["H"] if which == "W13" else case["I"]
    n = w[0].shape[0] // case["E"]
    codes = w[0][e * n: (e + 1) * n].view(torch.float8_e4m3fn).double()
    return codes * torch.repeat_interleave(torch.exp2(w[1][e * n: (e + 1) * n].double()), 32, dim=1)


def _exact_residual(case, st, y):
    n = y
    if case["post"]:
        n = _rms64(y) * st["w_post"].double()
    if case["gate"] != "none":
        gate = st["gate"].double()
        n = n * (gate.unsqueeze(1) if case["gate"] == "token" else gate)
    h = st["h"].double() + n * case["scale"]
    out = {"h": h}
    if case["next"]:
        out["x_next"] = _rms64(h) * st["w_next"].double()
    return out


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    op = case["op"]
    if op == "norm":
        w = st["w"].double() + (1.0 if case["unit_offset"] else 0.0)
        return _rms64(st["h"].double()) * w
    if op == "norm_residual":
        return _exact_residual(case, st, st["y"].double())
    x = st["x"].double() if op == "route" else _rms64(st["h"].double()) * st["w_pre"].double()
    logits = x @ st["w_router"].double().T
    bias = None if st["bias"] is None else st["bias"].double().cpu().numpy()
    ids, w = _exact_select(case, logits.cpu().numpy(), bias, case["scale"] if op == "route" else 1.0)
    if op == "route":
        out = {"ids": torch.from_numpy(ids).cuda(), "weights": torch.from_numpy(w).cuda()}
        if case["logits"]:
            out["logits"] = logits
        return out
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
    I = case["I"]
    for e in sorted(set(ids.reshape(-1).tolist())):
        t, j = np.nonzero(ids == e)
        rows = torch.from_numpy(t).cuda()
        gu = x[rows] @ _exact_expert_weights(case, st, "W13", e).T
        a = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y[rows] += torch.from_numpy(w[t, j]).cuda()[:, None] * (a @ _exact_expert_weights(case, st, "W2", e).T)
    out = _exact_residual(case, st, y)
    order = {"h": out["h"], "ids": torch.from_numpy(ids).cuda(), "weights": torch.from_numpy(w).cuda()}
    if "x_next" in out:
        order["x_next"] = out["x_next"]
    return order
