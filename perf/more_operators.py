"""The mixture-of-experts block's backward pass as measured cases: the way back
into token order (combine), the experts, the way out of it (dispatch), the
router and the norm.

Each case runs in two forms. With ``own`` false, ``run`` computes the operator
with elementary torch operations in 32 bits, rounded once at the end; with
``own`` true it calls the framework's entry point as a user does, on buffers
kept between calls. ``exact`` computes the same outputs in 64 bits.

Notation: T tokens, E experts, k experts per token, H hidden size, I
intermediate size, R = T k routed rows, sorted by expert. Row r of the sorted
batch holds slot perm[r] = t k + j; inv is the inverse map (-1: a dropped slot).
Sizes are this repository's own workload shapes or generic.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

EPS = 1e-6
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def _combine(name, T, E, k, H, drop=0.0):
    return {"op": "combine", "name": name, "T": T, "E": E, "k": k, "H": H, "drop": drop}


def _dispatch(name, T, E, k, H, drop=0.0, add=False, rows="bf16"):
    return {"op": "dispatch", "name": name, "T": T, "E": E, "k": k, "H": H, "drop": drop, "add": add, "rows": rows}


def _experts(name, T, E, k, H, I, idle=0, drop=0.0):
    return {"op": "experts", "name": name, "T": T, "E": E, "k": k, "H": H, "I": I, "idle": idle, "drop": drop}


def _norm(name, T, H, h="bf16", w="bf16", add=True, unit_offset=False):
    return {"op": "norm", "name": name, "T": T, "H": H, "h": h, "w": w, "add": add, "unit_offset": unit_offset}


def _route(name, T, E, k, H, score="softmax", renorm=True, scale=1.0, add=False):
    return {"op": "route", "name": name, "T": T, "E": E, "k": k, "H": H, "score": score, "renorm": renorm,
            "scale": scale, "add": add}


def listed():
    return [
        # a few tokens of a small fine-tuning batch, some slots dropped by a capacity limit
        _combine("combine_grad_13", 13, 64, 4, 2048, drop=0.1),
        # the large batch: bandwidth
        _combine("combine_grad_large", 8192, 128, 8, 4096),
        # a ragged batch of wide rows, some slots dropped, with the gradient that comes through the router added
        _dispatch("dispatch_grad_1021", 1021, 384, 6, 7168, drop=0.05, add=True),
        # the large batch
        _dispatch("dispatch_grad_large", 8192, 128, 8, 4096),
        # a small batch over a few small experts: launches and short products count
        _experts("experts_grad_64", 64, 16, 4, 1024, 512),
        # an odd batch at sizes that fill no tile, with experts that get no row and slots that are dropped
        _experts("experts_grad_ragged", 1000, 50, 6, 2880, 1472, idle=3, drop=0.02),
        # the large batch: matrix products
        _experts("experts_grad_large", 8192, 128, 8, 4096, 1536),
        # a few rows of the widest stream
        _norm("norm_grad_7", 7, 7168),
        # an odd batch of an fp32 stream
        _norm("norm_grad_2047_fp32", 2047, 7168, h="fp32", w="fp32"),
        # the large batch, the gradient of the residual path added
        _norm("norm_grad_large", 8192, 4096),
        # an odd few tokens over many experts, sigmoid scores
        _route("route_grad_61", 61, 256, 8, 7168, score="sigmoid", scale=2.5),
        # the large batch, with the gradient of a balancing loss on the logits
        _route("route_grad_large", 8192, 128, 8, 4096, add=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(lo, min(hi, _log(rng, lo, hi) // m * m))


def draw(rng):
    op = rng.choice(["combine", "dispatch", "experts", "norm", "route"])
    if op == "norm":
        return _norm(None, _log(rng, 1, 8192), _mult(rng, 256, 4096, 64), h=rng.choice(["bf16", "fp32"]),
                     w=rng.choice(["bf16", "fp32"]), add=rng.random() < 0.6, unit_offset=rng.random() < 0.3)
    if op == "experts":
        E = _log(rng, 4, 128)
        idle = rng.randint(0, E // 4)
        return _experts(None, _log(rng, 8, 4096), E, rng.randint(1, min(8, E - idle)), _mult(rng, 256, 4096, 64),
                        _mult(rng, 128, 1536, 64), idle=idle, drop=rng.choice([0.0, 0.0, 0.1]))
    E = _log(rng, 8, 384)
    k = rng.randint(1, min(8, E))
    if op == "route":
        return _route(None, _log(rng, 1, 8192), _log(rng, 8, 128), k, _mult(rng, 256, 4096, 64),
                      score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                      scale=rng.choice([1.0, 2.5]), add=rng.random() < 0.5)
    T, H, drop = _log(rng, 1, 8192), _mult(rng, 256, 4096, 64), rng.choice([0.0, 0.0, 0.1])
    if op == "combine":
        return _combine(None, T, E, k, H, drop=drop)
    return _dispatch(None, T, E, k, H, drop=drop, add=rng.random() < 0.5, rows=rng.choice(["bf16", "bf16", "fp32"]))


# ----------------------------------------------------------------- inputs

def _randn(g, shape, dtype, std=1.0, mean=0.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(mean, std, generator=g)


def _routing(st, case, seed):
    """k distinct experts a token (the first `idle` never), dropped slots, and
    the sorted batch's maps: expert_offsets, perm, inv."""
    rng = np.random.default_rng(seed * 7919 + 5)
    T, E, k, idle = case["T"], case["E"], case["k"], case.get("idle", 0)
    key = rng.random((T, E))
    key[:, :idle] = 2.0
    ids = np.argsort(key, axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < case["drop"]] = -1
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    order = order[flat[order] >= 0]
    counts = np.bincount(flat[order], minlength=E)
    bounds = np.concatenate([[0], np.cumsum(counts)])
    perm = np.zeros(T * k, dtype=np.int32)
    perm[: len(order)] = order
    inv = np.full(T * k, -1, dtype=np.int32)
    inv[order] = np.arange(len(order), dtype=np.int32)
    st["valid"], st["bounds"] = len(order), bounds
    for name, a in (("offsets", bounds.astype(np.int32)), ("perm", perm), ("inv", inv)):
        st[name] = torch.from_numpy(a).cuda()
    if case["op"] == "experts":
        # the plain form's plan: each expert's rows, padded to the longest
        most = max(1, int(counts.max()))
        st["pad"] = torch.from_numpy(np.minimum(bounds[:-1, None] + np.arange(most), T * k - 1)).cuda()
        st["on"] = torch.from_numpy(np.arange(most) < counts[:, None]).cuda()
        e, i = np.nonzero(np.arange(most) < counts[:, None])
        st["back"] = torch.from_numpy(e * most + i).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    st = {"case": case}
    T, H, op, bf = case["T"], case["H"], case["op"], torch.bfloat16
    if op in ("combine", "dispatch", "experts"):
        _routing(st, case, seed)
        k, rows = case["k"], case["T"] * case["k"]
    if op == "combine":
        st["dout"] = _randn(g, (T, H), bf, 0.01)
        st["y"] = _randn(g, (rows, H), torch.float32, 0.3)
        w = torch.rand((T, k), generator=g, device="cuda") + 0.1
        st["weights"] = w / w.sum(1, keepdim=True)
    elif op == "dispatch":
        st["dxs"] = _randn(g, (rows, H), _DT[case["rows"]], 0.01)
        st["add"] = _randn(g, (T, H), bf, 0.01) if case["add"] else None
    elif op == "experts":
        E, I = case["E"], case["I"]
        st["x"] = _randn(g, (rows, H), bf)
        st["dy"] = _randn(g, (rows, H), bf, 0.01)
        st["W13"] = _randn(g, (E, 2 * I, H), bf, 1.0 / math.sqrt(H))
        st["W2"] = _randn(g, (E, H, I), bf, 1.0 / math.sqrt(I))
    elif op == "norm":
        # rows of a residual stream: each at its own level, a few channels far above the rest
        h = _randn(g, (T, H), torch.float32) * torch.exp(_randn(g, (T, 1), torch.float32, 0.5))
        h[:, ::509] *= 8.0
        st["h"] = h.to(_DT[case["h"]])
        st["w"] = _randn(g, (H,), _DT[case["w"]], 0.1, 0.0 if case["unit_offset"] else 1.0)
        st["dx"] = _randn(g, (T, H), bf, 0.01)
        st["add"] = _randn(g, (T, H), _DT[case["h"]], 0.01) if case["add"] else None
    else:
        E, k = case["E"], case["k"]
        st["x"] = _randn(g, (T, H), bf)
        st["w_router"] = _randn(g, (E, H), bf, 1.0 / math.sqrt(H))
        st["logits"] = st["x"].float() @ st["w_router"].float().T
        st["ids"] = st["logits"].sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
        st["dw"] = _randn(g, (T, k), torch.float32, 0.01)
        st["add"] = _randn(g, (T, E), torch.float32, 1e-4) if case["add"] else None
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """The problem descriptions, outputs and workspaces that a user's program keeps."""
    from moe_routed_expert_routing_gb300 import binding as B

    case = st["case"]
    op, T, H = case["op"], case["T"], case["H"]

    def zeros(shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    st["B"] = B
    if op in ("combine", "dispatch", "experts"):
        E, k = case["E"], case["k"]
        st["experts"] = B.Problem.make(T, E, k, H, case.get("I", 64))
    if op == "combine":
        st["dy_out"], st["dw_out"] = zeros((T * k, H)), zeros((T, k), torch.float32)
    elif op == "dispatch":
        st["dx_out"] = zeros((T, H))
    elif op == "experts":
        st["grad"] = B.ExpertGradProblem.make(st["experts"])
        st["ws"] = zeros(B.moe_expert_backward_workspace_size(st["grad"]), torch.uint8)
        st["dx_out"], st["dW13"], st["dW2"] = zeros((T * k, H)), torch.empty_like(st["W13"]), torch.empty_like(st["W2"])
    elif op == "norm":
        st["norm"] = B.NormProblem.make(T, H, h_dtype=_DT[case["h"]], w_dtype=_DT[case["w"]], eps=EPS,
                                        unit_offset=case["unit_offset"])
        st["ws"] = zeros(B.moe_norm_backward_workspace_size(st["norm"]), torch.uint8)
        st["dh_out"], st["dw_out"] = torch.empty_like(st["h"]), torch.empty_like(st["w"])
    else:
        st["router"] = B.RouterProblem.make(
            T, case["E"], case["k"], H, score=B.MOE_SCORE_SOFTMAX if case["score"] == "softmax" else B.MOE_SCORE_SIGMOID,
            renormalize=case["renorm"], scale=case["scale"])
        st["ws"] = zeros(B.moe_route_backward_workspace_size(st["router"]), torch.uint8)
        st["dx_out"], st["dw_out"] = torch.empty_like(st["x"]), torch.empty_like(st["w_router"])
        st["dl_out"] = torch.empty_like(st["logits"])


# ------------------------------------------------------------- plain forms

def _plain_combine(case, st):
    k = case["k"]
    dout = st["dout"].float()
    kept = (st["inv"] >= 0).float().view(-1, k)
    y = st["y"][st["inv"].clamp(min=0).long()].view(case["T"], k, -1)
    dw = (dout[:, None, :] * y).sum(2) * kept
    slot = st["perm"].long()
    on = (torch.arange(len(slot), device="cuda") < st["valid"]).float()
    dy = dout[slot // k] * (st["weights"].reshape(-1)[slot] * on)[:, None]
    return {"dy": dy.to(torch.bfloat16), "dw": dw}


def _plain_dispatch(case, st):
    k = case["k"]
    kept = (st["inv"] >= 0).float().view(-1, k, 1)
    dx = (st["dxs"][st["inv"].clamp(min=0).long()].float().view(case["T"], k, -1) * kept).sum(1)
    if st["add"] is not None:
        dx = dx + st["add"].float()
    return {"dx": dx.to(torch.bfloat16)}


def _plain_experts(case, st):
    I = case["I"]
    on = st["on"][:, :, None].float()
    x, dy = st["x"][st["pad"]].float() * on, st["dy"][st["pad"]].float() * on
    W13, W2 = st["W13"].float(), st["W2"].float()
    gu = x @ W13.transpose(1, 2)
    g, u = gu[:, :, :I], gu[:, :, I:]
    s = 1.0 / (1.0 + torch.exp(-g))
    da = dy @ W2
    dgu = torch.cat([da * u * s * (1.0 + g * (1.0 - s)), da * g * s], 2)
    dx = torch.zeros((case["T"] * case["k"], case["H"]), device="cuda")
    dx[: st["valid"]] = (dgu @ W13).view(-1, case["H"])[st["back"]]
    return {"dx": dx.to(torch.bfloat16), "dW13": (dgu.transpose(1, 2) @ x).to(torch.bfloat16),
            "dW2": (dy.transpose(1, 2) @ (g * s * u)).to(torch.bfloat16)}


def _plain_norm(case, st):
    h, dx, w = st["h"].float(), st["dx"].float(), st["w"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    q = dx * (w + 1.0 if case["unit_offset"] else w)
    dh = r * (q - h * (r * r * (q * h).mean(1, keepdim=True)))
    if st["add"] is not None:
        dh = dh + st["add"].float()
    return {"dh": dh.to(st["h"].dtype), "dw": (dx * h * r).sum(0).to(st["w"].dtype)}


def _plain_route(case, st):
    logits, ids, dw = st["logits"], st["ids"].long(), st["dw"]
    if case["score"] == "softmax":
        ex = torch.exp(logits - logits.amax(1, keepdim=True))
        score = ex / ex.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    c = score.gather(1, ids)
    if case["renorm"]:
        total = c.sum(1, keepdim=True)
        dc = (dw - (dw * c).sum(1, keepdim=True) / total) / total
    else:
        dc = dw
    dc = torch.zeros_like(logits).scatter_(1, ids, dc * case["scale"])
    if case["score"] == "softmax":
        dl = score * (dc - (dc * score).sum(1, keepdim=True))
    else:
        dl = dc * score * (1.0 - score)
    if st["add"] is not None:
        dl = dl + st["add"]
    return {"dx": (dl @ st["w_router"].float()).to(torch.bfloat16),
            "dw": (dl.T @ st["x"].float()).to(torch.bfloat16), "dl": dl}


_PLAIN = {"combine": _plain_combine, "dispatch": _plain_dispatch, "experts": _plain_experts, "norm": _plain_norm,
          "route": _plain_route}


# ------------------------------------------------------- the framework's calls

def _run_own(st):
    B, op = st["B"], st["case"]["op"]
    if op == "combine":
        B.moe_combine_backward(st["experts"], st["dout"], st["inv"], st["weights"], st["dy_out"], y_sorted=st["y"],
                               d_weights=st["dw_out"])
        return {"dy": st["dy_out"], "dw": st["dw_out"]}
    if op == "dispatch":
        B.moe_dispatch_backward(st["experts"], st["dxs"], st["inv"], st["dx_out"], dx_add=st["add"])
        return {"dx": st["dx_out"]}
    if op == "experts":
        B.moe_expert_backward(st["grad"], st["x"], st["offsets"], st["W13"], st["W2"], st["dy"], st["ws"],
                              dx_sorted=st["dx_out"], dW13=st["dW13"], dW2=st["dW2"])
        return {"dx": st["dx_out"], "dW13": st["dW13"], "dW2": st["dW2"]}
    if op == "norm":
        B.moe_norm_backward(st["norm"], st["h"], st["w"], st["dx"], st["dh_out"], st["ws"], dh_add=st["add"],
                            dw=st["dw_out"])
        return {"dh": st["dh_out"], "dw": st["dw_out"]}
    B.moe_route_backward(st["router"], st["x"], st["w_router"], st["logits"], st["ids"], st["dw"], st["ws"],
                         d_logits_add=st["add"], dx=st["dx_out"], dw_router=st["dw_out"], d_logits=st["dl_out"])
    return {"dx": st["dx_out"], "dw": st["dw_out"], "dl": st["dl_out"]}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state["case"], state)


# ------------------------------------------------------------------- work

def work(case):
    T, H, op = case["T"], case["H"], case["op"]
    if op == "norm":
        hb, wb = (4 if case["h"] == "fp32" else 2), (4 if case["w"] == "fp32" else 2)
        return {"bytes": T * H * ((3 if case["add"] else 2) * hb + 2) + 2 * H * wb, "flops": 11 * T * H}
    if op == "route":
        E, k = case["E"], case["k"]
        return {"bytes": 4 * T * H + 4 * E * H + 4 * T * E * (3 if case["add"] else 2) + 8 * T * k,
                "flops": 4 * T * H * E}
    k = case["k"]
    rows = T * k * (1.0 - case["drop"])
    if op == "combine":
        return {"bytes": int(6 * rows * H + 2 * T * H + 12 * T * k), "flops": int(3 * rows * H)}
    if op == "dispatch":
        b = 4 if case["rows"] == "fp32" else 2
        return {"bytes": int(b * rows * H + 2 * T * H * (2 if case["add"] else 1) + 4 * T * k), "flops": int(rows * H)}
    # the experts that the rows touch on average; every expert's gradient is written
    E, I = case["E"], case["I"]
    live = E - case["idle"]
    touched = live * (1.0 - (1.0 - 1.0 / live) ** rows)
    return {"bytes": int(6 * H * I * (touched + E) + 6 * rows * H), "flops": int(16 * rows * H * I)}


# ---------------------------------------------------------- exact, 64 bits

def _exact_experts(case, st):
    I, b = case["I"], st["bounds"]
    dx = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
    dW13 = torch.zeros(st["W13"].shape, dtype=torch.float64, device="cuda")
    dW2 = torch.zeros(st["W2"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        lo, hi = int(b[e]), int(b[e + 1])
        if lo == hi:
            continue
        x, dy = st["x"][lo:hi].double(), st["dy"][lo:hi].double()
        wg, wu, w2 = st["W13"][e, :I].double(), st["W13"][e, I:].double(), st["W2"][e].double()
        g, u, da = x @ wg.T, x @ wu.T, dy @ w2
        sig = torch.sigmoid(g)
        silu = g * sig
        dg, du = da * u * (sig + silu * (1.0 - sig)), da * silu
        dx[lo:hi] = dg @ wg + du @ wu
        dW13[e, :I], dW13[e, I:] = dg.T @ x, du.T @ x
        dW2[e] = dy.T @ (silu * u)
    return {"dx": dx, "dW13": dW13, "dW2": dW2}


def _exact_route(case, st):
    l, ids, dw = st["logits"].double(), st["ids"].long(), st["dw"].double()
    T, E, k = case["T"], case["E"], case["k"]
    lg = l.gather(1, ids)
    soft = case["score"] == "softmax"
    p = torch.softmax(l, 1) if soft else torch.sigmoid(l)
    c = p.gather(1, ids)
    dl = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    if case["renorm"] and soft:
        # a softmax over the chosen logits alone
        v = torch.softmax(lg, 1)
        dl.scatter_(1, ids, case["scale"] * v * (dw - (dw * v).sum(1, keepdim=True)))
    else:
        if case["renorm"]:
            s = c.sum(1, keepdim=True)
            dc = case["scale"] * (dw * s - (dw * c).sum(1, keepdim=True)) / (s * s)
        else:
            dc = case["scale"] * dw
        if soft:
            dl -= p * (dc * c).sum(1, keepdim=True)
            dl.scatter_add_(1, ids, dc * c)
        else:
            dl.scatter_(1, ids, dc * c * torch.sigmoid(-lg))
    if case["add"]:
        dl += st["add"].double()
    return {"dx": dl @ st["w_router"].double(), "dw": dl.T @ st["x"].double(), "dl": dl}


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    T, H, op = case["T"], case["H"], case["op"]
    if op == "experts":
        return _exact_experts(case, st)
    if op == "route":
        return _exact_route(case, st)
    if op == "norm":
        h, dx, w = st["h"].double(), st["dx"].double(), st["w"].double()
        if case["unit_offset"]:
            w = 1.0 + w
        rms = torch.sqrt(h.square().sum(1, keepdim=True) / H + EPS)
        n = h / rms
        dn = dx * w
        dh = (dn - n * ((dn * n).sum(1, keepdim=True) / H)) / rms
        if case["add"]:
            dh = dh + st["add"].double()
        return {"dh": dh, "dw": (dx * n).sum(0)}
    k, V = case["k"], st["valid"]
    slot = st["perm"][:V].long()
    if op == "combine":
        dy = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        for lo in range(0, V, 8192):
            s = slot[lo: lo + 8192]
            d = st["dout"][s // k].double()
            dy[lo: lo + len(s)] = d * st["weights"].double().view(-1)[s, None]
            dw[s] = (d * st["y"][lo: min(V, lo + 8192)].double()).sum(1)
        return {"dy": dy, "dw": dw.view(T, k)}
    dx = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    dx.index_add_(0, slot // k, st["dxs"][:V].double())
    return {"dx": dx + st["add"].double() if case["add"] else dx}
