"""The block's gradients on the GPU against 64-bit forms, at the sizes, types,
strides and masks where they can go wrong.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32; bf16 outputs
add half a step of their own, 2^-8):

* combine: dy is one product, u; dw is a sum of H products, in a thread at most
  H / 256 + 8 of them one after the other, then 13 levels: (H / 256 + 21) u of the
  sum of |products|.
* dispatch: k + 1 terms one after the other: (k + 1) u of the sum of |terms|.
* norm: the row sums run over at most 64 terms a thread and 10 levels, 74 u;
  r another 4 u, and six roundings: 90 u = 5.4e-6 of the terms; dw adds its own sum over the
  rows, (T / 152 + 64) u at most (rows of a block one after the other, then blocks).
* route: the exponentials' arguments are off by u times their size (at most 40
  here), two exponentials and the sums some 20 u: 64 u = 4e-6 of the terms, and the products
  2^-16 of |dl| each (two bf16 parts) and what the tensor cores' sums lose.
* experts: backward_reference.experts.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import backward_reference as back
import block_reference as ref
from parity import bf16_half_ulp

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
DT = {"bf16": BF, "fp32": F32}


@pytest.fixture(scope="module")
def B():
    from moe_routed_expert_routing_gb300.build import build
    build()
    from moe_routed_expert_routing_gb300 import binding
    return binding


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, shape, dtype=BF, std=1.0, mean=0.0):
    return torch.empty(shape, device="cuda").normal_(mean, std, generator=g).to(dtype)


def empty(shape, dtype=BF, fill=7.0):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


def check(got, want, tol, what):
    dtype = got.dtype
    got = ref.f64(got)
    if not got.size:
        return
    assert np.isfinite(got).all(), what
    if dtype == BF:
        tol = tol * (1 + 2.0 ** -8) + bf16_half_ulp(want) * (1 + 1e-3)
    err, tol = np.abs(got - want), np.broadcast_to(tol + 1e-30, want.shape)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), f"{what}: error {err[worst]:.3e} at {worst}, allowed {tol[worst]:.3e}"


def count(n):
    return None if n is None else torch.tensor([n], dtype=I32, device="cuda")


def routing(seed, T, E, k, drop=0.0):
    """ids with dropped slots, and the sorted batch's maps, by the dispatch's rule."""
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    flat = ids.reshape(-1)
    order = np.concatenate([np.nonzero(flat == e)[0] for e in range(E)]).astype(np.int64)
    inv = np.full(T * k, -1, dtype=np.int32)
    inv[order] = np.arange(len(order))
    return ids, inv, len(order)


ROWS = [(1, 4, 1, 64, 0.0), (1, 8, 8, 7168, 0.3), (5, 16, 3, 192, 0.5), (37, 64, 6, 2880, 0.1), (129, 384, 6, 1024, 0.0),
        (600, 20, 9, 512, 0.2), (3, 64, 64, 320, 0.2), (2, 4, 2, 9216, 1.0), (2, 4, 2, 33024, 0.0)]


# ------------------------------------------------------------------ combine and dispatch

@pytest.mark.parametrize("T,E,k,H,drop", ROWS)
def test_combine_backward(B, T, E, k, H, drop):
    _, inv, valid = routing(T + H, T, E, k, drop)
    g = gen(T + k)
    p = B.Problem.make(T, E, k, H, 64, capacity=T * k + 3)
    dout, y = randn(g, (T, H)), randn(g, (p.cap, H), F32)
    w = torch.rand((T, k), generator=g, device="cuda")
    dy, dw = empty((p.cap, H)), empty((T, k), F32)
    d_inv = torch.from_numpy(inv).cuda()
    B.moe_combine_backward(p, dout, d_inv, w, dy, y_sorted=y, d_weights=dw)
    rows, want_dw, mag = back.combine(ref.f64(dout), ref.f64(y), inv, ref.f64(w))
    check(dw, want_dw, (H / 256 + 21) * U * mag, "dw")
    if valid:
        want = np.stack([rows[r] for r in range(valid)])
        check(dy[:valid], want, U * np.abs(want), "dy")
    assert (dy[valid:] == 7.0).all()
    # without the weights' gradient: the same rows
    dy2 = empty((p.cap, H))
    B.moe_combine_backward(p, dout, d_inv, w, dy2)
    assert torch.equal(dy, dy2)


@pytest.mark.parametrize("T,E,k,H,drop", ROWS)
@pytest.mark.parametrize("rows", ["bf16", "fp32"])
def test_dispatch_backward(B, T, E, k, H, drop, rows):
    _, inv, valid = routing(T + H, T, E, k, drop)
    g = gen(T + k)
    p = B.Problem.make(T, E, k, H, 64)
    dxs, add = randn(g, (p.cap, H), DT[rows]), randn(g, (T, H))
    dxs[valid:] = float("nan")           # rows that no slot holds
    d_inv = torch.from_numpy(inv).cuda()
    for other in (None, add):
        dx = empty((T, H))
        B.moe_dispatch_backward(p, dxs, d_inv, dx, dx_add=other)
        want, mag = back.dispatch(ref.f64(dxs), inv, T, k, ref.f64(other))
        check(dx, want, (k + 1) * U * mag, "dx")
    same = add.clone()                   # in place
    B.moe_dispatch_backward(p, dxs, d_inv, same, dx_add=same)
    assert torch.equal(same, dx)


def test_rows_of_absent_tokens_stay(B):
    T, E, k, H = 9, 8, 2, 256
    _, inv, _ = routing(3, T, E, k)
    g = gen(3)
    p = B.Problem.make(T, E, k, H, 64)
    dout, y, w = randn(g, (T, H)), randn(g, (T * k, H), F32), torch.rand((T, k), generator=g, device="cuda")
    d_inv = torch.from_numpy(inv).cuda()
    full_dy, full_dw, full_dx = empty((T * k, H)), empty((T, k), F32), empty((T, H))
    B.moe_combine_backward(p, dout, d_inv, w, full_dy, y_sorted=y, d_weights=full_dw)
    B.moe_dispatch_backward(p, full_dy, d_inv, full_dx)
    for n, rows in [(4, 4), (0, 0), (-2, 0), (50, T)]:
        dy, dw, dx = empty((T * k, H)), empty((T, k), F32), empty((T, H))
        B.moe_combine_backward(p, dout, d_inv, w, dy, y_sorted=y, d_weights=dw, d_num_tokens=count(n))
        B.moe_dispatch_backward(p, full_dy, d_inv, dx, d_num_tokens=count(n))
        here = torch.from_numpy(inv[: rows * k].astype(np.int64)).cuda()
        away = torch.from_numpy(inv[rows * k:].astype(np.int64)).cuda()
        assert torch.equal(dy[here], full_dy[here]) and (dy[away] == 7.0).all()
        assert torch.equal(dw[:rows], full_dw[:rows]) and (dw[rows:] == 7.0).all()
        assert torch.equal(dx[:rows], full_dx[:rows]) and (dx[rows:] == 7.0).all()


def test_rows_outside_the_batch_count_as_dropped(B):
    T, E, k, H = 2, 4, 2, 64
    p = B.Problem.make(T, E, k, H, 64)
    inv = torch.tensor([0, 4, 1 << 30, -7], dtype=I32, device="cuda")    # cap is 4
    g = gen(1)
    dout, y, w = randn(g, (T, H)), randn(g, (4, H), F32), torch.rand((T, k), generator=g, device="cuda")
    dy, dw, dx = empty((4, H)), empty((T, k), F32), empty((T, H))
    B.moe_combine_backward(p, dout, inv, w, dy, y_sorted=y, d_weights=dw)
    B.moe_dispatch_backward(p, dy, inv, dx)
    assert (dy[1:] == 7.0).all() and (dw.view(-1)[1:] == 0).all()
    assert torch.equal(dx[0], dy[0]) and (dx[1] == 0).all()


# ------------------------------------------------------------------ experts

def expert_inputs(seed, counts, H, I, spare=0):
    g = gen(seed)
    bounds = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows, E = int(bounds[-1]), len(counts)
    x, dy = randn(g, (rows + spare, H)), randn(g, (rows + spare, H), BF, 0.5)
    x[rows:], dy[rows:] = float("nan"), float("nan")       # rows past the last expert's
    W13, W2 = randn(g, (E, 2 * I, H), BF, H ** -0.5), randn(g, (E, H, I), BF, I ** -0.5)
    return x, dy, W13, W2, bounds


def expert_problem(B, counts, H, I, spare=0, **kw):
    rows, E = int(sum(counts)) + spare, len(counts)
    return B.ExpertGradProblem.make(B.Problem.make(max(rows, 1), E, 1, H, I), **kw)


def run_experts(B, p, x, dy, W13, W2, bounds, **out):
    ws = torch.zeros(B.moe_expert_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    B.moe_expert_backward(p, x, torch.from_numpy(bounds).cuda(), W13, W2, dy, ws, **out)
    assert B.moe_last_device_error(ws) == 0
    return out


@pytest.mark.parametrize("counts,H,I,spare", [
    ([1], 64, 64, 0),
    ([0, 3, 0], 64, 64, 5),
    ([16, 0, 15, 17], 192, 64, 0),
    ([63, 64, 65, 1, 127, 128, 129], 128, 192, 100),
    ([255, 256, 257], 320, 448, 0),
    ([0, 0, 0, 515, 0], 512, 256, 1),
    ([40, 30, 20, 10, 5, 2, 1, 0] * 4, 256, 128, 64),
    ([300, 7], 1088, 576, 0),
    ([0, 0], 128, 64, 9),                 # nothing routed
    ([1500, 1300], 256, 128, 3),          # many K blocks a tile
    ([256, 384, 385, 513], 192, 128, 0),  # a last tile of 128 rows, of 129, of 1
])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_expert_backward(B, counts, H, I, spare, kind):
    x, dy, W13, W2, bounds = expert_inputs(sum(counts) + H, counts, H, I, spare)
    p = expert_problem(B, counts, H, I, spare, dx_dtype=DT[kind], dw_dtype=DT[kind])
    out = run_experts(B, p, x, dy, W13, W2, bounds, dx_sorted=empty(x.shape, DT[kind]),
                      dW13=empty(W13.shape, DT[kind], float("nan")), dW2=empty(W2.shape, DT[kind], float("nan")))
    n = int(bounds[-1])
    want, tol = back.experts(ref.f64(x[:n]), ref.f64(dy[:n]), ref.f64(W13), ref.f64(W2), bounds)
    check(out["dx_sorted"][:n], want["dx"], tol["dx"], "dx")
    check(out["dW13"], want["dW13"], tol["dW13"], "dW13")
    check(out["dW2"], want["dW2"], tol["dW2"], "dW2")
    assert (out["dx_sorted"][n:] == 7.0).all()


@pytest.mark.parametrize("H,I", [(64, 64), (192, 128), (384, 320)])
def test_expert_backward_halved_tiles(B, H, I):
    """Up to 128 rows an expert on average: tiles split between the CTAs of a pair at 32 or 64 rows, whole
    ones beside them, even and odd numbers of K blocks."""
    counts = [1, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 255, 256, 257, 0, 320]
    assert 24 * len(counts) < sum(counts) + 5 <= 128 * len(counts)
    x, dy, W13, W2, bounds = expert_inputs(H + I, counts, H, I, 5)
    p = expert_problem(B, counts, H, I, 5, dx_dtype=F32, dw_dtype=F32)
    out = run_experts(B, p, x, dy, W13, W2, bounds, dx_sorted=empty(x.shape, F32), dW13=empty(W13.shape, F32),
                      dW2=empty(W2.shape, F32))
    n = int(bounds[-1])
    want, tol = back.experts(ref.f64(x[:n]), ref.f64(dy[:n]), ref.f64(W13), ref.f64(W2), bounds)
    check(out["dx_sorted"][:n], want["dx"], tol["dx"], "dx")
    check(out["dW13"], want["dW13"], tol["dW13"], "dW13")
    check(out["dW2"], want["dW2"], tol["dW2"], "dW2")
    assert (out["dx_sorted"][n:] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_expert_backward_many_units(B, kind):
    """More than 128 rows an expert and more than six tiles of the products for each CTA pair."""
    counts, H, I = [200, 0, 513], 4096, 704
    tiles = 3 * (6 * 16 + 16 * 3) + 3 * 16
    assert tiles > 6 * 76 and sum(counts) > 128 * len(counts)
    x, dy, W13, W2, bounds = expert_inputs(12, counts, H, I)
    p = expert_problem(B, counts, H, I, dx_dtype=DT[kind], dw_dtype=DT[kind])
    out = run_experts(B, p, x, dy, W13, W2, bounds, dx_sorted=empty(x.shape, DT[kind]),
                      dW13=empty(W13.shape, DT[kind], float("nan")), dW2=empty(W2.shape, DT[kind], float("nan")))
    want, tol = back.experts(ref.f64(x), ref.f64(dy), ref.f64(W13), ref.f64(W2), bounds)
    for n, key in (("dx_sorted", "dx"), ("dW13", "dW13"), ("dW2", "dW2")):
        check(out[n], want[key], tol[key], n)


def test_expert_backward_one_output_at_a_time(B):
    counts, H, I = [70, 0, 130], 256, 192
    x, dy, W13, W2, bounds = expert_inputs(5, counts, H, I)
    p = expert_problem(B, counts, H, I)
    outs = {"dx_sorted": x.shape, "dW13": W13.shape, "dW2": W2.shape}
    full = run_experts(B, p, x, dy, W13, W2, bounds, **{n: empty(s) for n, s in outs.items()})
    again = run_experts(B, p, x, dy, W13, W2, bounds, **{n: empty(s) for n, s in outs.items()})
    for n, s in outs.items():
        assert torch.equal(full[n], again[n]), n          # the same bits every time
        one = run_experts(B, p, x, dy, W13, W2, bounds, **{n: empty(s)})
        assert torch.equal(one[n], full[n]), n


def test_expert_backward_accumulates(B):
    counts, H, I = [70, 0, 33], 192, 128
    x, dy, W13, W2, bounds = expert_inputs(6, counts, H, I)
    p = expert_problem(B, counts, H, I, dw_dtype=F32)
    out = run_experts(B, p, x, dy, W13, W2, bounds, dW13=empty(W13.shape, F32), dW2=empty(W2.shape, F32))
    p = expert_problem(B, counts, H, I, dw_dtype=F32, accumulate=True)
    g = gen(7)
    old = {"dW13": randn(g, W13.shape, F32), "dW2": randn(g, W2.shape, F32)}
    acc = run_experts(B, p, x, dy, W13, W2, bounds, **{n: v.clone() for n, v in old.items()})
    for n in old:
        assert torch.equal(acc[n], old[n] + out[n]), n
        assert torch.equal(acc[n][1], old[n][1]), n       # an expert without rows adds nothing


def test_expert_backward_keeps_experts_apart(B):
    """Rows of infinities and NaN in one expert leave every other expert's gradients as they are."""
    counts, H, I = [65, 50, 3, 200], 128, 64
    x, dy, W13, W2, bounds = expert_inputs(8, counts, H, I)
    p = expert_problem(B, counts, H, I)
    names = {"dx_sorted": x.shape, "dW13": W13.shape, "dW2": W2.shape}
    clean = run_experts(B, p, x, dy, W13, W2, bounds, **{n: empty(s) for n, s in names.items()})
    x2, dy2 = x.clone(), dy.clone()
    x2[65:115], dy2[65:115] = float("nan"), float("inf")
    got = run_experts(B, p, x2, dy2, W13, W2, bounds, **{n: empty(s) for n, s in names.items()})
    for e in (0, 2, 3):
        assert torch.equal(got["dW13"][e], clean["dW13"][e]) and torch.equal(got["dW2"][e], clean["dW2"][e])
    keep = torch.ones(len(x), dtype=torch.bool, device="cuda")
    keep[65:115] = False
    assert torch.equal(got["dx_sorted"][keep], clean["dx_sorted"][keep])
    assert torch.isnan(got["dW13"][1]).any()


def test_expert_backward_offsets_are_clamped(B):
    counts, H, I = [20, 12], 64, 64
    x, dy, W13, W2, bounds = expert_inputs(9, counts, H, I)
    p = expert_problem(B, counts, H, I)
    wild = np.array([-5, 20, 1 << 30], dtype=np.int32)
    a = run_experts(B, p, x, dy, W13, W2, bounds, dx_sorted=empty(x.shape), dW13=empty(W13.shape))
    b = run_experts(B, p, x, dy, W13, W2, wild, dx_sorted=empty(x.shape), dW13=empty(W13.shape))
    assert torch.equal(a["dx_sorted"], b["dx_sorted"]) and torch.equal(a["dW13"], b["dW13"])


def test_expert_backward_extreme_gates(B):
    """Gates far out, where the exponential overflows or the slope vanishes, give finite gradients."""
    counts, H, I = [40], 64, 64
    x, dy, W13, W2, bounds = expert_inputs(10, counts, H, I)
    W13[:, :I] *= 60.0
    p = expert_problem(B, counts, H, I, dx_dtype=F32, dw_dtype=F32)
    out = run_experts(B, p, x, dy, W13, W2, bounds, dx_sorted=empty(x.shape, F32), dW13=empty(W13.shape, F32),
                      dW2=empty(W2.shape, F32))
    want, tol = back.experts(ref.f64(x), ref.f64(dy), ref.f64(W13), ref.f64(W2), bounds)
    for n, key in (("dx_sorted", "dx"), ("dW13", "dW13"), ("dW2", "dW2")):
        check(out[n], want[key], tol[key], n)


def test_expert_backward_into_the_middle_of_a_buffer(B):
    """Outputs and inputs that are 16-byte aligned and no more."""
    counts, H, I = [40, 100], 128, 64
    x, dy, W13, W2, bounds = expert_inputs(11, counts, H, I)
    for dt in (BF, F32):
        p = expert_problem(B, counts, H, I, dx_dtype=dt, dw_dtype=dt)
        names = {"dx_sorted": x.shape, "dW13": W13.shape, "dW2": W2.shape}
        want = run_experts(B, p, x, dy, W13, W2, bounds, **{n: empty(s, dt) for n, s in names.items()})

        def shifted(t):
            step = 16 // t.element_size()
            buf = torch.zeros(t.numel() + step, dtype=t.dtype, device="cuda")
            buf[step:] = t.reshape(-1)
            return buf[step:].view(t.shape)

        got = run_experts(B, p, shifted(x), shifted(dy), shifted(W13), shifted(W2), bounds,
                          **{n: shifted(empty(s, dt)) for n, s in names.items()})
        for n in names:
            assert torch.equal(got[n], want[n]), n


def test_offsets_beyond_32_bits(B):
    """Rows and weights whose elements pass 2^31: the last ones come out right."""
    T, k, H, E = 8192, 9, 32768, 16
    _, inv, valid = routing(5, T, E, k)
    g = gen(5)
    p = B.Problem.make(T, E, k, H, 64)
    assert p.cap * H > 2 ** 31
    dout, w = randn(g, (T, H)), torch.rand((T, k), generator=g, device="cuda")
    y = torch.empty((p.cap, H), device="cuda").normal_(generator=g)
    dy, dw, dx, d_inv = empty((p.cap, H)), empty((T, k), F32), empty((T, H)), torch.from_numpy(inv).cuda()
    B.moe_combine_backward(p, dout, d_inv, w, dy, y_sorted=y, d_weights=dw)
    B.moe_dispatch_backward(p, dy, d_inv, dx)
    slot = np.argsort(inv)[-3:]                       # the slots of the last rows of the batch
    for s in slot:
        t, r = int(s) // k, int(inv[s])
        a, b = ref.f64(dout[t]), ref.f64(y[r])
        check(dy[r], float(w.view(-1)[s]) * a, U * np.abs(a), "dy")
        assert abs(float(dw.view(-1)[s]) - (a * b).sum()) <= (H / 256 + 21) * U * np.abs(a * b).sum()
        rows = [int(v) for v in inv[t * k: t * k + k]]
        terms = ref.f64(dy[rows])
        check(dx[t], terms.sum(0), (k + 1) * U * np.abs(terms).sum(0), "dx")
    del y, dy, dx, dout
    E, H, I = 264, 4096, 1024
    counts = [0] * (E - 2) + [70, 30]
    x, dgy, _, _, bounds = expert_inputs(12, [70, 30], H, I)
    bounds = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    W13, W2 = randn(g, (E, 2 * I, H), BF, H ** -0.5), randn(g, (E, H, I), BF, I ** -0.5)
    assert W13.numel() > 2 ** 31
    p = expert_problem(B, counts, H, I)
    out = run_experts(B, p, x, dgy, W13, W2, bounds, dx_sorted=empty(x.shape), dW13=torch.empty_like(W13),
                      dW2=torch.empty_like(W2))
    want, tol = back.experts(ref.f64(x), ref.f64(dgy), ref.f64(W13[-2:]), ref.f64(W2[-2:]), [0, 70, 100])
    check(out["dx_sorted"], want["dx"], tol["dx"], "dx")
    check(out["dW13"][-2:], want["dW13"], tol["dW13"], "dW13")
    check(out["dW2"][-2:], want["dW2"], tol["dW2"], "dW2")
    assert not out["dW13"][: E - 2].any() and not out["dW2"][: E - 2].any()


# ------------------------------------------------------------------ norm

def rows_apart(t, stride):
    if not stride or stride == t.shape[1]:
        return t.contiguous()
    buf = torch.full((t.shape[0], stride), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, : t.shape[1]] = t
    return buf[:, : t.shape[1]]


@pytest.mark.parametrize("T,H,h,w,stride,offset,add", [
    (1, 64, "bf16", "bf16", 0, False, False),
    (1, 7168, "bf16", "bf16", 0, False, True),
    (7, 7168, "bf16", "fp32", 0, True, True),
    (3, 2880, "fp32", "fp32", 2888, True, True),
    (17, 448, "bf16", "fp32", 512, False, False),
    (257, 4096, "fp32", "bf16", 0, False, True),
    (1031, 1536, "bf16", "bf16", 1544, True, True),
    (5, 8192, "bf16", None, 0, False, True),
    (2, 16384, "fp32", "bf16", 0, False, True),
    (170, 12288, "bf16", "bf16", 0, False, False),
    (3, 32768, "bf16", "fp32", 0, False, True),
    (160, 20480, "fp32", "bf16", 0, False, True),
    (3000, 128, "bf16", "bf16", 0, False, False),
    (5000, 256, "fp32", "fp32", 0, False, True),
    (16, 576, "fp32", "bf16", 584, True, True),
    (17, 64, "bf16", "bf16", 0, False, True),
    (900, 8192, "fp32", "fp32", 0, False, True),
    (400, 8192, "bf16", None, 8200, False, False),
])
def test_norm_backward(B, T, H, h, w, stride, offset, add):
    g = gen(T + H)
    hh = rows_apart((randn(g, (T, H), F32) * torch.exp(randn(g, (T, 1), F32, 1.0))).to(DT[h]), stride)
    ww = None if w is None else randn(g, (H,), DT[w], 0.2, 0.0 if offset else 1.0)
    dx = rows_apart(randn(g, (T, H)), stride)
    more = rows_apart(randn(g, (T, H), DT[h]), stride) if add else None
    dh = empty((T, stride or H), DT[h])
    dw = empty((H,), DT[w or "bf16"])
    p = B.NormProblem.make(T, H, h_dtype=DT[h], w_dtype=DT[w or "bf16"], eps=1e-5, unit_offset=offset, h_stride=stride,
                           x_stride=stride, y_stride=stride, out_stride=stride)
    ws = torch.full((B.moe_norm_backward_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
    B.moe_norm_backward(p, hh, ww, dx, dh[:, :H], ws, dh_add=more, dw=dw)
    want, want_dw, mag, mag_dw = back.norm(ref.f64(hh), ref.f64(dx), ref.f64(ww), 1e-5, offset, ref.f64(more))
    check(dh[:, :H], want, 90 * U * mag, "dh")
    check(dw, want_dw, (90 + T / 152 + 64) * U * mag_dw, "dw")
    if stride:
        assert (dh[:, H:] == 7.0).all()
    # without the weight's gradient, and in place
    dh2 = hh.clone() if not stride else None
    if dh2 is not None:
        B.moe_norm_backward(p, dh2, ww, dx, dh2, ws, dh_add=more)
        assert torch.equal(dh2, dh)
        if add:
            same = more.clone()
            B.moe_norm_backward(p, hh, ww, dx, same, ws, dh_add=same)
            assert torch.equal(same, dh)


def test_norm_backward_zero_rows_and_token_count(B):
    T, H = 9, 512
    g = gen(1)
    h, dx, w = randn(g, (T, H)), randn(g, (T, H)), randn(g, (H,), BF, 0.1, 1.0)
    h[2] = 0
    h[3] = 1e-30
    h[8], dx[8] = float("nan"), float("nan")          # a row past every count below
    p = B.NormProblem.make(T, H, eps=1e-6)
    ws = torch.empty(B.moe_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    for n, rows in [(8, 8), (5, 5), (0, 0), (-3, 0)]:
        dh, dw = empty((T, H)), empty((H,))
        B.moe_norm_backward(p, h, w, dx, dh, ws, dw=dw, d_num_tokens=count(n))
        want, want_dw, mag, mag_dw = back.norm(ref.f64(h)[:rows], ref.f64(dx)[:rows], ref.f64(w)) if rows else (
            np.zeros((0, H)), np.zeros(H), np.zeros((0, H)), np.zeros(H))
        check(dh[:rows], want, 90 * U * mag, "dh")
        check(dw, want_dw, 160 * U * mag_dw, "dw")
        assert (dh[rows:] == 7.0).all()


# ------------------------------------------------------------------ router

def test_norm_backward_many_rows_and_token_count(B):
    T, H = 700, 1088
    g = gen(2)
    h, dx, w = randn(g, (T, H)), randn(g, (T, H)), randn(g, (H,), BF, 0.1, 1.0)
    p = B.NormProblem.make(T, H, eps=1e-6)
    ws = torch.zeros(B.moe_norm_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    for n, rows in [(699, 699), (153, 153), (1, 1), (0, 0), (-1, 0), (4000, T)]:
        h2, dx2 = h.clone(), dx.clone()
        h2[rows:], dx2[rows:] = float("nan"), float("nan")
        dh, dw = empty((T, H)), empty((H,))
        B.moe_norm_backward(p, h2, w, dx2, dh, ws, dw=dw, d_num_tokens=count(n))
        want, want_dw, mag, mag_dw = back.norm(ref.f64(h)[:rows], ref.f64(dx)[:rows], ref.f64(w)) if rows else (
            np.zeros((0, H)), np.zeros(H), np.zeros((0, H)), np.zeros(H))
        check(dh[:rows], want, 90 * U * mag, "dh")
        check(dw, want_dw, 160 * U * mag_dw, "dw")
        assert (dh[rows:] == 7.0).all()
    assert B.moe_last_device_error(ws) == 0


def route_inputs(B, seed, T, E, k, H, score, renorm):
    g = gen(seed)
    x, w = randn(g, (T, H)), randn(g, (E, H), BF, H ** -0.5)
    logits = (x.float() @ w.float().T) * 2
    ids, _, _ = ref.route(ref.f64(logits), k, score, renorm)
    dw = randn(g, (T, k), F32)
    return x, w, logits, torch.from_numpy(ids).cuda(), dw


def run_route(B, p, x, w, logits, ids, dwt, add=None, dtype=BF, n=None, wanted=("dx", "dw", "dl")):
    ws = torch.zeros(B.moe_route_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    dx = empty(x.shape) if "dx" in wanted else None
    dw = empty(w.shape, dtype) if "dw" in wanted else None
    dl = empty(logits.shape, F32) if "dl" in wanted else None
    B.moe_route_backward(p, x, w, logits, ids, dwt, ws, d_logits_add=add, dx=dx, dw_router=dw, d_logits=dl,
                         d_num_tokens=count(n))
    return dx, dw, dl, B.moe_last_device_error(ws)


@pytest.mark.parametrize("T,E,k,H", [(1, 8, 2, 64), (3, 5, 5, 192), (61, 256, 8, 512), (130, 1000, 40, 128), (300, 64, 6, 320),
                                     (700, 24, 1, 1024), (2000, 130, 8, 256), (6, 1024, 64, 64)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward(B, T, E, k, H, score, renorm):
    x, w, logits, ids, dwt = route_inputs(B, T + E, T, E, k, H, score, renorm)
    add = randn(gen(2), (T, E), F32, 0.1) if T % 2 else None
    dtype = F32 if T % 3 == 0 else BF
    p = B.RouterProblem.make(T, E, k, H, score=0 if score == "softmax" else 1, renormalize=renorm, scale=1.5)
    dx, dw, dl, err = run_route(B, p, x, w, logits, ids, dwt, add, dtype)
    assert err == 0
    want, mag = back.route(ref.f64(logits), ref.f64(ids).astype(int), ref.f64(dwt), score, renorm, 1.5)
    if add is not None:
        want, mag = want + ref.f64(add), mag + np.abs(ref.f64(add))
    check(dl, want, 64 * U * mag, "dl")
    # the products, from the logits' gradient as it came out
    d, xx, ww = ref.f64(dl), ref.f64(x), ref.f64(w)
    Ep = (E + 63) // 64 * 64
    check(dx, d @ ww, (2.0 ** -16 + back.mma_rel(2 * Ep)) * (np.abs(d) @ np.abs(ww)), "dx")
    check(dw, d.T @ xx, (2.0 ** -16 + back.mma_rel(2 * T) + 152 * U) * (np.abs(d).T @ np.abs(xx)), "dw")


def test_route_backward_masks(B):
    """Switched-off experts, rows with nothing left, logits that are not finite, repeated and invalid ids."""
    T, E, k, H = 8, 12, 3, 64
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            x, w, logits, _, dwt = route_inputs(B, 3, T, E, k, H, score, renorm)
            logits[0] = float("-inf")
            logits[1, 3:] = float("-inf")
            logits[2, 5], logits[2, 6] = float("nan"), float("inf")
            logits[3] = -200.0                      # sigmoid scores underflow, their ratios do not
            logits[4] *= 20.0
            ids, _, _ = ref.route(ref.f64(logits), k, score, renorm)
            ids[5] = [4, 4, 7]                      # the same expert twice
            ids[6] = [2, -1, -1]
            p = B.RouterProblem.make(T, E, k, H, score=0 if score == "softmax" else 1, renormalize=renorm)
            d_ids = torch.from_numpy(ids).cuda()
            dx, dw, dl, err = run_route(B, p, x, w, logits, d_ids, dwt)
            assert err == 0
            want, mag = back.route(ref.f64(logits), ids, ref.f64(dwt), score, renorm)
            check(dl, want, 300 * U * mag, "dl")    # row 4: arguments up to 200 in size
            assert (dl[0] == 0).all() and torch.isfinite(dx).all() and torch.isfinite(dw).all()
            bad = ids.copy()
            bad[7] = [1, E, -9]
            _, _, dl2, err = run_route(B, p, x, w, logits, torch.from_numpy(bad).cuda(), dwt)
            assert err == B.MOE_DEVERR_BAD_EXPERT_ID
            want, mag = back.route(ref.f64(logits), bad, ref.f64(dwt), score, renorm)
            check(dl2, want, 300 * U * mag, "dl")


@pytest.mark.parametrize("T", [5, 400])
def test_route_backward_reports_invalid_ids_for_every_output(B, T):
    E, k, H = 16, 2, 64
    x, w, logits, ids, dwt = route_inputs(B, 6, T, E, k, H, "softmax", True)
    p = B.RouterProblem.make(T, E, k, H)
    for wanted in (("dx",), ("dw",), ("dl",)):
        for bad in (E, -2, 1 << 30):
            wrong = ids.clone()
            wrong[T - 1, 1] = bad
            assert run_route(B, p, x, w, logits, wrong, dwt, wanted=wanted)[3] == B.MOE_DEVERR_BAD_EXPERT_ID
        assert run_route(B, p, x, w, logits, ids, dwt, wanted=wanted)[3] == 0


@pytest.mark.parametrize("T,E,k", [(128, 64, 8), (200, 8, 1), (250, 16, 1), (256, 300, 4), (1, 1, 1)])
def test_route_backward_hot_experts(B, T, E, k):
    """Few slots, most of them of one expert; some tokens without any."""
    H = 1088
    x, w, logits, ids, dwt = route_inputs(B, 7, T, E, k, H, "sigmoid", True)
    hot = ids.clone()
    hot[:, 0] = E - 1
    for j in range(1, k):
        hot[:, j] = torch.where(hot[:, j] == E - 1, E - 2, hot[:, j])
    hot[T // 2] = -1
    p = B.RouterProblem.make(T, E, k, H, score=1)
    dx, dw, dl, err = run_route(B, p, x, w, logits, hot, dwt, dtype=F32)
    assert err == 0
    want, mag = back.route(ref.f64(logits), ref.f64(hot).astype(int), ref.f64(dwt), "sigmoid", True)
    check(dl, want, 64 * U * mag, "dl")
    d, xx, ww = ref.f64(dl), ref.f64(x), ref.f64(w)
    Ep = (E + 63) // 64 * 64
    check(dx, d @ ww, (2.0 ** -16 + back.mma_rel(2 * Ep)) * (np.abs(d) @ np.abs(ww)), "dx")
    check(dw, d.T @ xx, (2.0 ** -16 + back.mma_rel(2 * T) + 152 * U) * (np.abs(d).T @ np.abs(xx)), "dw")
    assert (dx[T // 2] == 0).all()


def test_route_backward_token_count_and_single_outputs(B):
    T, E, k, H = 300, 40, 4, 192
    x, w, logits, ids, dwt = route_inputs(B, 4, T, E, k, H, "softmax", True)
    p = B.RouterProblem.make(T, E, k, H)
    full = run_route(B, p, x, w, logits, ids, dwt)
    for i, name in enumerate(("dx", "dw", "dl")):
        one = run_route(B, p, x, w, logits, ids, dwt, wanted=(name,))[i]
        assert torch.equal(one, full[i]), name
    x2, l2, d2 = x.clone(), logits.clone(), dwt.clone()
    for n, rows in [(290, 290), (37, 37), (0, 0), (-1, 0), (1000, 300)]:
        x2[rows:], l2[rows:], d2[rows:] = float("nan"), float("nan"), float("nan")
        dx, dw, dl, _ = run_route(B, p, x2, w, l2, ids, d2, n=n)
        x2, l2, d2 = x.clone(), logits.clone(), dwt.clone()
        assert torch.equal(dx[:rows], full[0][:rows]) and (dx[rows:] == 7.0).all()
        assert torch.equal(dl[:rows], full[2][:rows]) and (dl[rows:] == 7.0).all()
        d, xx = ref.f64(full[2])[:rows], ref.f64(x)[:rows]
        check(dw, d.T @ xx, (2.0 ** -16 + back.mma_rel(2 * T) + 152 * U) * (np.abs(d).T @ np.abs(xx)), "dw")


# ------------------------------------------------------------------ together

def block_case(B, seed, T, E, k, H, I):
    g = gen(seed)
    return {"h": randn(g, (T, H)), "w_pre": randn(g, (H,), BF, 0.1, 1.0), "w_router": randn(g, (E, H), BF, H ** -0.5),
            "W13": randn(g, (E, 2 * I, H), BF, H ** -0.5), "W2": randn(g, (E, H, I), BF, I ** -0.5),
            "dout": randn(g, (T, H), BF)}


class Step:
    """One training step's forward and backward of a block, on buffers kept between steps."""

    def __init__(self, B, c, T, E, k, H, I):
        def new(*shape, dtype=BF):
            return torch.empty(shape, dtype=dtype, device="cuda")

        def ws(n):
            return torch.zeros(n, dtype=torch.uint8, device="cuda")

        self.B, self.c = B, c
        self.experts, self.router, self.norm = B.Problem.make(T, E, k, H, I), B.RouterProblem.make(T, E, k, H), B.NormProblem.make(T, H)
        self.grad = B.ExpertGradProblem.make(self.experts)
        self.bufs = B.Buffers(self.experts)
        self.x, self.ids, self.weights, self.logits = new(T, H), new(T, k, dtype=I32), new(T, k, dtype=F32), new(T, E, dtype=F32)
        self.route_ws, self.route_bws = ws(B.moe_route_workspace_size(self.router)), ws(B.moe_route_backward_workspace_size(self.router))
        self.expert_bws, self.norm_bws = ws(B.moe_expert_backward_workspace_size(self.grad)), ws(B.moe_norm_backward_workspace_size(self.norm))
        self.dy, self.dxs, self.dx, self.dh = new(T * k, H), new(T * k, H), new(T, H), new(T, H)
        self.dweights, self.dW13, self.dW2 = new(T, k, dtype=F32), new(E, 2 * I, H), new(E, H, I)
        self.dw_router, self.dw_pre = new(E, H), new(H)

    def forward(self):
        B, c, b = self.B, self.c, self.bufs
        B.moe_norm(self.norm, c["h"], c["w_pre"], self.x)
        B.moe_route(self.router, self.x, c["w_router"], self.ids, self.weights, self.route_ws, logits=self.logits)
        B.moe_dispatch(self.experts, self.ids, b.expert_offsets, b.perm, b.inv, b.ws, x=self.x, x_sorted=b.x_sorted)
        B.moe_expert_compute(self.experts, b.x_sorted, b.expert_offsets, c["W13"], c["W2"], b.y_sorted, b.ws)
        B.moe_combine(self.experts, b.y_sorted, b.inv, self.weights, b.out)

    def backward(self):
        B, c, b = self.B, self.c, self.bufs
        # the stream's row is h + out: its gradient reaches h past the block, and the block's out
        B.moe_combine_backward(self.experts, c["dout"], b.inv, self.weights, self.dy, y_sorted=b.y_sorted, d_weights=self.dweights)
        B.moe_expert_backward(self.grad, b.x_sorted, b.expert_offsets, c["W13"], c["W2"], self.dy, self.expert_bws,
                              dx_sorted=self.dxs, dW13=self.dW13, dW2=self.dW2)
        B.moe_route_backward(self.router, self.x, c["w_router"], self.logits, self.ids, self.dweights, self.route_bws,
                             dx=self.dx, dw_router=self.dw_router)
        B.moe_dispatch_backward(self.experts, self.dxs, b.inv, self.dx, dx_add=self.dx)
        B.moe_norm_backward(self.norm, c["h"], c["w_pre"], self.dx, self.dh, self.norm_bws, dh_add=c["dout"], dw=self.dw_pre)

    def outputs(self):
        return {"dh": self.dh, "dw_pre": self.dw_pre, "dw_router": self.dw_router, "dW13": self.dW13, "dW2": self.dW2}

    def errors(self):
        return [self.B.moe_last_device_error(w) for w in (self.route_ws, self.bufs.ws, self.route_bws, self.expert_bws)]


def autograd_block(c, ids, k):
    """The block in 64 bits with torch's differentiation, the choice of experts given."""
    leaf = {n: c[n].double().cpu().requires_grad_() for n in ("h", "w_pre", "w_router", "W13", "W2")}
    h = leaf["h"]
    x = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * leaf["w_pre"]
    p = torch.softmax(x @ leaf["w_router"].T, 1).gather(1, ids)
    p = p / p.sum(1, keepdim=True)
    I = leaf["W2"].shape[2]
    y = torch.zeros_like(h)
    for e in range(leaf["W2"].shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        gu = x[t] @ leaf["W13"][e].T
        y = y.index_add(0, t, p[t, j, None] * ((torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ leaf["W2"][e].T))
    (h + y).backward(c["dout"].double().cpu())
    return {"dh": h.grad, "dw_pre": leaf["w_pre"].grad, "dw_router": leaf["w_router"].grad, "dW13": leaf["W13"].grad,
            "dW2": leaf["W2"].grad}


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 128, 64), (50, 16, 4, 256, 192), (700, 8, 2, 512, 256)])
def test_whole_block_against_autograd(B, T, E, k, H, I):
    """Forward and backward of a block. Between the operators rows go through bf16 some four times (x, y's and
    x's gradients, the experts' inner rows), 2^-8 each at most and independent: 2 of those by their rms keep every
    result within 2 * 2^-8 of its norm, and a quarter of that is what uniform roundings come to."""
    c = block_case(B, T + E, T, E, k, H, I)
    s = Step(B, c, T, E, k, H, I)
    s.forward()
    s.backward()
    assert s.errors() == [0, 0, 0, 0]
    want = autograd_block(c, s.ids.cpu().long(), k)
    for n, got in s.outputs().items():
        off = (got.double().cpu() - want[n]).norm() / want[n].norm()
        assert off <= 2 * 2.0 ** -8, (n, float(off))


def test_step_in_a_graph_and_on_another_stream(B):
    """A captured step gives the eager step's bits, replayed with new inputs and on a stream of its own."""
    T, E, k, H, I = 130, 16, 4, 256, 128
    c = block_case(B, 1, T, E, k, H, I)
    s = Step(B, c, T, E, k, H, I)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    first = {n: v.clone() for n, v in s.outputs().items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.forward()
        s.backward()
    for v in s.outputs().values():
        v.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    for n, v in s.outputs().items():
        assert torch.equal(v, first[n]), n
    other = block_case(B, 2, T, E, k, H, I)
    for n in c:
        c[n].copy_(other[n])
    graph.replay()
    torch.cuda.synchronize()
    replayed = {n: v.clone() for n, v in s.outputs().items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        t = Step(B, other, T, E, k, H, I)
        t.forward()
        t.backward()
    stream.synchronize()
    for n, v in t.outputs().items():
        assert torch.equal(v, replayed[n]), n
    assert s.errors() == [0, 0, 0, 0]
