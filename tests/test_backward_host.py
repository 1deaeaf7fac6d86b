"""Host checks of the gradients' entry points (no GPU): what is out of range,
missing, misaligned or too short is refused before any CUDA call; and the
tests' own 64-bit gradients against central differences of the forward."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import backward_reference as back
import block_reference as ref
from moe_routed_expert_routing_gb300 import build as build_mod

FAKE = 1 << 40      # never dereferenced: every call below is refused first
NULL, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def B():
    build_mod.build()
    from moe_routed_expert_routing_gb300 import binding
    return binding


def each(args, nulls, aligns):
    """(changed arguments, status) for every pointer that may not be missing or misaligned."""
    for i in nulls:
        yield args[:i] + [None] + args[i + 1:], NULL
    for i in aligns:
        yield args[:i] + [FAKE + 8] + args[i + 1:], ALIGN


def test_combine_backward_refusals(B):
    f = B.load_library().moe_combine_backward
    p = ctypes.byref(B.Problem.make(4, 8, 2, 128, 64))
    ok = [FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE]
    for args, status in each(ok, (0, 1, 2, 3, 5), (0, 1, 5)):
        assert f(p, *args, None) == status, args
    assert f(None, *ok, None) == NULL
    assert f(ctypes.byref(B.Problem.make(4, 8, 2, 100, 64)), *ok, None) == ALIGN
    assert f(ctypes.byref(B.Problem.make(4, 8, 9, 128, 64)), *ok, None) == SHAPE


def test_dispatch_backward_refusals(B):
    f = B.load_library().moe_dispatch_backward
    p = ctypes.byref(B.Problem.make(4, 8, 2, 128, 64))
    ok = [FAKE, FAKE, FAKE, None, FAKE]
    for args, status in each(ok, (0, 1, 4), (0, 2, 4)):
        assert f(p, 0, *args, None) == status, args
    assert f(p, 2, *ok, None) == SHAPE
    assert f(p, -1, *ok, None) == SHAPE
    assert f(None, 0, *ok, None) == NULL


def grad(B, dx=0, dw=0, accumulate=False, **kw):
    args = dict(T_max=4, E=8, k=2, H=128, I=64)
    args.update(kw)
    return B.ExpertGradProblem.make(B.Problem.make(**args), dx, dw, accumulate)


@pytest.mark.parametrize("kw,status", [
    (dict(H=100), ALIGN), (dict(E=0), SHAPE), (dict(dx=2), SHAPE), (dict(dw=-1), SHAPE), (dict(dw=0, accumulate=True), SHAPE),
    (dict(dw=1, accumulate=2), SHAPE), (dict(H=256, I=128, weight_layout=1), UNSUPPORTED),
    (dict(H=256, I=128, weight_layout=2), UNSUPPORTED), (dict(capacity=7), SHAPE),
    (dict(E=1, k=1, H=1 << 30, I=1 << 20), SHAPE),
])
def test_expert_backward_description(B, kw, status):
    p = grad(B, **kw)
    with pytest.raises(B.MoeError) as ei:
        B.moe_expert_backward_workspace_size(p)
    assert ei.value.status == status
    f = B.load_library().moe_expert_backward
    assert f(ctypes.byref(p), *[FAKE] * 8, FAKE, 1 << 50, None) == status


def test_expert_backward_pointers_and_workspace(B):
    f = B.load_library().moe_expert_backward
    p = grad(B)
    need = B.moe_expert_backward_workspace_size(p)
    assert need % 256 == 0 and need >= 6 * 8 * 64
    P = ctypes.byref(p)
    ok = [FAKE] * 8
    for args, status in each(ok, (0, 1, 2, 3, 4), (0, 2, 3, 4, 5, 6, 7)):
        assert f(P, *args, FAKE, need, None) == status, args
    assert f(P, *ok[:5], None, None, None, FAKE, need, None) == NULL      # nothing wanted
    assert f(P, *ok, None, need, None) == NULL
    assert f(P, *ok, FAKE + 16, need, None) == ALIGN
    assert f(P, *ok, FAKE, need - 1, None) == WORKSPACE
    assert f(None, *ok, FAKE, need, None) == NULL
    # a larger capacity needs a larger workspace
    assert B.moe_expert_backward_workspace_size(grad(B, capacity=1000)) >= 6 * 1000 * 64


def test_norm_backward_refusals(B):
    f = B.load_library().moe_norm_backward
    q = B.NormProblem.make(4, 256)
    need = B.moe_norm_backward_workspace_size(q)
    p = ctypes.byref(q)
    ok = [FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE]
    for args, status in each(ok, (0, 2, 5), (0, 1, 2, 3, 5, 6)):
        assert f(p, *args, FAKE, need, None) == status, args
    assert f(p, *ok, None, need, None) == NULL
    assert f(p, *ok, FAKE, need - 256, None) == WORKSPACE
    assert f(None, *ok, FAKE, need, None) == NULL
    for bad, status in [(dict(T_max=0), SHAPE), (dict(H=100), ALIGN), (dict(H=32832), SHAPE), (dict(eps=0.0), SHAPE),
                        (dict(x_stride=260), ALIGN), (dict(y_stride=64), SHAPE)]:
        args = dict(T_max=4, H=256)
        args.update(bad)
        n = B.NormProblem.make(**args)
        assert f(ctypes.byref(n), *ok, FAKE, 1 << 50, None) == status
        with pytest.raises(B.MoeError) as ei:
            B.moe_norm_backward_workspace_size(n)
        assert ei.value.status == status


def test_route_backward_refusals(B):
    f = B.load_library().moe_route_backward
    q = B.RouterProblem.make(4, 16, 2, 128)
    need = B.moe_route_backward_workspace_size(q)
    p = ctypes.byref(q)
    # x, w_router, logits, ids, d_weights, add, tokens, dx, dw, d_logits
    ok = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE]
    for args, status in each(ok, (0, 1, 2, 3, 4), (0, 1, 2, 3, 4, 5, 7, 8, 9)):
        assert f(p, 0, *args, FAKE, need, None) == status, args
    assert f(p, 0, *ok[:7], None, None, None, FAKE, need, None) == NULL
    assert f(p, 2, *ok, FAKE, need, None) == SHAPE
    assert f(p, 0, *ok, FAKE, need - 1, None) == WORKSPACE
    assert f(p, 0, *ok, None, need, None) == NULL
    assert f(None, 0, *ok, FAKE, need, None) == NULL
    for bad, status in [(dict(k=0), SHAPE), (dict(H=100), ALIGN), (dict(E=1025), SHAPE), (dict(score=2), SHAPE),
                        (dict(scale=float("nan")), SHAPE), (dict(T_max=1 << 27, E=1, k=1, H=1 << 30), SHAPE)]:
        args = dict(T_max=4, E=16, k=2, H=128)
        args.update(bad)
        r = B.RouterProblem.make(**args)
        assert f(ctypes.byref(r), 0, *ok, FAKE, 1 << 60, None) == status, bad


def test_binding_refuses_what_does_not_fit(B):
    bf, host = torch.bfloat16, torch.zeros
    p = B.Problem.make(4, 8, 2, 128, 64)
    with pytest.raises(ValueError, match="d_out must be a CUDA tensor"):
        B.moe_combine_backward(p, host((4, 128), dtype=bf), FAKE, FAKE, FAKE)
    with pytest.raises(ValueError, match="dx_sorted must be a CUDA tensor"):
        B.moe_dispatch_backward(p, host((8, 128), dtype=bf), FAKE, FAKE)
    with pytest.raises(ValueError, match="float16"):
        B.moe_dispatch_backward(p, host((8, 128), dtype=torch.float16), FAKE, FAKE)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.moe_expert_backward(grad(B), host((8, 128), dtype=bf), FAKE, FAKE, FAKE, FAKE, host(1))
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.moe_norm_backward(B.NormProblem.make(4, 256), host((4, 256), dtype=bf), None, FAKE, FAKE, host(1))
    with pytest.raises(ValueError, match="float64"):
        B.moe_route_backward(B.RouterProblem.make(4, 16, 2, 128), FAKE, FAKE, FAKE, FAKE, FAKE, host(1),
                             dw_router=host((16, 128), dtype=torch.float64))


# ------------------------------------------------ the references by differences

def differences(f, v, eps=1e-6):
    """Gradient of the scalar f at v by central differences."""
    out = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        keep = v[i]
        v[i] = keep + eps
        up = f()
        v[i] = keep - eps
        out[i] = (up - f()) / (2 * eps)
        v[i] = keep
    return out


def test_reference_norm_by_differences():
    rng = np.random.default_rng(0)
    h, w, dx = rng.standard_normal((3, 8)), rng.standard_normal(8), rng.standard_normal((3, 8))
    for offset in (False, True):
        f = lambda: (ref.norm(h, w, 0.1, offset) * dx).sum()  # noqa: E731
        dh, dw, _, _ = back.norm(h, dx, w, 0.1, offset)
        assert np.allclose(dh, differences(f, h), atol=1e-8)
        assert np.allclose(dw, differences(f, w), atol=1e-8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_reference_route_by_differences(score, renormalize):
    rng = np.random.default_rng(1)
    l, dw = rng.standard_normal((4, 7)), rng.standard_normal((4, 3))
    ids, _, _ = ref.route(l, 3, score, renormalize)
    f = lambda: (ref.route(l, 3, score, renormalize, scale=1.7)[1] * dw).sum()  # noqa: E731
    dl, _ = back.route(l, ids, dw, score, renormalize, 1.7)
    assert np.allclose(dl, differences(f, l), atol=1e-8)


def test_reference_experts_and_rows_by_differences():
    rng = np.random.default_rng(2)
    T, E, k, H, I = 5, 3, 2, 4, 3
    x, W13, W2 = rng.standard_normal((T, H)), rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    ids = np.array([[0, 2], [2, -1], [0, 2], [-1, -1], [2, 0]])     # expert 1 gets no row
    w, dout = rng.random((T, k)), rng.standard_normal((T, H))
    flat = ids.reshape(-1)
    order = [s for e in range(E) for s in np.nonzero(flat == e)[0]]
    inv = np.full(T * k, -1)
    inv[order] = np.arange(len(order))
    bounds = [0, 3, 3, 7]
    f = lambda: (ref.experts(x, ids, w, W13, W2) * dout).sum()  # noqa: E731
    xs = x[np.array(order) // k]
    y = np.zeros((len(order), H))
    for e in (0, 2):
        rows = slice(bounds[e], bounds[e + 1])
        gu = xs[rows] @ W13[e].T
        y[rows] = (gu[:, :I] * back.sigmoid(gu[:, :I]) * gu[:, I:]) @ W2[e].T
    dy, dw, _ = back.combine(dout, y, inv, w)
    dy = np.stack([dy[r] for r in range(len(order))])
    got, _ = back.experts(xs, dy, W13, W2, bounds)
    dx, _ = back.dispatch(got["dx"], inv, T, k)
    assert np.allclose(dx, differences(f, x), atol=1e-7)
    assert np.allclose(dw, differences(f, w), atol=1e-7)
    assert np.allclose(got["dW13"], differences(f, W13), atol=1e-7)
    assert np.allclose(got["dW2"], differences(f, W2), atol=1e-7)
