"""Host checks of the block's entry points (no GPU): descriptions that are out
of range, missing or misaligned buffers and short workspaces are refused
before any CUDA call, and the binding refuses tensors that do not fit."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import block_reference as ref
from moe_routed_expert_routing_gb300 import build as build_mod

FAKE = 1 << 40      # never dereferenced: every call below is refused first
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def B():
    build_mod.build()
    from moe_routed_expert_routing_gb300 import binding
    return binding


@pytest.mark.parametrize("bad,status", [
    (dict(T_max=0), SHAPE), (dict(H=0), SHAPE), (dict(H=100), ALIGN), (dict(H=32832), SHAPE), (dict(h_dtype=2), SHAPE),
    (dict(w_dtype=-1), SHAPE), (dict(eps=0.0), SHAPE), (dict(eps=-1e-6), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(eps=float("inf")), SHAPE), (dict(residual_scale=float("nan")), SHAPE), (dict(gate=4), SHAPE),
    (dict(h_stride=64), SHAPE), (dict(y_stride=260), ALIGN), (dict(x_stride=-8), SHAPE), (dict(out_stride=1 << 41), SHAPE),
    (dict(gate_stride=257), ALIGN),
])
def test_norm_description(B, bad, status):
    so = B.load_library()
    args = dict(T_max=4, H=256)
    args.update(bad)
    p = ctypes.byref(B.NormProblem.make(**args))
    assert so.moe_norm(p, FAKE, FAKE, None, FAKE, None) == status
    assert so.moe_norm_residual(p, FAKE, FAKE, None, FAKE, None, None, FAKE, None, None) == status


def test_norm_pointers(B):
    so = B.load_library()
    p = ctypes.byref(B.NormProblem.make(4, 256))
    assert so.moe_norm(None, FAKE, FAKE, None, FAKE, None) == NULL
    assert so.moe_norm(p, None, FAKE, None, FAKE, None) == NULL
    assert so.moe_norm(p, FAKE, None, None, None, None) == NULL
    assert so.moe_norm(p, FAKE + 2, FAKE, None, FAKE, None) == ALIGN
    assert so.moe_norm(p, FAKE, FAKE + 8, None, FAKE, None) == ALIGN
    assert so.moe_norm_residual(p, FAKE, None, None, None, None, None, FAKE, None, None) == NULL
    assert so.moe_norm_residual(p, FAKE, FAKE, None, None, None, None, None, None, None) == NULL
    assert so.moe_norm_residual(p, FAKE, FAKE + 4, None, None, None, None, FAKE, None, None) == ALIGN
    assert so.moe_norm_residual(p, FAKE, FAKE, None, None, None, None, FAKE, FAKE + 4, None) == ALIGN
    g = ctypes.byref(B.NormProblem.make(4, 256, gate=B.MOE_GATE_CHANNEL))
    assert so.moe_norm_residual(g, FAKE, FAKE, None, None, None, None, FAKE, None, None) == NULL


ROUTER = dict(T_max=4, E=16, k=2, H=128)


@pytest.mark.parametrize("bad,status", [
    (dict(T_max=0), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=17), SHAPE),
    (dict(E=128, k=65), SHAPE), (dict(H=100), ALIGN), (dict(H=0), SHAPE), (dict(score=2), SHAPE), (dict(renormalize=2), SHAPE),
    (dict(n_group=3), SHAPE), (dict(n_group=0), SHAPE), (dict(E=64, n_group=64), SHAPE),
    (dict(n_group=4, topk_group=5), SHAPE), (dict(n_group=4, topk_group=0), SHAPE), (dict(group_top=3), SHAPE),
    (dict(group_top=2), SHAPE), (dict(n_group=16, topk_group=4, group_top=2), SHAPE),
    (dict(n_group=4, topk_group=1, k=5), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(T_max=1 << 28), SHAPE),
])
def test_router_description(B, bad, status):
    args = dict(ROUTER)
    args.update(bad)
    p = B.RouterProblem.make(**args)
    with pytest.raises(B.MoeError) as ei:
        B.moe_route_workspace_size(p)
    assert ei.value.status == status
    assert B.load_library().moe_route(ctypes.byref(p), FAKE, FAKE, None, None, FAKE, FAKE, None, FAKE, 1 << 40, None) == status


def test_router_pointers_and_workspace(B):
    so = B.load_library()
    r = B.RouterProblem.make(**ROUTER)
    need = B.moe_route_workspace_size(r)
    p = ctypes.byref(r)
    assert need % 256 == 0 and need >= 4 * 4 * 16
    assert so.moe_route(None, FAKE, FAKE, None, None, FAKE, FAKE, None, FAKE, need, None) == NULL
    for i in (0, 1, 4, 5, 7):
        args = [FAKE, FAKE, None, None, FAKE, FAKE, None, FAKE]
        args[i] = None
        assert so.moe_route(p, *args, need, None) == NULL, i
        args[i] = FAKE + 4
        assert so.moe_route(p, *args, need, None) == ALIGN, i
    assert so.moe_route(p, FAKE, FAKE, FAKE + 4, None, FAKE, FAKE, None, FAKE, need, None) == ALIGN
    assert so.moe_route(p, FAKE, FAKE, None, None, FAKE, FAKE, FAKE + 8, FAKE, need, None) == ALIGN
    assert so.moe_route(p, FAKE, FAKE, None, None, FAKE, FAKE, None, FAKE, need - 1, None) == WORKSPACE


def layer(B, norm=None, router=None, experts=None):
    e = dict(T_max=4, E=16, k=2, H=128, I=64)
    e.update(experts or {})
    r = dict(ROUTER)
    r.update(router or {})
    n = dict(T_max=4, H=128)
    n.update(norm or {})
    return B.LayerProblem.make(B.Problem.make(**e), B.RouterProblem.make(**r), B.NormProblem.make(**n))


@pytest.mark.parametrize("parts,status", [
    (dict(norm=dict(T_max=5)), SHAPE), (dict(norm=dict(H=192)), SHAPE), (dict(router=dict(E=15)), SHAPE),
    (dict(router=dict(k=3)), SHAPE), (dict(experts=dict(I=100)), ALIGN), (dict(norm=dict(eps=0.0)), SHAPE),
    (dict(experts=dict(T_max=129), router=dict(T_max=129), norm=dict(T_max=129)), SHAPE),
    (dict(experts=dict(H=16448), router=dict(H=16448), norm=dict(H=16448)), SHAPE),
])
def test_layer_description(B, parts, status):
    p = layer(B, **parts)
    with pytest.raises(B.MoeError) as ei:
        B.moe_layer_workspace_size(p)
    assert ei.value.status == status


def test_layer_pointers_and_workspace(B):
    so = B.load_library()
    p = layer(B)
    need = B.moe_layer_workspace_size(p)
    assert need >= B.moe_workspace_size(p.experts)
    ok = [FAKE, None, FAKE, None, FAKE, FAKE, None, None, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE]
    P = ctypes.byref(p)
    assert so.moe_layer(None, *ok, need, None) == NULL
    for i in (0, 2, 4, 5, 10, 11, 12, 13, 14, 16):
        args = list(ok)
        args[i] = None
        assert so.moe_layer(P, *args, need, None) == NULL, i
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 14, 15, 16):
        args = list(ok)
        args[i] = FAKE + 4
        assert so.moe_layer(P, *args, need, None) == ALIGN, i
    assert so.moe_layer(P, *ok, need - 256, None) == WORKSPACE
    gated = layer(B, norm=dict(gate=B.MOE_GATE_TOKEN))
    assert so.moe_layer(ctypes.byref(gated), *ok, need, None) == NULL


@pytest.mark.parametrize("capacity", [8, 9, 100, 1 << 29, 1 << 30, (1 << 30) + 4, (1 << 31) - 1])
def test_layer_workspace_does_not_follow_the_capacity(B, capacity):
    """The layer's sorted rows are its own: T_max * k of them whatever larger capacity the experts' description
    names (twice that capacity would not fit 32 bits)."""
    so = B.load_library()
    need = B.moe_layer_workspace_size(layer(B))
    p = layer(B, experts=dict(capacity=capacity))
    assert B.moe_layer_workspace_size(p) == need
    args = [FAKE, None, FAKE, None, FAKE, FAKE, None, None, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE]
    assert so.moe_layer(ctypes.byref(p), *args, need - 256, None) == WORKSPACE
    with pytest.raises(B.MoeError) as ei:      # fewer rows than slots are refused as in moe_forward
        B.moe_layer_workspace_size(layer(B, experts=dict(capacity=7)))
    assert ei.value.status == SHAPE


class _Rows:
    """Stands in for a CUDA tensor: device, type, shape and strides."""
    is_cuda = True

    def __init__(self, dtype, shape, strides):
        self.dtype, self.shape, self._strides = dtype, shape, strides

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def numel(self):
        return int(np.prod(self.shape))

    def is_contiguous(self):
        return self._strides == (self.shape[1], 1)

    def data_ptr(self):
        return FAKE


def test_binding_checks_rows(B):
    bf = torch.bfloat16
    assert B._need_rows(_Rows(bf, (4, 256), (256, 1)), "h", bf, 4, 256, 0) == FAKE
    assert B._need_rows(_Rows(bf, (4, 256), (264, 1)), "h", bf, 4, 256, 264) == FAKE
    for t, rows, stride in [(_Rows(bf, (3, 256), (256, 1)), 4, 0), (_Rows(bf, (4, 256), (264, 1)), 4, 0),
                            (_Rows(bf, (4, 256), (256, 1)), 4, 264), (_Rows(bf, (4, 128), (264, 1)), 4, 264),
                            (_Rows(bf, (4, 256), (264, 2)), 4, 264), (_Rows(torch.float32, (4, 256), (256, 1)), 4, 0)]:
        with pytest.raises(ValueError, match="h"):
            B._need_rows(t, "h", bf, rows, 256, stride)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.moe_norm(B.NormProblem.make(4, 256), torch.zeros((4, 256), dtype=bf), None, FAKE)
    with pytest.raises(ValueError, match="float32"):
        B.NormProblem.make(4, 256, h_dtype=torch.float16)
    with pytest.raises(ValueError, match="gate"):
        B.moe_norm_residual(B.NormProblem.make(4, 256), FAKE, FAKE, FAKE, gate=FAKE)


def test_reference_router_by_brute_force():
    """The tests' own 64-bit router against every subset of experts, on tiny sizes."""
    rng = np.random.default_rng(0)
    for _ in range(30):
        l = rng.integers(-3, 4, (3, 6)).astype(np.float64)
        ids, w, _ = ref.route(l, 3, "softmax", False)
        p = np.exp(l) / np.exp(l).sum(1, keepdims=True)
        for t in range(3):
            pairs = sorted(((-l[t, e], e) for e in range(6)))[:3]
            assert list(ids[t]) == [e for _, e in pairs]
            assert np.allclose(w[t], p[t, ids[t]])
    ids, w, _ = ref.route(np.array([[1.0, 5.0, 4.0, 2.0]]), 2, "sigmoid", True, None, 2, 1, 2)
    assert list(ids[0]) == [2, 3]
    s = 1 / (1 + np.exp(-np.array([1.0, 5.0, 4.0, 2.0])))
    best = 0 if s[0] + s[1] > s[2] + s[3] else 1
    assert all(i // 2 == best for i in ids[0])
