"""moe_layer in the forms that its shape, its description and its kernels' waits
bring about: rows beyond the routed slots, K parts of the down product, the
one-kernel form's rows over several CTAs, waits that run out; and the precision
that an fp32 residual stream shows."""
from __future__ import annotations

import time

import numpy as np
import pytest
import torch

import block_reference as ref
from test_gpu_block import B, LayerCase  # noqa: F401  (B is the module's fixture)

pytestmark = pytest.mark.gpu

OUTPUTS = ("ids", "weights", "h", "x_next")


def same_bits(a, b, what=""):
    for key in OUTPUTS:
        if a[key] is not None:
            assert torch.equal(a[key], b[key]), (what, key)


@pytest.mark.parametrize("form", [0, 2])
def test_layer_capacity_beyond_the_slots(B, form):
    """A capacity far above T * k, in the workspace of the plain description: the same bits."""
    c = LayerCase(B, T=4, E=32, k=4, H=256, I=128, form=form)
    want = c.run()
    c.verify(want)
    for capacity in (17, (1 << 30) + 5, (1 << 31) - 1):
        q = B.Problem.make(4, 32, 4, 256, 128, forward_form=form, capacity=capacity)
        c.p = B.LayerProblem.make(q, c.router, c.norm)
        assert B.moe_layer_workspace_size(c.p) == c.ws.numel()
        o = {key: None if v is None else torch.full_like(v, 3) for key, v in want.items()}
        perm = o["perm"]
        o["perm"] = perm.data_ptr()          # T * k entries, which is what the call writes
        c.call(o)
        same_bits(o, want, capacity)
        assert torch.equal(perm, want["perm"]) and torch.equal(o["offsets"], want["offsets"])
        assert B.moe_last_device_error(c.ws) == 0


HEADER_BYTES = 256 + 4 * (1024 + 6)   # error word block, readiness counts, counters


@pytest.mark.parametrize("form,layout", [(0, 0), (0, 2), (2, 0), (2, 2)],
                         ids=["separate", "separate_mxfp8", "one_kernel", "one_kernel_mxfp8"])
def test_layer_wait_limit_reports_and_recovers(B, form, layout):
    """Readiness counts that no gate-up unit can bring to the target make the down units' waits run out after 2 s.
    The call says so, takes no second limit (a CTA that gave up counts itself for the rounds it leaves out, so the
    others do not wait for it), leaves every counter at zero, and the workspace gives the same bits afterwards."""
    c = LayerCase(B, T=4, E=64, k=4, H=512, I=256, layout=layout, form=form)
    clean = c.run()
    assert B.moe_last_device_error(c.ws) == 0
    c.ws[256:256 + 4 * 64].view(torch.int32).fill_(-(1 << 30))
    torch.cuda.synchronize()
    t0 = time.time()
    c.run()
    torch.cuda.synchronize()
    took = time.time() - t0
    assert B.moe_last_device_error(c.ws) & B.MOE_DEVERR_WAIT_TIMEOUT
    assert 1.5 < took < 3.5, took
    assert int(c.ws[4:HEADER_BYTES].count_nonzero()) == 0
    B.moe_clear_device_error(c.ws)
    same_bits(c.run(), clean)
    assert B.moe_last_device_error(c.ws) == 0


# (layer, K parts of its down product): at least four 128-wide K blocks a part, up to 16-row tiles' few units
SPLITS = [
    (dict(T=1, E=8, k=4, H=512, I=1024), 2),
    (dict(T=1, E=8, k=4, H=512, I=2048, gate=1), 4),
    (dict(T=3, E=24, k=2, H=384, I=1280, h="fp32", score=1, bias=True), 2),     # five K blocks a part
    (dict(T=2, E=16, k=3, H=256, I=2560, post=False, gate=2), 4),
    (dict(T=16, E=32, k=2, H=320, I=2048, h="fp32", nxt=False), 4),             # H ends inside a tile; rows of 16 bits only
    (dict(T=1, E=8, k=4, H=512, I=896), 1),                                     # seven K blocks: none
]


def parts_used(c):
    """K parts whose buffers the last call wrote: the workspace behind its header was 0xA5 before it. Of the larger
    buffers only unused parts, T * k pairs of fp32 rows each, and the sorted copy of x (half of that, where rows are
    gathered) stay untouched."""
    p = c.experts
    blocks = p.I // 128 if p.I % 128 == 0 else 1
    most = 4 if blocks % 4 == 0 else 2 if blocks % 2 == 0 else 1
    part = 4 * 2 * p.T_max * p.k * p.H
    untouched = 4 * int((c.ws[4608:].view(torch.int32) == -0x5A5A5A5B).sum())
    return most - untouched // part


@pytest.mark.parametrize("layout", [0, 1, 2], ids=["rows", "packed", "mxfp8"])
@pytest.mark.parametrize("form", [0, 2], ids=["separate", "one_kernel"])
@pytest.mark.parametrize("case,parts", SPLITS, ids=lambda v: "I{I}".format(**v) if isinstance(v, dict) else f"parts{v}")
def test_layer_splits_the_down_product(B, case, parts, form, layout):
    if layout and case["H"] % 128:
        pytest.skip("packed and MXFP8 weights come in tiles of 128 rows")
    c = LayerCase(B, form=form, layout=layout, **case)
    c.ws[4608:].fill_(0xA5)
    o = c.run()
    torch.cuda.synchronize()
    assert parts_used(c) == parts
    c.verify(o)
    same_bits(c.run(), o)
    n = c.T - 1                          # fewer tokens than the description's, by the device count
    fewer = c.run(T_dev=n)
    for key, fill in (("h", 7.0), ("x_next", 7.0), ("ids", -9), ("weights", -9.0)):
        if o[key] is not None:
            assert torch.equal(fewer[key][:n], o[key][:n]) and (fewer[key][n:] == fill).all(), key


# The one-kernel form's tail: a token's row in several items (of 1024 columns, or 2048 with MXFP8 weights) on
# several CTAs, the last of them partly filled; the row sums meet through the GPU-wide count.
TAILS = [
    dict(T=1, E=8, k=2, H=2880, I=128),
    dict(T=5, E=16, k=3, H=2880, I=192, h="fp32", gate=1),
    dict(T=16, E=16, k=2, H=7168, I=128, post=False, gate=3),
    dict(T=9, E=8, k=2, H=7168, I=128, nxt=False, gate=2, w="fp32"),
    dict(T=3, E=8, k=2, H=7168, I=128, h="fp32", layout=2),
    dict(T=17, E=16, k=2, H=2880, I=128, h="fp32", offset=True),          # more tokens than the router's last CTA takes
    dict(T=40, E=64, k=4, H=1088, I=64, score=1, bias=True, post=False, nxt=False),
    dict(T=128, E=256, k=2, H=1152, I=128, layout=2, gate=1),
    dict(T=2, E=4, k=1, H=16384, I=64, stride=16392),
]


@pytest.mark.parametrize("case", TAILS, ids=lambda c: "T{T}E{E}k{k}H{H}I{I}".format(**c))
def test_layer_one_kernel_tail(B, case):
    c = LayerCase(B, form=2, **case)
    o = c.run()
    c.verify(o)
    for _ in range(8):                   # the sums in any order of the CTAs give the same bits
        same_bits(c.run(), o)
    for n in (0, c.T // 2):
        fewer = c.run(T_dev=n)
        for key, fill in (("h", 7.0), ("x_next", 7.0), ("ids", -9), ("weights", -9.0)):
            if o[key] is not None:
                assert torch.equal(fewer[key][:n], o[key][:n]) and (fewer[key][n:] == fill).all(), (key, n)
    assert B.moe_last_device_error(c.ws) == 0
    assert int(c.ws[4:HEADER_BYTES].count_nonzero()) == 0


def test_layer_one_kernel_form_is_refused_where_it_does_not_fit(B):
    """MXFP8 weights and more than two paired rows an expert on average: 32-row tiles, which the form does not have.
    Nothing is launched."""
    c = LayerCase(B, T=3, E=4, k=2, H=256, I=128, layout=2, form=2)
    with pytest.raises(B.MoeError) as ei:
        c.run()
    assert ei.value.status == 5
    torch.cuda.synchronize()
    assert int(c.ws.count_nonzero()) == 0


@pytest.mark.parametrize("case", [
    dict(T=1, E=8, k=4, H=512, I=1024),                       # K parts
    dict(T=8, E=8, k=4, H=2048, I=512),
    dict(T=8, E=8, k=4, H=2048, I=512, path=2),               # 16-row tiles, asked for
    dict(T=64, E=16, k=4, H=1024, I=256),                     # 32-row tiles
    dict(T=128, E=8, k=4, H=512, I=256),                      # 128-row tiles
    dict(T=8, E=16, k=2, H=7168, I=128),
    dict(T=5, E=8, k=2, H=1024, I=512, layout=2),
    dict(T=64, E=8, k=2, H=512, I=256, layout=2),
    dict(T=5, E=8, k=2, H=1024, I=512, form=2),
], ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_layer_precision_of_an_fp32_stream(B, case):
    """The block's output as an fp32 stream shows it. x and h count with 16 bits: a relative 2^-17 of each element,
    through gate, up and down together at most 2^-16 of the output's rms; sums truncate by up to 2^-23 for each of
    their K / 16 steps; the norm's r is within 4e-6, and enters gate, up and their product."""
    c = LayerCase(B, h="fp32", post=False, nxt=False, **case)
    o = c.run()
    c.verify(o)
    h = ref.f64(c.h)
    v = ref.norm(h, ref.f64(c.w_pre), 1e-6)
    y = c.scale * ref.experts(v, o["ids"].cpu().numpy(), ref.f64(o["weights"]), c.ref13, c.ref2)
    off = np.sqrt(((ref.f64(o["h"]) - h - y) ** 2).mean() / (y ** 2).mean())
    stored = 2.0 ** -24 * np.sqrt((h ** 2).mean() / (y ** 2).mean())
    assert off <= 2.0 ** -16 + (case["H"] + case["I"]) / 16 * 2.0 ** -23 + 3 * 4e-6 + stored, off
