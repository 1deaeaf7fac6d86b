"""moe_layer in the forms that its shape, its description and its kernels' waits
bring about: rows beyond the routed slots, K parts of the down product, the
one-kernel form's rows over several CTAs, waits that run out."""
from __future__ import annotations

import time

import pytest
import torch

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
