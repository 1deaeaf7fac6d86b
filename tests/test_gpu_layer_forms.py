"""moe_layer in the forms that its shape, its description and its kernels' waits
bring about: rows beyond the routed slots, K parts of the down product, the
one-kernel form's rows over several CTAs, waits that run out."""
from __future__ import annotations

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
