"""The example that runs the block's operators together: the decoder (moe_layer
in a graph) and the prompt (the operators one by one) give the same stream."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_prompt_and_decoder_agree():
    from moe_routed_expert_routing_gb300.build import build
    build()
    spec = importlib.util.spec_from_file_location("moe_block_example", os.path.join(ROOT, "examples", "moe_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    diff, finite = example.main(["--blocks", "2", "--prompt", "160", "--batch", "5", "--steps", "4", "--shape",
                                 "16,2,256,128"])
    assert finite
    # bf16 roundings of x, h and y in each of two blocks (2^-9 each, relative), and
    # now and then an expert on the edge of the selection
    assert diff < 0.05
