"""Programmatic dependent launch, read from the sources (host only).

A kernel lets its dependents start (``pdl_trigger``) when one thread of each of
its blocks has said so. The library's kernels count on every kernel two or more
launches back having completed by then, so each thread of a kernel that triggers
has to have waited for the kernel ahead (``pdl_wait``) first, on every way
through it: a wait in the trigger's own block or in one around it, not behind a
condition, or two waits behind a condition and its negation.
"""
from __future__ import annotations

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_routed_expert_routing_gb300", "csrc")


def kernels(text):
    """(name, body) of every __global__ function of a source without comments."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for m in re.finditer(r"__global__", text):
        start = text.index("{", m.end())
        depth = 0
        for i in range(start, len(text)):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            if depth == 0:
                break
        yield re.findall(r"(\w+)\s*\(", text[m.end():start].split("__grid_constant__")[0])[-1], text[start:i + 1]


def calls(body, name):
    """(position, blocks around it, condition or None) of each call `name();`: the blocks as the
    positions of their braces, the condition that of an `if` (or "else") without braces."""
    for m in re.finditer(rf"\b{name}\(\);", body):
        blocks = []
        for i, c in enumerate(body[:m.start()]):
            if c == "{":
                blocks.append(i)
            elif c == "}":
                blocks.pop()
        before = body[:m.start()].rstrip()
        statement = re.split(r"[;{}]", before)[-1].strip()
        yield m.start(), tuple(blocks), re.sub(r"\s+", " ", statement) or None


def unwaited(body):
    """Triggers of a kernel that some thread may reach without a wait."""
    waits = list(calls(body, "pdl_wait"))
    bad = []
    for at, blocks, _ in calls(body, "pdl_trigger"):
        ahead = [(b, c) for p, b, c in waits if p < at and blocks[:len(b)] == b]
        always = any(c is None for _, c in ahead)
        conditions = {c[2:].strip() for _, c in ahead if c and c.startswith("if")}     # with their brackets
        if not always and not any(f"(!{c})" in conditions for c in conditions):
            bad.append(at)
    return bad


def sources():
    return sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")))


@pytest.mark.parametrize("name", sources())
def test_every_thread_waits_before_dependents_may_start(name):
    with open(os.path.join(CSRC, name)) as f:
        for kernel, body in kernels(f.read()):
            assert not unwaited(body), (name, kernel)


def test_what_the_reading_tells_apart():
    assert not unwaited("{ pdl_wait(); if (x) { y(); } pdl_trigger(); }")
    assert not unwaited("{ for (;;) { if (p) { pdl_wait(); pdl_trigger(); } } }")
    assert not unwaited("{ if (!(a && b)) pdl_wait(); f(); if (a && b) pdl_wait(); pdl_trigger(); }")
    assert unwaited("{ if (w != 2) pdl_wait(); pdl_trigger(); }")
    assert unwaited("{ if (a) { pdl_wait(); } pdl_trigger(); }")
    assert unwaited("{ pdl_trigger(); pdl_wait(); }")


def test_kernels_are_found():
    found = set()
    for name in sources():
        with open(os.path.join(CSRC, name)) as f:
            found |= {k for k, body in kernels(f.read()) if "pdl_trigger" in body}
    assert {"act_grad_kernel", "products_kernel", "select_kernel", "norm_backward_few_kernel"} <= found
