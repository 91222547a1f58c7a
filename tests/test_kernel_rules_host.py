"""Rules of the kernels that break without a failing result, read from their source."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_scaled_fp4_pre_gb300", "csrc")


def kernels(name: str) -> dict:
    """Body of every __global__ function of a file, comments removed."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = {}
    for m in re.finditer(r"__global__\b", text):
        start = text.index("{\n", m.end())
        head = text[m.end():start]
        depth, i = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        found[re.findall(r"(\w+)\(", head.replace("__launch_bounds__(", ""))[-1]
              if "(" in head else head] = text[start:i]
    return found


def test_the_reader_finds_the_kernels():
    assert {"few_logits_kernel", "few_expert_kernel"} <= set(kernels("few.cu"))
    assert {"linear_kernel", "linear_pair_kernel", "linear_split_kernel"} <= set(kernels("linear.cu"))


def met_always(body: str, at: int) -> bool:
    """Whether some cluster barrier before `at` is met whatever the call's sizes: its statement
    is under no condition but CLUSTER, or under one whose block holds `at` too."""
    for m in re.finditer(r"ptx::cluster_(?:wait|sync)\(\)", body[:at]):
        line = body[body.rindex("\n", 0, m.start()) + 1:m.start()]
        cond = re.search(r"if \((.*)\)\s*$", line)
        if cond and cond.group(1) != "CLUSTER":
            continue
        depth = low = 0
        for ch in body[m.start():at]:
            depth += {"{": 1, "}": -1}.get(ch, 0)
            low = min(low, depth)
        if low == 0:
            return True
    return False


@pytest.mark.parametrize("name", ["few.cu", "linear.cu"])
def test_no_store_to_another_block_before_every_block_runs(name):
    # shared memory of another block of the cluster may be accessed only once it has started
    seen = 0
    for kernel, body in kernels(name).items():
        at = body.find("st_cluster")
        if at >= 0:
            seen += 1
            assert met_always(body, at), kernel
    assert seen


@pytest.mark.parametrize("name", ["few.cu", "linear.cu"])
def test_no_block_leaves_with_copies_in_flight(name):
    # also after a wait that ran out: waits with a flag of their own, not the block's abort
    seen = 0
    for kernel, body in kernels(name).items():
        issue = [body.rfind(f) for f in ("tma_load_2d", "tma_load_3d", "bulk_load")]
        if max(issue) >= 0:
            seen += 1
            assert "&never" in body[max(issue):], kernel
    assert seen
