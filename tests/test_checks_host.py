"""Calls that read a workspace's error bits stay on the stream that they are given: read from
their source."""
from __future__ import annotations

import os
import re

import pytest

from tests.test_kernel_rules_host import CSRC


def function(name: str, file: str) -> str:
    with open(os.path.join(CSRC, file)) as f:
        text = f.read()
    start = text.index(f"moe_status {name}(")
    return text[start:text.index("\n}\n", start)]


@pytest.mark.parametrize("name,file", [("moe_attention_check", "attn_api.cu"),
                                       ("moe_check", "api.cu"),
                                       ("moe_linear_check", "ops.cu")])
def test_a_check_uses_no_other_stream(name, file):
    # cudaMemset on the default stream is not ordered with what another stream runs next
    body = function(name, file)
    assert not re.search(r"\bcudaMem(?:cpy|set)\(", body)
    assert "read_flags(" in body and re.search(r"if \(flag && .*clear_flags\(", body)
