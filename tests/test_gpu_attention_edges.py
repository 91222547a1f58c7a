"""Attention at the ends of what its arguments may be."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests.attention64 import Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 40])
def test_a_scale_whose_logits_have_no_fp32(new):
    # queries of 0: every logit is 0 whatever the scale, and the output the values' mean
    p = Paged(new=[new], old=[30])
    p.q.zero_()
    out = torch.full_like(p.q, 77.0)
    for scale in (2.4e38, 3.4e38):                     # finite; times log2 e they are not
        with pytest.raises(mx.MoeError) as e:
            p.run(out=out, scale=scale)
        assert e.value.status == mx.MOE_ERR_INVALID_ARG
    assert torch.all(out == 77)
    for scale in (2.3e38, 1e-45):
        out, lse = p.run(scale=scale)
        p.check(out, lse, scale)
