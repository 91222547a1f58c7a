"""A key with a NaN shows in both outputs of the tokens that see it, and in no other's."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests.attention64 import Paged

pytestmark = pytest.mark.gpu


# few rows: whole and cut items; tiles: rows for one row tile and for both, cut and whole; a prefix
# in one pass or for each sequence
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,old,shared", [
    ([1, 1], [40, 40], 0), ([1], [3000], 0), ([3, 1], [500, 70], 0), ([12, 20], [100, 0], 0),
    ([12], [3000], 0), ([150], [20], 0), ([300], [1500], 0), ([1, 1, 1], [5, 9, 30], 64),
    ([40, 20], [0, 7], 256)])
def test_nan_in_a_key(new, old, shared, D):
    p = Paged(new=new, old=old, shared=shared, D=D)
    for mode in (mx.MOE_SHARED_ALWAYS, mx.MOE_SHARED_NEVER) if shared else (mx.MOE_SHARED_AUTO,):
        mx.moe_attention_set_shared(p.ws, mode)
        clean, clean_lse = p.run()
        first = p.lens[0] - new[0]                    # position of the first new token
        for j in sorted({0, shared // 2, first // 2, first, p.lens[0] - 1}):
            page, r = p.slot(0, j)
            kept = p.k[page, 1, r, 3].clone()
            p.k[page, 1, r, 3] = float("nan")
            out, lse = p.run()
            p.k[page, 1, r, 3] = kept
            sees = torch.zeros(p.T, p.hq, dtype=torch.bool, device="cuda")
            for b, n in enumerate(new):
                if b == 0 or j < shared:
                    i0 = max(0, j - (p.lens[b] - n))
                    sees[p.cu[b] + i0:p.cu[b] + n, p.hq // p.hk:] = True
            assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all(), j
            # The others' running maxima may be raised at another tile, so their terms round
            # differently.  Each side is within 2^-8 sum p |v| and one rounding, 2^-8, of the
            # exact value: the two within 4 2^-8 of the largest |v|, and a little.
            seen = torch.nan_to_num(p.v).abs().max().double()
            apart = (out[~sees].double() - clean[~sees].double()).abs()
            assert torch.all(apart <= seen * 2.0 ** -6 * 1.05), j
            assert torch.all((lse[~sees] - clean_lse[~sees]).abs()
                             <= (clean_lse[~sees].abs() + 1) * 2.0 ** -18), j
