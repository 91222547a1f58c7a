"""One key that outweighs all others: the output is its value row, so that a row of the cache that
is lost, doubled or taken from another place is an error of the output's size, however long the
context.

A needle's logit is 20 or more above every other key's, of which there are fewer than 2^13: the
others weigh under 2^13 e^-20 < 2^-15 together, with values below 8 of size (normal, 5 sigma and
more) an error under 2^-11; the needle's weight and the output are each rounded by 2^-8."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests.attention64 import Paged

pytestmark = pytest.mark.gpu


def needles(p, at, i=0):
    """Gives head h of new token i of sequence b a needle at at(b, h), by a direction of its own in
    keys that are otherwise 0 in it, and checks that the output is the value row there."""
    G = p.hq // p.hk
    # head h of a kv head's group asks along dimension h % G: 16 * 16 / sqrt(D) >= 22
    p.q.zero_()
    p.k[..., :G] = torch.where(torch.isnan(p.k[..., :G]), p.k[..., :G], 0)
    want = torch.empty(len(p.new), p.hq, p.D, dtype=torch.float64, device="cuda")
    for b in range(len(p.new)):
        for h in range(p.hq):
            g, d = divmod(h, G)
            page, r = p.slot(b, at(b, h))
            p.q[p.cu[b] + i, h, d] = 16.0
            p.k[page, g, r, d] = 16.0
            want[b, h] = p.v[page, g, r].double()
    out, lse = p.run()
    got = out[[p.cu[b] + i for b in range(len(p.new))]].double()
    assert want.abs().max() < 8
    assert torch.all((got - want).abs() <= want.abs() * 2.0 ** -7 * 1.01 + 2.0 ** -11)


CONTEXTS = [1000, 2500, 5000]


def places(length, page):
    """Positions about the ends of tiles, pages and boxes, and everywhere between."""
    edges = {0, 1, length - 1, length - 2}
    for step in (16, 64, 128, page):
        for k in (1, 2, 3, length // step // 2, length // step - 1, length // step):
            edges |= {k * step - 1, k * step}
    edges |= set(range(7, length, length // 60))
    return sorted(e for e in edges if 0 <= e < length)


# new tokens and heads that take the few-row kernel, one row tile, two row tiles; q heads of one kv
# head ask for needles of their own
@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("D,new,q_heads,kv_heads", [(128, 1, 32, 4), (64, 1, 16, 2),
                                                    (128, 9, 32, 4), (64, 40, 16, 2),
                                                    (128, 70, 32, 4)])
def test_needles(D, new, q_heads, kv_heads, shared, page):
    common = 768 if shared else 0
    p = Paged(new=[new] * 3, old=[c - common - new for c in CONTEXTS], q_heads=q_heads,
              kv_heads=kv_heads, D=D, page=page, shared=common, uniform=True)
    keys = p.k.clone()
    spots = [places(c - new + 1, page) for c in CONTEXTS]       # seen by the first new token
    for k in range(-(-max(map(len, spots)) // q_heads)):
        def at(b, h):
            # the prefix's rows are every sequence's: a head has its needle there in all of them
            first, x = (s[(k * q_heads + h) % len(s)] for s in (spots[0], spots[b]))
            return first if min(first, x) < common else x
        p.k.copy_(keys)
        needles(p, at, i=0 if k % 2 else new - 1)


@pytest.mark.parametrize("page", [16, 128])
def test_needles_of_a_long_context(page):
    # a range of keys a block, and an item of more parts than any other here
    p = Paged(new=[1], old=[8100], q_heads=64, kv_heads=8, page=page, uniform=True)
    keys = p.k.clone()
    for k in range(4):
        p.k.copy_(keys)
        needles(p, lambda b, h: (h * 127 + k * 31) % p.lens[0])
