"""A paged cache, its batch and attention over it in 64 bits."""
from __future__ import annotations

import math
import random

import torch

import block_scaled_fp4_pre_gb300 as mx


def turns64(dims, positions):
    """cos and sin [tokens, pairs] of a rotation, magnitude included, in 64 bits."""
    d = dims.rotary_dim
    i = torch.arange(0, d, 2, dtype=torch.float64) / d
    base, m = dims.base, 1.0
    if dims.scaling == mx.MOE_ROPE_NTK:
        base *= dims.factor ** (d / (d - 2))
    w = base ** -i
    if dims.scaling == mx.MOE_ROPE_LINEAR:
        w = w / dims.factor
    if dims.scaling == mx.MOE_ROPE_YARN:
        t = dims.original_length * w / (2 * math.pi)
        g = ((t - dims.beta_slow) / (dims.beta_fast - dims.beta_slow)).clamp(0, 1)
        w, m = w * g + w / dims.factor * (1 - g), 0.1 * math.log(dims.factor) + 1
    m = dims.magnitude or m
    a = positions.cpu().double().unsqueeze(1) * w
    return m * torch.cos(a), m * torch.sin(a)


def rotated64(dims, x, positions):
    """The rotation of x [tokens, heads, D] and, beside it, |a| + |b| of each pair (0 for what is
    copied)."""
    cos, sin = (t.unsqueeze(1) for t in turns64(dims, positions))
    y, size = x.cpu().double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    d = dims.rotary_dim
    first, second = (slice(0, d // 2), slice(d // 2, d)) if dims.layout == mx.MOE_ROPE_HALF \
        else (slice(0, d, 2), slice(1, d, 2))
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    size[..., first] = size[..., second] = a.abs() + b.abs()
    return y, size


class Paged:
    """Sequences of `old` tokens behind `shared` common ones and `new` new ones.  The cache's rows
    that no sequence reaches hold NaN."""

    def __init__(self, new, old, q_heads=8, kv_heads=2, D=128, page=16, shared=0, seed=0,
                 uniform=False, spare=0, max_shared=None, tail=0, wide=0, q_size=2.0,
                 share=mx.MOE_SHARED_ALWAYS):
        rng, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.shared, self.D, self.page = new, shared, D, page
        self.hq, self.hk = q_heads, kv_heads
        # a length below 0 new tokens' worth: old < 0 leaves the first new tokens out
        self.lens = [max(0, shared + o + n) for n, o in zip(new, old)]
        common = shared // page
        counts = [max(0, -(-n // page) - common) for n in self.lens]
        ids = list(range(common + sum(counts) + spare))
        rng.shuffle(ids)
        width = max([1, common] + [-(-n // page) for n in self.lens]) + wide
        self.table = torch.full((len(new), width), -7, dtype=torch.int32)
        self.table[0, :common] = torch.tensor(ids[:common], dtype=torch.int32)
        at = common
        for b, k in enumerate(counts):
            self.table[b, common:common + k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
            at += k
        self.T = sum(new) + tail
        shape = (len(ids), kv_heads, page, D)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
                          for _ in range(2))
        for b in range(len(new)):
            at = [self.slot(b, j) for j in range(shared if b else 0, self.lens[b])]
            if at:
                p, r = (torch.tensor(x, device="cuda") for x in zip(*at))
                for cache in (self.k, self.v):
                    cache[p, :, r] = torch.randn(len(at), kv_heads, D, generator=g,
                                                 device="cuda").bfloat16()
        self.q = (torch.randn(self.T, q_heads, D, generator=g, device="cuda") * q_size).bfloat16()
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu = cu
        self.dims = mx.make_attention_dims(q_heads, kv_heads, D, len(ids), page, max(1, self.T),
                                           (self.T if max_shared is None else max_shared)
                                           if shared else 0)
        self.batch = mx.make_kv_batch(
            torch.tensor(self.lens, dtype=torch.int32, device="cuda"), self.table.cuda(), self.T,
            cu_new=None if uniform else torch.tensor(cu, dtype=torch.int32, device="cuda"),
            max_new=max(1, max(new)), shared_len=shared)
        self.ws = torch.empty(mx.moe_attention_workspace_size(self.dims), dtype=torch.uint8,
                              device="cuda").fill_(255)
        mx.moe_attention_workspace_init(self.dims, self.ws)
        mx.moe_attention_set_shared(self.ws, share)

    def slot(self, b, j):
        return int(self.table[0 if j < self.shared else b, j // self.page]), j % self.page

    def rows(self, cache, b):
        """A sequence's rows [length, kv heads, D] of a cache, in 64 bits."""
        at = [self.slot(b, j) for j in range(self.lens[b])]
        if not at:
            return cache.new_zeros(0, self.hk, self.D).double()
        p, r = (torch.tensor(x, device="cuda") for x in zip(*at))
        return cache[p, :, r].double()

    def run(self, q=None, out=None, lse=True, scale=None, stream=None):
        q = self.q if q is None else q
        out = torch.full_like(q, 77.0) if out is None else out
        l = torch.full((self.T, self.hq), 77.0, device="cuda") if lse else None
        mx.moe_attention(self.dims, self.batch, q, self.k, self.v, out, self.ws, lse=l,
                         scale=scale, stream=stream)
        mx.moe_attention_check(self.ws, stream)
        return out, l

    def check(self, out, lse, scale=None):
        """Every output within its tolerance of 64 bits.  With s a logit, its products and sums
        in fp32 are off by e = (D + 4) 2^-23 scale sum |q k|, a probability by 2 e and its
        rounding to bf16, 2^-8, relatively; sums over n keys add n 2^-23, joining parts of
        them 2^-20; and the output is rounded once, 2^-8."""
        scale = self.D ** -0.5 if scale is None else scale
        G = self.hq // self.hk
        for b, n in enumerate(self.new):
            K, V = self.rows(self.k, b), self.rows(self.v, b)
            t0 = self.cu[b]
            for i in range(n):
                end = self.lens[b] - n + i + 1
                q = self.q[t0 + i].double().view(self.hk, G, self.D)
                got = out[t0 + i].double().view(self.hk, G, self.D)
                if end <= 0:
                    assert torch.all(got == 0)
                    if lse is not None:
                        assert torch.all(lse[t0 + i] == -math.inf)
                    continue
                k, v = K[:end].permute(1, 2, 0), V[:end].transpose(0, 1)
                s = q @ k * scale
                e = ((q.abs() @ k.abs()) * scale * (self.D + 4) * 2.0 ** -23).amax(-1, True)
                top = torch.logsumexp(s, -1, keepdim=True)
                p = torch.exp(s - top)
                want, size = p @ v, p @ v.abs()
                tol = size * (2.0 ** -8 + 2 * torch.expm1(e) + end * 2.0 ** -23 + 2.0 ** -20)
                tol = tol + (want.abs() + tol) * 2.0 ** -8
                worst = ((got - want).abs() / tol).max()
                assert worst <= 1, (b, i, end, float(worst))
                if lse is not None:
                    l = lse[t0 + i].double().view(self.hk, G, 1)
                    tol = e + end * 2.0 ** -23 + (top.abs() + 1) * 2.0 ** -21
                    assert torch.all((l - top).abs() <= tol), (b, i, end)
        assert torch.all(out[self.cu[-1]:] == 77.0)
        if lse is not None:
            assert torch.all(lse[self.cu[-1]:] == 77.0)

    def check_rows(self, out, lse):
        """As check, sequence by sequence and head by head."""
        G, scale = self.hq // self.hk, self.D ** -0.5
        for b, n in enumerate(self.new):
            K, V = self.rows(self.k, b), self.rows(self.v, b)
            L, t = self.lens[b], slice(self.cu[b], self.cu[b + 1])
            ends = torch.arange(L - n + 1, L + 1, device="cuda").view(n, 1)
            hidden = torch.arange(L, device="cuda") >= ends
            for h in range(self.hq):
                q, k, v = self.q[t, h].double(), K[:, h // G], V[:, h // G]
                s = (q @ k.T * scale).masked_fill_(hidden, -math.inf)
                e = ((q.abs() @ k.abs().T).masked_fill_(hidden, 0).amax(-1, True) * scale
                     * (self.D + 4) * 2.0 ** -23)
                top = torch.logsumexp(s, -1, keepdim=True)
                p = torch.exp(s - top)
                want, size = p @ v, p @ v.abs()
                tol = size * (2.0 ** -8 + 2 * torch.expm1(e) + ends * 2.0 ** -23 + 2.0 ** -20)
                tol = tol + (want.abs() + tol) * 2.0 ** -8
                assert torch.all((out[t, h].double() - want).abs() <= tol), (b, h)
                tol = e + ends * 2.0 ** -23 + (top.abs() + 1) * 2.0 ** -21
                assert torch.all((lse[t, h].double().view(n, 1) - top).abs() <= tol), (b, h)
