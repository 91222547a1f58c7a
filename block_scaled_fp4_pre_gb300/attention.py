"""The half of a decoder block that holds attention, on the package's operators, and the whole
block with the expert half of block.py.

    q, k, v  = rows of the projection before           the last block's `out`, [T, (Hq + 2 Hkv) D]
    cache   <- rotated k, v; q rotated                  moe_kv_append
    attn     = softmax(q K^T / sqrt(D)) V               moe_attention over the paged cache
    out      = the expert half on attn and residual     block.ExpertBlock, whose projection is the
                                                        next block's q, k, v

`python -m block_scaled_fp4_pre_gb300.attention --sequences 4 --context 4096` times one decode
step of a block with random weights.
"""
from __future__ import annotations

import argparse

import torch

import block_scaled_fp4_pre_gb300 as mx
from block_scaled_fp4_pre_gb300 import block as blk


class Attention:
    """A layer's paged cache, rotation (of the caller's frequencies, if given) and buffers, for up
    to dims.max_tokens tokens a step.

    The workspace (42 MB and more at 128 elements a head) holds nothing between calls: layers whose
    calls follow one another on one stream can share that of the first, `ws`."""

    def __init__(self, dims: mx.AttentionDims, rope: mx.RopeDims, device="cuda",
                 frequencies=None, ws=None):
        u8, bf = torch.uint8, torch.bfloat16
        self.dims, self.rope = dims, rope
        self.table = torch.empty(mx.moe_rope_table_size(rope), dtype=u8, device=device)
        if frequencies is None:
            mx.moe_rope_prepare(rope, self.table)
        else:
            mx.moe_rope_prepare_frequencies(rope, frequencies, self.table)
        self.k_cache, self.v_cache = (torch.zeros(dims.cache_shape, dtype=bf, device=device)
                                      for _ in range(2))
        self.ws = ws
        if ws is None:
            self.ws = torch.empty(mx.moe_attention_workspace_size(dims), dtype=u8, device=device)
            mx.moe_attention_workspace_init(dims, self.ws)
        self.q, self.attn = (torch.empty(dims.max_tokens, dims.q_heads, dims.head_dim, dtype=bf,
                                         device=device) for _ in range(2))

    def forward(self, qkv, batch: mx.KvBatch, stream=None):
        """qkv bf16 [T, (q_heads + 2 kv_heads) * head_dim] of the batch's new tokens -> bf16
        [T, q_heads * head_dim], a view of a buffer that the next call overwrites.  Rows of tokens
        that the batch leaves out keep what they held."""
        d, T = self.dims, qkv.shape[0]
        heads = (d.q_heads, d.kv_heads, d.kv_heads)
        q, k, v = qkv.unflatten(1, (sum(heads), d.head_dim)).split(heads, 1)
        rotated, attn = self.q[:T], self.attn[:T]
        mx.moe_kv_append(d, batch, k, v, self.k_cache, self.v_cache, self.ws, rope=self.rope,
                         table=self.table, q=q, q_out=rotated, stream=stream)
        mx.moe_attention(d, batch, rotated, self.k_cache, self.v_cache, attn, self.ws,
                         stream=stream)
        return attn.flatten(1)

    def check(self, stream=None) -> None:
        """Synchronises and raises what the kernels recorded (a page outside the cache)."""
        mx.moe_attention_check(self.ws, stream)


class DecoderBlock:
    """One decoder block between two projections: from a block's q, k, v rows to the next's."""

    def __init__(self, attention: Attention, experts: blk.ExpertBlock):
        self.attention, self.experts = attention, experts

    def forward(self, qkv, residual, batch: mx.KvBatch, routing=None, stream=None):
        """residual bf16 [T, H] is updated in place; the rest as the halves' forward."""
        attn = self.attention.forward(qkv, batch, stream)
        return self.experts.forward(attn, residual, routing, stream)

    def check(self, stream=None) -> None:
        self.attention.check(stream)
        self.experts.check(stream)


def random_decoder_block(dims: mx.MoeDims, attention: mx.AttentionDims, rope: mx.RopeDims,
                         seed: int = 0) -> DecoderBlock:
    """A block with N(0, 1/sqrt(K)) weights on the current device."""
    features = attention.q_heads * attention.head_dim
    nxt = features + 2 * attention.kv_heads * attention.head_dim
    return DecoderBlock(Attention(attention, rope), blk.random_block(dims, features, nxt, seed))


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--sequences", type=int, default=1, help="1..16, one new token each")
    ap.add_argument("--context", type=int, default=4096, help="tokens of each sequence")
    ap.add_argument("--shared", type=int, default=0, help="of them in common (whole pages of 64)")
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=256)
    ap.add_argument("--topk", type=int, default=6)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    B, page = a.sequences, 64
    if not 1 <= B <= blk.FEW_TOKENS:
        ap.error("--sequences: 1..16")
    if a.shared % page or not 0 <= a.shared < a.context:
        ap.error("--shared: whole pages of 64, below --context")
    common = a.shared // page
    own = -(-a.context // page) - common
    dims = mx.make_dims(a.hidden, a.inter, a.experts, a.topk, B)
    attention = mx.make_attention_dims(a.heads, a.kv_heads, 128, common + B * own, page, B, B)
    block = random_decoder_block(dims, attention, mx.make_rope_dims(128))
    pages = torch.arange(common + B * own, dtype=torch.int32, device="cuda")
    table = torch.cat((pages[:common].expand(B, common), pages[common:].view(B, own)), 1)
    lens = torch.full((B,), a.context, dtype=torch.int32, device="cuda")
    batch = mx.make_kv_batch(lens, table.contiguous(), B, shared_len=a.shared)
    for cache in (block.attention.k_cache, block.attention.v_cache):
        cache.normal_()
    qkv = torch.randn(B, (a.heads + 2 * a.kv_heads) * 128, device="cuda").bfloat16()
    residual = torch.randn(B, a.hidden, device="cuda").bfloat16()
    start = residual.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    block.forward(qkv, residual, batch)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.capture_begin()
        residual.copy_(start)
        block.forward(qkv, residual, batch)
        graph.capture_end()
    for _ in range(10):
        graph.replay()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    block.check()
    print(f"{B} sequences of {a.context} tokens, {a.shared} in common: "
          f"{begin.elapsed_time(end) * 1e3 / a.steps:.1f} us a block (hidden {a.hidden}, "
          f"{a.heads} heads on {a.kv_heads}, inter {a.inter}, {a.experts} experts, top-{a.topk}; "
          "the same tokens each step, so what they use may stay in L2)")


if __name__ == "__main__":
    main()
