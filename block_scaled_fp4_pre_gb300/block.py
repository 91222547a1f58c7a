"""The half of a decoder block that holds the expert layer, on the package's operators.

    o        = attn Wo^T                       moe_linear_forward (MXFP4 x MXFP4)
    residual = residual + o, h = norm(...)     moe_rmsnorm_mxfp8
    m        = expert layer of h               moe_few_forward, or moe_pre_dispatch and
                                               moe_forward above 16 tokens
    residual = residual + m, (q, sf) = norm    moe_rmsnorm_mxfp8, the MXFP8 pair
    out      = (q, sf) Wn^T                    moe_linear_forward_pair (MXFP8 x MXFP4)

Wn is the projection that comes next (the next block's, or the output head's).  Up to 16
tokens the block routes itself, in six kernels; more take their routing from the caller.
`python -m block_scaled_fp4_pre_gb300.block --tokens 4` times one with random weights.
"""
from __future__ import annotations

import argparse

import torch

import block_scaled_fp4_pre_gb300 as mx

FEW_TOKENS = 16


def quantised(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Canonical MXFP4 codes and scales of an fp32 matrix [N, K]."""
    N, K = w.shape
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(N, K // 32, dtype=torch.uint8, device=w.device)
    mx.moe_quantize_mxfp4(w, codes, scales)
    return codes, scales


class Linear:
    """Prepared weights and a workspace of one MXFP4 linear product."""

    def __init__(self, codes, scales, max_rows: int, mma_type: int):
        N, K = codes.shape[0], codes.shape[1] * 2
        self.dims = mx.make_linear_dims(N, K, max_rows, mma_type)
        u8, dev = torch.uint8, codes.device
        self.prepared = torch.empty(mx.moe_linear_weights_size(self.dims), dtype=u8, device=dev)
        mx.moe_linear_prepare(self.dims, codes, scales, self.prepared)
        self.ws = torch.empty(mx.moe_linear_workspace_size(self.dims), dtype=u8, device=dev)
        mx.moe_linear_workspace_init(self.dims, self.ws)


class ExpertBlock:
    """Buffers and weights of one half block, for up to dims.max_tokens tokens.

    wo and wn are (codes, scales) of [H, attn features] and [next features, H]; prepared is
    the expert layer's blob, router bf16 [E, H], the gammas bf16 [H]."""

    def __init__(self, dims: mx.MoeDims, wo, prepared, router, wn, gamma_in, gamma_out,
                 eps: float = 1e-6):
        T, H, dev = dims.max_tokens, dims.hidden, prepared.device
        self.dims, self.prepared, self.router, self.eps = dims, prepared, router, eps
        self.gamma_in, self.gamma_out = gamma_in, gamma_out
        self.wo = Linear(*wo, T, mx.MOE_MMA_MXF4xMXF4)
        self.wn = Linear(*wn, T, mx.MOE_MMA_FP8xFP4)
        self.ws = torch.empty(mx.moe_workspace_size(dims), dtype=torch.uint8, device=dev)
        mx.moe_workspace_init(dims, self.ws)
        bf = torch.bfloat16
        self.o, self.h, self.m = (torch.empty(T, H, dtype=bf, device=dev) for _ in range(3))
        self.ids = torch.empty(T, dims.topk, dtype=torch.int32, device=dev)
        self.weights = torch.empty(T, dims.topk, dtype=torch.float32, device=dev)
        self.q = torch.empty(T, H, dtype=torch.uint8, device=dev)
        self.sf = torch.empty(mx.moe_mxfp8_scale_bytes(T, H, mx.MOE_SF_128X4), dtype=torch.uint8,
                              device=dev)
        self.out = torch.empty(T, self.wn.dims.out_features, dtype=bf, device=dev)

    def forward(self, attn, residual, routing=None, stream=None):
        """attn bf16 [T, features], residual bf16 [T, H] (updated in place) -> bf16 [T, next
        features], a view of a buffer that the next call overwrites.  routing: (ids, weights)
        for the expert layer instead of the block's router; needed above 16 tokens."""
        T, k = attn.shape[0], self.dims.topk
        # before the residual changes
        if routing is None and T > FEW_TOKENS:
            raise ValueError(f"{T} tokens: above {FEW_TOKENS} the routing is the caller's")
        for t, dtype in zip(routing or (), (torch.int32, torch.float32)):
            if t.dtype is not dtype or t.shape != (T, k) or not t.is_contiguous():
                raise ValueError(f"routing: need contiguous {dtype} [{T}, {k}], got {t.dtype} "
                                 f"{list(t.shape)}")
        o, h, m, q, out = (b[:T] for b in (self.o, self.h, self.m, self.q, self.out))
        mx.moe_linear_forward(self.wo.dims, self.wo.prepared, attn, o, self.wo.ws, stream)
        mx.moe_rmsnorm_mxfp8(o, self.gamma_in, self.eps, residual=residual, residual_out=residual,
                             y=h, stream=stream)
        if T <= FEW_TOKENS:
            ids, weights = routing or (self.ids, self.weights)
            mx.moe_few_forward(self.dims, self.prepared, None if routing else self.router, h, ids,
                               weights, T, self.ws, m, stream)
        else:
            mx.moe_pre_dispatch(self.dims, h, *routing, T, self.ws, stream)
            mx.moe_forward(self.dims, self.prepared, self.ws, m, T, stream)
        mx.moe_rmsnorm_mxfp8(m, self.gamma_out, self.eps, q, self.sf, residual=residual,
                             residual_out=residual, stream=stream)
        mx.moe_linear_forward_pair(self.wn.dims, self.wn.prepared, q, self.sf, T, out, self.wn.ws,
                                   stream)
        return out

    def check(self, stream=None) -> None:
        """Synchronises and raises what the kernels recorded (a routing error, a timeout)."""
        mx.moe_check(self.ws, stream)
        mx.moe_linear_check(self.wo.ws, stream)
        mx.moe_linear_check(self.wn.ws, stream)


def random_block(dims: mx.MoeDims, attn_features: int, next_features: int, seed: int = 0):
    """A block with N(0, 1/sqrt(K)) weights on the current device."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5

    E, H, I = dims.num_experts, dims.hidden, dims.inter
    can = []
    for rows, K in ((2 * I, H), (H, I)):
        parts = [quantised(normal(rows, K)) for _ in range(E)]
        can += [torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])]
    prepared = torch.empty(mx.moe_prepared_weights_size(dims), dtype=torch.uint8, device="cuda")
    mx.moe_prepare_weights(dims, *can, prepared)
    torch.cuda.synchronize()
    gammas = [(1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    return ExpertBlock(dims, quantised(normal(H, attn_features)), prepared,
                       normal(E, H).bfloat16(), quantised(normal(next_features, H)), *gammas)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1, help="1..16")
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=256)
    ap.add_argument("--topk", type=int, default=6)
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    if not 1 <= a.tokens <= FEW_TOKENS:
        ap.error("--tokens: 1..16")
    dims = mx.make_dims(a.hidden, a.inter, a.experts, a.topk, a.tokens)
    block = random_block(dims, a.hidden, a.hidden)
    attn = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    residual = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    start = residual.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    block.forward(attn, residual)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.capture_begin()
        residual.copy_(start)
        block.forward(attn, residual)
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
    print(f"{a.tokens} tokens: {begin.elapsed_time(end) * 1e3 / a.steps:.1f} us a half block "
          f"(hidden {a.hidden}, inter {a.inter}, {a.experts} experts, top-{a.topk}; the same "
          "tokens each step, so their experts' weights may stay in L2)")


if __name__ == "__main__":
    main()
