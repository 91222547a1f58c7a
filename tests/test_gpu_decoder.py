"""The attention half and the whole decoder block: prompts, then decode steps, through the paged
cache, against 64 bits."""
from __future__ import annotations

import sys

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from block_scaled_fp4_pre_gb300 import attention as att
from tests.attention64 import rotated64

pytestmark = pytest.mark.gpu

HQ, HK, D, PAGE = 6, 2, 64, 16
ROPE = dict(head_dim=D, rotary_dim=48, layout=mx.MOE_ROPE_INTERLEAVED, scaling=mx.MOE_ROPE_YARN,
            factor=4.0, original_length=128.0)


def rows(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, (HQ + 2 * HK) * D, generator=g, device="cuda").bfloat16()


class Model:
    """What each sequence has been given, with its attention in 64 bits from the bf16 values that
    the layer holds (rotated queries and keys rounded once)."""

    def __init__(self, rope, sequences):
        self.rope = rope
        self.k, self.v = ([[] for _ in range(sequences)] for _ in range(2))

    def step(self, b, qkv, first):
        n = qkv.shape[0]
        pos = torch.arange(first, first + n)
        q, k, v = qkv.cpu().unflatten(1, (HQ + 2 * HK, D)).split((HQ, HK, HK), 1)
        self.k[b].append(rotated64(self.rope, k, pos)[0].bfloat16())
        self.v[b].append(v)
        return self.attend(b, rotated64(self.rope, q, pos)[0].bfloat16())

    def attend(self, b, q):
        """Outputs of the last rows and the tolerance: as attention64's, and half a step more of a
        rotated value's rounding on either side (it may round the other way next to a tie), which
        moves a logit by scale sum |q k| 2^-8 of the few values that do."""
        n, K, V = q.shape[0], torch.cat(self.k[b]).double(), torch.cat(self.v[b]).double()
        L = K.shape[0]
        hidden = torch.arange(L) > torch.arange(L - n, L).view(n, 1)
        out, tol = torch.empty(n, HQ, D, dtype=torch.float64), torch.empty(n, HQ, D,
                                                                            dtype=torch.float64)
        for h in range(HQ):
            k, v, x = K[:, h // (HQ // HK)], V[:, h // (HQ // HK)], q[:, h].double()
            s = (x @ k.T * D ** -0.5).masked_fill_(hidden, float("-inf"))
            p = torch.softmax(s, -1)
            out[:, h] = p @ v
            # a value next to a tie: one in a few hundred, so two of a row's products at most,
            # each at most the largest |q k| of the row times 2^-7
            e = 2 * (x.abs().amax(-1, True) * k.abs().amax()) * D ** -0.5 * 2.0 ** -7
            size = p @ v.abs()
            tol[:, h] = size * (2.0 ** -8 + 2 * torch.expm1(e + 2.0 ** -14) + 2.0 ** -16)
        return out, tol + (out.abs() + tol) * 2.0 ** -8


def make(tokens, sequences, width, shared_tokens=0):
    rope = mx.make_rope_dims(**ROPE)
    pages = sequences * width
    dims = mx.make_attention_dims(HQ, HK, D, pages, PAGE, tokens, shared_tokens)
    a = att.Attention(dims, rope)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).int().cuda()
    return a, rope, table.view(sequences, width)


def test_prompts_then_steps():
    lens = [37, 5, 90]
    a, rope, table = make(sum(lens), 3, 8)
    model = Model(rope, 3)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 37, 42, 132], dtype=torch.int32, device="cuda")
    qkv = rows(132, 1)
    out = a.forward(qkv, mx.make_kv_batch(seq, table, 132, cu_new=cu, max_new=90))
    a.check()
    got = out.cpu().double().view(-1, HQ, D)
    for b in range(3):
        t = slice(int(cu[b]), int(cu[b + 1]))
        want, tol = model.step(b, qkv[t], 0)
        assert torch.all((got[t] - want).abs() <= tol)
    step = mx.make_kv_batch(seq, table, 3)                # the same arrays, one token each
    for i in range(20):
        seq += 1
        qkv = rows(3, 10 + i)
        got = a.forward(qkv, step).cpu().double().view(3, HQ, D)
        for b in range(3):
            want, tol = model.step(b, qkv[b:b + 1], lens[b] + i)
            assert torch.all((got[b:b + 1] - want).abs() <= tol)
    a.check()


def test_steps_replayed_from_a_graph():
    # one captured step serves every length: the lengths are on the device
    a, rope, table = make(2, 2, 8)
    b, _, _ = make(2, 2, 8)
    seq = torch.zeros(2, dtype=torch.int32, device="cuda")
    batch = mx.make_kv_batch(seq, table, 2)
    qkv, out = rows(2, 0), torch.empty(2, HQ * D, dtype=torch.bfloat16, device="cuda")
    a.forward(qkv, batch)                                  # (length 0: nothing is appended)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.capture_begin()
        out.copy_(a.forward(qkv, batch))
        graph.capture_end()
    for i in range(40):
        seq += torch.tensor([1, i % 2], dtype=torch.int32, device="cuda")
        qkv.copy_(rows(2, 100 + i))
        graph.replay()
        assert torch.equal(out, b.forward(qkv, batch))
    assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)
    a.check()


def test_a_prefix_in_common():
    # one sequence's prompt serves the others; then each goes on by itself
    a, rope, table = make(40, 4, 8, 40)
    table[1:, :2] = table[0, :2]
    model = Model(rope, 4)
    seq = torch.full((4,), 32, dtype=torch.int32, device="cuda")
    prompt = rows(32, 1)
    first = mx.make_kv_batch(seq[:1], table[:1], 32)
    a.forward(prompt, first)
    model.step(0, prompt, 0)
    for b in range(1, 4):
        model.k[b], model.v[b] = list(model.k[0]), list(model.v[0])
    mx.moe_attention_set_shared(a.ws, mx.MOE_SHARED_ALWAYS)
    for n in (3, 1, 1, 10):
        seq += n
        qkv = rows(4 * n, 50 + n)
        got = a.forward(qkv, mx.make_kv_batch(seq, table, 4 * n, shared_len=32))
        got = got.cpu().double().view(4, n, HQ, D)
        for b in range(4):
            want, tol = model.step(b, qkv[b * n:(b + 1) * n], int(seq[b]) - n)
            assert torch.all((got[b] - want).abs() <= tol)
    a.check()


def test_whole_block_is_its_halves(monkeypatch, capsys):
    H, T = 512, 5
    dims = mx.make_dims(H, 256, 16, 4, T)
    adims = mx.make_attention_dims(HQ, HK, D, 5 * 4, PAGE, T)
    block = att.random_decoder_block(dims, adims, mx.make_rope_dims(**ROPE))
    other = att.Attention(adims, mx.make_rope_dims(**ROPE))
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(5, 4)
    seq = torch.zeros(5, dtype=torch.int32, device="cuda")
    batch = mx.make_kv_batch(seq, table, T)
    res = torch.randn(T, H, device="cuda").bfloat16()
    kept, qkv = res.clone(), rows(T, 9)
    for _ in range(4):
        seq += 1
        nxt = block.forward(qkv, res, batch).clone()
        attn = other.forward(qkv, batch)
        want = block.experts.forward(attn, kept)
        assert torch.equal(nxt, want) and torch.equal(res, kept)
        assert nxt.shape == qkv.shape and torch.isfinite(nxt).all()
        qkv = nxt                                          # the next block's rows
    block.check()
    argv = ("attention --sequences 3 --context 300 --shared 128 --hidden 512 --inter 256 "
            "--experts 16 --topk 4 --heads 8 --kv-heads 2 --steps 3")
    monkeypatch.setattr(sys, "argv", argv.split())
    att.main()
    assert "3 sequences of 300 tokens" in capsys.readouterr().out
