"""Attention over the paged cache against 64 bits (tolerances: attention64.Paged.check)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import block_scaled_fp4_pre_gb300 as mx
from tests.attention64 import Paged

pytestmark = pytest.mark.gpu


def both(**kw):
    p = Paged(**kw)
    out, lse = p.run()
    p.check(out, lse)
    return p, out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 5001])
def test_one_token(length, D):
    both(new=[1], old=[length - 1], D=D, uniform=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (3, 1), (4, 4), (7, 1), (10, 2), (16, 1),
                                              (34, 2), (40, 1), (128, 1)])
def test_head_groups(q_heads, kv_heads, D):
    both(new=[1, 1, 1], old=[70, 0, 401], q_heads=q_heads, kv_heads=kv_heads, D=D, uniform=True)


@pytest.mark.parametrize("q_heads,kv_heads", [(100, 1), (255, 1), (256, 1), (1024, 4)])
def test_large_head_groups(q_heads, kv_heads):
    both(new=[1, 3, 2], old=[70, 0, 401], q_heads=q_heads, kv_heads=kv_heads, D=64, shared=16)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(page):
    both(new=[1, 3, 70], old=[300, 513, 0], page=page, spare=5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 3, 5, 16, 31, 32, 33, 63, 65, 127, 128, 129, 300, 700])
def test_prompts(n, D):
    both(new=[n], old=[0], D=D, uniform=True)
    both(new=[n, n], old=[3, 200], D=D, uniform=True)


@pytest.mark.parametrize("D,q_heads,kv_heads,new,old,shared", [
    (128, 32, 8, [3000], [0], 0), (64, 13, 13, [124, 90, 78] * 6, [0] * 18, 768),
    (128, 39, 13, [157, 142, 150] * 4, [88, 474, 200] * 4, 0), (64, 2, 2, [1000] * 30, [0] * 30, 0),
    (128, 8, 8, [2100, 1], [1000, 5000], 0)])
def test_many_tiles(D, q_heads, kv_heads, new, old, shared):
    # long enough lines for every block to have several items and products queued behind them
    p = Paged(new=new, old=old, q_heads=q_heads, kv_heads=kv_heads, D=D, page=128, shared=shared)
    for mode in ((mx.MOE_SHARED_ALWAYS, mx.MOE_SHARED_NEVER) if shared else (0,)):
        mx.moe_attention_set_shared(p.ws, mode)
        for _ in range(3):
            p.check_rows(*p.run())


def test_ragged_batch():
    both(new=[1, 0, 17, 200, 0, 2, 1, 64, 0], old=[40, 30, 0, 129, 0, 1000, 0, 64, 5], page=32)


def test_many_sequences():
    g = torch.Generator().manual_seed(5)
    old = torch.randint(0, 90, (300,), generator=g).tolist()
    both(new=[1] * 300, old=old, q_heads=4, uniform=True)
    new = torch.randint(0, 4, (300,), generator=g).tolist()
    both(new=new, old=old, q_heads=4)


@pytest.mark.parametrize("q_heads", [2, 40])
def test_most_sequences(q_heads):
    g = torch.Generator().manual_seed(6)
    p = Paged(new=[1] * 4096, old=torch.randint(0, 40, (4096,), generator=g).tolist(),
              q_heads=q_heads, kv_heads=1, D=64, uniform=True)
    p.check(*p.run())


@pytest.mark.parametrize("shared", [0, 32])
@pytest.mark.parametrize("q_heads", [8, 80])
def test_no_sequence_has_a_token(q_heads, shared):
    both(new=[0, 0, 0], old=[5, 0, 700], q_heads=q_heads, shared=shared, tail=3)


def test_sequences_without_a_token_give_zeros():
    # padded rows of a decode batch: length 0, one new token
    p, out, lse = both(new=[1, 1, 1, 1], old=[-1, 20, -1, 0], uniform=True)
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0)
    # prompts whose first tokens lie before the sequence
    both(new=[5, 9, 40], old=[-5, -4, -39])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,uniform", [([1] * 9, True), ([3] * 5, True), ([40, 1, 0, 17], False),
                                         ([1, 1], True)])
@pytest.mark.parametrize("shared", [16, 128, 400])
def test_shared_prefix(new, uniform, shared, D):
    old = [(37 * i) % 150 for i in range(len(new))]
    p, out, lse = both(new=new, old=old, uniform=uniform, shared=shared, D=D)
    # the same with the prefix computed for each sequence: by choice, or for want of workspace
    mx.moe_attention_set_shared(p.ws, mx.MOE_SHARED_NEVER)
    o2, l2 = p.run()
    p.check(o2, l2)
    q = Paged(new=new, old=old, uniform=uniform, shared=shared, D=D, max_shared=0)
    o3, l3 = q.run()
    assert torch.equal(o2, o3) and torch.equal(l2, l3)


def test_one_sequence_with_a_shared_prefix():
    both(new=[1], old=[40], shared=64, uniform=True)
    both(new=[300], old=[40], shared=64, uniform=True)


def test_a_prefix_that_pays_is_shared_by_itself():
    # 16 MB of keys and values, 40 times: one pass by the estimate, as when it is asked for
    p = Paged(new=[1] * 40, old=[3 * i for i in range(40)], shared=16384, q_heads=8, page=64,
              share=mx.MOE_SHARED_AUTO, uniform=True)
    a, l = p.run()
    mx.moe_attention_set_shared(p.ws, mx.MOE_SHARED_ALWAYS)
    b, m = p.run()
    assert torch.equal(a, b) and torch.equal(l, m)
    mx.moe_attention_set_shared(p.ws, mx.MOE_SHARED_NEVER)
    c, _ = p.run()
    assert not torch.equal(a, c)
    p.check(a, l)


def test_more_rows_than_the_blocks_take_together():
    # the prefix's items outnumber the blocks: some whole, some cut
    both(new=[40] * 20, old=[i for i in range(20)], shared=48, q_heads=128, kv_heads=16, D=64,
         uniform=True)


def test_shared_prefix_of_sequences_that_end_inside_it():
    both(new=[1] * 6, old=[10, -100, -1, -129, -200, 0], shared=128, uniform=True)


def test_long_prefix_of_many():
    both(new=[1] * 40, old=[5 * i for i in range(40)], shared=2048, q_heads=16, uniform=True)


def test_drafts_over_a_long_context():
    both(new=[6, 6], old=[4000, 2500], q_heads=12, page=64, uniform=True)


def test_rows_behind_the_last_sequence_are_left():
    p = Paged(new=[2, 5], old=[30, 3], tail=9)
    p.q[-9:] = float("nan")
    out, lse = p.run()
    p.check(out, lse)


@pytest.mark.parametrize("new", [[1, 1], [50, 7]])
def test_strides(new):
    p = Paged(new=new, old=[33, 64])
    a, l = p.run()
    wide = torch.full((p.T, p.hq * p.D + 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[:, 8:8 + p.hq * p.D]
    q.copy_(p.q.view(p.T, -1))
    into = torch.full((p.T, p.hq * p.D + 40), 5.0, dtype=torch.bfloat16, device="cuda")
    p.run(q, into[:, 16:16 + p.hq * p.D])
    assert torch.equal(into[:, 16:16 + p.hq * p.D], a.view(p.T, -1))
    assert torch.all(into[:, :16] == 5) and torch.all(into[:, 16 + p.hq * p.D:] == 5)
    b, none = p.run(lse=False)
    assert none is None and torch.equal(a, b)


@pytest.mark.parametrize("new,old", [([1], [700]), ([90], [10])])
def test_large_and_small_logits(new, old):
    for size, scale in ((60.0, 1.0), (1e-3, None), (2.0, 1e-6)):
        p = Paged(new=new, old=old, q_size=size)
        out, lse = p.run(scale=scale)
        p.check(out, lse, scale)


def test_ascending_logits():
    # each key's logit above the ones before it: the running maximum moves at every tile
    p = Paged(new=[1, 60], old=[2000, 1000], q_heads=4)
    p.q.fill_(1.0)
    for b in range(2):
        for j in range(p.lens[b]):
            page, r = p.slot(b, j)
            p.k[page, :, r] = j / 8
    out, lse = p.run()
    p.check(out, lse)


def test_same_bits_again_and_captured():
    p = Paged(new=[1, 30, 1], old=[3000, 900, 2], shared=64, q_heads=16)
    a, l = p.run()
    for _ in range(5):
        b, m = p.run()
        assert torch.equal(a, b) and torch.equal(l, m)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    out, lse = torch.zeros_like(a), torch.zeros_like(l)
    with torch.cuda.stream(side):
        graph.capture_begin()
        mx.moe_attention(p.dims, p.batch, p.q, p.k, p.v, out, p.ws, lse=lse)
        graph.capture_end()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(l, lse)
    # other lengths and pages in the same arrays
    seq, cu, pages = p.batch.tensors
    p.lens[0] -= 1500
    seq[0] = p.lens[0]
    graph.replay()
    torch.cuda.synchronize()
    p.check(out, lse)


@pytest.mark.parametrize("D", [64, 128])
def test_same_bits_whatever_the_blocks_order(D):
    # several hundred items, some with two blocks' parts, joined by whichever comes last: long
    # scans on some SMs leave the last blocks of a call waiting for the first ones to end
    p = Paged(new=[2500], old=[700], q_heads=32, kv_heads=8, D=D, page=128)
    a, l = p.run()
    p.check_rows(a, l)
    side = torch.cuda.Stream()
    for rows in (1, 3, 10, 20, 30, 50):
        long = torch.ones(rows, 1 << 20, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            long.cumsum(1)
        b, m = p.run()
        assert torch.equal(l, m) and torch.equal(a, b)
        torch.cuda.synchronize()


@pytest.mark.parametrize("new", [[1, 2], [90, 1, 300]])
def test_offsets_past_32_bits(new):
    # the same pages at the end of caches of more than 2^32 elements, appended there and read
    p = Paged(new=new, old=[700] * len(new), page=256, q_heads=16, kv_heads=8)
    a, l = p.run()
    pages, more = p.k.shape[0], 16384
    dims = mx.make_attention_dims(p.hq, p.hk, p.D, pages + more, p.page, p.T)
    batch = mx.make_kv_batch(p.batch.tensors[0], p.batch.tensors[2] + more, p.T,
                             cu_new=p.batch.tensors[1], max_new=max(new))
    ws = torch.empty(mx.moe_attention_workspace_size(dims), dtype=torch.uint8, device="cuda")
    mx.moe_attention_workspace_init(dims, ws)
    k, v = (torch.empty(dims.cache_shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[more:], v[more:] = p.k, p.v
    rows = [torch.empty(p.T, p.hk, p.D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, n in enumerate(new):
        for i in range(n):
            page, r = p.slot(b, p.lens[b] - n + i)
            for cache, far, row in zip((p.k, p.v), (k, v), rows):
                row[p.cu[b] + i] = cache[page, :, r]
                far[more + page, :, r] = 5.0
    mx.moe_kv_append(dims, batch, *rows, k, v, ws)
    out, lse = torch.empty_like(a), torch.empty_like(l)
    mx.moe_attention(dims, batch, p.q, k, v, out, ws, lse=lse)
    mx.moe_attention_check(ws)
    assert torch.equal(out, a) and torch.equal(lse, l)


def test_calls_on_two_streams():
    calls = [Paged(new=[1] * 40, old=[997] * 40, uniform=True, seed=1),
             Paged(new=[300, 70], old=[500, 900], shared=64, seed=2)]
    want = [p.run() for p in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[(torch.full_like(a, 77.0), torch.full_like(l, 77.0)) for _ in range(20)]
           for a, l in want]
    torch.cuda.synchronize()
    for i in range(20):
        for p, outs, stream in zip(calls, got, streams):
            mx.moe_attention(p.dims, p.batch, p.q, p.k, p.v, outs[i][0], p.ws, lse=outs[i][1],
                             stream=stream)
    for p, stream in zip(calls, streams):
        mx.moe_attention_check(p.ws, stream)
    for (a, l), outs in zip(want, got):
        assert all(torch.equal(a, b) and torch.equal(l, m) for b, m in outs)


@pytest.mark.parametrize("new", [1, 300])
def test_a_workspace_after_a_timeout(new):
    # as a call that gave up leaves it: the flag set and counters of parts begun
    p = Paged(new=[new], old=[9000], q_heads=32, kv_heads=8, uniform=True)
    a, l = p.run()
    words = p.ws.view(torch.int32)
    words[0] = 2
    words[256:512] = 1
    with pytest.raises(mx.MoeError) as e:
        mx.moe_attention_check(p.ws)
    assert e.value.status == mx.MOE_ERR_TIMEOUT
    b, m = p.run()
    assert torch.equal(a, b) and torch.equal(l, m)


@pytest.mark.parametrize("new", [1, 50])
def test_bad_pages_are_reported(new):
    p = Paged(new=[new, new], old=[200, 200])
    good, _ = p.run()
    seq, cu, pages = p.batch.tensors
    for bad in (-1, p.dims.num_pages, 2 ** 31 - 1, -2 ** 31):
        kept = int(pages[1, 3])
        pages[1, 3] = bad
        with pytest.raises(mx.MoeError) as e:
            p.run()
        assert e.value.status == mx.MOE_ERR_PAGE
        pages[1, 3] = kept
    seq[1] = 16 * pages.shape[1] + 5 * new     # longer than its row of the table
    with pytest.raises(mx.MoeError) as e:
        p.run()
    assert e.value.status == mx.MOE_ERR_PAGE
    seq[1] = p.lens[1]
    again, _ = p.run()
    assert torch.equal(good, again)


def test_refusals():
    p = Paged(new=[2, 2], old=[30, 30], shared=16)
    f, D, kept = mx.lib(), p.dims, p.k.clone()
    out = torch.full_like(p.q, 77.0)
    seq, cu, pages = (t.data_ptr() for t in p.batch.tensors)
    good = dict(seq=seq, cu=cu, pages=pages, batch=2, tokens=4, max_new=2, pages_ld=3, shared=16)

    def call(batch=None, q=p.q.data_ptr(), ldq=1024, k=p.k.data_ptr(), v=p.v.data_ptr(), scale=1.0,
             o=out.data_ptr(), ldo=1024, lse=None, append=True):
        b = mx.KvBatch(*(batch or good).values())
        a = f.moe_attention(ctypes.byref(D), ctypes.byref(b), q, ldq, k, v, scale, o, ldo, lse,
                            p.ws.data_ptr(), p.ws.nbytes, None)
        c = append and f.moe_kv_append(ctypes.byref(D), ctypes.byref(b), None, None, None, None, 0,
                                       None, 0, q, ldq, o, ldo, k, v, p.ws.data_ptr(),
                                       p.ws.nbytes, None)
        return a, c

    bad, ok = mx.MOE_ERR_INVALID_ARG, mx.MOE_OK
    for change in (dict(batch=0), dict(batch=4097), dict(batch=-1), dict(tokens=-1),
                   dict(tokens=5), dict(seq=None), dict(pages=None), dict(seq=seq + 2),
                   dict(cu=cu + 1), dict(pages=pages + 2), dict(pages_ld=0), dict(max_new=0),
                   dict(max_new=5), dict(shared=8), dict(shared=-16), dict(shared=64),
                   dict(cu=None, batch=3)):
        assert call(good | change) == (bad, bad), change
    assert f.moe_attention(ctypes.byref(D), None, 16, 1024, 128, 128, 1.0, 16, 1024, None,
                           p.ws.data_ptr(), p.ws.nbytes, None) == bad
    for change in (dict(q=None), dict(q=p.q.data_ptr() + 8), dict(o=None),
                   dict(o=out.data_ptr() + 2), dict(k=None), dict(k=p.k.data_ptr() + 16),
                   dict(v=None), dict(v=p.v.data_ptr() + 64), dict(ldq=8), dict(ldq=1028)):
        assert call(**change) == (bad, bad), change
    for change in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                   dict(scale=float("inf")), dict(lse=out.data_ptr() + 2), dict(ldo=1020),
                   dict(ldo=0)):
        assert call(**change, append=False)[0] == bad, change
    assert call(good | dict(tokens=0, cu=None), q=None, o=None) == (ok, ok)

    ref, b, rope = ctypes.byref(D), ctypes.byref(p.batch), mx.make_rope_dims(128)
    kv = (p.q.data_ptr(), 1024, p.q.data_ptr(), 1024, p.k.data_ptr(), p.v.data_ptr(),
          p.ws.data_ptr(), p.ws.nbytes, None)
    q = p.q.data_ptr()
    t = torch.zeros(512, dtype=torch.uint8, device="cuda").data_ptr()
    small = mx.make_rope_dims(64)
    for r, table, pos, src, lds, dst, ldd in (
            (rope, None, None, None, 0, None, 0), (None, t, None, None, 0, None, 0),
            (rope, t, None, q, 1024, None, 1024), (rope, t, None, None, 0, q, 1024),
            (None, None, None, q, 1024, q, 1024), (small, t, None, None, 0, None, 0),
            (rope, t + 8, None, None, 0, None, 0), (rope, t, t + 1, None, 0, None, 0),
            (rope, t, None, q, 1024, q, 1032), (rope, t, None, q, 1016, q, 1016),
            (rope, t, None, q + 8, 1024, q + 8, 1024)):
        assert f.moe_kv_append(ref, b, None if r is None else ctypes.byref(r), table, pos, src, lds,
                               dst, ldd, *kv) == bad
    torch.cuda.synchronize()
    assert torch.all(out == 77) and torch.equal(p.k, kept)


def test_the_binding_refuses_other_tensors():
    p = Paged(new=[2, 2], old=[30, 30])
    out = torch.full_like(p.q, 77.0)
    for change in (dict(q=p.q.float()), dict(q=p.q[:3]), dict(q=p.q.cpu()), dict(k=p.k[1:]),
                   dict(k=p.k.transpose(1, 2)), dict(v=p.v.cpu()), dict(v=p.v.half()),
                   dict(out=out[:, :4]), dict(out=out.transpose(0, 1)), dict(ws=p.ws.cpu()),
                   dict(lse=torch.empty(4, 8)), dict(lse=torch.empty(3, 8, device="cuda")),
                   dict(lse=torch.empty(4, 8, device="cuda", dtype=torch.float64))):
        a = dict(q=p.q, k=p.k, v=p.v, out=out, ws=p.ws, lse=None) | change
        with pytest.raises((ValueError, mx.MoeError)):
            mx.moe_attention(p.dims, p.batch, a["q"], a["k"], a["v"], a["out"], a["ws"],
                             lse=a["lse"])
    with pytest.raises(mx.MoeError):
        mx.make_kv_batch(p.batch.tensors[0].cpu(), p.batch.tensors[2], 4)
    torch.cuda.synchronize()
    assert torch.all(out == 77)


@pytest.mark.parametrize("change", [dict(q_heads=16), dict(page_size=32), dict(max_tokens=3),
                                    dict(num_pages=1)])
def test_a_workspace_of_other_dims_is_refused(change):
    p = Paged(new=[2, 2], old=[30, 30])
    d = {n: getattr(p.dims, n) for n, _ in p.dims._fields_}
    p.dims = mx.make_attention_dims(**(d | change))
    out = torch.empty_like(p.q)
    b = mx.KvBatch.from_buffer_copy(p.batch)
    b.tokens = min(b.tokens, p.dims.max_tokens)
    assert mx.lib().moe_attention(
        ctypes.byref(p.dims), ctypes.byref(b), p.q.data_ptr(), 2048, p.k.data_ptr(),
        p.v.data_ptr(), 1.0, out.data_ptr(), 2048, None, p.ws.data_ptr(), p.ws.nbytes, None) \
        == mx.MOE_ERR_WORKSPACE_MISMATCH
