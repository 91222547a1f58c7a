"""The operators of the attention half of a decoder block, as cases to measure: rotary
positions, the append of keys and values to a paged cache, and attention over that cache for
single tokens, drafted tokens, prompts and batches that share a prefix.

`run` computes a case in its plain form (elementary torch operations in 32 bits, angles in 64,
each output rounded once) or, where `own` is true, through the package's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

# A cache is [pages, kv heads, page size, head dim]; a sequence's tokens lie in the pages that
# its row of the page table names, in order.


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # One token's queries and keys in a decode step of a 4096-wide model (32 + 8 heads).
        _rope("rope_1x40x128", 1, 40, 128, 128, "half", "none", 4096),
        # A long prompt read in pieces: far positions, half of each head rotated in adjacent
        # pairs, frequencies stretched for the long context.
        _rope("rope_8191x40x128_part", 8191, 40, 128, 64, "interleaved", "yarn", 1 << 20),
        # One token of one user: latency.
        _append("append_1", 1, 1, 1, 4096, 32, 8, 128, 64, 128, "half", "none", 11),
        # Four ragged prompts of a narrower model into small pages.
        _append("append_4_prompts", 4, 700, 1024, 0, 20, 4, 64, 16, 32, "interleaved",
                "linear", 12),
        # A prefill chunk of 16 long sequences.
        _append("append_16x1000", 16, 900, 1024, 30000, 32, 8, 128, 64, 128, "half", "yarn", 13),
        # One user, a short context: latency.
        _attention("decode_1_short", 1, 1, 1, 900, 1100, 0, 32, 8, 128, 64, 21),
        # One user, a long context: the cache's bytes.
        _attention("decode_1_long", 1, 1, 1, 131000, 131072, 0, 32, 8, 128, 64, 22),
        # A ragged batch of a narrower model with small pages, no common prefix.
        _attention("decode_48_ragged", 48, 1, 1, 64, 6000, 0, 14, 2, 64, 16, 23),
        # Many users behind one long system prompt.
        _attention("decode_64_prefix", 64, 1, 1, 100, 2000, 8192, 32, 8, 128, 64, 24),
        # Drafted tokens of a few users, the prefix common.
        _attention("draft_8x5_prefix", 8, 5, 5, 30, 3000, 16384, 32, 8, 128, 128, 25),
        # Ragged questions about one shared document.
        _attention("questions_32_prefix", 32, 17, 250, 0, 0, 8192, 32, 8, 128, 64, 26),
        # A whole prompt.
        _attention("prompt_16384", 1, 16384, 16384, 0, 0, 0, 32, 8, 128, 64, 27),
    ]


def _rope(name, tokens, heads, dim, rotary, layout, scaling, far):
    c = {"op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rotary": rotary,
         "layout": layout, "scaling": scaling, "far": far}
    return {"name": name, **c} if name else c


def _append(name, batch, new_lo, new_hi, before, q_heads, kv_heads, dim, page, rotary, layout,
            scaling, pick):
    """`batch` sequences with new_lo..new_hi new tokens each behind about `before` older ones."""
    c = {"op": "append", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "before": before,
         "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "rotary": rotary,
         "layout": layout, "scaling": scaling, "pick": pick}
    return {"name": name, **c} if name else c


def _attention(name, batch, new_lo, new_hi, own_lo, own_hi, shared, q_heads, kv_heads, dim, page,
               pick):
    """`batch` sequences of `shared` common tokens, own_lo..own_hi older ones of their own and
    new_lo..new_hi new ones, which ask."""
    c = {"op": "attention", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "own_lo": own_lo,
         "own_hi": own_hi, "shared": shared, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
         "page": page, "pick": pick}
    return {"name": name, **c} if name else c


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


MOST_FLOPS = 4 * 128 * 32 * 16384 * 16384 / 2       # the whole prompt's
MOST_BYTES = 1.2e9


def draw(rng):
    op = rng.choice(("rope", "append", "attention", "attention", "attention"))
    pick = rng.randrange(1 << 30)
    layout = rng.choice(("half", "interleaved"))
    scaling = rng.choice(("none", "linear", "ntk", "yarn"))
    while True:
        dim = rng.choice((64, 128))
        kv = _log_int(rng, 1, 16)
        q = kv * rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
        page = rng.choice((16, 32, 64, 128))
        if op == "rope":
            dim = rng.choice((64, 80, 128, 192, 256))
            c = _rope(None, _log_int(rng, 1, 16384), rng.randint(1, 48), dim,
                      rng.choice((dim, dim // 2, dim // 4)), layout, scaling,
                      _log_int(rng, 1 << 10, 1 << 20))
            cost = c["tokens"] * c["heads"] * dim * 4
        elif op == "append":
            hi = _log_int(rng, 1, 4096)
            c = _append(None, _log_int(rng, 1, 64), rng.randint(max(1, hi // 2), hi), hi,
                        rng.randint(0, 8192), q, kv, dim, page, rng.choice((dim, dim // 2)),
                        layout, scaling, pick)
            cost = c["batch"] * hi * (q + 2 * kv) * dim * 4 * 4
        else:
            kind = rng.choice(("decode", "draft", "prompt", "question"))
            batch = _log_int(rng, 1, 128)
            shared = page * _log_int(rng, 1, 32768 // page) if rng.random() < 0.6 else 0
            hi = {"decode": 1, "draft": rng.randint(2, 8), "prompt": _log_int(rng, 64, 16384),
                  "question": _log_int(rng, 9, 512)}[kind]
            lo = hi if kind in ("decode", "draft") else rng.randint(max(1, hi // 4), hi)
            own_hi = _log_int(rng, 16, 65536) if kind != "question" else 0
            if kind == "prompt" and rng.random() < 0.5:
                own_hi = 0
            c = _attention(None, batch, lo, hi, rng.randint(own_hi // 8, own_hi), own_hi, shared,
                           q, kv, dim, page, pick)
            cost = (shared + batch * (hi + own_hi)) * kv * dim * 4 + batch * hi * q * dim * 4
            if 4 * dim * q * batch * hi * (shared + own_hi + hi) > MOST_FLOPS:
                continue
        if q <= 96 and cost <= MOST_BYTES:
            return c


def _lengths(c):
    """New tokens and older tokens of its own, for each sequence of a case."""
    rng = random.Random(c["pick"])
    new = [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    if c["op"] == "append":
        return new, [rng.randint(c["before"] // 2, c["before"]) for _ in new]
    return new, [rng.randint(c["own_lo"], c["own_hi"]) for _ in new]


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"]
        # what is not rotated is copied
        return {"bytes": 4 * n * c["dim"] + 4 * c["tokens"], "flops": 3 * n * c["rotary"]}
    new, old = _lengths(c)
    T = sum(new)
    if c["op"] == "append":
        heads = c["q_heads"] + 2 * c["kv_heads"]
        return {"bytes": 4 * T * heads * c["dim"],
                "flops": 3 * T * (c["q_heads"] + c["kv_heads"]) * c["rotary"]}
    keys = sum(n * (c["shared"] + o) + n * (n + 1) // 2 for n, o in zip(new, old))
    cached = c["shared"] + sum(n + o for n, o in zip(new, old))
    return {"bytes": 4 * cached * c["kv_heads"] * c["dim"] + 4 * T * c["q_heads"] * c["dim"]
            + 4 * T * c["q_heads"],
            "flops": 4 * c["dim"] * c["q_heads"] * keys}


# ---------------------------------------------------------------------------
# Rotary frequencies

BASE = 10000.0
SCALINGS = {  # factor, trained length
    "none": (1.0, 0.0), "linear": (4.0, 0.0), "ntk": (8.0, 0.0), "yarn": (16.0, 65536.0)}
BETA_FAST, BETA_SLOW = 32.0, 1.0


def _frequencies(c):
    """Radians a position of each rotated pair, in 64 bits, and the rotation's magnitude."""
    d = c["rotary"]
    factor, trained = SCALINGS[c["scaling"]]
    i = torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d
    if c["scaling"] == "ntk":
        return (BASE * factor ** (d / (d - 2.0))) ** -i, 1.0
    f = BASE ** -i
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "yarn":
        turns = trained * f / (2 * math.pi)
        keep = ((turns - BETA_SLOW) / (BETA_FAST - BETA_SLOW)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1
    return f, 1.0


# ---------------------------------------------------------------------------
# Inputs

def _normal(g, *shape, scale=1.0):
    x = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda") * scale)
    return x


def _batch(s, c):
    """Page table and lengths: pages handed out in random order, the common prefix's once."""
    new, old = _lengths(c)
    page, shared = c["page"], c.get("shared", 0)
    rng = random.Random(c["pick"] + 1)
    lens = [shared + o + n for n, o in zip(new, old)]
    common = shared // page
    counts = [-(-n // page) - common for n in lens]
    total = common + sum(counts)
    ids = list(range(total))
    rng.shuffle(ids)
    table = torch.zeros(len(lens), max(-(-n // page) for n in lens), dtype=torch.int32)
    at = common
    for b, k in enumerate(counts):
        table[b, :common] = torch.tensor(ids[:common], dtype=torch.int32)
        table[b, common:common + k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
        at += k
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["new"], s["lens"], s["pages"] = new, lens, total
    s["table"] = table.cuda()
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["cu"] = None if c["new_lo"] == c["new_hi"] else torch.tensor(cu, dtype=torch.int32).cuda()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rope":
        s["x"] = _normal(g, c["tokens"], c["heads"], c["dim"])
        start = torch.randint(0, max(1, c["far"] - c["tokens"]), (1,), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(c["tokens"], device="cuda")).int()
    else:
        _batch(s, c)
        T, hq, hk, d = sum(s["new"]), c["q_heads"], c["kv_heads"], c["dim"]
        cache = (s["pages"], hk, c["page"], d)
        if c["op"] == "append":
            # the rows that the projection wrote: queries, keys and values side by side
            qkv = _normal(g, T, hq + 2 * hk, d)
            s["q"], s["k"], s["v"] = qkv.split((hq, hk, hk), 1)
            s["k_cache"], s["v_cache"] = (torch.zeros(cache, dtype=torch.bfloat16, device="cuda")
                                          for _ in range(2))
        else:
            # logits of standard deviation 2 and values with a mean, as trained heads have
            s["q"] = _normal(g, T, hq, d, scale=2.0)
            s["k_cache"] = _normal(g, *cache)
            s["v_cache"] = _normal(g, *cache).add_(0.5)
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a user's program keeps: outputs, the rotation's table, a workspace."""
    import block_scaled_fp4_pre_gb300 as mx
    c = s["case"]
    u8, bf = torch.uint8, torch.bfloat16
    if c["op"] != "attention":
        factor, trained = SCALINGS[c["scaling"]]
        s["rope"] = mx.make_rope_dims(
            c["dim"], c["rotary"],
            mx.MOE_ROPE_HALF if c["layout"] == "half" else mx.MOE_ROPE_INTERLEAVED, BASE,
            {"none": mx.MOE_ROPE_UNSCALED, "linear": mx.MOE_ROPE_LINEAR, "ntk": mx.MOE_ROPE_NTK,
             "yarn": mx.MOE_ROPE_YARN}[c["scaling"]], factor, trained, BETA_FAST, BETA_SLOW)
        s["rope_table"] = torch.empty(mx.moe_rope_table_size(s["rope"]), dtype=u8, device="cuda")
        mx.moe_rope_prepare(s["rope"], s["rope_table"])
    if c["op"] == "rope":
        s["out"] = torch.empty_like(s["x"])
        return
    T = sum(s["new"])
    shared = c.get("shared", 0)
    d = s["dims"] = mx.make_attention_dims(c["q_heads"], c["kv_heads"], c["dim"], s["pages"],
                                           c["page"], T, T if shared else 0)
    s["batch"] = mx.make_kv_batch(s["seq_lens"], s["table"], T, cu_new=s["cu"],
                                  max_new=max(s["new"]), shared_len=shared)
    s["ws"] = torch.empty(mx.moe_attention_workspace_size(d), dtype=u8, device="cuda")
    mx.moe_attention_workspace_init(d, s["ws"])
    s["out"] = torch.empty(T, c["q_heads"], c["dim"], dtype=bf, device="cuda")
    if c["op"] == "attention":
        s["lse"] = torch.empty(T, c["q_heads"], dtype=torch.float32, device="cuda")


# ---------------------------------------------------------------------------
# One pass

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "rope":
        return _rotate(s["x"], s["positions"], c)
    if c["op"] == "append":
        return _append_plain(s, c)
    return _attention_plain(s, c)


def _run_own(s, c):
    import block_scaled_fp4_pre_gb300 as mx
    if c["op"] == "rope":
        mx.moe_rope(s["rope"], s["rope_table"], s["x"], s["positions"], s["out"])
        return s["out"]
    if c["op"] == "append":
        mx.moe_kv_append(s["dims"], s["batch"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                         s["ws"], rope=s["rope"], table=s["rope_table"], q=s["q"],
                         q_out=s["out"])
        return {"q": s["out"], "k": s["k_cache"], "v": s["v_cache"]}
    mx.moe_attention(s["dims"], s["batch"], s["q"], s["k_cache"], s["v_cache"], s["out"], s["ws"],
                     lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------------------
# The plain forms

def _rotate(x, positions, c):
    """Rotates the first c["rotary"] elements of each head of x [tokens, heads, dim]."""
    f, magnitude = _frequencies(c)
    angle = positions.double().unsqueeze(1) * f
    cos = (torch.cos(angle) * magnitude).float().unsqueeze(1)
    sin = (torch.sin(angle) * magnitude).float().unsqueeze(1)
    r, rest = x[..., :c["rotary"]].float(), x[..., c["rotary"]:]
    if c["layout"] == "half":
        a, b = r.chunk(2, -1)
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((r.bfloat16(), rest), -1)


def _places(s, c):
    """Position in its sequence, page and row of each new token."""
    new = torch.tensor(s["new"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"), new)
    first = (s["seq_lens"] - new)[seq]
    begin = (torch.cumsum(new, 0) - new)[seq]
    p = first + torch.arange(len(seq), device="cuda") - begin
    return p, s["table"][seq, p // c["page"]].long(), p % c["page"]


def _append_plain(s, c):
    p, page, row = _places(s, c)
    s["k_cache"][page, :, row] = _rotate(s["k"], p, c)
    s["v_cache"][page, :, row] = s["v"]
    return {"q": _rotate(s["q"], p, c), "k": s["k_cache"], "v": s["v_cache"]}


def _attention_plain(s, c):
    hq, hk, d, page = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    G = hq // hk
    T = sum(s["new"])
    out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, hq, dtype=torch.float32, device="cuda")
    t0 = 0
    for b, (n, length) in enumerate(zip(s["new"], s["lens"])):
        pages = s["table"][b, :-(-length // page)].long()
        limit = torch.arange(length - n + 1, length + 1, device="cuda").view(n, 1, 1)
        masked = torch.arange(length, device="cuda") >= limit             # [n, 1, L]
        # one kv head after another where its scores are large, all together where small
        step = hk if n * hq * length <= 1 << 26 else 1
        for h in range(0, hk, step):
            heads = slice(h, h + step)
            k, v = (x[pages, heads].transpose(0, 1).reshape(step, -1, d)[:, :length].float()
                    for x in (s["k_cache"], s["v_cache"]))
            q = s["q"][t0:t0 + n, h * G:(h + step) * G].float().view(n, step, G, d)
            q = q.transpose(0, 1).reshape(step, n * G, d) * d ** -0.5
            sc = (q @ k.transpose(1, 2)).view(step, n, G, length)
            sc.masked_fill_(masked, -math.inf)
            top = sc.amax(-1, keepdim=True)
            sc.sub_(top).exp_()
            total = sc.sum(-1, keepdim=True)
            o = (sc.view(step, n * G, length) @ v).view(step, n, G, d) / total
            out[t0:t0 + n, h * G:(h + step) * G] = o.transpose(0, 1).reshape(n, step * G, d)
            lse[t0:t0 + n, h * G:(h + step) * G] = \
                (top + torch.log(total)).squeeze(-1).transpose(0, 1).reshape(n, step * G)
        t0 += n
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, written apart from the plain forms

def _turned64(x, positions, c):
    """The rotation as a product of complex numbers."""
    d, half = c["rotary"], c["rotary"] // 2
    factor, trained = SCALINGS[c["scaling"]]
    rates, size = [], 1.0
    for i in range(half):
        base = BASE * factor ** (d / (d - 2)) if c["scaling"] == "ntk" else BASE
        w = math.exp(-2 * i / d * math.log(base))
        if c["scaling"] == "linear":
            w /= factor
        elif c["scaling"] == "yarn":
            turns = trained * w / math.tau
            slow = min(1.0, max(0.0, (BETA_FAST - turns) / (BETA_FAST - BETA_SLOW)))
            w = w * (1 - slow) + w * slow / factor
        rates.append(w)
    if c["scaling"] == "yarn":
        size = 1 + 0.1 * math.log(factor)
    turn = torch.polar(torch.full((len(positions), 1, half), size, dtype=torch.float64,
                                  device="cuda"),
                       positions.double().view(-1, 1, 1)
                       * torch.tensor(rates, dtype=torch.float64, device="cuda"))
    y = x.double()
    first, second = (slice(0, half), slice(half, d)) if c["layout"] == "half" \
        else (slice(0, d, 2), slice(1, d, 2))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "rope":
        return _turned64(s["x"], s["positions"], c)
    hq, hk, d, page = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    first = [0]
    for n in s["new"]:
        first.append(first[-1] + n)
    if c["op"] == "append":
        where = [(length - n + i, b) for b, (n, length) in enumerate(zip(s["new"], s["lens"]))
                 for i in range(n)]
        p = torch.tensor([w[0] for w in where], device="cuda")
        table = s["table"].cpu().tolist()
        slot = torch.tensor([table[b][i // page] * page + i % page for i, b in where],
                            device="cuda")
        caches = {}
        for name, rows in (("k", _turned64(s["k"], p, c)), ("v", s["v"].double())):
            flat = s[name + "_cache"].double().transpose(1, 2).reshape(-1, hk, d)
            flat[slot] = rows
            caches[name] = flat.view(-1, page, hk, d).transpose(1, 2)
        return {"q": _turned64(s["q"], p, c), **caches}
    if 4.0 * d * hq * sum(n * L for n, L in zip(s["new"], s["lens"])) > 1.0e13:
        return None
    out = torch.empty(first[-1], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(first[-1], hq, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lens"]):
        n = s["new"][b]
        at = torch.arange(length, device="cuda")
        slot = s["table"][b].long()[at // page] * (hk * page) + at % page
        for h in range(hk):
            k, v = (x.view(-1, d)[slot + h * page].double() for x in (s["k_cache"], s["v_cache"]))
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                end = length - n + i + m                  # what the last of these rows sees
                rows = slice(first[b] + i, first[b] + i + m)
                for j in range(h * (hq // hk), (h + 1) * (hq // hk)):
                    z = s["q"][rows, j].double() @ k[:end].T / math.sqrt(d)
                    z = z + torch.full_like(z, -math.inf).triu(end - m + 1)
                    lse[rows, j] = torch.logsumexp(z, -1)
                    out[rows, j] = torch.exp(z - lse[rows, j].unsqueeze(-1)) @ v[:end]
    return {"out": out, "lse": lse}
