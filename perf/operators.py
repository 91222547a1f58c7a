"""The operators around the expert layer, as cases to measure: RMSNorm with an MXFP8
output, the MXFP4 linear product, and the whole expert layer for a few tokens.

`run` computes a case in its plain form (elementary torch operations in 32 bits, each
output rounded once) or, where `own` is true, through the package's entry points.
"""
from __future__ import annotations

import torch

own = False

E2M1_STEPS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
              (3.5, True), (5.0, False))       # (threshold, reached by a tie), codes 1..7
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # One token of a decode step between two layers of a 4096-wide model.
        {"name": "norm_1x4096", "op": "norm", "rows": 1, "K": 4096, "layout": "128x4",
         "residual": True, "y": True},
        # A small ragged batch of a narrower model; the first norm, with no residual yet.
        {"name": "norm_333x1408", "op": "norm", "rows": 333, "K": 1408, "layout": "packed",
         "residual": False, "y": False},
        # A large prefill between two layers.
        {"name": "norm_16384x4096", "op": "norm", "rows": 16384, "K": 4096, "layout": "128x4",
         "residual": True, "y": True},
        # One token through a 4096 x 4096 projection: latency and the weight's bytes.
        {"name": "linear_1x4096x4096", "op": "linear", "rows": 1, "N": 4096, "K": 4096,
         "act": "mxfp4"},
        # A decode batch through a shared expert's gate/up projection, on the norm's pair.
        {"name": "linear_24x4096x4096_pair", "op": "linear", "rows": 24, "N": 4096, "K": 4096,
         "act": "mxfp8_pair"},
        # Ragged in every direction: an odd number of outputs, K not a whole scale block.
        {"name": "linear_317x1001x1056", "op": "linear", "rows": 317, "N": 1001, "K": 1056,
         "act": "mxfp8"},
        # A prefill of four prompts of 1024 tokens through a down projection.
        {"name": "linear_4096x4096x2048_pair", "op": "linear", "rows": 4096, "N": 4096,
         "K": 2048, "act": "mxfp8_pair"},
        # The large prefill, both operands in 4 bits.
        {"name": "linear_16384x4096x4096", "op": "linear", "rows": 16384, "N": 4096, "K": 4096,
         "act": "mxfp4"},
        # A small expert layer with odd counts, as a draft model's.
        {"name": "few_3_small", "op": "few", "T": 3, "H": 640, "I": 384, "E": 12, "k": 3,
         "mma": "mxf4xmxf4"},
        # One token through the full-size layer: the decode step of a single user.
        {"name": "few_1", "op": "few", "T": 1, "H": 4096, "I": 2048, "E": 256, "k": 6,
         "mma": "mxf4xmxf4"},
        # A few users, or one with drafted tokens, on 8-bit activations.
        {"name": "few_5_w4a8", "op": "few", "T": 5, "H": 4096, "I": 2048, "E": 256, "k": 6,
         "mma": "fp8xfp4"},
        # The most tokens the few-token form takes.
        {"name": "few_16", "op": "few", "T": 16, "H": 4096, "I": 2048, "E": 256, "k": 6,
         "mma": "mxf4xmxf4"},
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("norm", "linear", "few"))
    while True:
        if op == "norm":
            c = {"op": op, "rows": _log_int(rng, 1, 16384), "K": 128 * _log_int(rng, 1, 64),
                 "layout": rng.choice(("packed", "128x4")), "residual": rng.random() < 0.7,
                 "y": rng.random() < 0.7}
            if c["rows"] * c["K"] <= 16384 * 4096:
                return c
        elif op == "linear":
            act = rng.choice(("mxfp4", "mxfp8", "mxfp8_pair"))
            k = 128 * _log_int(rng, 1, 64) if act == "mxfp8_pair" else 32 * _log_int(rng, 4, 256)
            c = {"op": op, "rows": _log_int(rng, 1, 16384), "N": _log_int(rng, 64, 8192), "K": k,
                 "act": act}
            if c["rows"] * c["N"] * c["K"] <= 16384 * 4096 * 4096:
                return c
        else:
            e = _log_int(rng, 4, 256)
            c = {"op": op, "T": _log_int(rng, 1, 16), "H": 128 * _log_int(rng, 2, 32),
                 "I": 128 * _log_int(rng, 1, 16), "E": e, "k": rng.randint(1, min(6, e)),
                 "mma": rng.choice(("mxf4xmxf4", "fp8xfp4"))}
            return c


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["K"]
        per = 2 + 1 + 1 / 32 + (4 if c["residual"] else 0) + (2 if c["y"] else 0)
        return {"bytes": n * per + 2 * c["K"], "flops": 6 * n}
    if c["op"] == "linear":
        m, n, k = c["rows"], c["N"], c["K"]
        x = m * k * (33 / 32 if c["act"] == "mxfp8_pair" else 2)
        return {"bytes": x + n * k * (1 / 2 + 1 / 32) + 2 * m * n, "flops": 2 * m * n * k}
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    touched = E * (1 - (1 - k / E) ** T)           # expected distinct experts
    return {"bytes": touched * 3 * I * H * (1 / 2 + 1 / 32) + 2 * E * H + 4 * T * H + 8 * T * k,
            "flops": 6 * T * k * I * H + 2 * T * E * H}


# ---------------------------------------------------------------------------
# Inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _mxfp4_weights(g, *shape):
    """Canonical MXFP4 of N(0, 1/sqrt(K)) rows: packed codes and scale bytes."""
    K = shape[-1]
    w = (_normal(g, *shape) * K ** -0.5).view(*shape[:-1], K // 32, 32)
    e = _exponent(w.abs().amax(-1), 0.75, 3)
    v = torch.ldexp(w, -e.unsqueeze(-1))
    a = v.abs()
    code = (v < 0).to(torch.uint8) * 8
    for i, (t, tie) in enumerate(E2M1_STEPS):
        code += (a >= t) if tie else (a > t)
    code = code.view(*shape[:-1], K // 2, 2)
    return code[..., 0] | code[..., 1] << 4, (e + 127).to(torch.uint8)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "norm":
        rows, K = c["rows"], c["K"]
        # activations with a few channels far larger than the rest, as hidden states have
        ch = 1 + 20 * (torch.rand(K, generator=g, device="cuda") < 0.004)
        s["x"] = (_normal(g, rows, K) * ch).bfloat16()
        s["gamma"] = (1 + 0.2 * _normal(g, K)).bfloat16()
        s["residual"] = (3 * _normal(g, rows, K) * ch).bfloat16() if c["residual"] else None
    elif c["op"] == "linear":
        m, n, k = c["rows"], c["N"], c["K"]
        x = _normal(g, m, k).bfloat16()
        if c["act"] == "mxfp8_pair":
            q, e = _quantise8(x.float())
            s["q"], s["sf"] = q.view(torch.uint8), _block_scales((e + 127).to(torch.uint8))
        else:
            s["x"] = x
        s["codes"], s["scales"] = _mxfp4_weights(g, n, k)
    else:
        T, H, I, E = c["T"], c["H"], c["I"], c["E"]
        s["x"] = _normal(g, T, H).bfloat16()
        s["router"] = (_normal(g, E, H) * H ** -0.5).bfloat16()
        u8 = torch.uint8
        for name, r, K in (("w1", 2 * I, H), ("w2", H, I)):
            s[name] = torch.empty(E, r, K // 2, dtype=u8, device="cuda")
            s[name + "s"] = torch.empty(E, r, K // 32, dtype=u8, device="cuda")
            for e in range(0, E, 16):
                s[name][e:e + 16], s[name + "s"][e:e + 16] = _mxfp4_weights(
                    g, min(16, E - e), r, K)
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a user's program keeps: outputs, weights in the package's layout, workspaces."""
    import block_scaled_fp4_pre_gb300 as mx
    c = s["case"]
    u8, bf = torch.uint8, torch.bfloat16
    if c["op"] == "norm":
        rows, K = c["rows"], c["K"]
        s["layout"] = mx.MOE_SF_128X4 if c["layout"] == "128x4" else mx.MOE_SF_PACKED
        s["q"] = torch.empty(rows, K, dtype=u8, device="cuda")
        s["sf"] = torch.empty(mx.moe_mxfp8_scale_bytes(rows, K, s["layout"]), dtype=u8,
                              device="cuda")
        s["residual_out"] = torch.empty(rows, K, dtype=bf, device="cuda") if c["residual"] else None
        s["y"] = torch.empty(rows, K, dtype=bf, device="cuda") if c["y"] else None
    elif c["op"] == "linear":
        mma = mx.MOE_MMA_MXF4xMXF4 if c["act"] == "mxfp4" else mx.MOE_MMA_FP8xFP4
        d = s["dims"] = mx.make_linear_dims(c["N"], c["K"], c["rows"], mma)
        s["prepared"] = torch.empty(mx.moe_linear_weights_size(d), dtype=u8, device="cuda")
        mx.moe_linear_prepare(d, s["codes"], s["scales"], s["prepared"])
        s["ws"] = torch.empty(mx.moe_linear_workspace_size(d), dtype=u8, device="cuda")
        mx.moe_linear_workspace_init(d, s["ws"])
        s["out"] = torch.empty(c["rows"], c["N"], dtype=bf, device="cuda")
    else:
        mma = mx.MOE_MMA_MXF4xMXF4 if c["mma"] == "mxf4xmxf4" else mx.MOE_MMA_FP8xFP4
        T, k = c["T"], c["k"]
        d = s["dims"] = mx.make_dims(c["H"], c["I"], c["E"], k, T, mma)
        s["prepared"] = torch.empty(mx.moe_prepared_weights_size(d), dtype=u8, device="cuda")
        mx.moe_prepare_weights(d, s.pop("w1"), s.pop("w1s"), s.pop("w2"), s.pop("w2s"),
                               s["prepared"])
        s["ws"] = torch.empty(mx.moe_workspace_size(d), dtype=u8, device="cuda")
        mx.moe_workspace_init(d, s["ws"])
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
        s["out"] = torch.empty(T, c["H"], dtype=bf, device="cuda")


# ---------------------------------------------------------------------------
# One pass

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "norm":
        return _norm(s, c)
    if c["op"] == "linear":
        return _linear(s, c)
    return _few(s, c)


def _run_own(s, c):
    import block_scaled_fp4_pre_gb300 as mx
    if c["op"] == "norm":
        mx.moe_rmsnorm_mxfp8(s["x"], s["gamma"], EPS, s["q"], s["sf"], s["layout"],
                             residual=s["residual"], residual_out=s["residual_out"], y=s["y"])
        return {"q": s["q"].view(torch.float8_e4m3fn), "sf": s["sf"].view(torch.float8_e8m0fnu),
                "residual": s["residual_out"], "y": s["y"]}
    if c["op"] == "linear":
        if c["act"] == "mxfp8_pair":
            mx.moe_linear_forward_pair(s["dims"], s["prepared"], s["q"], s["sf"], c["rows"],
                                       s["out"], s["ws"])
        else:
            mx.moe_linear_forward(s["dims"], s["prepared"], s["x"], s["out"], s["ws"])
        return s["out"]
    mx.moe_few_forward(s["dims"], s["prepared"], s["router"], s["x"], s["ids"], s["weights"],
                       c["T"], s["ws"], s["out"])
    return {"out": s["out"], "ids": s["ids"], "weights": s["weights"]}


# ---------------------------------------------------------------------------
# The plain forms

def _exponent(amax, top, bits):
    """Smallest e >= -127 with amax <= top * 2^(bits + e), 0.5 <= top < 1."""
    m, ex = torch.frexp(amax)
    e = ex - bits + (m > top)
    return torch.where(amax > 0, e.clamp(min=-127), -127)


def _quantise4(x):
    """MXFP4 of fp32 rows, as the values it stands for."""
    v = x.unflatten(-1, (-1, 32))
    e = _exponent(v.abs().amax(-1), 0.75, 3).unsqueeze(-1)
    v = torch.ldexp(v, -e)
    a = v.abs()
    r = torch.zeros_like(a)
    for i, (t, tie) in enumerate(E2M1_STEPS):
        r += ((a >= t) if tie else (a > t)) * (E2M1_VALUES[i + 1] - E2M1_VALUES[i])
    return torch.ldexp(torch.where(v < 0, -r, r), e).flatten(-2)


def _quantise8(x):
    """MXFP8 of fp32 rows: E4M3 values and each group's exponent."""
    v = x.unflatten(-1, (-1, 32))
    e = _exponent(v.abs().amax(-1), 0.875, 9)
    return torch.ldexp(v, -e.unsqueeze(-1)).flatten(-2).to(torch.float8_e4m3fn), e


def _quantise8_values(x):
    q, e = _quantise8(x)
    return torch.ldexp(q.float().unflatten(-1, (-1, 32)), e.unsqueeze(-1)).flatten(-2)


def _block_scales(sf):
    """Row-major scale bytes [rows, K/32] in the 128x4 block layout, padded rows zero."""
    rows, n = sf.shape
    blocks = -(-rows // 128)
    full = torch.zeros(blocks * 128, n, dtype=sf.dtype, device=sf.device)
    full[:rows] = sf
    return full.view(blocks, 4, 32, n // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _unblock_scales(sf, rows, n):
    blocks = -(-rows // 128)
    return sf.view(blocks, n // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, n)[:rows]


def _weight_values(codes, scales):
    """fp32 values of canonical MXFP4 weights [..., K/2], [..., K/32]."""
    table = torch.tensor([(1 - 2 * (b >> 3)) * E2M1_VALUES[b & 7] for b in range(16)],
                         device=codes.device)
    pairs = torch.stack((table.repeat(16), table.repeat_interleave(16)), -1)
    v = pairs[codes.int()].flatten(-2)
    e = scales.int() - 127
    return torch.ldexp(v.unflatten(-1, (-1, 32)), e.unsqueeze(-1)).flatten(-2)


def _norm(s, c):
    r = s["x"].float()
    if c["residual"]:
        r = r + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    q, e = _quantise8(y)
    sf = (e + 127).to(torch.uint8)
    sf = _block_scales(sf) if c["layout"] == "128x4" else sf.reshape(-1)
    return {"q": q, "sf": sf.view(torch.float8_e8m0fnu),
            "residual": r.bfloat16() if c["residual"] else None,
            "y": y.bfloat16() if c["y"] else None}


def _linear(s, c):
    if c["act"] == "mxfp8_pair":
        m, k = c["rows"], c["K"]
        e = _unblock_scales(s["sf"], m, k // 32).int() - 127
        x = torch.ldexp(s["q"].view(torch.float8_e4m3fn).float().view(m, k // 32, 32),
                        e.unsqueeze(-1)).flatten(-2)
    else:
        x = (_quantise4 if c["act"] == "mxfp4" else _quantise8_values)(s["x"].float())
    return (x @ _weight_values(s["codes"], s["scales"]).T).bfloat16()


def _few(s, c):
    k, I = c["k"], c["I"]
    quantise = _quantise4 if c["mma"] == "mxf4xmxf4" else _quantise8_values
    x = s["x"].float()
    top, ids = torch.sort(x @ s["router"].float().T, dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(-1, keepdim=True)
    xq = quantise(x).repeat_interleave(k, 0).unsqueeze(-1)             # [T*k, H, 1]
    flat = ids.reshape(-1)
    gu = torch.bmm(_weight_values(s["w1"][flat], s["w1s"][flat]), xq).squeeze(-1)
    gate, up = gu[:, :I], gu[:, I:]
    h = quantise(gate / (1 + torch.exp(-gate)) * up)
    y = torch.bmm(_weight_values(s["w2"][flat], s["w2s"][flat]), h.unsqueeze(-1)).squeeze(-1)
    out = (y.view(-1, k, c["H"]) * w.unsqueeze(-1)).sum(1)
    return {"out": out.bfloat16(), "ids": ids.int(), "weights": w}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, written apart from the plain forms

def _grid64(x, top, mant, emin):
    """Microscaled rounding in double: a power-of-two scale per 32 that brings the
    largest magnitude to at most `top`, then the nearest value with `mant` mantissa bits
    and exponents from `emin`, ties to even.  Returns (scaled values, scales)."""
    v = x.reshape(*x.shape[:-1], -1, 32)
    amax = v.abs().max(-1, keepdim=True).values
    e = torch.ceil(torch.log2(amax / top)).clamp(-127, 127)
    e = torch.where(amax <= top * torch.exp2(e - 1), e - 1, e)       # log2 rounded up
    e = torch.where(amax > top * torch.exp2(e), e + 1, e).clamp(min=-127)   # or down
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    v = v * torch.exp2(-e)
    ex = torch.frexp(v)[1].double() - 1
    step = torch.exp2(ex.clamp(min=emin) - mant)
    return torch.round(v / step) * step, torch.exp2(e)


def _values64(x, act):
    q, s = _grid64(x, 6.0, 1, 0) if act in ("mxfp4", "mxf4xmxf4") else _grid64(x, 448.0, 3, -6)
    return (q * s).reshape(x.shape)


def _weights64(codes, scales):
    lo, hi = codes & 15, codes >> 4
    n = torch.stack((lo, hi), -1).reshape(*codes.shape[:-1], -1)
    m, ex = (n & 1).double(), ((n >> 1) & 3).double()
    mag = torch.where(ex > 0, (1 + m / 2) * torch.exp2(ex - 1), m / 2)
    v = torch.where(n > 7, -mag, mag)
    s = torch.exp2(scales.double() - 127)
    return (v.reshape(*scales.shape, 32) * s.unsqueeze(-1)).reshape(v.shape)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "norm":
        r = s["x"].double()
        if c["residual"]:
            r = r + s["residual"].double()
        y = r / torch.sqrt((r ** 2).sum(-1, keepdim=True) / c["K"] + EPS) * s["gamma"].double()
        q, sc = _grid64(y, 448.0, 3, -6)
        sc = sc.squeeze(-1)
        if c["layout"] == "128x4":
            rows = torch.arange(-(-c["rows"] // 128) * 128, device=sc.device)
            full = torch.full((len(rows), sc.shape[1]), 2.0 ** -127, dtype=torch.float64,
                              device=sc.device)
            full[:c["rows"]] = sc
            col = torch.arange(sc.shape[1], device=sc.device)
            at = ((rows // 128 * (sc.shape[1] // 4)).unsqueeze(1) + col // 4) * 512 \
                + ((rows % 32) * 16 + rows % 128 // 32 * 4).unsqueeze(1) + col % 4
            sc = torch.empty(full.numel(), dtype=torch.float64, device=sc.device)
            sc[at.reshape(-1)] = full.reshape(-1)
        return {"q": q.reshape(c["rows"], c["K"]), "sf": sc.reshape(-1),
                "residual": r if c["residual"] else None, "y": y if c["y"] else None}
    if c["op"] == "linear":
        if c["act"] == "mxfp8_pair":
            m, n = c["rows"], c["K"] // 32
            rows = torch.arange(m, device="cuda").unsqueeze(1)
            col = torch.arange(n, device="cuda")
            at = (rows // 128 * (n // 4) + col // 4) * 512 + rows % 32 * 16 \
                + rows % 128 // 32 * 4 + col % 4
            sc = torch.exp2(s["sf"][at].double() - 127)
            x = s["q"].view(torch.float8_e4m3fn).double().reshape(m, n, 32) * sc.unsqueeze(-1)
            x = x.reshape(m, -1)
        else:
            x = _values64(s["x"].double(), c["act"])
        return x @ _weights64(s["codes"], s["scales"]).T
    T, H, I, k = c["T"], c["H"], c["I"], c["k"]
    x = s["x"].double()
    logits = (x @ s["router"].double().T).cpu()
    order = [sorted(range(c["E"]), key=lambda e, t=t: (-float(logits[t, e]), e))[:k]
             for t in range(T)]
    ids = torch.tensor(order, dtype=torch.int32, device="cuda")
    w = torch.softmax(torch.gather(logits, 1, ids.long().cpu()), -1).cuda()
    xq = _values64(x, c["mma"])
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in sorted({e for row in order for e in row}):
        t = torch.tensor([i for i in range(T) if e in order[i]], device="cuda")
        gu = xq[t] @ _weights64(s["w1"][e], s["w1s"][e]).T
        h = _values64(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:], c["mma"])
        y = h @ _weights64(s["w2"][e], s["w2s"][e]).T
        out[t] += (w[t] * (ids[t] == e)).sum(-1, keepdim=True) * y
    return {"out": out, "ids": ids, "weights": w}
