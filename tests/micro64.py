"""Microscaled formats in 64 bits with numpy, for tests: quantisers and decoders written
from the format definitions (one power-of-two scale per 32 values, E2M1 or E4M3 elements,
round to nearest, ties to even)."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
TOP = {"e2m1": 6.0, "e4m3": 448.0}


def bf16(a: np.ndarray) -> np.ndarray:
    """Nearest bf16 of float values (ties to even), as float64; finite input."""
    b = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def exponents(x: np.ndarray, kind: str) -> np.ndarray:
    """Smallest e >= -127 with amax <= top * 2^e per group of 32 (amax 0: -127)."""
    amax = np.abs(x.reshape(*x.shape[:-1], -1, 32)).max(-1)
    e = np.full(amax.shape, -127, np.int64)
    nz = amax > 0
    guess = np.floor(np.log2(np.where(nz, amax, 1.0) / TOP[kind])).astype(np.int64) - 1
    for _ in range(4):                       # the exact inequality decides, not the log
        guess += np.where(amax > TOP[kind] * np.exp2(guess.astype(np.float64)), 1, 0)
    e[nz] = np.maximum(guess[nz], -127)
    return e


def round_elements(v: np.ndarray, kind: str) -> np.ndarray:
    """Nearest element value of scaled values."""
    mant, emin = (1, 0) if kind == "e2m1" else (3, -6)
    ex = np.frexp(v)[1].astype(np.float64) - 1
    step = np.exp2(np.maximum(ex, emin) - mant)
    return np.rint(v / step) * step


def quantise(x: np.ndarray, kind: str):
    """(element values, exponents) of rows x [..., K]."""
    x = np.asarray(x, np.float64)
    e = exponents(x, kind)
    v = x.reshape(*e.shape, 32) * np.exp2(-e.astype(np.float64))[..., None]
    return round_elements(v, kind).reshape(x.shape), e


def values(x: np.ndarray, kind: str) -> np.ndarray:
    """What the quantised rows stand for."""
    q, e = quantise(x, kind)
    return (q.reshape(*e.shape, 32) * np.exp2(e.astype(np.float64))[..., None]).reshape(q.shape)


def e2m1_decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Values of packed codes [..., K/2] with scale bytes [..., K/32]."""
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = np.where(n > 7, -1.0, 1.0) * E2M1[n & 7]
    s = np.exp2(scales.astype(np.float64) - 127)
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(n.shape)


def e2m1_pack(values_: np.ndarray) -> np.ndarray:
    """Packed codes of element values."""
    code = np.searchsorted(E2M1, np.abs(values_)).astype(np.uint8) | \
        (np.signbit(values_).astype(np.uint8) << 3)
    return code[..., 0::2] | code[..., 1::2] << 4


def e4m3_decode(codes: np.ndarray) -> np.ndarray:
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8) * np.exp2(e - 7.0), m / 8 * 2.0 ** -6)
    return np.where(c & 128, -v, v)


def mxfp4_weights(rng, *shape):
    """Canonical MXFP4 (codes, scale bytes) of N(0, 1/sqrt(K)) rows."""
    w = rng.standard_normal(shape).astype(np.float32).astype(np.float64) * shape[-1] ** -0.5
    q, e = quantise(w, "e2m1")
    return e2m1_pack(q), (e + 127).astype(np.uint8)


def sf_offsets(rows: int, groups: int) -> np.ndarray:
    """Byte of (row, group) in the 128x4 block layout."""
    r, s = np.arange(rows)[:, None], np.arange(groups)[None, :]
    return (r // 128 * (groups // 4) + s // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + s % 4
