"""Rotary positions, the paged key-value cache and attention in fp64 — oracle
side (TEST INFRASTRUCTURE).

Plain numpy written from the definitions in include/kq.h; shares no code with
the library. 16-bit values are numpy float16, or bf16 as uint16 bit patterns.
"""
from __future__ import annotations

import numpy as np

from oracle import formats as F

PAGE = 32
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


# ---- element types

def bf16_bits(x: np.ndarray) -> np.ndarray:
    """uint16 bf16 patterns of x rounded to fp32, then to nearest even."""
    u = np.asarray(x, np.float32).view(np.uint32)
    r = (u + 0x7FFF + ((u >> 16) & 1)) >> 16
    return np.where(np.isnan(np.asarray(x, np.float32)), 0x7FC0, r).astype(np.uint16)


def widen(x: np.ndarray) -> np.ndarray:
    """fp64 of fp32, fp16, or bf16 bit patterns."""
    with np.errstate(invalid="ignore"):   # signalling NaN
        if x.dtype == np.uint16:
            return (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        return x.astype(np.float64)


def narrow(x: np.ndarray, kind: str) -> np.ndarray:
    """x rounded to fp32 and from there to the type."""
    with np.errstate(over="ignore"):
        x = np.asarray(x, np.float32)
        return x if kind == "f32" else x.astype(np.float16) if kind == "f16" else bf16_bits(x)


# ---- rotary positions

def freqs(scaling: str, rot: int, base: float, factor: float = 1.0, original: int = 0, fast: float = 32.0,
          slow: float = 1.0):
    """(radians per position [rot / 2], factor on cos and sin)."""
    i = np.arange(rot // 2)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        g = np.clip((original * f / (2 * np.pi) - slow) / (fast - slow), 0.0, 1.0)
        return g * f + (1 - g) * f / factor, 0.1 * np.log(factor) + 1 if factor > 1 else 1.0
    return f, 1.0


def rope(x: np.ndarray, positions, f: np.ndarray, m: float, interleaved: bool) -> np.ndarray:
    """x fp64 [tokens][heads][dim] rotated by the complex unit of each pair."""
    rot = 2 * len(f)
    th = np.asarray(positions, np.float64)[:, None] * f
    w = m * np.exp(1j * th)[:, None, :]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y = x.copy()
    z = (x[..., a] + 1j * x[..., b]) * w
    y[..., a], y[..., b] = z.real, z.imag
    return y


# ---- the cache

def place(kind: str, is_v: bool, p, d):
    """Index of channel d of page position p in its region (elements; bytes for q8_0)."""
    p, d = np.asarray(p), np.asarray(d)
    r, t = 4 * (p // 8) + p % 4, p // 4 % 2
    if kind == "q8_0":
        if is_v:
            return d // 32 * 1024 + (p // 8 * 16 + d % 16) * 16 + d % 32 // 16 * 8 + p % 8
        return d // 32 * 1024 + (d % 32 // 8 * 16 + r) * 16 + t * 8 + d % 8
    if is_v:
        return d // 16 * 512 + (p // 8 * 16 + d % 16) * 8 + p % 8
    return (d // 32 * 2 + t) * 512 + (d % 32 // 8 * 16 + r) * 8 + d % 8


def region_bytes(kind: str, D: int) -> int:
    return 34 * D if kind == "q8_0" else 64 * D


def q8_blocks(x: np.ndarray):
    """(codes int8 [..][D], scales float16 [..][D / 32]) of fp32 rows; a block without a finite scale: codes 0, scale NaN."""
    rows = x.reshape(-1, 32).astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        d = (np.abs(rows).max(-1) / np.float32(127)).astype(np.float16)
    bad = ~np.isfinite(rows).all(-1) | ~np.isfinite(d)
    f = F.quantize("q8_0", np.where(bad[:, None], np.float32(0), rows))
    q = f["q"].reshape(-1, 32).astype(np.int8)
    d = np.where(bad, np.float16(np.nan), f["d"].reshape(-1).view(np.float16))
    return q.reshape(x.shape), d.reshape(*x.shape[:-1], x.shape[-1] // 32)


def put(region: np.ndarray, kind: str, is_v: bool, p: int, row: np.ndarray) -> None:
    """One position's fp64 row [D] into a region (uint8)."""
    D = row.shape[0]
    at = place(kind, is_v, p, np.arange(D))
    if kind == "q8_0":
        q, d = q8_blocks(narrow(row, "f32"))
        region[at] = q.view(np.uint8)
        region[32 * D:].view(np.uint16)[np.arange(D // 32) * 32 + p] = d.view(np.uint16)
    else:
        region.view(np.uint16)[at] = narrow(row, kind).view(np.uint16)


def get(region: np.ndarray, kind: str, is_v: bool) -> np.ndarray:
    """fp64 values [32][D] of a region."""
    D = region.shape[-1] // (34 if kind == "q8_0" else 64)
    p, d = np.arange(PAGE)[:, None], np.arange(D)[None]
    at = place(kind, is_v, p, d)
    if kind == "q8_0":
        scales = region[32 * D:].view(np.float16).astype(np.float64)
        with np.errstate(invalid="ignore"):
            return region[at].view(np.int8).astype(np.float64) * scales[d // 32 * 32 + p]
    raw = region.view(np.uint16)[at]
    return widen(raw.view(np.float16) if kind == "f16" else raw)


def tokens(q_start, lens):
    """(row, sequence, index, position) of every token of a batch."""
    for s in range(len(lens)):
        n = q_start[s + 1] - q_start[s]
        for i in range(n):
            yield q_start[s] + i, s, i, lens[s] - n + i


# ---- attention

def visible(at: int, length: int, window: int, tree=None, first_new: int = 0) -> np.ndarray:
    """Which of `length` positions the query at position `at` sees."""
    j = np.arange(length)
    ok = j <= at
    if window:
        ok &= j > at - window
    if tree is not None:
        bits = np.array([(tree >> k) & 1 for k in range(64)], bool)
        among = j - first_new
        ok &= (among < 0) | ((among < 64) & bits[np.clip(among, 0, 63)])
    return ok


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, ok: np.ndarray):
    """(out [D], sum w |v| / sum w, largest score, score error unit, sum |v| / sum w) of one query over the visible keys."""
    k, v = k[ok], v[ok]
    D = q.shape[0]
    none = np.zeros(v.shape[-1])
    if not len(k):
        return none, none, 0.0, 0.0, none
    with np.errstate(invalid="ignore", over="ignore"):
        t = scale * (k @ q)
        if not np.isnan(t).any() and t.max() == -np.inf:
            return none, none, 0.0, 0.0, none
        w = np.exp(t - t.max())
        unit = float(scale * (np.abs(k) @ np.abs(q)).max()) * (D + 8) * 2.0 ** -23 + float(np.abs(t).max()) * 2.0 ** -22
        return (w @ v) / w.sum(), (w @ np.abs(v)) / w.sum(), float(np.abs(t).max()), unit, np.abs(v).sum(0) / w.sum()


def attention_tolerance(out, mass, unit, spread, n_keys, kind, weight_step, lost=2.0 ** -25):
    """What an output may be off by: its rounding; and, relative to the weighted
    mass of |v|: errors of the scores (fp32 products and sums over the channels,
    the scale) on both sides of the quotient, of exp2 (2^-21), of the sums over
    the keys in fp32, of the weights' rounding; and `lost`, what the smallest
    weights may be off by, relative to the largest."""
    rel = 2 * unit + 2.0 ** -20 + 2 * (n_keys + 16) * 2.0 ** -24 + weight_step
    return HALF_STEP[kind] * (np.abs(out) + mass * rel) + mass * rel + spread * lost + 2.0 ** -25
