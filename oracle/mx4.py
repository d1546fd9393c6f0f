"""Microscaled 4-bit matrices, the router and the whole mixture-of-experts
layer in fp64 — oracle side (TEST INFRASTRUCTURE).

Plain numpy written from the definitions in include/kq.h: blocks of 32
elements of a row, scale byte s = 2^(s - 127) (255: NaN), 4-bit codes (sign,
two exponent bits, one mantissa bit). Products of a code, a scale and a 16- or
32-bit activation are exact in fp64; the sums' errors (about K * 2^-53) are
far below every tolerance.
"""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def widen(x: np.ndarray) -> np.ndarray:
    """fp64 of fp32, fp16, or bf16 given as uint16 bit patterns."""
    if x.dtype == np.uint16:
        return (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return x.astype(np.float64)


def nearest_code(a: np.ndarray) -> np.ndarray:
    """Code (0..7) of the magnitudes a: the nearest magnitude, on ties the one
    whose mantissa bit (the code's lowest) is 0; the largest beyond it."""
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    code = np.arange(8)
    # of the (at most two) nearest codes the even one: order by (distance, odd)
    return np.argmin(np.where(d == best, code % 2, 2), axis=-1)


def quantize(x: np.ndarray):
    """(codes [R][K] of 0..15, scale bytes [R][K/32]) of x [R][K]."""
    v = widen(np.asarray(x))
    R, K = v.shape
    b = v.reshape(R, K // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = np.frexp(amax)[1] - 1                      # floor(log2(amax)) where amax > 0
    s = np.where(amax > 0, np.clip(e - 2 + 127, 0, 254), 0)
    a = np.ldexp(np.abs(b), -(s[..., None] - 127))
    code = nearest_code(a) | (np.signbit(b).astype(np.int64) << 3)
    code = np.where(bad[..., None], 0, code)
    s = np.where(bad, 255, s)
    return code.reshape(R, K).astype(np.uint8), s.astype(np.uint8)


def planes(codes: np.ndarray, scales: np.ndarray):
    """The bytes of the two planes."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8), scales.astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 values [R][K]: code times scale (up to 6 * 2^127; scale 255 NaN), as the products take them."""
    sign = np.where(codes & 8, -1.0, 1.0)
    s = np.repeat(scales.astype(np.int64), BLOCK, axis=1)
    return np.where(s == 255, np.nan, sign * np.ldexp(MAGNITUDES[codes & 7], (s - 127).astype(np.int32)))


def dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values as fp32 and bf16 hold them: infinite from 2^128 on."""
    v = values(codes, scales)
    return np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)


def product(w: np.ndarray, x: np.ndarray):
    """y [M][N] and sum |w x| for values w [N][K], x [M][K]."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def route(x: np.ndarray, W: np.ndarray, top_k: int, renorm: bool):
    """ids, weights [M][top_k] and the logits [M][E]."""
    l = x @ W.T
    key = np.where(np.isnan(l), -np.inf, l)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
    best = np.take_along_axis(l, ids, 1)
    with np.errstate(invalid="ignore"):
        p = np.exp(best - best[:, :1])
        total = p.sum(1) if renorm else np.exp(l - best[:, :1]).sum(1)
        return ids.astype(np.int32), p / total[:, None], l


def silu(z: np.ndarray) -> np.ndarray:
    return z / (1.0 + np.exp(-z))


def moe_layer(x, gate, up, down, ids, weights, unit: float = 2.0 ** -23):
    """y [M][H] for values x [M][H], gate, up [E][I][H], down [E][H][I] and the
    given routes, and a bound on the error of sums taken in fp32: every
    addition rounds by at most `unit` of the sum of magnitudes."""
    M, H = x.shape
    inter = gate.shape[1]
    y, bound = np.zeros((M, H)), np.zeros((M, H))
    for m in range(M):
        for j in range(ids.shape[1]):
            e, p = int(ids[m, j]), weights[m, j]
            g, u = gate[e] @ x[m], up[e] @ x[m]
            dg, du = (np.abs(gate[e]) @ np.abs(x[m]) * (H + 64) * unit, np.abs(up[e]) @ np.abs(x[m]) * (H + 64) * unit)
            h = silu(g) * u
            # |silu'| <= 1.1; eight roundings from the sums to h
            dh = 1.1 * np.abs(u) * dg + (np.abs(silu(g)) + 1.1 * dg) * du + 8 * unit * np.abs(h)
            y[m] += p * (down[e] @ h)
            a = np.abs(down[e])
            bound[m] += p * (a @ dh + (inter + 64 + 8 * ids.shape[1]) * unit * (a @ np.abs(h)))
    return y, bound
