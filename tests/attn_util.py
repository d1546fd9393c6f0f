"""Batches for the tests of rotary positions, the paged cache and attention:
seeded inputs in numpy, their upload, and the oracle's results."""
import numpy as np

import block_quantized_gemv_kq_amd as kq
from oracle import attn as A
from tests import gpu_util as U

TYPE_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
NP_TYPE = {"f32": np.float32, "f16": np.float16, "bf16": np.uint16}


def narrow(x, kind):
    """Random values as the type holds them."""
    return A.narrow(np.asarray(x, np.float64), kind)


def dev(a):
    """Upload; uint16 patterns and other unsigned types go as bytes-compatible signed ones."""
    a = np.ascontiguousarray(a)
    signed = {np.dtype(np.uint16): np.int16, np.dtype(np.uint64): np.int64}.get(a.dtype)
    return U.to_dev(a.view(signed) if signed else a)


def host(t, kind):
    """Download as the type's numpy form."""
    a = U.to_host(t)
    return a.view(NP_TYPE[kind]) if kind != "f32" else a


class Batch:
    """Sequences with `new` tokens and `lens` positions; pages anywhere in a
    cache of `spare` more pages than needed; `gap` rows before the first and
    behind the last sequence that belong to none."""

    def __init__(self, seed, new, lens, gap=(0, 0), spare=3, width=None):
        rng = np.random.default_rng(seed)
        self.new, self.lens = list(new), list(lens)
        self.S = len(self.new)
        self.q_start = np.concatenate([[gap[0]], gap[0] + np.cumsum(self.new)]).astype(np.int32) if self.S else np.array([gap[0]], np.int32)
        self.T = int(self.q_start[-1]) + gap[1]
        counts = [-(-n // A.PAGE) for n in self.lens]
        self.width = width or max([1] + counts)
        self.n_pages = sum(counts) + spare
        ids = rng.permutation(self.n_pages).astype(np.int32)
        # entries behind a sequence's pages name no page at all: they must not be followed
        self.table = np.where(rng.random((max(self.S, 1), self.width)) < 0.5, -5, 0x7fffffff).astype(np.int32)
        at = 0
        for s, c in enumerate(counts):
            self.table[s, :c] = ids[at:at + min(c, self.width)]   # a table may be narrower than a sequence
            at += c
        self.dev = None

    def upload(self):
        if self.dev is None:
            self.dev = [dev(self.table), dev(self.q_start), dev(np.array(self.lens + [0], np.int32))]
        return kq.kq_kv_batch(self.dev[0], self.width, self.dev[1], self.dev[2], self.S, self.T)

    def tokens(self):
        return A.tokens(self.q_start, self.lens)


def random_cache(seed, batch, kind, kv_heads, D, spread=1.0):
    """cache_with of normal values."""
    rng = np.random.default_rng(seed)
    return cache_with(batch, kind, kv_heads, D, lambda is_v, length: rng.standard_normal((length, kv_heads, D)) * spread)


def cache_with(batch, kind, kv_heads, D, rows):
    """(k, v) uint8 [pages][kv_heads][region] with the sequences' positions
    holding rows(is_v, length) [length][kv_heads][D] and every other byte of every
    page 0xFF (NaN in all 16-bit types and in the scales), and the values fp64
    per sequence [len][kv_heads][D]."""
    nb = A.region_bytes(kind, D)
    pools, values = [], []
    for is_v in (False, True):
        pool = np.full((batch.n_pages, kv_heads, nb), 0xFF, np.uint8)
        vals = []
        for s, length in enumerate(batch.lens):
            x = rows(is_v, length)
            if kind == "q8_0":
                codes, scales = A.q8_blocks(A.narrow(x, "f32"))
                got = codes.astype(np.float64) * np.repeat(scales.astype(np.float64), 32, -1)
            else:
                raw = narrow(x, kind)
                got = A.widen(raw)
            pos = np.arange(length)
            page, p = batch.table[s, pos // A.PAGE], pos % A.PAGE
            at = A.place(kind, is_v, p[:, None], np.arange(D)[None])
            for h in range(kv_heads):
                flat = pool[:, h]
                if kind == "q8_0":
                    flat[page[:, None], at] = codes[:, h].view(np.uint8)
                    sc = 32 * D + 2 * (np.arange(D // 32)[None] * 32 + p[:, None])
                    b = scales[:, h].copy().view(np.uint8).reshape(length, D // 32, 2)
                    flat[page[:, None], sc] = b[..., 0]
                    flat[page[:, None], sc + 1] = b[..., 1]
                else:
                    b = raw[:, h].copy().view(np.uint8).reshape(length, D, 2)
                    flat[page[:, None], 2 * at] = b[..., 0]
                    flat[page[:, None], 2 * at + 1] = b[..., 1]
            vals.append(got)
        pools.append(pool)
        values.append(vals)
    return pools, values


def cache_of(kind, pools, kv_heads, D, extra=0):
    """(struct, device buffers)."""
    k, v = dev(pools[0]), dev(pools[1])
    return kq.kq_kv_cache(kind, k, v, pools[0].shape[0], kv_heads, D), (k, v)


def attention(batch, values, q, heads, kv_heads, D, scale, window, tree, kind, weight_step, lost=2.0 ** -25):
    """The oracle's rows and their tolerances: {row: (out [heads][D], tolerance)}."""
    got = {}
    for row, s, i, at in batch.tokens():
        n, length = batch.new[s], batch.lens[s]
        ok = A.visible(at, length, window, None if tree is None else int(tree[row]), length - n)
        outs, tols = [], []
        for h in range(heads):
            kh = h // (heads // kv_heads)
            k, v = values[0][s][:, kh], values[1][s][:, kh]
            out, mass, _, unit, spread = A.attend(q[row, h], k, v, scale, ok)
            outs.append(out)
            tols.append(A.attention_tolerance(out, mass, unit, spread, int(ok.sum()), kind, weight_step, lost))
        got[row] = (np.array(outs), np.array(tols))
    return got


def check_rows(got, want, T, canary, what):
    """Rows of `want` within their tolerances, infinities and NaN where `want` has them, every other row still the canary's."""
    for row in range(T):
        if row not in want:
            assert np.array_equal(got[row].view(np.uint16), canary[row].view(np.uint16)), f"{what}: row {row} belongs to none"
            continue
        out, tol = want[row]
        y = A.widen(got[row]).reshape(out.shape)
        # where there is no finite result or tolerance, the value itself: |y - inf| <= inf holds for every y
        fine = np.isfinite(out) & np.isfinite(tol)
        with np.errstate(invalid="ignore"):
            bad = np.where(fine, ~(np.abs(y - out) <= tol), ~((y == out) | (np.isnan(y) & np.isnan(out))))
        if bad.any():
            i = tuple(np.argwhere(bad)[0])
            raise AssertionError(f"{what}: row {row}: {bad.sum()} outputs off; first {i}: got {y[i]!r} want {out[i]!r} tolerance {tol[i]!r}")
