"""Rotary positions and the write into the paged cache, against the fp64 oracle.

Angles and products are 64-bit and results go through fp32, so an output is off
by half a step of its type and half a step of fp32 (f32: the latter alone), and
cached bytes equal those that the oracle's fp32 values give."""
import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import attn as A
from tests import attn_util as T
from tests import gpu_util as U

pytestmark = pytest.mark.gpu


def spec(rng, rot, pairs, positions=None, scaling="none"):
    f, m = kq.kq_rope_freqs(scaling, rot, 1e4, 4.0, 2048)
    fd = U.to_dev(f)
    return kq.kq_rope_spec(fd, rot, pairs, m, None if positions is None else U.to_dev(positions)), f, m


def within(y, want, kind):
    step = A.HALF_STEP[kind] + (0 if kind == "f32" else 2.0 ** -24)
    tiny = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[kind]
    return np.abs(A.widen(y) - want) <= np.abs(want) * step * (1 + 2.0 ** -20) + tiny + 1e-14


@pytest.mark.parametrize("xk,ok", [("f32", "f32"), ("f32", "f16"), ("f16", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,heads,D,rot,pairs,pad", [
    (1, 1, 32, 2, 0, 0), (1, 5, 128, 128, 0, 0), (7, 3, 64, 64, 1, 8), (9, 2, 96, 42, 0, 3), (17, 4, 256, 100, 1, 1),
    (33, 1, 160, 160, 0, 0), (8, 9, 224, 6, 1, 0)])
def test_rope(xk, ok, tokens, heads, D, rot, pairs, pad):
    rng = np.random.default_rng([tokens, heads, D, rot])
    positions = np.concatenate([[0, 1, 131071, -3, 2**31 - 1], rng.integers(0, 1 << 20, tokens)])[:tokens].astype(np.int32)
    rope, f, m = spec(rng, rot, pairs, positions, "yarn" if D == 128 else "none")
    ld = heads * D + pad
    x = T.narrow(rng.standard_normal((tokens, ld)), xk)
    xd, y0 = T.dev(x), T.narrow(rng.standard_normal((tokens, ld + 5)), ok)
    yd = T.dev(y0)
    print("rope", xk, ok, tokens, heads, D, rot, pairs, flush=True)
    kq.kq_rope(rope, xk, xd, ld, ok, yd, ld + 5, tokens, heads, D)
    y = T.host(yd, ok)
    want = A.rope(A.widen(x)[:, :heads * D].reshape(tokens, heads, D), positions, f, m, bool(pairs)).reshape(tokens, -1)
    assert within(y[:, :heads * D], want, ok).all()
    assert np.array_equal(y[:, heads * D:], y0[:, heads * D:])   # what lies between rows stays
    assert np.array_equal(T.host(xd, xk), x)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_rope_in_place(kind):
    rng = np.random.default_rng(5)
    positions = rng.integers(0, 9999, 21).astype(np.int32)
    rope, f, m = spec(rng, 64, 0, positions)
    x = T.narrow(rng.standard_normal((21, 6 * 64)), kind)
    out, xd = T.dev(np.zeros_like(x)), T.dev(x)
    kq.kq_rope(rope, kind, xd, 384, kind, out, 384, 21, 6, 64)
    kq.kq_rope(rope, kind, xd, 384, kind, xd, 384, 21, 6, 64)
    assert np.array_equal(T.host(xd, kind), T.host(out, kind))


def test_rope_many_tokens():
    rng = np.random.default_rng(6)
    positions = np.arange(5003, dtype=np.int32)
    rope, f, m = spec(rng, 32, 1, positions)
    x = rng.standard_normal((5003, 96)).astype(np.float32)
    y = U.empty_dev((5003, 96))
    kq.kq_rope(rope, "f32", U.to_dev(x), 96, "f32", y, 96, 5003, 3, 32)
    want = A.rope(x.astype(np.float64).reshape(5003, 3, 32), positions, f, m, True).reshape(5003, 96)
    assert within(U.to_host(y), want, "f32").all()


BATCHES = [
    ([1], [1]), ([1], [2]), ([1, 1, 1], [8, 9, 33]), ([5], [5]), ([16], [40]), ([0, 3, 0, 0, 40, 1], [7, 35, 0, 64, 45, 1]),
    ([64], [64]), ([9, 31], [41, 31]), ([3], [2]), ([4, 2], [1, 0]),
]


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("new,lens", BATCHES)
@pytest.mark.parametrize("xk,heads,kv_heads,D,rot,pairs", [
    ("f32", 4, 2, 64, 64, 0), ("bf16", 3, 3, 96, 20, 1), ("f16", 0, 1, 32, 0, 0), ("f32", 8, 1, 128, 128, 1), ("f16", 2, 2, 256, 130, 0)])
def test_append_and_read(kind, new, lens, xk, heads, kv_heads, D, rot, pairs):
    """Every byte of the cache, the rotated q, and the rows read back."""
    rng = np.random.default_rng([len(new), sum(new), D])
    b = T.Batch(D, new, lens, gap=(2, 3))
    nb = A.region_bytes(kind, D)
    pools = [rng.integers(0, 256, (b.n_pages, kv_heads, nb), dtype=np.uint8) for _ in range(2)]
    row = (heads + 2 * kv_heads) * D + (0 if D == 64 else 7)
    x = T.narrow(rng.standard_normal((b.T, row)), xk)
    xd = T.dev(x)
    rope, f, m = spec(rng, rot, pairs, scaling="linear") if rot else (None, None, None)
    cache, (kd, vd) = T.cache_of(kind, pools, kv_heads, D)
    q0 = T.narrow(rng.standard_normal((b.T, max(heads, 1) * D)), "f16")
    qd = T.dev(q0)
    print("append", kind, new, lens, xk, heads, kv_heads, D, flush=True)
    kq.kq_kv_append(cache, b.upload(), rope, xk, xd[:, heads * D:], row, xd[:, (heads + kv_heads) * D:], row,
                    xd if heads else None, row, "f16", qd if heads else None, max(heads, 1) * D, heads)
    q, kb, vb = T.host(qd, "f16"), U.to_host(kd), U.to_host(vd)
    wide = A.widen(x)
    mine = {r: (s, i, at) for r, s, i, at in b.tokens() if at >= 0}
    for r in range(b.T):
        if r not in mine or not heads:
            assert np.array_equal(q[r], q0[r])
            continue
        want = wide[r, :heads * D].reshape(1, heads, D)
        want = A.rope(want, [mine[r][2]], f, m, bool(pairs)) if rot else want
        assert within(q[r], want.reshape(-1), "f16").all(), r
    back = {}
    for r, (s, i, at) in mine.items():
        k = wide[r, heads * D:(heads + kv_heads) * D].reshape(1, kv_heads, D)
        v = wide[r, (heads + kv_heads) * D:][:kv_heads * D].reshape(kv_heads, D)
        k = (A.rope(k, [at], f, m, bool(pairs)) if rot else k)[0]
        page = b.table[s, at // 32]
        for h in range(kv_heads):
            A.put(pools[0][page, h], kind, False, at % 32, k[h])
            A.put(pools[1][page, h], kind, True, at % 32, v[h])
            back[r, h] = [A.get(p[page, h], kind, w)[at % 32] for p, w in zip(pools, (False, True))]
    assert np.array_equal(kb, pools[0]) and np.array_equal(vb, pools[1])

    for ok in ("f32", "f16", "bf16"):
        width = kv_heads * D
        o0 = T.narrow(rng.standard_normal((2, b.T, width + 1)), ok)
        od = [T.dev(o) for o in o0]
        kq.kq_kv_read(cache, b.upload(), ok, od[0], width + 1, od[1], width + 1)
        for which, (o, before) in enumerate(zip(od, o0)):
            got = T.host(o, ok)
            for r in range(b.T):
                want = before[r].copy()
                for h in range(kv_heads):
                    if (r, h) in back:
                        want[h * D:(h + 1) * D] = A.narrow(back[r, h][which], ok)
                assert np.array_equal(got[r], want, equal_nan=ok != "bf16"), (ok, which, r)


def test_append_positions_of_its_own():
    """Tokens of a tree share positions: rotation by the caller's, place by the cache's."""
    rng = np.random.default_rng(8)
    b = T.Batch(1, [4, 3], [10, 35])
    positions = np.array([6, 7, 7, 8, 32, 33, 33], np.int32)
    rope, f, m = spec(rng, 64, 0, positions)
    x = rng.standard_normal((7, 128)).astype(np.float32)
    pools = [np.zeros((b.n_pages, 1, 64 * 64), np.uint8) for _ in range(2)]
    cache, (kd, vd) = T.cache_of("f16", pools, 1, 64)
    xd = U.to_dev(x)
    kq.kq_kv_append(cache, b.upload(), rope, "f32", xd, 128, xd[:, 64:], 128)
    for r, s, i, at in b.tokens():
        k = A.rope(x[r, :64].astype(np.float64).reshape(1, 1, 64), positions[r:r + 1], f, m, False)[0, 0]
        A.put(pools[0][b.table[s, at // 32], 0], "f16", False, at % 32, k)
        A.put(pools[1][b.table[s, at // 32], 0], "f16", True, at % 32, x[r, 64:].astype(np.float64))
    assert np.array_equal(U.to_host(kd), pools[0]) and np.array_equal(U.to_host(vd), pools[1])


def test_append_bad_pages():
    """Ids outside the cache and positions behind the table: nothing is stored, q is rotated, reads give NaN."""
    rng = np.random.default_rng(9)
    b = T.Batch(2, [40, 2, 3], [40, 70, 200], width=3)
    b.table[0, 0] = -1
    b.table[1, 2] = b.n_pages
    for s in range(3):
        b.table[s] = np.where((b.table[s] >= 0) & (b.table[s] < b.n_pages), b.table[s], -1)
    rope, f, m = spec(rng, 32, 0)
    x = T.narrow(rng.standard_normal((45, 96)), "f16")
    pools = [np.full((b.n_pages, 1, 34 * 32), 7, np.uint8) for _ in range(2)]
    cache, (kd, vd) = T.cache_of("q8_0", pools, 1, 32)
    xd, qd = T.dev(x), T.dev(np.zeros((45, 32), np.float16))
    kq.kq_kv_append(cache, b.upload(), rope, "f16", xd, 96, xd[:, 32:], 96, xd[:, 64:], 96, "f16", qd, 32, 1)
    k, v = U.empty_dev((45, 32)), U.empty_dev((45, 32))
    kq.kq_kv_read(cache, b.upload(), "f32", k, 32, v, 32)
    k, v, q = U.to_host(k), U.to_host(v), T.host(qd, "f16")
    for r, s, i, at in b.tokens():
        page = b.table[s, at // 32] if at // 32 < 3 else -1
        want = A.rope(A.widen(x[r, 64:]).reshape(1, 1, 32), [at], f, m, False).reshape(-1)
        assert within(q[r], want, "f16").all()
        assert np.isnan(k[r]).all() == np.isnan(v[r]).all() == (page < 0), r
        if page >= 0:
            kr = A.rope(A.widen(x[r, :32]).reshape(1, 1, 32), [at], f, m, False).reshape(-1)
            A.put(pools[0][page, 0], "q8_0", False, at % 32, kr)
            A.put(pools[1][page, 0], "q8_0", True, at % 32, A.widen(x[r, 32:64]))
    assert np.array_equal(U.to_host(kd), pools[0]) and np.array_equal(U.to_host(vd), pools[1])


@pytest.mark.parametrize("n", [1, 8, 11])
def test_append_values_at_the_ends(n):
    """Q8_0 blocks with zeros, ties, subnormal scales, infinities and NaN; 16-bit types past their range."""
    rng = np.random.default_rng(10)
    rows = rng.standard_normal((11, 2, 32)).astype(np.float32)
    rows[0] = 0
    rows[1] = 127 * np.float32(2.0 ** -20)
    rows[1, :, ::3] = 2.5 * np.float32(2.0 ** -20)
    rows[2] = np.arange(-16, 16) * np.float32(0.5)
    rows[3, 0, 5] = np.inf
    rows[4, 1, 6] = np.nan
    rows[5, 0, 0] = 1e7
    rows[6] = 1e-7
    rows[7] = 1e-12
    rows[8, :, 31] = -70000
    rows = rows[:n].reshape(n, 64)
    b = T.Batch(3, [n], [n])
    for kind in ("q8_0", "f16", "bf16"):
        pools = [np.zeros((b.n_pages, 1, A.region_bytes(kind, 64)), np.uint8) for _ in range(2)]
        cache, (kd, vd) = T.cache_of(kind, pools, 1, 64)
        xd = U.to_dev(rows)
        kq.kq_kv_append(cache, b.upload(), None, "f32", xd, 64, xd, 64)
        for is_v, got in ((False, U.to_host(kd)), (True, U.to_host(vd))):
            have = A.get(got[b.table[0, 0], 0], kind, is_v)[:n]
            want = np.zeros_like(got[0, 0])
            for p in range(n):
                A.put(want, kind, is_v, p, rows[p].astype(np.float64))
            assert np.array_equal(have, A.get(want, kind, is_v)[:n], equal_nan=True), (kind, is_v)
