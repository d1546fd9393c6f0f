"""Attention where scores are far apart or far from zero, against the fp64 oracle."""
import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import attn as A
from tests import attn_util as T
from tests import gpu_util as U

pytestmark = pytest.mark.gpu

BOTH = [("f16", "f16"), ("bf16", "bf16"), ("f16", "q8_0"), ("bf16", "q8_0")]


def attend(decode, kind, cache_kind, b, pools, q, kv_heads, D, scale, window=0, tree=None):
    """The call's rows [T][heads * D]; q [T][heads * D] as the type holds it."""
    heads = q.shape[1] // D
    cache, keep = T.cache_of(cache_kind, pools, kv_heads, D)
    batch = b.upload()
    qd, od = T.dev(q), T.dev(np.zeros_like(q))
    size = (kq.kq_attn_decode_workspace_bytes if decode else kq.kq_attn_prompt_workspace_bytes)(cache, batch, heads)
    ws = U.empty_dev((size + 16,), "uint8")
    ws.fill_(0xFF)
    print("attn", "decode" if decode else "prompt", b.new, b.lens, kind, cache_kind, heads, kv_heads, D, window, size, flush=True)
    if decode:
        kq.kq_attn_decode(kind, qd, heads * D, cache, batch, od, heads * D, heads, scale, window, None if tree is None else T.dev(tree), ws, size)
    else:
        kq.kq_attn_prompt(kind, qd, heads * D, cache, batch, od, heads * D, heads, scale, window, ws, size)
    return T.host(od, kind)


# The largest scores of a query, times log2(e), in its type's range: fp16 2^29 and
# more, bf16 2^33 and more, where neighbouring fp32 values are 64 and 1024 apart.
# Keys are one number times ones, so equal keys have equal scores, and the others
# are behind by more than 2^20: their weights are 0 and the result is the mean of V
# over the visible keys of the largest number, off by its rounding and by the
# sums' and the quotient's in fp32 (each at most 2^-24 of the mass, under 16 in
# all), and over 8-bit caches by the weights' (two bf16 parts with V's scale).
LARGE = {"f16": 2000.0, "bf16": 20000.0}


def tolerance(out, v, kind, cache_kind):
    return A.HALF_STEP[kind] * np.abs(out) + np.abs(v).mean(0) * (2.0 ** -20 + (2.0 ** -16 if cache_kind == "q8_0" else 0.0)) + 2.0 ** -25


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window", [
    ([20], [150], 3, 1, 128, 0), ([20, 3], [3000, 500], 3, 1, 128, 0), ([30, 11], [150, 77], 4, 2, 64, 40), ([40], [400], 32, 1, 128, 0),
    ([30], [200], 4, 1, 256, 0), ([50], [333], 33, 1, 160, 100), ([9], [70], 2, 2, 32, 0)])
def test_large_scores(decode, kind, cache_kind, sign, new, lens, heads, kv_heads, D, window):
    rng = np.random.default_rng(60)
    b = T.Batch(61, new, lens)

    def rows(is_v, length):
        if is_v:
            return rng.standard_normal((length, kv_heads, D))
        size = np.where(rng.random((length, kv_heads)) < 0.05, 1.0, rng.choice([0.25, 0.5], (length, kv_heads)))
        if sign < 0:
            size = np.where(size == 1.0, 0.25, 2.0 * size)   # the smallest number has the largest score
        return np.broadcast_to((sign * LARGE[kind] * size)[..., None], (length, kv_heads, D))
    pools, values = T.cache_with(b, cache_kind, kv_heads, D, rows)
    size = LARGE[kind] * rng.uniform(0.9, 1.0, (b.T, heads, 1))
    q = T.narrow(np.broadcast_to(size, (b.T, heads, D)).reshape(b.T, heads * D), kind)
    got = attend(decode, kind, cache_kind, b, pools, q, kv_heads, D, 1.0, window)
    want = {}
    for row, s, i, at in b.tokens():
        ok = A.visible(at, b.lens[s], window)
        outs, tols = [], []
        for h in range(heads):
            k, v = values[0][s][ok, h // (heads // kv_heads)], values[1][s][ok, h // (heads // kv_heads)]
            v = v[k[:, 0] == k[:, 0].max()]
            outs.append(v.mean(0))
            tols.append(tolerance(outs[-1], v, kind, cache_kind))
        want[row] = (np.array(outs), np.array(tols))
    T.check_rows(got, want, b.T, got, f"{new} {lens}")


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window", [([20], [150], 3, 1, 128, 0), ([9, 3], [2000, 500], 4, 1, 64, 0)])
def test_scores_that_grow_large(decode, kind, cache_kind, new, lens, heads, kv_heads, D, window):
    """Small scores first, then ones beyond 2^22, then ones far larger, and each the other way round in other heads."""
    rng = np.random.default_rng(62)
    b = T.Batch(63, new, lens)
    top = LARGE[kind]

    def rows(is_v, length):
        if is_v:
            return rng.standard_normal((length, kv_heads, D))
        steps = np.repeat(top * 2.0 ** np.array([-30, -12, -9, -7, -3, 0]), -(-length // 6))[:length]
        return np.broadcast_to(steps[:, None, None], (length, kv_heads, D))
    pools, values = T.cache_with(b, cache_kind, kv_heads, D, rows)
    size = top * np.where(np.arange(heads) % 2, -1.0, 1.0)[:, None] * rng.uniform(0.9, 1.0, (b.T, heads, 1))
    q = T.narrow(np.broadcast_to(size, (b.T, heads, D)).reshape(b.T, heads * D), kind)
    got = attend(decode, kind, cache_kind, b, pools, q, kv_heads, D, 1.0, window)
    want = {}
    for row, s, i, at in b.tokens():
        ok = A.visible(at, b.lens[s], window)
        outs, tols = [], []
        for h in range(heads):
            k, v = values[0][s][ok, 0], values[1][s][ok, 0]
            t = (k[:, 0] if h % 2 == 0 else -k[:, 0])
            v = v[t == t.max()]
            outs.append(v.mean(0))
            tols.append(tolerance(outs[-1], v, kind, cache_kind))
        want[row] = (np.array(outs), np.array(tols))
    T.check_rows(got, want, b.T, got, f"{new} {lens}")


# What a weight's rounding is off by, relative (one 16-bit value, or two parts).
ONE = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TWO = {"f16": 2.0 ** -22, "bf16": 2.0 ** -16, "q8_0": 2.0 ** -16}
# What the smallest weights may be off by besides: those of fp16 are multiples of
# 2^-24, rounded by half of that, and the largest is 2^14.5 or more (2^15, and two
# roundings). bf16 has no such border near the range of a softmax.
LOST = 2.0 ** -39.5


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D", [([20], [150], 6, 1, 128), ([20], [1500], 6, 1, 64), ([33], [333], 32, 1, 128)])
def test_large_and_small_scores_side_by_side(decode, kind, cache_kind, new, lens, heads, kv_heads, D):
    """Heads of one key-value head: every second one has large scores, the others ordinary ones, with ordinary tolerances."""
    rng = np.random.default_rng(64)
    b = T.Batch(65, new, lens)

    def rows(is_v, length):
        if is_v:
            return rng.standard_normal((length, kv_heads, D))
        return np.broadcast_to(LARGE[kind] * rng.choice([0.25, 0.5, 1.0], (length, kv_heads, 1)), (length, kv_heads, D))
    pools, values = T.cache_with(b, cache_kind, kv_heads, D, rows)
    size = np.where(np.arange(heads) % 2, 4.0 / (LARGE[kind] * D), LARGE[kind])[:, None] * rng.uniform(0.9, 1.0, (b.T, heads, 1))
    q = T.narrow(np.broadcast_to(size, (b.T, heads, D)).reshape(b.T, heads * D), kind)
    got = attend(decode, kind, cache_kind, b, pools, q, kv_heads, D, 1.0)
    step = TWO["q8_0" if cache_kind == "q8_0" else kind] if decode or cache_kind == "q8_0" else ONE[kind]
    want = T.attention(b, values, A.widen(q).reshape(b.T, heads, D), heads, kv_heads, D, 1.0, 0, None, kind, step, LOST)
    for row, s, i, at in b.tokens():
        ok = A.visible(at, b.lens[s], 0)
        k, v = values[0][s][ok, 0], values[1][s][ok, 0]
        v = v[k[:, 0] == k[:, 0].max()]
        for h in range(0, heads, 2):
            want[row][0][h], want[row][1][h] = v.mean(0), tolerance(v.mean(0), v, kind, cache_kind)
    T.check_rows(got, want, b.T, got, f"{new} {lens}")


# One key far above the rest, with a small V, and all the others equally far below:
# what they have in common adds up, and their weights' rounding with it. (Over 8-bit
# caches decode sums codes with 128 added, three times the mass here at most: its
# chains have one rounding per 32 keys, the tolerance two per key.)
GAPS = [9.0, 11.890625, 13.0, 13.859375, 14.90625, 16.109375, 17.5, 21.0]


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window,width", [
    ([1], [3000], 4, 1, 64, 0, None), ([1], [60], 2, 2, 128, 0, None), ([9], [2000], 4, 1, 64, 0, 40000), ([3, 1], [500, 3000], 4, 2, 96, 2999, None),
    ([40], [700], 32, 1, 128, 0, None), ([2], [1500], 1, 1, 256, 0, None)])
def test_small_weights(decode, kind, cache_kind, new, lens, heads, kv_heads, D, window, width):
    for gap in GAPS:
        rng = np.random.default_rng(66)
        b = T.Batch(67, new, lens, width=width)

        def rows(is_v, length):
            if is_v:
                v = rng.uniform(0.5, 1.5, (length, kv_heads, D))
                v[0] *= 2.0 ** -20
                return v
            k = rng.standard_normal((length, kv_heads, D))
            k[..., :32] = 0.0           # a block of its own
            k[0, :, 0] = gap
            return k
        pools, values = T.cache_with(b, cache_kind, kv_heads, D, rows)
        q = np.zeros((b.T, heads, D))
        q[..., 0] = 1.0
        q = T.narrow(q.reshape(b.T, heads * D), kind)
        got = attend(decode, kind, cache_kind, b, pools, q, kv_heads, D, 1.0, window)
        step = TWO["q8_0" if cache_kind == "q8_0" else kind] if decode or cache_kind == "q8_0" else ONE[kind]
        want = T.attention(b, values, A.widen(q).reshape(b.T, heads, D), heads, kv_heads, D, 1.0, window, None, kind, step, LOST)
        T.check_rows(got, want, b.T, got, f"{new} {lens} gap {gap}")


def test_a_long_tail_far_below():
    """131071 positions, all but the first 17.5 below it: their share (0.0033) comes out whole, in a token's call and a prompt's."""
    heads, D, length = 2, 32, 131071
    rng = np.random.default_rng(68)
    b = T.Batch(69, [1], [length])

    def rows(is_v, length):
        x = np.ones((length, 1, D)) if is_v else np.zeros((length, 1, D))
        x[0] = 0.0 if is_v else 17.5 / D
        return x
    for kind, cache_kind in BOTH:
        pools, values = T.cache_with(b, cache_kind, 1, D, rows)
        q = T.narrow(np.ones((1, heads * D)), kind)
        sink = float(values[0][0][0, 0].sum())
        tail = (length - 1) * np.exp(-sink)
        want = tail / (1 + tail)
        for decode in (True, False):
            got = A.widen(attend(decode, kind, cache_kind, b, pools, q, 1, D, 1.0))
            # its rounding; the weights' (2^-11 and 2^-8 at most); sums of 131071 in 512 parts of at most 1024 in fp32
            tol = want * (A.HALF_STEP[kind] + (TWO["q8_0" if cache_kind == "q8_0" else kind] if decode else ONE[kind]) + 2 * 1024 * 2.0 ** -24)
            assert (np.abs(got - want) <= tol).all(), (kind, cache_kind, decode, got, want)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("far", [1.0 / 64, 1.0 / 16, 1.0 / 8, 1.0])
@pytest.mark.parametrize("new,lens,heads,kv_heads,D", [([40], [160], 32, 1, 64), ([50], [700], 16, 1, 128)])
def test_scores_that_rise_from_far_below(decode, kind, cache_kind, far, new, lens, heads, kv_heads, D):
    """The first pages' scores are hugely negative, at many sizes, and their V large; the others' are ordinary."""
    rng = np.random.default_rng(90)
    b = T.Batch(91, new, lens)
    top = LARGE[kind]

    def rows(is_v, length):
        first = (np.arange(length) < 70)[:, None, None]
        if is_v:
            return np.where(first, 300.0, 1.0) * rng.standard_normal((length, kv_heads, D))
        return np.broadcast_to(np.where(first, -top * far, rng.uniform(0.5, 2.0, (length, kv_heads, 1)) / (top * D)), (length, kv_heads, D))
    pools, values = T.cache_with(b, cache_kind, kv_heads, D, rows)
    q = T.narrow(np.broadcast_to(top * rng.uniform(0.5, 1.0, (b.T, heads, 1)), (b.T, heads, D)).reshape(b.T, heads * D), kind)
    got = attend(decode, kind, cache_kind, b, pools, q, kv_heads, D, 1.0)
    step = TWO["q8_0" if cache_kind == "q8_0" else kind] if decode or cache_kind == "q8_0" else ONE[kind]
    wide, want = A.widen(q).reshape(b.T, heads, D), {}
    for row, s, i, at in b.tokens():
        ok = A.visible(at, b.lens[s], 0)
        ok[:70] = False        # their weights are below 2^-10000
        outs = [A.attend(wide[row, h], values[0][s][:, 0], values[1][s][:, 0], 1.0, ok) for h in range(heads)]
        want[row] = (np.array([o[0] for o in outs]), np.array([A.attention_tolerance(*o[:2], *o[3:], int(ok.sum()), kind, step, LOST) for o in outs]))
    T.check_rows(got, want, b.T, got, f"{new} {lens}")
