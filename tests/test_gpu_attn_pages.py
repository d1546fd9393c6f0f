"""Attention where some pages' ids are invalid: what the other rows get. The ids'
places are read as page 0's until they are masked, so page 0 is part of the
checks: its rows, and none of its values where a query sees no page 0."""
import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import attn as A
from tests import attn_util as T
from tests import gpu_util as U
from tests.test_gpu_attn_range import BOTH, LOST, ONE, TWO, attend

pytestmark = pytest.mark.gpu


def check(decode, kind, cache_kind, new, lens, heads, kv_heads, D, window, bad, width=None, trees=False):
    """bad: (sequence, page of its) whose id is invalid."""
    rng = np.random.default_rng(70)
    b = T.Batch(71, new, lens, width=width)
    pools, values = T.random_cache(72, b, cache_kind, kv_heads, D)
    # page 0 of the cache belongs to no sequence: large finite values, which must show nowhere
    for s in range(b.S):
        n = -(-lens[s] // A.PAGE)
        if (b.table[s, :n] == 0).any():
            spare = [i for i in range(1, b.n_pages) if not (b.table == i).any()][0]
            at = b.table[s, :n] == 0
            for pool in pools:
                pool[spare] = pool[0]
            b.table[s, :n][at] = spare
    for is_v, pool in enumerate(pools):
        for h in range(kv_heads):
            for p in range(A.PAGE):
                A.put(pool[0, h], cache_kind, bool(is_v), p, np.full(D, 50.0 + p))
    for i, (s, page) in enumerate(bad):
        b.table[s, page] = [-1, b.n_pages, 0x7fffffff, -2 ** 31][i % 4]
    q = T.narrow(rng.standard_normal((b.T, heads * D)), kind)
    tree = None
    if trees:
        tree = np.zeros(b.T, np.uint64)
        for row, s, i, at in b.tokens():
            tree[row] = np.uint64(1 << i)
    got = attend(decode, kind, cache_kind, b, pools, q, kv_heads, D, D ** -0.5, window, tree)
    step = TWO["q8_0" if cache_kind == "q8_0" else kind] if decode or cache_kind == "q8_0" else ONE[kind]
    want = T.attention(b, values, A.widen(q).reshape(b.T, heads, D), heads, kv_heads, D, np.float32(D ** -0.5).astype(np.float64), window, tree,
                       kind, step, LOST if cache_kind != "q8_0" else 2.0 ** -25)
    clean = 0
    for row, s, i, at in b.tokens():
        ok = A.visible(at, lens[s], window, None if tree is None else int(tree[row]), lens[s] - new[s])
        if any(ok[32 * page:32 * page + 32].any() for t, page in bad if t == s):
            want[row] = tuple(np.full((heads, D), np.nan) for _ in range(2))
        else:
            clean += 1
    assert 0 < clean < b.T
    T.check_rows(got, want, b.T, got, f"{new} {lens} {bad}")


CASES = [
    # new, lens, heads, kv_heads, D, window, bad
    ([3, 2, 4, 1], [66, 40, 130, 30], 4, 2, 64, 0, [(0, 2), (1, 0)]),
    ([6, 3], [300, 70], 4, 2, 128, 40, [(0, 0), (0, 5), (0, 8)]),      # behind and inside the windows
    ([40, 1], [40, 90], 8, 2, 96, 0, [(0, 1)]),
    ([30, 7], [2000, 700], 4, 1, 64, 500, [(0, 3), (0, 62), (1, 10)]),
    ([2, 2], [700, 900], 2, 1, 256, 0, [(1, 12)]),
]


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window,bad", CASES)
def test_rows_beside_bad_pages(decode, kind, cache_kind, new, lens, heads, kv_heads, D, window, bad):
    check(decode, kind, cache_kind, new, lens, heads, kv_heads, D, window, bad)


@pytest.mark.parametrize("kind,cache_kind", BOTH)
def test_rows_beside_bad_pages_of_large_tiles(kind, cache_kind):
    check(False, kind, cache_kind, [300, 30], [300, 200], 8, 1, 128, 0, [(0, 3)])
    check(False, kind, cache_kind, [400], [900], 8, 2, 128, 200, [(0, 2), (0, 20)])


@pytest.mark.parametrize("kind,cache_kind", BOTH)
def test_rows_beside_bad_pages_of_wide_tiles(kind, cache_kind):
    check(True, kind, cache_kind, [9, 5], [200, 500], 4, 1, 64, 150, [(0, 0), (0, 6), (1, 10)], width=1 + 160000000 // (34 * 64 * 2))


@pytest.mark.parametrize("kind,cache_kind", BOTH)
def test_branches_beside_a_bad_page(kind, cache_kind):
    """Rows that see of the new tokens themselves alone, with the new tokens in two pages, one of them bad."""
    check(True, kind, cache_kind, [8, 3], [36, 40], 4, 2, 64, 20, [(0, 1)], trees=True)
