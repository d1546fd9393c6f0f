"""Attention over the paged cache against the fp64 oracle: decode and verify
passes, and prompts. Every byte of the cache that no sequence owns is 0xFF (NaN
in every type), as are the positions behind a sequence in its last page."""
import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import attn as A
from tests import attn_util as T
from tests import gpu_util as U

pytestmark = pytest.mark.gpu

# What a weight's rounding is off by, relative: one 16-bit value, or two parts
# of 8 (bf16; also the 8-bit caches') or 11 bits.
ONE = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TWO = {"f16": 2.0 ** -22, "bf16": 2.0 ** -16, "q8_0": 2.0 ** -16}


def run(decode, seed, new, lens, kind, cache_kind, heads, kv_heads, D, window=0, trees=False, gap=(0, 0), pad=(0, 0), spread=1.0,
        width=None, change=None, scale=None):
    rng = np.random.default_rng(seed)
    b = T.Batch(seed, new, lens, gap=gap, width=width)
    pools, values = T.random_cache(seed + 1, b, cache_kind, kv_heads, D)
    if change:
        change(b, pools, values)
    q = T.narrow(rng.standard_normal((b.T, heads * D + pad[0])) * spread, kind)
    out0 = T.narrow(rng.standard_normal((b.T, heads * D + pad[1])), kind)
    tree = None
    if trees:
        tree = np.zeros(b.T, np.uint64)
        for row, s, i, at in b.tokens():
            parent = int(tree[row - 1 - rng.integers(0, i)]) if i else 0
            tree[row] = parent | 1 << i
        if b.T > 2:
            tree[b.q_start[0]] &= np.uint64(~1 & (1 << 64) - 1)   # a row that does not see itself
    cache, keep = T.cache_of(cache_kind, pools, kv_heads, D)
    qd, od = T.dev(q), T.dev(out0)
    td = None if tree is None else T.dev(tree)
    batch = b.upload()
    scale = scale or D ** -0.5
    size = (kq.kq_attn_decode_workspace_bytes if decode else kq.kq_attn_prompt_workspace_bytes)(cache, batch, heads)
    ws = U.empty_dev((size + 512,), "uint8")
    ws.fill_(0xFF)
    print("attn", "decode" if decode else "prompt", new, lens, kind, cache_kind, heads, kv_heads, D, window, size, flush=True)
    if decode:
        kq.kq_attn_decode(kind, qd, heads * D + pad[0], cache, batch, od, heads * D + pad[1], heads, scale, window, td, ws[256:], size)
    else:
        kq.kq_attn_prompt(kind, qd, heads * D + pad[0], cache, batch, od, heads * D + pad[1], heads, scale, window, ws[256:], size)
    out, guard = T.host(od, kind), U.to_host(ws)
    assert (guard[:256] == 0xFF).all() and (guard[256 + size:] == 0xFF).all()
    assert np.array_equal(out[:, heads * D:], out0[:, heads * D:])
    step = TWO["q8_0" if cache_kind == "q8_0" else kind] if decode or cache_kind == "q8_0" else ONE[kind]
    wide = A.widen(q)[:, :heads * D].reshape(b.T, heads, D)
    want = T.attention(b, values, wide, heads, kv_heads, D, np.float32(scale).astype(np.float64), window, tree, kind, step)
    T.check_rows(np.ascontiguousarray(out[:, :heads * D]), want, b.T, np.ascontiguousarray(out0[:, :heads * D]), f"{new} {lens}")
    return b, out


BOTH = [("f16", "f16"), ("bf16", "bf16"), ("f16", "q8_0"), ("bf16", "q8_0")]
DECODES = [
    # new, lens, heads, kv_heads, D, window
    ([1], [1], 1, 1, 32, 0), ([1], [31], 4, 1, 64, 0), ([1, 1, 1], [32, 33, 64], 8, 2, 128, 0), ([1, 1], [0, 5], 2, 2, 64, 0),
    ([2, 0, 3, 1], [1, 40, 100, 7], 6, 2, 96, 0), ([16], [50], 4, 1, 128, 0), ([1] * 64, list(range(1, 129, 2)), 5, 1, 32, 0),
    ([8, 8], [300, 8], 24, 8, 64, 0), ([1], [97], 16, 1, 256, 0), ([7, 2], [64, 65], 3, 3, 160, 0), ([64], [70], 2, 1, 64, 0),
    ([20], [21], 5, 1, 192, 0), ([30], [95], 2, 2, 224, 0), ([1, 3], [100, 90], 4, 2, 128, 1), ([5, 1], [70, 200], 4, 4, 64, 33),
    ([9], [129], 8, 1, 128, 40), ([3], [8], 2, 1, 64, 1000), ([16], [90], 8, 1, 256, 0), ([33], [33], 8, 2, 96, 0),
]


@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window", DECODES)
def test_decode(kind, cache_kind, new, lens, heads, kv_heads, D, window):
    run(True, 1, new, lens, kind, cache_kind, heads, kv_heads, D, window)


@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window", [
    ([1], [5000], 4, 1, 64, 0), ([1, 1, 1], [3001, 10, 700], 4, 2, 128, 0), ([16, 5], [1500, 2000], 8, 2, 64, 0),
    ([1], [4096], 2, 2, 256, 0), ([3, 1], [2500, 2000], 4, 2, 32, 1500), ([40], [1999], 8, 1, 128, 0)])
def test_decode_split(kind, cache_kind, new, lens, heads, kv_heads, D, window):
    """Lengths that are split over workgroups and joined."""
    run(True, 2, new, lens, kind, cache_kind, heads, kv_heads, D, window)


@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window", [
    ([8], [8], 4, 2, 64, 0), ([16, 16, 16], [100, 33, 16], 4, 2, 128, 0), ([7, 1], [2000, 40], 2, 1, 96, 0), ([64], [100], 1, 1, 32, 0),
    ([5, 9], [64, 80], 4, 1, 64, 20)])
def test_decode_trees(kind, cache_kind, new, lens, heads, kv_heads, D, window):
    run(True, 3, new, lens, kind, cache_kind, heads, kv_heads, D, window, trees=True)


PROMPTS = [
    ([1], [1], 1, 1, 32, 0), ([33], [33], 4, 1, 64, 0), ([5, 70, 0, 1], [5, 70, 9, 1], 4, 2, 128, 0), ([130], [130], 2, 2, 64, 0),
    ([40, 64], [100, 64], 6, 2, 96, 0), ([31], [200], 8, 1, 128, 0), ([300], [300], 3, 1, 64, 0), ([2, 3], [1, 2], 2, 1, 64, 0),
    ([100], [100], 5, 1, 256, 0), ([65, 3], [65, 90], 4, 4, 160, 0), ([90], [90], 4, 1, 192, 0), ([50], [51], 2, 1, 224, 0),
    ([128], [128], 4, 2, 64, 1), ([100, 20], [150, 400], 4, 2, 128, 40), ([200], [200], 2, 1, 64, 64), ([60], [60], 8, 1, 32, 500),
]


@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window", PROMPTS)
def test_prompt(kind, cache_kind, new, lens, heads, kv_heads, D, window):
    run(False, 4, new, lens, kind, cache_kind, heads, kv_heads, D, window)


@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window", [
    ([40], [3000], 2, 1, 64, 0), ([33, 100], [2500, 900], 4, 2, 128, 0), ([20], [4000], 2, 2, 96, 1700)])
def test_prompt_split(kind, cache_kind, new, lens, heads, kv_heads, D, window):
    run(False, 5, new, lens, kind, cache_kind, heads, kv_heads, D, window)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
def test_rows_of_none_and_strides(decode, kind, cache_kind):
    """Rows before and behind the sequences keep what they held; rows apart by odd numbers of elements."""
    run(decode, 6, [3, 5], [40, 70], kind, cache_kind, 4, 2, 64, gap=(2, 4), pad=(3, 5), width=9)
    run(decode, 7, [3, 5], [40, 70], kind, cache_kind, 4, 2, 64, gap=(1, 1), pad=(8, 16))


@pytest.mark.parametrize("decode", [True, False])
def test_many_sequences(decode):
    n = 64 if decode else 200
    run(decode, 8, [1] * n, [1 + (7 * i) % 90 for i in range(n)], "f16", "f16", 2, 1, 32)
    if not decode:
        run(decode, 9, [i % 5 for i in range(150)], [i % 5 + i % 37 for i in range(150)], "bf16", "q8_0", 2, 2, 32, gap=(1, 2))


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
def test_peaked_and_large_scores(decode, kind, cache_kind):
    run(decode, 10, [5], [150], kind, cache_kind, 4, 2, 64, spread=30.0)
    run(decode, 11, [5], [150], kind, cache_kind, 4, 2, 64, spread=0.0)
    run(decode, 12, [5], [150], kind, cache_kind, 4, 2, 64, scale=1e-30)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", [("f16", "f16"), ("bf16", "q8_0")])
@pytest.mark.parametrize("heads,kv_heads", [(1024, 1), (1024, 1024), (1023, 341)])
def test_most_heads(decode, kind, cache_kind, heads, kv_heads):
    run(decode, 42, [1, 1], [40, 170], kind, cache_kind, heads, kv_heads, 32)


def test_most_sequences():
    """4096 sequences, most of them without new tokens."""
    lens = [(7 * s) % 50 for s in range(4096)]
    new = [1 if s % 61 == 60 and lens[s] else 0 for s in range(4096)]
    run(False, 43, new, lens, "f16", "f16", 2, 1, 32)


def poison(which, where):
    """Puts infinities and NaN into K or V of one position, in the cache and the values."""
    def change(b, pools, values):
        s, p = where
        page = b.table[s, p // 32]
        D = values[which][s].shape[-1]
        for h in range(pools[which].shape[1]):
            row = values[which][s][p, h]
            row[0], row[1], row[D - 1] = np.inf, np.nan, -np.inf
            A.put(pools[which][page, h], "f16" if row_kind[0] == "f16" else row_kind[0], bool(which), p % 32, row)
    row_kind = ["f16"]
    change.kind = row_kind
    return change


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("new,lens,window,where", [
    ([4], [40], 0, 38), ([4], [70], 3, 64), ([6], [100], 0, 97), ([2], [64], 0, 10), ([12], [33], 5, 20)])
def test_not_finite_in_masked_places(decode, kind, new, lens, window, where):
    """A position with infinities and NaN in V reaches the queries that see it and no other."""
    change = poison(1, (0, where))
    change.kind[0] = kind
    run(decode, 13, new, lens, kind, kind, 4, 2, 64, window, change=change)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
def test_not_finite_keys(decode, kind, cache_kind):
    """NaN in K of a position: queries that see it are NaN, earlier ones are not."""
    def change(b, pools, values):
        page = b.table[0, 1]
        for h in range(2):
            row = values[0][0][36, h]
            row[:32] = np.nan
            A.put(pools[0][page, h], cache_kind, False, 4, row)
    b, out = run(decode, 14, [6], [40], kind, cache_kind, 4, 2, 64, change=change)
    got = np.isnan(A.widen(out))
    assert not got[:2].any() and got[2:].all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("decode", [True, False])
def test_bad_scale_in_a_masked_place(decode, kind):
    """A Q8_0 block of V that reads as NaN reaches the queries that see it and no other."""
    def change(b, pools, values):
        for h in range(2):
            row = values[1][0][38, h]
            row[32:] = np.nan
            A.put(pools[1][b.table[0, 1], h], "q8_0", True, 6, row)
    b, out = run(decode, 15, [4], [40], kind, "q8_0", 4, 2, 64, change=change)
    got = np.isnan(A.widen(out)).reshape(4, 4, 64)
    assert not got[:2].any() and got[2:, :, 32:].all() and not got[2:, :, :32].any()


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kind,cache_kind", BOTH)
def test_bad_pages(decode, kind, cache_kind):
    """A page id outside the cache: NaN for the queries that see it. A sequence longer than its table: NaN for all."""
    rng = np.random.default_rng(16)
    b = T.Batch(16, [3, 2, 4, 1], [66, 40, 130, 30])
    pools, values = T.random_cache(17, b, cache_kind, 2, 64)
    b.table[0, 2] = -1            # positions 64, 65
    b.table[1, 0] = b.n_pages     # positions 0..31
    b.width = 4
    b.table = np.ascontiguousarray(b.table[:, :4])   # sequence 2 has 5 pages
    q = T.narrow(rng.standard_normal((10, 256)), kind)
    cache, keep = T.cache_of(cache_kind, pools, 2, 64)
    qd, od = T.dev(q), T.dev(np.zeros_like(q))
    batch = b.upload()
    fn = kq.kq_attn_decode if decode else kq.kq_attn_prompt
    size = (kq.kq_attn_decode_workspace_bytes if decode else kq.kq_attn_prompt_workspace_bytes)(cache, batch, 4)
    ws = U.empty_dev((size + 16,), "uint8")
    fn(kind, qd, 256, cache, batch, od, 256, 4, 0.125, workspace=ws, workspace_bytes=size)
    bad = np.isnan(A.widen(T.host(od, kind))).all(-1)
    assert bad.tolist() == [False, True, True, True, True, True, True, True, True, False]
    # behind a window of 8 the bad page is not seen from position 39, and is from 38 (31 .. 38)
    fn(kind, qd, 256, cache, batch, od, 256, 4, 0.125, 8, workspace=ws, workspace_bytes=size)
    out = A.widen(T.host(od, kind))
    assert np.isnan(out).all(-1).tolist() == [False, True, True, True, False, True, True, True, True, False]
    assert not np.isnan(out[4]).any()


@pytest.mark.parametrize("decode", [True, False])
def test_starts_that_do_not_ascend(decode):
    """Arrays that hold nonsense touch nothing outside the buffers, and the call ends."""
    torch = U.torch_cuda()
    b = T.Batch(18, [3, 2, 4], [66, 40, 700])
    pools, _ = T.random_cache(19, b, "f16", 2, 64)
    cache, keep = T.cache_of("f16", pools, 2, 64)
    for starts, lens in (([9, 0, 9, 0], [700, 700, 700]), ([-5, 4, 2**31 - 1, 3], [2**31 - 1, -7, 50]), ([0, 9, 0, 9], [3, 704, 2**30])):
        batch = b.upload()
        b.dev[1].copy_(torch.tensor(starts, dtype=torch.int32))
        b.dev[2][:3].copy_(torch.tensor(lens, dtype=torch.int32))
        q = T.dev(np.ones((9 + 8, 256), np.float16))
        out = T.dev(np.full((9 + 8, 256), 5, np.float16))
        size = (kq.kq_attn_decode_workspace_bytes if decode else kq.kq_attn_prompt_workspace_bytes)(cache, batch, 4)
        ws = U.empty_dev((size + 512,), "uint8")
        ws.fill_(0xFF)
        fn = kq.kq_attn_decode if decode else kq.kq_attn_prompt
        fn("f16", q, 256, cache, batch, out, 256, 4, 0.125, workspace=ws, workspace_bytes=size)
        guard = U.to_host(ws)
        assert (guard[size:] == 0xFF).all()
        assert (T.host(out, "f16")[9:] == 5).all()


def test_same_bits_again():
    """Two calls, and one on another stream, give the same bits; a call's workspace needs no contents."""
    torch = U.torch_cuda()
    for decode in (True, False):
        b = T.Batch(20, [2, 7], [3000, 500])
        pools, _ = T.random_cache(21, b, "bf16", 2, 128)
        cache, keep = T.cache_of("bf16", pools, 2, 128)
        q = T.dev(T.narrow(np.random.default_rng(22).standard_normal((9, 8 * 128)), "bf16"))
        batch = b.upload()
        size = (kq.kq_attn_decode_workspace_bytes if decode else kq.kq_attn_prompt_workspace_bytes)(cache, batch, 8)
        fn = kq.kq_attn_decode if decode else kq.kq_attn_prompt
        got = []
        torch.cuda.synchronize()
        for i in range(3):
            stream = torch.cuda.Stream() if i == 2 else torch.cuda.current_stream()
            ws = U.empty_dev((size,), "uint8")
            ws.fill_(0xFF if i else 0)
            out = torch.zeros_like(q)
            torch.cuda.synchronize()
            fn("bf16", q, 1024, cache, batch, out, 1024, 8, 0.1, workspace=ws, workspace_bytes=size, stream=stream)
            got.append(T.host(out, "bf16"))
        assert np.array_equal(got[0], got[1]) and np.array_equal(got[0], got[2])


def test_page_past_4_gib():
    """Pages whose bytes lie past 4 GiB in both buffers, written, read back and attended to."""
    torch = U.torch_cuda()
    D, kv_heads = 128, 4
    nb = kq.kq_kv_page_bytes("f16", kv_heads, D)
    n_pages = (5 << 30) // nb
    k = torch.empty(n_pages * nb, dtype=torch.uint8, device="cuda")
    v = torch.empty(n_pages * nb, dtype=torch.uint8, device="cuda")
    k.fill_(0xFF)
    v.fill_(0xFF)
    rng = np.random.default_rng(23)
    b = T.Batch(24, [40], [40])
    x = T.narrow(rng.standard_normal((40, 3 * kv_heads * D)), "f16")
    xd, w, row = T.dev(x), kv_heads * D, 3 * kv_heads * D
    outs = []
    for ids in ([n_pages - 1, n_pages - 2], [0, 1]):
        b.table[0, :2] = ids
        b.dev = None
        cache, batch = kq.kq_kv_cache("f16", k, v, n_pages, kv_heads, D), b.upload()
        kq.kq_kv_append(cache, batch, None, "f16", xd[:, w:], row, xd[:, 2 * w:], row)
        kb, vb = T.dev(np.zeros((40, w), np.float16)), T.dev(np.zeros((40, w), np.float16))
        kq.kq_kv_read(cache, batch, "f16", kb, w, vb, w)
        assert np.array_equal(T.host(kb, "f16"), x[:, w:2 * w]) and np.array_equal(T.host(vb, "f16"), x[:, 2 * w:])
        for decode in (True, False):
            out = T.dev(np.zeros((40, w), np.float16))
            size = (kq.kq_attn_decode_workspace_bytes if decode else kq.kq_attn_prompt_workspace_bytes)(cache, batch, kv_heads)
            assert size == 0
            (kq.kq_attn_decode if decode else kq.kq_attn_prompt)("f16", xd, row, cache, batch, out, w, kv_heads, 0.09)
            outs.append(T.host(out, "f16"))
    assert np.array_equal(outs[0], outs[2]) and np.array_equal(outs[1], outs[3]) and np.isfinite(outs[0]).all()


def test_graph_follows_the_arrays():
    """A captured step (append, decode) replayed as the sequences grow: each replay equals the eager call."""
    torch = U.torch_cuda()
    rng = np.random.default_rng(25)
    heads, kv_heads, D = 8, 2, 128
    row = (heads + 2 * kv_heads) * D
    b = T.Batch(26, [1, 1, 1], [1500, 62, 400], width=60)
    pools, _ = T.random_cache(27, b, "q8_0", kv_heads, D)
    free = [p for p in range(b.n_pages) if p not in set(b.table[b.table >= 0].tolist())]
    b.table[1, 2:4] = free[:2]
    cache, keep = T.cache_of("q8_0", pools, kv_heads, D)
    batch = b.upload()
    f, m = kq.kq_rope_freqs("none", D, 1e4)
    rope = kq.kq_rope_spec(U.to_dev(f), D, 0, m)
    x = U.empty_dev((3, row))
    q, out = T.dev(np.zeros((3, heads * D), np.float16)), T.dev(np.zeros((3, heads * D), np.float16))
    size = kq.kq_attn_decode_workspace_bytes(cache, batch, heads)
    ws = U.empty_dev((size,), "uint8")

    def step():
        kq.kq_kv_append(cache, batch, rope, "f32", x[:, heads * D:], row, x[:, (heads + kv_heads) * D:], row, x, row, "f16", q,
                        heads * D, heads)
        kq.kq_attn_decode("f16", q, heads * D, cache, batch, out, heads * D, heads, D ** -0.5, workspace=ws, workspace_bytes=size)

    x.copy_(torch.from_numpy(rng.standard_normal((3, row)).astype(np.float32)))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(5):
        x.copy_(torch.from_numpy(rng.standard_normal((3, row)).astype(np.float32)))
        b.dev[2][1] += 1       # the second sequence grows into its next page
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = T.host(out, "f16").copy()
        out.zero_()
        step()
        assert np.array_equal(got, T.host(out, "f16")) and np.isfinite(got).all() and (got != 0).any()


def test_prompts_on_two_streams_and_in_a_graph():
    """Two prompt calls at once (their own workspaces) and a captured one, replayed: the bits of calls alone."""
    torch = U.torch_cuda()
    heads, kv_heads, D = 8, 1, 128
    b = T.Batch(50, [60, 3], [1500, 300])
    pools, _ = T.random_cache(51, b, "bf16", kv_heads, D)
    cache, keep = T.cache_of("bf16", pools, kv_heads, D)
    batch = b.upload()
    rng = np.random.default_rng(52)
    qs = [T.narrow(rng.standard_normal((b.T, heads * D)), "bf16") for _ in range(2)]
    size = kq.kq_attn_prompt_workspace_bytes(cache, batch, heads)
    assert size > 0
    qd, outs = [T.dev(q) for q in qs], [T.dev(np.zeros_like(q)) for q in qs]
    ws = [U.empty_dev((size,), "uint8") for _ in qs]

    def call(i):
        kq.kq_attn_prompt("bf16", qd[i], heads * D, cache, batch, outs[i], heads * D, heads, 0.1, 700, ws[i], size)

    alone = []
    for i in range(2):
        call(i)
        alone.append(T.host(outs[i], "bf16").copy())
        assert np.isfinite(A.widen(alone[i])).all() and (alone[i] != 0).any()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                call(i)
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(T.host(outs[i], "bf16"), alone[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        call(0)
    for rep in range(3):
        outs[0].zero_()
        if rep == 1:
            qd[0].copy_(qd[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(T.host(outs[0], "bf16"), alone[min(rep, 1)])


LARGE = [
    # enough columns for tiles of 256: new, lens, heads, kv_heads, D, window
    ([130], [130], 8, 1, 128, 0), ([300], [333], 4, 1, 160, 0), ([200, 150], [200, 700], 16, 2, 128, 0), ([140], [140], 8, 1, 256, 0),
    ([257], [300], 5, 1, 192, 0), ([150], [900], 8, 1, 224, 100), ([400], [400], 4, 1, 128, 33), ([128], [2200], 16, 1, 128, 0),
    ([160], [2150], 8, 1, 256, 1500),
]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window", LARGE)
def test_prompt_large_tiles(kind, new, lens, heads, kv_heads, D, window, capfd):
    """Tiles of 256 columns (two groups of waves a phase apart), whole and split."""
    with U.tuning({"log": "1"}):
        run(False, 30, new, lens, kind, kind, heads, kv_heads, D, window)
    assert "tile=256" in capfd.readouterr().err


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("new,lens,window,where", [([300], [300], 0, 290), ([300], [310], 0, 5), ([300], [300], 60, 100), ([280], [700], 200, 410)])
def test_not_finite_in_masked_places_of_large_tiles(kind, new, lens, window, where):
    change = poison(1, (0, where))
    change.kind[0] = kind
    run(False, 31, new, lens, kind, kind, 4, 1, 128, window, change=change)


def test_bad_pages_of_large_tiles():
    """A page id outside the cache in the middle, and a sequence longer than its table."""
    def change(b, pools, values):
        b.table[0, 3] = -1       # positions 96..127
    b = T.Batch(32, [300, 30], [300, 200])
    pools, values = T.random_cache(33, b, "bf16", 1, 128)
    b.table[0, 3] = -1
    b.width = 10
    b.table = np.ascontiguousarray(b.table[:, :10])
    b.lens[1] = 400              # 13 pages
    cache, keep = T.cache_of("bf16", pools, 1, 128)
    q = T.narrow(np.random.default_rng(34).standard_normal((330, 8 * 128)), "bf16")
    qd, od = T.dev(q), T.dev(np.zeros_like(q))
    batch = b.upload()
    size = kq.kq_attn_prompt_workspace_bytes(cache, batch, 8)
    ws = U.empty_dev((size + 16,), "uint8")
    kq.kq_attn_prompt("bf16", qd, 1024, cache, batch, od, 1024, 8, 0.1, workspace=ws, workspace_bytes=size)
    out = A.widen(T.host(od, "bf16"))
    nan = np.isnan(out)
    assert not nan[:96].any() and nan[96:].all()


def test_long_walks():
    """Walks of more steps than the lanes hold places for, whole and with a window."""
    for window in (0, 4500):
        run(False, 35, [130], [9000], "bf16", "bf16", 8, 1, 128, window)
        run(False, 36, [10], [9000], "f16", "q8_0", 2, 1, 64, window)
        run(True, 37, [2], [9000], "f16", "f16", 2, 1, 64, window)


WIDE = [
    # tiles of 32 columns: new, lens, heads, kv_heads, D, window, trees
    ([5], [60], 4, 1, 64, 0, False), ([5, 17, 1], [900, 17, 33], 8, 1, 64, 0, False), ([20], [700], 6, 2, 64, 130, False),
    ([9, 12], [200, 500], 4, 1, 32, 0, True), ([33], [2500], 2, 1, 64, 0, True),
]


@pytest.mark.parametrize("kind,cache_kind", BOTH)
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window,trees", WIDE)
def test_decode_wide_tiles(kind, cache_kind, new, lens, heads, kv_heads, D, window, trees, capfd):
    with U.tuning({"log": "1"}):
        run(True, 38, new, lens, kind, cache_kind, heads, kv_heads, D, window, trees, width=1 + 160000000 // (34 * D * 2 * kv_heads))
    err = capfd.readouterr().err
    assert "tile=32" in err and "k_attn_join" in err


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("new,lens,heads,kv_heads,D,window,trees", [([6], [300], 4, 1, 96, 0, False), ([18, 2], [90, 1000], 8, 2, 128, 50, False),
                                                                    ([10], [400], 5, 1, 256, 0, True), ([7], [200], 3, 1, 160, 0, False)])
def test_decode_wide_tiles_of_long_heads(kind, new, lens, heads, kv_heads, D, window, trees, capfd):
    with U.tuning({"log": "1"}):
        run(True, 39, new, lens, kind, kind, heads, kv_heads, D, window, trees, width=1 + 160000000 // (64 * D * 2 * kv_heads))
    assert "tile=32" in capfd.readouterr().err


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("new,lens,window,where", [([6], [40], 0, 36), ([6], [300], 0, 5), ([6], [300], 60, 100), ([9], [700], 200, 510)])
def test_not_finite_in_masked_places_of_wide_tiles(kind, new, lens, window, where):
    change = poison(1, (0, where))
    change.kind[0] = kind
    run(True, 40, new, lens, kind, kind, 4, 1, 128, window, width=10000, change=change)


def test_decode_variants(capfd):
    """Tiles of 16 unless the table's pages are many; a table of a few pages needs no join."""
    for new, lens, cache_kind, D, width, tile, join in (
            (1, 60, "f16", 64, 2, 16, False), (5, 60, "q8_0", 64, 4, 16, False), (5, 300, "f16", 64, 10, 16, True),
            (4, 300, "f16", 64, 20000, 16, True), (5, 300, "q8_0", 128, 20000, 16, True)):
        with U.tuning({"log": "1"}):
            run(True, 41, [new], [lens], "f16", cache_kind, 4, 1, D, width=width)
        err = capfd.readouterr().err
        assert f"tile={tile}" in err and ("k_attn_join" in err) == join


def test_a_layer_from_projection_to_projection():
    """q|k|v of a quantised product into the cache, attention, and the o projection, for a prompt and then
    decode steps: each stage against the oracle on the stage's own input."""
    torch = U.torch_cuda()
    from oracle import ref as R
    rng = np.random.default_rng(40)
    hidden, heads, kv_heads, D = 256, 8, 2, 64
    row = (heads + 2 * kv_heads) * D
    Wqkv, fq = U.quantize_both("affine4", (rng.standard_normal((row, hidden)) * 0.1).astype(np.float32))
    Wo, fo = U.quantize_both("q8_0", (rng.standard_normal((hidden, heads * D)) * 0.1).astype(np.float32))
    Wqkv, Wo = U.to_dev(Wqkv), U.to_dev(Wo)
    f, m = kq.kq_rope_freqs("yarn", D, 1e4, 4.0, 64)
    fd = U.to_dev(f)
    b = T.Batch(41, [20, 33], [20, 33], width=3)
    free = [p for p in range(b.n_pages) if p not in set(b.table[(b.table >= 0) & (b.table < b.n_pages)].tolist())]
    b.table[0, 1] = free[0]
    pools = [np.full((b.n_pages, kv_heads, 34 * D), 0xFF, np.uint8) for _ in range(2)]
    cache, (kd, vd) = T.cache_of("q8_0", pools, kv_heads, D)
    rope = kq.kq_rope_spec(fd, D, kq.KQ_ROPE_HALF, m)
    for step in range(4):
        if step:
            b.new = [1, 1]
            b.lens = [n + 1 for n in b.lens]
            b.q_start = np.array([0, 1, 2], np.int32)
            b.T = 2
            b.dev = None
        batch = b.upload()
        x = rng.standard_normal((b.T, hidden)).astype(np.float16)
        qkv = U.empty_dev((b.T, row))
        xd = U.to_dev(x)
        for t0 in range(0, b.T, kq.KQ_MAX_M):
            n = min(kq.KQ_MAX_M, b.T - t0)
            kq.kq_gemv("affine4", Wqkv, xd[t0:], qkv[t0:], row, hidden, n)
        q, out = T.dev(np.zeros((b.T, heads * D), np.float16)), T.dev(np.zeros((b.T, heads * D), np.float16))
        kq.kq_kv_append(cache, batch, rope, "f32", qkv[:, heads * D:], row, qkv[:, (heads + kv_heads) * D:], row, qkv, row, "f16", q,
                        heads * D, heads)
        decode = step > 0
        size = (kq.kq_attn_decode_workspace_bytes if decode else kq.kq_attn_prompt_workspace_bytes)(cache, batch, heads)
        ws = U.empty_dev((size + 16,), "uint8")
        (kq.kq_attn_decode if decode else kq.kq_attn_prompt)("f16", q, heads * D, cache, batch, out, heads * D, heads, D ** -0.5,
                                                             workspace=ws, workspace_bytes=size)
        y = U.empty_dev((b.T, hidden))
        kq.kq_gemv("q8_0", Wo, out, y, hidden, heads * D, b.T)

        hq = U.to_host(qkv)
        ref, bound = R.gemv("affine4", fq, x)
        U.assert_parity(hq, ref, bound, "q|k|v")
        for r, s, i, at in b.tokens():
            k = A.rope(hq[r, heads * D:(heads + kv_heads) * D].astype(np.float64).reshape(1, kv_heads, D), [at], f, m, False)[0]
            v = hq[r, (heads + kv_heads) * D:].astype(np.float64).reshape(kv_heads, D)
            for h in range(kv_heads):
                A.put(pools[0][b.table[s, at // 32], h], "q8_0", False, at % 32, k[h])
                A.put(pools[1][b.table[s, at // 32], h], "q8_0", True, at % 32, v[h])
        assert np.array_equal(U.to_host(kd), pools[0]) and np.array_equal(U.to_host(vd), pools[1])
        values = [[np.stack([np.concatenate([A.get(pool[p, h], "q8_0", w) for p in b.table[s, :-(-b.lens[s] // 32)]])[:b.lens[s]]
                             for h in range(kv_heads)], 1) for s in range(2)] for pool, w in zip(pools, (False, True))]
        q16, o16 = T.host(q, "f16"), T.host(out, "f16")
        want = T.attention(b, values, A.widen(q16).reshape(b.T, heads, D), heads, kv_heads, D, D ** -0.5, 0, None, "f16", TWO["q8_0"])
        T.check_rows(o16, want, b.T, o16, f"step {step}")
        ref, bound = R.gemv("q8_0", fo, o16)
        U.assert_parity(U.to_host(y), ref, bound, "o")
