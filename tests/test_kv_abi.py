"""What the rotary, cache and attention calls refuse, on the host before any HIP
call (the addresses are never dereferenced); the frequencies; the layout."""
import ctypes

import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import attn as A

ADDR = 0x10000   # aligned to everything
F32, F16, BF16 = kq.KQ_F32, kq.KQ_F16, kq.KQ_BF16
ARG, SHAPE, ALIGN = kq.KQ_ERR_ARG, kq.KQ_ERR_SHAPE, kq.KQ_ERR_ALIGN


def cache(type="f16", k=ADDR, v=ADDR, n_pages=9, kv_heads=2, head_dim=64, reserved=0):
    c = kq.kq_kv_cache(1, k, v, n_pages, kv_heads, head_dim)
    c.type, c.reserved = kq._kv_type(type), reserved
    return c


def batch(table=ADDR, width=4, q_start=ADDR, lens=ADDR, n_seqs=2, n_tokens=5):
    return kq.kq_kv_batch(table, width, q_start, lens, n_seqs, n_tokens)


def rope(freqs=ADDR, rot=32, pairs=0, m=1.0, positions=ADDR):
    return kq.kq_rope_spec(freqs, rot, pairs, m, positions)


def refuse(fn, cases, empty=()):
    for change, want in cases:
        assert fn(**change) == want, (change, want, fn(**change))
        assert kq.last_error(), change
    for change in empty:
        assert fn(**change) == kq.KQ_OK, (change, kq.last_error())


def at(s):
    return None if s is None else ctypes.addressof(s)


BAD_CACHE = [({"c": cache(type=0)}, ARG), ({"c": cache(type=3)}, ARG), ({"c": cache(kv_heads=0)}, ARG),
             ({"c": cache(kv_heads=kq.KQ_MAX_HEADS + 1)}, ARG), ({"c": cache(head_dim=0)}, SHAPE),
             ({"c": cache(head_dim=80)}, SHAPE), ({"c": cache(head_dim=288)}, SHAPE), ({"c": cache(head_dim=-32)}, SHAPE),
             ({"c": cache(reserved=1)}, ARG), ({"c": cache(n_pages=0)}, ARG), ({"c": cache(n_pages=1 << 31)}, ARG),
             ({"c": None}, ARG), ({"b": None}, ARG), ({"b": batch(n_seqs=-1)}, ARG),
             ({"b": batch(n_seqs=kq.KQ_MAX_SEQS + 1)}, ARG), ({"b": batch(n_tokens=-1)}, ARG),
             ({"b": batch(n_tokens=kq.KQ_MAX_TOKENS + 1)}, ARG), ({"b": batch(width=0)}, ARG),
             ({"b": batch(width=1 << 26)}, ARG)]
BAD_POINTERS = [({"c": cache(k=None)}, ARG), ({"c": cache(v=None)}, ARG), ({"c": cache(k=ADDR + 8)}, ALIGN),
                ({"c": cache(v=ADDR + 4)}, ALIGN), ({"b": batch(table=None)}, ARG), ({"b": batch(q_start=None)}, ARG),
                ({"b": batch(lens=None)}, ARG), ({"b": batch(table=ADDR + 2)}, ALIGN),
                ({"b": batch(q_start=ADDR + 1)}, ALIGN), ({"b": batch(lens=ADDR + 2)}, ALIGN)]
EMPTY = [{"b": batch(n_tokens=0)}, {"b": batch(n_seqs=0)}, {"b": batch(None, 4, None, None, 2, 0), "c": cache(k=None, v=None)}]


def bad_rows(key, ld, type_size):
    return [({key: None}, ARG), ({ld: 127}, ARG), ({ld: (1 << 35) + 1}, ARG), ({key: ADDR + type_size // 2}, ALIGN)]


def test_rope_refusals():
    def fn(r=rope(), xtype=F16, x=ADDR, ldx=128, otype=F32, out=ADDR + 4096, ldo=128, T=3, heads=2, D=64):
        return kq.lib().kq_rope(at(r), xtype, x, ldx, otype, out, ldo, T, heads, D, None)
    refuse(fn, [({"r": None}, ARG), ({"r": rope(freqs=None)}, ARG), ({"r": rope(positions=None)}, ARG),
                ({"r": rope(rot=0)}, SHAPE), ({"r": rope(rot=31)}, SHAPE), ({"r": rope(rot=66)}, SHAPE),
                ({"r": rope(pairs=2)}, ARG), ({"r": rope(m=float("nan"))}, ARG), ({"r": rope(m=float("inf"))}, ARG),
                ({"r": rope(freqs=ADDR + 4)}, ALIGN), ({"r": rope(positions=ADDR + 2)}, ALIGN), ({"xtype": 3}, ARG),
                ({"otype": -1}, ARG), ({"T": -1}, ARG), ({"T": kq.KQ_MAX_TOKENS + 1}, ARG), ({"heads": 0}, ARG),
                ({"heads": kq.KQ_MAX_HEADS + 1}, ARG), ({"D": 48}, SHAPE), ({"D": 0}, SHAPE), ({"D": 512}, SHAPE),
                ({"out": ADDR}, ARG), ({"out": ADDR, "otype": F16, "ldo": 256}, ARG)]
           + bad_rows("x", "ldx", 2) + bad_rows("out", "ldo", 4), [{"T": 0}, {"T": 0, "x": None, "out": None}])


def test_append_refusals():
    def fn(c=cache(), b=batch(), r=rope(positions=None), xtype=F32, k=ADDR, ldk=128, v=ADDR, ldv=128, q=ADDR, ldq=128, otype=F16,
           q_out=ADDR + 4096, ldo=128, heads=2):
        return kq.lib().kq_kv_append(at(c), at(b), at(r), xtype, k, ldk, v, ldv, q, ldq, otype, q_out, ldo, heads, None)
    refuse(fn, BAD_CACHE + BAD_POINTERS + bad_rows("k", "ldk", 4) + bad_rows("v", "ldv", 4) + bad_rows("q_out", "ldo", 2)
           + bad_rows("q", "ldq", 4)[1:] + [
               ({"xtype": 4}, ARG), ({"otype": 3}, ARG), ({"heads": 0}, ARG), ({"heads": kq.KQ_MAX_HEADS + 1}, ARG),
               ({"r": rope(freqs=None)}, ARG), ({"r": rope(rot=80)}, SHAPE), ({"r": rope(positions=ADDR + 1)}, ALIGN),
               ({"q_out": ADDR}, ARG)],
           EMPTY + [{"b": batch(n_tokens=0), "q": None, "heads": 0, "otype": 9}])


def test_read_refusals():
    def fn(c=cache(), b=batch(), otype=F32, k=ADDR, ldk=128, v=ADDR, ldv=128):
        return kq.lib().kq_kv_read(at(c), at(b), otype, k, ldk, v, ldv, None)
    refuse(fn, BAD_CACHE + BAD_POINTERS + bad_rows("k", "ldk", 4) + bad_rows("v", "ldv", 4) + [({"otype": 3}, ARG)], EMPTY)


ATTN = [({"type": F32}, ARG), ({"type": 3}, ARG), ({"type": BF16}, ARG), ({"c": cache("bf16")}, ARG), ({"heads": 0}, ARG),
        ({"heads": 3}, SHAPE), ({"heads": 2 * kq.KQ_MAX_HEADS}, ARG), ({"scale": 0.0}, ARG), ({"scale": -1.0}, ARG),
        ({"scale": float("nan")}, ARG), ({"scale": float("inf")}, ARG), ({"scale": 3e38}, ARG), ({"window": -1}, ARG),
        ({"window": kq.KQ_MAX_WINDOW + 1}, ARG)] + bad_rows("q", "ldq", 2) + bad_rows("out", "ldo", 2)


def test_decode_refusals():
    wide = batch(width=1000)
    need = kq.kq_attn_decode_workspace_bytes(cache(), wide, 2)
    assert need > 0

    def fn(c=cache(), b=wide, type=F16, q=ADDR, ldq=128, out=ADDR, ldo=128, heads=2, scale=1.0, window=0, tree=None, ws=ADDR,
           wsb=need):
        return kq.lib().kq_attn_decode(type, q, ldq, at(c), at(b), out, ldo, heads, scale, window, tree, ws, wsb, None)
    refuse(fn, BAD_CACHE + BAD_POINTERS + ATTN + [
        ({"b": batch(n_tokens=65)}, ARG), ({"b": batch(n_seqs=65)}, ARG), ({"tree": ADDR + 4}, ALIGN), ({"ws": None}, ARG),
        ({"wsb": need - 1}, ARG), ({"wsb": -1}, ARG), ({"ws": ADDR + 8}, ALIGN)], EMPTY)


def test_prompt_refusals():
    wide = batch(width=5000)
    need = kq.kq_attn_prompt_workspace_bytes(cache(), wide, 2)
    assert need > 0

    def fn(c=cache(), b=wide, type=F16, q=ADDR, ldq=128, out=ADDR, ldo=128, heads=2, scale=1.0, window=0, ws=ADDR, wsb=need):
        return kq.lib().kq_attn_prompt(type, q, ldq, at(c), at(b), out, ldo, heads, scale, window, ws, wsb, None)
    refuse(fn, BAD_CACHE + BAD_POINTERS + ATTN + [({"ws": None}, ARG), ({"wsb": need - 1}, ARG), ({"ws": ADDR + 8}, ALIGN)], EMPTY)


def test_workspace_sizes():
    """Nothing where a table row is one short chunk; the errors of an invalid shape."""
    for fn in (kq.kq_attn_decode_workspace_bytes, kq.kq_attn_prompt_workspace_bytes):
        assert fn(cache(), batch(width=1), 2) == 0
        assert fn(cache(k=None, v=None), batch(None, 9999, None, None, 2, 5), 2) > 0
        assert fn(cache(), batch(width=9999, n_tokens=0), 2) == 0
        for bad in ((cache(head_dim=40), batch(), 2), (cache(), batch(), 3), (cache(), batch(width=0), 2)):
            with pytest.raises(kq.KQError):
                fn(*bad)


def test_page_bytes():
    assert kq.kq_kv_page_bytes("f16", 8, 128) == 8 * 128 * 32 * 2
    assert kq.kq_kv_page_bytes("bf16", 1, 32) == 2048
    assert kq.kq_kv_page_bytes("q8_0", 8, 128) == 8 * 32 * (128 // 32) * kq.kq_block_bytes("q8_0")
    L = kq.lib()
    assert L.kq_kv_page_bytes(0, 8, 128) == ARG and L.kq_kv_page_bytes(1, 0, 128) == ARG
    assert L.kq_kv_page_bytes(1, 8, 100) == SHAPE


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot,base,factor", [(2, 1e4, 2.0), (64, 1e4, 8.0), (128, 1e6, 4.0), (256, 5e5, 0.5)])
def test_freqs(scaling, rot, base, factor):
    f, m = kq.kq_rope_freqs(scaling, rot, base, factor, 4096)
    want, wm = A.freqs(scaling, rot, base, factor, 4096)
    assert f.shape == (rot // 2,) and np.allclose(f, want, rtol=1e-13, atol=0) and abs(m - wm) < 1e-15


def test_freqs_by_hand():
    f, m = kq.kq_rope_freqs("none", 4, 100.0)
    assert f[0] == 1.0 and abs(f[1] - 0.1) < 1e-16 and m == 1.0
    f, m = kq.kq_rope_freqs("ntk", 4, 100.0, 4.0)            # base 100 * 4^2
    assert abs(f[1] - 1 / 40) < 1e-16 and m == 1.0
    f, m = kq.kq_rope_freqs("linear", 4, 100.0, 10.0)
    assert f[0] == 0.1 and m == 1.0
    # turns over 100 positions: 15.9 of the first pair (halfway between 1 and 30.8), 0.159 of the second
    f, m = kq.kq_rope_freqs("yarn", 4, 1e4, 10.0, 100, 2 * 100 / (2 * np.pi) - 1.0, 1.0)
    assert abs(f[0] - 0.55) < 1e-15 and abs(f[1] - 0.001) < 1e-17 and abs(m - (0.1 * np.log(10.0) + 1)) < 1e-15


def test_freqs_refusals():
    out, m = np.empty(128), ctypes.c_double()
    args = dict(scaling=0, rot=64, base=1e4, factor=1.0, n=0, fast=32.0, slow=1.0, out=out.ctypes.data, m=ctypes.addressof(m))

    def fn(**change):
        a = {**args, **change}
        return kq.lib().kq_rope_freqs(*a.values())
    refuse(fn, [({"rot": 0}, SHAPE), ({"rot": 3}, SHAPE), ({"rot": 258}, SHAPE), ({"scaling": 4}, ARG), ({"scaling": -1}, ARG),
                ({"base": 0.0}, ARG), ({"base": float("inf")}, ARG), ({"factor": 0.0}, ARG), ({"factor": float("nan")}, ARG),
                ({"out": None}, ARG), ({"m": None}, ARG), ({"scaling": 3}, ARG), ({"scaling": 3, "n": 8, "fast": 1.0}, ARG)],
           [{}, {"scaling": 3, "n": 8}])


def test_names():
    assert kq.KV_TYPES == {"f16": 1, "bf16": 2, "q8_0": 8}
    with pytest.raises(KeyError):
        kq.kq_kv_page_bytes("f32", 1, 32)


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
@pytest.mark.parametrize("D", [32, 96, 256])
def test_layout_is_one_to_one(kind, D):
    p, d = np.meshgrid(np.arange(32), np.arange(D), indexing="ij")
    for is_v in (False, True):
        assert np.array_equal(np.sort(A.place(kind, is_v, p, d).ravel()), np.arange(32 * D))
