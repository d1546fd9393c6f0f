"""The rotary, cache and attention calls at the most rows, the most sequences and far positions:
sampled rows against 64-bit results from the same stored values."""
import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import attn as A
from tests import attn_util as T
from tests import gpu_util as U
from tests.test_gpu_attn_range import LOST, ONE, TWO

pytestmark = pytest.mark.gpu


def setup(new, lens, kind, cache_kind, heads, kv_heads, D, spare=1):
    """Rows of normal values, and a cache that is filled by kq_kv_append with all of each sequence's positions."""
    torch = U.torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(80)
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[kind]
    S, L = len(new), sum(lens)
    counts = [-(-n // A.PAGE) for n in lens]
    n_pages, width = sum(counts) + spare, max(counts)
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor(np.cumsum([0] + counts[:-1]), device="cuda")
    table = ids[(first[:, None] + torch.arange(width, device="cuda")).clamp(max=n_pages - 1)].contiguous()
    starts = torch.tensor(np.cumsum([0] + list(new)), dtype=torch.int32, device="cuda")
    all_starts = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda")
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nb = kq.kq_kv_page_bytes(cache_kind, kv_heads, D)
    pools = [torch.full((n_pages * nb,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = kq.kq_kv_cache(cache_kind, *pools, n_pages, kv_heads, D)
    w = kv_heads * D
    k, v = (torch.randn(L, w, generator=g, device="cuda").to(dt) for _ in range(2))
    for at in range(0, L, kq.KQ_MAX_TOKENS):   # a part of one sequence, or all of them
        n = min(kq.KQ_MAX_TOKENS, L - at)
        if n == L:
            kq.kq_kv_append(cache, kq.kq_kv_batch(table, width, all_starts, ld, S, L), None, kind, k, w, v, w)
        else:
            assert S == 1
            part, upto = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([at + n], dtype=torch.int32, device="cuda")
            kq.kq_kv_append(cache, kq.kq_kv_batch(table, width, part, upto, 1, n), None, kind, k[at:], w, v[at:], w)
    q = torch.randn(sum(new), heads * D, generator=g, device="cuda").to(dt)
    return cache, kq.kq_kv_batch(table, width, starts, ld, S, sum(new)), q, k, v


def attend_and_check(decode, new, lens, kind, cache_kind, heads, kv_heads, D, window, rows):
    torch = U.torch_cuda()
    cache, batch, q, k, v = setup(new, lens, kind, cache_kind, heads, kv_heads, D)
    out = torch.full_like(q, float("nan"))
    size = (kq.kq_attn_decode_workspace_bytes if decode else kq.kq_attn_prompt_workspace_bytes)(cache, batch, heads)
    ws = torch.empty(size + 16, dtype=torch.uint8, device="cuda")
    print("attn", decode, new[:3], lens[:3], kind, cache_kind, size, flush=True)
    scale = D ** -0.5
    (kq.kq_attn_decode if decode else kq.kq_attn_prompt)(kind, q, heads * D, cache, batch, out, heads * D, heads, scale, window,
                                                         workspace=ws, workspace_bytes=size)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    starts, first = np.cumsum([0] + list(new)), np.cumsum([0] + list(lens))
    step = TWO["q8_0" if cache_kind == "q8_0" else kind] if decode or cache_kind == "q8_0" else ONE[kind]
    for row in rows:
        s = int(np.searchsorted(starts, row, side="right")) - 1
        at = lens[s] - new[s] + int(row - starts[s])
        lo = max(at - window + 1, 0) if window else 0
        n = at + 1 - lo
        for h in {(row * 7) % heads}:
            kh = slice(h // (heads // kv_heads) * D, (h // (heads // kv_heads) + 1) * D)
            kk, vv = (x[first[s] + lo:first[s] + at + 1, kh].double().cpu().numpy() for x in (k, v))
            if cache_kind == "q8_0":
                kk, vv = ((lambda c, d: c.astype(np.float64) * np.repeat(d.astype(np.float64), 32, -1))(*A.q8_blocks(A.narrow(x, "f32"))) for x in (kk, vv))
            y = out[row, h * D:(h + 1) * D].double().cpu().numpy()
            want, mass, _, unit, spread = A.attend(q[row, h * D:(h + 1) * D].double().cpu().numpy(), kk, vv, float(np.float32(scale)), np.ones(n, bool))
            # sums of a chain: one per 32 keys of a wave's pages, and the chunks' join
            tol = A.attention_tolerance(want, mass, unit, spread, n // 32 + 1024, kind, step, LOST if cache_kind != "q8_0" else 2.0 ** -25)
            assert (np.abs(y - want) <= tol).all(), (row, h, float(np.abs(y - want).max()), float(tol.min()))


@pytest.mark.parametrize("kind,cache_kind", [("f16", "f16"), ("bf16", "bf16"), ("f16", "q8_0")])
def test_decode_far_away(kind, cache_kind):
    """New tokens behind three million positions, all of them or a window seen."""
    attend_and_check(True, [3], [3000017], kind, cache_kind, 2, 1, 32, 0, [0, 2])
    attend_and_check(True, [1], [3000017], kind, cache_kind, 2, 1, 32, 2000003, [0])


@pytest.mark.parametrize("kind,cache_kind,window", [("bf16", "bf16", 0), ("f16", "q8_0", 5000)])
def test_prompt_of_the_most_tokens(kind, cache_kind, window):
    n = kq.KQ_MAX_TOKENS
    attend_and_check(False, [n], [n], kind, cache_kind, 1, 1, 32, window, [0, 1, 31, 32, 100, 4097, n // 2 + 3, n - 129, n - 2, n - 1])


def test_prompts_of_the_most_sequences_and_tokens():
    new = [256 + (7 * s) % 31 - 15 for s in range(4096)]
    new[-1] += kq.KQ_MAX_TOKENS - sum(new)
    starts = np.cumsum([0] + new)
    rows = [0, 5, kq.KQ_MAX_TOKENS - 1] + [int(starts[s]) + d for s in (1, 63, 64, 65, 2047, 4000, 4095) for d in (-1, 0, 1, 40, 200)]
    attend_and_check(False, new, new, "f16", "f16", 2, 1, 32, 0, rows)
    attend_and_check(False, new, new, "bf16", "q8_0", 2, 2, 32, 50, rows)


def test_rotation_of_the_most_tokens():
    torch = U.torch_cuda()
    n, D = kq.KQ_MAX_TOKENS, 32
    f, m = kq.kq_rope_freqs("none", D, 1e4)
    x = torch.randn(n, D, generator=torch.Generator(device="cuda").manual_seed(81), device="cuda").half()
    positions = torch.arange(2 ** 31 - n, 2 ** 31, dtype=torch.int64, device="cuda").to(torch.int32)
    y = torch.zeros_like(x)
    kq.kq_rope(kq.kq_rope_spec(U.to_dev(f), D, kq.KQ_ROPE_HALF, m, positions), "f16", x, D, "f16", y, D, n, 1, D)
    rows = [0, 1, 7, 8, n // 2, n - 9, n - 8, n - 1]
    got, xs = y[rows].cpu().numpy().astype(np.float64), x[rows].cpu().numpy().astype(np.float64)
    want = A.rope(xs[:, None], [2 ** 31 - n + r for r in rows], f, m, False)[:, 0]
    # the angle is rounded to 64 bits (2^31 * 2^-53, relative 2^-22 of a radian) in both, then half a step
    assert (np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -20 * np.abs(xs).max() + 2.0 ** -25).all()
