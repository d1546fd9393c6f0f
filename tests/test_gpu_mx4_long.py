"""Conversions of matrices that one grid, or 32-bit offsets, do not reach."""
import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import mx4 as X
from tests import gpu_util as U
from tests.test_gpu_mx4 import activations, as_type, check, dev, random_planes, upload

pytestmark = pytest.mark.gpu


def test_more_than_2_to_35_contiguous_elements():
    """2^23 + 3 rows of 4096: every row is 1.5 but those around powers of two and the last, which are random."""
    t = U.torch_cuda()
    K, R = 4096, (1 << 23) + 3
    rng = np.random.default_rng(71)
    rows = np.unique(np.concatenate([[0, 1], *[np.arange(p - 2, p + 2) for p in (1 << 20, 1 << 21, 1 << 22, 3 << 21)],
                                     np.arange((1 << 23) - 2, R)]))
    xs = as_type(activations(rng, rows.size, K), "bf16")
    c, s = X.quantize(xs)
    at = t.from_numpy(rows).to("cuda")
    x = t.full((R, K), 1.5, dtype=t.bfloat16, device="cuda")
    x[at] = t.from_numpy(xs.view(np.int16)).to("cuda").view(t.bfloat16)
    codes, scales = t.zeros((R, K // 2), dtype=t.uint8, device="cuda"), t.zeros((R, K // 32), dtype=t.uint8, device="cuda")
    kq.kq_mx4_quantize("bf16", x, K, codes, scales, R, K)
    pc, ps = X.planes(c, s)
    assert np.array_equal(codes[at].cpu().numpy(), pc) and np.array_equal(scales[at].cpu().numpy(), ps)
    x.zero_()
    kq.kq_mx4_dequantize(codes, scales, "bf16", x, K, R, K)
    assert np.array_equal(x[at].float().cpu().numpy().astype(np.float64), X.dequantize(c, s))
    x[at], codes[at], scales[at] = 1.5, 0x77, 125   # 1.5 is 6 times 2^-2
    for i in range(0, R, 1 << 20):
        part = slice(i, min(R, i + (1 << 20)))
        assert bool((codes[part] == 0x77).all()) and bool((scales[part] == 125).all()) and bool((x[part] == 1.5).all()), i


@pytest.mark.parametrize("kind", ("f32", "bf16"))
def test_rows_that_lie_far_apart(kind):
    """Twenty rows 2^27 + 1 elements apart, past 4 GiB in bytes; what lies between them stays."""
    t = U.torch_cuda()
    R, K, ld = 20, 96, (1 << 27) + 1
    rng = np.random.default_rng(72)
    xs = as_type(activations(rng, R, K), kind)
    dtype = t.float32 if kind == "f32" else t.bfloat16
    flat = t.zeros((R - 1) * ld + K, dtype=dtype, device="cuda")
    view = flat.as_strided((R, K), (ld, 1))
    view.copy_(t.from_numpy(xs if kind == "f32" else xs.view(np.int16)).to("cuda").view(dtype))
    codes, scales = U.empty_dev((R, K // 2), "uint8"), U.empty_dev((R, K // 32), "uint8")
    kq.kq_mx4_quantize(kind, flat, ld, codes, scales, R, K)
    c, s = X.quantize(xs)
    pc, ps = X.planes(c, s)
    assert np.array_equal(U.to_host(codes), pc) and np.array_equal(U.to_host(scales), ps)
    view.zero_()
    kq.kq_mx4_dequantize(codes, scales, kind, flat, ld, R, K)
    assert np.array_equal(view.float().cpu().numpy().astype(np.float64), X.dequantize(c, s))
    view.zero_()
    assert not bool(flat.any())


def test_outputs_past_32_bit_offsets():
    """Products of the most rows: 2^31 outputs of 64 columns and 2^25 rows of activations times 72 weights."""
    t = U.torch_cuda()
    N, K, M = kq.KQ_MX4_MAX_ROWS, 32, 64
    rng = np.random.default_rng(73)
    c, s = random_planes(rng, 50, K)
    bc, bs = X.planes(c, s)
    at = t.from_numpy(np.concatenate([np.arange(3), N // 2 + np.arange(-4, 5), N - 38 + np.arange(38)])).to("cuda")
    codes, scales = t.zeros((N, K // 2), dtype=t.uint8, device="cuda"), t.full((N, K // 32), 127, dtype=t.uint8, device="cuda")
    codes[at], scales[at] = t.from_numpy(bc).to("cuda"), t.from_numpy(bs).to("cuda")
    w = X.dequantize(c, s)
    for kind in ("bf16", "f32"):
        x = as_type(activations(rng, M, K), kind)
        y = t.full((M, N), float("nan"), device="cuda")
        kq.kq_mx4_gemv(codes, scales, kind, dev(x), y, N, K, M)
        check(y[:, at].cpu().numpy(), *X.product(w, X.widen(x)), K, what=kind)
        y[:, at] = 0.0
        assert all(not bool(row.any()) for row in y)   # a NaN counts
        del y
    # the same planes as the activations of a product of two matrices
    n = 72
    wc, ws = random_planes(rng, n, K)
    pw = upload(wc, ws)
    y = t.full((N, n), float("nan"), dtype=t.bfloat16, device="cuda")
    kq.kq_mx4_gemm(codes, scales, pw[0].ptr, pw[1].ptr, "bf16", y, N, n, K)
    check(y[at].view(t.int16).cpu().numpy().view(np.uint16), *X.product(X.dequantize(wc, ws), w), K, "bf16")
    y[at] = 0.0
    assert not any(bool(part.any()) for part in y.split(1 << 22))


@pytest.mark.parametrize("M", (1, 3))
def test_experts_past_32_bit_offsets(M):
    """1024 experts of 4160 x 2080: every plane of codes passes 4 GiB, and the chosen experts are the last ones and some
    on both sides of 4 GiB; the others' scales are NaN."""
    t = U.torch_cuda()
    E, H, inter, top_k = 1024, 2080, 4160, 4
    used = [0, 991, 992, 1023]   # 4.33 MB an expert: 4 GiB lies in expert 992
    rng = np.random.default_rng((74, M))
    planes, host = [], []
    for n, k in ((inter, H), (inter, H), (H, inter)):
        codes = t.zeros((E, n, k // 2), dtype=t.uint8, device="cuda")
        scales = t.full((E, n, k // 32), 255, dtype=t.uint8, device="cuda")
        values = np.zeros((len(used), n, k))
        for i, e in enumerate(used):
            c, s = random_planes(rng, n, k, 119, 123)
            bc, bs = X.planes(c, s)
            codes[e], scales[e] = t.from_numpy(bc).to("cuda"), t.from_numpy(bs).to("cuda")
            values[i] = X.dequantize(c, s)
        planes += [codes, scales]
        host.append(values)
    assert planes[0].numel() > 1 << 32 and inter * H // 2 * 991 < 1 << 32 < inter * H // 2 * 993
    W = np.full((E, H), -0.01, np.float32)
    for i, e in enumerate(used):
        W[e] = 0.001 * (i + 1)
    x = as_type(np.abs(rng.standard_normal((M, H))) + 0.1, "bf16")
    y, ids, wts = U.empty_dev((M, H)), U.empty_dev((M, top_k), "int32"), U.empty_dev((M, top_k))
    nb = kq.kq_mx4_moe_layer_workspace_bytes(H, inter, M, top_k, E)
    ws = U.empty_dev((nb,), "uint8")
    kq.kq_mx4_moe_layer("bf16", dev(x), "f32", dev(W), *planes, y, ids, wts, H, inter, M, top_k, E, True, ws, nb)
    got = U.to_host(ids)
    assert (got == used[::-1]).all()
    ref, bound = X.moe_layer(X.widen(x), *host, np.searchsorted(used, got), U.to_host(wts).astype(np.float64))
    assert (np.abs(U.to_host(y) - ref) <= bound).all()
