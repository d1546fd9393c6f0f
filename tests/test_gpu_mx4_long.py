"""Conversions of matrices that one grid, or 32-bit offsets, do not reach."""
import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import mx4 as X
from tests import gpu_util as U
from tests.test_gpu_mx4 import activations, as_type

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
