"""Which kernels the microscaled calls run where: the shapes here reach every
variant (a shape of another group that moves to another kernel shows here), and
each result is compared with the oracle under the bounds of
tests/test_gpu_mx4.py. The rules ask for the number of compute units; the table
is for the 256 of an MI355X."""
import re

import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import mx4 as X
from tests import gpu_util as U
from tests.test_gpu_mx4 import Layer, activations, as_type, check, dev, random_planes, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def whole_card():
    n = U.torch_cuda().cuda.get_device_properties(0).multi_processor_count
    if n != 256:
        pytest.skip(f"{n} compute units")


def launches(capfd, call):
    """[(kernel, its log line)] of the call."""
    capfd.readouterr()
    with U.tuning({"log": "1"}):
        call()
        U.torch_cuda().cuda.synchronize()
    return [(m[1], m[0]) for m in re.finditer(r"kq: (\S+) .*", capfd.readouterr().err)]


GEMV = [  # N, K, M, types, column tiles, row tiles, chunks
    (100, 160, 8, ("f16", "bf16"), 1, 1, 4), (100, 256, 1, ("f16", "bf16"), 1, 1, 4),
    (6129, 2400, 9, ("f16", "bf16"), 1, 2, 2), (6144, 2048, 16, ("f16", "bf16"), 1, 2, 2),
    (6144, 2048, 13, ("f16", "bf16"), 1, 2, 2), (6144, 2048, 12, ("f16", "bf16"), 1, 1, 2),   # two workgroups of one tile fit
    (6128, 2048, 16, ("f16", "bf16"), 1, 1, 2), (6144, 2016, 9, ("f16", "bf16"), 1, 1, 2), (19456, 2048, 9, ("f16", "bf16"), 1, 1, 2),
    (1000, 160, 64, ("f16", "bf16"), 1, 1, 2),
    (1801, 160, 32, ("f16", "bf16"), 1, 1, 2), (2064, 160, 32, ("f16", "bf16"), 2, 1, 1), (1500, 256, 49, ("f16", "bf16"), 2, 1, 1),
    (8192, 160, 17, ("f16", "bf16"), 2, 2, 1), (8200, 128, 32, ("f16", "bf16"), 2, 2, 1),
    (4000, 128, 48, ("f16", "bf16"), 3, 1, 1), (4000, 96, 33, ("f16", "bf16"), 3, 1, 1),
    (8192, 128, 48, ("f16", "bf16"), 3, 2, 1), (8209, 96, 40, ("f16", "bf16"), 3, 2, 1),
    (4000, 128, 64, ("f16", "bf16"), 4, 1, 1), (4000, 96, 49, ("f16", "bf16"), 4, 1, 1),
    (8192, 128, 64, ("f16", "bf16"), 4, 2, 1), (8209, 96, 50, ("f16", "bf16"), 4, 2, 1),
    (1000, 160, 64, ("f32",), 1, 1, 1), (6128, 128, 16, ("f32",), 1, 1, 1), (6144, 160, 1, ("f32",), 1, 2, 1),
    (3100, 128, 32, ("f32",), 1, 2, 1), (12288, 128, 1, ("f32",), 1, 4, 1), (3201, 288, 64, ("f32",), 1, 4, 1),
]


@pytest.mark.parametrize("N,K,M,kind,ct,rt,u", [(n, k, m, t, *c) for n, k, m, ts, *c in GEMV for t in ts])
def test_gemv(capfd, N, K, M, kind, ct, rt, u):
    rng = np.random.default_rng((N, K, M, 21))
    codes, scales = random_planes(rng, N, K)
    pc, ps = upload(codes, scales)
    x = as_type(activations(rng, M, K), kind)
    xd, y = dev(x), U.empty_dev((M, N))
    (name, line), = launches(capfd, lambda: kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, xd, y, N, K, M))
    assert name == "k_mx4_gemv" and line.endswith(f"ct={ct} rt={rt} u={u}"), line
    check(U.to_host(y), *X.product(X.dequantize(codes, scales), X.widen(x)), K, what=line)


@pytest.mark.parametrize("M,N,K,tile", [(4096, 2048, 96, "160x256"), (2049, 4000, 160, "160x256"),
                                        (2048, 2560, 128, "192x128"), (1900, 2561, 160, "192x128"),
                                        (4096, 12032, 128, "256x256"), (4100, 12000, 96, "256x256"),
                                        (300, 6144, 256, "64x64"), (513, 999, 96, "64x64"), (40, 300, 768, "64x64"),
                                        (40, 300, 800, None), (512, 512, 1024, None), (1, 1, 896, None), (513, 512, 1024, "64x64")])
@pytest.mark.parametrize("kind", ("f32", "bf16"))
def test_gemm(capfd, M, N, K, tile, kind):
    t = U.torch_cuda()
    rng = np.random.default_rng((M, N, K, 22))
    a, w = random_planes(rng, M, K, 127, 128), random_planes(rng, N, K, 127, 128)   # exact sums: multiples of 1/4
    pa, pw = upload(*a), upload(*w)
    y = t.full((M, N), float("nan"), dtype=t.float32 if kind == "f32" else t.bfloat16, device="cuda")
    (name, line), = launches(capfd, lambda: kq.kq_mx4_gemm(pa[0].ptr, pa[1].ptr, pw[0].ptr, pw[1].ptr, kind, y, M, N, K))
    assert (name == "k_mx4_gemm_small") if tile is None else (name == "k_mx4_gemm" and line.endswith("tile=" + tile)), line
    av, wv = (t.from_numpy(X.dequantize(*p).astype(np.float32)).to("cuda").double() for p in (a, w))
    assert t.equal(y, (av @ wv.T.contiguous()).to(y.dtype))


LAYER = [  # M, E, hidden, inter, top_k, (gate and up's tiles, columns in 16 bits), choice in that kernel, parts of the down projection
    (1, 8, 64, 32, 2, 1, 4, True, 1), (1, 512, 64, 32, 8, 1, 4, True, 1),
    (1, 513, 64, 32, 8, 1, 4, False, 1), (1, 64, 64, 256, 64, 2, 4, False, 1),
    (2, 300, 2048, 64, 3, 1, 4, False, 1), (7, 9, 1056, 32, 9, 1, 8, False, 1), (8, 9, 1056, 32, 9, 1, 8, False, 7),
    (16, 16, 128, 1056, 8, 2, 8, False, 16), (40, 256, 160, 64, 4, 1, 4, False, 16), (40, 256, 160, 128, 8, 2, 4, False, 16),
    (3, 6, 64, 32, 2, 1, 4, False, 1), (16, 4, 1024, 64, 2, 1, 8, False, 8),
]


@pytest.mark.parametrize("kind", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("M,E,H,inter,top_k,tiles,cols,chooses,parts", LAYER)
def test_layer(capfd, kind, M, E, H, inter, top_k, tiles, cols, chooses, parts):
    rng = np.random.default_rng((M, E, H, 23))
    L = Layer(rng, E, H, inter)
    x, W = as_type(activations(rng, M, H), kind), as_type(rng.standard_normal((E, H)) * H ** -0.5, kind)
    got = []
    seen = launches(capfd, lambda: got.append(L.run(x, kind, W, kind, top_k, True)))
    names = [n for n, _ in seen]
    assert names == ["k_route_logits"] + ["k_route_select"] * (not chooses) + ["k_mx4_gate_up", "k_mx4_down"] + ["k_mx4_down_sum"] * (parts > 1), names
    line = dict(seen)
    assert f"tiles={tiles} cols={4 if kind == 'f32' else cols} chooses={int(chooses)}" in line["k_mx4_gate_up"], line
    assert f",{parts}) block" in line["k_mx4_down"] and line["k_mx4_down"].endswith("u=4 slots=1" if M == 1 else "u=2 slots=3"), line
    y, ids, wts = got[0]
    ref, bound = X.moe_layer(X.widen(x), *L.host, ids, wts.astype(np.float64))
    assert np.array_equal(ids, X.route(X.widen(x), X.widen(W), top_k, True)[0])
    assert (np.abs(y - ref) <= bound + 2.0 ** -120).all()


@pytest.mark.parametrize("kind", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("ld,offset,vec", [(64, 0, 1), (72, 0, 1), (71, 0, 0), (64, 1, 0)])
def test_conversions(capfd, kind, ld, offset, vec):
    t = U.torch_cuda()
    R, K = 5, 64
    rng = np.random.default_rng((ld, offset))
    xs = as_type(activations(rng, R, K), kind)
    dtype = getattr(t, {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}[kind])
    flat = t.zeros(R * ld + offset, dtype=dtype, device="cuda")
    view = flat[offset:].as_strided((R, K), (ld, 1), offset)
    view.copy_(dev(xs).view(dtype))
    codes, scales = U.empty_dev((R, K // 2), "uint8"), U.empty_dev((R, K // 32), "uint8")
    base = flat.data_ptr() + offset * flat.element_size()
    (name, line), = launches(capfd, lambda: kq.kq_mx4_quantize(kind, base, ld, codes, scales, R, K))
    assert name == "k_mx4_quantize" and line.endswith(f"vec={vec}"), line
    c, s = X.quantize(xs)
    assert np.array_equal(U.to_host(codes), X.planes(c, s)[0]) and np.array_equal(U.to_host(scales), s)
    view.zero_()
    (name, line), = launches(capfd, lambda: kq.kq_mx4_dequantize(codes, scales, kind, base, ld, R, K))
    assert name == "k_mx4_dequantize" and line.endswith(f"vec={vec}"), line
    want = X.dequantize(c, s)
    if kind == "f16":
        want = want.astype(np.float16).astype(np.float64)
    assert np.array_equal(view.double().cpu().numpy(), want)
