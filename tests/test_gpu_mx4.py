"""Microscaled 4-bit matrices, the router and the whole mixture-of-experts layer
on the GPU against the fp64 oracle.

Tolerances, from the arithmetic: quantised planes and dequantised values are
exact. A product of K terms is summed in fp32 by at most K + 64 additions (the
64 for joining the waves), each off by at most 2^-23 of the sum of magnitudes
(2^-24 rounded to nearest; the matrix instruction may truncate), so |error| <=
(K + 64) 2^-23 sum|w x|. Signs of the roundings vary, so the 2-norm over many
outputs is held to 4 sqrt(K + 64) 2^-23 of that of sum|w x| / sqrt(K) besides. An
output rounded to 16 bits adds half a step of its own."""
import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import mx4 as X
from tests import gpu_util as U
from tests.test_gpu_canary import GUARD, Guarded

pytestmark = pytest.mark.gpu

TYPES = ("f32", "f16", "bf16")
UNIT = 2.0 ** -23


def as_type(a, kind):
    """fp64/fp32 array -> the type's host array (bf16 as uint16 bits, nearest even)."""
    a = np.asarray(a, np.float32)
    if kind == "f32":
        return a
    if kind == "f16":
        with np.errstate(over="ignore"):
            return a.astype(np.float16)
    b = a.view(np.uint32)
    r = (b + 0x7FFF + ((b >> 16) & 1)) >> 16
    return np.where(np.isnan(a), 0x7FC0, r).astype(np.uint16)


def dev(a):
    return U.to_dev(a.view(np.int16) if a.dtype == np.uint16 else a)


def random_planes(rng, R, K, lo=118, hi=136):
    """Codes and scales of a random matrix (every code, scales 2^-9 to 2^8)."""
    return rng.integers(0, 16, (R, K)).astype(np.uint8), rng.integers(lo, hi, (R, K // 32)).astype(np.uint8)


class Plane:
    """A plane in device memory between 0xFF bytes: codes of -6 and NaN scales,
    so that whatever is read past it shows in the result."""

    def __init__(self, bytes_):
        t = U.torch_cuda()
        n = bytes_.size
        self.buf = t.full((GUARD + n + GUARD,), 0xFF, dtype=t.uint8, device="cuda")
        self.buf[GUARD:GUARD + n] = t.from_numpy(np.ascontiguousarray(bytes_).reshape(-1)).to("cuda")
        self.ptr = self.buf.data_ptr() + GUARD


def upload(codes, scales):
    c, s = X.planes(codes, scales)
    return Plane(c), Plane(s)


def check(y, ref, mags, K, kind="f32", what=""):
    eps = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    y = X.widen(y)
    tiny = 2.0 ** -24 if kind == "f16" else 2.0 ** -126
    bound = (K + 64) * UNIT * mags
    assert np.isfinite(y).all(), what
    err = np.abs(y - ref)
    lim = bound + eps * (np.abs(ref) + bound) + tiny
    assert (err <= lim).all(), (what, np.argwhere(err > lim)[:3], (err / lim).max())
    if kind == "f32" and y.size >= 64:
        rel = np.linalg.norm(err) / np.linalg.norm(mags / np.sqrt(K))
        assert rel <= 4 * np.sqrt(K + 64) * UNIT, (what, rel)


# ------------------------------------------------------------------ quantise

SPECIAL = np.array([0.0, -0.0, 1.0, -1.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.0, 7.9, 0.2499, 2.501,
                    -5.0, -0.25, 4.0, 1e-3, 1e-6, 3e-8, 6e-8, -3e-5, 65504.0, 1e-38, 1e-40, 1.4e-45, 3.0e38, -3.3e38, 2.0 ** -126])


def quantise_inputs(rng, R, K):
    """Rows of normals, blocks of ties, zeros, tiny, huge, infinite and NaN values."""
    x = (rng.standard_normal((R, K)) * np.exp(rng.standard_normal((R, 1)) * 4)).astype(np.float32)
    b = x.reshape(R * K // 32, 32)
    for i in range(b.shape[0]):
        pick = i % 9
        if pick == 1:
            b[i] = SPECIAL * 2.0 ** rng.integers(-3, 4) if i % 2 else SPECIAL
        elif pick == 2:
            b[i] = 0.0
        elif pick == 3:
            b[i] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 32) * rng.choice([-1, 1], 32)
        elif pick == 4:
            b[i] *= 2.0 ** -140
        elif pick == 5 and i % 2:
            b[i, i % 32] = [np.inf, -np.inf, np.nan][i % 3]
    return x


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("R,K,ld", [(1, 32, 32), (9, 32, 32), (3, 96, 96), (7, 2560, 2560), (5, 2080, 2096),
                                    (4, 64, 71), (33, 160, 161), (2, 9728, 9728)])
def test_quantize(kind, R, K, ld):
    rng = np.random.default_rng((R, K))
    x = np.full((R, ld), np.nan, np.float32)
    with np.errstate(over="ignore"):
        x[:, :K] = quantise_inputs(rng, R, K)
    xt = as_type(x, kind)
    codes, scales = Guarded(R * K // 2), Guarded(R * K // 32)
    kq.kq_mx4_quantize(kind, dev(xt), ld, codes.ptr, scales.ptr, R, K)
    codes.check(fully_written=False, what="codes")
    scales.check(fully_written=False, what="scales")
    c, s = X.planes(*X.quantize(xt[:, :K]))
    got_c = U.to_host(codes.buf)[GUARD:GUARD + R * K // 2].reshape(R, -1)
    got_s = U.to_host(scales.buf)[GUARD:GUARD + R * K // 32].reshape(R, -1)
    assert np.array_equal(got_s, s)
    assert np.array_equal(got_c, c)


def test_quantize_unaligned_base():
    rng = np.random.default_rng(4)
    x = as_type(rng.standard_normal(1 + 3 * 64), "f16")
    d = dev(x)
    codes, scales = U.empty_dev((3, 32), "uint8"), U.empty_dev((3, 2), "uint8")
    kq.kq_mx4_quantize("f16", d.data_ptr() + 2, 64, codes, scales, 3, 64)
    c, s = X.planes(*X.quantize(x[1:].reshape(3, 64)))
    assert np.array_equal(U.to_host(codes), c) and np.array_equal(U.to_host(scales), s)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("R,K,ld", [(1, 32, 32), (17, 96, 96), (5, 2080, 2096), (4, 64, 71), (3, 4096, 4096)])
def test_dequantize(kind, R, K, ld):
    rng = np.random.default_rng((R, K, 1))
    codes, scales = random_planes(rng, R, K, 0, 256)   # every scale byte, NaN among them
    pc, ps = upload(codes, scales)
    size = 4 if kind == "f32" else 2
    out = U.torch_cuda().full((GUARD + R * ld * size + GUARD,), 0x5A, dtype=U.torch_cuda().uint8, device="cuda")
    kq.kq_mx4_dequantize(pc.ptr, ps.ptr, kind, out.data_ptr() + GUARD, ld, R, K)
    h = U.to_host(out)
    assert (h[:GUARD] == 0x5A).all() and (h[GUARD + R * ld * size:] == 0x5A).all()
    got = h[GUARD:GUARD + R * ld * size].view({"f32": np.float32, "f16": np.float16, "bf16": np.uint16}[kind]).reshape(R, ld)
    assert (np.ascontiguousarray(got[:, K:]).view(np.uint8) == 0x5A).all()   # what lies between rows stays
    want = X.dequantize(codes, scales)
    if kind == "f16":
        with np.errstate(over="ignore"):
            want = want.astype(np.float16).astype(np.float64)
    assert np.array_equal(X.widen(got[:, :K].copy()), want, equal_nan=True)


def test_quantize_empty_and_idempotent():
    kq.kq_mx4_quantize("f32", None, 32, None, None, 0, 32)
    rng = np.random.default_rng(6)
    x = dev(as_type(rng.standard_normal((20, 512)), "bf16"))
    c, s, v = U.empty_dev((20, 256), "uint8"), U.empty_dev((20, 16), "uint8"), U.empty_dev((20, 512), "float16")
    c2, s2, v2 = U.empty_dev((20, 256), "uint8"), U.empty_dev((20, 16), "uint8"), U.empty_dev((20, 512), "float16")
    kq.kq_mx4_quantize("bf16", x, 512, c, s, 20, 512)
    kq.kq_mx4_dequantize(c, s, "bf16", v, 512, 20, 512)
    kq.kq_mx4_quantize("bf16", v, 512, c2, s2, 20, 512)
    kq.kq_mx4_dequantize(c2, s2, "bf16", v2, 512, 20, 512)
    assert np.array_equal(U.to_host(v).view(np.uint16), U.to_host(v2).view(np.uint16))


# ------------------------------------------------------------------ gemv

GEMV_SHAPES = [(1, 32), (15, 96), (16, 128), (17, 160), (333, 1056), (48, 2560), (100, 4096), (31, 9728), (5, 16416)]


def activations(rng, M, K):
    """Rows whose channels differ by large factors, as hidden states do."""
    return rng.standard_normal((M, K)) * np.exp(1.5 * rng.standard_normal(K))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("N,K", GEMV_SHAPES)
@pytest.mark.parametrize("M", (1, 5, 16, 17, 33, 64))
def test_gemv(kind, N, K, M):
    rng = np.random.default_rng((N, K, M))
    codes, scales = random_planes(rng, N, K)
    pc, ps = upload(codes, scales)
    x = as_type(activations(rng, M, K), kind)
    y = Guarded(4 * M * N)
    xd = dev(x)
    kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, xd, y.ptr, N, K, M)
    y.check(what=f"{kind} {N}x{K} M={M}")
    got = U.to_host(y.buf)[GUARD:GUARD + 4 * M * N].view(np.float32).reshape(M, N)
    check(got, *X.product(X.dequantize(codes, scales), X.widen(x)), K, what=f"{kind} {N}x{K} M={M}")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M", (2, 3, 4, 6, 7, 8, 9, 12, 15, 24, 32, 48, 49, 63))
def test_gemv_every_width(kind, M):
    N, K = 130, 1184
    rng = np.random.default_rng((M, 77))
    codes, scales = random_planes(rng, N, K)
    pc, ps = upload(codes, scales)
    x = as_type(activations(rng, M, K), kind)
    y = U.empty_dev((M, N))
    kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, dev(x), y, N, K, M)
    check(U.to_host(y), *X.product(X.dequantize(codes, scales), X.widen(x)), K, what=f"{kind} M={M}")


@pytest.mark.parametrize("kind", TYPES)
def test_gemv_unit_vectors_give_the_weights(kind):
    """x = a unit vector picks one weight exactly, with every code and the scales 2^-100 to 2^100."""
    N, K, M = 40, 224, 56
    rng = np.random.default_rng(9)
    codes, scales = random_planes(rng, N, K, 27, 228)
    pc, ps = upload(codes, scales)
    w = X.dequantize(codes, scales)
    for k0 in range(0, K, M):
        x = np.zeros((M, K))
        x[np.arange(M), k0 + np.arange(M)] = 1.0
        y = U.empty_dev((M, N))
        kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, dev(as_type(x, kind)), y, N, K, M)
        assert np.array_equal(U.to_host(y).astype(np.float64), w[:, k0:k0 + M].T)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("K", (160, 256))
def test_gemv_non_finite(kind, K):
    """A NaN scale spoils its rows alone, a NaN or infinite activation its
    columns alone; a zero weight times infinity is NaN."""
    N, M = 37, 6
    rng = np.random.default_rng((K, 3))
    codes, scales = random_planes(rng, N, K)
    scales[5, 1] = scales[36, K // 32 - 1] = 255
    codes[7, 40], codes[8, 40] = 0, 3
    x = activations(rng, M, K)
    x[1, 2] = np.nan
    x[4, 40] = np.inf
    pc, ps = upload(codes, scales)
    y = U.empty_dev((M, N))
    xt = as_type(x, kind)
    kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, dev(xt), y, N, K, M)
    got = U.to_host(y)
    with np.errstate(invalid="ignore"):
        want = X.widen(xt) @ X.dequantize(codes, scales).T
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want)) and (got[np.isinf(want)] == want[np.isinf(want)]).all()
    assert np.isfinite(got[[0, 2, 3, 5]][:, [i for i in range(N) if i not in (5, 36)]]).all()


def test_gemv_extreme_activations():
    """fp32 activations at both ends of the range, 24 bits each; fp16 and bf16 denormals."""
    N, K = 33, 64
    rng = np.random.default_rng(12)
    codes, scales = random_planes(rng, N, K, 126, 129)
    pc, ps = upload(codes, scales)
    w = X.dequantize(codes, scales)
    for kind, scale in (("f32", 2.0 ** 120), ("f32", 2.0 ** -100), ("f16", 2.0 ** -20), ("bf16", 2.0 ** -118), ("f16", 2.0 ** 12)):
        x = as_type(rng.standard_normal((3, K)) * scale, kind)
        y = U.empty_dev((3, N))
        kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, dev(x), y, N, K, 3)
        ref, mags = X.product(w, X.widen(x))
        err = np.abs(U.to_host(y) - ref)
        assert (err <= (K + 64) * UNIT * mags).all(), (kind, scale, (err / mags).max())


# ------------------------------------------------------------------ gemm

@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 64, 256), (3, 17, 96), (64, 64, 512), (65, 63, 160), (77, 1000, 1056),
                                   (130, 258, 2560), (16, 333, 9728), (200, 5, 288), (33, 129, 480)])
def test_gemm(kind, M, N, K):
    rng = np.random.default_rng((M, N, K))
    a, w = random_planes(rng, M, K), random_planes(rng, N, K)
    pa, pw = upload(*a), upload(*w)
    size = 4 if kind == "f32" else 2
    y = Guarded(size * M * N, elem=size)
    kq.kq_mx4_gemm(pa[0].ptr, pa[1].ptr, pw[0].ptr, pw[1].ptr, kind, y.ptr, M, N, K)
    y.check(fully_written=size * M * N % 4 == 0, what=f"{kind} {M}x{N}x{K}")
    got = U.to_host(y.buf)[GUARD:GUARD + size * M * N].view({"f32": np.float32, "f16": np.float16, "bf16": np.uint16}[kind])
    ref, mags = X.product(X.dequantize(*w), X.dequantize(*a))
    if kind == "f16":   # what fp16 cannot hold is infinite there
        sure = np.abs(ref) + (K + 64) * UNIT * mags < 65504
        got = np.where(sure, got.reshape(M, N), 0)
        ref, mags = np.where(sure, ref, 0), np.where(sure, mags, 0)
    check(got.reshape(M, N), ref, mags, K, kind, f"{kind} {M}x{N}x{K}")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,N,K", [(4096, 2048, 96), (2049, 4000, 544), (300, 20001, 256), (20001, 300, 1280),   # 160 x 256 tiles
                                   (2048, 2560, 160), (1900, 2561, 2592), (2000, 2500, 384),                  # 192 x 128
                                   (4100, 12000, 96), (4099, 12001, 1184), (4096, 12032, 1280),               # 256 x 256
                                   (300, 6143, 2592), (300, 6144, 2560), (40, 300, 256), (513, 999, 96),      # 64 x 64
                                   (64, 2560, 9728), (33, 1570, 5856), (512, 512, 3200)])                     # 32 x 32
def test_gemm_tiles(kind, M, N, K):
    """Every tile shape; every result bit for bit, as the sums are exact in fp32."""
    t = U.torch_cuda()
    dtype = {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[kind]
    rng = np.random.default_rng((M, N))
    # magnitudes up to 6 and scales of 1: multiples of 1/4 up to 36 K < 2^24 / 4 are exact in any order
    a, w = random_planes(rng, M, K, 127, 128), random_planes(rng, N, K, 127, 128)
    pa, pw = upload(*a), upload(*w)
    y = t.full((M, N), float("nan"), dtype=dtype, device="cuda")
    kq.kq_mx4_gemm(pa[0].ptr, pa[1].ptr, pw[0].ptr, pw[1].ptr, kind, y, M, N, K)
    av, wv = (t.from_numpy(X.dequantize(*p).astype(np.float32)).to("cuda").double() for p in (a, w))
    assert t.equal(y, (av @ wv.T.contiguous()).to(dtype))


def test_gemm_nan_scales_stay_in_their_rows():
    M, N, K = 70, 90, 160
    rng = np.random.default_rng(21)
    a, w = random_planes(rng, M, K), random_planes(rng, N, K)
    a[1][3, 4] = w[1][50, 0] = w[1][89, 4] = 255
    pa, pw = upload(*a), upload(*w)
    y = U.empty_dev((M, N))
    kq.kq_mx4_gemm(pa[0].ptr, pa[1].ptr, pw[0].ptr, pw[1].ptr, "f32", y, M, N, K)
    want = np.zeros((M, N), bool)
    want[3] = True
    want[:, [50, 89]] = True
    assert np.array_equal(np.isnan(U.to_host(y)), want)


# ------------------------------------------------------------------ router

def run_route(xt, Wt, xk, wk, top_k, renorm):
    M, K = xt.shape
    E = Wt.shape[0]
    ids, wts = Guarded(4 * M * top_k), Guarded(4 * M * top_k)
    n = kq.kq_moe_route_workspace_bytes(M, E)
    ws = Guarded(n, elem=2)
    kq.kq_moe_route(xk, dev(xt), wk, dev(Wt), M, K, E, top_k, renorm, ids.ptr, wts.ptr, ws.ptr, n)
    ids.check(what="ids")
    wts.check(fully_written=False, what="weights")
    ws.check(fully_written=False, what="workspace")
    cut = lambda g, d: U.to_host(g.buf)[GUARD:GUARD + 4 * M * top_k].view(d).reshape(M, top_k)   # noqa: E731
    return cut(ids, np.int32), cut(wts, np.float32)


@pytest.mark.parametrize("xk,wk", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("M,K,E,top_k", [(1, 32, 1, 1), (1, 2048, 128, 8), (3, 96, 5, 5), (16, 2048, 128, 8), (17, 160, 65, 3),
                                         (64, 512, 512, 10), (5, 64, 1024, 64), (2, 4096, 257, 12), (48, 320, 64, 1)])
@pytest.mark.parametrize("renorm", (True, False))
def test_route(xk, wk, M, K, E, top_k, renorm):
    rng = np.random.default_rng((M, K, E))
    xt, Wt = as_type(rng.standard_normal((M, K)), xk), as_type(rng.standard_normal((E, K)) * K ** -0.5, wk)
    ids, wts = run_route(xt, Wt, xk, wk, top_k, renorm)
    rid, rw, _ = X.route(X.widen(xt), X.widen(Wt), top_k, renorm)
    assert np.array_equal(ids, rid)
    # 64-bit logits and softmax, one rounding to fp32 (half a step, and 2^-30 for the 64-bit steps)
    assert (np.abs(wts - rw) <= (2.0 ** -24 + 2.0 ** -30) * rw).all()


def test_route_ties_and_close_logits():
    """Equal logits go to the lower index; logits that differ in the last bit of
    fp64-exact sums are told apart where fp32 sums would not."""
    K, E = 64, 200
    W = np.zeros((E, K), np.float32)
    W[:, 0] = 1.0
    W[70:75, 1] = 2.0 ** -30          # five experts ahead by 2^-30
    W[130, 1] = 2.0 ** -29
    x = np.ones((2, K), np.float32)
    x[1, 1] = -1.0
    ids, wts = run_route(x, W, "f32", "f32", 8, True)
    assert ids[0].tolist() == [130, 70, 71, 72, 73, 74, 0, 1]
    assert ids[1].tolist() == [0, 1, 2, 3, 4, 5, 6, 7]
    assert np.allclose(wts, 0.125, rtol=1e-6)


def test_route_non_finite():
    K, E = 32, 70
    rng = np.random.default_rng(2)
    W, x = rng.standard_normal((E, K)).astype(np.float32), rng.standard_normal((3, K)).astype(np.float32)
    W[5, 3] = np.nan                  # one expert's logit is NaN for every token
    x[1, 0] = np.nan                  # every logit of this token is NaN
    ids, wts = run_route(x, W, "f32", "f32", 4, True)
    rid, rw, _ = X.route(X.widen(x), X.widen(W), 4, True)
    assert np.array_equal(ids, rid) and ids[1].tolist() == [0, 1, 2, 3]
    assert np.isnan(wts[1]).all() and np.allclose(wts[[0, 2]], rw[[0, 2]], rtol=2.0 ** -23)
    assert np.isnan(run_route(x, W, "f32", "f32", 4, False)[1]).all()


# ------------------------------------------------------------------ layer

class Layer:
    def __init__(self, rng, E, H, inter):
        self.E, self.H, self.I = E, H, inter
        self.host, self.planes = [], []
        for n, k in ((inter, H), (inter, H), (H, inter)):
            c, s = random_planes(rng, E * n, k, 119, 123)
            self.host.append(X.dequantize(c, s).reshape(E, n, k))
            self.planes += list(upload(c, s))

    def run(self, x, xk, W, wk, top_k, renorm, ws=None, out=None):
        M = x.shape[0]
        n = kq.kq_mx4_moe_layer_workspace_bytes(self.H, self.I, M, top_k, self.E)
        ws = Guarded(n, elem=2) if ws is None else ws
        out = out or [Guarded(4 * M * self.H), Guarded(4 * M * top_k), Guarded(4 * M * top_k)]
        kq.kq_mx4_moe_layer(xk, dev(x), wk, dev(W), *[p.ptr for p in self.planes], *[o.ptr for o in out], self.H, self.I, M,
                            top_k, self.E, renorm, ws.ptr, n)
        ws.check(fully_written=False, what="workspace")
        for o in out:
            o.check(fully_written=False)
        cut = lambda g, d: U.to_host(g.buf)[GUARD:GUARD + g.n].view(d).reshape(M, -1)   # noqa: E731
        return cut(out[0], np.float32), cut(out[1], np.int32), cut(out[2], np.float32)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,E,H,inter,top_k", [(1, 8, 32, 32, 2), (1, 16, 256, 128, 4), (1, 1, 96, 160, 1), (2, 5, 160, 96, 5),
                                               (7, 40, 512, 224, 3), (16, 32, 128, 256, 8), (33, 4, 96, 64, 2), (64, 12, 256, 96, 6),
                                               (64, 3, 64, 512, 1), (3, 300, 64, 32, 10)])
def test_layer(kind, M, E, H, inter, top_k):
    rng = np.random.default_rng((M, E, H))
    L = Layer(rng, E, H, inter)
    x, W = as_type(activations(rng, M, H), kind), as_type(rng.standard_normal((E, H)) * H ** -0.5, kind)
    for renorm in (True, False):
        y, ids, wts = L.run(x, kind, W, kind, top_k, renorm)
        rid, rw, _ = X.route(X.widen(x), X.widen(W), top_k, renorm)
        assert np.array_equal(ids, rid)
        assert (np.abs(wts - rw) <= (2.0 ** -24 + 2.0 ** -30) * rw).all()
        ref, bound = X.moe_layer(X.widen(x), *L.host, ids, wts.astype(np.float64))
        err = np.abs(y - ref)
        assert (err <= bound + 2.0 ** -120).all(), (kind, renorm, (err / bound).max())
        again = L.run(x, kind, W, kind, top_k, renorm)
        assert all(np.array_equal(a, b) for a, b in zip((y, ids, wts), again))


def test_layer_all_tokens_on_one_expert():
    """Every slot of 64 tokens on the same two experts; the others' weights are NaN and never read."""
    rng = np.random.default_rng(31)
    E, H, inter, M = 9, 128, 96, 64
    L = Layer(rng, E, H, inter)
    W = np.zeros((E, H), np.float32)
    W[2], W[7] = 1.0, 0.5
    W[[0, 1, 3, 4, 5, 6, 8]] = -1.0
    for i, n in enumerate((inter, inter, H)):
        s = L.planes[2 * i + 1]
        per = n * (H if i < 2 else inter) // 32
        view = s.buf[GUARD:GUARD + E * per].view(E, per)
        view[[0, 1, 3, 4, 5, 6, 8]] = 255
    x = np.abs(rng.standard_normal((M, H))).astype(np.float32)
    y, ids, wts = L.run(x, "f32", W, "f32", 2, True)
    assert (ids == [2, 7]).all()
    ref, bound = X.moe_layer(X.widen(x), *L.host, ids, wts.astype(np.float64))
    assert (np.abs(y - ref) <= bound).all()


def test_layer_bad_rows_stay_alone():
    """A token of NaN gives NaN in its own row; the others keep the bits they have without it."""
    rng = np.random.default_rng(32)
    L = Layer(rng, 8, 96, 64)
    W = as_type(rng.standard_normal((8, 96)), "f16")
    x = as_type(rng.standard_normal((5, 96)), "f16")
    good = L.run(x, "f16", W, "f16", 2, True)
    bad = x.copy()
    bad[3, 17] = np.nan
    y, ids, wts = L.run(bad, "f16", W, "f16", 2, True)
    assert np.isnan(y[3]).all() and np.isnan(wts[3]).all() and ids[3].tolist() == [0, 1]
    keep = [0, 1, 2, 4]
    assert np.array_equal(y[keep], good[0][keep]) and np.array_equal(ids[keep], good[1][keep])


# ------------------------------------------------------------------ together

def test_quantise_then_multiply_and_route_into_packed_experts():
    """A model's path: weights quantised on the GPU, a prompt through the product of two microscaled matrices, a decode
    token through the same weights, and the router's output taken by kq_moe_ffn with Q4_0 experts."""
    from oracle import formats as F
    from oracle import ref as R
    from synth import inputs as S
    t = U.torch_cuda()
    rng = np.random.default_rng(41)
    N, K, M = 200, 384, 70
    Wf, xp = rng.standard_normal((N, K)).astype(np.float32) * 0.02, as_type(activations(rng, M, K), "bf16")
    wc, ws_, ac, as_ = (U.empty_dev(s, "uint8") for s in ((N, K // 2), (N, K // 32), (M, K // 2), (M, K // 32)))
    y, yd = U.empty_dev((M, N)), U.empty_dev((1, N))
    kq.kq_mx4_quantize("f32", dev(Wf), K, wc, ws_, N, K)
    xd = dev(xp)
    kq.kq_mx4_quantize("bf16", xd, K, ac, as_, M, K)
    kq.kq_mx4_gemm(ac, as_, wc, ws_, "f32", y, M, N, K)
    kq.kq_mx4_gemv(wc, ws_, "bf16", xd, yd, N, K, 1)
    w, a = X.dequantize(*X.quantize(Wf)), X.dequantize(*X.quantize(xp))
    check(U.to_host(y), *X.product(w, a), K, what="prompt")
    check(U.to_host(yd), *X.product(w, X.widen(xp[:1])), K, what="decode")
    # router + Q4_0 experts
    E, H, inter, top_k, m = 8, 128, 64, 2, 3
    Wr, x = as_type(rng.standard_normal((E, H)), "f16"), as_type(rng.standard_normal((m, H)), "f16")
    ids, wts = U.empty_dev((m, top_k), "int32"), U.empty_dev((m, top_k))
    n = kq.kq_moe_route_workspace_bytes(m, E)
    wsp = U.empty_dev((n,), "uint8")
    xg = dev(x)
    kq.kq_moe_route("f16", xg, "f16", dev(Wr), m, H, E, top_k, True, ids, wts, wsp, n)
    mats, devw = [], []
    for which, (r, c) in enumerate([(inter, H), (inter, H), (H, inter)]):
        Ws = [S.weights((91, e, which, 0), r, c) for e in range(E)]
        devw.append(U.to_dev(np.concatenate([kq.kq_pack("q4_0", v) for v in Ws])))
        mats.append([F.quantize("q4_0", v) for v in Ws])
    yf, h = U.empty_dev((m, H)), U.empty_dev((m, top_k, inter), "float16")
    nb = kq.kq_moe_ffn_workspace_bytes(H, inter, m, top_k)
    wsf = t.empty(nb, dtype=t.uint8, device="cuda")
    kq.kq_moe_ffn("q4_0", *devw, xg, ids, wts, yf, h, H, inter, m, top_k, E, wsf, nb)
    rid, rw, _ = X.route(X.widen(x), X.widen(Wr), top_k, True)
    yr, ad, *_ = R.moe_ffn("q4_0", *mats, x, rid, rw.astype(np.float32), h_override=U.to_host(h))
    U.assert_parity(U.to_host(yf), yr, ad, "router into kq_moe_ffn")


def test_captured_and_on_another_stream():
    """Every call captured into one graph, replayed with new inputs and eager work between; equal bits to eager calls.
    Two graphs with workspaces of their own replayed on two streams at once."""
    t = U.torch_cuda()
    rng = np.random.default_rng(51)
    E, H, inter, M, top_k, N = 16, 256, 128, 4, 3, 300
    L = Layer(rng, E, H, inter)
    W = dev(as_type(rng.standard_normal((E, H)) * H ** -0.5, "bf16"))
    pw = upload(*random_planes(rng, N, H))
    n = kq.kq_mx4_moe_layer_workspace_bytes(H, inter, M, top_k, E)

    class Set:
        def __init__(self):
            self.x = t.zeros((M, H), dtype=t.bfloat16, device="cuda")
            self.c, self.s = t.empty((M, H // 2), dtype=t.uint8, device="cuda"), t.empty((M, H // 32), dtype=t.uint8, device="cuda")
            self.v, self.y1, self.y2 = (t.empty(s, device="cuda") for s in ((M, H), (M, N), (M, N)))
            self.y3, self.ids, self.w = t.empty((M, H), device="cuda"), t.empty((M, top_k), dtype=t.int32, device="cuda"), t.empty((M, top_k), device="cuda")
            self.ws = t.empty(n, dtype=t.uint8, device="cuda")

        def run(self):
            kq.kq_mx4_quantize("bf16", self.x, H, self.c, self.s, M, H)
            kq.kq_mx4_dequantize(self.c, self.s, "f32", self.v, H, M, H)
            kq.kq_mx4_gemm(self.c, self.s, pw[0].ptr, pw[1].ptr, "f32", self.y1, M, N, H)
            kq.kq_mx4_gemv(pw[0].ptr, pw[1].ptr, "bf16", self.x, self.y2, N, H, M)
            kq.kq_mx4_moe_layer("bf16", self.x, "bf16", W, *[p.ptr for p in L.planes], self.y3, self.ids, self.w, H, inter, M,
                                top_k, E, True, self.ws, n)

        def outputs(self):
            return [a.clone() for a in (self.c, self.s, self.v, self.y1, self.y2, self.y3, self.ids, self.w)]

    sets = [Set(), Set()]
    xs = [t.from_numpy(rng.standard_normal((M, H))).to("cuda", t.bfloat16) for _ in range(5)]
    want = []
    for x in xs:
        sets[0].x.copy_(x)
        sets[0].run()
        want.append(sets[0].outputs())
    graphs, streams = [], [t.cuda.Stream(), t.cuda.Stream()]
    for s, st in zip(sets, streams):
        st.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(st):
            s.run()
        st.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=st):
            s.run()
        graphs.append(g)
    for i in range(5):
        for k in (0, 1):
            with t.cuda.stream(streams[k]):
                sets[k].x.copy_(xs[(i + k) % 5])
                graphs[k].replay()
        t.cuda.synchronize()
        for k in (0, 1):
            got = sets[k].outputs()
            assert all(t.equal(a, b) for a, b in zip(got, want[(i + k) % 5])), (i, k)
        _ = (xs[i].float() @ xs[i].float().T).sum().item()   # eager work and a synchronisation between replays


# ------------------------------------------------------------------ ways the work is shared out

@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("N,K,M", [(1000, 2080, 64),   # few row tiles: groups of 16 columns (16-bit types)
                                   (1000, 2048, 50), (37, 13056, 33),
                                   (1801, 160, 64), (1500, 544, 49),     # groups of 32
                                   (8200, 160, 17), (8209, 256, 48), (8207, 96, 64),   # two row tiles
                                   (1601, 160, 61), (3201, 288, 64), (12305, 128, 3), (12305, 160, 16)])   # fp32: two and four
def test_gemv_shared_out(kind, N, K, M):
    rng = np.random.default_rng((N, K, M, 3))
    codes, scales = random_planes(rng, N, K)
    pc, ps = upload(codes, scales)
    x = as_type(activations(rng, M, K), kind)
    y = Guarded(4 * M * N)
    xd = dev(x)
    kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, xd, y.ptr, N, K, M)
    y.check(what=f"{kind} {N}x{K} M={M}")
    got = U.to_host(y.buf)[GUARD:GUARD + 4 * M * N].view(np.float32).reshape(M, N)
    check(got, *X.product(X.dequantize(codes, scales), X.widen(x)), K, what=f"{kind} {N}x{K} M={M}")


@pytest.mark.parametrize("kind", TYPES)
def test_longest_rows(kind):
    """K at its limit: quantised, dequantised and multiplied in both products."""
    K, M, N = 1 << 20, 5, 3
    rng = np.random.default_rng(61)
    x = as_type(activations(rng, M, K) * 0.01, kind)
    codes, scales = random_planes(rng, N, K)
    pw = upload(codes, scales)
    w = X.dequantize(codes, scales)
    c, s, y, yg = U.empty_dev((M, K // 2), "uint8"), U.empty_dev((M, K // 32), "uint8"), U.empty_dev((M, N)), U.empty_dev((M, N))
    xd = dev(x)
    kq.kq_mx4_quantize(kind, xd, K, c, s, M, K)
    rc, rs = X.quantize(x)
    pc, ps = X.planes(rc, rs)
    assert np.array_equal(U.to_host(c), pc) and np.array_equal(U.to_host(s), ps)
    kq.kq_mx4_gemv(pw[0].ptr, pw[1].ptr, kind, xd, y, N, K, M)
    check(U.to_host(y), *X.product(w, X.widen(x)), K, what="gemv")
    kq.kq_mx4_gemm(c, s, pw[0].ptr, pw[1].ptr, "f32", yg, M, N, K)
    check(U.to_host(yg), *X.product(w, X.dequantize(rc, rs)), K, what="gemm")


def test_many_rows_past_32_bit_offsets():
    """A matrix whose code plane passes 4 GiB: the last rows are the last rows."""
    t = U.torch_cuda()
    K, N = 1024, (1 << 23) + 5
    codes = t.zeros((N, K // 2), dtype=t.uint8, device="cuda")
    scales = t.full((N, K // 32), 127, dtype=t.uint8, device="cuda")
    rng = np.random.default_rng(62)
    c, s = random_planes(rng, 40, K)
    bc, bs = X.planes(c, s)
    codes[-40:] = t.from_numpy(bc).to("cuda")
    scales[-40:] = t.from_numpy(bs).to("cuda")
    x = as_type(activations(rng, 2, K), "bf16")
    y = U.empty_dev((2, N))
    kq.kq_mx4_gemv(codes, scales, "bf16", dev(x), y, N, K, 2)
    assert not bool(y[:, :-40].any())
    check(y[:, -40:].cpu().numpy(), *X.product(X.dequantize(c, s), X.widen(x)), K)
    ac, as_ = X.quantize(x)
    pa = upload(ac, as_)
    kq.kq_mx4_gemm(pa[0].ptr, pa[1].ptr, codes, scales, "f32", y, 2, N, K)
    assert not bool(y[:, :-40].any())
    check(y[:, -40:].cpu().numpy(), *X.product(X.dequantize(c, s), X.dequantize(ac, as_)), K)
    v = t.empty((40, K), dtype=t.float32, device="cuda")
    kq.kq_mx4_dequantize(codes[-40:], scales[-40:], "f32", v, K, 40, K)
    kq.kq_mx4_quantize("f32", v, K, codes, scales, 40, K)   # into the first rows
    back = t.empty((40, K), dtype=t.float32, device="cuda")
    kq.kq_mx4_dequantize(codes, scales, "f32", back, K, 40, K)
    assert t.equal(v, back)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,E,H,inter,top_k", [(1, 300, 160, 96, 7), (1, 512, 256, 64, 64), (1, 700, 96, 32, 5),     # one token: chosen in the experts' kernel, or not
                                               (1, 1024, 64, 32, 64), (1, 9, 96, 2080, 8), (1, 3, 12320, 32, 2),
                                               (64, 64, 32, 32, 64), (64, 80, 64, 32, 64),                             # every expert, 4096 slots
                                               (64, 9, 160, 96, 3), (40, 5, 256, 544, 2), (33, 2, 64, 1056, 2),       # eight columns in a pass
                                               (3, 7, 8352, 64, 3), (20, 3, 16384, 32, 1), (6, 4, 96, 8224, 2),       # long rows
                                               (16, 8, 2048, 64, 4), (9, 8, 1056, 160, 8), (2, 40, 2080, 224, 33)])
def test_layer_shared_out(kind, M, E, H, inter, top_k):
    rng = np.random.default_rng((M, E, H, 5))
    L = Layer(rng, E, H, inter)
    x, W = as_type(activations(rng, M, H), kind), as_type(rng.standard_normal((E, H)) * H ** -0.5, kind)
    y, ids, wts = L.run(x, kind, W, kind, top_k, False)
    rid, rw, _ = X.route(X.widen(x), X.widen(W), top_k, False)
    assert np.array_equal(ids, rid)
    assert (np.abs(wts - rw) <= (2.0 ** -24 + 2.0 ** -30) * rw).all()
    ref, bound = X.moe_layer(X.widen(x), *L.host, ids, wts.astype(np.float64))
    err = np.abs(y - ref)
    assert (err <= bound + 2.0 ** -120).all(), (err / bound).max()


def test_one_token_captured_on_two_streams():
    """Decode as it is captured: the one-token layer and the router, replayed on two streams at once, with workspaces of
    their own that hold what other calls left there."""
    t = U.torch_cuda()
    rng = np.random.default_rng(63)
    E, H, inter, top_k = 48, 512, 96, 6
    L = Layer(rng, E, H, inter)
    W = dev(as_type(rng.standard_normal((E, H)) * H ** -0.5, "f16"))
    n = kq.kq_mx4_moe_layer_workspace_bytes(H, inter, 1, top_k, E)
    nr = kq.kq_moe_route_workspace_bytes(1, E)

    class Set:
        def __init__(self):
            self.x = t.zeros((1, H), dtype=t.float16, device="cuda")
            self.y, self.ids, self.w = t.empty((1, H), device="cuda"), t.empty((1, top_k), dtype=t.int32, device="cuda"), t.empty((1, top_k), device="cuda")
            self.ids2, self.w2 = t.empty_like(self.ids), t.empty_like(self.w)
            self.ws = t.full((max(n, nr),), 0xFF, dtype=t.uint8, device="cuda")

        def run(self):
            kq.kq_mx4_moe_layer("f16", self.x, "f16", W, *[p.ptr for p in L.planes], self.y, self.ids, self.w, H, inter, 1,
                                top_k, E, True, self.ws, n)
            kq.kq_moe_route("f16", self.x, "f16", W, 1, H, E, top_k, True, self.ids2, self.w2, self.ws, nr)

        def outputs(self):
            return [a.clone() for a in (self.y, self.ids, self.w, self.ids2, self.w2)]

    xs = [t.from_numpy(rng.standard_normal((1, H))).to("cuda", t.float16) for _ in range(6)]
    sets, want = [Set(), Set()], []
    for x in xs:
        sets[0].x.copy_(x)
        sets[0].run()
        want.append(sets[0].outputs())
        assert t.equal(want[-1][1], want[-1][3]) and t.equal(want[-1][2], want[-1][4])
    graphs, streams = [], [t.cuda.Stream(), t.cuda.Stream()]
    for s, st in zip(sets, streams):
        st.wait_stream(t.cuda.current_stream())
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=st):
            s.run()
        graphs.append(g)
    for i in range(6):
        for k in (0, 1):
            with t.cuda.stream(streams[k]):
                sets[k].x.copy_(xs[(i + k) % 6])
                graphs[k].replay()
        t.cuda.synchronize()
        for k in (0, 1):
            assert all(t.equal(a, b) for a, b in zip(sets[k].outputs(), want[(i + k) % 6])), (i, k)
        _ = (xs[i].float() ** 2).sum().item()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("N,K,M", [(6143, 2080, 9), (6161, 2048, 16), (6129, 2048, 13)])
def test_gemv_two_row_tiles_of_up_to_16_columns(kind, N, K, M):
    rng = np.random.default_rng((N, K, M, 4))
    codes, scales = random_planes(rng, N, K)
    pc, ps = upload(codes, scales)
    x = as_type(activations(rng, M, K), kind)
    y = Guarded(4 * M * N)
    xd = dev(x)
    kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, xd, y.ptr, N, K, M)
    y.check(what=f"{kind} {N}x{K} M={M}")
    got = U.to_host(y.buf)[GUARD:GUARD + 4 * M * N].view(np.float32).reshape(M, N)
    check(got, *X.product(X.dequantize(codes, scales), X.widen(x)), K, what=f"{kind} {N}x{K} M={M}")
