"""Microscaled products at the ends of the scale's range: a weight is its code
times its scale for every scale byte but 255, up to 6 * 2^127, whatever the
activations' type, and only a result past fp32 is infinite.

A product with a power of two is exact in fp32 unless it leaves fp32's normal
range: those tests ask for equal bits (results below 2^-126 may be zero).
Sums are held to the bound of tests/test_gpu_mx4.py, (K + 64) 2^-23 sum|w x|."""
import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import mx4 as X
from tests import gpu_util as U
from tests.test_gpu_mx4 import TYPES, UNIT, Layer, Plane, as_type, check, dev, upload

pytestmark = pytest.mark.gpu

ENDS = np.array([0, 1, 2, 3, 4, 60, 127, 200, 250, 251, 252, 253, 254], np.uint8)


def ends_planes(rng, R, K, bytes_=ENDS):
    """Every code with scale bytes of `bytes_`, several of them in each row."""
    return rng.integers(0, 16, (R, K)).astype(np.uint8), rng.choice(bytes_, (R, K // 32)).astype(np.uint8)


def same_power(got, want):
    """Equal bits, except that what is below fp32's normal range may be zero."""
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    tiny = np.abs(want) < 2.0 ** -126
    assert (got[~tiny] == want[~tiny]).all(), np.argwhere((got != want) & ~tiny)[:4]
    assert ((got[tiny] == want[tiny]) | (got[tiny] == 0)).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("N,K,M", [(40, 224, 1), (40, 256, 8), (6160, 2048, 16), (70, 224, 56), (70, 96, 33),
                                   (1500, 544, 49), (8200, 160, 17), (8207, 96, 48), (8207, 96, 64), (12305, 128, 5)])
def test_gemv_unit_vectors(kind, N, K, M):
    """x = a power of two in one place picks one weight, up and down the range."""
    rng = np.random.default_rng((N, K, M, 9))
    codes, scales = ends_planes(rng, N, K)
    pc, ps = upload(codes, scales)
    w = X.values(codes, scales)
    for power, k0 in ((-14, 0), (14, K - M if K > M else 0), (0, K // 2)):
        at = (k0 + np.arange(M)) % K
        x = np.zeros((M, K))
        x[np.arange(M), at] = 2.0 ** power
        y = U.empty_dev((M, N))
        kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, dev(as_type(x, kind)), y, N, K, M)
        same_power(U.to_host(y).astype(np.float64), (w[:, at] * 2.0 ** power).T)


@pytest.mark.parametrize("kind,power", [("f32", -133), ("f32", -126), ("f32", -149 + 20), ("bf16", -133), ("bf16", -127), ("f16", -24), ("f16", -15)])
def test_gemv_denormal_activations(kind, power):
    """A denormal power of two (from 2^-133 on for fp32: what lies below is dropped) times weights about 2^100."""
    N, K, M = 37, 160, 20
    rng = np.random.default_rng((3, power + 200))
    codes, scales = ends_planes(rng, N, K, np.array([226, 227, 229], np.uint8))
    pc, ps = upload(codes, scales)
    w = X.values(codes, scales)
    at = rng.integers(0, K, M)
    x = np.zeros((M, K))
    x[np.arange(M), at] = 2.0 ** power
    y = U.empty_dev((M, N))
    kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, dev(as_type(x, kind)), y, N, K, M)
    assert np.array_equal(U.to_host(y).astype(np.float64), (w[:, at] * 2.0 ** power).T)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M", (1, 5, 17, 33, 64))
@pytest.mark.parametrize("N,K", [(50, 160), (37, 1184), (8200, 128)])
def test_gemv_sums(kind, N, K, M):
    """Sums over blocks of every scale at once; columns 1, 4, .. are zero at the large blocks, so that the small ones
    count there. Magnitudes stay below 2^127."""
    rng = np.random.default_rng((N, K, M, 10))
    codes, scales = ends_planes(rng, N, K, np.array([100, 126, 127, 128, 250, 252, 253, 254], np.uint8))
    large = np.arange(K // 32) % 3 == 1
    scales[:, ~large] = rng.choice(np.array([100, 126, 127, 128], np.uint8), (N, int((~large).sum())))
    pc, ps = upload(codes, scales)
    x = np.clip(rng.standard_normal((M, K)), -4, 4) * 2.0 ** -14 * 32 / K
    x[1::3, np.repeat(large, 32)] = 0.0
    xt = as_type(x, kind)
    y = U.empty_dev((M, N))
    kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, dev(xt), y, N, K, M)
    check(U.to_host(y), *X.product(X.values(codes, scales), X.widen(xt)), K, what=f"{kind} M={M}")


@pytest.mark.parametrize("kind", TYPES)
def test_gemv_infinite_activations_at_large_scales(kind):
    """An infinite activation times a weight that is not zero is infinite, times zero NaN, at every scale; blocks beside
    it do not change that, and a NaN scale spoils its rows alone."""
    N, K, M = 60, 160, 3
    rng = np.random.default_rng(17)
    codes, scales = ends_planes(rng, N, K)
    scales[11, 3] = scales[59, 4] = 255
    x = np.full((M, K), 2.0 ** -20)
    x[1, 70], x[2, 133] = np.inf, -np.inf
    pc, ps = upload(codes, scales)
    y = U.empty_dev((M, N))
    xt = as_type(x, kind)
    kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, dev(xt), y, N, K, M)
    got = U.to_host(y)
    with np.errstate(invalid="ignore"):
        want = X.widen(xt) @ X.values(codes, scales).T
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want)) and (got[np.isinf(want)] == want[np.isinf(want)]).all()


@pytest.mark.parametrize("M,N,K", [(40, 300, 256), (33, 129, 480), (33, 40, 1056), (16, 333, 1280), (2049, 4000, 96), (4100, 12000, 96)])
def test_gemm_unit_rows(M, N, K):
    """Activation rows with one element of a power of two pick one weight."""
    rng = np.random.default_rng((M, N, K, 11))
    wc, wsc = ends_planes(rng, N, K)
    pw = upload(wc, wsc)
    w = X.values(wc, wsc)
    y = U.empty_dev((M, N))
    for power in (-14, 14, -120, 126):
        at = rng.integers(0, K, M)
        ac, asc = np.zeros((M, K), np.uint8), np.full((M, K // 32), 127 + power, np.uint8)
        ac[np.arange(M), at] = 2
        pa = upload(ac, asc)
        kq.kq_mx4_gemm(pa[0].ptr, pa[1].ptr, pw[0].ptr, pw[1].ptr, "f32", y, M, N, K)
        same_power(U.to_host(y).astype(np.float64), (w[:, at] * 2.0 ** power).T)


@pytest.mark.parametrize("M,N,K", [(40, 300, 256), (33, 40, 1056), (300, 900, 160)])
def test_gemm_sums(M, N, K):
    """Large weights with small activations and the reverse: the values' scales, up to 2^127, meet their opposites."""
    rng = np.random.default_rng((M, N, K, 12))
    a, w = ends_planes(rng, M, K), ends_planes(rng, N, K)
    asc = rng.integers(0, 255, (1, K // 32))
    a = (a[0], np.repeat(asc, M, 0).astype(np.uint8))
    w = (w[0], np.repeat(254 - asc, N, 0).astype(np.uint8))
    pa, pw = upload(*a), upload(*w)
    y = U.empty_dev((M, N))
    kq.kq_mx4_gemm(pa[0].ptr, pa[1].ptr, pw[0].ptr, pw[1].ptr, "f32", y, M, N, K)
    check(U.to_host(y), *X.product(X.values(*w), X.values(*a)), K, what=f"{M}x{N}x{K}")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,E,H,inter,top_k", [(1, 8, 160, 96, 3), (9, 6, 128, 160, 2), (40, 5, 256, 96, 2)])
@pytest.mark.parametrize("which", ("up", "down"))
def test_layer(kind, M, E, H, inter, top_k, which):
    """Experts whose up or down projection reaches 6 * 2^127, with h or the other projection as small."""
    rng = np.random.default_rng((M, E, H, 13))
    L = Layer(rng, E, H, inter)
    i, n, k = (1, inter, H) if which == "up" else (2, H, inter)
    c, s = ends_planes(rng, E * n, k, np.array([128, 250, 252, 253, 254], np.uint8))
    L.host[i] = X.values(c, s).reshape(E, n, k)
    L.planes[2 * i:2 * i + 2] = [Plane(p) for p in X.planes(c, s)]
    x = as_type(rng.standard_normal((M, H)) * 2.0 ** -13, kind)
    W = as_type(rng.standard_normal((E, H)) * 64.0, kind)
    y, ids, wts = L.run(x, kind, W, kind, top_k, True)
    assert np.isfinite(y).all()
    ref, bound = X.moe_layer(X.widen(x), *L.host, ids, wts.astype(np.float64))
    err = np.abs(y - ref)
    assert (err <= bound).all(), (kind, (err / bound).max())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("N,K,M", [(37, 13056, 33), (20, 16416, 1), (50, 9728, 64), (33, 20000, 9)])
def test_gemv_long_rows(kind, N, K, M):
    """Rows that a wave walks in several steps, the large scales in some of them."""
    rng = np.random.default_rng((N, K, M, 14))
    codes, scales = ends_planes(rng, N, K, np.array([100, 127, 128], np.uint8))
    scales[::2, K // 64] = 254
    scales[1::3, K // 32 - 1] = 253
    pc, ps = upload(codes, scales)
    x = rng.standard_normal((M, K))
    x[:, K // 64 * 32:K // 64 * 32 + 32] *= 2.0 ** -14
    x[:, -32:] *= 2.0 ** -13
    xt = as_type(x, kind)
    y = U.empty_dev((M, N))
    kq.kq_mx4_gemv(pc.ptr, ps.ptr, kind, dev(xt), y, N, K, M)
    check(U.to_host(y), *X.product(X.values(codes, scales), X.widen(xt)), K, what=f"{kind} M={M}")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,E,H,inter,top_k", [(3, 5, 8352, 64, 3), (20, 3, 16384, 32, 1), (1, 3, 12320, 32, 2), (6, 4, 96, 8224, 2)])
def test_layer_long_rows(kind, M, E, H, inter, top_k):
    """The same in the layer: up rows with a block at 2^126 or 2^127, down rows with a large scale on codes of zero."""
    rng = np.random.default_rng((M, E, H, 15))
    L = Layer(rng, E, H, inter)
    # up rows about 2^-86, a block of some at 2^126 or 2^127: u up to about 2^120, h to 2^107; down weights about 2^-79
    c, s = ends_planes(rng, E * inter, H, np.array([40, 41], np.uint8))
    s[::5, H // 64], s[2::5, H // 32 - 1] = 254, 253
    L.host[1], L.planes[2:4] = X.values(c, s).reshape(E, inter, H), [Plane(p) for p in X.planes(c, s)]
    c, s = ends_planes(rng, E * H, inter, np.array([47, 48, 49], np.uint8))
    s[::7, inter // 64] = 200   # met by the down projection's waves, on weights of zero
    c[::7, inter // 64 * 32:inter // 64 * 32 + 32] = 0
    L.host[2], L.planes[4:6] = X.values(c, s).reshape(E, H, inter), [Plane(p) for p in X.planes(c, s)]
    x = as_type(np.clip(rng.standard_normal((M, H)), -3, 3) * 2.0 ** -14, kind)
    W = as_type(rng.standard_normal((E, H)), kind)
    y, ids, wts = L.run(x, kind, W, kind, top_k, True)
    assert np.isfinite(y).all()
    ref, bound = X.moe_layer(X.widen(x), *L.host, ids, wts.astype(np.float64))
    assert (np.abs(y - ref) <= bound).all()
