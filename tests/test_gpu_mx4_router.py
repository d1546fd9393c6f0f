"""Logits that are not finite, in the router and in the layer that chooses its
experts in the gate and up kernel (one token) or before it. Weights within half
a step of fp32 (2^-24) and 2^-30 for the steps in 64 bits."""
import numpy as np
import pytest

from oracle import mx4 as X
from tests.test_gpu_mx4 import Layer, run_route

pytestmark = pytest.mark.gpu


def router(kind, rng, M, K, E):
    """Router rows and activations (positive, so that the logit of a row with an infinity is that infinity)."""
    W = rng.standard_normal((E, K)).astype(np.float32) * K ** -0.5
    x = np.abs(rng.standard_normal((M, K))).astype(np.float32) + 0.1
    if kind == "minus":          # some experts at minus infinity
        W[[1, 4, E - 1], 3] = -np.inf
    elif kind == "plus":
        W[2, 5] = np.inf
    elif kind == "all minus":
        W[:, 0] = -np.inf
    elif kind == "minus and nan":   # both come last, by index among themselves
        W[[0, 3], 3] = -np.inf
        W[1, 2] = np.nan
    elif kind == "two finite":
        W[2:, 0] = -np.inf
    return W, x


@pytest.mark.parametrize("kind", ("minus", "plus", "all minus", "minus and nan", "two finite"))
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("M,E,top_k", [(1, 6, 6), (3, 6, 4), (2, 70, 5), (1, 130, 64)])
def test_logits_not_finite(kind, renorm, M, E, top_k):
    K, inter = 64, 32
    rng = np.random.default_rng((M, E, top_k))
    W, x = router(kind, rng, M, K, E)
    with np.errstate(invalid="ignore"):
        rid, rw, logits = X.route(X.widen(x), X.widen(W), top_k, renorm)
    enter = np.take_along_axis(logits, rid, 1) if renorm else logits
    # what the header says: NaN where a NaN, plus infinity or nothing but minus infinity enters the sum
    nan = np.isnan(enter).any(1) | (enter == np.inf).any(1) | (enter == -np.inf).all(1)
    assert np.array_equal(np.isnan(rw), np.repeat(nan[:, None], top_k, 1))
    L = Layer(rng, E, K, inter)
    runs = [run_route(x, W, "f32", "f32", top_k, renorm), L.run(x, "f32", W, "f32", top_k, renorm)[1:]]
    for ids, wts in runs:
        assert np.array_equal(ids, rid)
        assert np.array_equal(np.isnan(wts), np.isnan(rw))
        assert (np.abs(wts - rw)[~nan] <= (2.0 ** -24 + 2.0 ** -30) * rw[~nan]).all()
        minus = np.take_along_axis(logits, ids, 1) == -np.inf
        assert (wts[minus & ~nan[:, None]] == 0).all()
    y, ids, wts = L.run(x, "f32", W, "f32", top_k, renorm)
    assert np.isnan(y[nan]).all()
    ref, bound = X.moe_layer(X.widen(x)[~nan], *L.host, ids[~nan], wts[~nan].astype(np.float64))
    assert (np.abs(y[~nan] - ref) <= bound + 2.0 ** -120).all()
