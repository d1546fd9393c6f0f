"""Frequencies at the ends of the range: finite ones, or a refusal."""
import ctypes

import numpy as np
import pytest

import block_quantized_gemv_kq_amd as kq
from oracle import attn as A

NONE, LINEAR, NTK, YARN = range(4)


def call(scaling, rot, base, factor):
    f, m = np.full(128, np.nan), ctypes.c_double(0.0)
    st = kq.lib().kq_rope_freqs(scaling, rot, base, factor, 4096, 32.0, 1.0, f.ctypes.data, ctypes.addressof(m))
    return st, f[:rot // 2]


@pytest.mark.parametrize("scaling,rot,base,factor", [
    (LINEAR, 64, 1e4, 1e-310), (YARN, 64, 1e4, 1e-320), (NTK, 4, 1e4, 1e200), (NTK, 4, 1e4, 1e-200), (NONE, 256, 5e-324, 1.0)])
def test_frequencies_that_are_not_finite(scaling, rot, base, factor):
    st, _ = call(scaling, rot, base, factor)
    assert st == kq.KQ_ERR_ARG and "infinite" in kq.last_error()


@pytest.mark.parametrize("scaling,rot,base,factor", [
    (NONE, 2, 5e-324, 1.0), (NONE, 128, 1e308, 1.0), (NONE, 128, 1e-300, 1.0), (LINEAR, 64, 1e4, 1e-300), (LINEAR, 64, 1e4, 1e300),
    (NTK, 4, 1e4, 1e150), (NTK, 2, 1e4, 1e300), (NTK, 4, 1e4, 1e-150), (YARN, 64, 1e4, 1e-300)])
def test_frequencies_at_the_ends(scaling, rot, base, factor):
    st, f = call(scaling, rot, base, factor)
    want, _ = A.freqs(["none", "linear", "ntk", "yarn"][scaling], rot, base, factor, 4096)
    assert st == kq.KQ_OK and np.isfinite(f).all() and np.allclose(f, want, rtol=1e-12, atol=1e-320)
