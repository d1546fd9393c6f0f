"""Attention calls whose results would overwrite what they read: refused on the
host before any HIP call (the addresses are never dereferenced)."""
import ctypes

import pytest

import block_quantized_gemv_kq_amd as kq

ADDR = 0x10000   # aligned to everything


@pytest.mark.parametrize("type", ["f16", "bf16"])
@pytest.mark.parametrize("decode", [True, False])
def test_out_is_not_q(decode, type):
    cache = kq.kq_kv_cache(type, ADDR, ADDR, 9, 2, 64)

    def call(n_tokens, out, ldo):
        batch = kq.kq_kv_batch(ADDR, 4, ADDR, ADDR, 2, n_tokens)
        args = [kq._type(type), ADDR, 128, ctypes.addressof(cache), ctypes.addressof(batch), out, ldo, 2, 1.0, 0]
        return kq.lib().kq_attn_decode(*args, None, None, 0, None) if decode else kq.lib().kq_attn_prompt(*args, None, 0, None)
    assert call(5, ADDR, 128) == kq.KQ_ERR_ARG and "out must not be q" in kq.last_error()
    assert call(5, ADDR, 256) == kq.KQ_ERR_ARG and "out must not be q" in kq.last_error()
    assert call(0, ADDR, 128) == kq.KQ_OK      # nothing is written
