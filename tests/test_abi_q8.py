"""The 8-bit cache's entry points without a GPU: host-side validation returns its status before
any CUDA call, the binding refuses tensors that do not fit, and the page layout."""
import ctypes

import numpy as np
import pytest
import torch

import head_latent_attention_attn_b200 as mla
from mla_inputs import CONFIGS
from tests import q8_reference as Q
from tests.test_abi_host import FAKE, P, _dims


def test_page_bytes(mla_lib):
    for c in CONFIGS.values():
        want = Q.page_bytes(c.kv_lora_rank, c.num_kv_groups * c.rope_dim)
        assert mla.mla_q8_page_bytes(_dims(c)) == (want if c.kv_lora_rank % 64 == 0 else -1)
    assert mla.mla_q8_page_bytes(_dims(page_size=32)) == -1
    assert mla.mla_q8_page_bytes(_dims(kv_lora_rank=576)) == -1
    assert mla.mla_q8_page_bytes(_dims(kv_lora_rank=72)) == -1


def _append(d, **kw):
    a = dict(c_kv=FAKE, k_r=FAKE, cos=FAKE, sin=FAKE, table=FAKE, maxp=4, start=FAKE, lens=None,
             batch=2, n=1, cache=FAKE, npages=8, err=None)
    a.update(kw)
    return mla.lib().mla_cache_append_q8(ctypes.byref(d), *a.values(), None)


def _read(d, **kw):
    a = dict(cache=FAKE, npages=8, table=FAKE, maxp=4, start=FAKE, lens=None, batch=2, n=1,
             out=FAKE, err=None)
    a.update(kw)
    return mla.lib().mla_cache_read_q8(ctypes.byref(d), *a.values(), None)


def _decode(d, **kw):
    a = dict(q=FAKE, cache=FAKE, npages=100, table=FAKE, maxp=4, lens=FAKE, batch=2, qlen=1,
             maxlen=256, causal=1, splits=1, ws=P(0x10000), wsb=1 << 20, o=FAKE, lse=FAKE)
    a.update(kw)
    return mla.lib().mla_decode_attn_q8(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("call", [_append, _read])
def test_append_and_read_validation(mla_lib, call):
    assert call(_dims(num_kv_groups=3)) == mla.MLA_ERR_INVALID_ARG
    assert call(_dims(page_size=32)) == mla.MLA_ERR_UNSUPPORTED
    assert call(_dims(kv_lora_rank=1024)) == mla.MLA_ERR_UNSUPPORTED
    assert call(_dims(kv_lora_rank=72)) == mla.MLA_ERR_UNSUPPORTED
    for k in ("cache", "table", "start"):
        assert call(_dims(), **{k: None}) == mla.MLA_ERR_INVALID_ARG
    assert call(_dims(), cache=P(0x10008)) == mla.MLA_ERR_INVALID_ARG
    for bad in (dict(batch=-1), dict(n=-1), dict(npages=0), dict(npages=1 << 31), dict(maxp=0)):
        assert call(_dims(), **bad) == mla.MLA_ERR_INVALID_ARG
    assert call(_dims(), batch=(1 << 31) - 1, n=(1 << 31) - 1) == mla.MLA_ERR_UNSUPPORTED
    assert call(_dims(), batch=0) == mla.MLA_OK
    assert call(_dims(), n=0) == mla.MLA_OK


def test_append_only_and_read_only_validation(mla_lib):
    for k in ("c_kv", "k_r", "cos", "sin"):
        assert _append(_dims(), **{k: None}) == mla.MLA_ERR_INVALID_ARG
    assert _append(_dims(), c_kv=P(0x10008)) == mla.MLA_ERR_INVALID_ARG
    assert _read(_dims(), out=None) == mla.MLA_ERR_INVALID_ARG
    assert _read(_dims(), out=P(0x10008)) == mla.MLA_ERR_INVALID_ARG


def test_decode_validation(mla_lib):
    assert _decode(_dims(page_size=32)) == mla.MLA_ERR_UNSUPPORTED
    assert _decode(_dims(kv_lora_rank=1024)) == mla.MLA_ERR_UNSUPPORTED
    assert _decode(_dims(kv_lora_rank=504)) == mla.MLA_ERR_UNSUPPORTED    # not whole blocks of 64
    assert _decode(_dims(), qlen=0) == mla.MLA_ERR_INVALID_ARG
    assert _decode(_dims(), causal=2) == mla.MLA_ERR_INVALID_ARG
    assert _decode(_dims(), lens=None) == mla.MLA_ERR_INVALID_ARG
    assert _decode(_dims(), cache=P(0x10008)) == mla.MLA_ERR_INVALID_ARG
    assert _decode(_dims(), ws=None) == mla.MLA_ERR_WORKSPACE
    assert _decode(_dims(), splits=4, wsb=4096) == mla.MLA_ERR_WORKSPACE
    assert _decode(_dims(), batch=0) == mla.MLA_OK


def test_binding_refuses(mla_lib):
    d = _dims()
    c = torch.zeros(2, 1, 512, dtype=torch.bfloat16)
    with pytest.raises(mla.MlaError):        # CPU tensors
        mla.mla_cache_append_q8(d, c, c, c, c, c, c, c)
    with pytest.raises(mla.MlaError):
        mla.mla_cache_append_q8(d, None, c, c, c, c, c, c)
    with pytest.raises(mla.MlaError):
        mla.mla_cache_read_q8(d, c, c, c, c)
    with pytest.raises(mla.MlaError):
        mla.mla_decode_attn_q8(d, c, c, c, c, 64, c, c, c)


def test_reference_quantiser():
    """The test reference itself, against torch's e4m3 rounding and by its invariants."""
    rng = np.random.default_rng(0)
    x = torch.from_numpy((rng.standard_normal((50, 128)) * np.exp(3 * rng.standard_normal((50, 1)))).astype(np.float32)).to(torch.bfloat16)
    bits = x.view(torch.int16).numpy().view(np.uint16)
    codes, byte = Q.quantise(bits)
    e = byte.astype(np.int64) - 127
    y = x.float().reshape(50, 2, 64)
    amax = y.abs().amax(-1).numpy().astype(np.float64)
    assert np.all(amax * 2.0 ** -e <= 448) and np.all(amax * 2.0 ** (1 - e) > 448)
    z = torch.ldexp(y, torch.from_numpy(-e)[..., None]).to(torch.float8_e4m3fn)
    assert np.array_equal(z.view(torch.uint8).numpy().reshape(50, 128), codes)
