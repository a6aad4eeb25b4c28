"""mla_prefill_attn's entry point without a GPU: host-side validation returns its status before any
CUDA call, and the binding refuses tensors that do not fit."""
import ctypes

import pytest
import torch

import head_latent_attention_attn_b200 as mla
from tests.test_abi_host import FAKE, P, _dims


def _prefill(d, **kw):
    a = dict(q=FAKE, k=FAKE, kts=128 * 128, khs=128, kr=FAKE, krts=64, v=FAKE, vts=128 * 128,
             vhs=128, lens=FAKE, q_lens=None, batch=2, qlen=5, kvlen=64, causal=1, o=FAKE, lse=FAKE,
             err=None)
    a.update(kw)
    return mla.lib().mla_prefill_attn(ctypes.byref(d), *a.values(), None)


def test_validation(mla_lib):
    bad, unsupported = mla.MLA_ERR_INVALID_ARG, mla.MLA_ERR_UNSUPPORTED
    assert _prefill(_dims(num_kv_groups=3)) == bad
    for k in ("q", "k", "kr", "v", "lens", "o", "lse"):
        assert _prefill(_dims(), **{k: None}) == bad
    for k in ("q", "k", "kr", "v", "o"):
        assert _prefill(_dims(), **{k: P(0x10008)}) == bad
    for kw in (dict(batch=-1), dict(qlen=0), dict(kvlen=0), dict(causal=2)):
        assert _prefill(_dims(), **kw) == bad
    # strides: a head's numbers, a token's heads, multiples of 8, below TMA's limit
    for kw in (dict(khs=120), dict(vhs=120), dict(kts=128 * 128 - 8), dict(vts=127 * 128),
               dict(krts=56), dict(khs=129), dict(kts=128 * 128 + 4), dict(vts=1 << 33)):
        assert _prefill(_dims(), **kw) == bad
    assert _prefill(_dims(qk_nope_dim=136)) == unsupported
    assert _prefill(_dims(v_head_dim=136)) == unsupported
    assert _prefill(_dims(rope_dim=72)) == unsupported
    assert _prefill(_dims(rope_dim=4, num_kv_groups=2, kv_lora_rank=512)) == unsupported
    assert _prefill(_dims(), batch=1 << 20, qlen=1 << 22) == unsupported       # too many units
    assert _prefill(_dims(), batch=0) == mla.MLA_OK


def test_binding_refuses(mla_lib):
    d = _dims()
    t = torch.zeros(1, 4, 128, 192, dtype=torch.bfloat16)
    for args in ((t,) * 7, (None,) * 7, (t[0],) + (t,) * 6):
        with pytest.raises(mla.MlaError):
            mla.mla_prefill_attn(d, *args)
    with pytest.raises(mla.MlaError):
        mla._per_token(t, "k_nope", t.shape)             # a CPU tensor
