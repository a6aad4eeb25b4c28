"""Sizes and strides at the ends of their types, without a GPU: refused or planned for, never wrapped."""
import pytest

import head_latent_attention_attn_b200 as mla
from tests.test_abi_host import _dims
from tests.test_abi_prefill import _prefill

BIG = (1 << 31) - 1


def test_prefill_sizes(mla_lib):
    """Row and token counts that 32-bit tile arithmetic would wrap on, or whose units take longer than
    a wait in the kernel may."""
    d = _dims(num_heads=1, qk_nope_dim=8, v_head_dim=8, rope_dim=0)
    small = dict(kts=8, khs=8, vts=8, vhs=8, kr=None, krts=0, batch=1)
    for kw in (dict(qlen=BIG), dict(kvlen=BIG), dict(qlen=(1 << 25) + 1), dict(kvlen=(1 << 25) + 1)):
        assert _prefill(d, **{**small, **kw}) == mla.MLA_ERR_UNSUPPORTED
    many = _dims(num_heads=1 << 30, num_kv_groups=1)
    wide = dict(kts=1 << 37, khs=128, vts=1 << 37, vhs=128, kvlen=1)
    assert _prefill(many, batch=1 << 30, qlen=1 << 12, **wide) == mla.MLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("stride", [1 << 61, (1 << 62) + 8, 1 << 58])
def test_prefill_head_strides(mla_lib, which, stride):
    assert _prefill(_dims(), **{which + "hs": stride}) == mla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("q", [3, 256])
def test_workspace_of_a_context_without_a_bound(mla_lib, q):
    """The larger workspace of a context that it cannot hold is the plain one."""
    d = _dims()
    for n in (BIG, BIG - 62):
        plain = mla.mla_decode_workspace_size(d, 1, q, n)
        assert plain > 0 and mla.mla_decode_q8_workspace_size(d, 1, q, n) == plain
    n = 1 << 20
    assert mla.mla_decode_q8_workspace_size(d, 1, q, n) > mla.mla_decode_workspace_size(d, 1, q, n)


def test_supported_widths(mla_lib):
    """The row widths that mla.h names for the decode are the ones that a plan exists for."""
    for H, q in ((1, 1), (32, 1), (33, 1), (16, 3), (64, 1), (65, 1), (128, 1), (128, 3)):
        for r in (8, 72, 128, 384, 440, 448, 472, 480, 504, 512):
            for R in (0, 8, 16, 32, 64, 72, 96, 104, 128):
                d = _dims(num_heads=H, num_kv_groups=1, kv_lora_rank=r, rope_dim=R)
                pair = q * H > 64 and r % 128 == 0 and R in (32, 64, 128)
                want = r + R <= 640 and (pair or q * H <= 32 or r + R <= 576)
                assert (mla.mla_decode_workspace_size(d, 2, q, 300) > 0) == want, (H, q, r, R)
