"""Tensors that start where the calls allow and no other test puts them: queries on 16 bytes but not 32,
decode outputs on any element, prefill operands and outputs on 16 bytes. The same bits, and nothing
written outside."""
import numpy as np
import pytest
import torch

import head_latent_attention_attn_b200 as mla
from tests.test_gpu_prefill_expanded import make
from tests.test_gpu_q8 import Filled, bf, cu, decode

pytestmark = pytest.mark.gpu


class Shifted:
    """A tensor `shift` elements into a buffer of sevens."""

    def __init__(self, shape, dtype, shift, values=None):
        n = int(np.prod(shape))
        self.buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
        self.t = self.buf[shift:shift + n].view(shape)
        self.shift, self.n = shift, n
        if values is not None:
            self.t.copy_(values)

    def outside_is_untouched(self):
        return bool((self.buf[:self.shift] == 7.0).all()) and bool((self.buf[self.shift + self.n:] == 7.0).all())


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("q_shift,o_shift", [(8, 0), (0, 8), (24, 4), (16, 1), (8, 3)])
@pytest.mark.parametrize("name,q", [("deepseek_v2", 2), ("hybrid", 3), ("qwen25_7b", 1), ("pair_r256", 2)])
def test_decode(name, q, q_shift, o_shift, q8):
    f = Filled(name, [400, 70], seed=q)
    d, q_bits = f.dims, f.query(q)
    cache = f.cache if q8 else f.bf16_cache()
    fn = mla.mla_decode_attn_q8 if q8 else mla.mla_decode_attn
    H, r = d.num_heads, d.kv_lora_rank
    for ns in (0, 1, 3):
        want = decode(d, fn, q_bits, cache, f.table, f.lens, True, ns)
        x = bf(q_bits)
        qs = Shifted(x.shape, torch.bfloat16, q_shift, x)
        o, lse = Shifted((2, q, H, r), torch.bfloat16, o_shift), Shifted((2, q, H), torch.float32, o_shift)
        ws = torch.zeros(mla.mla_decode_workspace_size(d, 2, q, 400, ns), dtype=torch.uint8, device="cuda")
        fn(d, qs.t, cache, cu(f.table), cu(np.array(f.lens, np.int32)), 400, ws, o.t, lse.t, num_splits=ns)
        assert mla.mla_get_device_status(ws.view(torch.int32)[:1]) == mla.MLA_OK
        assert torch.equal(o.t, want[0]) and torch.equal(lse.t, want[1])
        assert o.outside_is_untouched() and lse.outside_is_untouched()


@pytest.mark.parametrize("shift", [8, 16, 24])
@pytest.mark.parametrize("H,n", [(4, 700), (96, 300)])
def test_prefill(H, n, shift):
    dn, dr, dv, q = 64, 16, 72, 150
    d = mla.make_dims(H, 1, 64, dn, dr, dv, 64, 0.11)
    x = {k: bf(v) for k, v in make(2, q, n, H, 1, dn, dr, dv, seed=shift).items()}
    lens, ql = cu(np.array([n, 200], np.int32)), cu(np.array([150, 99], np.int32))
    out = []
    for s in (0, shift):
        t = {k: Shifted(v.shape, torch.bfloat16, s, v).t for k, v in x.items()}
        o, lse = Shifted((2, q, H, dv), torch.bfloat16, s), Shifted((2, q, H), torch.float32, s // 8)
        mla.mla_prefill_attn(d, t["q"], t["k"], t["kr"], t["v"], lens, o.t, lse.t, q_lens=ql)
        assert o.outside_is_untouched() and lse.outside_is_untouched()
        out.append((o.t.clone(), lse.t.clone()))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    # an address that is not on 16 bytes is refused
    bad = Shifted(x["v"].shape, torch.bfloat16, 4, x["v"]).t
    with pytest.raises(mla.MlaError) as e:
        mla.mla_prefill_attn(d, x["q"], x["k"], x["kr"], bad, lens, out[0][0], out[0][1], q_lens=ql)
    assert e.value.status == mla.MLA_ERR_INVALID_ARG
