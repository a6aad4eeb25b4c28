"""Sizes at the ends of what the calls of the 8-bit cache and the expanded prefill take: caches and
outputs whose offsets pass 32 bits, and calls with nothing to do."""
import numpy as np
import pytest
import torch

import head_latent_attention_attn_b200 as mla
from tests import q8_reference as Q
from tests.test_gpu_prefill_expanded import make, run
from tests.test_gpu_q8 import Filled, bf, bits_of, cu, decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["deepseek_v2", "hybrid"])
def test_pages_past_4_gib(name):
    """The same tokens in the last pages of a cache of more than 2^32 bytes: the append, the rows read
    back and the attention are those of a small cache."""
    f = Filled(name, [200, 65], seed=6)
    d, r = f.dims, f.dims.kv_lora_rank
    pages = 2 ** 32 // f.pages.shape[1] + 100
    shift = pages - f.P
    big = torch.zeros((pages, f.pages.shape[1]), dtype=torch.uint8, device="cuda")
    table = np.where(f.table >= 0, f.table + shift, -1).astype(np.int32)
    lens, zero = cu(np.array(f.lens, np.int32)), cu(np.zeros(2, np.int32))
    mla.mla_cache_append_q8(d, bf(f.c_bits), bf(f.k_bits), cu(f.cos), cu(f.sin), cu(table), zero, big,
                            new_lens=lens, dev_error=f.err)
    rows = [torch.zeros((2, 200, d.row_width), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    mla.mla_cache_read_q8(d, f.cache, cu(f.table), zero, rows[0], read_lens=lens, dev_error=f.err)
    mla.mla_cache_read_q8(d, big, cu(table), zero, rows[1], read_lens=lens, dev_error=f.err)
    assert torch.equal(rows[0], rows[1]) and bool(rows[0][0, 199, :r].any())
    q_bits = f.query(2)
    want = decode(d, mla.mla_decode_attn_q8, q_bits, f.cache, f.table, f.lens)
    got = decode(d, mla.mla_decode_attn_q8, q_bits, big, table, f.lens)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert mla.mla_get_device_status(f.err) == mla.MLA_OK


def test_rows_past_2_31_numbers():
    """A read-back of more than 2^31 numbers (one page over and over): the last rows as the first."""
    f = Filled("hybrid", [64], seed=7)
    n = 2 ** 31 // f.dims.row_width // 64 * 64 + 128
    table = torch.full((1, n // 64), int(f.table[0, 0]), dtype=torch.int32, device="cuda")
    out = torch.zeros((1, n, f.dims.row_width), dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_read_q8(f.dims, f.cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"), out,
                          dev_error=f.err)
    want = Q.rows(f.cache.cpu().numpy(), 256, 64)[f.table[0, 0]]
    for at in (0, n // 128 * 64, n - 64):
        assert np.array_equal(Q.bf16_to_f64(bits_of(out[0, at:at + 64])), want)
    assert mla.mla_get_device_status(f.err) == mla.MLA_OK


def test_prefill_outputs_past_2_31_numbers():
    """Query rows and outputs of more than 2^31 numbers over a short context, every row the same query:
    the rows that see all of it give the same bits, the last rows included."""
    H, dn, dv, L = 16, 128, 128, 130
    q = 2 ** 31 // (H * dv) + 300
    d = mla.make_dims(H, 1, 64, dn, 0, dv, 64, dn ** -0.5)
    g = torch.Generator("cuda")
    g.manual_seed(8)
    one = torch.randn((1, 1, H, dn), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((1, L, H, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    qs = one.expand(1, q, H, dn).contiguous()
    o = torch.zeros((1, q, H, dv), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((1, q, H), device="cuda")
    mla.mla_prefill_attn(d, qs, k, None, v, torch.tensor([L], dtype=torch.int32, device="cuda"), o, lse,
                         causal=False)
    p = torch.softmax(torch.einsum("hd,thd->ht", one[0, 0].double(), k[0].double()) * dn ** -0.5, -1)
    ref = torch.einsum("ht,thd->hd", p, v[0].double())
    # weights and o rounded to bf16 (2^-8 each), scores in fp32
    assert float((o[0, 0].double() - ref).abs().max()) <= 2.0 ** -7 * float(v.abs().max())
    for at in (q // 2, q - 300, q - 1):
        assert torch.equal(o[0, at], o[0, 0]) and torch.equal(lse[0, at], lse[0, 0])
    assert bool((o == o[:, :1]).all())


def test_nothing_to_do():
    """Batches of none, calls of no tokens and rows: accepted, nothing touched."""
    f = Filled("qwen25_7b", [70], seed=8)
    d, before = f.dims, f.cache.clone()
    H, G, r, dr = d.num_heads, d.num_kv_groups, d.kv_lora_rank, d.rope_dim
    table, zero = cu(f.table), torch.zeros(1, dtype=torch.int32, device="cuda")

    def bf16(*shape):
        return torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")

    def f32(*shape):
        return torch.full(shape, 7.0, device="cuda")

    mla.mla_cache_append_q8(d, bf16(1, 0, r), bf16(1, 0, G, dr), f32(1, 0, G, dr // 2), f32(1, 0, G, dr // 2),
                            table, zero, f.cache)
    mla.mla_cache_append_q8(d, bf16(0, 3, r), bf16(0, 3, G, dr), f32(0, 3, G, dr // 2), f32(0, 3, G, dr // 2),
                            table[:0], zero[:0], f.cache)
    mla.mla_cache_append_q8(d, bf16(1, 5, r), bf16(1, 5, G, dr), f32(1, 5, G, dr // 2), f32(1, 5, G, dr // 2),
                            table, zero, f.cache, new_lens=zero)
    mla.mla_cache_read_q8(d, f.cache, table, zero, bf16(1, 0, d.row_width))
    mla.mla_cache_read_q8(d, f.cache, table[:0], zero[:0], bf16(0, 4, d.row_width))
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    mla.mla_decode_attn_q8(d, bf16(0, 1, H, d.row_width), f.cache, table[:0], zero[:0], 70, ws, bf16(0, 1, H, r),
                           f32(0, 1, H))
    mla.mla_prefill_attn(d, bf16(0, 3, H, 128 + dr), bf16(0, 9, H, 128), bf16(0, 9, G, dr), bf16(0, 9, H, 128),
                         zero[:0], bf16(0, 3, H, 128), f32(0, 3, H))
    x = make(2, 5, 9, 4, 1, 128, 64, 128)
    o, lse, st = run(mla.make_dims(4, 1, 64, 128, 64, 128, 64, 0.1), x, [9, 0], [0, 0])
    assert st == mla.MLA_OK and bool((o == 7.0).all()) and bool((lse == 7.0).all())
    assert torch.equal(f.cache, before)
    assert mla.mla_get_device_status(ws.view(torch.int32)[:1]) == mla.MLA_OK


@pytest.mark.parametrize("name,q", [("deepseek_v2", 1), ("qwen3_30b_a3b", 4)])
def test_a_context_of_seconds_in_one_range(name, q):
    """One page over and over as a context of 130M tokens that one cluster works through alone, longer
    than a wait in the kernel may take: its last tile is waited for from the start."""
    f = Filled(name, [64], seed=9)
    d, H, r = f.dims, f.dims.num_heads, f.dims.kv_lora_rank
    n = 2_000_000 * 64 + 17
    table = torch.full((1, n // 64 + 1), int(f.table[0, 0]), dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    x = bf(f.query(q))
    ws = torch.zeros(mla.mla_decode_workspace_size(d, 1, q, n, 1), dtype=torch.uint8, device="cuda")
    for fn, cache in ((mla.mla_decode_attn_q8, f.cache), (mla.mla_decode_attn, f.bf16_cache())):
        o = torch.zeros((1, q, H, r), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((1, q, H), device="cuda")
        fn(d, x, cache, table, lens, n, ws, o, lse, num_splits=1)
        assert mla.mla_get_device_status(ws.view(torch.int32)[:1]) == mla.MLA_OK
        assert bool(torch.isfinite(o.float()).all()) and bool((lse > np.log(n) - 30).all())
