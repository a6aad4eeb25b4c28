"""Infinities and NaN inside an attended context: a row that sees one gives NaN, whatever way the
sequence is cut, and a row that does not see it is as it would be without it."""
import numpy as np
import pytest
import torch

import head_latent_attention_attn_b200 as mla
from tests import q8_reference as Q
from tests.test_gpu_q8 import SHAPES, Filled, bf, bits_of, cu, decode, to_bits

pytestmark = pytest.mark.gpu

NAN, INF, NINF = 0x7FC1, 0x7F80, 0xFF80


def poison(f, b, pos, col, bits=NAN):
    """Latent column `col` of token `pos` of sequence b written again, as `bits`."""
    f.c_bits[b, pos, col] = bits
    B = len(f.lens)
    at, n = np.full(B, pos, np.int32), np.zeros(B, np.int32)
    n[b] = 1
    row = slice(pos, pos + 1)
    mla.mla_cache_append_q8(f.dims, bf(f.c_bits[:, row]), bf(f.k_bits[:, row]), cu(f.cos[:, row]),
                            cu(f.sin[:, row]), cu(f.table), cu(at), f.cache, new_lens=cu(n),
                            dev_error=f.err)


def both(f, q_bits, ns=0, causal=True):
    """(o, lse) over the 8-bit cache and over the bf16 cache of the same rows."""
    yield decode(f.dims, mla.mla_decode_attn_q8, q_bits, f.cache, f.table, f.lens, causal, ns)
    yield decode(f.dims, mla.mla_decode_attn, q_bits, f.bf16_cache(), f.table, f.lens, causal, ns)


@pytest.mark.parametrize("col", [5, 300])
@pytest.mark.parametrize("name", ["deepseek_v2", "qwen3_128"])
def test_a_bad_block_in_either_latent_half_reaches_every_row(name, col, monkeypatch):
    """Each CTA of the two-CTA kernel scores its half of the latent; the rows that the other owns get
    those scores packed. A NaN among them has to arrive as one."""
    monkeypatch.setitem(SHAPES, "qwen3_128", (128, 4, 512, 8))
    f = Filled(name, [200, 90], seed=1)
    q_bits = f.query(1)
    clean = list(both(f, q_bits, 1))
    poison(f, 0, 70, col)
    for (o, lse), (o0, lse0) in zip(both(f, q_bits, 1), clean):
        assert bool(torch.isfinite(o0.float()).all())
        assert bool(torch.isnan(o[0].float()).all())
        assert torch.equal(o[1], o0[1]) and torch.equal(lse[1], lse0[1])


@pytest.mark.parametrize("ns", [1, 3, 7, 20])
@pytest.mark.parametrize("name,q", [("hybrid", 1), ("qwen3_30b_a3b", 1), ("rows_64", 1), ("deepseek_v2", 1),
                                    ("pair_r256", 3)])
def test_a_bad_block_is_not_lost_with_its_piece(name, q, ns):
    """One context of 20 pages held whole, in 3 pieces (merged a warp a row), 7 and 20 (a block a row):
    a bad block in one of the pieces, then in every page, makes o and lse NaN whatever the cut."""
    f = Filled(name, [1280], seed=2)
    q_bits = f.query(q)
    for o, lse in both(f, q_bits, ns):
        assert bool(torch.isfinite(o.float()).all()) and bool(torch.isfinite(lse).all())
    poison(f, 0, 700, 3)
    for _ in range(2):
        for o, lse in both(f, q_bits, ns):
            assert bool(torch.isnan(lse).all()) and bool(torch.isnan(o.float()).all())
        for page in range(20):
            poison(f, 0, 64 * page, 60, INF)
