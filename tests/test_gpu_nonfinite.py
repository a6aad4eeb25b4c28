"""Infinities and NaN inside an attended context: a row that sees one gives NaN, whatever way the
sequence is cut, and a row that does not see it is as it would be without it."""
import numpy as np
import pytest
import torch

import head_latent_attention_attn_b200 as mla
from tests import q8_reference as Q
from tests.test_gpu_q8 import SHAPES, Filled, bf, bits_of, bounds_of, cu, decode

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


def rows_that_see_nothing_bad_are_clean(f, q_bits, o, lse, clean, bad, what):
    """`bad`: {sequence: first bad position}. Rows that see it are NaN; the others are within the
    bound of the 64-bit formula over the finite rows `clean`, whose other tokens they share."""
    H, G, r, dr = SHAPES[f.name]
    n_q = q_bits.shape[1]
    got, gl = Q.bf16_to_f64(bits_of(o)), lse.double().cpu().numpy()
    scale = float(np.float32(f.dims.softmax_scale))
    qf = Q.bf16_to_f64(q_bits)
    for b, L in enumerate(f.lens):
        pos = np.arange(L)
        row = clean[f.table[b, pos // 64], pos % 64]
        last = np.repeat(L - n_q + np.arange(n_q), H)
        x = qf[b].reshape(n_q * H, -1)
        ro, rl = Q.attention(x, row, row[:, :r], scale, pos[None] <= last[:, None])
        tol, rel, d = bounds_of(x, row, row[:, :r], scale)
        g, l = got[b].reshape(n_q * H, r), gl[b].reshape(-1)
        sees = last >= bad.get(b, L)
        assert np.isnan(g[sees]).all() and np.isnan(l[sees]).all(), what
        assert np.isfinite(g[~sees]).all() and np.isfinite(l[~sees]).all(), what
        assert np.all((np.abs(g - ro) - rel * np.abs(ro))[~sees] <= tol[~sees]), what
        assert np.all(np.abs(l - rl)[~sees] <= (d + 2.0 ** -22 * np.abs(rl))[~sees]), what


@pytest.mark.parametrize("ns", [0, 1, 3])
@pytest.mark.parametrize("name,q,lens", [
    ("hybrid", 4, [1000, 130, 4]), ("hybrid", 77, [333, 90]), ("qwen3_30b_a3b", 2, [200, 65]),
    ("qwen25_7b", 2, [64, 300]), ("rank_448", 5, [70, 513]), ("rank_192", 9, [90, 400]),
    ("deepseek_v2", 3, [300, 67]), ("deepseek_v2", 80, [300, 100]), ("pair_r256", 2, [191, 66]),
    ("no_rope", 6, [69, 70])])
def test_a_bad_block_does_not_reach_rows_that_do_not_see_it(name, q, lens, ns):
    """The chunk's own tokens: the last one bad in one sequence, one in the middle in another. Over
    the 8-bit cache, with its pages converted first, and over the bf16 cache (NaN; infinities too)."""
    f = Filled(name, lens, seed=q)
    r = f.dims.kv_lora_rank
    q_bits = f.query(q)
    clean = Q.rows(f.cache.cpu().numpy(), r, f.R)
    bad = {0: lens[0] - 1, 1: lens[1] - q + (q + 1) // 2}
    poison(f, 0, bad[0], r - 1)
    poison(f, 1, bad[1], 0, INF)
    for i, (o, lse) in enumerate(both(f, q_bits, ns)):
        rows_that_see_nothing_bad_are_clean(f, q_bits, o, lse, clean, bad, f"cache {i}")
    o, lse = decode(f.dims, mla.mla_decode_attn_q8, q_bits, f.cache, f.table, f.lens, True, ns,
                    mla.mla_decode_q8_workspace_size)
    rows_that_see_nothing_bad_are_clean(f, q_bits, o, lse, clean, bad, "converted first")
    # infinities among finite numbers in a bf16 cache: a score of +inf or NaN (as the query's signs
    # make it) or -inf, whose weight is zero
    full = torch.from_numpy(clean).to(torch.bfloat16).cuda()
    for b, t in bad.items():
        full[f.table[b, t // 64], t % 64, [0, r - 1]] = torch.tensor([float("inf"), float("-inf")]).to(full)
    o, lse = decode(f.dims, mla.mla_decode_attn, q_bits, full, f.table, f.lens, True, ns)
    H = f.dims.num_heads
    for b, L in enumerate(lens):
        sees = torch.arange(L - q, L) >= bad.get(b, L)
        assert bool(torch.isfinite(o[b, ~sees].float()).all()) and bool(torch.isfinite(lse[b, ~sees]).all())
