"""Infinities and NaN inside an attended context: a row that sees one gives NaN, whatever way the
sequence is cut, and a row that does not see it is as it would be without it."""
import numpy as np
import pytest
import torch

import head_latent_attention_attn_b200 as mla
from tests import q8_reference as Q
from tests.test_gpu_prefill_expanded import check, make, run
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


def number(bits):
    return float(Q.bf16_to_f64(np.array([bits], np.uint16))[0])


# heads, groups, d_n, d_r, d_v; query rows, keys, lengths, query lengths
PREFILL = {
    "clusters": (4, 1, 128, 64, 128, 77, 1100, [1100, 333, 77], [77, 70, 77]),
    "two_row_tiles": (2, 1, 64, 0, 64, 300, 700, [700, 301, 513], [300, 300, 130]),
    "odd": (3, 3, 96, 24, 72, 260, 260, [260, 200, 131], [260, 199, 131]),
    "short_of_rows": (2, 2, 40, 64, 128, 200, 150, [150, 3, 0], [200, 200, 200]),
    "many_units": (96, 1, 64, 16, 64, 300, 700, [700, 650, 257], [300, 257, 257]),
    "one_token": (4, 1, 16, 8, 16, 1, 130, [130, 1, 128], [1, 1, 1]),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", sorted(PREFILL))
def test_prefill_values_reach_only_rows_that_see_them(name, causal):
    """Infinities and NaN among the values of single tokens, at the chunk's borders and inside it: a row
    that sees one has it in that column, on top of what it has without (and NaN where both signs
    meet); every other number keeps its bits."""
    H, G, dn, dr, dv, q, n, lens, q_lens = PREFILL[name]
    d = mla.make_dims(H, G, 64, dn, dr, dv, 64, 1.0 / np.sqrt(dn + dr))
    x = make(len(lens), q, n, H, G, dn, dr, dv, seed=q)
    rng = np.random.default_rng(n)
    marks = []                                   # (sequence, token, head, column, bits)
    for b, (L, m) in enumerate(zip(lens, q_lens)):
        at = {L - 1, L - 2, L - m, L - m + 1, L - m + 63, L - m + 127, L - m + 128, L - m + 129,
              L - m + 255, L - m + 256, 0, L // 2}
        at |= {int(t) for t in rng.integers(max(L - m, 0), max(L, 1), 4)}
        marks += [(b, t, int(rng.integers(H)), int(rng.integers(dv)), bits)
                  for t in sorted(at) if 0 <= t < L for bits in (NAN, INF, NINF)]
    y = {k: v.copy() for k, v in x.items()}
    for b, t, h, c, bits in marks:
        x["v"][b, t, h, c] = 0
        y["v"][b, t, h, c] = bits
    o0, lse0, st0 = run(d, x, lens, q_lens, causal, packed=dr > 0)
    o, lse, st = run(d, y, lens, q_lens, causal, packed=dr > 0)
    assert st == st0 == mla.MLA_OK
    want, got = Q.bf16_to_f64(bits_of(o0)), Q.bf16_to_f64(bits_of(o))
    for b, t, h, c, bits in marks:
        L, m = lens[b], q_lens[b]
        last = L - m + np.arange(m) if causal else np.full(m, L - 1)
        with np.errstate(invalid="ignore"):
            want[b, :m, h, c] += np.where(last >= t, number(bits), 0.0)
    assert torch.equal(lse, lse0)
    bad = np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))
    assert bad.size == 0, f"{len(bad)} numbers differ, first {bad[:4].tolist()}"


@pytest.mark.parametrize("name", sorted(PREFILL))
def test_prefill_keys_reach_only_rows_that_see_them(name):
    """A NaN in a key, and one in a group's rotary key: o and lse are NaN in the rows that see it, and
    the others keep their bits."""
    H, G, dn, dr, dv, q, n, lens, q_lens = PREFILL[name]
    d = mla.make_dims(H, G, 64, dn, dr, dv, 64, 1.0 / np.sqrt(dn + dr))
    x = make(len(lens), q, n, H, G, dn, dr, dv, seed=q)
    o0, lse0, _ = run(d, x, lens, q_lens)
    y = {k: v.copy() for k, v in x.items()}
    sees = np.zeros((len(lens), q, H), bool)
    for b, (L, m) in enumerate(zip(lens, q_lens)):
        pos = L - m + np.arange(m)
        for t in {L - 1, L - (m + 1) // 2}:
            if 0 <= t < L:
                h = (t + b) % H
                y["k"][b, t, h, dn - 1] = NAN
                sees[b, :m, h] |= pos >= t
                if dr and t == L - 1:
                    g = (h + 1) % H // (H // G)
                    y["kr"][b, t, g, 0] = NAN
                    sees[b, :m, g * (H // G):(g + 1) * (H // G)] |= (pos >= t)[:, None]
    o, lse, st = run(d, y, lens, q_lens)
    assert st == mla.MLA_OK
    s = torch.from_numpy(sees).cuda()
    assert bool(torch.isnan(lse[s]).all()) and bool(torch.isnan(o[s].float()).all())
    assert torch.equal(lse[~s], lse0[~s]) and torch.equal(o[~s], o0[~s])


def test_prefill_units_after_one_with_bad_values():
    """A CTA that takes over units, and a unit with nothing bad right after one that has it: only the
    heads with bad values differ, over and over."""
    H, G, dn, dr, dv, q, n, lens, q_lens = PREFILL["many_units"]
    d = mla.make_dims(H, G, 64, dn, dr, dv, 64, 1.0 / np.sqrt(dn + dr))
    x = make(len(lens), q, n, H, G, dn, dr, dv, seed=5)
    o0, lse0, _ = run(d, x, lens, q_lens)
    y = {k: v.copy() for k, v in x.items()}
    heads = np.arange(0, H, 3)
    for b, L in enumerate(lens):
        y["v"][b, L - 1, heads] = NAN            # seen by the last row only
    for _ in range(5):
        o, lse, _ = run(d, y, lens, q_lens)
        assert torch.equal(lse, lse0)
        for b, m in enumerate(q_lens):
            assert bool(torch.isnan(o[b, m - 1, heads].float()).all())
            o[b, m - 1, heads] = o0[b, m - 1, heads]
        assert torch.equal(o, o0)


def test_prefill_of_many_short_prompts_with_garbage_behind_them():
    """Hundreds of units of one to three tiles, whose last tile ends inside or behind its context: the
    CTAs take over unit after unit while the tiles of the one before are still on their way."""
    H, G, dn, dr, dv, B, q = 96, 1, 64, 16, 64, 12, 300
    d = mla.make_dims(H, G, 64, dn, dr, dv, 64, 1.0 / np.sqrt(dn + dr))
    x = make(B, q, q, H, G, dn, dr, dv, seed=9)
    lens = [300, 1, 130, 128, 77, 256, 200, 257, 5, 129, 64, 260]
    for b, L in enumerate(lens):
        for k in ("k", "kr", "v"):
            x[k][b, L:] = NAN
        x["q"][b, L:] = NAN
    o0, lse0, st = run(d, x, lens, lens)
    assert st == mla.MLA_OK
    check(d, x, lens, lens, True, o0, lse0, [0, 47, 95])
    for _ in range(20):
        o, lse, _ = run(d, x, lens, lens)
        assert torch.equal(o, o0) and torch.equal(lse, lse0)


@pytest.mark.parametrize("name,q", [("deepseek_v2", 2), ("hybrid", 3), ("qwen3_30b_a3b", 1), ("rows_64", 1)])
def test_a_bad_query_row_stays_alone(name, q):
    """A NaN in one head's query (in either latent half): that row is NaN, and the others are what they
    are without it but for the roundings that a reference moved at other tiles brings: each side is
    within its bound of the formula, so they are within twice that of one another."""
    f = Filled(name, [700, 65], seed=3)
    H, G, r, dr = SHAPES[name]
    q_bits = f.query(q)
    clean = list(both(f, q_bits))
    kv = Q.rows(f.cache.cpu().numpy(), r, f.R)
    scale = float(np.float32(f.dims.softmax_scale))
    tol, lt = np.zeros((2, q * H, 1)), np.zeros((2, q * H))
    for b, L in enumerate(f.lens):
        row = kv[f.table[b, np.arange(L) // 64], np.arange(L) % 64]
        t, rel, d = bounds_of(Q.bf16_to_f64(q_bits)[b].reshape(q * H, -1), row, row[:, :r], scale)
        tol[b], lt[b] = t, d
    tol, lt = cu(tol.reshape(2, q, H, 1)), cu(lt.reshape(2, q, H))
    for col in (1, r - 1, r + f.R - 1):
        bad = q_bits.copy()
        bad[0, q - 1, H // 2, col] = NAN
        row = (0, q - 1, H // 2)
        for (o, lse), (o0, lse0) in zip(both(f, bad), clean):
            assert bool(torch.isnan(o[row].float()).all()) and bool(torch.isnan(lse[row]))
            o[row], lse[row] = o0[row], lse0[row]
            e = (o.double() - o0.double()).abs() - 2 * rel * o0.double().abs()
            assert bool((e <= 2 * tol).all())
            assert bool(((lse - lse0).abs() <= 2 * (lt + 2.0 ** -22 * lse0.abs())).all())
