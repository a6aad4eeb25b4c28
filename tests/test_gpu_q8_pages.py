"""The 8-bit cache's pages as a whole: the same tokens give the same bytes however they were appended."""
import numpy as np
import pytest

import head_latent_attention_attn_b200 as mla
from tests import q8_reference as Q
from tests.test_gpu_q8 import SHAPES, Filled, bf, check_attention, cu, decode, dims_of, to_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["deepseek_v2", "rank_320", "rank_448", "rank_192", "qwen25_7b", "one_head"])
def test_pages_do_not_depend_on_the_call(name):
    """5000 tokens in one call, in calls of a few and a token at a time: every byte of the pages is
    equal, the scale bytes past r / 64 are zero, and bytes of slots that hold no token stay."""
    H, G, r, dr = SHAPES[name]
    R, n, P = G * dr, 5000, 80
    rng = np.random.default_rng(r)
    table = rng.permutation(P)[:79].reshape(1, 79).astype(np.int32)
    bits = to_bits(rng.standard_normal((1, n, r)) * np.exp(2 * rng.standard_normal((1, n, 1))))
    bits[0, 17, 3] = 0x7F80
    k_bits = to_bits(rng.standard_normal((1, n, G, dr)))
    ang = rng.uniform(-40, 40, (1, n, G, dr // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    before = rng.integers(0, 256, (P, Q.page_bytes(r, R))).astype(np.uint8)
    start = 3
    want = Q.append(before, bits, k_bits, cos, sin, table, np.array([start]))
    sc = want[:, Q.PS * (r + 2 * R):].reshape(P, 64, 8)
    pos = start + np.arange(n)
    rest = sc[table[0, pos // 64], pos % 64]
    rest[:, r // 64:] = 0
    sc[table[0, pos // 64], pos % 64] = rest
    for cuts in ([0, n], [0, 4096, 4100, n], [0, 1, 2, 3, 1000, 1001, n]):
        cache = cu(before)
        for a, b in zip(cuts, cuts[1:]):
            mla.mla_cache_append_q8(dims_of(name), bf(bits[:, a:b]), bf(k_bits[:, a:b]), cu(cos[:, a:b]),
                                    cu(sin[:, a:b]), cu(table), cu(np.array([start + a], np.int32)), cache)
        bad = np.argwhere(cache.cpu().numpy() != want)
        assert bad.size == 0, f"cuts {cuts}: {len(bad)} bytes differ, first {bad[:4].tolist()}"


@pytest.mark.parametrize("name", ["deepseek_v2", "qwen3_30b_a3b", "rank_192"])
@pytest.mark.parametrize("power", [-100, -60, 14, 100])
def test_attention_over_any_scale(name, power):
    """Latents of about 2^power and queries of about 2^-power, without keys: scores of order one that
    come from the scaled codes alone, so that o, lse and the softmax tell a wrong scale."""
    f = Filled(name, [150, 64], seed=4, size=2.0 ** power)
    B = len(f.lens)
    f.k_bits[...] = 0
    mla.mla_cache_append_q8(f.dims, bf(f.c_bits), bf(f.k_bits), cu(f.cos), cu(f.sin), cu(f.table),
                            cu(np.zeros(B, np.int32)), f.cache, new_lens=cu(np.array(f.lens, np.int32)),
                            dev_error=f.err)
    q_bits = to_bits(Q.bf16_to_f64(f.query(1)) * 2.0 ** -power)
    o, lse = decode(f.dims, mla.mla_decode_attn_q8, q_bits, f.cache, f.table, f.lens)
    check_attention(o, lse, q_bits, f)
    spread = lse.max() - lse.min()
    assert float(spread) > 1e-3, "scores that say nothing"
    assert mla.mla_get_device_status(f.err) == mla.MLA_OK
