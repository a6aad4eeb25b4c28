"""mla_prefill_attn on the GPU against the 64-bit formula: head layouts, lengths around the
tile sizes, padded batches, rows that see nothing, garbage past a context, strides; and the run
of a chunk through the 8-bit cache (append, read back, expand, expanded attention) against the
absorbed attention over the same cache."""
import numpy as np
import pytest
import torch

import head_latent_attention_attn_b200 as mla
from tests import q8_reference as Q
from tests.test_gpu_q8 import SHAPES, Filled, bf, bits_of, cu, dims_of, to_bits

pytestmark = pytest.mark.gpu


def make(B, q, n, H, G, dn, dr, dv, seed=0, sigma=1.5):
    rng = np.random.default_rng(seed)
    t = {"q": rng.standard_normal((B, q, H, dn + dr)) * sigma,
         "k": rng.standard_normal((B, n, H, dn)), "kr": rng.standard_normal((B, n, G, dr)),
         "v": rng.standard_normal((B, n, H, dv))}
    return {k: to_bits(x) for k, x in t.items()}


def run(d, x, lens, q_lens=None, causal=True, packed=False, stream=None):
    B, q, H, _ = x["q"].shape
    dn, dv = d.qk_nope_dim, d.v_head_dim
    o = torch.full((B, q, H, dv), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, q, H), 7.0, device="cuda")
    k, v, kr = bf(x["k"]), bf(x["v"]), bf(x["kr"])
    if packed:                               # halves of one projection, columns of wider rows
        kv = torch.cat([k, v], -1)
        k, v = kv[..., :dn], kv[..., dn:]
        rows = torch.cat([torch.full_like(kr.flatten(2)[..., :1], float("nan")).expand(-1, -1, 16),
                          kr.flatten(2)], -1).contiguous()
        kr = rows[..., 16:].unflatten(-1, x["kr"].shape[2:])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_prefill_attn(d, bf(x["q"]), k, kr, v, cu(np.array(lens, np.int32)), o, lse,
                         q_lens=None if q_lens is None else cu(np.array(q_lens, np.int32)),
                         causal=causal, dev_error=err, stream=stream)
    return o, lse, mla.mla_get_device_status(err)


def check(d, x, lens, q_lens, causal, o, lse, heads=None):
    """Bounds: scores are fp32 sums of exact products, off by d <= 2^-20 scale |q|.|k| (192 terms
    of 2^-24 and the exponent's fma); exp2 and log2 are good to about 2^-21; a weight is rounded
    to bf16 while the sum is not, and o is rounded once more. bf16 has 8 significant bits: its
    step just above a power of two is 2^-7 of the value, so a rounding is off by up to half of
    that, 2^-8 of the value (torch.finfo(torch.bfloat16).eps / 2)."""
    B, q, H, _ = x["q"].shape
    G = x["kr"].shape[2]
    got, gl = Q.bf16_to_f64(bits_of(o)), lse.double().cpu().numpy()
    f = {k: Q.bf16_to_f64(v) for k, v in x.items()}
    scale = float(np.float32(d.softmax_scale))
    for b in range(B):
        L, m = lens[b], q if q_lens is None else q_lens[b]
        assert np.all(got[b, m:] == 7.0) and np.all(gl[b, m:] == 7.0), "rows past q_lens"
        if m == 0:
            continue
        pos = L - m + np.arange(m) if causal else np.full(m, L - 1)
        for h in (range(H) if heads is None else heads):
            key = np.concatenate([f["k"][b, :, h], f["kr"][b, :, h // (H // G)]], -1)[:L]
            val = f["v"][b, :L, h]
            seen = np.arange(L)[None] <= pos[:, None]
            ro, rl = Q.attention(f["q"][b, :m, h], key, val, scale, seen)
            gone = ~seen.any(1)
            assert np.all(got[b, :m, h][gone] == 0) and np.all(np.isneginf(gl[b, :m, h][gone]))
            here = ~gone
            if not here.any():
                continue
            s = scale * (np.abs(f["q"][b, :m, h]) @ np.abs(key).T).max(-1)
            e = 2.0 ** -20 * s + 2.0 ** -20
            tol = (2 * e + 2.0 ** -8 + 2.0 ** -14)[:, None] * np.abs(val).max()
            err = np.abs(got[b, :m, h] - ro) - 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(ro)
            assert np.all(err[here] <= tol[here]), f"b {b} h {h}: o is {(err / tol)[here].max():.2f} of its bound"
            el = np.abs(gl[b, :m, h][here] - rl[here])
            lt = (e + 2.0 ** -22 * np.abs(rl))[here]
            assert np.all(el <= lt), f"b {b} h {h}: lse is {(el / lt).max():.2f} of its bound"


# heads, groups, d_n, d_r, d_v
LAYOUTS = {"many": (96, 1, 64, 16, 64), "mla": (4, 1, 128, 64, 128), "grouped": (8, 4, 128, 8, 128), "no_rope": (2, 1, 64, 0, 64),
           "odd": (3, 3, 96, 24, 72), "tiny": (4, 1, 16, 8, 16), "wide_v": (2, 2, 40, 64, 128)}


def dims(name):
    H, G, dn, dr, dv = LAYOUTS[name]
    return mla.make_dims(H, G, 64, dn, dr, dv, 64, 1.0 / np.sqrt(dn + dr))


@pytest.mark.parametrize("name", sorted(set(LAYOUTS) - {"many"}))
@pytest.mark.parametrize("q,n,lens,q_lens,causal", [
    (1, 1, [1, 1], None, True),
    (1, 300, [300, 1], None, True),
    (5, 70, [70, 5], [5, 3], True),
    (128, 128, [128, 127], [128, 100], True),
    (129, 257, [257, 200], [129, 1], True),
    (256, 256, [256, 129], [256, 129], True),
    (300, 700, [700, 513], [300, 257], True),
    (77, 333, [333, 90], [60, 77], False),
    (300, 200, [200, 128], None, False),
])
def test_matches_the_formula(name, q, n, lens, q_lens, causal):
    H, G, dn, dr, dv = LAYOUTS[name]
    x = make(len(lens), q, n, H, G, dn, dr, dv, seed=q + n)
    d = dims(name)
    o, lse, st = run(d, x, lens, q_lens, causal)
    assert st == mla.MLA_OK
    check(d, x, lens, q_lens, causal, o, lse)
    o2, lse2, _ = run(d, x, lens, q_lens, causal, packed=dr % 8 == 0 and dr > 0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("name,q,n,lens,q_lens,causal,heads", [
    ("mla", 40, 2300, [2300, 130, 1000], [40, 3, 40], True, None),      # clusters of eight
    ("odd", 300, 1100, [1100, 300], [300, 130], True, None),            # of four, two row tiles
    ("no_rope", 129, 2100, [2100], None, False, None),
    ("many", 300, 700, [700, 650], [300, 257], True, [0, 37, 95]),      # more units than SMs
    ("many", 700, 700, [700, 0, 129, 400], [700, 300, 129, 0], True, [1, 64, 94]),
    ("many", 256, 1500, [1500, 1], None, False, [5, 90]),
])
def test_few_and_many_units(name, q, n, lens, q_lens, causal, heads):
    """Few query rows over a long context (the CTAs of a cluster share the tiles of a unit), and
    more units than SMs (CTAs take over units, of very different lengths)."""
    H, G, dn, dr, dv = LAYOUTS[name]
    x = make(len(lens), q, n, H, G, dn, dr, dv, seed=q + n)
    o, lse, st = run(dims(name), x, lens, q_lens, causal)
    assert st == mla.MLA_OK
    check(dims(name), x, lens, q_lens, causal, o, lse, heads)
    for _ in range(3):
        o2, lse2, _ = run(dims(name), x, lens, q_lens, causal)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H", [2, 9, 16, 20, 25, 33, 44, 60, 80])
@pytest.mark.parametrize("dv", [8, 72, 128])
def test_clusters_of_every_size(H, dv):
    """From eight CTAs a unit down to one as the heads grow, and values whose columns they do not
    share evenly; a sequence too short for each of them to have a tile."""
    x = make(1, 21, 2100, H, 1, 128, 8, dv, seed=H)
    d = mla.make_dims(H, 1, 64, 128, 8, dv, 64, 136 ** -0.5)
    for L, ql in ((2100, 21), (300, 5), (2100, 0)):
        o, lse, st = run(d, x, [L], [ql])
        assert st == mla.MLA_OK
        check(d, x, [L], [ql], True, o, lse, [0, H - 1])


def test_rows_that_see_nothing():
    """Contexts of zero, and shorter than the rows (whose first positions are negative)."""
    x = make(4, 200, 150, 4, 1, 128, 64, 128)
    for lens, q_lens, causal in (([0, 150, 3, 100], [200, 200, 200, 0], True),
                                 ([0, 150, 3, 100], [200, 0, 200, 7], False)):
        o, lse, st = run(dims("mla"), x, lens, q_lens, causal)
        assert st == mla.MLA_OK
        check(dims("mla"), x, lens, q_lens, causal, o, lse)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3.38e38])
def test_what_lies_past_a_context_is_not_used(fill):
    lens, q_lens = [130, 1, 255, 128], [130, 1, 200, 128]
    x = make(4, 200, 300, 4, 1, 128, 64, 128, seed=3)
    want = run(dims("mla"), x, lens, q_lens)
    y = {k: v.copy() for k, v in x.items()}
    bits = to_bits(np.array([fill]))[0]
    for b, L in enumerate(lens):
        for k in ("k", "kr", "v"):
            y[k][b, L:] = bits
        y["q"][b, q_lens[b]:] = bits
    got = run(dims("mla"), y, lens, q_lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("sigma", [8.0, 60.0])
def test_peaked_softmax(sigma):
    """Scores of hundreds: the reference moves, O is rescaled, single tokens take all weight."""
    x = make(2, 150, 900, 4, 1, 128, 64, 128, seed=5, sigma=sigma)
    x["q"][0, ::3] = 0                        # rows whose weights are all equal
    o, lse, _ = run(dims("mla"), x, [900, 400], [150, 99])
    check(dims("mla"), x, [900, 400], [150, 99], True, o, lse)


def test_increasing_scores_rescale_every_tile():
    """Keys that grow along the context: every tile moves the reference of every row."""
    x = make(1, 256, 1024, 2, 1, 64, 0, 64, seed=6)
    k = Q.bf16_to_f64(x["k"]) * 0.01 + 1.0
    x["k"] = to_bits(k * (1 + np.arange(1024) / 16)[None, :, None, None])
    x["q"] = to_bits(np.abs(Q.bf16_to_f64(x["q"])) * 0.2)
    d = mla.make_dims(2, 1, 64, 64, 0, 64, 64, 0.125)
    o, lse, _ = run(d, x, [1024], None)
    check(d, x, [1024], None, True, o, lse)


def test_bad_lengths_are_flagged():
    x = make(3, 40, 64, 4, 1, 128, 64, 128, seed=7)
    want = run(dims("mla"), x, [64, 64, 64])
    for lens, q_lens in (([64, 65, 64], None), ([64, -1, 64], None), ([64, 64, 64], [40, 41, 40]),
                         ([64, 64, 64], [40, -1, 40])):
        o, lse, st = run(dims("mla"), x, lens, q_lens)
        assert st == mla.MLA_ERR_DEVICE_BOUNDS
        assert torch.equal(o[0], want[0][0]) and torch.equal(o[2], want[0][2])
        seen = o[1].float()[0 if q_lens is None or q_lens[1] > 0 else 40:]
        assert bool((seen == 0).all())


@pytest.mark.parametrize("name", ["grouped", "many"])
def test_same_bits_again_in_a_graph_and_on_side_streams(name):
    """Few units (clusters) and more units than SMs (CTAs take over units)."""
    H, G, dn, dr, dv = LAYOUTS[name]
    x = make(2, 300, 600, H, G, dn, dr, dv, seed=8)
    lens, ql = [600, 280], [300, 280]
    d = dims(name)
    want = run(d, x, lens, ql)
    t = {k: bf(v) for k, v in x.items()}
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    sl, qs = cu(np.array(lens, np.int32)), cu(np.array(ql, np.int32))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_prefill_attn(d, t["q"], t["k"], t["kr"], t["v"], sl, o, lse, q_lens=qs)
    g.replay()
    torch.cuda.synchronize()
    for b in range(2):
        assert torch.equal(o[b, :ql[b]], want[0][b, :ql[b]])
    t["v"].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o[0], (want[0][0].float() * 2).to(torch.bfloat16))
    t["v"].mul_(0.5)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, (a, c) in zip(streams, outs):
            mla.mla_prefill_attn(d, t["q"], t["k"], t["kr"], t["v"], sl, a, c, q_lens=qs, stream=s)
    torch.cuda.synchronize()
    for a, c in outs:
        assert torch.equal(a, want[0]) and torch.equal(c, want[1])


@pytest.mark.parametrize("name", ["deepseek_v2", "qwen3_30b_a3b"])
def test_a_chunk_through_the_8_bit_cache(name):
    """The calls as a server makes them: a chunk is appended to a context in the 8-bit cache; the
    context is read back, its keys and values are expanded, and the chunk attends in the expanded
    form. The absorbed form over the same cache gives the same o and lse but for roundings."""
    H, G, r, dr = SHAPES[name]
    dn = dv = 128
    q, lens = 70, [290, 133]
    f = Filled(name, lens, seed=11)
    d, rng = f.dims, f.rng
    n, B = max(lens), len(lens)
    w_uk = bf(to_bits(rng.standard_normal((H, dn, r)) / np.sqrt(r)))
    w_uv = bf(to_bits(rng.standard_normal((H, dv, r)) / np.sqrt(r)))
    q_nope, q_pe = bf(to_bits(rng.standard_normal((B, q, H, dn)))), bf(to_bits(rng.standard_normal((B, q, H, dr))))
    pos = np.array(lens)[:, None] - q + np.arange(q)[None]
    th = 10000.0 ** (-2.0 * np.arange(dr // 2) / dr)
    ang = np.broadcast_to((pos[..., None] * th)[:, :, None], (B, q, G, dr // 2))
    cos, sin = cu(np.cos(ang).astype(np.float32)), cu(np.sin(ang).astype(np.float32))
    sl = cu(np.array(lens, np.int32))
    # absorbed
    q_ext = torch.empty((B, q, H, d.row_width), dtype=torch.bfloat16, device="cuda")
    mla.mla_absorb_q(d, q_nope, q_pe, cos, sin, w_uk, q_ext)
    ws = torch.zeros(mla.mla_decode_workspace_size(d, B, q, n), dtype=torch.uint8, device="cuda")
    o_lat = torch.empty((B, q, H, r), dtype=torch.bfloat16, device="cuda")
    lse_a = torch.empty((B, q, H), device="cuda")
    o_a = torch.empty((B, q, H, dv), dtype=torch.bfloat16, device="cuda")
    mla.mla_decode_attn_q8(d, q_ext, f.cache, cu(f.table), sl, n, ws, o_lat, lse_a)
    mla.mla_out_up(d, o_lat, w_uv, o_a)
    # expanded
    rows = torch.zeros((B, n, d.row_width), dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_read_q8(d, f.cache, cu(f.table), cu(np.zeros(B, np.int32)), rows, read_lens=sl)
    c = rows[..., :r].contiguous()[:, :, None].expand(B, n, H, r).contiguous()
    k, v = (torch.empty((B, n, H, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mla.mla_out_up(d, c, w_uk, k)
    mla.mla_out_up(d, c, w_uv, v)
    # the rotated query is the absorbed query's slot of the head's group
    g = torch.arange(H, device="cuda") // (H // G)
    rot = q_ext[..., r:].unflatten(-1, (G, dr))[:, :, torch.arange(H, device="cuda"), g]
    o_e, lse_e = torch.empty_like(o_a), torch.empty_like(lse_a)
    mla.mla_prefill_attn(d, torch.cat([q_nope, rot], -1).contiguous(), k, rows[..., r:].unflatten(-1, (G, dr)), v,
                         sl, o_e, lse_e)
    assert mla.mla_get_device_status(ws.view(torch.int32)[:1]) == mla.MLA_OK
    # Roundings to bf16 (2^-8 at most, 2^-8 / sqrt(3) in the mean square) that only one side has:
    # o_lat, its pieces, o_a, k, v, o_e, the absorbed query, and the weights of each side; eight
    # of them add up to less than 2^-8 sqrt(8 / 3) of o in the 2-norm, and scores that differ by
    # 2^-8 sqrt(2 / 3) |s| (|s| < 6) / sqrt(128) to less than that again.
    a, e = o_a.float(), o_e.float()
    assert float((a - e).norm() / e.norm()) <= 2 * 2.0 ** -8 * (8 / 3) ** 0.5
    assert float((lse_a - lse_e).abs().max()) <= 2.0 ** -8 * 6
