"""The 8-bit latent cache on the GPU: the append bit for bit against the byte-level definition,
the read-back exact, and the attention over it bit for bit equal to mla_decode_attn over the
same rows in bf16 and within the rounding bound of the 64-bit formula."""
import numpy as np
import pytest
import torch

import head_latent_attention_attn_b200 as mla
from tests import q8_reference as Q

pytestmark = pytest.mark.gpu

# name: heads, groups, rank, rotary width of a group
SHAPES = {
    "deepseek_v2": (128, 1, 512, 64),
    "qwen3_30b_a3b": (32, 4, 512, 8),
    "qwen25_7b": (28, 4, 128, 8),
    "hybrid": (16, 1, 256, 64),
    "one_head": (1, 1, 64, 8),
    "no_rope": (16, 1, 512, 0),
    "rank_448": (8, 1, 448, 64),
    "rows_64": (64, 1, 512, 64),          # one CTA with 64 query columns, no room to spare
    "rank_320": (128, 1, 320, 64),        # 64-row blocks of the one-CTA kernel
    "rank_192": (24, 2, 192, 24),
    "rope_128": (128, 4, 128, 32),        # the widest rotary part, two-CTA kernel
    "pair_r256": (96, 2, 256, 16),        # 96 of 128 rows, rotary half of 16
}


def dims_of(name, scale=0.1):
    H, G, r, dr = SHAPES[name]
    return mla.make_dims(H, G, r, 128, dr, 128, 64, scale)


def bf(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def to_bits(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Filled:
    """A cache of `lens` tokens a sequence in shuffled pages, written by the append; bytes that
    no token owns are 0xff (scales and keys of NaN)."""

    def __init__(self, name, lens, seed=0, size=1.0, spare=2):
        H, G, r, dr = SHAPES[name]
        self.name, self.lens, self.R = name, [int(x) for x in lens], G * dr
        self.dims = dims_of(name, 1.0 / np.sqrt(128 + dr))
        rng = self.rng = np.random.default_rng(seed)
        B, n = len(lens), max(lens)
        need = [(x + 63) // 64 for x in self.lens]
        self.P = sum(need) + spare
        perm = rng.permutation(self.P).astype(np.int32)
        self.table = np.full((B, max(need)), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m]
            at += m
        self.c_bits = to_bits(rng.standard_normal((B, n, r)) * size * np.exp(0.7 * rng.standard_normal(r)))
        self.k_bits = to_bits(rng.standard_normal((B, n, G, dr)))
        ang = rng.uniform(-30, 30, (B, n, G, dr // 2))
        self.cos, self.sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
        self.pages = np.full((self.P, Q.page_bytes(r, self.R)), 0xFF, np.uint8)
        self.cache = cu(self.pages)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.mla_cache_append_q8(self.dims, bf(self.c_bits), bf(self.k_bits), cu(self.cos),
                                cu(self.sin), cu(self.table), cu(np.zeros(B, np.int32)), self.cache,
                                new_lens=cu(np.array(self.lens, np.int32)), dev_error=self.err)

    def bf16_cache(self):
        """The same tokens in a bf16 cache (NaN elsewhere), through the read-back."""
        r, B, n = self.dims.kv_lora_rank, len(self.lens), max(self.lens)
        out = torch.empty((B, n, self.dims.row_width), dtype=torch.bfloat16, device="cuda")
        mla.mla_cache_read_q8(self.dims, self.cache, cu(self.table), cu(np.zeros(B, np.int32)), out,
                              read_lens=cu(np.array(self.lens, np.int32)), dev_error=self.err)
        full = torch.full((self.P, 64, self.dims.row_width), float("nan"), dtype=torch.bfloat16,
                          device="cuda")
        for b, L in enumerate(self.lens):
            pos = np.arange(L)
            full[torch.from_numpy(self.table[b, pos // 64]).long().cuda(),
                 torch.from_numpy(pos % 64).cuda()] = out[b, :L]
        return full

    def query(self, q, sigma=1.3):
        H, G, r, dr = SHAPES[self.name]
        D = r + self.R
        x = self.rng.standard_normal((len(self.lens), q, H, D)) * sigma * np.sqrt((128 + dr) / D)
        x[..., r:] *= (np.arange(self.R) // max(dr, 1))[None] == (np.arange(H) // (H // G))[:, None]
        return to_bits(x)


def decode(dims, fn, q_bits, cache, table, lens, causal=True, num_splits=0,
           size=mla.mla_decode_workspace_size):
    B, q, H, _ = q_bits.shape
    o = torch.full((B, q, H, dims.kv_lora_rank), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, q, H), 7.0, device="cuda")
    n = size(dims, B, q, max(lens), num_splits)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    fn(dims, bf(q_bits), cache, cu(table), cu(np.array(lens, np.int32)), max(lens), ws, o, lse,
       causal=causal, num_splits=num_splits)
    assert mla.mla_get_device_status(ws.view(torch.int32)[:1]) == mla.MLA_OK
    return o, lse


@pytest.mark.parametrize("name", ["deepseek_v2", "qwen25_7b", "hybrid", "no_rope", "rank_192"])
@pytest.mark.parametrize("n", [1, 5, 67, 200])
def test_append_is_the_definition(name, n):
    """Every byte of the cache: written tokens as defined, all other bytes as they were; a
    padded batch with a count of zero among its counts; zeros, the largest and smallest numbers,
    infinities and NaN among the values."""
    H, G, r, dr = SHAPES[name]
    rng = np.random.default_rng(n)
    B, P = 4, 40
    start = rng.integers(0, 150, B).astype(np.int32)
    lens = np.array([n, 0, n // 2, n], np.int32)
    maxp = int((start.max() + n + 63) // 64)
    table = rng.permutation(P)[:B * maxp].reshape(B, maxp).astype(np.int32)
    c = rng.standard_normal((B, n, r)) * np.exp(2 * rng.standard_normal((B, n, 1)))
    bits = to_bits(c)
    bits[0, 0, :64] = 0                                     # a block of zeros
    if r >= 128:
        bits[0, 0, 64:128] = rng.integers(0, 0x80, 64)      # only subnormals
    bits[3, 0, :64] = to_bits(np.full(64, 3.38e38))         # the largest: saturates
    bits[3, n - 1, :64] = to_bits(448 * 2.0 ** rng.integers(-9, 3, 64))   # powers on the border
    if n > 4:
        bits[0, 1, 5], bits[0, 2, 63], bits[0, 3, 0] = 0x7F80, 0xFF80, 0x7FC1
        bits[0, 4, :] = to_bits(np.tile([449.0, 480.0, 464.0, -465.0, 17.0, 0.0146, 2.0 ** -9, 2.0 ** -10], r // 8))
    k_bits = to_bits(rng.standard_normal((B, n, G, dr)) * 3)
    ang = rng.uniform(-40, 40, (B, n, G, dr // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    R = G * dr
    before = rng.integers(0, 256, (P, Q.page_bytes(r, R))).astype(np.uint8)
    want = Q.append(before, bits, k_bits, cos, sin, table, start, lens)
    cache, err = cu(before), torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_cache_append_q8(dims_of(name), bf(bits), bf(k_bits), cu(cos), cu(sin), cu(table),
                            cu(start), cache, new_lens=cu(lens), dev_error=err)
    got = cache.cpu().numpy()
    # a token's scale bytes past r / 64 hold nothing
    sc = slice(Q.PS * (r + 2 * R), None)
    a, b = got[:, sc].reshape(P, 64, 8), want[:, sc].reshape(P, 64, 8)
    assert np.array_equal(a[..., :r // 64], b[..., :r // 64])
    got[:, sc] = want[:, sc]
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{len(bad)} bytes differ, first {bad[:4].tolist()}"
    assert mla.mla_get_device_status(err) == mla.MLA_OK
    # a slot that no token was written to keeps all 8 of its scale bytes
    untouched = np.ones((P, 64), bool)
    for s in range(B):
        pos = start[s] + np.arange(lens[s])
        untouched[table[s, pos // 64], pos % 64] = False
    assert np.array_equal(a[untouched], before[:, sc].reshape(P, 64, 8)[untouched])


@pytest.mark.parametrize("name", ["deepseek_v2", "qwen25_7b", "no_rope", "rank_192", "rank_448", "one_head"])
@pytest.mark.parametrize("shift", [0, 1])
def test_append_of_many_tokens(name, shift):
    """Enough tokens for warps of several: every byte as defined, with counts that end inside a warp,
    a count out of range and pages that are not there; keys and angles that start on any element."""
    H, G, r, dr = SHAPES[name]
    R, B, n, P = G * dr, 5, 1003, 90
    rng = np.random.default_rng(shift + r)
    start = rng.integers(0, 70, B).astype(np.int32)
    lens = np.array([n, 0, 515, n + 1, n], np.int32)        # n + 1: appends none, flagged
    maxp = (70 + n + 63) // 64
    table = rng.permutation(P)[:B * maxp].reshape(B, maxp).astype(np.int32)
    table[0, 3], table[4, 5] = -1, P
    bits = to_bits(rng.standard_normal((B, n, r)) * np.exp(2 * rng.standard_normal((B, n, 1))))
    bits[0, :, 63], bits[2, 100, 0] = 0x7F80, 0x7FC1
    bits[4, 7] = 0x0003                                     # subnormals
    k_bits = to_bits(rng.standard_normal((B, n, G, dr)) * 3)
    ang = rng.uniform(-40, 40, (B, n, G, dr // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)

    def at(x):                                              # contiguous, `shift` elements in
        flat = torch.cat([x.new_zeros(shift), x.flatten()])
        return flat[shift:].view(x.shape)

    before = rng.integers(0, 256, (P, Q.page_bytes(r, R))).astype(np.uint8)
    want = Q.append(before, bits, k_bits, cos, sin, table, start, np.where(lens > n, 0, lens))
    cache, err = cu(before), torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_cache_append_q8(dims_of(name), bf(bits), at(bf(k_bits)), at(cu(cos)), at(cu(sin)),
                            cu(table), cu(start), cache, new_lens=cu(lens), dev_error=err)
    assert mla.mla_get_device_status(err) == mla.MLA_ERR_DEVICE_BOUNDS
    got = cache.cpu().numpy()
    sc = slice(Q.PS * (r + 2 * R), None)
    a, b = got[:, sc].reshape(P, 64, 8), want[:, sc].reshape(P, 64, 8)
    assert np.array_equal(a[..., :r // 64], b[..., :r // 64])
    written = np.zeros((P, 64), bool)
    for s in range(B):
        pos = start[s] + np.arange(0 if lens[s] > n else lens[s])
        page = table[s, pos // 64]
        ok = (page >= 0) & (page < P)
        written[page[ok], pos[ok] % 64] = True
    assert np.array_equal(a[~written], before[:, sc].reshape(P, 64, 8)[~written])
    got[:, sc] = want[:, sc]
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{len(bad)} bytes differ, first {bad[:4].tolist()}"


@pytest.mark.parametrize("dr", [2, 4, 12])
def test_append_of_narrow_groups(dr):
    """Rotary groups that four pairs at a time do not divide: the keys as defined."""
    G, r, B, n, P = 4, 64, 2, 2100, 70
    dims = mla.make_dims(8, G, r, 128, dr, 128, 64, 0.1)
    rng = np.random.default_rng(dr)
    table = rng.permutation(P)[:B * 34].reshape(B, 34).astype(np.int32)
    bits = to_bits(rng.standard_normal((B, n, r)))
    k_bits = to_bits(rng.standard_normal((B, n, G, dr)) * 3)
    ang = rng.uniform(-40, 40, (B, n, G, dr // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    for m in (9, n):
        before = rng.integers(0, 256, (P, Q.page_bytes(r, G * dr))).astype(np.uint8)
        zero = np.zeros(B, np.int32)
        want = Q.append(before, bits[:, :m], k_bits[:, :m], cos[:, :m], sin[:, :m], table, zero)
        cache = cu(before)
        mla.mla_cache_append_q8(dims, bf(bits[:, :m]), bf(k_bits[:, :m]), cu(cos[:, :m]), cu(sin[:, :m]),
                                cu(table), cu(zero), cache)
        keep = Q.PS * (r + 2 * G * dr)
        assert np.array_equal(cache.cpu().numpy()[:, :keep], want[:, :keep])


@pytest.mark.parametrize("name", ["deepseek_v2", "qwen3_30b_a3b", "no_rope", "rank_192", "one_head"])
@pytest.mark.parametrize("n,start", [(1, 63), (9, 60), (130, 0), (64, 1)])
def test_read_back_is_exact(name, n, start):
    """Rows of pages of random bytes (every code, every scale byte) are the values they stand
    for; rows at and past read_lens are left as they were."""
    H, G, r, dr = SHAPES[name]
    R, D, B, P = G * dr, SHAPES[name][2] + SHAPES[name][1] * SHAPES[name][3], 3, 16
    rng = np.random.default_rng(start + n)
    pages = rng.integers(0, 256, (P, Q.page_bytes(r, R))).astype(np.uint8)
    codes = pages[:, :Q.PS * r]
    codes[(codes & 127) == 127] = 0x7E                       # codes the append never writes
    sc = pages[:, Q.PS * (r + 2 * R):]
    sc[...] = np.where(sc < 17, 255, np.where((sc > 246) & (sc < 255), 246, sc))
    maxp = (start + n + 63) // 64
    table = rng.permutation(P)[:B * maxp].reshape(B, maxp).astype(np.int32)
    lens = np.array([n, n // 2, 0], np.int32)
    want = Q.rows(pages, r, R)
    out = torch.full((B, n, D), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_cache_read_q8(dims_of(name), cu(pages), cu(table), cu(np.full(B, start, np.int32)), out,
                          read_lens=cu(lens), dev_error=err)
    got = Q.bf16_to_f64(bits_of(out))
    for b in range(B):
        pos = start + np.arange(lens[b])
        ref = want[table[b, pos // 64], pos % 64]
        assert np.array_equal(got[b, :lens[b]], ref, equal_nan=True)
        assert np.all(got[b, lens[b]:] == 7.0)
    assert mla.mla_get_device_status(err) == mla.MLA_OK


@pytest.mark.parametrize("shift", [0, 8, 16, 24])
def test_read_back_to_rows_on_any_16_bytes(shift):
    """Rows that start `shift` bf16 numbers behind a 512-byte boundary: the same bits, and nothing
    outside them."""
    f = Filled("hybrid", [130, 64], seed=shift)
    B, n, D = 2, 130, f.dims.row_width
    buf = torch.full((B * n * D + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[shift:shift + B * n * D].view(B, n, D)
    lens = torch.tensor(f.lens, dtype=torch.int32, device="cuda")
    mla.mla_cache_read_q8(f.dims, f.cache, cu(f.table), torch.zeros_like(lens), out, read_lens=lens,
                          dev_error=f.err)
    want = Q.rows(f.cache.cpu().numpy(), 256, 64)
    got = Q.bf16_to_f64(bits_of(out))
    for b in range(B):
        pos = np.arange(f.lens[b])
        assert np.array_equal(got[b, :f.lens[b]], want[f.table[b, pos // 64], pos % 64])
        assert np.all(got[b, f.lens[b]:] == 7.0)
    assert torch.all(buf[:shift] == 7.0) and torch.all(buf[shift + B * n * D:] == 7.0)


def test_faults_are_flagged_and_skipped():
    """Bad page ids, positions past the table or below zero and counts outside [0, n] set the
    bounds bit; what they cover is not written or read, and the rest is."""
    name = "qwen25_7b"
    H, G, r, dr = SHAPES[name]
    R, D, n, P = G * dr, r + G * dr, 70, 8
    rng = np.random.default_rng(1)
    bits, k_bits = to_bits(rng.standard_normal((5, n, r))), to_bits(rng.standard_normal((5, n, G, dr)))
    cos = np.ones((5, n, G, dr // 2), np.float32)
    sin = np.zeros_like(cos)
    table = np.array([[0, 1], [2, P], [3, -1], [4, 5], [6, 7]], np.int32)
    start = np.array([0, 0, 0, -3, 64], np.int32)
    before = np.zeros((P, Q.page_bytes(r, R)), np.uint8)
    want = Q.append(before, bits, k_bits, cos, sin, table, start)
    cache, err = cu(before), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (bf(bits), bf(k_bits), cu(cos), cu(sin), cu(table), cu(start))
    mla.mla_cache_append_q8(dims_of(name), *args, cache, dev_error=err)
    assert mla.mla_get_device_status(err, reset=True) == mla.MLA_ERR_DEVICE_BOUNDS
    got = cache.cpu().numpy()
    lim = Q.PS * (r + 2 * R)
    assert np.array_equal(got[:, :lim], want[:, :lim])
    out = torch.full((5, n, D), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.mla_cache_read_q8(dims_of(name), cache, cu(table), cu(start), out, dev_error=err)
    assert mla.mla_get_device_status(err, reset=True) == mla.MLA_ERR_DEVICE_BOUNDS
    ref, o = Q.rows(want, r, R), Q.bf16_to_f64(bits_of(out))
    for b in range(5):
        for t in range(n):
            pos = int(start[b]) + t
            pg = table[b, pos // 64] if 0 <= pos < 128 else -1
            if 0 <= pg < P:
                assert np.array_equal(o[b, t], ref[pg, pos % 64])
            else:
                assert np.all(o[b, t] == 7.0)
    for lens in ([n + 1, 0, 0, 0, 0], [-1, 0, 0, 0, 0]):
        c2 = cu(before)
        mla.mla_cache_append_q8(dims_of(name), *args, c2, new_lens=cu(np.array(lens, np.int32)), dev_error=err)
        assert mla.mla_get_device_status(err, reset=True) == mla.MLA_ERR_DEVICE_BOUNDS
        assert not c2.any()
        out.fill_(7.0)
        mla.mla_cache_read_q8(dims_of(name), cache, cu(table), cu(start), out,
                              read_lens=cu(np.array(lens, np.int32)), dev_error=err)
        assert mla.mla_get_device_status(err, reset=True) == mla.MLA_ERR_DEVICE_BOUNDS
        assert bool((out == 7.0).all())


def bounds_of(q, k, v, scale):
    """How far o and lse may be off (per row): scores are fp32 sums of exact products (each
    partial sum of the two-CTA kernel rounded by 2^-16 of it), so a score is off by
    d <= 2^-15 max_l scale |q| . |k_l|; exp2 and log2 are approximations to about 2^-21. A weight
    is then off by d + 2^-8 (its bf16 rounding) relatively, and a piece and o by 2^-8 each."""
    s = scale * (np.abs(q) @ np.abs(k).T).max(-1)
    d = 2.0 ** -15 * s + 2.0 ** -20
    top = np.abs(v).max()
    return (2 * d + 2.0 ** -8 + 2.0 ** -14)[:, None] * top, 2.0 ** -7 * (1 + 2.0 ** -6), d


def check_attention(o, lse, q_bits, f, causal=True):
    """o, lse of all sequences against the 64-bit formula over the rows that the pages hold."""
    H, G, r, dr = SHAPES[f.name]
    kv = Q.rows(f.cache.cpu().numpy(), r, f.R)
    got, gl = Q.bf16_to_f64(bits_of(o)), lse.double().cpu().numpy()
    qf = Q.bf16_to_f64(q_bits)
    n_q = q_bits.shape[1]
    scale = float(np.float32(f.dims.softmax_scale))
    for b, L in enumerate(f.lens):
        pos = np.arange(L)
        row = kv[f.table[b, pos // 64], pos % 64]
        last = np.repeat(L - n_q + np.arange(n_q) if causal else np.full(n_q, L - 1), H)
        x = qf[b].reshape(n_q * H, -1)
        ro, rl = Q.attention(x, row, row[:, :r], scale, pos[None] <= last[:, None])
        tol, rel, d = bounds_of(x, row, row[:, :r], scale)
        e = np.abs(got[b].reshape(n_q * H, r) - ro) - rel * np.abs(ro)
        assert np.all(e <= tol), f"seq {b}: o is {(e / tol).max():.2f} of its bound"
        el = np.abs(gl[b].reshape(-1) - rl)
        lt = d + 2.0 ** -22 * np.abs(rl)
        assert np.all(el <= lt), f"seq {b}: lse is {(el / lt).max():.2f} of its bound"


CASES = [
    ("deepseek_v2", [517, 64, 65, 1, 200], 1, True),
    ("deepseek_v2", [300, 130], 3, True),
    ("qwen3_30b_a3b", [60, 1500, 63, 129, 1], 1, True),
    ("qwen3_30b_a3b", [200, 77], 2, False),
    ("qwen25_7b", [777, 64, 2], 1, True),
    ("hybrid", [3001, 12], 1, True),
    ("hybrid", [1000, 4], 4, True),
    ("hybrid", [333, 90], 77, True),
    ("one_head", [1, 2, 63, 700], 1, True),
    ("no_rope", [130, 64], 1, True),
    ("rank_448", [513, 3], 1, True),
    ("rows_64", [450, 65], 1, True),
    ("rank_320", [257, 64], 1, True),
    ("rank_192", [90, 400], 5, True),
    ("rope_128", [260, 31], 1, True),
    ("pair_r256", [191, 70], 1, True),
]


@pytest.mark.parametrize("name,lens,q,causal", CASES)
def test_decode_equals_bf16_cache_and_formula(name, lens, q, causal):
    f = Filled(name, lens, seed=q)
    q_bits = f.query(q)
    for ns in (0, 1, 3):
        o, lse = decode(f.dims, mla.mla_decode_attn_q8, q_bits, f.cache, f.table, f.lens, causal, ns)
        o2, lse2 = decode(f.dims, mla.mla_decode_attn, q_bits, f.bf16_cache(), f.table, f.lens, causal, ns)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), f"splits {ns}"
        check_attention(o, lse, q_bits, f, causal)
    assert mla.mla_get_device_status(f.err) == mla.MLA_OK


@pytest.mark.parametrize("name,lens,q,ns", [
    ("deepseek_v2", [300, 90, 80], 80, 0),       # one range a block: the rows lie over the partials
    ("deepseek_v2", [300, 5, 64], 4, 0),         # sequences cut between ranges: behind them
    ("deepseek_v2", [300, 5, 64], 4, 3),
    ("hybrid", [700, 33], 33, 0),
    ("rank_192", [130, 64], 9, 0),               # 64-row blocks of the one-CTA kernel
    ("deepseek_v2", [130, 64], 2, 0),            # two blocks: nothing to gain, the same size
])
def test_pages_converted_once(name, lens, q, ns):
    """The larger workspace gives the same bits, again and with what the last call left in it."""
    f = Filled(name, lens, seed=q)
    q_bits = f.query(q)
    plain = mla.mla_decode_workspace_size(f.dims, len(lens), q, max(lens), ns)
    large = mla.mla_decode_q8_workspace_size(f.dims, len(lens), q, max(lens), ns)
    assert large >= plain and (large > plain or q in (2, 80))
    want = decode(f.dims, mla.mla_decode_attn, q_bits, f.bf16_cache(), f.table, f.lens, True, ns)
    for _ in range(2):
        got = decode(f.dims, mla.mla_decode_attn_q8, q_bits, f.cache, f.table, f.lens, True, ns,
                     mla.mla_decode_q8_workspace_size)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    B, H, r = len(lens), f.dims.num_heads, f.dims.kv_lora_rank
    ws = torch.full((large,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    o = torch.empty((B, q, H, r), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, q, H), device="cuda")
    table = f.table.copy()
    for bad in (False, True):                    # a page id out of range: flagged, the others right
        if bad:
            table[1, 0] = f.P + 5
        mla.mla_decode_attn_q8(f.dims, bf(q_bits), f.cache, cu(table), cu(np.array(f.lens, np.int32)),
                               max(lens), ws, o, lse, num_splits=ns)
        st = mla.mla_get_device_status(ws.view(torch.int32)[:1], reset=True)
        assert st == (mla.MLA_ERR_DEVICE_BOUNDS if bad else mla.MLA_OK)
        for b in range(B):
            if not (bad and b == 1):
                assert torch.equal(o[b], want[0][b]) and torch.equal(lse[b], want[1][b])


@pytest.mark.parametrize("name", ["deepseek_v2", "qwen3_30b_a3b"])
@pytest.mark.parametrize("size,sigma", [(2.0 ** 14, 2.0 ** -13), (2.0 ** -60, 1.0), (8.0, 2.0)])
def test_decode_scale_range(name, size, sigma):
    """Scales above 2^7 (two factors), far below one, and a peaked softmax."""
    f = Filled(name, [150, 64], seed=4, size=size)
    q_bits = f.query(1, sigma=sigma)
    if size < 1:
        f.k_bits[...] = 0
    o, lse = decode(f.dims, mla.mla_decode_attn_q8, q_bits, f.cache, f.table, f.lens)
    o2, lse2 = decode(f.dims, mla.mla_decode_attn, q_bits, f.bf16_cache(), f.table, f.lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_attention(o, lse, q_bits, f)


def test_bad_page_and_length_are_flagged():
    f = Filled("qwen25_7b", [200, 130, 90], seed=2)
    q_bits = f.query(1)
    want, _ = decode(f.dims, mla.mla_decode_attn_q8, q_bits, f.cache, f.table, f.lens)
    for table, lens in ((f.table.copy(), list(f.lens)), (f.table, [f.lens[0], 300, f.lens[2]])):
        if lens == f.lens:
            table[1, 1] = f.P + 1000
        B = 3
        o = torch.empty((B, 1, 28, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((B, 1, 28), device="cuda")
        ws = torch.zeros(mla.mla_decode_workspace_size(f.dims, B, 1, 200), dtype=torch.uint8, device="cuda")
        mla.mla_decode_attn_q8(f.dims, bf(q_bits), f.cache, cu(table), cu(np.array(lens, np.int32)),
                               200, ws, o, lse)
        assert mla.mla_get_device_status(ws.view(torch.int32)[:1], reset=True) == mla.MLA_ERR_DEVICE_BOUNDS
        assert torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])


@pytest.mark.parametrize("name", ["deepseek_v2", "qwen3_30b_a3b"])
def test_graph_replay_and_side_streams(name):
    """Append and decode captured into a graph and replayed on other inputs; the same calls on
    two side streams at once with workspaces of their own."""
    f = Filled(name, [320, 70], seed=9)
    H, G, r, dr = SHAPES[name]
    q0 = bf(f.query(1))
    q1 = bf(f.query(1))
    table, lens = cu(f.table), cu(np.array(f.lens, np.int32))
    at = cu(np.array([x - 1 for x in f.lens], np.int32))
    c = [bf(to_bits(f.rng.standard_normal((2, 1, r)))) for _ in range(2)]
    k, cos, sin = bf(f.k_bits[:, :1]), cu(f.cos[:, :1]), cu(f.sin[:, :1])
    ws = [torch.zeros(mla.mla_decode_workspace_size(f.dims, 2, 1, 320), dtype=torch.uint8, device="cuda")
          for _ in range(3)]

    def step(cin, qin, o, lse, w, cache):
        mla.mla_cache_append_q8(f.dims, cin, k, cos, sin, table, at, cache)
        mla.mla_decode_attn_q8(f.dims, qin, cache, table, lens, 320, w, o, lse)

    def fresh():
        return (torch.zeros((2, 1, H, r), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((2, 1, H), device="cuda"))

    want = []
    for i in range(2):
        o, lse = fresh()
        step(c[i], (q0, q1)[i], o, lse, ws[0], f.cache)
        want.append((o.clone(), lse.clone()))
    assert not torch.equal(want[0][0], want[1][0])
    cin, qin, (o, lse) = c[0].clone(), q0.clone(), fresh()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(cin, qin, o, lse, ws[0], f.cache)
    for i in (0, 1, 0):
        cin.copy_(c[i])
        qin.copy_((q0, q1)[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [f.cache.clone() for _ in range(2)]
    outs = [fresh() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                step(c[i], (q0, q1)[i], *outs[i], ws[1 + i], caches[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])


@pytest.mark.parametrize("name,lens,q", [
    ("deepseek_v2", [4096] * 48, 1), ("qwen3_30b_a3b", [4096, 300, 1024, 2048] * 32, 1),
    ("rows_64", [3000, 500] * 24, 1), ("hybrid", [65536], 4)])
def test_long_runs_give_the_same_bits(name, lens, q):
    """Thousands of pages a call, where the warps of a CTA contend for shared memory and each
    other's buffers: every one of ten calls gives the bits of the bf16 cache."""
    f = Filled(name, lens, seed=3)
    q_bits = f.query(q)
    want = decode(f.dims, mla.mla_decode_attn, q_bits, f.bf16_cache(), f.table, f.lens)
    for i in range(10):
        got = decode(f.dims, mla.mla_decode_attn_q8, q_bits, f.cache, f.table, f.lens)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), f"call {i}"
