"""What is measured of the 8-bit latent cache and of the expanded prefill attention.

Four operators, each in its plain form (elementary torch operations in 32 bits, ``own`` false)
and as a user calls it through the package (``own`` true):

* write:   mla_cache_append_q8, then mla_cache_read_q8 of the rows just written. A cache row's
           latent is held as e4m3 codes with one power-of-two scale per 64 columns, so what
           comes back is the values that the codes stand for, with the rotated keys (bf16).
* read:    mla_cache_read_q8 of a stretch of every sequence, dequantised to bf16 rows.
* decode:  mla_decode_attn_q8, the absorbed attention of q new rows over the paged 8-bit cache.
* prefill: mla_prefill_attn, the same attention in its expanded form (a key and a value per
           head, the rotary key shared by the heads of a group) over a padded batch.

A page of the 8-bit cache holds 64 tokens: the latent codes in blocks of 64 columns
([r/64][64 tokens][64]), the rotated keys ([64 tokens][R] bf16), and 8 scale bytes a token
(exponent + 127 of column block k in byte k; 255 marks a block with a non-finite value).
"""
import math
import random

import torch

own = False

PS = 64            # tokens a page
E_MIN, E_MAX = -110, 119

# heads, key groups, rank, nope width, rotary width of a group, value width
SHAPES = {
    "deepseek_v2": (128, 1, 512, 128, 64, 128),
    "qwen3_30b_a3b": (32, 4, 512, 128, 8, 128),
    "qwen25_7b": (28, 4, 128, 128, 8, 128),
    "hybrid": (16, 1, 256, 128, 64, 128),
}


def listed():
    return [
        # one decode step's new rows of a 64-sequence batch at context 8192: launch latency
        {"name": "write_step_64", "op": "write", "shape": "deepseek_v2", "batch": 64, "n": 1,
         "start": 8191, "ragged": False},
        # prompts stored chunk by chunk, of uneven lengths in a padded batch
        {"name": "write_prompts_4x4097", "op": "write", "shape": "deepseek_v2", "batch": 4, "n": 4097,
         "start": 0, "ragged": True},
        # a few short prefixes fetched for the next chunk
        {"name": "read_3x1000", "op": "read", "shape": "qwen3_30b_a3b", "batch": 3, "n": 1000,
         "start": 37, "ragged": True},
        # one long document's whole context
        {"name": "read_1m", "op": "read", "shape": "hybrid", "batch": 1, "n": 1 << 20, "start": 0,
         "ragged": False},
        # one user, a short context: latency
        {"name": "decode_1x1000", "op": "decode", "shape": "hybrid", "batch": 1, "q": 1, "ctx": 1000,
         "lo": 1000},
        # steady serving of the 128-head layer
        {"name": "decode_64x8192", "op": "decode", "shape": "deepseek_v2", "batch": 64, "q": 1,
         "ctx": 8192, "lo": 8192},
        # a large batch of uneven contexts
        {"name": "decode_128_ragged", "op": "decode", "shape": "qwen3_30b_a3b", "batch": 128, "q": 1,
         "ctx": 32768, "lo": 1024},
        # four drafted tokens over one very long context
        {"name": "decode_1m_q4", "op": "decode", "shape": "hybrid", "batch": 1, "q": 4,
         "ctx": 1 << 20, "lo": 1 << 20},
        # a chunk of new tokens over the paged cache
        {"name": "decode_chunk_256", "op": "decode", "shape": "deepseek_v2", "batch": 1, "q": 256,
         "ctx": 4096, "lo": 4096},
        # a small odd padded batch
        {"name": "prefill_3x77", "op": "prefill", "shape": "hybrid", "batch": 3, "q": 77, "ctx": 333,
         "causal": True},
        # a chunk over a longer context, 128 heads
        {"name": "prefill_1024_of_4096", "op": "prefill", "shape": "deepseek_v2", "batch": 1, "q": 1024,
         "ctx": 4096, "causal": True},
        # whole prompts at once, grouped rotary keys
        {"name": "prefill_2x4096", "op": "prefill", "shape": "qwen3_30b_a3b", "batch": 2, "q": 4096,
         "ctx": 4096, "causal": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    tops = {}
    for c in listed():
        w = work(c)
        tops[c["op"]] = max(tops.get(c["op"], 0.0), w["bytes"] / 6e12 + w["flops"] / 1.2e15)
    op = rng.choice(["write", "read", "decode", "decode", "prefill", "prefill"])
    while True:
        c = {"op": op, "shape": rng.choice(sorted(SHAPES))}
        if op in ("write", "read"):
            c.update(batch=_log(rng, 1, 64), n=_log(rng, 1, 1 << 16), start=rng.randrange(0, 300),
                     ragged=rng.random() < 0.6)
        elif op == "decode":
            ctx = _log(rng, 64, 1 << 19)
            q = rng.choice([1, 1, 1, 2, 3, 5, _log(rng, 8, 300)])
            ctx = max(ctx, q)
            c.update(batch=_log(rng, 1, 128), q=q, ctx=ctx,
                     lo=ctx if rng.random() < 0.4 else max(q, ctx // 16))
        else:
            q = _log(rng, 1, 4096)
            c.update(batch=_log(rng, 1, 8), q=q, ctx=q + rng.choice([0, rng.randrange(0, 5000)]),
                     causal=rng.random() < 0.8)
        w = work(c)
        if w["bytes"] / 6e12 + w["flops"] / 1.2e15 <= 0.9 * tops[op]:
            return c


# ---- what a case says, apart from any seed ---------------------------------------------------

def _lens(case):
    """Lengths of a case's sequences: (rows written, read or queried, context), by the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B = case["batch"]
    if case["op"] in ("write", "read"):
        n = case["n"]
        rows = [rng.randrange(0, n + 1) if case["ragged"] else n for _ in range(B)]
        rows[rng.randrange(B)] = n
        return rows, [case["start"] + x for x in rows]
    if case["op"] == "decode":
        lens = [rng.randint(case["lo"], case["ctx"]) for _ in range(B)]
        lens[rng.randrange(B)] = case["ctx"]
        return [case["q"]] * B, lens
    rows = [rng.randint((case["q"] + 1) // 2, case["q"]) for _ in range(B)]
    rows[0] = case["q"]
    lens = [rng.randint(x, case["ctx"]) for x in rows]
    lens[0] = case["ctx"]
    return rows, lens


def work(case):
    H, G, r, dn, dr, dv = SHAPES[case["shape"]]
    R, D, nb = G * dr, r + G * dr, r // 64
    rows, lens = _lens(case)
    row8 = r + 2 * R + nb
    if case["op"] == "write":     # read the new rows and angles, write the codes, read them, write rows
        return {"bytes": sum(rows) * (2 * D + 4 * R + 2 * row8 + 2 * D), "flops": 0}
    if case["op"] == "read":
        return {"bytes": sum(rows) * (row8 + 2 * D), "flops": 0}
    if case["op"] == "decode":
        q = case["q"]
        seen = sum(q * L - q * (q - 1) // 2 for L in lens)
        return {"bytes": sum(lens) * row8 + len(lens) * q * H * (2 * D + 2 * r + 4),
                "flops": 2 * seen * H * (D + r)}
    seen = sum(x * L - x * (x - 1) // 2 if case["causal"] else x * L for x, L in zip(rows, lens))
    return {"bytes": sum(rows) * H * (2 * (dn + dr) + 2 * dv + 4)
            + sum(lens) * (2 * H * (dn + dv) + 2 * R), "flops": 2 * seen * H * (dn + dr + dv)}


# ---- inputs -----------------------------------------------------------------------------------

def _angles(B, n, start, G, dr, dev):
    """cos and sin [B, n, G, dr/2] of each pair's angle at positions start .. start + n - 1."""
    j = torch.arange(dr // 2, dtype=torch.float64, device=dev)
    theta = 10000.0 ** (-2.0 * j / dr)
    ang = (start + torch.arange(n, dtype=torch.float64, device=dev))[:, None, None] * theta
    ang = ang.expand(n, G, dr // 2)[None].expand(B, n, G, dr // 2)
    return ang.cos().float().contiguous(), ang.sin().float().contiguous()


def _latents(g, shape, dev):
    """Normed latents: rows of unit size whose columns differ in size."""
    x = torch.randn(shape, generator=g, device=dev)
    return (x * torch.exp(0.5 * torch.randn(shape[-1], generator=g, device=dev))).to(torch.bfloat16)


def _make_pages(g, num_pages, r, R, dev):
    """Pages as a filled cache holds them: every token's latent quantised, its keys beside it."""
    pages = torch.zeros(num_pages, PS * (r + 2 * R + 8), dtype=torch.uint8, device=dev)
    for p0 in range(0, num_pages, 4096):
        p1 = min(num_pages, p0 + 4096)
        codes, e = _quantise(_latents(g, (p1 - p0, PS, r), dev).float())
        keys = torch.randn(p1 - p0, PS, R, generator=g, device=dev).to(torch.bfloat16)
        lat, key, sc = _planes(pages[p0:p1], r, R)
        lat.copy_(codes.view(p1 - p0, PS, r // 64, 64).transpose(1, 2))
        key.copy_(keys)
        sc[..., :r // 64] = (e + 127).to(torch.uint8)
    return pages


def _table(g, lens, dev, spare=3):
    """A shuffled block table for contexts `lens` and the number of pages; -1 past a context."""
    need = [-(-max(x, 1) // PS) for x in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    at = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=dev)
    k = 0
    for b, m in enumerate(need):
        at[b, :m] = perm[k:k + m]
        k += m
    return at, total


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev)
    g.manual_seed(seed)
    H, G, r, dn, dr, dv = SHAPES[case["shape"]]
    R, D, B = G * dr, r + G * dr, case["batch"]
    rows, lens = _lens(case)
    s = {"op": case["op"], "dims": SHAPES[case["shape"]], "scale": (dn + dr) ** -0.5}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if case["op"] in ("write", "read"):
        n = case["n"]
        s["table"], total = _table(g, [case["start"] + n] * B, dev)
        s["start"], s["rows"] = i32([case["start"]] * B), i32(rows)
        s["out"] = torch.zeros(B, n, D, dtype=torch.bfloat16, device=dev)
        if case["op"] == "write":
            s["cache"] = torch.zeros(total, PS * (r + 2 * R + 8), dtype=torch.uint8, device=dev)
            s["c_kv"] = _latents(g, (B, n, r), dev)
            s["k_r"] = torch.randn(B, n, G, dr, generator=g, device=dev).to(torch.bfloat16)
            s["cos"], s["sin"] = _angles(B, n, case["start"], G, dr, dev)
        else:
            s["cache"] = _make_pages(g, total, r, R, dev)
        return s
    s["lens"] = i32(lens)
    if case["op"] == "decode":
        q = case["q"]
        s["table"], total = _table(g, lens, dev)
        s["cache"] = _make_pages(g, total, r, R, dev)
        s["max_len"] = max(lens)
        qe = torch.randn(B, q, H, D, generator=g, device=dev) * (1.3 * math.sqrt((dn + dr) / D))
        group = torch.arange(H, device=dev) // (H // G)
        slot = (torch.arange(R, device=dev) // dr)[None, :] == group[:, None]
        qe[..., r:] *= slot
        s["q"] = qe.to(torch.bfloat16)
        s["o"] = torch.zeros(B, q, H, r, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(B, q, H, device=dev)
        if own:
            import head_latent_attention_attn_b200 as mla
            s["ws"] = torch.zeros(mla.mla_decode_workspace_size(_dims(s), B, q, s["max_len"]),
                                  dtype=torch.uint8, device=dev)
        return s
    q, n = case["q"], case["ctx"]
    s["rows"], s["causal"] = i32(rows), case["causal"]
    s["q"] = (1.5 * torch.randn(B, q, H, dn + dr, generator=g, device=dev)).to(torch.bfloat16)
    # the up-projection of a packed weight leaves [k_nope | v] of a head side by side
    kv = torch.randn(B, n, H, dn + dv, generator=g, device=dev).to(torch.bfloat16)
    s["k_nope"], s["v"] = kv[..., :dn], kv[..., dn:]
    row = torch.randn(B, n, D, generator=g, device=dev).to(torch.bfloat16)   # cache rows read back
    s["k_pe"] = row[..., r:].unflatten(-1, (G, dr))
    s["o"] = torch.zeros(B, q, H, dv, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros(B, q, H, device=dev)
    return s


# ---- plain forms ------------------------------------------------------------------------------

def _planes(pages, r, R):
    """Views of pages [P, bytes]: codes [P, r/64, 64, 64] e4m3, keys [P, 64, R] bf16, scales [P, 64, 8]."""
    P = pages.shape[0]
    a, b = PS * r, PS * (r + 2 * R)
    lat = pages[:, :a].unflatten(1, (r // 64, PS, 64)).view(torch.float8_e4m3fn)
    keys = pages[:, a:b].view(torch.bfloat16).view(P, PS, R)
    return lat, keys, pages[:, b:].unflatten(1, (PS, 8))


def _quantise(x):
    """e4m3 codes of x [..., r] and the exponent of every 64 columns (finite x)."""
    y = x.unflatten(-1, (-1, 64))
    amax = y.abs().amax(-1)
    m, e = torch.frexp(amax)                      # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)     # least e with amax 2^-e <= 448
    e = torch.where(amax == 0, torch.full_like(e, E_MIN), e).clamp(E_MIN, E_MAX)
    return torch.ldexp(y, -e[..., None]).to(torch.float8_e4m3fn).flatten(-2), e


def _rows32(pages, r, R):
    """Rows [P, 64, r + R] fp32 that pages [P, bytes] stand for."""
    lat, keys, sc = _planes(pages, r, R)
    e = sc[..., :r // 64].to(torch.int32) - 127
    x = torch.ldexp(lat.float().transpose(1, 2), e[..., None]).flatten(-2)
    return torch.cat([x, keys.float()], -1)


def _plain_read(s):
    H, G, r, dn, dr, dv = s["dims"]
    R = G * dr
    B, n = s["out"].shape[:2]
    t = torch.arange(n, device=s["out"].device)
    pos = s["start"].long()[:, None] + t                                    # [B, n]
    page, slot = s["table"].gather(1, pos // PS).long(), pos % PS
    lat, keys, sc = _planes(s["cache"], r, R)
    x = lat.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()   # [B, n, r/64, 64]
    e = sc[page, slot, :r // 64].to(torch.int32) - 127
    got = torch.cat([torch.ldexp(x, e[..., None]).to(torch.bfloat16).flatten(-2), keys[page, slot]], -1)
    return torch.where((t < s["rows"][:, None])[..., None], got, s["out"])


def _plain_write(s):
    H, G, r, dn, dr, dv = s["dims"]
    R, half = G * dr, dr // 2
    B, n = s["c_kv"].shape[:2]
    codes, e = _quantise(s["c_kv"].float())
    x0, x1 = s["k_r"][..., :half].float(), s["k_r"][..., half:].float()
    key = torch.cat([x0 * s["cos"] - x1 * s["sin"], x1 * s["cos"] + x0 * s["sin"]], -1)
    t = torch.arange(n, device=codes.device)
    pos = s["start"].long()[:, None] + t
    b, k = torch.nonzero(t < s["rows"][:, None], as_tuple=True)
    at = pos[b, k]
    page, slot = s["table"][b, at // PS].long(), at % PS
    lat, keys, sc = _planes(s["cache"], r, R)
    lat.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)[b, k].unflatten(-1, (-1, 64))
    keys[page, slot] = key.to(torch.bfloat16).view(B, n, R)[b, k]
    sc[page, slot, :r // 64] = (e + 127).to(torch.uint8)[b, k]
    return _plain_read(s)


def _softmax(x, seen):
    """Softmax of x over its last dim where `seen`, and the logarithm of its sum; zeros and -inf
    where a row sees nothing."""
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    return p / torch.where(l > 0, l, torch.ones_like(l)), lse[..., 0]


def _plain_decode(s):
    H, G, r, dn, dr, dv = s["dims"]
    R = G * dr
    B, q = s["q"].shape[:2]
    rows = _rows32(s["cache"][s["table"].clamp(min=0).long().flatten()], r, R).view(B, -1, r + R)
    x = torch.bmm(s["q"].float().view(B, q * H, r + R), rows.transpose(1, 2)) * s["scale"]
    t = torch.arange(rows.shape[1], device=x.device)
    last = s["lens"].long()[:, None] - q + torch.arange(q, device=x.device)   # [B, q]
    seen = (t <= last[..., None])[:, :, None].expand(B, q, H, -1).reshape(x.shape)
    p, lse = _softmax(x, seen)
    o = torch.bmm(p, rows[..., :r])
    return o.to(torch.bfloat16).view(B, q, H, r), lse.view(B, q, H)


def _plain_prefill(s):
    H, G, r, dn, dr, dv = s["dims"]
    B, q = s["q"].shape[:2]
    n = s["v"].shape[1]
    dev = s["q"].device
    keys = torch.cat([s["k_nope"], s["k_pe"].repeat_interleave(H // G, 2)], -1).float()
    x = torch.matmul(s["q"].float().transpose(1, 2), keys.permute(0, 2, 3, 1)) * s["scale"]
    i, t = torch.arange(q, device=dev), torch.arange(n, device=dev)
    L, rows = s["lens"].long()[:, None, None], s["rows"].long()[:, None, None]
    last = L - rows + i[:, None] if s["causal"] else L - 1
    seen = ((t <= last) & (t < L)).expand(B, q, n)[:, None]
    p, lse = _softmax(x, seen)
    o = torch.matmul(p, s["v"].float().transpose(1, 2)).transpose(1, 2).to(torch.bfloat16)
    real = i < rows[..., 0]                                                   # [B, q]
    return (torch.where(real[..., None, None], o, s["o"]),
            torch.where(real[..., None], lse.transpose(1, 2), s["lse"]))


# ---- one pass ---------------------------------------------------------------------------------

def _dims(s):
    import head_latent_attention_attn_b200 as mla
    H, G, r, dn, dr, dv = s["dims"]
    return mla.make_dims(H, G, r, dn, dr, dv, PS, s["scale"])


def run(s):
    if not own:
        return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode,
                "prefill": _plain_prefill}[s["op"]](s)
    import head_latent_attention_attn_b200 as mla
    dims = _dims(s)
    if s["op"] == "write":
        mla.mla_cache_append_q8(dims, s["c_kv"], s["k_r"], s["cos"], s["sin"], s["table"],
                                s["start"], s["cache"], new_lens=s["rows"])
    if s["op"] in ("write", "read"):
        mla.mla_cache_read_q8(dims, s["cache"], s["table"], s["start"], s["out"],
                              read_lens=s["rows"])
        return s["out"]
    if s["op"] == "decode":
        mla.mla_decode_attn_q8(dims, s["q"], s["cache"], s["table"], s["lens"], s["max_len"],
                               s["ws"], s["o"], s["lse"])
    else:
        mla.mla_prefill_attn(dims, s["q"], s["k_nope"], s["k_pe"], s["v"], s["lens"], s["o"],
                             s["lse"], q_lens=s["rows"], causal=s["causal"])
    return s["o"], s["lse"]


# ---- the definition in 64 bits ----------------------------------------------------------------

def _exact_page_rows(pages, r, R):
    """Rows [P, 64, r + R] fp64 of pages, from the bits of their bytes."""
    P = pages.shape[0]
    c = pages[:, :PS * r].reshape(P, r // 64, PS, 64).to(torch.int64)
    sign, ex, man = 1.0 - 2.0 * (c >> 7).double(), (c >> 3) & 15, (c & 7).double()
    val = torch.where(ex == 0, man * 2.0 ** -9, (8.0 + man) * torch.exp2((ex - 10).double()))
    sc = pages[:, PS * (r + 2 * R):].reshape(P, PS, 8)[..., :r // 64].double()
    lat = (sign * val) * torch.exp2(sc - 127.0).transpose(1, 2)[..., None]
    k = pages[:, PS * r:PS * (r + 2 * R)].reshape(P, PS, R, 2).to(torch.int64)
    bits = ((k[..., 1] << 8 | k[..., 0]) << 16).to(torch.int32)
    return torch.cat([lat.transpose(1, 2).reshape(P, PS, r), bits.view(torch.float32).double()], -1)


def _exact_quantised(x):
    """What x [..., r] stands for after e4m3 with a power of two per 64 columns."""
    y = x.double().reshape(*x.shape[:-1], -1, 64)
    big = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(big.clamp(min=2.0 ** -200) / 448.0))
    e = torch.where(big * torch.exp2(-(e - 1)) <= 448.0, e - 1, e)
    e = torch.where(big * torch.exp2(-e) > 448.0, e + 1, e).clamp(E_MIN, E_MAX)
    z = y * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(z / step) * step * torch.exp2(e)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    H, G, r, dn, dr, dv = s["dims"]
    R, D = G * dr, r + G * dr
    rows, lens = _lens(case)
    dev = s["table"].device if "table" in s else s["q"].device
    if s["op"] == "write":
        lat = _exact_quantised(s["c_kv"])
        z = torch.complex(s["k_r"][..., :dr // 2].double(), s["k_r"][..., dr // 2:].double())
        z = z * torch.complex(s["cos"].double(), s["sin"].double())
        out = torch.cat([lat, torch.cat([z.real, z.imag], -1).flatten(-2)], -1)
        for b, m in enumerate(rows):
            out[b, m:] = 0
        return out
    if s["op"] == "read":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
        for b, m in enumerate(rows):
            if m:
                st = case["start"]
                got = _exact_page_rows(s["cache"][s["table"][b, :-(-(st + m) // PS)].long()], r, R)
                out[b, :m] = got.reshape(-1, D)[st:st + m]
        return out
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=dev)
    for b, (m, L) in enumerate(zip(rows, lens)):
        if s["op"] == "decode":
            kv = _exact_page_rows(s["cache"][s["table"][b, :-(-L // PS)].long()], r, R)
            kv = kv.reshape(-1, D)[:L]
        for h in ([slice(0, H)] if s["op"] == "decode" and m * H <= 512 else
                  [slice(k, k + 1) for k in range(H)]):
            qh = s["q"][b, :m, h].double()                                     # [m, heads, d]
            if s["op"] == "decode":
                x = torch.einsum("qhd,td->qht", qh, kv)
            else:
                key = torch.cat([s["k_nope"][b, :L, h.start], s["k_pe"][b, :L, h.start // (H // G)]], -1)
                x = (qh[:, 0] @ key.double().T)[:, None]
            x = x * s["scale"]
            if case.get("causal", True):
                hide = torch.ones(m, L, dtype=torch.bool, device=dev).triu(L - m + 1)
                x.masked_fill_(hide[:, None], -math.inf)
            lse[b, :m, h] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[b, :m, h, None])
            val = kv[:, :r] if s["op"] == "decode" else s["v"][b, :L, h.start].double()
            o[b, :m, h] = torch.einsum("qht,tc->qhc", p, val)
    return o, lse
