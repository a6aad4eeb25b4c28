"""The 8-bit latent cache and attention over it in numpy, from their definitions: the byte
layout of a page, quantisation with exact arithmetic in 64 bits, the values that pages stand
for, and masked softmax attention in 64 bits. Shares no code with the library."""
from __future__ import annotations

import numpy as np

PS = 64
E_MIN, E_MAX = -110, 119


def page_bytes(r: int, R: int) -> int:
    return PS * (r + 2 * R + 8)


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16_bits(x: np.ndarray) -> np.ndarray:
    """Values that fit in bf16 exactly, as bits."""
    f = np.asarray(x, dtype=np.float32)
    u = f.view(np.uint32)
    assert not np.any(u[np.isfinite(f)] & 0xFFFF), "not a bf16 value"
    return (u >> 16).astype(np.uint16)


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (NaN for 0x7f and 0xff)."""
    c = np.arange(256)
    ex, man = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (8.0 + man) * 2.0 ** (ex - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def quantise(c_bits: np.ndarray):
    """(codes uint8 [..., r], scale bytes uint8 [..., r/64]) of bf16 bits [..., r]."""
    x = bf16_to_f64(c_bits).reshape(*c_bits.shape[:-1], -1, 64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(-1)
    e = np.full(amax.shape, E_MIN)
    for cand in range(E_MAX, E_MIN - 1, -1):      # least e of the range with amax 2^-e <= 448
        e = np.where(amax <= 448.0 * 2.0 ** cand, cand, e)
    e = np.where(amax > 448.0 * 2.0 ** E_MAX, E_MAX, e)
    z = np.abs(x) * 2.0 ** -e[..., None].astype(np.float64)
    # positive codes are ordered like their values: nearest, ties to the even code
    vals = e4m3_values()[:127]
    hi = np.clip(np.searchsorted(vals, z, side="left"), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dh, dl = np.abs(vals[hi] - z), np.abs(z - vals[lo])
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    sign = (c_bits.reshape(x.shape) >> 15).astype(np.int64)
    code = np.where(bad[..., None], 0, code | (sign << 7))
    byte = np.where(bad, 255, e + 127)
    return code.astype(np.uint8).reshape(c_bits.shape), byte.astype(np.uint8)


def rotate_bits(k_bits, cos, sin):
    """bf16 bits of the rotated keys [..., G, d_r] (fp32, separately rounded, ties to even)."""
    half = k_bits.shape[-1] // 2
    x = (k_bits.astype(np.uint32) << 16).view(np.float32)
    x0, x1 = x[..., :half], x[..., half:]
    y = np.concatenate([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).astype(np.float32)
    u = y.view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def append(pages, c_bits, k_bits, cos, sin, table, start, new_lens=None):
    """pages uint8 [P, bytes] after the append (a copy)."""
    pages = pages.copy()
    B, n, r = c_bits.shape
    R = k_bits.shape[2] * k_bits.shape[3]
    codes, scales = quantise(c_bits)
    keys = rotate_bits(k_bits, cos, sin).reshape(B, n, R).view(np.uint8) if R else None
    for b in range(B):
        for t in range(n if new_lens is None else int(new_lens[b])):
            pos = int(start[b]) + t
            if pos < 0 or pos // PS >= table.shape[1]:
                continue
            pg, s = int(table[b, pos // PS]), pos % PS
            if not 0 <= pg < pages.shape[0]:
                continue
            row = pages[pg]
            for k in range(r // 64):
                at = k * PS * 64 + s * 64
                row[at:at + 64] = codes[b, t, 64 * k:64 * k + 64]
            if R:
                at = PS * r + s * 2 * R
                row[at:at + 2 * R] = keys[b, t]
            at = PS * (r + 2 * R) + 8 * s
            row[at:at + r // 64] = scales[b, t]
    return pages


def rows(pages, r, R):
    """fp64 rows [P, 64, r + R] that pages stand for."""
    P = pages.shape[0]
    c = e4m3_values()[pages[:, :PS * r]].reshape(P, r // 64, PS, 64)
    sc = pages[:, PS * (r + 2 * R):].reshape(P, PS, 8)[..., :r // 64].astype(np.float64)
    f = np.where(sc == 255, np.nan, 2.0 ** (sc - 127.0))
    lat = (c * f.transpose(0, 2, 1)[..., None]).transpose(0, 2, 1, 3).reshape(P, PS, r)
    k = np.ascontiguousarray(pages[:, PS * r:PS * (r + 2 * R)]).view(np.uint16).reshape(P, PS, R)
    return np.concatenate([lat, bf16_to_f64(k)], -1)


def attention(q, k, v, scale, seen):
    """o [rows, dv], lse [rows] of softmax(scale q k^T) v in 64 bits over the tokens `seen`
    [rows, tokens]; a row that sees nothing gives zeros and -inf. Unseen tokens do not enter."""
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.where(seen, scale * (q @ np.where(seen.any(0)[:, None], k, 0.0).T), -np.inf)
    m = s.max(-1, keepdims=True, initial=-np.inf)
    p = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = p.sum(-1, keepdims=True)
    o = (p / np.where(l > 0, l, 1.0)) @ np.where(seen.any(0)[:, None], v, 0.0)
    lse = np.where(l > 0, np.where(np.isfinite(m), m, 0.0) + np.log(np.where(l > 0, l, 1.0)), -np.inf)
    return o, lse[:, 0]
