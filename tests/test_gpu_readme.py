"""The README's prefill chunk over an 8-bit cache, run as it stands there."""
import os
import re

import numpy as np
import pytest
import torch

import head_latent_attention_attn_b200 as mla
from tests.test_gpu_q8 import bf, cu, to_bits

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("H,G,r,d_n,d_r,d_v", [(8, 2, 128, 64, 16, 96), (16, 1, 256, 128, 64, 128)])
def test_expanded_chunk(H, G, r, d_n, d_r, d_v):
    """Its o and lse are the absorbed form's (its last call, over the same cache) but for roundings, for
    value and key widths that differ as well."""
    text = open(os.path.join(ROOT, "README.md")).read()
    code = re.search(r"A prefill chunk over an 8-bit cache.*?```python\n(.*?)```", text, re.S).group(1)
    rng = np.random.default_rng(r)
    B, q, L = 2, 70, 70
    dims = mla.make_dims(H, G, r, d_n, d_r, d_v, 64, (d_n + d_r) ** -0.5)
    th = 10000.0 ** (-2.0 * np.arange(d_r // 2) / d_r)
    ang = np.broadcast_to((np.arange(q)[:, None] * th)[None, :, None], (B, q, G, d_r // 2))
    cos, sin = cu(np.cos(ang).astype(np.float32)), cu(np.sin(ang).astype(np.float32))
    new = lambda *shape: bf(to_bits(rng.standard_normal(shape)))  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    empty = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    s = dict(torch=torch, mla=mla, dims=dims, B=B, n=L, H=H, G=G, r=r, d_n=d_n, d_r=d_r, d_v=d_v, num_pages=5,
             c_kv_new=new(B, q, r), k_r_new=new(B, q, G, d_r), cos_new=cos, sin_new=sin, cos_q=cos, sin_q=sin,
             q_nope=new(B, q, H, d_n), q_pe=new(B, q, H, d_r),
             w_uk=bf(to_bits(rng.standard_normal((H, d_n, r)) / np.sqrt(r))),
             w_uv=bf(to_bits(rng.standard_normal((H, d_v, r)) / np.sqrt(r))),
             block_table=ints([[3, 1], [0, 4]]), start_pos=ints([0, 0]), q_lens=ints([q, q]),
             seq_lens=ints([L, L]), max_seq_len=L, q_ext=empty(B, q, H, r + G * d_r), o=empty(B, q, H, d_v),
             o_latent=empty(B, q, H, r), lse=torch.empty((B, q, H), device="cuda"),
             ws=torch.zeros(mla.mla_decode_workspace_size(dims, B, q, L), dtype=torch.uint8, device="cuda"))
    before, after = code.split("# later tokens")
    exec(before, s)
    o, lse = s["o"].clone(), s["lse"].clone()
    exec("# later tokens" + after, s)
    assert mla.mla_get_device_status(s["ws"].view(torch.int32)[:1]) == mla.MLA_OK
    o_a = torch.empty_like(o)
    mla.mla_out_up(dims, s["o_latent"], s["w_uv"], o_a)
    # Roundings to bf16 (2^-8 at most, 2^-8 / sqrt(3) in the mean square) that only one side has: o_lat,
    # its pieces, o_a, k, v, o, the absorbed query, and the weights of each side; eight of them add up
    # to less than 2^-8 sqrt(8 / 3) of o in the 2-norm, and scores that differ by 2^-8 sqrt(2 / 3) |s|
    # (|s| < 6) / sqrt(64) to less than that again.
    a, e = o_a.float(), o.float()
    assert float((a - e).norm() / e.norm()) <= 2 * 2.0 ** -8 * (8 / 3) ** 0.5
    assert float((s["lse"] - lse).abs().max()) <= 2.0 ** -8 * 6
