// append.cuh - one new token's cache row, written by one warp: the latent row moves as
// 16-byte vectors, the rotary pairs are rotated in fp32 (separately rounded multiply /
// subtract / add) and rounded to bf16 with ties to even. Used by cache_append_kernel and,
// folded into the query absorption, by the one-call decode step; the rotation also by the
// 8-bit cache's append.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

namespace mla {

// One rotary pair: fp32 with separately rounded products and sums, then bf16 with ties to even.
MLA_DEVICE void rotate_pair(uint16_t k0, uint16_t k1, float c, float s, uint16_t* y0, uint16_t* y1) {
  const float x0 = bf16_bits_to_f32(k0);
  const float x1 = bf16_bits_to_f32(k1);
  *y0 = f32_to_bf16_rne(__fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s)));
  *y1 = f32_to_bf16_rne(__fadd_rn(__fmul_rn(x1, c), __fmul_rn(x0, s)));
}

// Rotary key of every group of one token, by `lanes` lanes, one pair (x_j, x_{j + d_r/2}) per lane
// and step.
MLA_DEVICE void rotate_keys(const uint16_t* kr, const float* cs, const float* sn, int groups,
                            int rope_dim, int lane, uint16_t* dst, int lanes = 32) {
  const int half = rope_dim / 2;
  const int npairs = groups * half;
  for (int idx = lane; idx < npairs; idx += lanes) {
    const int g = idx / half;
    const int at = g * half + idx;             // g * rope_dim + j
    rotate_pair(kr[at], kr[at + half], cs[idx], sn[idx], &dst[at], &dst[at + half]);
  }
}

// Token gw = b * n_new + t of the batch (0 <= gw < batch * n_new); all 32 lanes call it.
MLA_DEVICE void append_token(const AppendParams& p, int64_t gw, int lane) {
  const int b = int(gw / p.n_new);
  const int t = int(gw - int64_t(b) * p.n_new);
  const int64_t pos = int64_t(p.start_pos[b]) + t;
  const int64_t lp = pos >= 0 ? pos / p.page_size : -1;
  if (pos < 0 || lp >= p.max_pages) {
    if (lane == 0 && p.dev_error) atomicOr(p.dev_error, MLA_DEVERR_BOUNDS);
    return;
  }
  const int32_t page = p.block_table[int64_t(b) * p.max_pages + lp];
  if (page < 0 || page >= p.num_pages) {
    if (lane == 0 && p.dev_error) atomicOr(p.dev_error, MLA_DEVERR_BOUNDS);
    return;
  }
  const int D = p.r + p.groups * p.rope_dim;
  uint16_t* dst = p.cache + (int64_t(page) * p.page_size + pos % p.page_size) * D;

  // latent: exact copy, 8 bf16 per 16-byte vector (r % 8 == 0, rows 16-byte aligned)
  const uint4* src4 = reinterpret_cast<const uint4*>(p.c_kv + gw * p.r);
  uint4* dst4 = reinterpret_cast<uint4*>(dst);
  for (int i = lane; i < p.r / 8; i += 32) dst4[i] = src4[i];

  const int64_t npairs = int64_t(p.groups) * (p.rope_dim / 2);
  rotate_keys(p.k_r + gw * 2 * npairs, p.rope_cos + gw * npairs, p.rope_sin + gw * npairs,
              p.groups, p.rope_dim, lane, dst + p.r);
}

}  // namespace mla
