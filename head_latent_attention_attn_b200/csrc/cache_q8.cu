// cache_q8.cu - mla_cache_append_q8 and mla_cache_read_q8: new tokens quantised into the paged
// 8-bit latent cache (q8.cuh), and stretches of it read back as bf16 rows.
//
// Append, one warp per token: a lane holds 8 columns (16 bytes) of each half of 256 columns, so
// the 8 lanes of a 64-column block find its largest magnitude with three shuffles on the bf16
// bits, and codes of a block leave as 64 consecutive bytes. Both directions are bound by memory:
// a token is 2 r + 2 R bytes in and r + 2 R + r/64 out (or the reverse).
//
// Read, one warp per 8 tokens: a lane takes 16 codes of one token from each column block (the
// warp reads 512 consecutive bytes of a block when the tokens share a page), all loads issued
// before the first use, and writes 32 consecutive bytes; four lanes make a full 128-byte line. One
// 32-byte store fills a sector of L2 where two of 16 bytes visit it twice (rows that start on
// 16-byte boundaries only still need those), and the keys' loads go out with the codes': 1M rows of
// 256 + 64 columns take 166 us (6.5 TB/s), 181 with a loop over the keys before the first
// conversion, 191 with 16-byte stores too. Six blocks an SM instead of four: 206 (spills).
#include "append.cuh"
#include "q8.cuh"

namespace mla {

// Page and slot of position pos of sequence b; false (and the bounds bit) when outside.
MLA_DEVICE bool q8_locate(const int32_t* block_table, int32_t max_pages, int64_t num_pages,
                          int32_t* dev_error, int b, int64_t pos, int64_t* page, int* slot) {
  const int64_t lp = pos >= 0 ? pos / kQ8Tok : -1;
  int64_t pg = -1;
  if (lp >= 0 && lp < max_pages) pg = block_table[int64_t(b) * max_pages + lp];
  if (pg < 0 || pg >= num_pages) {
    if (dev_error) atomicOr(dev_error, MLA_DEVERR_BOUNDS);
    return false;
  }
  *page = pg;
  *slot = int(pos % kQ8Tok);
  return true;
}

// Rows of sequence b that a call covers: all n, or the caller's count if it is within [0, n]
// (else none, and the bounds bit).
MLA_DEVICE int q8_rows(const int32_t* lens, int b, int n, int32_t* dev_error) {
  if (lens == nullptr) return n;
  const int m = lens[b];
  if (m >= 0 && m <= n) return m;
  if (dev_error) atomicOr(dev_error, MLA_DEVERR_BOUNDS);
  return 0;
}

__global__ void __launch_bounds__(256) cache_append_q8_kernel(AppendQ8Params p) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t gw = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (gw >= int64_t(p.batch) * p.n_new) return;
  const int b = int(gw / p.n_new);
  const int t = int(gw - int64_t(b) * p.n_new);
  if (t >= q8_rows(p.new_lens, b, p.n_new, lane == 0 && t == 0 ? p.dev_error : nullptr)) return;
  // the row's loads are issued before the block table's, which they do not wait for
  const uint4* src = reinterpret_cast<const uint4*>(p.c_kv + gw * p.r);
  uint4 x[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = 256 * h + 8 * lane;
    x[h] = c < p.r ? ld_stream_v4(src + c / 8) : make_uint4(0, 0, 0, 0);
  }
  int64_t page;
  int slot;
  if (!q8_locate(p.block_table, p.max_pages, p.num_pages, lane == 0 ? p.dev_error : nullptr, b,
                 int64_t(p.start_pos[b]) + t, &page, &slot))
    return;
  const int R = p.groups * p.rope_dim;
  uint8_t* dst = p.cache + page * q8_page_bytes(p.r, R);

  uint32_t scales[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {x[h].x, x[h].y, x[h].z, x[h].w};
    uint32_t top = 0;                          // largest magnitude bits, non-finite included
#pragma unroll
    for (int i = 0; i < 4; ++i)
      top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool bad = top >= 0x7F80u;           // the block holds an infinity or a NaN
    const uint32_t s = bad ? kQ8Bad : q8_scale_byte(top);
    // 2^-(s - 127), exact in fp32 (s - 127 in [-110, 119]); a bad block's codes are zero
    const float f = bad ? 0.0f : __uint_as_float((254u - s) << 23);
    uint32_t code[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = w[2 * i], c = w[2 * i + 1];
      code[i] = q8_encode2(__uint_as_float(a << 16) * f, __uint_as_float(a & 0xFFFF0000u) * f) |
                (q8_encode2(__uint_as_float(c << 16) * f, __uint_as_float(c & 0xFFFF0000u) * f)
                 << 16);
    }
    const int c = 256 * h + 8 * lane;
    if (c < p.r)
      *reinterpret_cast<uint2*>(dst + (c / kQ8Cols) * kQ8BlockBytes + slot * kQ8Cols +
                                c % kQ8Cols) =
          bad ? make_uint2(0, 0) : make_uint2(code[0], code[1]);
    uint32_t word = s << (8 * (lane >> 3));    // byte of this lane's block
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    word |= __shfl_xor_sync(0xffffffffu, word, 16);
    scales[h] = word;
  }
  if (lane == 0)
    *reinterpret_cast<uint2*>(dst + q8_scales_offset(p.r, R) + slot * kQ8ScaleBytes) =
        make_uint2(scales[0], scales[1]);
  const int64_t pairs = R / 2;
  rotate_keys(p.k_r + gw * R, p.rope_cos + gw * pairs, p.rope_sin + gw * pairs, p.groups,
              p.rope_dim, lane, reinterpret_cast<uint16_t*>(dst + q8_keys_offset(p.r)) + slot * R);
}

__global__ void __launch_bounds__(256) cache_read_q8_kernel(ReadQ8Params p) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t gw = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int per_seq = (p.n + 7) / 8;           // warps per sequence, 8 tokens each
  const int b = int(gw / per_seq);
  if (b >= p.batch) return;
  const int t = int(gw - int64_t(b) * per_seq) * 8 + (lane >> 2), part = lane & 3;
  if (p.out_table && lane == 0 && t % kQ8Tok == 0)
    p.out_table[int64_t(b) * (p.n / kQ8Tok) + t / kQ8Tok] = b * (p.n / kQ8Tok) + t / kQ8Tok;
  if (t >= q8_rows(p.read_lens, b, p.n, lane == 0 && t == 0 ? p.dev_error : nullptr)) return;
  int64_t page;
  int slot;
  if (!q8_locate(p.block_table, p.max_pages, p.num_pages, part == 0 ? p.dev_error : nullptr, b,
                 (p.start_pos ? int64_t(p.start_pos[b]) : 0) + t, &page, &slot))
    return;
  const int R = p.R, nb = p.r / kQ8Cols;
  const uint8_t* src = p.cache + page * q8_page_bytes(p.r, R);
  uint4 codes[kQ8MaxBlocks];
#pragma unroll
  for (int k = 0; k < kQ8MaxBlocks; ++k)
    if (k < nb)
      codes[k] = ld_stream_v4(src + k * kQ8BlockBytes + slot * kQ8Cols + 16 * part);
  const uint2 sc = *reinterpret_cast<const uint2*>(src + q8_scales_offset(p.r, R) +
                                                   slot * kQ8ScaleBytes);
  uint16_t* row = p.out + (int64_t(b) * p.n + t) * (p.r + R);
  const uint8_t* keys = src + q8_keys_offset(p.r) + slot * R * 2;
  // 16 keys of every 64 are this lane's; the first 64 are loaded with the codes
  auto load_keys = [&](int c, uint4* x) {
    if (c < R) x[0] = ld_stream_v4(keys + 2 * c);
    if (c + 8 < R) x[1] = ld_stream_v4(keys + 2 * c + 16);
  };
  auto store_keys = [&](int c, const uint4* x) {
    uint4* dst = reinterpret_cast<uint4*>(row + p.r + c);
    if (p.wide) {                              // R % 16 == 0 then
      if (c < R) st_global_v8(dst, x[0], x[1]);
    } else {
      if (c < R) dst[0] = x[0];
      if (c + 8 < R) dst[1] = x[1];
    }
  };
  uint4 first[2];
  load_keys(16 * part, first);
#pragma unroll
  for (int k = 0; k < kQ8MaxBlocks; ++k) {
    if (k >= nb) break;
    const uint32_t s = ((k < 4 ? sc.x : sc.y) >> (8 * (k & 3))) & 0xFFu;
    uint32_t v[8];
    q8_decode16(codes[k], q8_factor(s), v);
    uint4* dst = reinterpret_cast<uint4*>(row + k * kQ8Cols + 16 * part);
    const uint4 lo = make_uint4(v[0], v[1], v[2], v[3]), hi = make_uint4(v[4], v[5], v[6], v[7]);
    if (p.wide) {
      st_global_v8(dst, lo, hi);
    } else {
      dst[0] = lo;
      dst[1] = hi;
    }
  }
  store_keys(16 * part, first);
  for (int c = 64 + 16 * part; c < R; c += 64) {
    uint4 x[2];
    load_keys(c, x);
    store_keys(c, x);
  }
}

cudaError_t launch_cache_append_q8(const AppendQ8Params& p, cudaStream_t stream) {
  const int64_t blocks = (int64_t(p.batch) * p.n_new + 7) / 8;
  return launch_pdl(cache_append_q8_kernel, dim3(unsigned(blocks)), dim3(256), 0, stream, 1, p);
}

cudaError_t launch_cache_read_q8(const ReadQ8Params& params, cudaStream_t stream) {
  ReadQ8Params p = params;
  p.wide = (p.r + p.R) % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
  const int64_t blocks = (int64_t(p.batch) * ((p.n + 7) / 8) + 7) / 8;
  return launch_pdl(cache_read_q8_kernel, dim3(unsigned(blocks)), dim3(256), 0, stream, 1, p);
}

}  // namespace mla
