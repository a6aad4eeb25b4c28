// cache_q8.cu - mla_cache_append_q8 and mla_cache_read_q8: new tokens quantised into the paged
// 8-bit latent cache (q8.cuh), and stretches of it read back as bf16 rows.
//
// Append: four lanes hold a token's block of 64 columns, 16 (32 bytes) each, so its largest magnitude
// takes two shuffles of packed bf16 bits and its codes leave as 64 consecutive bytes; the same lanes
// rotate the token's keys. A token is 2 r + 2 R bytes in, with 4 R of angles, and r + 2 R + 8 out:
// bound by memory once there are many (32 x 8192 tokens of 512 + 64 columns: 83 us, of 256 + 64: 60,
// at 6.5 and 5.7 TB/s), by latency for a decode step (2.1 us).
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

// Four rotary pairs j .. j + 3 of a group: half % 4 == 0, keys 8-byte and angles 16-byte aligned.
struct KeyQuad {
  uint2 k0, k1;
  float4 c, s;
  int at;                                      // of x_j in the token's keys
  MLA_DEVICE void load(const uint16_t* kr, const float* cs, const float* sn, int idx, int half) {
    at = idx / half * half + idx;
    k0 = *reinterpret_cast<const uint2*>(kr + at);
    k1 = *reinterpret_cast<const uint2*>(kr + at + half);
    c = *reinterpret_cast<const float4*>(cs + idx);
    s = *reinterpret_cast<const float4*>(sn + idx);
  }
  MLA_DEVICE void store(uint16_t* dst, int half) const {
    uint16_t y0[4], y1[4];
    rotate_pair(uint16_t(k0.x), uint16_t(k1.x), c.x, s.x, &y0[0], &y1[0]);
    rotate_pair(uint16_t(k0.x >> 16), uint16_t(k1.x >> 16), c.y, s.y, &y0[1], &y1[1]);
    rotate_pair(uint16_t(k0.y), uint16_t(k1.y), c.z, s.z, &y0[2], &y1[2]);
    rotate_pair(uint16_t(k0.y >> 16), uint16_t(k1.y >> 16), c.w, s.w, &y0[3], &y1[3]);
    *reinterpret_cast<uint2*>(dst + at) =
        make_uint2(y0[0] | uint32_t(y0[1]) << 16, y0[2] | uint32_t(y0[3]) << 16);
    *reinterpret_cast<uint2*>(dst + at + half) =
        make_uint2(y1[0] | uint32_t(y1[1]) << 16, y1[2] | uint32_t(y1[3]) << 16);
  }
};

// Tokens of a warp (TOK): more of them share the work of finding their place (some 150 of 420
// instructions a token with one). At 32 x 8192 tokens of 512 + 64 columns one takes 141 us, two 97,
// four 83 and eight 91; at 64 x 8192 of 128 + 32 columns four take 91 us and eight, which leave a
// lane as much work as four do there, 74. A few tokens want short warps: 1024 of 512 + 64 columns
// take 2.2 us with one a warp and 3.0 with four, 4096 take 4.2 and 3.2.
constexpr int64_t kManyTokens = 4096;

// TOK tokens a warp, from token TOK * warp of the batch on. Four lanes hold a (token, block of 64
// columns), 16 columns each; a pass of the warp is eight of those, the tokens of a block side by
// side, so that codes leave in stretches of 64 * TOK bytes.
template <int TOK>
__global__ void __launch_bounds__(256) cache_append_q8_kernel(AppendQ8Params p) {
  constexpr int kStep = kQ8MaxBlocks / TOK;    // blocks of a pass
  constexpr int kLanes = 32 / TOK;             // lanes of a token
  grid_dep_wait();
  grid_dep_launch();
  const int64_t gw0 = ((int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5) * TOK;
  const int64_t tokens = int64_t(p.batch) * p.n_new;
  if (gw0 >= tokens) return;
  const int lane = threadIdx.x & 31, part = lane & 3, tk = (lane >> 2) % TOK;
  const int blk0 = (lane >> 2) / TOK;
  const int64_t gw = gw0 + tk;
  int b = 0, t = 0;
  bool mine = gw < tokens;
  const bool reports = part == 0 && blk0 == 0;
  if (mine) {
    // 64-bit divisions take some 100 instructions
    b = tokens <= int64_t(UINT32_MAX) ? int(uint32_t(gw) / uint32_t(p.n_new)) : int(gw / p.n_new);
    t = int(gw - int64_t(b) * p.n_new);
    mine = t < q8_rows(p.new_lens, b, p.n_new, reports && t == 0 ? p.dev_error : nullptr);
  }
  if (!__any_sync(0xffffffffu, mine)) return;
  // the row's loads are issued before the block table's, which they do not wait for
  const uint4* src = reinterpret_cast<const uint4*>(p.c_kv + gw * p.r) + 2 * part;
  const int nb = p.r / kQ8Cols;
  uint4 x[TOK][2];
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int k = blk0 + i * kStep;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      x[i][h] = mine && k < nb ? ld_stream_v4(src + 8 * k + h) : make_uint4(0, 0, 0, 0);
  }
  const int R = p.groups * p.rope_dim, half = p.rope_dim / 2, npairs = R / 2;
  const uint16_t* kr = p.k_r + gw * R;
  const float *cs = p.rope_cos + gw * npairs, *sn = p.rope_sin + gw * npairs;
  const int key_lane = part + 4 * blk0;
  KeyQuad keys;
  if (mine && p.quads && 4 * key_lane < npairs) keys.load(kr, cs, sn, 4 * key_lane, half);
  int64_t page = 0;
  int slot = 0;
  if (mine)
    mine = q8_locate(p.block_table, p.max_pages, p.num_pages, reports ? p.dev_error : nullptr, b,
                     int64_t(p.start_pos[b]) + t, &page, &slot);
  uint8_t* dst = p.cache + page * q8_page_bytes(p.r, R);

  uint8_t* codes = dst + slot * kQ8Cols + 16 * part;
  uint64_t scales = 0;                         // byte k: block k, of this lane's; 0 past r / 64
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int k = blk0 + i * kStep;
    if (i * kStep >= nb) break;
    const uint32_t w[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                           x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
    uint32_t tops = 0;                         // largest magnitude bits, non-finite included
#pragma unroll
    for (int j = 0; j < 8; ++j) tops = max_u16x2(tops, w[j] & 0x7FFF7FFFu);
    tops = max_u16x2(tops, __shfl_xor_sync(0xffffffffu, tops, 1));
    tops = max_u16x2(tops, __shfl_xor_sync(0xffffffffu, tops, 2));
    const uint32_t top = max(tops & 0xFFFFu, tops >> 16);
    const bool bad = top >= 0x7F80u;           // the block holds an infinity or a NaN
    const uint32_t s = bad ? kQ8Bad : q8_scale_byte(top);
    // 2^-(s - 127) in both halves: a normal bf16, as s - 127 is in [-110, 119]. A product is exact
    // but for those below 2^-126, whose code is zero anyway. A bad block's codes are zero.
    const uint32_t f = (254u - s) * 0x00800080u;
    uint32_t code[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = mul_bf16x2(w[2 * j], f), c = mul_bf16x2(w[2 * j + 1], f);
      code[j] = __byte_perm(q8_encode2(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u)),
                            q8_encode2(__uint_as_float(c << 16), __uint_as_float(c & 0xFFFF0000u)),
                            0x5410);
      code[j] = bad ? 0u : code[j];
    }
    if (mine && k < nb)
      *reinterpret_cast<uint4*>(codes + k * kQ8BlockBytes) =
          make_uint4(code[0], code[1], code[2], code[3]);
    scales |= uint64_t(k < nb ? s : 0u) << (8 * k);
  }
#pragma unroll
  for (int o = 4 * TOK; o < 32; o <<= 1) scales |= __shfl_xor_sync(0xffffffffu, scales, o);
  if (!mine) return;
  if (reports)
    *reinterpret_cast<uint64_t*>(dst + q8_scales_offset(p.r, R) + slot * kQ8ScaleBytes) = scales;
  uint16_t* row = reinterpret_cast<uint16_t*>(dst + q8_keys_offset(p.r)) + slot * R;
  if (p.quads) {
    for (int q = 4 * key_lane; q < npairs;) {
      keys.store(row, half);
      q += 4 * kLanes;
      if (q < npairs) keys.load(kr, cs, sn, q, half);
    }
  } else {
    rotate_keys(kr, cs, sn, p.groups, p.rope_dim, key_lane, row, kLanes);
  }
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

cudaError_t launch_cache_append_q8(const AppendQ8Params& params, cudaStream_t stream) {
  AppendQ8Params p = params;
  auto on = [](const void* at, size_t n) { return reinterpret_cast<uintptr_t>(at) % n == 0; };
  p.quads = p.rope_dim % 8 == 0 && on(p.k_r, 8) && on(p.rope_cos, 16) && on(p.rope_sin, 16);
  const int64_t tokens = int64_t(p.batch) * p.n_new;
  const int tok = tokens < kManyTokens ? 1 : p.r <= 2 * kQ8Cols ? 8 : 4;
  const dim3 grid(unsigned((tokens + 8 * tok - 1) / (8 * tok)));
  return launch_pdl(tok == 1   ? cache_append_q8_kernel<1>
                    : tok == 4 ? cache_append_q8_kernel<4>
                               : cache_append_q8_kernel<8>,
                    grid, dim3(256), 0, stream, 1, p);
}

cudaError_t launch_cache_read_q8(const ReadQ8Params& params, cudaStream_t stream) {
  ReadQ8Params p = params;
  p.wide = (p.r + p.R) % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
  const int64_t blocks = (int64_t(p.batch) * ((p.n + 7) / 8) + 7) / 8;
  return launch_pdl(cache_read_q8_kernel, dim3(unsigned(blocks)), dim3(256), 0, stream, 1, p);
}

}  // namespace mla
