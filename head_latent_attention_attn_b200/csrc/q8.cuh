// q8.cuh - the 8-bit latent cache: layout of a page and the conversions to and from it.
//
// A page holds 64 tokens. Its bytes are three planes, in this order:
//   codes   [r/64][64 tokens][64]   e4m3 code of latent column 64 k + j of token t
//   keys    [64 tokens][R]          rotated keys of every group, bf16 (R = G * d_r)
//   scales  [64 tokens][8]          byte k: exponent + 127 of the token's column block k
// The codes are blocked by 64 columns so that 8 tokens of a block are 512 consecutive bytes
// (one 16-byte load a lane) and a thread's 16 codes become two 16-byte chunks of the
// 128-byte-swizzled bf16 operand tile without a shared-memory bank conflict.
//
// Scales are powers of two: a code times its scale is exact in bf16 (4 significant bits), so
// what attention multiplies is exactly what the cache holds, and a group's relative error is
// e4m3's own half step, 2^-4. Byte 255 marks a block that held an infinity or a NaN; the
// whole block reads back as NaN.
#pragma once

#include "ptx.cuh"

namespace mla {

constexpr int kQ8Tok = 64;             // tokens per page
constexpr int kQ8Cols = 64;            // latent columns per scale
constexpr int kQ8MaxBlocks = 8;        // r <= 512
constexpr int kQ8BlockBytes = kQ8Tok * kQ8Cols;
constexpr int kQ8ScaleBytes = kQ8MaxBlocks;   // per token
constexpr int kQ8ExpMin = -110;        // smallest scale 2^-110: every nonzero value is a normal bf16
constexpr int kQ8ExpMax = 119;         // largest scale 2^119: 448 * 2^119 is finite in bf16
constexpr uint32_t kQ8Bad = 255;       // scale byte of a block with a non-finite value

__host__ __device__ inline int64_t q8_page_bytes(int r, int R) {
  return int64_t(kQ8Tok) * (r + 2 * R + kQ8ScaleBytes);
}
__host__ __device__ inline int q8_keys_offset(int r) { return kQ8Tok * r; }
__host__ __device__ inline int q8_scales_offset(int r, int R) { return kQ8Tok * (r + 2 * R); }

// Scale byte of a block whose largest finite magnitude has the bf16 bits `amax` (sign clear):
// exponent e = least e with amax * 2^-e <= 448 = 1.75 * 2^8, clamped. amax = m * 2^(E-127) with
// m <= 1.75 exactly when its 7 mantissa bits are <= 0x60.
MLA_DEVICE uint32_t q8_scale_byte(uint32_t amax) {
  const int s = int(amax >> 7) - 8 + ((amax & 0x7Fu) > 0x60u ? 1 : 0);
  return uint32_t(min(max(s, kQ8ExpMin + 127), kQ8ExpMax + 127));
}

// Two e4m3 codes of lo * f and hi * f, round to nearest even, saturating (lo in the low byte).
MLA_DEVICE uint32_t q8_encode2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

MLA_DEVICE uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The factor (bf16, in both halves) that takes re-biased codes of a block with scale byte s to
// their values. A code's bits placed as sign | 4-bit exponent | mantissa of a bf16 stand for
// its value times 2^-120, so the factor is 2^(s - 127 + 120). Scales above 2^7 (s > 134) do
// not fit one bf16 factor: those blocks multiply twice (q8_decode16's `big`).
constexpr uint32_t kQ8OneFactorMax = 134;
MLA_DEVICE uint32_t q8_factor(uint32_t s) {
  const uint32_t f = s == kQ8Bad ? 0x7FC0u : ((s > kQ8OneFactorMax ? 254u : s + 120u) << 7);
  return f | (f << 16);
}
MLA_DEVICE uint32_t q8_factor2(uint32_t s) {
  const uint32_t f = (s > kQ8OneFactorMax && s != kQ8Bad) ? (s - 7u) << 7 : 0x3F80u;
  return f | (f << 16);
}

// 16 codes to 16 bf16 values (exact): bytes are spread to the high halves of 16-bit lanes, the
// exponent and mantissa move down by 4 beside the sign, and one multiplication re-biases and
// scales. (The conversion instruction goes to fp16 and would need a second conversion through
// fp32; this is 2.5 integer or half operations a value.)
MLA_DEVICE void q8_decode16(const uint4& codes, uint32_t factor, uint32_t* v) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __byte_perm(w[i], 0u, 0x1404), b = __byte_perm(w[i], 0u, 0x3424);
    v[2 * i] = mul_bf16x2(((a >> 4) & 0x07F007F0u) | (a & 0x80008000u), factor);
    v[2 * i + 1] = mul_bf16x2(((b >> 4) & 0x07F007F0u) | (b & 0x80008000u), factor);
  }
}

// 16 bytes of global memory, kept out of L1 (each byte is used once).
MLA_DEVICE uint4 ld_stream_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

}  // namespace mla
