// q8.cuh - the 8-bit latent cache: layout of a page and the conversions to and from it.
//
// A page holds 64 tokens. Its bytes are three planes, in this order:
//   codes   [r/64][64 tokens][64]   e4m3 code of latent column 64 k + j of token t
//   keys    [64 tokens][R]          rotated keys of every group, bf16 (R = G * d_r)
//   scales  [64 tokens][8]          byte k: exponent + 127 of the token's column block k; 0 past r/64
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
constexpr int kQ8ExpMin = -110;        // 2^-110: every nonzero value is a normal bf16
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

MLA_DEVICE uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

MLA_DEVICE uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The scale 2^(s - 127) of scale byte s as bf16, in both halves: s is its exponent field. A
// NaN for the byte of a non-finite block.
MLA_DEVICE uint32_t q8_factor(uint32_t s) {
  return s == kQ8Bad ? 0x7FC07FC0u : s * 0x00800080u;
}

// 16 codes to 16 bf16 values (exact): codes to fp16 pairs by the conversion instruction, each
// half to fp32, whose upper halves are the bf16 values (4 significant bits), then one packed
// multiplication by the scale. On B200 that is 10.4 cycles of a scheduler for 4 codes of a
// warp. Moving the bits with integer operations, which all share the half-rate ALU pipe, takes
// 16 (two byte permutes, two shifts, four logic operations and two multiplications).
MLA_DEVICE void q8_decode16(const uint4& codes, uint32_t factor, uint32_t* v) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t f[4];
    asm("{\n\t.reg .b16 c0, c1, h0, h1, h2, h3;\n\t.reg .b32 p0, p1;\n\t"
        "mov.b32 {c0, c1}, %4;\n\t"
        "cvt.rn.f16x2.e4m3x2 p0, c0;\n\t"
        "cvt.rn.f16x2.e4m3x2 p1, c1;\n\t"
        "mov.b32 {h0, h1}, p0;\n\t"
        "mov.b32 {h2, h3}, p1;\n\t"
        "cvt.f32.f16 %0, h0;\n\tcvt.f32.f16 %1, h1;\n\t"
        "cvt.f32.f16 %2, h2;\n\tcvt.f32.f16 %3, h3;\n\t}"
        : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
        : "r"(w[i]));
    v[2 * i] = mul_bf16x2(__byte_perm(f[0], f[1], 0x7632), factor);
    v[2 * i + 1] = mul_bf16x2(__byte_perm(f[2], f[3], 0x7632), factor);
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

// 32 bytes of global memory, 32-byte aligned.
MLA_DEVICE void ld_global_v8(const void* p, uint4* lo, uint4* hi) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(lo->x), "=r"(lo->y), "=r"(lo->z), "=r"(lo->w), "=r"(hi->x), "=r"(hi->y),
                 "=r"(hi->z), "=r"(hi->w)
               : "l"(p)
               : "memory");
}

// 32 bytes to global memory, 32-byte aligned: a whole sector of a line in one access.
MLA_DEVICE void st_global_v8(void* p, const uint4& lo, const uint4& hi) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(lo.x),
               "r"(lo.y), "r"(lo.z), "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
               : "memory");
}

}  // namespace mla
