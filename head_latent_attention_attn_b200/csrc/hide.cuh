// hide.cuh - tokens that some rows of a tile do not see. Their weights are 0 there, but the tensor core
// multiplies them all the same.
#pragma once

#include "ptx.cuh"

namespace mla {

// Whether the bf16 pairs of a 16-byte chunk are all finite: 0 * x is 0 or, for an infinity or a NaN,
// NaN, which the sums keep.
MLA_DEVICE uint32_t times_zero(uint32_t x, uint32_t sum) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(sum));
  return r;
}

// 64 bf16 numbers of a token (128 bytes at `row`, shared memory) that a product with the weights of a
// block of query rows reads, when some of the rows (or, with `none`, all) do not see the token. Their
// weight is 0, and 0 times an infinity or a NaN must not reach their O: such numbers become zeros (with
// `none` all do). Returns whether there were any (false with `none`).
MLA_DEVICE bool hide_token(uint8_t* row, bool none, int lane) {
  // chunks in another order a lane: rows are 128 bytes apart, so that eight lanes at the same chunk
  // would be in the same banks
  auto at = [&](int i) { return reinterpret_cast<uint4*>(row + 16 * ((i + lane) & 7)); };
  if (none) {
#pragma unroll
    for (int i = 0; i < 8; ++i) *at(i) = make_uint4(0, 0, 0, 0);
    return false;
  }
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = *at(i + j);
    uint32_t a = 0, b = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a = times_zero(x[j].y, times_zero(x[j].x, a));
      b = times_zero(x[j].w, times_zero(x[j].z, b));
    }
    sum |= a | b;
  }
  if ((sum & 0x7FFF7FFFu) == 0) return false;    // (zeros of either sign)
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    uint32_t* w = reinterpret_cast<uint32_t*>(at(i));
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = (w[j] & 0x7F80u) == 0x7F80u ? 0xFFFF0000u : 0xFFFFFFFFu;
      const uint32_t hi = (w[j] & 0x7F800000u) == 0x7F800000u ? 0xFFFFu : 0xFFFFFFFFu;
      w[j] &= lo & hi;
    }
  }
  return true;
}

}  // namespace mla
