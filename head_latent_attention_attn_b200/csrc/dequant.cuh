// dequant.cuh - the part of the decode kernels that turns pages of the 8-bit cache (q8.cuh)
// into the bf16 tiles that the UMMAs read.
//
// A page's codes go from memory to the registers of the dequantising warps and from there, as
// bf16, into the cache slot: no shared memory holds them in between, which the largest shapes
// do not have. A warp converts 8 tokens (lane: token lane / 4, 16 of the 64 columns); its loads
// of the next page are issued as soon as this page's codes have left the registers. In the one-CTA
// kernel the TMA producer brings pages into L2 ahead of them.
//
// What this costs is issue slots, which the softmax warps of the same SM need: some 12 cycles of
// a scheduler for 4 codes of a warp. So the 8-bit cache saves memory, not time. The one-CTA kernel
// takes 1.0 to 1.2 times what it takes over the bf16 cache, for 0.54 to 0.61 of the bytes: 16 rows
// over 1M tokens 130 us (122 over bf16), 64 rows over 1M tokens 159 (138), 128 ragged sequences of
// 32 heads 402 from a cool start and 432 in a long run (390 and 410), 64 rows over 64 x 8192 of r
// 512 139 (134). The two-CTA kernel takes 1.3 times: 64 x 8192 tokens of 128 heads 236 (183).
// Measured and slower: 16 warps of half the blocks, two pages ahead in registers, converting before
// the slot is free, S^T begun on half a page, PV by latent chunk so that the slot's first blocks are
// free early.
#pragma once

#include "decode_sched.cuh"
#include "q8.cuh"

namespace mla {

constexpr uint32_t kBlk8Bytes = kDecodeTok * 128;   // one 64 x 64 bf16 block of a slot
constexpr int kDequantPrefetch = 3;                 // pages that the L2 prefetch runs ahead

MLA_DEVICE void st_shared_v4(uint32_t saddr, const uint32_t* v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

// `bytes` (a multiple of 16) at p, 16-byte aligned, into L2.
MLA_DEVICE void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Tile by tile along [r0, r1): the page of each, its first position and its context length.
struct PageWalk {
  UnitWalk w;
  int t;
  MLA_DEVICE explicit PageWalk(const UnitWalk& u) : w(u), t(0) {}
  MLA_DEVICE PageWalk(const DecodeParams& p, int cg, int r0, int b, int s) : w{b, s}, t(r0) {
    w.load(p, cg);
  }
  MLA_DEVICE int32_t page(const DecodeParams& p) const {
    return p.block_table[int64_t(w.b) * p.max_pages + (t - w.s)];
  }
  // to the next tile; the caller stops at r1
  MLA_DEVICE void next(const DecodeParams& p, int cg, int r1) {
    if (++t == w.s + w.tiles && t < r1) {
      w.s += w.tiles;
      ++w.b;
      w.load(p, cg);
    }
  }
};

// Bring the pages of the tiles up to `upto` (exclusive of r1) into L2; one thread.
MLA_DEVICE void prefetch_pages(const DecodeParams& p, int cg, int r1, int upto,
                               PageWalk& ahead) {
  const int64_t page_bytes = q8_page_bytes(p.r, p.D - p.r);
  while (ahead.t < r1 && ahead.t <= upto) {
    const int32_t page = ahead.page(p);
    if (page >= 0 && page < p.num_pages)
      prefetch_l2(static_cast<const uint8_t*>(p.cache_q8) + page * page_bytes,
                  uint32_t(page_bytes));
    ahead.next(p, cg, r1);
  }
}

// All pages of tiles [r0, r1), whose first is of sequence b, which starts at tile s. This warp
// converts the NG 8-token groups from NG * grp on of the page's column blocks [blk0, blk0 + nb),
// nb <= NB, into the slot's blocks 0, 1, ... It waits for empty[slot] and arrives on full[slot]
// once. The last `hidden` tokens of a context, which none of the block's rows sees, become zeros.
template <int NB, int NG>
MLA_DEVICE void dequant_pages(const DecodeParams& p, int cg, int r0, int r1, int b, int s, int grp,
                              int blk0, int nb, int hidden, uint8_t* slots, uint32_t slot_bytes,
                              uint64_t* full, uint64_t* empty, const WaitCtx& wc) {
  const int lane = threadIdx.x & 31, part = lane & 3;
  const int tok = 8 * NG * grp + (lane >> 2);       // of the first group; + 8 g
  const int not_live = hidden + tok;
  const int R = p.D - p.r;
  const int64_t page_bytes = q8_page_bytes(p.r, R);
  const uint8_t* cache = static_cast<const uint8_t*>(p.cache_q8);
  const uint32_t code_off = uint32_t(blk0 * kQ8BlockBytes + tok * kQ8Cols + 16 * part);
  const uint32_t scale_off = uint32_t(q8_scales_offset(p.r, R) + tok * kQ8ScaleBytes);
  const uint32_t st0 = smem_u32(slots) + tok * 128 + (((2 * part) ^ (tok & 7)) << 4);

  PageWalk next(p, cg, r0, b, s);        // the tile to fetch; its page id is read a tile ahead
  int32_t page = next.page(p);
  uint4 codes[NG][NB];
  uint2 scales[NG];
  int live;                              // tokens that some row sees from `tok` on
  auto fetch = [&]() {
    if (page < 0 || page >= p.num_pages) page = 0;       // the TMA producer reports it
    const uint8_t* src = cache + page * page_bytes;
    // rows past those are loaded too (they are part of the page) but not used
    live = next.w.L - (next.t - next.w.s) * kDecodeTok - not_live;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (k < nb)
          codes[g][k] = ld_stream_v4(src + code_off + k * kQ8BlockBytes + g * 8 * kQ8Cols);
      scales[g] = *reinterpret_cast<const uint2*>(src + scale_off + g * 8 * kQ8ScaleBytes);
    }
    next.next(p, cg, r1);
    if (next.t < r1) page = next.page(p);
  };

  fetch();
  SlotRing ring(p.nslot);
  for (int jj = 0, n = r1 - r0; jj < n; ++jj, ring.next()) {
    if (jj >= p.nslot &&
        !__all_sync(0xffffffffu, mbar_wait(&empty[ring.slot], (ring.round - 1) & 1, wc)))
      break;
    const uint32_t at = st0 + ring.slot * slot_bytes;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (live <= 8 * g) {
        // they may hold anything: they become zeros (0-weight x garbage must not reach O)
        scales[g] = make_uint2(0, 0);
#pragma unroll
        for (int k = 0; k < NB; ++k) codes[g][k] = make_uint4(0, 0, 0, 0);
      }
      const uint64_t sc = (uint64_t(scales[g].y) << 32 | scales[g].x) >> (8 * blk0);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (k >= nb) break;
        uint32_t v[8];
        q8_decode16(codes[g][k], q8_factor(uint32_t(sc >> (8 * k)) & 0xFFu), v);
        st_shared_v4(at + k * kBlk8Bytes + g * 1024, v);
        st_shared_v4((at ^ 16u) + k * kBlk8Bytes + g * 1024, v + 4);
      }
    }
    // no proxy fence here: the UMMA issuer fences after it has waited for full[slot]
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[ring.slot]);
    if (next.t < r1) fetch();
  }
}

}  // namespace mla
