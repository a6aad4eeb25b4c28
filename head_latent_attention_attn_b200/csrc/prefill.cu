// prefill.cu - mla_prefill_attn on sm_100a: attention in its expanded form, a key and a value
// per head, the rotary key shared by the heads of a group.
//
//   s[i, t] = scale (q_nope[i] . k_nope[t] + q_pe[i] . k_pe[t]),  o = softmax(s) v
//
// Against the absorbed form over the latent (r + d_r columns of scores, r of output) this needs
// d_n + d_r + d_v multiplications a (query, token) pair instead of 2 r + d_r: 320 instead of 1088
// for the DeepSeek-V2 layer. It pays once a context's keys and values are expanded for enough
// query rows, as in a prefill chunk. A 128 x 128 tile of one head is 128 * 128 * (192 + 128)
// multiplications, 1280 cycles of an SM's tensor core, against 1024 cycles for its exponentials and
// 80 KB of operands that the heads' other query tiles find in L2.
//
// Measured on B200: 1024 rows over 4096 tokens of 128 heads in 281 us from a cool start (1.07
// PFLOP/s) and 331 us in a long run (910 TFLOP/s), where the card holds 990 W by lowering its clock
// to 1.62 GHz; a library matrix product sustains 1365 TFLOP/s there. Causal 4096 rows, 2 x 32
// heads of 136 + 128: 301 and 340 us. A group's tile takes 3500 to 3700 cycles (scores 270 to read
// and find their maximum, 1400 for the weights, 1600 from the last weights to the next scores),
// two groups' products 2560 of them. So the chain of a group's hand-overs bounds a cool card and
// its power a warm one: taking up to half of the exponentials to the FMA units by a polynomial
// gained nothing cool and lost 15 %, and a last wave spread over the idle SMs gained nothing warm.
//
// One CTA works on 256 query rows of a head, as two groups of 128 (one per softmax warpgroup).
// While a group's scores are in the hands of its softmax, the tensor cores work for the other:
//   S_g = Q_g K^T       UMMA M=128 rows, N=128 tokens, both operands in shared memory
//   O_g += P_g V        UMMA M=128 rows, N=d_v, A = P in TMEM (bf16 over S's columns), V MN-major
// TMEM lane = query row, so a thread owns a row: its 128 scores sit in registers, and maximum
// and sum need no exchange. TMEM: O_0, O_1, S_0, S_1, 128 columns each.
//
// Shared memory: Q of both groups 96 KB, three 32 KB slots through which K (unrotated part) and V
// tiles pass in turn, two 16 KB slots for the rotary part of K.
//
// Roles (384 threads): warp 0 TMA producer, warp 1 UMMA issuer, warp 2 scheduler, warps 4-7 and
// 8-11 the rows of group 0 and 1. Registers: 168 a thread at launch, 72 for the first group of
// warps, 216 for the rows'.
//
// The grid has one CTA per unit (256 rows of a head), but a CTA that runs takes over further
// units of CTAs not launched yet (cluster launch control): loads, scores and outputs of
// neighbouring units overlap, where a CTA per unit spent 10 of 46 us (causal 4096 rows) on its
// start, its first loads and its last group's output.
//
// Few units (a short chunk over a long context) leave most SMs idle: then a cluster of up to eight
// CTAs shares a unit's tiles (kSplit), and merges its parts through distributed shared memory.
//
// Softmax in the log2 domain with a reference maximum that moves only when a score exceeds it by
// more than 8 (weights stay <= 256), so that O is rescaled rarely; the row itself then does it.
#include <math.h>

#include "hide.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mla {

namespace {

constexpr int kRows = 128;                       // query rows of a group
constexpr int kTok = 128;                        // tokens of a tile
constexpr int kThreads = 384;
constexpr uint32_t kBlk = 128 * 128;             // 128 rows x 64 bf16, 16 KB
constexpr int kSlots = 3;
constexpr uint32_t kColO = 0, kColS = 256;       // + 128 g
constexpr int kRegsLaunch = 168, kRegsIssue = 72, kRegsRows = 216;
// setmaxnreg may only lower a group's share by .dec and raise it by .inc
static_assert(kRegsIssue <= kRegsLaunch && kRegsRows >= kRegsLaunch, "register shares");
static_assert(kRegsIssue + 2 * kRegsRows <= 3 * kRegsLaunch,
              "the groups' registers exceed what the block is launched with");
constexpr float kLazyThreshold = 8.0f;           // log2 units
constexpr float kRefInit = -3.0e38f;             // finite: see decode.cu
constexpr float kLn2 = 0.69314718055994530942f;

constexpr uint32_t kQOff = 0;                    // [group][nope 2 blocks, rope 1 block]
constexpr uint32_t kQGroup = 3 * kBlk;
constexpr uint32_t kSlotOff = 2 * kQGroup;       // K unrotated / V, 2 blocks each
constexpr uint32_t kRopeOff = kSlotOff + kSlots * 2 * kBlk;
constexpr uint32_t kMiscOff = kRopeOff + 2 * kBlk;
constexpr uint32_t kBars = 4 + 2 * kSlots + 10 + 6;
constexpr uint32_t kInfoOff = kMiscOff + 16;     // [2] unit descriptions, 32 bytes each
constexpr uint32_t kRespOff = kInfoOff + 64;     // answer of the launch control, 16 bytes
constexpr uint32_t kBadOff = kRespOff + 16;      // [4] see bad_unit
constexpr uint32_t kBarOff = kBadOff + 16;
constexpr uint32_t kSmem = kBarOff + 8 * kBars + 1024;   // + alignment slack
static_assert(kSmem <= 232448, "shared memory of a CTA");

// What a CTA works on: 256 query rows from row0 of head h of sequence b, which has L tokens and
// ql query rows; group g's rows see nt[g] tiles from tile t0 on. h < 0: no further unit.
struct Unit {
  int row0, h, b, L, ql, nt[2], t0;
  MLA_DEVICE int tiles() const { return max(nt[0], nt[1]); }
  // first position that some row of the unit does not see
  MLA_DEVICE int first_hidden(const PrefillParams& p) const {
    return p.causal ? min(L, L - ql + row0 + 1) : L;
  }
};

// Unit u of the grid, or with split > 1 the part of its tiles that CTA `rank` of the cluster takes.
MLA_DEVICE Unit make_unit(const PrefillParams& p, int u, int rank, int split) {
  // Units in blocks of head_block heads whose keys and values share L2; in a block the query
  // tiles with the most tokens first (a causal chunk's last rows), so that the last are short.
  const int heads = p.heads * p.batch, qts = (p.q_len + 2 * kRows - 1) / (2 * kRows);
  const int blk = u / (p.head_block * qts), at = u - blk * p.head_block * qts;
  const int hb = min(p.head_block, heads - blk * p.head_block);
  const int bh = blk * p.head_block + at % hb;
  Unit w;
  w.row0 = (qts - 1 - at / hb) * 2 * kRows;
  w.b = bh / p.heads;
  w.h = bh - w.b * p.heads;
  w.L = p.seq_lens[w.b];
  w.ql = p.q_lens ? p.q_lens[w.b] : p.q_len;
  if (w.L < 0 || w.L > p.kv_len || w.ql < 0 || w.ql > p.q_len) {
    if (p.dev_error) atomicOr(p.dev_error, MLA_DEVERR_BOUNDS);
    w.L = 0;
    w.ql = max(0, min(w.ql, p.q_len));
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int first = w.row0 + g * kRows, last = min(first + kRows, w.ql) - 1;
    const int seen =
        first >= w.ql ? 0 : p.causal ? max(0, min(w.L, w.L - w.ql + last + 1)) : w.L;
    w.nt[g] = (seen + kTok - 1) / kTok;
  }
  const int n = w.tiles(), end = n * (rank + 1) / split;
  w.t0 = n * rank / split;
#pragma unroll
  for (int g = 0; g < 2; ++g) w.nt[g] = max(0, min(w.nt[g], end) - w.t0);
  return w;
}

// A phase counter of an mbarrier: the wait for its n-th completion takes parity n % 2.
struct Phase {
  uint32_t n = 0;
  MLA_DEVICE uint32_t next() { return n++ & 1u; }
  MLA_DEVICE uint32_t last() const { return (n - 1) & 1u; }
};

// A CTA's part of a unit for the cluster's merge, over Q, K and V: O as [group][column / 4][row],
// then reference and sum as [group][row].
MLA_DEVICE float4* stage_o(uint8_t* base, int g, int col4, int row) {
  return reinterpret_cast<float4*>(base) + (g * 32 + col4) * kRows + row;
}
MLA_DEVICE float2* stage_ml(uint8_t* base, int g, int row) {
  return reinterpret_cast<float2*>(base + 2 * 32 * kRows * 16) + g * kRows + row;
}

// Position in the ring of K and V slots.
struct Ring {
  int slot = 0;
  uint32_t round = 0;
  MLA_DEVICE void next() {
    if (++slot == kSlots) {
      slot = 0;
      ++round;
    }
  }
};

}  // namespace

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + kMiscOff);
  volatile int* abort_flag = reinterpret_cast<int*>(base + kMiscOff) + 1;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(base + kBarOff);   // [group]
  uint64_t* q_empty = q_full + 2;                // [group] every product with the unit's Q done
  uint64_t* full = q_empty + 2;                  // [slot] K or V tile landed
  uint64_t* empty = full + kSlots;               // [slot]
  uint64_t* s_full = empty + kSlots;             // [group] scores computed
  uint64_t* p_full = s_full + 2;                 // [group][half] weights of 64 tokens written
  uint64_t* pv_done = p_full + 4;                // [group] PV of the group's tile done
  uint64_t* o_free = pv_done + 2;                // [group] O of the unit read
  uint64_t* info_full = o_free + 2;              // [2]
  uint64_t* info_empty = info_full + 2;          // [2]
  uint64_t* resp_full = info_empty + 2;
  uint64_t* want = resp_full + 1;                // the producer is about to need a unit
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{abort_flag, p.dev_error};

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);              // the group's four warps
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&info_full[i], 1);
      mbar_init(&info_empty[i], 10);             // producer, issuer, 8 row warps
    }
    mbar_init(resp_full, 1);
    mbar_init(want, 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(base + kBadOff)[i] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // set-up above may overlap the previous kernel; from here on global memory is touched
  grid_dep_wait();
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int nb = (p.dn + 63) / 64, vb = (p.dv + 63) / 64;   // 64-column blocks
  const int rope = p.dr > 0 ? 1 : 0;

  // The k-th unit of this CTA, from the scheduler; false when there is none (or on an abort).
  // Called by one thread (kWarp false) or a whole warp.
  auto next_unit = [&](uint32_t k, Unit* w, bool whole_warp) -> bool {
    bool ok = mbar_wait(&info_full[k & 1], (k >> 1) & 1, wc);
    if (whole_warp) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    const int* src = reinterpret_cast<const int*>(base + kInfoOff + 32 * (k & 1));
    w->row0 = src[0];
    w->h = src[1];
    w->b = src[2];
    w->L = src[3];
    w->ql = src[4];
    w->nt[0] = src[5];
    w->nt[1] = src[6];
    w->t0 = src[7];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(&info_empty[k & 1]);
    return w->h >= 0;
  };

  if (warp < 4) {
    reg_dec<kRegsIssue>();
    if (warp == 0) {
      // =================================== TMA producer ===================================
      if (elect_one()) {
        prefetch_tensormap(&p.tm_k);
        prefetch_tensormap(&p.tm_v);
        prefetch_tensormap(&p.tm_q);
        Ring ring;
        Phase q_ph[2];
        uint32_t tile = 0;                       // K tiles so far: rope slot tile % 2
        bool ok = true;
        Unit w;
        for (uint32_t k = 0; ok && next_unit(k, &w, false); ++k) {
          const int kg = w.h / p.heads_per_group, n = w.tiles();
          auto load_q = [&](int g) {
            if (q_ph[g].n > 0) ok = ok && mbar_wait(&q_empty[g], q_ph[g].last(), wc);
            if (!ok) return;
            q_ph[g].next();
            uint8_t* dst = base + kQOff + g * kQGroup;
            mbar_arrive_expect_tx(&q_full[g], uint32_t(nb + rope) * kBlk);
            for (int i = 0; i < nb; ++i)
              tma_load_4d(dst + i * kBlk, &p.tm_q, 64 * i, w.h, w.row0 + g * kRows, w.b,
                          &q_full[g]);
            if (rope)
              tma_load_4d(dst + 2 * kBlk, &p.tm_qr, 0, w.h, w.row0 + g * kRows, w.b, &q_full[g]);
          };
          // Next slot of the ring: K and V tiles in turn. A K tile's rotary part goes to rope
          // slot tile % 2, which is free when the ring slot of V of two tiles before is: its
          // release follows every product with that tile's keys.
          auto load_tile = [&](int t, bool v) {
            if (ring.round > 0) ok = ok && mbar_wait(&empty[ring.slot], (ring.round - 1) & 1, wc);
            if (!ok) return;
            uint8_t* dst = base + kSlotOff + ring.slot * 2 * kBlk;
            uint64_t* bar = &full[ring.slot];
            if (v) {
              mbar_arrive_expect_tx(bar, uint32_t(vb) * kBlk);
              for (int i = 0; i < vb; ++i)
                tma_load_4d(dst + i * kBlk, &p.tm_v, 64 * i, w.h, (w.t0 + t) * kTok, w.b, bar);
            } else {
              mbar_arrive_expect_tx(bar, uint32_t(nb + rope) * kBlk);
              for (int i = 0; i < nb; ++i)
                tma_load_4d(dst + i * kBlk, &p.tm_k, 64 * i, w.h, (w.t0 + t) * kTok, w.b, bar);
              if (rope)
                tma_load_4d(base + kRopeOff + (tile & 1) * kBlk, &p.tm_kr, 0, kg, (w.t0 + t) * kTok,
                            w.b, bar);
              ++tile;
            }
            ring.next();
          };
          if (w.nt[0] > 0) load_q(0);
          if (n > 0) load_tile(0, false);
          if (w.nt[1] > 0) load_q(1);
          // the next unit is asked for with the last tile: asked for earlier, a CTA would sit on
          // a unit that an idle one could have begun
          if (n == 0) mbar_arrive(want);
          for (int t = 0; ok && t < n; ++t) {
            if (t == n - 1) mbar_arrive(want);
            load_tile(t, true);
            if (t + 1 < n) load_tile(t + 1, false);
          }
        }
        // never leave while copies into this CTA's shared memory are in flight
        for (int g = 0; g < 2; ++g)
          if (q_ph[g].n > 0) mbar_wait_bounded(&q_full[g], q_ph[g].last(), 200000000ull);
        for (int i = 0; i < kSlots; ++i) {
          const uint32_t used = ring.round + (i < ring.slot ? 1 : 0);
          if (used > 0) mbar_wait_bounded(&full[i], (used - 1) & 1, 200000000ull);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // =================================== UMMA issuer ====================================
      if (elect_one()) {
        const uint32_t idesc_s = make_idesc_bf16(kRows, kTok, 0, 0);
        const uint32_t idesc_o = make_idesc_bf16(kRows, 64 * vb, 0, 1);
        const uint64_t q0 = make_sdesc(smem_u32(base + kQOff), 16, 1024, kSw128);
        const uint64_t k0 = make_sdesc(smem_u32(base + kSlotOff), 16, 1024, kSw128);
        const uint64_t r0 = make_sdesc(smem_u32(base + kRopeOff), 16, 1024, kSw128);
        const uint64_t v0 = make_sdesc(smem_u32(base + kSlotOff), kBlk, 1024, kSw128);
        const int ns = (p.dn + 15) / 16, nr = (p.dr + 15) / 16;   // K steps of 16 columns
        Ring ring;                               // the next tile to wait for
        Phase q_ph[2], p_ph[2], o_ph[2];
        uint32_t tile = 0;
        int k_slot = 0, v_slot = 0;              // slots of the current K and V tiles
        bool ok = true;
        auto wait_tile = [&]() -> int {
          const int slot = ring.slot;
          ok = ok && mbar_wait(&full[slot], ring.round & 1, wc);
          tc_fence_after();
          ring.next();
          return slot;
        };
        auto scores = [&](int g, bool last) {
          const uint32_t d = tmem + kColS + 128 * g;
          const uint64_t qa = q0 + ((g * kQGroup) >> 4);
          const uint64_t kb = k0 + ((k_slot * 2 * kBlk) >> 4);
          for (int i = 0; i < ns; ++i) {
            const uint64_t o = uint64_t(((i >> 2) * kBlk + (i & 3) * 32) >> 4);
            umma_bf16(d, qa + o, kb + o, idesc_s, i > 0 ? 1u : 0u);
          }
          const uint64_t qr = qa + ((2 * kBlk) >> 4), kr = r0 + (((tile & 1) * kBlk) >> 4);
          for (int i = 0; i < nr; ++i) umma_bf16(d, qr + 2 * i, kr + 2 * i, idesc_s, 1u);
          umma_commit(&s_full[g]);
          if (last) umma_commit(&q_empty[g]);
        };
        auto values = [&](int g, bool first) {
          const uint64_t vd = v0 + ((v_slot * 2 * kBlk) >> 4);
          if (first) {                           // O of the unit before has been read
            if (o_ph[g].n > 0) ok = ok && mbar_wait(&o_free[g], o_ph[g].last(), wc);
            o_ph[g].next();
          }
          const uint32_t parity = p_ph[g].next();
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i) {
            if (i % 4 == 0) {                     // the first half while the second is computed
              ok = ok && mbar_wait(&p_full[2 * g + i / 4], parity, wc);
              if (!ok) return;
              tc_fence_after();
            }
            umma_bf16_ts(tmem + kColO + 128 * g, tmem + kColS + 128 * g + 8 * i,
                         vd + ((i * 2048) >> 4), idesc_o, (!first || i > 0) ? 1u : 0u);
          }
          umma_commit(&pv_done[g]);
        };
        Unit w, after;
        bool have_after = false;                 // `after` holds the unit after w
        bool begun = false;                      // group 0's first scores of w are issued
        for (uint32_t k = 0; ok; ++k) {
          if (have_after) {
            w = after;
            have_after = false;
            if (w.h < 0) break;
          } else if (!next_unit(k, &w, false)) {
            break;
          }
          const int n = w.tiles();
          if (n == 0) continue;
          if (!begun) k_slot = wait_tile();
#pragma unroll
          for (int g = 0; g < 2; ++g)
            if (w.nt[g] > 0 && !(g == 0 && begun)) {
              ok = ok && mbar_wait(&q_full[g], q_ph[g].next(), wc);
              tc_fence_after();
              if (ok) scores(g, w.nt[g] == 1);
            }
          begun = false;
          if (ok) umma_commit(&empty[k_slot]);
          // The weights P_g(t) lie over S_g(t); the products with them are issued before the
          // scores S_g(t + 1) that overwrite both, and the tensor core works in order.
          for (int t = 0; ok && t < n; ++t) {
            v_slot = wait_tile();
            ++tile;
            bool have_k = false;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if (ok && t < w.nt[g]) values(g, t == 0);
              if (g == 1 && ok) umma_commit(&empty[v_slot]);
              if (ok && t + 1 < w.nt[g]) {
                if (!have_k) k_slot = wait_tile();
                have_k = true;
                if (ok) scores(g, t + 2 == w.nt[g]);
              }
              // Group 0 is done with this unit: its first scores of the next one, if that has
              // come in, go ahead of group 1's last product and keep its rows busy meanwhile.
              if (g == 0 && ok && t + 1 == n) {
                if (mbar_test_wait(&info_full[(k + 1) & 1], ((k + 1) >> 1) & 1)) {
                  next_unit(k + 1, &after, false);
                  have_after = true;
                  if (after.h >= 0 && after.nt[0] > 0 &&
                      mbar_test_wait(&full[ring.slot], ring.round & 1) &&
                      mbar_test_wait(&q_full[0], q_ph[0].n & 1)) {
                    q_ph[0].next();
                    k_slot = wait_tile();
                    if (ok) scores(0, after.nt[0] == 1);
                    begun = true;
                  }
                }
              }
            }
            if (ok && t + 1 < n) umma_commit(&empty[k_slot]);
          }
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ===================================== scheduler ====================================
      if (elect_one()) {
        const int split = kSplit ? p.split : 1, rank = kSplit ? int(cluster_ctarank()) : 0;
        int u = int(blockIdx.x) / split;
        for (uint32_t k = 0;; ++k) {
          Unit w;
          if (u >= 0) w = make_unit(p, u, rank, split);
          else w.h = -1;
          if (k >= 2 && !mbar_wait(&info_empty[k & 1], ((k >> 1) - 1) & 1, wc)) break;
          int* dst = reinterpret_cast<int*>(base + kInfoOff + 32 * (k & 1));
          dst[1] = w.h;
          if (u >= 0) {
            dst[0] = w.row0;
            dst[2] = w.b;
            dst[3] = w.L;
            dst[4] = w.ql;
            dst[5] = w.nt[0];
            dst[6] = w.nt[1];
            dst[7] = w.t0;
          }
          mbar_arrive(&info_full[k & 1]);
          if (u < 0) break;
          if (kSplit) {                          // one unit a cluster
            u = -1;
            continue;
          }
          if (!mbar_wait(want, k & 1, wc)) break;
          mbar_arrive_expect_tx(resp_full, 16);
          try_cancel_cta(base + kRespOff, resp_full);
          // (this wait ends by itself: the answer is the hardware's)
          if (!mbar_wait_bounded(resp_full, k & 1, kWaitLimitNs)) {
            *abort_flag = 1;
            if (p.dev_error) atomicOr(p.dev_error, MLA_DEVERR_TIMEOUT);
            break;
          }
          u = cancelled_cta(base + kRespOff);
          fence_proxy_async_smem();              // read before the next answer is written
        }
      }
      __syncwarp();
    }
  } else {
    // ======================================= rows =========================================
    reg_inc<kRegsRows>();
    const int g = (warp - 4) >> 2;
    const int sp = warp & 3;
    const uint32_t lane_base = uint32_t(32 * sp) << 16;
    const uint32_t t_s = tmem + lane_base + kColS + 128 * g;
    const uint32_t t_o = tmem + lane_base + kColO + 128 * g;
    const float c = p.scale_log2;
    Ring v_ring;                                 // the K or V tile before the next V tile
    uint32_t tiles = 0;                          // of this group so far
    bool ok = true;
    Unit w, staged;                              // kSplit: the unit whose part is in O
    staged.h = -1;
    float m_part = kRefInit, l_part = 0.0f;
    bool bad_part = false;
    // The k-th unit has values among those that some row does not see which are infinite or NaN. The
    // stamp of a unit four before may go: no group is three units behind the other.
    volatile uint32_t* bad_unit = reinterpret_cast<uint32_t*>(base + kBadOff);
    // Those values, taken out of the tiles, for the rows that see them: column e + i of this thread's
    // row in o[i].
    auto add_hidden = [&](const Unit& u, int ng, float* o, int e) {
      const int qi = u.row0 + g * kRows + 32 * sp + lane;
      const int last = min(min(u.L - 1, u.L - u.ql + qi), (u.t0 + ng) * kTok - 1);
#pragma unroll 1
      for (int t = max(u.first_hidden(p), u.t0 * kTok); t <= last; ++t) {
        const uint16_t* v = p.v + (int64_t(u.b) * p.kv_len + t) * p.v_token + u.h * p.v_head + e;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          if (e + i >= p.dv) break;
          const uint4 x = *reinterpret_cast<const uint4*>(v + i);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((w[j] & 0x7F80u) == 0x7F80u) o[i + 2 * j] += __uint_as_float(w[j] << 16);
            if ((w[j] & 0x7F800000u) == 0x7F800000u)
              o[i + 2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
          }
        }
      }
    };
    for (uint32_t k = 0; ok && next_unit(k, &w, true); ++k) {
      const int n = w.tiles(), ng = g == 0 ? w.nt[0] : w.nt[1];
      const int L = w.L, ql = w.ql;
      const int qi = w.row0 + g * kRows + 32 * sp + lane;     // query row of this thread
      // last token that this row sees (may be negative)
      const int lim = min(L - 1, p.causal ? L - ql + qi : L - 1);
      const int hidden = w.first_hidden(p);
      float m = kRefInit, l = 0.0f;
      for (int j = 0; j < n; ++j) {
        v_ring.next();                           // V of tile j
        const Ring at = v_ring;
        v_ring.next();
        if (j >= ng) continue;
        const uint32_t parity = tiles & 1;
        ++tiles;
        const int t0 = (w.t0 + j) * kTok;
        // Value rows past the context may hold anything, and a weight of 0 times NaN is NaN: zeros. Of a
        // token that some row of the unit does not see, infinities and NaN become zeros, and the rows
        // that see it add them at the end. Group 0 does this for its tiles, which the product of group
        // 1 meets after group 0's, and group 1 for those that only it has. Where there is a tile
        // before, that is done by the time the scores come (for every tile after them: 2 x 4096 causal
        // rows 344 us, 331 without any). Its scores also say that the slot's last keys had landed, so
        // that the phase waited for is this tile's; with the unit's first tile its own scores do.
        const bool hides = t0 + kTok > hidden && (g == 0 || j >= w.nt[0]);
        auto hide = [&]() {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[at.slot], at.round & 1, wc));
          const int tok = 32 * sp + lane;
          if (ok && t0 + tok >= hidden) {
            uint8_t* v = base + kSlotOff + at.slot * 2 * kBlk + tok * 128;
            bool bad = false;
            for (int e = 0; e < vb; ++e) bad |= hide_token(v + e * kBlk, t0 + tok >= L, lane);
            if (bad) bad_unit[k & 3] = k + 1;
          }
          fence_proxy_async_smem();
        };
        if (hides && j > 0) hide();
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&s_full[g], parity, wc));
        if (ok && hides && j == 0) hide();
        if (!ok) break;
        tc_fence_after();
        float s[kTok];
#pragma unroll
        for (int e = 0; e < kTok; e += 32) tmem_ld32(t_s + e, s + e);
        tmem_wait_ld();
        if (t0 + kTok - 1 > lim) {
#pragma unroll
          for (int e = 0; e < kTok; ++e)
            if (t0 + e > lim) s[e] = -INFINITY;
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max3(s[i], s[i + 4], s[i + 8]);
#pragma unroll
        for (int e = 12; e + 8 <= kTok; e += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], s[e + i], s[e + 4 + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], s[kTok - 4 + i]);
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
        float alpha = 1.0f;
        if (top > m + kLazyThreshold) {
          alpha = ex2_approx(m - top);           // 0 while m is still kRefInit
          l *= alpha;
          m = top;
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
          // O holds this row's earlier tiles, once their product is done
          ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[g], parity ^ 1u, wc));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int e = 0; e < 64 * vb; e += 16) {
            float o[16];
            tmem_ld16(t_o + e, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_st16(t_o + e, o);
          }
        }
        // weights 2^(s * scale - m), in pairs, half a tile at a time
        const float2 c2 = make_float2(c, c), m2 = make_float2(-m, -m);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int e = 64 * half; e < 64 * half + 64; e += 32) {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 y = fma_f32x2(make_float2(s[e + 2 * i], s[e + 2 * i + 1]), c2, m2);
              y.x = ex2_approx(y.x);
              y.y = ex2_approx(y.y);
              sum[i & 1] = add_f32x2(sum[i & 1], y);
              x[i] = cvt_bf16x2(y.x, y.y);
            }
            tmem_st16(t_s + e / 2, reinterpret_cast<const float*>(x));
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * g + half]);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      // ----------------------------------- epilogue --------------------------------------
      if (ng > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[g], (tiles - 1) & 1, wc));
        if (!ok) break;
        tc_fence_after();
      }
      if constexpr (kSplit) {                    // the cluster's merge follows below
        staged = w;
        m_part = m;
        l_part = l;
        bad_part = ng > 0 && bad_unit[k & 3] == k + 1;
        break;
      }
      const bool real = qi < ql, bad = ng > 0 && bad_unit[k & 3] == k + 1;
      const int64_t row = (int64_t(w.b) * p.q_len + qi) * p.heads + w.h;
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;          // NaN stays NaN
      if (real) p.lse[row] = l != 0.0f ? (m + __log2f(l)) * kLn2 : -INFINITY;
      uint16_t* out = p.o + row * p.dv;
#pragma unroll 1
      for (int e = 0; e < 64 * vb; e += 32) {
        float o[32];
        if (ng > 0) {
          tmem_ld32(t_o + e, o);
          tmem_wait_ld();
        }
        if (bad) add_hidden(w, ng, o, e);
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t x[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            x[y] = inv == 0.0f ? 0u : cvt_bf16x2(o[i + 2 * y] * inv, o[i + 2 * y + 1] * inv);
          if (real && e + i < p.dv)
            *reinterpret_cast<uint4*>(out + e + i) = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      if (ng > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[g]);
      }
    }
    // after a wait that ran out this CTA's rows stay unwritten; the error word tells
    tc_fence_before();
    if constexpr (kSplit) {
      // Unnormalised O, the reference and the sum into shared memory, once the products of both
      // groups have read Q, K and V there (all eight warps come here, after an abort too).
      named_bar_sync(1, 256);
      if (staged.h >= 0) {
        const bool any = (g == 0 ? staged.nt[0] : staged.nt[1]) > 0;
        const int at = 32 * sp + lane;
        *stage_ml(base, g, at) = make_float2(m_part, l_part);
#pragma unroll 1
        for (int e = 0; e < 64 * vb; e += 32) {
          float o[32];
          if (any) {
            tmem_ld32(t_o + e, o);
            tmem_wait_ld();
          }
          if (bad_part) add_hidden(staged, g == 0 ? staged.nt[0] : staged.nt[1], o, e);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *stage_o(base, g, (e + i) / 4, at) =
                any ? make_float4(o[i], o[i + 1], o[i + 2], o[i + 3])
                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        tc_fence_before();
      }
      cluster_sync_all();                        // every CTA's part is in its shared memory
      // This CTA merges its share of the columns of all rows: o = sum_i 2^(m_i - M) O_i / sum_i
      // 2^(m_i - M) l_i over the cluster's CTAs, M = max m_i (a part without tokens has l_i = 0
      // and the least m_i).
      const int qi = staged.row0 + g * kRows + 32 * sp + lane, rl = 32 * sp + lane;
      if (staged.h >= 0 && qi < staged.ql) {
        const int s = p.split, rank = int(cluster_ctarank());
        float m = kRefInit;
        for (int i = 0; i < s; ++i)
          m = fmaxf(m, ld_cluster_f32(map_to_rank(smem_u32(&stage_ml(base, g, rl)->x), i)));
        float wgt[8], l = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= s) break;
          const uint32_t at = map_to_rank(smem_u32(stage_ml(base, g, rl)), i);
          wgt[i] = ex2_approx(ld_cluster_f32(at) - m);
          l += wgt[i] * ld_cluster_f32(at + 4);
        }
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;        // NaN stays NaN
        const int64_t row = (int64_t(staged.b) * p.q_len + qi) * p.heads + staged.h;
        if (rank == 0) p.lse[row] = l != 0.0f ? (m + __log2f(l)) * kLn2 : -INFINITY;
        for (int e = 8 * rank; e < p.dv; e += 8 * s) {
          float o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i >= s) break;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 v =
                  ld_cluster_v4(map_to_rank(smem_u32(stage_o(base, g, e / 4 + q, rl)), i));
              o[4 * q] += wgt[i] * v.x;
              o[4 * q + 1] += wgt[i] * v.y;
              o[4 * q + 2] += wgt[i] * v.z;
              o[4 * q + 3] += wgt[i] * v.w;
            }
          }
          uint32_t x[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            x[y] = inv == 0.0f ? 0u : cvt_bf16x2(o[2 * y] * inv, o[2 * y + 1] * inv);
          *reinterpret_cast<uint4*>(p.o + row * p.dv + e) = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
    }
  }
  if constexpr (kSplit) {
    if (warp < 4) {
      __syncwarp();
      cluster_sync_all();
    }
    __syncwarp();                                // (the merge's rows; a warp comes as one)
    cluster_sync_all();                          // nobody leaves while its part may be read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

int prefill_max_clusters(int split) {
  // by device and cluster size, plus one; 0: not asked yet
  static std::atomic<int> known[64][kPrefillMaxSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < 64) {
    const int n = known[dev][split].load(std::memory_order_relaxed);
    if (n > 0) return n - 1;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(mla_prefill_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(kSmem)) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, mla_prefill_kernel<true>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < 64) known[dev][split].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <bool kSplit>
static cudaError_t launch_prefill_t(const PrefillParams& p, unsigned units, cudaStream_t stream) {
  static std::atomic<bool> known{false};
  cudaError_t e = check_launch_regs(mla_prefill_kernel<kSplit>, kRegsLaunch, &known);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(
      mla_prefill_kernel<kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
  if (e != cudaSuccess) return e;
  return launch_pdl(mla_prefill_kernel<kSplit>, dim3(units * p.split), dim3(kThreads), kSmem,
                    stream, p.split, p);
}

cudaError_t launch_prefill(const PrefillParams& p, cudaStream_t stream) {
  const unsigned units = unsigned((p.q_len + 2 * kRows - 1) / (2 * kRows)) * p.heads * p.batch;
  return p.split > 1 ? launch_prefill_t<true>(p, units, stream)
                     : launch_prefill_t<false>(p, units, stream);
}

}  // namespace mla
