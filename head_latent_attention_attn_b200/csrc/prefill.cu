// prefill.cu - mla_prefill_attn on sm_100a: attention in its expanded form, a key and a value
// per head, the rotary key shared by the heads of a group.
//
//   s[i, t] = scale (q_nope[i] . k_nope[t] + q_pe[i] . k_pe[t]),  o = softmax(s) v
//
// Against the absorbed form over the latent (r + d_r columns of scores, r of output) this needs
// d_n + d_r + d_v multiplications a (query, token) pair instead of 2 r + d_r: 320 instead of 1088
// for the DeepSeek-V2 layer. It pays once a context's keys and values are expanded for enough
// query rows, as in a prefill chunk. Bound by the tensor cores: a 128 x 128 tile of one head is
// 128 * 128 * (192 + 128) multiplications, 1280 cycles of an SM, against 1024 cycles for its
// exponentials and 80 KB of operands that the heads' other query tiles find in L2.
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
// Roles (384 threads): warp 0 TMA producer, warp 1 UMMA issuer, warps 4-7 and 8-11 the rows of
// group 0 and 1. Registers: 168 a thread at launch, 40 for the issuers' group, 232 for the rows'.
//
// Softmax in the log2 domain with a reference maximum that moves only when a score exceeds it by
// more than 8 (weights stay <= 256), so that O is rescaled rarely; the row itself then does it.
#include <math.h>

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
constexpr int kRegsLaunch = 168, kRegsIssue = 40, kRegsRows = 232;
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
constexpr uint32_t kBars = 2 + 2 * kSlots + 8;
constexpr uint32_t kSmem = kMiscOff + 64 + 8 * kBars + 1024;   // + alignment slack
static_assert(kSmem <= 232448, "shared memory of a CTA");

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + kMiscOff);
  volatile int* abort_flag = reinterpret_cast<int*>(base + kMiscOff) + 1;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(base + kMiscOff + 64);   // [2]
  uint64_t* full = q_full + 2;                   // [slot] K or V tile landed
  uint64_t* empty = full + kSlots;               // [slot]
  uint64_t* s_full = empty + kSlots;             // [group] scores computed
  uint64_t* p_full = s_full + 2;                 // [group][half] weights of 64 tokens written
  uint64_t* pv_done = p_full + 4;                // [group] PV of the group's tile done
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{abort_flag, p.dev_error};

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);              // the group's four warps
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // set-up above may overlap the previous kernel; from here on global memory is touched
  grid_dep_wait();
  grid_dep_launch();

  // the longest tiles first: a causal chunk's last rows see the most tokens
  const int qt = int(gridDim.x) - 1 - int(blockIdx.x);
  const int h = blockIdx.y, b = blockIdx.z;
  int L = p.seq_lens[b], ql = p.q_lens ? p.q_lens[b] : p.q_len;
  const bool bad = L < 0 || L > p.kv_len || ql < 0 || ql > p.q_len;
  if (bad) {
    if (threadIdx.x == 0 && p.dev_error) atomicOr(p.dev_error, MLA_DEVERR_BOUNDS);
    L = 0;
    ql = max(0, min(ql, p.q_len));
  }
  // tiles that group g's rows see: those of its last row
  const int row0 = qt * 2 * kRows;
  int nt[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int first = row0 + g * kRows, last = min(first + kRows, ql) - 1;
    const int seen = first >= ql ? 0 : p.causal ? max(0, min(L, L - ql + last + 1)) : L;
    nt[g] = (seen + kTok - 1) / kTok;
  }
  const int n = max(nt[0], nt[1]);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int nb = (p.dn + 63) / 64, vb = (p.dv + 63) / 64;   // 64-column blocks

  if (warp < 4) {
    reg_dec<kRegsIssue>();
    if (warp == 0) {
      // =================================== TMA producer ===================================
      if (n > 0 && elect_one()) {
        prefetch_tensormap(&p.tm_k);
        prefetch_tensormap(&p.tm_v);
        prefetch_tensormap(&p.tm_q);
        const int rope = p.dr > 0 ? 1 : 0, kg = h / p.heads_per_group;
        auto load_q = [&](int g) {
          uint8_t* dst = base + kQOff + g * kQGroup;
          mbar_arrive_expect_tx(&q_full[g], uint32_t(nb + rope) * kBlk);
          for (int k = 0; k < nb; ++k)
            tma_load_4d(dst + k * kBlk, &p.tm_q, 64 * k, h, row0 + g * kRows, b, &q_full[g]);
          if (rope) tma_load_4d(dst + 2 * kBlk, &p.tm_qr, 0, h, row0 + g * kRows, b, &q_full[g]);
        };
        // tile u / 2: K for even u, V for odd u. A K tile's rotary part goes to rope slot
        // (u / 2) % 2, which is free when the slot of unit u - 3 (V of two tiles before) is:
        // its release follows every product with that tile's keys.
        auto load_unit = [&](int u) {
          uint8_t* dst = base + kSlotOff + (u % kSlots) * 2 * kBlk;
          uint64_t* bar = &full[u % kSlots];
          const int t0 = (u / 2) * kTok;
          if (u & 1) {
            mbar_arrive_expect_tx(bar, uint32_t(vb) * kBlk);
            for (int k = 0; k < vb; ++k) tma_load_4d(dst + k * kBlk, &p.tm_v, 64 * k, h, t0, b, bar);
          } else {
            mbar_arrive_expect_tx(bar, uint32_t(nb + rope) * kBlk);
            for (int k = 0; k < nb; ++k) tma_load_4d(dst + k * kBlk, &p.tm_k, 64 * k, h, t0, b, bar);
            if (rope)
              tma_load_4d(base + kRopeOff + ((u / 2) & 1) * kBlk, &p.tm_kr, 0, kg, t0, b, bar);
          }
        };
        if (nt[0] > 0) load_q(0);
        int u = 0;
        load_unit(u++);
        if (nt[1] > 0) load_q(1);
        for (; u < 2 * n; ++u) {
          if (u >= kSlots && !mbar_wait(&empty[u % kSlots], (u / kSlots - 1) & 1, wc)) break;
          load_unit(u);
        }
        // never leave while copies into this CTA's shared memory are in flight
        for (int g = 0; g < 2; ++g)
          if (nt[g] > 0) mbar_wait_bounded(&q_full[g], 0, 200000000ull);
        for (int v = max(0, u - kSlots); v < u; ++v)
          mbar_wait_bounded(&full[v % kSlots], (v / kSlots) & 1, 200000000ull);
      }
      __syncwarp();
    } else if (warp == 1) {
      // =================================== UMMA issuer ====================================
      if (n > 0 && elect_one()) {
        const uint32_t idesc_s = make_idesc_bf16(kRows, kTok, 0, 0);
        const uint32_t idesc_o = make_idesc_bf16(kRows, 64 * vb, 0, 1);
        const uint64_t q0 = make_sdesc(smem_u32(base + kQOff), 16, 1024, kSw128);
        const uint64_t k0 = make_sdesc(smem_u32(base + kSlotOff), 16, 1024, kSw128);
        const uint64_t r0 = make_sdesc(smem_u32(base + kRopeOff), 16, 1024, kSw128);
        const uint64_t v0 = make_sdesc(smem_u32(base + kSlotOff), kBlk, 1024, kSw128);
        const int ns = (p.dn + 15) / 16, nr = (p.dr + 15) / 16;   // K steps of 16 columns
        bool ok = true;
        auto wait_unit = [&](int u) {
          ok = ok && mbar_wait(&full[u % kSlots], (u / kSlots) & 1, wc);
          tc_fence_after();
        };
        auto scores = [&](int g, int j) {
          const uint32_t d = tmem + kColS + 128 * g;
          const uint64_t qa = q0 + ((g * kQGroup) >> 4);
          const uint64_t kb = k0 + ((((2 * j) % kSlots) * 2 * kBlk) >> 4);
          for (int i = 0; i < ns; ++i) {
            const uint64_t o = uint64_t(((i >> 2) * kBlk + (i & 3) * 32) >> 4);
            umma_bf16(d, qa + o, kb + o, idesc_s, i > 0 ? 1u : 0u);
          }
          const uint64_t qr = qa + ((2 * kBlk) >> 4), kr = r0 + (((j & 1) * kBlk) >> 4);
          for (int i = 0; i < nr; ++i) umma_bf16(d, qr + 2 * i, kr + 2 * i, idesc_s, 1u);
          umma_commit(&s_full[g]);
        };
        auto values = [&](int g, int j) {
          const uint64_t vd = v0 + ((((2 * j + 1) % kSlots) * 2 * kBlk) >> 4);
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i) {
            if (i % 4 == 0) {                     // the first half while the second is computed
              ok = ok && mbar_wait(&p_full[2 * g + i / 4], j & 1, wc);
              if (!ok) return;
              tc_fence_after();
            }
            umma_bf16_ts(tmem + kColO + 128 * g, tmem + kColS + 128 * g + 8 * i,
                         vd + ((i * 2048) >> 4), idesc_o, (j > 0 || i > 0) ? 1u : 0u);
          }
          umma_commit(&pv_done[g]);
        };
        wait_unit(0);
        for (int g = 0; ok && g < 2; ++g)
          if (nt[g] > 0) {
            ok = mbar_wait(&q_full[g], 0, wc);
            tc_fence_after();
            if (ok) scores(g, 0);
          }
        if (ok) umma_commit(&empty[0]);
        // The weights P_g(j) lie over S_g(j); the products with them are issued before the
        // scores S_g(j + 1) that overwrite both, and the tensor core works in order.
        for (int j = 0; ok && j < n; ++j) {
          wait_unit(2 * j + 1);
          bool have_k = false;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (ok && j < nt[g]) values(g, j);
            if (g == 1 && ok) umma_commit(&empty[(2 * j + 1) % kSlots]);
            if (ok && j + 1 < nt[g]) {
              if (!have_k) wait_unit(2 * j + 2);
              have_k = true;
              if (ok) scores(g, j + 1);
            }
          }
          if (ok && j + 1 < n) umma_commit(&empty[(2 * j + 2) % kSlots]);
        }
      }
      __syncwarp();
    }
  } else {
    // ======================================= rows =========================================
    reg_inc<kRegsRows>();
    const int g = (warp - 4) >> 2;
    const int sp = warp & 3;
    const int qi = row0 + g * kRows + 32 * sp + lane;     // query row of this thread
    const uint32_t lane_base = uint32_t(32 * sp) << 16;
    const uint32_t t_s = tmem + lane_base + kColS + 128 * g;
    const uint32_t t_o = tmem + lane_base + kColO + 128 * g;
    // last token that this row sees (may be negative)
    const int lim = min(L - 1, p.causal ? L - ql + qi : L - 1);
    const float c = p.scale_log2;
    float m = kRefInit, l = 0.0f;
    const int ng = g == 0 ? nt[0] : nt[1];
    for (int j = 0; j < ng; ++j) {
      const bool got = __all_sync(0xffffffffu, mbar_wait(&s_full[g], j & 1, wc));
      if (!got) break;
      tc_fence_after();
      float s[kTok];
#pragma unroll
      for (int k = 0; k < kTok; k += 32) tmem_ld32(t_s + k, s + k);
      tmem_wait_ld();
      const int t0 = j * kTok;
      if (t0 + kTok - 1 > lim) {
#pragma unroll
        for (int k = 0; k < kTok; ++k)
          if (t0 + k > lim) s[k] = -INFINITY;
      }
      float mx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i] = max3(s[i], s[i + 4], s[i + 8]);
#pragma unroll
      for (int k = 12; k + 8 <= kTok; k += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], s[k + i], s[k + 4 + i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], s[kTok - 4 + i]);
      const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
      float alpha = 1.0f;
      if (top > m + kLazyThreshold) {
        alpha = ex2_approx(m - top);             // 0 while m is still kRefInit
        l *= alpha;
        m = top;
      }
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
        // O holds this row's earlier tiles, once their product is done
        const bool done = __all_sync(0xffffffffu, mbar_wait(&pv_done[g], (j - 1) & 1, wc));
        if (!done) break;
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < 64 * vb; k += 16) {
          float o[16];
          tmem_ld16(t_o + k, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] *= alpha;
          tmem_st16(t_o + k, o);
        }
      }
      if (t0 + kTok > L) {
        // value rows past the context may hold anything (0-weight x NaN is NaN): zero them. Both
        // groups do so; the second writes zeros over zeros.
        const int u = 2 * j + 1;
        const bool landed = __all_sync(
            0xffffffffu, mbar_wait(&full[u % kSlots], (u / kSlots) & 1, wc));
        if (!landed) break;
        const int tok = 32 * sp + lane;
        if (t0 + tok >= L) {
          uint8_t* v = base + kSlotOff + (u % kSlots) * 2 * kBlk + tok * 128;
          for (int k = 0; k < vb; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(v + k * kBlk + 16 * i) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      // weights 2^(s * scale - m), in pairs, half a tile at a time
      const float2 c2 = make_float2(c, c), m2 = make_float2(-m, -m);
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int k = 64 * half; k < 64 * half + 64; k += 32) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 e = fma_f32x2(make_float2(s[k + 2 * i], s[k + 2 * i + 1]), c2, m2);
            e.x = ex2_approx(e.x);
            e.y = ex2_approx(e.y);
            sum[i & 1] = add_f32x2(sum[i & 1], e);
            w[i] = cvt_bf16x2(e.x, e.y);
          }
          tmem_st16(t_s + k / 2, reinterpret_cast<const float*>(w));
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * g + half]);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }
    // ------------------------------------ epilogue ---------------------------------------
    bool fin = true;
    if (ng > 0) fin = __all_sync(0xffffffffu, mbar_wait(&pv_done[g], (ng - 1) & 1, wc));
    tc_fence_after();
    fin = fin && *abort_flag == 0;
    const bool real = qi < ql;
    const float inv = (fin && l > 0.0f) ? 1.0f / l : (l > 0.0f || l == 0.0f ? 0.0f : l);
    const int64_t row = (int64_t(b) * p.q_len + qi) * p.heads + h;
    if (real)
      p.lse[row] = (fin && l > 0.0f) ? (m + __log2f(l)) * kLn2 : (l == 0.0f ? -INFINITY : l);
    uint16_t* out = p.o + row * p.dv;
#pragma unroll 1
    for (int k = 0; k < p.dv; k += 16) {
      float o[16];
      if (ng > 0) {
        tmem_ld16(t_o + k, o);
        tmem_wait_ld();
      }
      if (real) {
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          if (k + i >= p.dv) break;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = l == 0.0f ? 0u : cvt_bf16x2(o[i + 2 * e] * inv, o[i + 2 * e + 1] * inv);
          *reinterpret_cast<uint4*>(out + k + i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    tc_fence_before();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

cudaError_t launch_prefill(const PrefillParams& p, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(
      mla_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
  if (e != cudaSuccess) return e;
  const dim3 grid((p.q_len + 2 * kRows - 1) / (2 * kRows), p.heads, p.batch);
  return launch_pdl(mla_prefill_kernel, grid, dim3(kThreads), kSmem, stream, 1, p);
}

}  // namespace mla
