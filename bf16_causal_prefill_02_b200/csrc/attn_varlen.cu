// attn_varlen.cu -- causal forward (prefill) attention over packed prompts of
// different lengths, sm_100a, BF16 and FP8 e4m3, head dims (128,128) and MLA
// (192,128).
//
// Sequence b holds query rows cu_q[b] .. cu_q[b+1] - 1 and key rows cu_k[b] ..
// cu_k[b+1] - 1 of the packed tensors.  Per sequence the mathematics is that
// of attn_fwd.cu (same P, same FP8 modes, key blocks counted from the
// sequence's first key); what differs is the way to it:
//
//   * The offsets are read on the device, so the host launches a bound on the
//     work, and resident CTAs take over blocks that have not started
//     (varlen_sched.cuh).  Ragged lengths need no schedule on the host and no
//     counter in memory, and a unit's loads overlap the last one's tail.
//   * Units run in groups of heads that share the L2, inside a group sequence
//     by sequence, each sequence's longest tiles first.
//   * The last key tile of a sequence ends in rows of the next one, or in rows
//     of nothing.  Their scores are masked (weights exactly 0), and V's rows
//     are set to 0 in shared memory before the product, so that what they hold
//     (infinities and NaN too) does not matter.
//
// Bound by the softmax chain of a tile (the tensor pipe is 41-61% busy): after
// a pause, 16/16 heads 192/128 over 12136 rows 326 us (1174 TFLOP/s), FP8 Lean
// P, 32/8 heads, 5060 rows in chunks over 19793 keys 268 us (1544), one prompt of
// 16384 rows 1246 us (1765), bf16 4096 rows 129 us (1066).
//
// Warps: 0-7 softmax and epilogue (a 16-lane group of TMEM rows each, threads
// t and t + 16 share a query row, one 64-key half of the tile each), 8 TMA
// producer, 9 tcgen05 issuer, 10 scheduler.  Tensor memory as in attn_fwd.cu:
// S0 [0,128), S1 [128,256) with P written over them, O [256,384), FP8: row
// sum [384,400), scales of P [400,408) and of V [408,416).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "attn_math.cuh"
#include "serving.h"
#include "sm100_ptx.cuh"
#include "varlen_sched.cuh"

namespace zq {

namespace {

constexpr int kSmThreads = 256;  // softmax
constexpr int kVarThreads = kSmThreads + 96;
constexpr int kProducer = 8, kIssuer = 9, kScheduler = 10;
constexpr uint32_t kS0 = 0, kO = 256, kRS = 384, kSFA = 400, kSFB = 408;
constexpr uint32_t kCols = 512;
// Degree of the software exp2: 4 (2.7e-6) measured the same as the 3 (7.5e-5)
// of the fixed-batch kernel and keeps the lse of short rows to fp32.
constexpr int kPolyDegree = 4;

template <int DT, int DQK>
struct VGeo {
  static constexpr int DV = 128;
  static constexpr int ES = DT == 0 ? 2 : 1;
  static constexpr int QROW = DQK * ES;
  static constexpr int NCH = (QROW + 127) / 128;         // 128-byte chunks (the last may be 64)
  static constexpr bool NARROW = QROW % 128 != 0;
  static constexpr int QBYTES = kTile * QROW;
  static constexpr int KBYTES = QBYTES;
  static constexpr int VBYTES = kTile * DV * ES;
  static constexpr int VCH = DV * ES / 128;
  static constexpr int QK_STEPS = QROW / 32;             // 32 bytes of K per MMA
  static constexpr int PV_STEPS = DT == 0 ? 8 : 4;       // 16 (bf16) / 32 (fp8) keys per MMA
  static constexpr int NS = DT == 1 ? 4 : (DQK == 128 ? 3 : 2);
  static constexpr bool SPLIT = NS == 2;                 // K and V refill independently (see attn_fwd.cu)
  static constexpr int OFF_K = QBYTES;
  static constexpr int OFF_V = OFF_K + NS * KBYTES;
  static constexpr int OFF_ONES = OFF_V + NS * VBYTES;   // FP8: e4m3 ones for the rounded row sum
  static constexpr int ONES_BYTES = DT == 1 ? 16384 : 0;
  static constexpr int OFF_SF = OFF_ONES + ONES_BYTES;   // FP8: [2 buf] 512 B scale tiles
  static constexpr int OFF_PREFIX = OFF_SF + (DT == 1 ? 1024 : 0);
  static constexpr int OFF_UNIT = OFF_PREFIX + kSchedChunks * 4;
  static constexpr int OFF_CLC = OFF_UNIT + 2 * 32;
  static constexpr int OFF_BAR = OFF_CLC + 16;
  static constexpr int NBAR = 4 * NS + 15;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;  // + alignment slack
  static_assert(SMEM <= 232448, "227 KB of shared memory per CTA");
};

// A work unit, as the scheduler hands it out (32 bytes of shared memory).
struct VUnit {
  int b, h;          // sequence, query head
  int q_row, rows;   // first packed query row of the tile, rows of it that are the sequence's
  int k_row, len_k;  // first packed key row of the sequence, its keys
  int lim0;          // last key its first row may see (before the clamp to len_k - 1)
  int n_kv;          // key tiles to visit; -1: no more units
};

template <int DT, int DQK, int MODE, int BS>
__global__ void __launch_bounds__(kVarThreads, 1)
    attn_varlen_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ2,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmK2,
                       const __grid_constant__ CUtensorMap tmV, const VarlenParams p) {
  using G = VGeo<DT, DQK>;
  constexpr int NS = G::NS, DV = G::DV;
  constexpr unsigned kFull = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::OFF_BAR);
  uint64_t* bar_kfull = bars;               // [NS] K_j (and V_j unless split) landed
  uint64_t* bar_kfree = bar_kfull + NS;     // [NS] split: QK_j done
  uint64_t* bar_vfull = bar_kfree + NS;     // [NS] split: V_j landed
  uint64_t* bar_vfree = bar_vfull + NS;     // [NS] PV_j done: the stage is free, O holds tiles <= j
  uint64_t* bar_sfull = bar_vfree + NS;     // [2] QK_j done
  uint64_t* bar_pfull = bar_sfull + 2;      // [2] P_j written
  uint64_t* bar_ufull = bar_pfull + 2;      // [2] unit slot filled
  uint64_t* bar_ufree = bar_ufull + 2;      // [2] unit slot read by all roles
  uint64_t* bar_q = bar_ufree + 2;          // Q landed
  uint64_t* bar_qfree = bar_q + 1;          // last QK of a unit done
  uint64_t* bar_ofinal = bar_qfree + 1;     // last PV of a unit done
  uint64_t* bar_ofree = bar_ofinal + 1;     // softmax read O of a unit
  uint64_t* bar_clc = bar_ofree + 1;        // the answer to a request for a block
  uint64_t* bar_want = bar_clc + 1;         // the producer issued a unit's last load
  uint64_t* bar_drain = bar_want + 1;       // after an abort: the issuer's work landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_drain + 1);  // (bars + NBAR)
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  VUnit* units = reinterpret_cast<VUnit*>(smem + G::OFF_UNIT);
  int* prefix = reinterpret_cast<int*>(smem + G::OFF_PREFIX);
  uint32_t* sf_smem = reinterpret_cast<uint32_t*>(smem + G::OFF_SF);  // layout: attn_fwd.cu
  void* clc = smem + G::OFF_CLC;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4 * NS; ++s) mbar_init(bars + s, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_sfull + s, 1);
      mbar_init(bar_pfull + s, kSmThreads + p.withhold);
      mbar_init(bar_ufull + s, 1);
      mbar_init(bar_ufree + s, 2 + kSmThreads / 32);  // producer, issuer, softmax warps
    }
    mbar_init(bar_q, 1);
    mbar_init(bar_qfree, 1);
    mbar_init(bar_ofinal, 1);
    mbar_init(bar_ofree, kSmThreads);
    mbar_init(bar_clc, 1);
    mbar_init(bar_want, 1);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (DT == 1) {  // e4m3 1.0 = 0x38
    uint32_t* ones = reinterpret_cast<uint32_t*>(smem + G::OFF_ONES);
    for (int i = threadIdx.x; i < G::ONES_BYTES / 4; i += kVarThreads) ones[i] = 0x38383838u;
    fence_proxy_async_smem();
  }
  launch_dependents();
  wait_previous_kernel();
  UnitCount count;  // (the scheduler's; beside the set-up of the others)
  if (warp == kScheduler) count = count_tiles<kTile>(p, prefix, lane);
  if (warp == kIssuer) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  if (warp == kProducer && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    if (G::NARROW) {
      tma_prefetch_desc(&tmQ2);
      tma_prefetch_desc(&tmK2);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint64_t lim = p.timeout_ns;
  int q_loads = 0, x_last = -1, xk_last = -1, xv_last = -1;  // last loads armed (drain)
  bool asked = false;                                        // a request for a block is out
  int clc_n = 0;

  auto fail = [&]() {
    *abort_flag = 1;
    if (p.status) atomicExch(p.status, -7 /* ZQ_ERR_TIMEOUT */);
  };
  // the k-th unit of this CTA
  auto unit_wait = [&](int k) -> bool { return mbar_wait(bar_ufull + (k & 1), (k >> 1) & 1, lim, abort_flag); };

  if (warp == kScheduler) {
    // ----------------------------------------------------------- scheduler
    const bool ok = schedule_units<kTile>(
        p, p.Hq, count, prefix, clc, bar_clc, bar_want, bar_ufull, bar_ufree, abort_flag, lane, asked, clc_n, [&](int slot, const SeqTile* s) {
          VUnit w = {};
          w.n_kv = -1;
          if (s) {
            w.b = s->b;
            w.h = s->h;
            w.q_row = s->q0 + s->t * kTile;
            w.rows = min(s->q1 - w.q_row, kTile);
            w.k_row = s->k0;
            w.len_k = s->k1 - s->k0;
            w.lim0 = p.causal ? s->t * kTile + w.len_k - (s->q1 - s->q0) : w.len_k - 1;
            // key tiles up to the last key that the tile's last row sees
            const int max_key = p.causal ? min(w.lim0 + w.rows - 1, w.len_k - 1) : w.len_k - 1;
            w.n_kv = max_key < 0 ? 0 : max_key / kTile + 1;
          }
          units[slot] = w;
        });
    if (!ok && lane == 0) fail();
  } else if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int jt = 0, nq = 0;
      bool ok = true;
      for (int k = 0;; ++k) {
        if (!unit_wait(k)) { ok = false; break; }
        const VUnit w = units[k & 1];
        mbar_arrive(bar_ufree + (k & 1));
        if (w.n_kv < 0) break;
        if (w.n_kv == 0) {
          mbar_arrive(bar_want);
          continue;
        }
        const int g = w.h / p.group;
        // Q of the previous unit is read until its last QK completes
        if (nq > 0 && !mbar_wait(bar_qfree, (nq - 1) & 1, lim, abort_flag)) { ok = false; break; }
        mbar_arrive_expect_tx(bar_q, G::QBYTES);
        ++q_loads;
#pragma unroll
        for (int c = 0; c < G::NCH; ++c) {
          const bool narrow = c == G::NCH - 1 && G::NARROW;
          tma_load_4d(smem + c * 16384, narrow ? (const void*)&tmQ2 : (const void*)&tmQ, bar_q, c * 128 / G::ES, w.h, w.q_row, 0);
        }
        auto load_k = [&](int j, int s) {
#pragma unroll
          for (int c = 0; c < G::NCH; ++c) {
            const bool narrow = c == G::NCH - 1 && G::NARROW;
            tma_load_4d(smem + G::OFF_K + s * G::KBYTES + c * 16384, narrow ? (const void*)&tmK2 : (const void*)&tmK,
                        bar_kfull + s, c * 128 / G::ES, g, w.k_row + j * kTile, 0);
          }
        };
        auto load_v = [&](int j, int s, uint64_t* bar) {
#pragma unroll
          for (int c = 0; c < G::VCH; ++c)
            tma_load_4d(smem + G::OFF_V + s * G::VBYTES + c * 16384, &tmV, bar, c * 128 / G::ES, g, w.k_row + j * kTile, 0);
        };
        if constexpr (!G::SPLIT) {
          for (int j = 0; j < w.n_kv; ++j) {
            const int x = jt + j, s = x % NS;
            if (!mbar_wait(bar_vfree + s, ((x / NS) & 1) ^ 1, lim, abort_flag)) { ok = false; break; }
            mbar_arrive_expect_tx(bar_kfull + s, G::KBYTES + G::VBYTES);
            x_last = x;
            load_k(j, s);
            load_v(j, s, bar_kfull + s);
          }
        } else {
          // K runs ahead of V inside the unit; each ring refills as its stages free
          int jk = 0, jv = 0;
          uint64_t t0 = 0;
          uint32_t idle = 0;
          while (jv < w.n_kv) {
            bool progressed = false;
            if (jk < w.n_kv) {
              const int x = jt + jk, s = x % NS;
              if (mbar_test_wait(smem_u32(bar_kfree + s), ((x / NS) & 1) ^ 1)) {
                mbar_arrive_expect_tx(bar_kfull + s, G::KBYTES);
                xk_last = x;
                load_k(jk, s);
                ++jk;
                progressed = true;
              }
            }
            if (jv < jk) {
              const int x = jt + jv, s = x % NS;
              if (mbar_test_wait(smem_u32(bar_vfree + s), ((x / NS) & 1) ^ 1)) {
                mbar_arrive_expect_tx(bar_vfull + s, G::VBYTES);
                xv_last = x;
                load_v(jv, s, bar_vfull + s);
                ++jv;
                progressed = true;
              }
            }
            if (progressed) {
              idle = 0;
            } else {
              if (idle == 0) t0 = globaltimer_ns();
              ++idle;
              __nanosleep(32);
              if ((idle & 63u) == 0 && (*abort_flag || globaltimer_ns() - t0 > lim)) {
                ok = false;
                break;
              }
            }
          }
        }
        if (!ok) break;
        mbar_arrive(bar_want);
        jt += w.n_kv;
        ++nq;
      }
      if (!ok) fail();
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, one elected lane issues (see attn_fwd.cu).
    const uint32_t sbase = smem_u32(smem);
    constexpr uint32_t idesc_qk = idesc_dense(DT == 0 ? 1u : 0u, 0u, 128, 128);
    constexpr uint32_t idesc_pv_bf16 = idesc_dense(1u, 1u, 128, DV);
    uint64_t dq[G::QK_STEPS], dk[G::QK_STEPS], dvv[G::PV_STEPS];
#pragma unroll
    for (int kk = 0; kk < G::QK_STEPS; ++kk) {
      const int pos = kk * 32, c = pos / 128;
      const bool narrow = c == G::NCH - 1 && G::NARROW;
      const uint32_t off = c * 16384 + (pos % 128);
      dq[kk] = smem_desc(sbase + off, 16, narrow ? 512 : 1024, narrow ? SW_64B : SW_128B);
      dk[kk] = smem_desc(sbase + G::OFF_K + off, 16, narrow ? 512 : 1024, narrow ? SW_64B : SW_128B);
    }
#pragma unroll
    for (int kk = 0; kk < G::PV_STEPS; ++kk)
      dvv[kk] = smem_desc(sbase + G::OFF_V + kk * (DT == 0 ? 16 : 32) * 128, 16384, 1024, SW_128B);
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(kFull, mbar_wait(bar, parity, lim, abort_flag));
    };
    auto issue_qk = [&](int x) -> bool {
      const int s = x % NS;
      if (!wait_all(bar_kfull + s, (x / NS) & 1)) return false;
      tc_fence_after();
      const uint32_t dS = tbase + kS0 + (x & 1) * 128;
      const uint64_t koff = (uint64_t)((s * G::KBYTES) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < G::QK_STEPS; ++kk) {
          if (DT == 0)
            mma_f16_ss(dS, dq[kk], dk[kk] + koff, idesc_qk, kk > 0);
          else
            mma_f8_ss(dS, dq[kk], dk[kk] + koff, idesc_qk, kk > 0);
        }
        if (G::SPLIT) tc_commit(bar_kfree + s);
        tc_commit(bar_sfull + (x & 1));
      }
      __syncwarp();
      return true;
    };
    // rows [from, 128) of V_x become 0: they are no keys of this sequence.
    // A row is 128 bytes at 128 * row of each chunk, whatever the swizzle.
    auto clear_tail = [&](int x, int from) -> bool {
      const int s = x % NS;
      if (G::SPLIT && !wait_all(bar_vfull + s, (x / NS) & 1)) return false;  // (else K_x's wait covered V_x)
#pragma unroll 1
      for (int c = 0; c < G::VCH; ++c) {
        uint4* dst = reinterpret_cast<uint4*>(smem + G::OFF_V + s * G::VBYTES + c * 16384);
        for (int i = from * 8 + lane; i < kTile * 8; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      return true;
    };
    auto issue_pv = [&](int x, int j) -> bool {
      const int s = x % NS;
      if (!wait_all(bar_pfull + (x & 1), (x >> 1) & 1)) return false;
      if (G::SPLIT && !wait_all(bar_vfull + s, (x / NS) & 1)) return false;
      tc_fence_after();
      uint64_t voff = (uint64_t)((s * G::VBYTES) >> 4);
      if (DT == 1) {  // leading offset: from V_s to the ones block
        const uint32_t lbo = (uint32_t)(G::OFF_ONES - (G::OFF_V + s * G::VBYTES));
        voff += ((uint64_t)(lbo >> 4) << 16) - ((uint64_t)(16384u >> 4) << 16);
      }
      const uint32_t aP = tbase + kS0 + (x & 1) * 128;
      if (elect_one()) {
        if (DT == 1 && BS)
          tmem_cp_32x128b_x4(tbase + kSFA + (x & 1) * 4, smem_desc(sbase + G::OFF_SF + (x & 1) * 512, 16, 128, SW_NONE));
#pragma unroll
        for (int kk = 0; kk < G::PV_STEPS; ++kk) {
          const uint32_t acc = (j > 0 || kk > 0) ? 1u : 0u;
          if (DT == 0) {
            mma_f16_ts(tbase + kO, aP + (kk >> 2) * 64 + (kk & 3) * 8, dvv[kk] + voff, idesc_pv_bf16, acc);
          } else {
            const uint32_t sfa = (tbase + kSFA + (x & 1) * 4) | ((uint32_t)kk << 30);
            const uint32_t sfb = (tbase + kSFB) | ((uint32_t)kk << 30);
            mma_mxf8_ts(tbase + kO, aP + (kk >> 1) * 64 + (kk & 1) * 8, dvv[kk] + voff, idesc_mx(1u, 128, DV + 16, kk, kk), sfa,
                        sfb, acc);
          }
        }
        tc_commit(bar_vfree + s);
      }
      __syncwarp();
      return true;
    };
    int jt = 0, nq = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!__all_sync(kFull, unit_wait(k))) { ok = false; break; }
      const int n_kv = units[k & 1].n_kv, len_k = units[k & 1].len_k;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ufree + (k & 1));
      if (n_kv < 0) break;
      if (n_kv == 0) continue;
      if (!wait_all(bar_q, nq & 1)) { ok = false; break; }
      const int end = len_k - (n_kv - 1) * kTile;  // rows of the last visited tile that are keys, if below 128
      if (!issue_qk(jt)) { ok = false; break; }
      for (int j = 1; j < n_kv; ++j) {
        if (!issue_qk(jt + j)) { ok = false; break; }
        // PV_0 overwrites O: the softmax must have read the last unit's
        if (j == 1 && nq > 0 && !wait_all(bar_ofree, (nq - 1) & 1)) { ok = false; break; }
        if (!issue_pv(jt + j - 1, j - 1)) { ok = false; break; }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(bar_qfree);  // (the last QK is done when this is)
      __syncwarp();
      if (n_kv == 1 && nq > 0 && !wait_all(bar_ofree, (nq - 1) & 1)) { ok = false; break; }
      if (end < kTile && !clear_tail(jt + n_kv - 1, end)) { ok = false; break; }
      if (!issue_pv(jt + n_kv - 1, n_kv - 1)) { ok = false; break; }
      if (elect_one()) tc_commit(bar_ofinal);
      __syncwarp();
      jt += n_kv;
      ++nq;
    }
    if (!ok && lane == 0) fail();
  } else {
    // ------------------------------------------------------ softmax (rows)
    const int qd = warp & 3, sub = warp >> 2, half = lane >> 4;
    const int row = qd * 32 + sub * 16 + (lane & 15);  // row of the tile == TMEM lane
    const uint32_t col_h = (uint32_t)half * 64;
    const uint32_t lane_off = (uint32_t)(qd * 32 + sub * 16) << 16;
    if (DT == 1 && sub == 0) {
      // scales of V and of the ones block: all 2^0; running mode: P's too
      const uint32_t q_off = (uint32_t)(qd * 32) << 16;
      tmem_st4(tbase + q_off + kSFB, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
      tmem_st4(tbase + q_off + kSFB + 4, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
      if (!BS) {
        tmem_st4(tbase + q_off + kSFA, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        tmem_st4(tbase + q_off + kSFA + 4, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
      }
      tmem_st_wait();
    }
    const int T = p.headroom_T;
    bool ok = true;
    int jt = 0, nq = 0;

    // O holds tiles < j at the old reference: rescale this thread's 64 columns
    // (and FP8's row sum) by f once PV_{j-1} has landed (rare)
    auto rescale_o = [&](int x, float f) -> bool {
      if (!__all_sync(kFull, mbar_wait(bar_vfree + (x - 1) % NS, ((x - 1) / NS) & 1, lim, abort_flag))) return false;
      tc_fence_after();
#pragma unroll 1
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t o[32];
        const uint32_t to = tbase + lane_off + kO + ch * 32;
        tmem_ld16x2_32<64>(to, o);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
        tmem_st16x2_32<64>(to, o);
      }
      if (DT == 1) {
        uint32_t rs;
        tmem_ld16x2_1<1>(tbase + lane_off + kRS, rs);
        tmem_ld_wait();
        tmem_st16x2_1<1>(tbase + lane_off + kRS, __float_as_uint(__uint_as_float(rs) * f));
      }
      return true;
    };

    for (int k = 0; ok; ++k) {
      if (!__all_sync(kFull, unit_wait(k))) { ok = false; break; }
      const VUnit w = units[k & 1];
      if (w.n_kv < 0) break;
      const int n_kv = w.n_kv;
      const int row_lim = p.causal ? min(w.lim0 + row, w.len_k - 1) : w.len_k - 1;
      const int min_lim = min(w.lim0, w.len_k - 1);  // keys up to here: seen by every row
      float yref = -INFINITY;  // BF16 / running mode: log2-domain reference
      int eref = kInvalidExp;  // FP8: reference exponent
      float l = 0.0f;          // BF16: this thread's half of the row sum
      float c = p.scale_log2, vscale = 1.0f;
      if (DT == 1) {
        const int di = p.descale_per_kv ? w.b * p.Hkv + w.h / p.group : 0;
        const float qds = p.q_descale ? p.q_descale[di] : 1.0f;
        const float kds = p.k_descale ? p.k_descale[di] : 1.0f;
        vscale = p.v_descale ? p.v_descale[di] : 1.0f;
        c = (p.scale_log2 * qds) * kds;
        // A scale of 0 (a head of zeros), or a product that vanishes: all scores
        // are 0.  A factor that leaves them 0, and not 0 itself, which would
        // turn the masked keys' -inf into NaN.
        if (c == 0.0f) c = kTiniest;
      }
      for (int j = 0; ok && j < n_kv; ++j) {
        const int x = jt + j, buf = x & 1;
        if (!__all_sync(kFull, mbar_wait(bar_sfull + buf, (x >> 1) & 1, lim, abort_flag))) { ok = false; break; }
        tc_fence_after();
        float s[64];
        {
          uint32_t a0[32], a1[32];
          const uint32_t ts = tbase + lane_off + kS0 + buf * 128;
          tmem_ld16x2_32<64>(ts, a0);
          tmem_ld16x2_32<64>(ts + 32, a1);
          tmem_ld_wait_regs(a0, a1);
#pragma unroll
          for (int cc = 0; cc < 32; ++cc) {
            s[cc] = __uint_as_float(a0[cc]);
            s[32 + cc] = __uint_as_float(a1[cc]);
          }
        }
        const int kbase = j * kTile + (int)col_h;
        const bool masked = j * kTile + kTile - 1 > min_lim;  // the same for all threads
        if (masked) {
#pragma unroll
          for (int cc = 0; cc < 64; ++cc)
            if (kbase + cc > row_lim) s[cc] = -INFINITY;
        }
        const float m = max64(s);
        const uint32_t tP = tbase + lane_off + kS0 + buf * 128;
        if constexpr (DT == 0) {
          const float ym = m * c;
          const float ymax = fmaxf(ym, __shfl_xor_sync(kFull, ym, 16));
          if (__builtin_expect(__any_sync(kFull, ymax > yref + 8.0f), 0)) {
            const float nref = fmaxf(yref, ymax);
            const float f = (nref == -INFINITY || yref == nref) ? 1.0f : ex2_approx(yref - nref);
            yref = nref;
            l *= f;
            if (j > 0 && !rescale_o(x, f)) { ok = false; break; }
          }
          const float nb = yref == -INFINITY ? 0.0f : -yref;
          uint32_t pk[32];
          float lp0 = 0.0f, lp1 = 0.0f;
          // A quarter (d_qk = 192: an eighth) of the pairs runs on the FMA pipe,
          // but not where keys are masked: the polynomial does not give 0 for
          // them.  (us, 1/4 / 1/8: 4096 rows, 32/8 heads 132 / 134; 192/128 339 / 330)
          auto weights = [&](auto poly) {
#pragma unroll
            for (int cc = 0; cc < 64; cc += 2) {
              float z0, z1, p0, p1;
              ffma2(z0, z1, s[cc], s[cc + 1], c, nb);
              if (poly.value && (cc & (DQK == 128 ? 6 : 14)) == 0) {
                exp2_poly_x2<kPolyDegree>(p0, p1, z0, z1);
              } else {
                p0 = ex2_approx(z0);
                p1 = ex2_approx(z1);
              }
              lp0 += p0;
              lp1 += p1;
              pk[cc / 2] = pack_bf16x2(p0, p1);
            }
          };
          if (masked)
            weights(std::false_type{});
          else
            weights(std::true_type{});
          l += lp0 + lp1;
          tmem_st16x2_32<64>(tP, pk);
        } else {
          int e, nref;
          if (BS) {
            e = m != -INFINITY ? (int)ceilf(m * c) - T : kInvalidExp;
            nref = next_ref(eref, max(e, __shfl_xor_sync(kFull, e, 16)), 32);
          } else {
            const float ym = m * c;
            yref = fmaxf(yref, fmaxf(ym, __shfl_xor_sync(kFull, ym, 16)));
            nref = yref != -INFINITY ? (int)ceilf(yref) - T : kInvalidExp;
            e = nref;
          }
          const bool grow = eref > kInvalidExp && nref != eref;
          if (__builtin_expect(j > 0 && __any_sync(kFull, grow), 0)) {
            if (!rescale_o(x, grow ? pow2i(max(eref - nref, -126)) : 1.0f)) { ok = false; break; }
          }
          eref = nref;
          const bool v = e > kInvalidExp;
          uint32_t pk[16];
          if (MODE == 0) {
            const float ne = v ? -(float)e : 0.0f;
#pragma unroll
            for (int cc = 0; cc < 64; cc += 4) {
              float z0, z1, z2, z3, p0, p1;
              ffma2(z0, z1, s[cc], s[cc + 1], c, ne);
              ffma2(z2, z3, s[cc + 2], s[cc + 3], c, ne);
              if ((cc & 4) == 0) {
                exp2_poly_x2<5>(p0, p1, z0, z1);  // (an error near fp32's moves fewest values across a rounding border)
              } else {
                p0 = ex2_approx(z0);
                p1 = ex2_approx(z1);
              }
              pk[cc / 4] = pack_e4m3x4(p0, p1, ex2_approx(z2), ex2_approx(z3));
            }
          } else {
            const float a = c * 0.0625f;  // 8c / 128
            const float magic = 12582912.0f;
            const float k0 = v ? (float)(56 - 8 * e) * 0.0078125f : 0.0f;
#pragma unroll
            for (int cc = 0; cc < 64; cc += 4) {
              const float u0 = fma_sat(s[cc], a, k0);
              const float u1 = fma_sat(s[cc + 1], a, k0);
              const float u2 = fma_sat(s[cc + 2], a, k0);
              const float u3 = fma_sat(s[cc + 3], a, k0);
              float x0, x1, x2, x3;
              ffma2(x0, x1, u0, u1, 128.0f, magic);
              ffma2(x2, x3, u2, u3, 128.0f, magic);
              pk[cc / 4] = prmt(prmt(__float_as_uint(x0), __float_as_uint(x1), 0x0040u),
                                prmt(__float_as_uint(x2), __float_as_uint(x3), 0x0040u), 0x5410u);
            }
          }
          tmem_st16x2_16<64>(tP, pk);
          if (BS) {
            const int sf = v ? min(max(e - eref + 127, 0), 254) : 0;
            reinterpret_cast<uint16_t*>(sf_smem + buf * 128 + (row & 31) * 4 + (row >> 5))[half] = (uint16_t)(sf * 0x0101u);
            fence_proxy_async_smem();
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_pfull + buf);
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if (n_kv > 0 && !__all_sync(kFull, mbar_wait(bar_ofinal, nq & 1, lim, abort_flag))) { ok = false; break; }
      tc_fence_after();
      uint32_t o[64];
      float L = 0.0f, lse_v = -INFINITY;
      if (n_kv > 0) {
        tmem_ld16x2_32<64>(tbase + lane_off + kO, *reinterpret_cast<uint32_t(*)[32]>(o));
        tmem_ld16x2_32<64>(tbase + lane_off + kO + 32, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
        uint32_t rs = 0u;
        if (DT == 1) tmem_ld16x2_1<1>(tbase + lane_off + kRS, rs);
        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(o), *reinterpret_cast<uint32_t(*)[32]>(o + 32));
        asm volatile("" : "+r"(rs)::"memory");
        if (DT == 1) L = __uint_as_float(rs);
        tc_fence_before();
        mbar_arrive(bar_ofree);
      } else {
#pragma unroll
        for (int q = 0; q < 64; ++q) o[q] = 0u;
      }
      if (DT == 0) L = l + __shfl_xor_sync(kFull, l, 16);
      // no visible key, or none above -inf (NaN stays NaN)
      const bool empty = L == 0.0f || (DT == 0 && yref == -INFINITY && L == L);
      const float inv = empty ? 0.0f : vscale / L;
      if (!empty) lse_v = ((DT == 0 ? yref : (float)eref) + __log2f(L)) * 0.6931471805599453f;
      const int row4 = row & ~3;
      const int64_t stride = (int64_t)p.Hq * DV;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)w.q_row + row4) * stride + w.h * DV + col_h;
      store_channels<0>(dst, stride, w.rows - row4, o, inv, empty, lane);
      store_channels<32>(dst + 32, stride, w.rows - row4, o, inv, empty, lane);
      if (row < w.rows && half == 0 && p.lse) p.lse[(int64_t)w.h * p.Tq + w.q_row + row] = lse_v;
      // the unit is done: its slot may name the unit after next
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ufree + (k & 1));
      jt += n_kv;
      if (n_kv > 0) ++nq;
    }
    if (!ok && lane == 0) fail();
    tmem_ld_wait();
    tmem_st_wait();
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // asynchronous work already issued lands before the CTA frees its tensor
    // memory and exits; each wait is bounded again (see attn_fwd.cu)
    if (warp == kProducer && lane == 0) {
      if (q_loads > 0) mbar_wait_bounded(bar_q, (q_loads - 1) & 1, lim);
      for (int x = max(x_last - NS + 1, 0); x <= x_last; ++x) mbar_wait_bounded(bar_kfull + x % NS, (x / NS) & 1, lim);
      for (int x = max(xk_last - NS + 1, 0); x <= xk_last; ++x) mbar_wait_bounded(bar_kfull + x % NS, (x / NS) & 1, lim);
      for (int x = max(xv_last - NS + 1, 0); x <= xv_last; ++x) mbar_wait_bounded(bar_vfull + x % NS, (x / NS) & 1, lim);
    }
    if (warp == kScheduler && asked) mbar_wait_bounded(bar_clc, clc_n & 1, lim);
    if (warp == kIssuer) {
      if (elect_one()) tc_commit(bar_drain);
      __syncwarp();
      mbar_wait_bounded(bar_drain, 0, lim);
    }
    __syncthreads();
  }
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tbase, kCols);
  }
}

template <int DT, int DQK, int MODE, int BS>
cudaError_t launch_variant(const VarlenLaunch& a, cudaStream_t st) {
  using G = VGeo<DT, DQK>;
  const VarlenParams& p = a.p;
  CUtensorMap mQ, mQ2, mK, mK2, mV;
  if (!make_map(&mQ, a.q, G::ES, 1, p.Tq, p.Hq, DQK, 128 / G::ES, CU_TENSOR_MAP_SWIZZLE_128B, kTile) ||
      !make_map(&mK, a.k, G::ES, 1, p.Tk > 0 ? p.Tk : 1, p.Hkv, DQK, 128 / G::ES, CU_TENSOR_MAP_SWIZZLE_128B, kTile) ||
      !make_map(&mV, a.v, G::ES, 1, p.Tk > 0 ? p.Tk : 1, p.Hkv, G::DV, 128 / G::ES, CU_TENSOR_MAP_SWIZZLE_128B, kTile))
    return cudaErrorInvalidValue;
  mQ2 = mQ;
  mK2 = mK;
  if (G::NARROW && (!make_map(&mQ2, a.q, G::ES, 1, p.Tq, p.Hq, DQK, 64 / G::ES, CU_TENSOR_MAP_SWIZZLE_64B, kTile) ||
                    !make_map(&mK2, a.k, G::ES, 1, p.Tk > 0 ? p.Tk : 1, p.Hkv, DQK, 64 / G::ES, CU_TENSOR_MAP_SWIZZLE_64B, kTile)))
    return cudaErrorInvalidValue;
  auto kern = attn_varlen_kernel<DT, DQK, MODE, BS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, dim3((unsigned)p.max_tiles * (unsigned)p.Hq), dim3(kVarThreads), G::SMEM, st, mQ, mQ2, mK, mK2, mV, p);
}

}  // namespace

cudaError_t launch_attention_varlen(const VarlenLaunch& a, cudaStream_t st) {
  if (a.p.max_tiles <= 0) return cudaSuccess;
  if (a.pairs) return launch_attention_varlen_pp(a, st);
  if (a.dtype == 0) return a.dqk == 128 ? launch_variant<0, 128, 0, 0>(a, st) : launch_variant<0, 192, 0, 0>(a, st);
  const bool bs = a.block_scale != 0;
  if (a.dqk == 128) {
    if (a.mode == 1) return bs ? launch_variant<1, 128, 1, 1>(a, st) : launch_variant<1, 128, 1, 0>(a, st);
    return bs ? launch_variant<1, 128, 0, 1>(a, st) : launch_variant<1, 128, 0, 0>(a, st);
  }
  if (a.mode == 1) return bs ? launch_variant<1, 192, 1, 1>(a, st) : launch_variant<1, 192, 1, 0>(a, st);
  return bs ? launch_variant<1, 192, 0, 1>(a, st) : launch_variant<1, 192, 0, 0>(a, st);
}

}  // namespace zq
