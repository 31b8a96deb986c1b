// attn_varlen_pp.cu -- BF16 attention over packed prompts, head dims (128,
// 128), with two 128-row query tiles per CTA that share their keys.
//
// The mathematics of attn_varlen.cu and the schedule on the SM of attn_pp.cu:
// each of the two tiles has its own softmax team of four warps (a thread per
// query row) and its own MMA issuer, keys come in tiles of 64 that both teams
// read from the same stage, and P has tensor-memory buffers of its own, so one
// team's softmax runs while the tensor core works for the other.
//
// The tiles are two consecutive ones of one head; the earlier stops at its own
// diagonal.  Which calls come here: use_varlen_pairs (serving.h).
//
// Bound by the softmax chain and, in longer runs, by the board's power: 32/8
// heads after a pause, 16384 rows 1679 us (1310 TFLOP/s), 12 prompts of 13.6K
// rows in all 281 us (995).
//
// Units come from varlen_sched.cuh.  The last key tile of a sequence: scores
// past the end are masked (weights exactly 0), and V's rows past it are set to
// 0 by both issuers, each before its own product (zeros over zeros for the
// second).
//
// Warps: 0-3 team 0, 4-7 team 1, 8 TMA producer, 9 and 10 issuers of teams 0
// and 1 (9 owns the tensor memory), 11 scheduler.  Tensor memory per team t:
// S_t [64t, +64), O_t [128 + 128t, +128), P_t,b [384 + 32 (2t + b), +32).
#include <type_traits>

#include "attn_math.cuh"
#include "serving.h"
#include "sm100_ptx.cuh"
#include "varlen_sched.cuh"

namespace zq {

namespace {

constexpr int kTeam = 128;
constexpr int kVppThreads = 2 * kTeam + 128;
constexpr int kProducer = 8, kIssuer0 = 9, kScheduler = 11;
constexpr uint32_t kCols = 512;
constexpr int kPolyDegree = 4;  // as attn_varlen.cu

struct VGeoPP {
  static constexpr int D = 128;
  static constexpr int KT = kPairKeyTile;
  static constexpr int ROW = D * 2;
  static constexpr int QBYTES = kTile * ROW;  // chunk c (64 channels) at c * 16 KB
  static constexpr int KBYTES = KT * ROW;     // chunk c at c * 8 KB
  static constexpr int STAGE = 2 * KBYTES;    // K_j then V_j
  static constexpr int QK_STEPS = ROW / 32;
  static constexpr int PV_STEPS = KT / 16;
  static constexpr int NS = 5;
  static constexpr int OFF_KV = 2 * QBYTES;
  static constexpr int OFF_PREFIX = OFF_KV + NS * STAGE;
  static constexpr int OFF_UNIT = OFF_PREFIX + kSchedChunks * 4;
  static constexpr int OFF_CLC = OFF_UNIT + 2 * 64;
  static constexpr int OFF_BAR = OFF_CLC + 16;
  static constexpr int NBAR = 2 * NS + 25;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;  // + alignment slack
  static_assert(SMEM <= 232448, "227 KB of shared memory per CTA");
  __device__ static constexpr uint32_t col_s(int t) { return 64u * t; }
  __device__ static constexpr uint32_t col_o(int t) { return 128u + 128u * t; }
  __device__ static constexpr uint32_t col_p(int t, int b) { return 384u + 32u * (2 * t + b); }
};

// A unit as the scheduler hands it out (64 bytes of shared memory).
struct PUnit {
  int h, k_row, len_k;    // query head, the sequence's first key row and its keys
  int n_max;              // key tiles to load; -1: no more units
  int q_row[2], rows[2];  // first packed query row, rows of the tile that are the sequence's
  int lim0[2];            // last key the first row may see (before the clamp)
  int n[2];               // key tiles each team visits
};
static_assert(sizeof(PUnit) <= 64, "a ring slot");

__global__ void __launch_bounds__(kVppThreads, 1)
    attn_varlen_pp_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const VarlenParams p) {
  using G = VGeoPP;
  constexpr int NS = G::NS;
  constexpr unsigned kFull = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::OFF_BAR);
  uint64_t* bar_kvfull = bars;             // [NS] K_j and V_j landed
  uint64_t* bar_kvfree = bar_kvfull + NS;  // [NS] both teams done with the stage (2 arrivals)
  uint64_t* bar_q = bar_kvfree + NS;       // [2] Q_t landed
  uint64_t* bar_qfree = bar_q + 2;         // [2] the unit's last QK_t done
  uint64_t* bar_sfull = bar_qfree + 2;     // [2] QK_t(j) done
  uint64_t* bar_sfree = bar_sfull + 2;     // [2] team t loaded S_t(j)
  uint64_t* bar_pfull = bar_sfree + 2;     // [2][2] team t wrote P_t(j) into buffer j & 1
  uint64_t* bar_pvdone = bar_pfull + 4;    // [2] PV_t(j) done
  uint64_t* bar_ofinal = bar_pvdone + 2;   // [2] the unit's last PV_t done
  uint64_t* bar_ofree = bar_ofinal + 2;    // [2] team t read O_t
  uint64_t* bar_ufull = bar_ofree + 2;     // [2] unit slot filled
  uint64_t* bar_ufree = bar_ufull + 2;     // [2] unit slot read by all roles
  uint64_t* bar_clc = bar_ufree + 2;       // the answer to a request for a block
  uint64_t* bar_want = bar_clc + 1;        // the producer issued a unit's last load
  uint64_t* bar_drain = bar_want + 1;      // after an abort: both issuers' work landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_drain + 1);  // (bars + NBAR)
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto unit = [&](int k) -> PUnit& { return *reinterpret_cast<PUnit*>(smem + G::OFF_UNIT + (k & 1) * 64); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_kvfull + s, 1);
      mbar_init(bar_kvfree + s, 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_q + t, 1);
      mbar_init(bar_qfree + t, 1);
      mbar_init(bar_sfull + t, 1);
      mbar_init(bar_sfree + t, kTeam);
      mbar_init(bar_pfull + 2 * t, kTeam + p.withhold);
      mbar_init(bar_pfull + 2 * t + 1, kTeam + p.withhold);
      mbar_init(bar_pvdone + t, 1);
      mbar_init(bar_ofinal + t, 1);
      mbar_init(bar_ofree + t, kTeam);
      mbar_init(bar_ufull + t, 1);
      mbar_init(bar_ufree + t, 3 + 2 * kTeam / 32);  // producer, issuers, softmax warps
    }
    mbar_init(bar_clc, 1);
    mbar_init(bar_want, 1);
    mbar_init(bar_drain, 2);
    *abort_flag = 0;
    fence_barrier_init();
  }
  launch_dependents();
  wait_previous_kernel();
  UnitCount count;  // (the scheduler's; beside the set-up of the others)
  if (warp == kScheduler) count = count_tiles<2 * kTile>(p, reinterpret_cast<int*>(smem + G::OFF_PREFIX), lane);
  if (warp == kIssuer0) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  if (warp == kProducer && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint64_t lim = p.timeout_ns;
  int q_loads0 = 0, q_loads1 = 0, x_last = -1;  // last loads armed (drain)
  bool asked = false;
  int clc_n = 0;

  auto fail = [&]() {
    *abort_flag = 1;
    if (p.status) atomicExch(p.status, -7 /* ZQ_ERR_TIMEOUT */);
  };
  auto unit_wait = [&](int k) -> bool { return mbar_wait(bar_ufull + (k & 1), (k >> 1) & 1, lim, abort_flag); };

  if (warp == kScheduler) {
    // ----------------------------------------------------------- scheduler
    const bool ok = schedule_units<2 * kTile>(
        p, p.Hq, count, reinterpret_cast<int*>(smem + G::OFF_PREFIX), smem + G::OFF_CLC, bar_clc, bar_want, bar_ufull, bar_ufree,
        abort_flag, lane, asked, clc_n, [&](int slot, const SeqTile* s) {
          PUnit w = {};
          w.n_max = -1;
          if (s) {
            w.n_max = 0;
            w.k_row = s->k0;
            w.len_k = s->k1 - s->k0;
            w.h = s->h;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int i0 = (2 * s->t + t) * kTile;  // first row in the sequence
              w.q_row[t] = s->q0 + i0;
              w.rows[t] = min(s->q1 - w.q_row[t], kTile);  // (0 or less: a tile past the sequence)
              w.lim0[t] = p.causal ? i0 + w.len_k - (s->q1 - s->q0) : w.len_k - 1;
              const int max_key = p.causal ? min(w.lim0[t] + w.rows[t] - 1, w.len_k - 1) : w.len_k - 1;
              w.n[t] = max_key < 0 || w.rows[t] <= 0 ? 0 : max_key / G::KT + 1;
              w.n_max = max(w.n_max, w.n[t]);
            }
          }
          unit(slot) = w;
        });
    if (!ok && lane == 0) fail();
  } else if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int jkv = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!unit_wait(k)) { ok = false; break; }
        const PUnit w = unit(k);
        mbar_arrive(bar_ufree + (k & 1));
        if (w.n_max < 0) break;
        if (w.n_max == 0) {
          mbar_arrive(bar_want);
          continue;
        }
        const int g = w.h / p.group;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          int& nq = t ? q_loads1 : q_loads0;
          if (!ok || w.n[t] == 0) continue;
          // Q_t of the previous unit is read until its last QK_t completes
          if (nq > 0 && !mbar_wait(bar_qfree + t, (nq - 1) & 1, lim, abort_flag)) { ok = false; break; }
          mbar_arrive_expect_tx(bar_q + t, G::QBYTES);
          ++nq;
#pragma unroll
          for (int c = 0; c < 2; ++c) tma_load_4d(smem + t * G::QBYTES + c * 16384, &tmQ, bar_q + t, c * 64, w.h, w.q_row[t], 0);
        }
        if (!ok) break;
        for (int j = 0; j < w.n_max; ++j) {
          const int x = jkv + j, s = x % NS;
          if (!mbar_wait(bar_kvfree + s, ((x / NS) & 1) ^ 1, lim, abort_flag)) { ok = false; break; }
          uint8_t* sk = smem + G::OFF_KV + s * G::STAGE;
          mbar_arrive_expect_tx(bar_kvfull + s, G::STAGE);
          x_last = x;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tma_load_4d(sk + c * 8192, &tmK, bar_kvfull + s, c * 64, g, w.k_row + j * G::KT, 0);
            tma_load_4d(sk + G::KBYTES + c * 8192, &tmV, bar_kvfull + s, c * 64, g, w.k_row + j * G::KT, 0);
          }
        }
        if (!ok) break;
        mbar_arrive(bar_want);
        jkv += w.n_max;
      }
      if (!ok) fail();
    }
  } else if (warp > kProducer) {
    // ------------------------------------------------------------ issuers
    // The whole warp runs the loop, one elected lane issues.
    const int t = warp - kIssuer0;
    const uint32_t sbase = smem_u32(smem);
    constexpr uint32_t idesc_qk = idesc_dense(1u, 0u, 128, G::KT);
    constexpr uint32_t idesc_pv = idesc_dense(1u, 1u, 128, G::D);
    uint64_t dq[G::QK_STEPS], dk[G::QK_STEPS], dvv[G::PV_STEPS];
#pragma unroll
    for (int kk = 0; kk < G::QK_STEPS; ++kk) {
      const int pos = kk * 32, c = pos / 128;
      dq[kk] = smem_desc(sbase + t * G::QBYTES + c * 16384 + pos % 128, 16, 1024, SW_128B);
      dk[kk] = smem_desc(sbase + G::OFF_KV + c * 8192 + pos % 128, 16, 1024, SW_128B);
    }
#pragma unroll
    for (int kk = 0; kk < G::PV_STEPS; ++kk)
      dvv[kk] = smem_desc(sbase + G::OFF_KV + G::KBYTES + kk * 16 * 128, 8192, 1024, SW_128B);
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(kFull, mbar_wait(bar, parity, lim, abort_flag));
    };
    const uint32_t dS = tbase + G::col_s(t), dO = tbase + G::col_o(t);
    // g: the team's tile count in this CTA; x: the CTA's K/V tile count; j: index in the unit
    auto issue_qk = [&](int g, int x) -> bool {
      const int s = x % NS;
      if (!wait_all(bar_kvfull + s, (x / NS) & 1)) return false;
      if (g > 0 && !wait_all(bar_sfree + t, (g - 1) & 1)) return false;
      tc_fence_after();
      const uint64_t koff = (uint64_t)((s * G::STAGE) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < G::QK_STEPS; ++kk) mma_f16_ss(dS, dq[kk], dk[kk] + koff, idesc_qk, kk > 0);
        tc_commit(bar_sfull + t);
      }
      __syncwarp();
      return true;
    };
    // rows [from, 64) of V_x become 0 (a row is 128 bytes at 128 * row of each chunk)
    auto clear_tail = [&](int x, int from) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint4* dst = reinterpret_cast<uint4*>(smem + G::OFF_KV + (x % NS) * G::STAGE + G::KBYTES + c * 8192);
        for (int i = from * 8 + lane; i < G::KT * 8; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    auto issue_pv = [&](int g, int x, int j) -> bool {
      const int s = x % NS, b = g & 1;
      if (!wait_all(bar_pfull + 2 * t + b, (g >> 1) & 1)) return false;
      tc_fence_after();
      const uint64_t voff = (uint64_t)((s * G::STAGE) >> 4);
      const uint32_t aP = tbase + G::col_p(t, b);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < G::PV_STEPS; ++kk)
          mma_f16_ts(dO, aP + kk * 8, dvv[kk] + voff, idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit(bar_pvdone + t);
        tc_commit(bar_kvfree + s);
      }
      __syncwarp();
      return true;
    };
    int jt = 0, jkv = 0, nq = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!__all_sync(kFull, unit_wait(k))) { ok = false; break; }
      const int n = t ? unit(k).n[1] : unit(k).n[0], n_max = unit(k).n_max, len_k = unit(k).len_k;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ufree + (k & 1));
      if (n_max < 0) break;
      if (n > 0) {
        if (!wait_all(bar_q + t, nq & 1)) { ok = false; break; }
        const int end = len_k - (n - 1) * G::KT;  // rows of the last visited tile that are keys, if below 64
        if (!issue_qk(jt, jkv)) { ok = false; break; }
        for (int j = 1; j < n; ++j) {
          if (!issue_qk(jt + j, jkv + j)) { ok = false; break; }
          // PV_t(0) overwrites O_t: the team must have read the last unit's
          if (j == 1 && nq > 0 && !wait_all(bar_ofree + t, (nq - 1) & 1)) { ok = false; break; }
          if (!issue_pv(jt + j - 1, jkv + j - 1, j - 1)) { ok = false; break; }
        }
        if (!ok) break;
        if (elect_one()) tc_commit(bar_qfree + t);  // (QK_t of the last tile is done when this is)
        __syncwarp();
        if (n == 1 && nq > 0 && !wait_all(bar_ofree + t, (nq - 1) & 1)) { ok = false; break; }
        if (end < G::KT) clear_tail(jkv + n - 1, end);
        if (!issue_pv(jt + n - 1, jkv + n - 1, n - 1)) { ok = false; break; }
        if (elect_one()) tc_commit(bar_ofinal + t);
        __syncwarp();
        jt += n;
        ++nq;
      }
      // key tiles this team skips: release its share of their stages once loaded
      for (int j = n; j < n_max; ++j) {
        const int x = jkv + j;
        if (!wait_all(bar_kvfull + x % NS, (x / NS) & 1)) { ok = false; break; }
        if (lane == 0) mbar_arrive(bar_kvfree + x % NS);
        __syncwarp();
      }
      jkv += n_max;
    }
    if (!ok && lane == 0) fail();
  } else {
    // ------------------------------------------------------ softmax teams
    const int t = warp >> 2, qd = warp & 3;
    const int row = qd * 32 + lane;  // row of the team's tile == TMEM lane
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const uint32_t tS = tbase + lane_off + G::col_s(t), tO = tbase + lane_off + G::col_o(t);
    const float c = p.scale_log2;
    bool ok = true;
    int jt = 0, nq = 0;

    // O_t holds tiles < j at the old reference: rescale this row once
    // PV_t(j - 1) has landed (rare)
    auto rescale_o = [&](int g, float f) -> bool {
      if (!__all_sync(kFull, mbar_wait(bar_pvdone + t, (g - 1) & 1, lim, abort_flag))) return false;
      tc_fence_after();
#pragma unroll 1
      for (int ch = 0; ch < G::D / 32; ++ch) {
        uint32_t o[32];
        tmem_ld32_x32(tO + ch * 32, o);
        tmem_ld_wait_on(o);
#pragma unroll
        for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
        tmem_st32_x32(tO + ch * 32, o);
      }
      return true;
    };

    for (int k = 0; ok; ++k) {
      if (!__all_sync(kFull, unit_wait(k))) { ok = false; break; }
      if (unit(k).n_max < 0) break;
      const PUnit& w = unit(k);
      const int n = t ? w.n[1] : w.n[0], h = w.h, rows = t ? w.rows[1] : w.rows[0];
      const int lim0 = t ? w.lim0[1] : w.lim0[0], q_row = t ? w.q_row[1] : w.q_row[0], len_k = w.len_k;
      const int row_lim = p.causal ? min(lim0 + row, len_k - 1) : len_k - 1;
      const int min_lim = min(lim0, len_k - 1);  // keys up to here: seen by every row
      float yref = -INFINITY, l = 0.0f;
      for (int j = 0; ok && j < n; ++j) {
        const int g = jt + j, buf = g & 1;
        if (!__all_sync(kFull, mbar_wait(bar_sfull + t, g & 1, lim, abort_flag))) { ok = false; break; }
        tc_fence_after();
        float s[64];
        {
          uint32_t a[64];
          tmem_ld32_x64(tS, a);
          tmem_ld_wait_on(a);
#pragma unroll
          for (int cc = 0; cc < 64; ++cc) s[cc] = __uint_as_float(a[cc]);
        }
        tc_fence_before();
        mbar_arrive(bar_sfree + t);  // S_t is free for QK_t(j + 1)
        const int kbase = j * G::KT;
        const bool masked = kbase + G::KT - 1 > min_lim;  // the same for all threads of the team
        if (masked) {
#pragma unroll
          for (int cc = 0; cc < 64; ++cc)
            if (kbase + cc > row_lim) s[cc] = -INFINITY;
        }
        const float ym = max64(s) * c;
        if (__builtin_expect(__any_sync(kFull, ym > yref + 8.0f), 0)) {
          const float nref = fmaxf(yref, ym);
          const float f = (nref == -INFINITY || yref == nref) ? 1.0f : ex2_approx(yref - nref);
          yref = nref;
          l *= f;
          if (j > 0 && !rescale_o(g, f)) { ok = false; break; }
        }
        const float nb = yref == -INFINITY ? 0.0f : -yref;
        uint32_t pk[32];
        float lp0 = 0.0f, lp1 = 0.0f;
        // An eighth of the pairs on the FMA pipe, but not where keys are masked:
        // the polynomial does not give 0 for them.  In halves, so that one
        // half's arguments, the other's exponentials and sums stand beside one
        // another: pair by pair the compiler bunched the exponentials, which
        // queue up (8192 rows 450-480 us by where the polynomial's pairs lie,
        // 449 in halves, 467 all at once).  Share on the FMA pipe, 16384 rows:
        // none 1911, 1/16 1777, 1/8 1754, 3/16 1806, 1/4 1798 us.
        auto weights = [&](auto poly) {
#pragma unroll
          for (int c0 = 0; c0 < 128; c0 += 32) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              if (c0 < 64) ffma2(s[c0 + i], s[c0 + i + 1], s[c0 + i], s[c0 + i + 1], c, nb);
              if (const int e = c0 - 32 + i; e >= 0 && e < 64) {
                if (poly.value && (e & 14) == 0) {
                  exp2_poly_x2<kPolyDegree>(s[e], s[e + 1], s[e], s[e + 1]);
                } else {
                  s[e] = ex2_approx(s[e]);
                  s[e + 1] = ex2_approx(s[e + 1]);
                }
              }
              if (const int f = c0 - 64 + i; f >= 0) {
                fadd2(lp0, lp1, s[f], s[f + 1]);
                pk[f / 2] = pack_bf16x2(s[f], s[f + 1]);
              }
            }
          }
        };
        if (masked)
          weights(std::false_type{});
        else
          weights(std::true_type{});
        l += lp0 + lp1;
        tmem_st32_x32(tbase + lane_off + G::col_p(t, buf), pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_pfull + 2 * t + buf);
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      float inv = 0.0f, lse_v = -INFINITY;
      bool empty = true;  // no visible key, or none above -inf (NaN stays NaN)
      if (n > 0) {
        if (!__all_sync(kFull, mbar_wait(bar_ofinal + t, nq & 1, lim, abort_flag))) { ok = false; break; }
        tc_fence_after();
        empty = l == 0.0f || (yref == -INFINITY && l == l);
        inv = empty ? 0.0f : 1.0f / l;
        if (!empty) lse_v = (yref + __log2f(l)) * 0.6931471805599453f;
      }
      const int row4 = row & ~3;
      const int64_t stride = (int64_t)p.Hq * G::D;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)q_row + row4) * stride + h * G::D;
#pragma unroll 1
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t o[64];
        if (n > 0) {
          tmem_ld32_x64(tO + ch * 64, o);
          tmem_ld_wait_on(o);
        } else {
#pragma unroll
          for (int q = 0; q < 64; ++q) o[q] = 0u;
        }
        if (ch == 1 && n > 0) {
          tc_fence_before();
          mbar_arrive(bar_ofree + t);  // O_t read: the next unit's PV_t(0) may overwrite it
        }
        store_channels<0>(dst + ch * 64, stride, rows - row4, o, inv, empty, lane);
        store_channels<32>(dst + ch * 64 + 32, stride, rows - row4, o, inv, empty, lane);
      }
      if (row < rows && p.lse) p.lse[(int64_t)h * p.Tq + q_row + row] = lse_v;
      // the unit is done: its slot may name the unit after next
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ufree + (k & 1));
      jt += n;
      if (n > 0) ++nq;
    }
    if (!ok && lane == 0) fail();
    tmem_ld_wait();
    tmem_st_wait();
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // asynchronous work already issued lands before the CTA frees its tensor
    // memory and exits; each wait is bounded again
    if (warp == kProducer && lane == 0) {
      if (q_loads0 > 0) mbar_wait_bounded(bar_q, (q_loads0 - 1) & 1, lim);
      if (q_loads1 > 0) mbar_wait_bounded(bar_q + 1, (q_loads1 - 1) & 1, lim);
      for (int x = max(x_last - NS + 1, 0); x <= x_last; ++x) mbar_wait_bounded(bar_kvfull + x % NS, (x / NS) & 1, lim);
    }
    if (warp == kScheduler && asked) mbar_wait_bounded(bar_clc, clc_n & 1, lim);
    if (warp == kIssuer0 || warp == kIssuer0 + 1) {
      if (elect_one()) tc_commit(bar_drain);
      __syncwarp();
      mbar_wait_bounded(bar_drain, 0, lim);
    }
    __syncthreads();
  }
  if (warp == kIssuer0) {
    tc_fence_after();
    tmem_dealloc(tbase, kCols);
  }
}

}  // namespace

cudaError_t launch_attention_varlen_pp(const VarlenLaunch& a, cudaStream_t st) {
  using G = VGeoPP;
  VarlenParams p = a.p;
  p.max_tiles = varlen_tiles(p.Tq, p.B, 2 * kTile);
  const int Tk = p.Tk > 0 ? p.Tk : 1;
  CUtensorMap mQ, mK, mV;
  if (!make_map(&mQ, a.q, 2, 1, p.Tq, p.Hq, G::D, 64, CU_TENSOR_MAP_SWIZZLE_128B, kTile) ||
      !make_map(&mK, a.k, 2, 1, Tk, p.Hkv, G::D, 64, CU_TENSOR_MAP_SWIZZLE_128B, G::KT) ||
      !make_map(&mV, a.v, 2, 1, Tk, p.Hkv, G::D, 64, CU_TENSOR_MAP_SWIZZLE_128B, G::KT))
    return cudaErrorInvalidValue;
  auto kern = attn_varlen_pp_kernel;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, dim3((unsigned)p.max_tiles * (unsigned)p.Hq), dim3(kVppThreads), G::SMEM, st, mQ, mK, mV, p);
}

}  // namespace zq
