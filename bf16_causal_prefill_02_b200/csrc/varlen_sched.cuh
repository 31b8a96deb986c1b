// varlen_sched.cuh -- how the packed-prompt kernels come to their work: query
// tiles of sequences whose offsets only the device knows, dealt to resident
// CTAs by taking over blocks of the grid that have not started.
//
// The grid is a bound on the tiles, (Tq + (ROWS - 1) B) / ROWS, times the
// heads.  A scheduler warp sums the tile counts of the sequences (prefix sums
// over chunks of them, in shared memory), turns block u into (sequence, tile,
// head), hands it to the other roles through a two-slot ring, and asks the
// hardware for the next block (clusterlaunchcontrol.try_cancel) when the
// producer has issued the current unit's last load: late enough that a CTA
// with a long unit does not hold a second one that an idle CTA could run
// (8192 rows, 4 heads: 91 against 125 us when asked a whole unit ahead),
// early enough for the answer to hide behind the stages still to be consumed.
//
// And how they write their output rows (store_channels).
#pragma once
#include <cstdint>

#include "attn_math.cuh"
#include "serving.h"
#include "sm100_ptx.cuh"

namespace zq {

constexpr int kSchedChunks = 256;  // prefix sums, one per chunk of sequences

__device__ __forceinline__ void clc_try_cancel(void* response, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(response)),
               "r"(smem_u32(bar))
               : "memory");
}
// The block index that the request took over, or -1: no block is left.
__device__ __forceinline__ int64_t clc_taken(const void* response) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(response))
      : "memory");
  return ok ? (int64_t)x : -1;
}

// Rows of sequence b: [first, last) of the queries or of the keys.  Offsets
// are clamped to the tensor; a sequence whose offsets descend has no rows.
__device__ __forceinline__ int offset_at(const int32_t* cu, int b, int total) { return min(max(cu[b], 0), total); }
template <int ROWS>
__device__ __forceinline__ int tiles_of(const VarlenParams& p, int b) {
  const int n = offset_at(p.cu_q, b + 1, p.Tq) - offset_at(p.cu_q, b, p.Tq);
  return n > 0 ? (n + ROWS - 1) / ROWS : 0;
}

// A query tile of a sequence, and the flat head (or head pair) of the unit.
struct SeqTile {
  int b, t, h;         // t counts tiles of ROWS rows
  int q0, q1, k0, k1;  // the sequence's query and key rows
};

// Sums the tile counts: prefix[c] holds the tiles of chunks 0 .. c of `per`
// sequences each.  By one warp, before the ring is in use.
struct UnitCount {
  int per, n_chunks, tiles;
};
template <int ROWS>
__device__ __forceinline__ UnitCount count_tiles(const VarlenParams& p, int* prefix, int lane) {
  constexpr unsigned kFull = 0xffffffffu;
  UnitCount u;
  u.per = (p.B + kSchedChunks - 1) / kSchedChunks;
  u.n_chunks = (p.B + u.per - 1) / u.per;
  int64_t total = 0;  // (offsets that are no ascending sequence may add up to anything: cut at the grid's bound)
  for (int c0 = 0; c0 < u.n_chunks; c0 += 32) {
    const int b0 = (c0 + lane) * u.per, b1 = min(b0 + u.per, p.B);
    int64_t n = 0;
    for (int b = b0; b < b1; ++b) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.cu_k + b));  // read once the unit is known
      n += tiles_of<ROWS>(p, b);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kFull, n, o);
      if (lane >= o) n += up;
    }
    if (c0 + lane < u.n_chunks) prefix[c0 + lane] = (int)min(total + n, (int64_t)p.max_tiles);
    total += __shfl_sync(kFull, n, 31);
  }
  __syncwarp();
  u.tiles = (int)min(total, (int64_t)p.max_tiles);
  return u;
}

// The scheduler warp's loop.  `heads` flat heads (p.head_group of them
// interleaved); publish(slot, tile) by lane 0 writes a ring slot,
// publish(slot, nullptr) the end.  bar_free / bar_full: the ring's two slots;
// bar_want: one phase per unit, the producer needs the next; bar_clc,
// response: the requests.  False: a wait ran out; `asked`
// tells whether a request is then still out, `n_asked` how many were answered.
template <int ROWS, class Publish>
__device__ __forceinline__ bool schedule_units(const VarlenParams& p, int heads, const UnitCount& count, int* prefix, void* response,
                                               uint64_t* bar_clc, uint64_t* bar_want, uint64_t* bar_full, uint64_t* bar_free,
                                               volatile int* abort_flag, int lane, bool& asked, int& n_asked, Publish publish) {
  constexpr unsigned kFull = 0xffffffffu;
  const uint64_t lim = p.timeout_ns;
  const int per = count.per, n_chunks = count.n_chunks, tiles = count.tiles;
  const int64_t n_units = (int64_t)tiles * heads;
  const int GH = p.head_group;
  bool last = false;
  int64_t u = blockIdx.x;
  for (int k = 0;; ++k) {
    if (k > 0 && !__all_sync(kFull, mbar_wait(bar_want, (k - 1) & 1, lim, abort_flag))) return false;
    // a block past the last unit is nobody's: ask on until none is left
    while (!last && u >= n_units) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar_clc, 16);
        clc_try_cancel(response, bar_clc);
      }
      asked = true;
      if (!__all_sync(kFull, mbar_wait(bar_clc, n_asked & 1, lim, abort_flag))) return false;
      asked = false;
      ++n_asked;
      u = clc_taken(response);
      fence_proxy_async_smem();
      __syncwarp();
      last = u < 0;
    }
    SeqTile w = {};
    if (!last) {
      const int gi = (int)u / (GH * tiles), gr = (int)u % (GH * tiles);  // (units fit 31 bits)
      const int e = gr / GH;
      w.h = gi * GH + gr % GH;
      // the chunk, then the sequence, that holds tile e
      int ch = 0;
      for (int c0 = 0; c0 < n_chunks; c0 += 32) {
        const unsigned le = __ballot_sync(kFull, c0 + lane < n_chunks && prefix[c0 + lane] <= e);
        ch += __popc(le);
        if (le != kFull) break;
      }
      int r = e - (ch > 0 ? prefix[ch - 1] : 0);  // tile in the chunk
      int nt = 0;
      for (int b0 = ch * per;; b0 += 32) {
        const int b = b0 + lane;
        const int n = b < min((ch + 1) * per, p.B) ? tiles_of<ROWS>(p, b) : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(kFull, sum, o);
          if (lane >= o) sum += up;
        }
        const unsigned le = __ballot_sync(kFull, sum <= r);
        if (le == kFull && b0 + 32 < (ch + 1) * per) {
          r -= __shfl_sync(kFull, sum, 31);
          continue;
        }
        const int at = min(__popc(le), 31);
        nt = __shfl_sync(kFull, n, at);
        r -= __shfl_sync(kFull, sum - n, at);
        w.b = min(b0 + at, p.B - 1);
        break;
      }
      w.t = max(nt - 1 - r, 0);  // longest rows first
      w.q0 = offset_at(p.cu_q, w.b, p.Tq), w.q1 = offset_at(p.cu_q, w.b + 1, p.Tq);
      w.k0 = offset_at(p.cu_k, w.b, p.Tk), w.k1 = max(offset_at(p.cu_k, w.b + 1, p.Tk), w.k0);
      u = n_units;  // ask for the next one
    }
    if (!__all_sync(kFull, mbar_wait(bar_free + (k & 1), ((k >> 1) & 1) ^ 1, lim, abort_flag))) return false;
    if (lane == 0) {
      publish(k & 1, last ? nullptr : &w);
      mbar_arrive(bar_full + (k & 1));
    }
    __syncwarp();
    if (last) return true;
  }
}

// Transposes 4 x 4 pieces of 16 bytes over each four lanes: v[j] of lane i
// becomes v[i] of lane j.
__device__ __forceinline__ void transpose_pieces(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
    const bool hi = lane & b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & b) continue;
      uint4 s = hi ? v[j] : v[j | b];
      s.x = __shfl_xor_sync(0xffffffffu, s.x, b);
      s.y = __shfl_xor_sync(0xffffffffu, s.y, b);
      s.z = __shfl_xor_sync(0xffffffffu, s.z, b);
      s.w = __shfl_xor_sync(0xffffffffu, s.w, b);
      if (hi)
        v[j] = s;
      else
        v[j | b] = s;
    }
  }
}

// Writes 32 channels of an output row per lane, o[OFF ..] scaled by inv (0
// where `empty`), as bf16.  Four adjacent lanes hold four adjacent rows and
// exchange pieces first, so that they write 64 bytes of one row together, not
// half a sector of a row each.  `out`: the first of the channels in the first
// of the four rows, `rows` (0 or less: none) of which are written, `stride`
// elements apart.  Each lane its own row / with the exchange (us): one tile per
// CTA, 32/8 heads 1024 rows bf16 19.1 / 17.8, 192/128 351 / 344, FP8 exact
// 346 / 334, Lean P 272 / 267; two tiles, 12 prompts 288 / 285, 16384 rows
// 1903 / 1869.
template <int OFF, int N>
__device__ __forceinline__ void store_channels(__nv_bfloat16* out, int64_t stride, int rows, const uint32_t (&o)[N], float inv, bool empty,
                                               int lane) {
  uint4 v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float f[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) f[z] = empty ? 0.0f : __uint_as_float(o[OFF + 8 * q + z]) * inv;
    v[q] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
  transpose_pieces(v, lane);
  out += (lane & 3) * 8;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (r < rows) *reinterpret_cast<uint4*>(out + r * stride) = v[r];
}

}  // namespace zq
