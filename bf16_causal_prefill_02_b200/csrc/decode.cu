// decode.cu -- attention of one new token per sequence over a paged cache.
//
//   s_c = scale * k_descale * q . k_c,  o = softmax(s) v * v_descale,
//   lse = logsumexp(s)      over the n = seqlens[b] cached keys c.
//
// Bound by reading the cache once: n * Hkv * (d_qk + d_v) elements against
// 2 * (Hq / Hkv) * (d_qk + d_v) operations a key.  So:
//   * The query heads of a kv head share every key and value that is read.
//     The products are m16n8k16 with the long side on the 16: S^T = K Q^T (16
//     keys by 8 heads) and O^T = V^T P^T (16 channels by 8 heads), so a group of
//     up to 8 heads leaves little of them empty; up to 16 take two products
//     side by side (NT = 2), larger groups further head tiles.
//   * P^T is rounded to bf16 twice, P = P_hi + P_lo, over a bf16 cache: the
//     tensor work is not what bounds the kernel and the output keeps the 32-bit
//     weights' precision.  Over an e4m3 cache P is f16, which is exact to 2^-11
//     from 2^-14 on; the weights are kept near the top of its range (Weights),
//     so that many keys far below one (an attention sink) still count.
//   * The cache's length is split.  All key tiles of all (sequence, kv head)
//     pairs form one line that is cut into equal pieces, one per warp, so
//     ragged lengths cost no balance.  A piece that holds a whole (sequence,
//     head) writes the output; a cut one writes (m, l, O) to the workspace and
//     decode_join_kernel joins the parts: M = max m_j, l = sum l_j 2^(m_j - M),
//     o = sum O_j 2^(m_j - M) / l.  The order is fixed, so runs repeat bit for
//     bit.  Where the table has room for few keys there is no line: the warps of
//     a block, or of a cluster of up to 8, share a (sequence, kv head) and join in
//     shared memory.
//     Pieces go to warps side by side: where the heads allow it, the 2 or 4
//     warps of a team walk the same keys of adjacent heads, so that the 256
//     (bf16) or 128 (e4m3) bytes that a head has of a key are read together
//     with its neighbours' (32/8 heads e4m3, 64 x 8192 keys: 181 us against
//     203 with heads apart).
//   * A warp streams its keys through a ring of cp.async stages of its own and
//     waits for no other warp: the start and the end of one's segment overlap
//     the others' streams on the SM.
// Keys past the end, and keys whose page is not in the cache, are not read:
// their rows are filled with zeros and masked, so what lies there (NaN too)
// does not matter.
#include <cuda_fp16.h>

#include <type_traits>

#include "paged.cuh"

namespace zq {

namespace {

constexpr int kHeads = 8;        // query heads per product (n8)
constexpr int kMaxHeads = 16;    // query heads per head tile
constexpr int kCtasPerSm = 2;
constexpr int kMaxEntries = 1280;  // warps that the workspace has room for
// What a segment costs beyond its tiles (first loads, last stores), in tiles:
// a piece of many short segments gets fewer of them (64 sequences of 1 to 4096
// keys, 32/8 heads bf16: 51 us with 1, 48 with 2, 44 with 4 and with 8).
constexpr int kSegmentCost = 4;
constexpr int kJoinWarps = 4;
constexpr int kItemWarps = 8;
constexpr int kJoinBatch = 8;  // parts' rows on their way at once
constexpr int kJoinAlone = 24;  // parts that one warp joins by itself
// The reference of the weights 2^(s - ref) moves when one would pass 2^kTop, to
// where the largest is 2^kHead.  bf16 weights have fp32's range: 2^8 and 1.
// f16's range ends at 2^16 and its 11 bits at 2^-14, so e4m3 caches take 2^15 and
// 2^11: weights down to 2^-25 of the largest keep their bits, and a smaller one
// is off by 2^-36 of the largest at most.  (With 2^8 and 1 a key 25.6 octaves
// above 10^5 others took all of their weight.  The time is the same: 128 x up to
// 16384 keys 176.0 us with 2^8 and 1, 176.0 with 2^15 and 2^7, 176.6 with 2^15
// and 2^11; 64 x 8192 keys 185.1, 185.5, 184.1.)
template <int FP8>
struct Weights {
  static constexpr float kTop = FP8 ? 15.0f : 8.0f;
  static constexpr float kHead = FP8 ? 11.0f : 0.0f;
};
constexpr unsigned kJoinStep = 733;  // prime, and no divisor of a number of entries (at most 1280)

struct DecodeParams {
  PagedKV c;
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* out;
  float* lse;
  float scale;   // softmax scale times log2(e)
  int Hq, group, head_tiles;
  int team;      // warps that walk the same keys of adjacent heads: 1, 2 or 4, dividing the flat head tiles
  int slot;      // floats of a part: O of 8 or 16 heads, then their (m, l)
  // workspace: who cuts what, then the parts
  // {sequence, flat head tile, parts, first part's entry} of a (sequence, head
  // tile) that is cut, parts = 0 where it is not: one per (sequence, head tile)
  // where by_item, else one per entry [piece][team], of the one it begins
  int4* cut;
  int by_item;
  // without a line: warps that share a (sequence, head tile), 1 or all of a
  // cluster of 2^cluster_log2 blocks
  int share, cluster_log2;
  float* part;   // [piece][team][2][slot]: slot 0 a segment begun by an earlier piece, slot 1 one left to later pieces
};

template <int DQK, int FP8, int NT>
struct DecGeo {
  static constexpr int DV = 128;
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int KCH = DQK * ES / 16;             // 16-byte pieces per key row
  static constexpr int VCH = DV * ES / 16;
  // keys per tile (one step of a warp): 8 or 10 KB either way
  static constexpr int KEYS = FP8 ? 32 : 16;
  static constexpr int KB = KEYS / 16;                  // 16-key blocks of a tile
  static constexpr int KBYTES = KEYS * KCH * 16;
  static constexpr int VBYTES = KEYS * VCH * 16;
  static constexpr int STAGE = KBYTES + VBYTES;
  static constexpr unsigned ALL = 0xffffffffu >> (32 - KEYS);
  static constexpr int WARPS = 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int FIT = 113 * 1024 / WARPS / STAGE;  // two CTAs per SM
  static constexpr int NS = FIT < 6 ? FIT : 6;
  static constexpr int RING = NS * STAGE;               // bytes per warp
  static constexpr int SMEM = WARPS * RING;
  static constexpr int QK_STEPS = DQK / 16;
  static_assert(NS >= 2, "a stage in use and one in flight");
  // place of piece ch of row r: pieces of eight rows fall in different banks
  __device__ static constexpr uint32_t at_k(int r, int ch) {
    return (uint32_t)(r * KCH + (KCH % 8 == 0 ? (ch ^ (r & 7)) : (ch ^ ((r >> 1) & 3)))) * 16;
  }
  __device__ static constexpr uint32_t at_v(int r, int ch) { return (uint32_t)(r * VCH + (ch ^ (r & 7))) * 16; }
};

// Transposes an 8 x 8 tile of 16-bit values that the warp holds two a lane.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// All blocks of the cluster; what they wrote to shared memory is visible after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Loads from the same place of block `rank`'s shared memory.
__device__ __forceinline__ uint32_t peer_address(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float2 ld_cluster2(const void* p, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(peer_address(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(const void* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer_address(p, rank))
               : "memory");
  return v;
}

__device__ __forceinline__ int keys_of(const PagedKV& c, int b) {
  const int64_t cap = (int64_t)c.table_width << c.page_shift;
  return (int)min((int64_t)max(c.seqlens[b], 0), cap);
}

// Running (m, l, O) of a row, a lane's four channels of O.
struct Part {
  float m = -INFINITY, l = 0.0f;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __device__ __forceinline__ void add(float2 st, float4 v) {
    const float nm = fmaxf(m, st.x), nb = nm == -INFINITY ? 0.0f : nm;
    const float fa = ex2_approx(m - nb), fb = ex2_approx(st.x - nb);
    l = l * fa + st.y * fb;
    a.x = a.x * fa + v.x * fb;
    a.y = a.y * fa + v.y * fb;
    a.z = a.z * fa + v.z * fb;
    a.w = a.w * fa + v.w * fb;
    m = nm;
  }
};

// LINE: the keys as one line in equal pieces, with parts for the join.  Else a
// (sequence, head tile) is one warp's or one block's, and nothing is left.
template <int DQK, int FP8, int NT, int LINE>
__global__ void __launch_bounds__(DecGeo<DQK, FP8, NT>::THREADS, kCtasPerSm) decode_kernel(const DecodeParams p) {
  using G = DecGeo<DQK, FP8, NT>;
  using W = Weights<FP8>;
  constexpr int DV = G::DV, NS = G::NS, WARPS = G::WARPS, THREADS = G::THREADS;
  constexpr unsigned kFull = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan[WARPS];
  __shared__ int64_t first_off[WARPS];
  __shared__ int first_b[WARPS];
  __shared__ float2 stat_s[WARPS][kMaxHeads];
  const PagedKV& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, ql = lane & 3;
  const int heads = c.Hkv * p.head_tiles / p.team;  // teams of flat head tiles
  launch_dependents();
  wait_previous_kernel();

  // ---- the line: b outermost, then the team's heads, then kSegmentCost
  // places without a tile and the key tiles
  auto places = [&](int b) -> int64_t {
    const int n = keys_of(c, b);
    return n > 0 ? (int64_t)((n + G::KEYS - 1) / G::KEYS + kSegmentCost) * heads : 0;
  };
  int64_t x = 0, x1 = 0, line = 0;  // this warp's piece
  int pieces = 0;
  const int per_cta = WARPS / p.team;
  const int piece = warp / p.team * gridDim.x + blockIdx.x;  // (few pieces are spread over the SMs)
  const int mine_at = piece * p.team + warp % p.team;        // this warp's entry of cut and part
  if constexpr (LINE) {
    const int per = (c.B + THREADS - 1) / THREADS;
    const int b0 = min((int)threadIdx.x * per, c.B), b1 = min(b0 + per, c.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += places(b);
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) scan[warp] = sum;
    __syncthreads();
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += scan[w];
      line += scan[w];
    }
    // No more pieces than places, so that none is empty, nor so many of one
    // (sequence, head) that joining them costs more than a longer piece: about
    // 0.5 us a tile against 0.02 us a part (8/2 heads bf16, 2 x 11382 keys:
    // 17.8 us with the 296 parts that the warps allow, 13.1 with 143).
    const int least = max((int)sqrtf((float)(line / ((int64_t)c.B * heads)) * (1.0f / 22.0f)), 1);
    pieces = (int)min((int64_t)gridDim.x * per_cta, max(line / least, (int64_t)1));
    const int64_t at0 = before + sum - mine;  // place of this thread's first sequence
    for (int w = 0; w < per_cta; ++w) {
      const int pw = w * gridDim.x + blockIdx.x;
      if (pw >= pieces) break;
      const int64_t y = line * pw / pieces;
      if (y < at0 || y >= at0 + mine) continue;
      int64_t at = at0;
      int b = b0;
      for (; b + 1 < b1; ++b) {
        const int64_t n = places(b);
        if (y < at + n) break;
        at += n;
      }
      first_b[w] = b;
      first_off[w] = y - at;
    }
    __syncthreads();
    if (piece < pieces) {
      x = line * piece / pieces;
      x1 = line * (piece + 1) / pieces;
    }
  }
  // sequences without keys: 0 and -inf
  for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
    if (keys_of(c, b) > 0) continue;
    if (LINE && p.by_item)
      for (int i = threadIdx.x; i < c.Hkv * p.head_tiles; i += THREADS) p.cut[b * c.Hkv * p.head_tiles + i] = make_int4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < p.Hq * DV / 2; i += THREADS)
      reinterpret_cast<uint32_t*>(p.out + (int64_t)b * p.Hq * DV)[i] = 0u;
    if (p.lse)
      for (int i = threadIdx.x; i < p.Hq; i += THREADS) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
  }

  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(smem + warp * G::RING));
  const int64_t krow = (int64_t)c.Hkv * (DQK * G::ES), vrow = (int64_t)c.Hkv * (DV * G::ES);
  int4 cut = make_int4(0, 0, 0, 0);  // the segment of this piece that is left to later ones

  int b = 0;
  int64_t off = 0;
  if (LINE && x < x1) {
    b = first_b[warp / p.team];
    off = first_off[warp / p.team];
  }
  const int flat = c.Hkv * p.head_tiles;
  // without a line: items are (sequence, flat head tile)
  const bool shared = !LINE && p.share > 1;
  const int ranks = LINE ? 1 : 1 << p.cluster_log2, rank = blockIdx.x & (ranks - 1);
  const unsigned items = (unsigned)c.B * flat;  // (at most 65535 * 4096)
  unsigned item = shared ? blockIdx.x >> p.cluster_log2 : blockIdx.x + warp * gridDim.x;
  while (LINE ? x < x1 : item < items) {
    if (!LINE) b = (int)(item / (unsigned)flat);
    const int len = keys_of(c, b);
    const int tiles = (len + G::KEYS - 1) / G::KEYS, span = tiles + kSegmentCost;
    int fh, t0 = 0, steps = tiles;
    int64_t start = 0;
    if constexpr (!LINE) {
      static_assert(WARPS == 4, "a shift by 2");
      fh = (int)item - b * flat;
      item += shared ? gridDim.x >> p.cluster_log2 : gridDim.x * WARPS;
      if (shared) {  // a part of the keys each (few: below 2^16 tiles)
        const int at = rank * WARPS + warp, sh = p.cluster_log2 + 2;
        t0 = tiles * at >> sh;
        steps = (tiles * (at + 1) >> sh) - t0;
      }
      if (len == 0 && !shared) continue;  // (shared: the barriers below are everyone's, whatever a length does meanwhile)
    } else {
      if (len == 0 || off >= (int64_t)span * heads) {
        off -= len == 0 ? 0 : (int64_t)span * heads;
        if (++b >= c.B) break;
        continue;
      }
      fh = (int)(off / span) * p.team + warp % p.team;
      const int r0 = (int)(off % span);
      const int r1 = (int)min((int64_t)span, r0 + (x1 - x));
      start = x - r0;  // the (sequence, team)'s first place
      x += r1 - r0;
      off += r1 - r0;
      t0 = max(r0 - kSegmentCost, 0);
      steps = r1 - kSegmentCost - t0;
      if (steps <= 0) continue;
    }
    const int g = fh / p.head_tiles, ht = fh % p.head_tiles;
    const int h0 = g * p.group + ht * kMaxHeads;            // first query head of the tile
    const int rows = min(kMaxHeads, p.group - ht * kMaxHeads);  // query heads in it

    // ---- the segment's keys: tile `step` holds keys key0 + step * 16 ...
    const int32_t* table = c.table + b * c.table_stride;
    const int key0 = t0 * G::KEYS;
    const char* kbase = c.k + (int64_t)g * (DQK * G::ES);
    const char* vbase = c.v + (int64_t)g * (DV * G::ES);
    const int page_mask = (1 << c.page_shift) - 1;
    const bool whole = page_mask >= 15;  // each 16-key block of a tile lies in one page
    // the page of key (step, lane % KEYS), or -1: not there
    auto page_at = [&](int step) -> int {
      const int key = key0 + step * G::KEYS + (lane & (G::KEYS - 1));
      int pg = -1;
      if (step < steps && key < len) pg = table[key >> c.page_shift];
      return (unsigned)pg < (unsigned)c.num_pages ? pg : -1;
    };
    // starts the loads of a tile into the stage at sk; returns which of its keys are there
    auto load = [&](int step, uint32_t sk, int pg) -> unsigned {
      const unsigned vm = __ballot_sync(kFull, pg >= 0) & G::ALL;
      const uint32_t sv = sk + G::KBYTES;
      const int kb = key0 + step * G::KEYS;
      if (whole) {
        // rows of a block at fixed distances.  Where a row is 8, 16 or 32
        // pieces, the lane's piece is the same in all of them.
        auto rows_of = [&](auto all) {
          auto copy = [&](uint32_t dst, const char* src, int r) {
            if constexpr (all.value)
              cp_async16(dst, src);
            else
              cp_async16(dst, src, (vm >> r) & 1u ? 16 : 0);
          };
#pragma unroll
          for (int blk = 0; blk < G::KB; ++blk) {
            const int64_t page = max(__shfl_sync(kFull, pg, blk * 16), 0);  // (a block's first key is there if any is)
            const int64_t row = (kb + blk * 16) & page_mask;
            const char* ks = kbase + page * c.k_page + row * krow;
            const char* vs = vbase + page * c.v_page + row * vrow;
            if constexpr (32 % G::KCH == 0) {
              constexpr int R = 32 / G::KCH;
              const int r0 = lane / G::KCH, ch = lane % G::KCH;
              const char* src = ks + r0 * krow + ch * 16;
#pragma unroll
              for (int i = 0; i < 16; i += R, src += R * krow) copy(sk + G::at_k(blk * 16 + i + r0, ch), src, blk * 16 + i + r0);
            } else {
#pragma unroll
              for (int i = 0; i < 16 * G::KCH / 32; ++i) {
                const int idx = i * 32 + lane, r = idx / G::KCH, ch = idx % G::KCH;
                copy(sk + G::at_k(blk * 16 + r, ch), ks + r * krow + ch * 16, blk * 16 + r);
              }
            }
            constexpr int R = 32 / G::VCH;
            const int r0 = lane / G::VCH, ch = lane % G::VCH;
            const char* src = vs + r0 * vrow + ch * 16;
#pragma unroll
            for (int i = 0; i < 16; i += R, src += R * vrow) copy(sv + G::at_v(blk * 16 + i + r0, ch), src, blk * 16 + i + r0);
          }
        };
        if (vm == G::ALL)
          rows_of(std::true_type{});
        else
          rows_of(std::false_type{});
      } else {
#pragma unroll 1
        for (int idx = lane; idx < G::KEYS * G::KCH; idx += 32) {
          const int r = idx / G::KCH, ch = idx % G::KCH, rp = __shfl_sync(kFull, pg, r);
          cp_async16(sk + G::at_k(r, ch), kbase + max(rp, 0) * c.k_page + ((kb + r) & page_mask) * krow + ch * 16, rp >= 0 ? 16 : 0);
        }
#pragma unroll 1
        for (int idx = lane; idx < G::KEYS * G::VCH; idx += 32) {
          const int r = idx / G::VCH, ch = idx % G::VCH, rp = __shfl_sync(kFull, pg, r);
          cp_async16(sv + G::at_v(r, ch), vbase + max(rp, 0) * c.v_page + ((kb + r) & page_mask) * vrow + ch * 16, rp >= 0 ? 16 : 0);
        }
      }
      return vm;
    };
    // ---- queries as B fragments: column (head) quad of each product, and the
    // score scale of the columns 2 ql, 2 ql + 1 that this lane holds of S^T
    uint32_t qb[NT][G::QK_STEPS][2];
    const float c2 = p.scale * (FP8 && c.k_descale ? c.k_descale[c.descale_per_head ? g : 0] : 1.0f);
    float cr[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * kHeads + quad;
      const bool there = h < rows;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + b * p.q_stride + (int64_t)(h0 + (there ? h : 0)) * DQK);
      if constexpr (!FP8) {
#pragma unroll
        for (int ks = 0; ks < G::QK_STEPS; ++ks) {
          qb[nt][ks][0] = there ? src[ks * 8 + ql] : 0u;
          qb[nt][ks][1] = there ? src[ks * 8 + 4 + ql] : 0u;
        }
        cr[nt][0] = cr[nt][1] = c2;
      } else {
        // f16 operands (an e4m3 value is exact in f16).  A power of two brings
        // the head's largest query to [1, 2), so the bf16 values fit f16's
        // range, exactly for all within 2^-14 of the largest; the factor goes
        // into the score scale.  Order: a lane's four bytes of a 16-byte key
        // piece are channels 4 ql .. 4 ql + 3.
        float big = 0.0f;
#pragma unroll
        for (int ks = 0; ks < G::QK_STEPS; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = there ? src[ks * 8 + 2 * ql + i] : 0u;
            qb[nt][ks][i] = w;
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
          }
        big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
        big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
        const int ex = (int)(__float_as_uint(big) >> 23);  // biased exponent (0: subnormal or zero)
        const int e = ex == 255 ? 0 : min(max(ex - 127, -126), 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e
#pragma unroll
        for (int ks = 0; ks < G::QK_STEPS; ++ks) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qb[nt][ks][i];
            qb[nt][ks][i] = pack_f16x2(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xffff0000u) * down);
          }
        }
        const float mine = c2 * __uint_as_float((uint32_t)(127 + e) << 23);
        cr[nt][0] = __shfl_sync(kFull, mine, ql * 8);
        cr[nt][1] = __shfl_sync(kFull, mine, ql * 8 + 4);
      }
    }

    // O^T: rows (channels) by heads.  bf16: row quad, quad + 8 of 16 i are
    // channels 16 i + quad, + 8; e4m3: 16 i + 2 quad, + 1.
    float o[NT][DV / 16][4];
    float ref[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < DV / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
      ref[nt][0] = ref[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
    }

    // One body for the filling, the steady state and the draining of the ring:
    // it loads tile `it` and works on tile it - (NS - 1).  (Unrolled over the
    // stages the code outgrew the instruction cache: 16/1 heads e4m3, 30 x
    // 13000 keys, 43.0 against 39.8 us.)
    unsigned have[NS];  // keys that are there, of tiles it - (NS - 1) .. it
#pragma unroll
    for (int i = 0; i < NS; ++i) have[i] = 0u;
    uint32_t s_load = 0, s_work = 0;  // stages, as byte offsets
    int pg = page_at(0);
#pragma unroll 1
    for (int it = 0; it < steps + NS - 1; ++it) {
      {
        // (the stage to be filled is that of the tile worked on last)
        __syncwarp();
#pragma unroll
        for (int i = 0; i + 1 < NS; ++i) have[i] = have[i + 1];
        have[NS - 1] = it < steps ? load(it, ring_u + s_load, pg) : 0u;
        cp_async_commit();
        pg = page_at(it + 1);
        s_load = s_load + G::STAGE == G::RING ? 0 : s_load + G::STAGE;
        if (it < NS - 1) continue;
        cp_async_wait<NS - 1>();
        __syncwarp();
        const uint32_t sk = ring_u + s_work, sv = sk + G::KBYTES;
        s_work = s_work + G::STAGE == G::RING ? 0 : s_work + G::STAGE;

        // S^T = K Q^T: of each 16 keys the lane holds quad (i < 2) and quad + 8 of heads 2 ql + (i & 1)
        float sc[NT][G::KB][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int kb = 0; kb < G::KB; ++kb) sc[nt][kb][0] = sc[nt][kb][1] = sc[nt][kb][2] = sc[nt][kb][3] = 0.0f;
        if constexpr (!FP8) {
          const int mr = (lane & 7) + ((lane >> 3) & 1) * 8, mc = lane >> 4;
#pragma unroll
          for (int ks = 0; ks < G::QK_STEPS; ++ks) {
            uint32_t a[4];
            ldmatrix_x4(a, sk + G::at_k(mr, 2 * ks + mc));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816<false>(sc[nt][0], a, qb[nt][ks][0], qb[nt][ks][1]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < G::QK_STEPS; ++ks) {
            uint32_t w[4], a[4];
            ldmatrix_x4(w, sk + G::at_k(lane, ks));
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
              e4m3x4_to_f16x4(w[2 * kb], a[0], a[2]);
              e4m3x4_to_f16x4(w[2 * kb + 1], a[1], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816<true>(sc[nt][kb], a, qb[nt][ks][0], qb[nt][ks][1]);
            }
          }
        }
        // log2 domain, mask
        const unsigned vm = have[0];
        float mx[NT][2];
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int kb = 0; kb < G::KB; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[nt][kb][i] *= cr[nt][i & 1];
        if (vm != G::ALL) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int kb = 0; kb < G::KB; ++kb)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!((vm >> (kb * 16 + quad + (i >> 1) * 8)) & 1u)) sc[nt][kb][i] = -INFINITY;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mx[nt][i] = fmaxf(sc[nt][0][i], sc[nt][0][2 + i]);
            if constexpr (G::KB == 2) mx[nt][i] = fmaxf(mx[nt][i], fmaxf(sc[nt][1][i], sc[nt][1][2 + i]));
            move |= mx[nt][i] > ref[nt][i] + W::kTop;
          }
        if (__any_sync(kFull, move)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float m = mx[nt][i];
              m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
              m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
              m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
              const float nref = fmaxf(ref[nt][i], m - W::kHead);
              const float f = (nref == -INFINITY || nref == ref[nt][i]) ? 1.0f : ex2_approx(ref[nt][i] - nref);
              ref[nt][i] = nref;
              l[nt][i] *= f;
#pragma unroll
              for (int n = 0; n < DV / 16; ++n) {
                o[nt][n][i] *= f;
                o[nt][n][2 + i] *= f;
              }
            }
        }
        uint32_t pb[NT][G::KB][2], pl[NT][2];  // P^T as B fragments: keys 2 ql, 2 ql + 1 (and + 8) of head quad
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float n0 = ref[nt][0] == -INFINITY ? 0.0f : ref[nt][0], n1 = ref[nt][1] == -INFINITY ? 0.0f : ref[nt][1];
#pragma unroll
          for (int kb = 0; kb < G::KB; ++kb)
#pragma unroll
            for (int kh = 0; kh < 2; ++kh) {
              const float p0 = ex2_approx(sc[nt][kb][2 * kh] - n0), p1 = ex2_approx(sc[nt][kb][2 * kh + 1] - n1);
              l[nt][0] += p0;
              l[nt][1] += p1;
              if constexpr (FP8) {
                pb[nt][kb][kh] = transpose_8x8(pack_f16x2(p0, p1));
              } else {
                const uint32_t w = pack_bf16x2(p0, p1);
                pb[nt][kb][kh] = transpose_8x8(w);
                pl[nt][kh] = transpose_8x8(pack_bf16x2(p0 - __uint_as_float(w << 16), p1 - __uint_as_float(w & 0xffff0000u)));
              }
            }
        }
        // O^T += V^T P^T
        if constexpr (!FP8) {
          const int vr = (lane & 7) + (lane >> 4) * 8, vc = (lane >> 3) & 1;
#pragma unroll
          for (int i = 0; i < DV / 16; ++i) {
            uint32_t a[4];
            ldmatrix_x4_trans(a, sv + G::at_v(vr, 2 * i + vc));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816<false>(o[nt][i], a, pb[nt][0][0], pb[nt][0][1]);
              mma_16816<false>(o[nt][i], a, pl[nt][0], pl[nt][1]);
            }
          }
        } else {
          // a 16-bit element of the transposed load is two channels of a key:
          // the even ones are rows quad, the odd ones rows quad + 8
#pragma unroll
          for (int i = 0; i < DV / 16; ++i) {
            uint32_t w[4], a[4];
            ldmatrix_x4_trans(w, sv + G::at_v(lane, i));
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
              e4m3x4_to_f16x4(prmt(w[2 * kb], 0u, 0x3120u), a[0], a[1]);
              e4m3x4_to_f16x4(prmt(w[2 * kb + 1], 0u, 0x3120u), a[2], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816<true>(o[nt][i], a, pb[nt][kb][0], pb[nt][kb][1]);
            }
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- the segment's end: to the output, to this piece's slot, or joined
    // with the other warps' parts.  O^T goes through the ring so that rows of
    // channels are written whole.
    const bool begins = t0 == 0, ends = t0 + steps == tiles;
    const float vds = FP8 && c.v_descale ? c.v_descale[c.descale_per_head ? g : 0] : 1.0f;
    float* const slot = p.part + ((int64_t)mine_at * 2 + (begins ? 1 : 0)) * p.slot;
    constexpr int PITCH = DV + 4;
    static_assert(NT * kHeads * PITCH * 4 <= G::RING, "all O fit the ring");
    auto turn_of = [&](int w) { return reinterpret_cast<float*>(smem + w * G::RING); };  // [8 or 16 heads][132]
    float* const turn = turn_of(warp);
    auto write_row = [&](int h, float m, float sum, float4 v) {
      const int64_t row = (int64_t)b * p.Hq + h0 + h;
      // no key was there (sum = 0): 0 and -inf; NaN stays NaN
      const bool empty = sum == 0.0f;
      const float inv = vds / sum;
      reinterpret_cast<uint2*>(p.out + row * DV)[lane] =
          empty ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
      if (p.lse && lane == 0) p.lse[row] = empty ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[nt][i] += __shfl_xor_sync(kFull, l[nt][i], 4);
        l[nt][i] += __shfl_xor_sync(kFull, l[nt][i], 8);
        l[nt][i] += __shfl_xor_sync(kFull, l[nt][i], 16);
#pragma unroll
        for (int n = 0; n < DV / 16; ++n) {
          float* dst = turn + (nt * kHeads + 2 * ql + i) * PITCH + n * 16;
          if constexpr (!FP8) {
            dst[quad] = o[nt][n][i];
            dst[quad + 8] = o[nt][n][2 + i];
          } else {
            *reinterpret_cast<float2*>(dst + 2 * quad) = make_float2(o[nt][n][i], o[nt][n][2 + i]);
          }
        }
      }
      if (shared) {
        if (quad == 0) {
          stat_s[warp][nt * kHeads + 2 * ql] = make_float2(ref[nt][0], l[nt][0]);
          stat_s[warp][nt * kHeads + 2 * ql + 1] = make_float2(ref[nt][1], l[nt][1]);
        }
        continue;
      }
      __syncwarp();
#pragma unroll
      for (int r = 0; r < kHeads; ++r) {
        const int h = nt * kHeads + r;
        const float m = __shfl_sync(kFull, ref[nt][r & 1], r >> 1), sum = __shfl_sync(kFull, l[nt][r & 1], r >> 1);
        if (h >= rows) break;
        const float4 v = *reinterpret_cast<const float4*>(turn + h * PITCH + lane * 4);
        if (!LINE || (begins && ends)) {
          write_row(h, m, sum, v);
        } else {
          reinterpret_cast<float4*>(slot + h * DV)[lane] = v;
          if (lane == 0) *reinterpret_cast<float2*>(slot + p.slot - NT * kHeads * 2 + 2 * h) = make_float2(m, sum);
        }
      }
      __syncwarp();
    }
    if (shared) {
      __syncthreads();
      for (int h = warp; h < rows; h += WARPS) {
        Part all;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) all.add(stat_s[w][h], *reinterpret_cast<const float4*>(turn_of(w) + h * PITCH + lane * 4));
        if (ranks == 1) {
          write_row(h, all.m, all.l, all.a);
        } else {  // the block's part, in warp 0's place
          __syncwarp();
          *reinterpret_cast<float4*>(turn_of(0) + h * PITCH + lane * 4) = all.a;
          if (lane == 0) stat_s[0][h] = make_float2(all.m, all.l);
        }
      }
      if (ranks == 1) {
        __syncthreads();  // (the rings are loaded again)
      } else {
        cluster_sync();
        for (int h = rank * WARPS + warp; h < rows; h += ranks * WARPS) {
          Part all;
          for (int r = 0; r < ranks; ++r) all.add(ld_cluster2(&stat_s[0][h], r), ld_cluster4(turn_of(0) + h * PITCH + lane * 4, r));
          write_row(h, all.m, all.l, all.a);
        }
        cluster_sync();  // (the others have read this block's part)
      }
    }
    if (LINE && begins) {
      // its parts: this piece's and those up to the one of its last place.
      // The piece of place y is the largest j with floor(line * j / pieces) <= y.
      const int64_t j = min(((start + span) * pieces - 1) / line, (int64_t)pieces - 1);
      const int4 mine = make_int4(b, fh, ends ? 0 : (int)(j - piece) + 1, mine_at);
      if (!p.by_item)
        cut = ends ? cut : mine;
      else if (lane == 0)
        p.cut[b * c.Hkv * p.head_tiles + fh] = mine;
    }
  }
  if (LINE && !p.by_item && lane == 0) p.cut[mine_at] = cut;
}

// Joins the parts of what was cut; blockIdx.y is the query head in the head
// tile.  BY_ITEM: a block for each (sequence, head tile), its warps share the
// parts.  Else a warp for each entry, which joins
// a few parts alone; the parts of one with many are shared by the block's
// warps.  Entries are dealt to the blocks in an order that is not theirs (a
// multiple modulo their number), because those of a team, or of equally long
// sequences, are cut at regular distances.
template <int BY_ITEM>
__global__ void __launch_bounds__((BY_ITEM ? kItemWarps : kJoinWarps) * 32) decode_join_kernel(const DecodeParams p, int entries) {
  constexpr int DV = 128, WARPS = BY_ITEM ? kItemWarps : kJoinWarps;
  constexpr unsigned kFull = 0xffffffffu;
  __shared__ float4 acc_s[WARPS][32];
  __shared__ float2 stat_s[WARPS];
  __shared__ int4 cut_s[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y;
  const int stats = p.slot / (DV + 2) * DV;  // where a part's (m, l) begin
  launch_dependents();
  wait_previous_kernel();
  // parts first, first + step, ...: 32 at a time, a lane each for (m, l), then
  // their O with weights that no longer depend on one another.  Slot 1 of the
  // entry that begins the segment, slot 0 of the same head's in later pieces.
  auto read = [&](Part& t, int at, int first, int step, int parts) {
    auto part = [&](int j) { return p.part + ((int64_t)(at + j * p.team) * 2 + (j == 0 ? 1 : 0)) * p.slot; };
    for (int j0 = first; j0 < parts; j0 += 32 * step) {
      const int n = min((parts - j0 + step - 1) / step, 32);
      auto o_of = [&](int i) { return reinterpret_cast<const float4*>(part(j0 + min(i, n - 1) * step) + r * DV)[lane]; };
      const float2 st = lane < n ? *reinterpret_cast<const float2*>(part(j0 + lane * step) + stats + 2 * r) : make_float2(-INFINITY, 0.0f);
      float4 v[kJoinBatch];
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) v[i] = o_of(i);
      float m = st.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      const float f = ex2_approx(st.x - (m == -INFINITY ? 0.0f : m));
      float l = st.y * f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int i0 = 0; i0 < n; i0 += kJoinBatch) {  // (the weights past the last part are 0)
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
          const float fi = i0 + i < n ? __shfl_sync(kFull, f, i0 + i) : 0.0f;
          a.x += v[i].x * fi;
          a.y += v[i].y * fi;
          a.z += v[i].z * fi;
          a.w += v[i].w * fi;
        }
        if (i0 + kJoinBatch < n) {
#pragma unroll
          for (int i = 0; i < kJoinBatch; ++i) v[i] = o_of(i0 + kJoinBatch + i);
        }
      }
      t.add(make_float2(m, l), a);
    }
  };
  auto write = [&](const Part& t, int4 d) {
    const int g = d.y / p.head_tiles, ht = d.y % p.head_tiles;
    const bool empty = t.l == 0.0f;
    const float vds = p.c.dtype == 1 && p.c.v_descale ? p.c.v_descale[p.c.descale_per_head ? g : 0] : 1.0f;
    const float inv = vds / t.l;
    const int64_t row = (int64_t)d.x * p.Hq + g * p.group + ht * kMaxHeads + r;
    reinterpret_cast<uint2*>(p.out + row * DV)[lane] =
        empty ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(t.a.x * inv, t.a.y * inv), pack_bf16x2(t.a.z * inv, t.a.w * inv));
    if (p.lse && lane == 0) p.lse[row] = empty ? -INFINITY : (t.m + log2f(t.l)) * 0.6931471805599453f;
  };
  auto share = [&](int4 e) {
    Part t;
    read(t, e.w, warp, WARPS, e.z);
    acc_s[warp][lane] = t.a;
    if (lane == 0) stat_s[warp] = make_float2(t.m, t.l);
    __syncthreads();
    if (warp == 0) {
      Part all;
#pragma unroll
      for (int v = 0; v < WARPS; ++v) all.add(stat_s[v], acc_s[v][lane]);
      write(all, e);
    }
  };
  auto rows_of = [&](int4 e) { return min(kMaxHeads, p.group - (e.y % p.head_tiles) * kMaxHeads); };
  if constexpr (BY_ITEM) {
    const int4 d = p.cut[blockIdx.x];
    if (d.z > 0 && r < rows_of(d)) share(d);
  } else {
    const int mine = (int)(((blockIdx.x * WARPS + warp) * kJoinStep) % (gridDim.x * WARPS));
    int4 d = mine < entries ? p.cut[mine] : make_int4(0, 0, 0, 0);
    if (r >= rows_of(d)) d.z = 0;
    if (d.z > 0 && d.z <= kJoinAlone) {
      Part t;
      read(t, d.w, 0, 1, d.z);
      write(t, d);
    }
    if (lane == 0) cut_s[warp] = d;
    __syncthreads();
    for (int w = 0; w < WARPS; ++w) {
      const int4 e = cut_s[w];
      if (e.z <= kJoinAlone) continue;
      share(e);
      __syncthreads();
    }
  }
}

template <int DQK, int FP8, int NT>
cudaError_t launch_kernel(DecodeParams& p, cudaStream_t st, int num_sms) {
  using G = DecGeo<DQK, FP8, NT>;
  p.slot = NT * kHeads * (G::DV + 2);
  // one piece per warp of the CTAs that are resident at once
  constexpr int most = kMaxEntries / G::WARPS;
  int grid = num_sms * kCtasPerSm < most ? num_sms * kCtasPerSm : most;
  const int entries = grid * G::WARPS;
  const int64_t items = (int64_t)p.c.B * p.c.Hkv * p.head_tiles;
  // Blocks of a (sequence, head tile) each where there are few, which then have
  // many parts (us, by item / by entry: 2 x 11382 keys 8/2 heads 13.1 / 17.8,
  // 11 x 244 keys 16/1 heads 10.2 / 14.5; but 19 x 70 keys 32/8 heads, 608
  // blocks, 11.4 / 9.9 and 86 x 1000 keys, 2752 blocks, 70 / 61).
  const int rows = p.group < kMaxHeads ? p.group : kMaxHeads;
  p.by_item = items * rows <= 4 * num_sms && items <= entries ? 1 : 0;
  // A table with room for few keys: nothing is cut, and nothing is left to join
  // in another launch.  A (sequence, head tile) is a cluster's of 1 to 8 blocks,
  // as many as are resident at once and have 8 tiles of the table each, as long
  // as a warp has no more than 8; or one warp's, where there are many and the
  // tables short.  Us, line / that, equal lengths, 32/8 heads bf16: 1 sequence of
  // 512 keys 7.8 / 5.2, 1024 8.6 / 5.8, 4096 11.4 / 9.2 (8192: 12.2 / 14.5, so the
  // line); 4 of 4096 19.2 / 15.9; 16 of 1024 21.5 / 15.2, of 1 to 1024 14.2 / 9.9
  // (4096: 52.0 / 45.6, but ragged ones are better off in the line); 64 of 512
  // 31.7 / 27.1; 256 of 64 23.3 / 17.7 by warps, 26.1 by blocks.  e4m3: 1 of 1024
  // 8.6 / 5.5; 16/1 heads, 64 of 2048 24.6 / 11.8, of 1 to 2048 22.5 / 11.1; 16/16
  // heads 192/128, 64 of 1 to 1024 38.4 / 42.8 by warps, so the line.  Clusters of
  // 1 / 2 / 4 / 8: 1 sequence bf16 of 256 keys 5.5 / 5.5 / 5.0 / 5.5, of 1024 11.8 /
  // 8.8 / 6.8 / 6.4.
  const int64_t tiles = (((int64_t)p.c.table_width << p.c.page_shift) + G::KEYS - 1) / G::KEYS;
  int cluster = 1;
  p.share = p.cluster_log2 = 0;
  if (items >= 4 * num_sms || (items > grid && tiles <= 4)) {
    if (tiles <= 16) p.share = 1;
  } else {
    while (cluster < 8 && tiles >= 16 * cluster && items * 2 * cluster <= grid) cluster *= 2;
    if (tiles <= 32 * cluster) p.share = cluster * G::WARPS;
  }
  if (p.share > 0) {
    while ((1 << p.cluster_log2) < cluster) ++p.cluster_log2;
    if (items * cluster < grid) grid = (int)items * cluster;
    grid -= grid % cluster;
  }
  auto kern = p.share > 0 ? decode_kernel<DQK, FP8, NT, 0> : decode_kernel<DQK, FP8, NT, 1>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_overlapped_cluster(kern, p.share > 0 ? (unsigned)cluster : 1u, dim3((unsigned)grid), dim3(G::THREADS), G::SMEM, st, p);
  if (e != cudaSuccess || p.share > 0) return e;
  if (p.by_item)
    return launch_overlapped(decode_join_kernel<1>, dim3((unsigned)items, (unsigned)rows), dim3(kItemWarps * 32), 0, st, p, entries);
  const unsigned blocks = (unsigned)((entries + kJoinWarps - 1) / kJoinWarps);
  return launch_overlapped(decode_join_kernel<0>, dim3(blocks, (unsigned)rows), dim3(kJoinWarps * 32), 0, st, p, entries);
}

template <int DQK, int FP8>
cudaError_t launch_variant(DecodeParams& p, cudaStream_t st, int num_sms) {
  return p.group <= kHeads ? launch_kernel<DQK, FP8, 1>(p, st, num_sms) : launch_kernel<DQK, FP8, 2>(p, st, num_sms);
}

constexpr size_t kCutBytes = (size_t)kMaxEntries * 16;

}  // namespace

size_t decode_workspace_bytes() { return kCutBytes + (size_t)kMaxEntries * 2 * kMaxHeads * (128 + 2) * 4; }

cudaError_t launch_decode(const DecodeLaunch& a, cudaStream_t st, int num_sms) {
  DecodeParams p;
  p.c = a.c;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.scale = a.scale_log2;
  p.Hq = a.Hq;
  p.group = a.Hq / a.c.Hkv;
  p.head_tiles = (p.group + kMaxHeads - 1) / kMaxHeads;
  const int heads = a.c.Hkv * p.head_tiles;
  p.team = heads % 4 == 0 ? 4 : heads % 2 == 0 ? 2 : 1;
  p.cut = static_cast<int4*>(a.workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kCutBytes);
  if (a.c.dtype == 1) return a.c.dqk == 128 ? launch_variant<128, 1>(p, st, num_sms) : launch_variant<192, 1>(p, st, num_sms);
  return a.c.dqk == 128 ? launch_variant<128, 0>(p, st, num_sms) : launch_variant<192, 0>(p, st, num_sms);
}

}  // namespace zq
