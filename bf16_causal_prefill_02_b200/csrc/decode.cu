// decode.cu -- attention of one new token per sequence over a paged cache.
//
//   s_c = scale * k_descale * q . k_c,  o = softmax(s) v * v_descale,
//   lse = logsumexp(s)      over the n = seqlens[b] cached keys c.
//
// Bound by reading the cache once: n * Hkv * (d_qk + d_v) elements against
// 2 * (Hq / Hkv) * (d_qk + d_v) operations a key.  So:
//   * The query heads of a kv head (16 at most; more go in further head
//     tiles) are the 16 rows of m16n8k16 products, and a key or value is read
//     from memory once for all of them.  The rows that a small group leaves
//     empty cost tensor work that is not what bounds the kernel.
//   * The cache's length is split.  All key tiles of all (sequence, kv head)
//     pairs form one line that is cut into equal pieces, one per warp, so
//     ragged lengths cost no balance.  A piece that holds a whole (sequence,
//     head) writes the output; a cut one writes (m, l, O) to the workspace and
//     decode_join_kernel joins the parts: M = max m_j, l = sum l_j 2^(m_j - M),
//     o = sum O_j 2^(m_j - M) / l.  The order is fixed, so runs repeat bit for
//     bit.
//   * A warp streams its keys through a ring of cp.async stages of its own and
//     waits for no other warp: the start and the end of one's segment overlap
//     the other seven's streams on the SM.
//   * With at most 8 query heads per kv head (SMALL) the product's other 8
//     rows carry what the rounding of the weights to bf16 leaves out: P = P_hi
//     + P_lo costs no further product, and rows 8-15 need no exponentials.
// Keys past the end, and keys whose page is not in the cache, are not read:
// their rows are filled with zeros and masked, so what lies there (NaN too)
// does not matter.
#include <cuda_fp16.h>

#include "paged.cuh"

namespace zq {

namespace {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kRows = 16;      // query heads per head tile
constexpr int kMaxCtas = 320;  // the workspace has room for their pieces
constexpr int kMaxPieces = kMaxCtas * kDecWarps;
constexpr int kCtasPerSm = 2;
constexpr int kSlot = kRows * 128 + 2 * kRows;  // floats of a part: O, then (m, l) per row
// What a segment costs beyond its tiles (first loads, last stores), in tiles:
// a piece of many short segments gets fewer of them.
constexpr int kSegmentCost = 2;
constexpr int kJoinWarps = 8;
constexpr int kJoinAlone = 8;  // parts that one warp joins by itself

struct DecodeParams {
  PagedKV c;
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* out;
  float* lse;
  float scale;
  int Hq, group, head_tiles;
  // workspace: who cuts what, then the parts
  int4* cut;     // [piece] {sequence, flat head tile, parts, 0} of the segment that this piece begins and does not finish
  float* part;   // [piece][2][kSlot]: slot 0 a segment begun by an earlier piece, slot 1 one left to later pieces
};

template <int DQK, int FP8>
struct DecGeo {
  static constexpr int DV = 128;
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int KW = FP8 ? 32 : 16;              // keys per tile (one step of a warp)
  static constexpr int KCH = DQK * ES / 16;             // 16-byte pieces per key row
  static constexpr int VCH = DV * ES / 16;
  static constexpr int KBYTES = KW * KCH * 16;
  static constexpr int VBYTES = KW * VCH * 16;
  static constexpr int STAGE = KBYTES + VBYTES;
  static constexpr int NS = DQK == 128 ? 3 : 2;         // stages that fit 113 KB (two CTAs per SM)
  static constexpr int RING = NS * STAGE;               // bytes per warp
  static constexpr int SMEM = kDecWarps * RING;
  static constexpr int QK_STEPS = DQK / 16;
  static_assert(SMEM <= 113 * 1024, "two CTAs per SM");
  // place of piece ch of row r: pieces of eight rows fall in different banks
  __device__ static constexpr uint32_t at_k(int r, int ch) {
    return (uint32_t)(r * KCH + (KCH % 8 == 0 ? (ch ^ (r & 7)) : (ch ^ ((r >> 1) & 3)))) * 16;
  }
  __device__ static constexpr uint32_t at_v(int r, int ch) { return (uint32_t)(r * VCH + (ch ^ (r & 7))) * 16; }
};

__device__ __forceinline__ int keys_of(const PagedKV& c, int b) {
  const int64_t cap = (int64_t)c.table_width << c.page_shift;
  return (int)min((int64_t)max(c.seqlens[b], 0), cap);
}

template <int DQK, int FP8, int SMALL>
__global__ void __launch_bounds__(kDecThreads, kCtasPerSm) decode_kernel(const DecodeParams p) {
  using G = DecGeo<DQK, FP8>;
  constexpr int DV = G::DV, KW = G::KW, NS = G::NS;
  constexpr int HF = SMALL ? 1 : 2;  // rows quad, and quad + 8 unless SMALL
  constexpr unsigned kFull = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan[kDecWarps];
  __shared__ int64_t first_off[kDecWarps];
  __shared__ int first_b[kDecWarps];
  const PagedKV& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, ql = lane & 3;
  const int heads = c.Hkv * p.head_tiles;
  launch_dependents();

  // ---- the line: b outermost, then the flat head tile, then kSegmentCost
  // places without a tile and the key tiles
  auto places = [&](int b) -> int64_t {
    const int n = keys_of(c, b);
    return n > 0 ? (int64_t)((n + KW - 1) / KW + kSegmentCost) * heads : 0;
  };
  int64_t x = 0, x1 = 0, line = 0;  // this warp's piece
  int pieces;
  const int piece = warp * gridDim.x + blockIdx.x;  // (few pieces are spread over the SMs)
  {
    const int per = (c.B + kDecThreads - 1) / kDecThreads;
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
    for (int w = 0; w < kDecWarps; ++w) {
      if (w < warp) before += scan[w];
      line += scan[w];
    }
    // no more pieces than places, so that none is empty
    pieces = (int)min((int64_t)gridDim.x * kDecWarps, line);
    const int64_t at0 = before + sum - mine;  // place of this thread's first sequence
    for (int w = 0; w < kDecWarps; ++w) {
      const int pw = w * gridDim.x + blockIdx.x;
      if (pw >= pieces) break;
      const int64_t y = line * pw / pieces;
      if (y < at0 || y >= at0 + mine) continue;
      int64_t at = at0;
      int b = b0;
      for (;; ++b) {
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
    for (int i = threadIdx.x; i < p.Hq * DV / 2; i += kDecThreads)
      reinterpret_cast<uint32_t*>(p.out + (int64_t)b * p.Hq * DV)[i] = 0u;
    if (p.lse)
      for (int i = threadIdx.x; i < p.Hq; i += kDecThreads) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
  }

  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(smem + warp * G::RING));
  int4 cut = make_int4(0, 0, 0, 0);  // the segment of this piece that is left to later ones

  int b = x < x1 ? first_b[warp] : 0;
  int64_t off = x < x1 ? first_off[warp] : 0;
  while (x < x1) {
    const int len = keys_of(c, b);
    const int tiles = (len + KW - 1) / KW, span = tiles + kSegmentCost;
    if (len == 0 || off >= (int64_t)span * heads) {
      off -= len == 0 ? 0 : (int64_t)span * heads;
      ++b;
      continue;
    }
    const int fh = (int)(off / span), r0 = (int)(off % span);
    const int r1 = (int)min((int64_t)span, r0 + (x1 - x));
    const int64_t start = x - r0;  // the (sequence, head)'s first place
    x += r1 - r0;
    off += r1 - r0;
    const int t0 = max(r0 - kSegmentCost, 0);
    const int steps = r1 - kSegmentCost - t0;
    if (steps <= 0) continue;
    const int g = fh / p.head_tiles, ht = fh % p.head_tiles;
    const int h0 = g * p.group + ht * kRows;          // first query head of the tile
    const int rows = min(kRows, p.group - ht * kRows);  // query heads in it

    // ---- queries as A fragments: rows quad and quad + 8
    uint32_t qa[G::QK_STEPS][4];
    if constexpr (SMALL) {
#pragma unroll
      for (int ks = 0; ks < G::QK_STEPS; ++ks) qa[ks][1] = qa[ks][3] = 0u;
    }
    const float c2 = p.scale * (FP8 && c.k_descale ? c.k_descale[c.descale_per_head ? g : 0] : 1.0f) * 1.4426950408889634f;
    float cr[2] = {c2, c2};
    {
      const __nv_bfloat16* qrow = p.q + b * p.q_stride + (int64_t)h0 * DQK;
#pragma unroll
      for (int hf = 0; hf < HF; ++hf) {
        const int r = quad + hf * 8;
        const bool there = r < rows;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(qrow + (int64_t)r * DQK);
        if constexpr (!FP8) {
#pragma unroll
          for (int ks = 0; ks < G::QK_STEPS; ++ks) {
            qa[ks][hf] = there ? src[ks * 8 + ql] : 0u;
            qa[ks][2 + hf] = there ? src[ks * 8 + 4 + ql] : 0u;
          }
        } else {
          // f16 operands (an e4m3 value is exact in f16).  A power of two
          // brings the row's largest query to [1, 2), so the bf16 values fit
          // f16's range, exactly for all within 2^-14 of the largest; the
          // factor goes into the score scale.  Element order: a lane's four
          // bytes of a 16-byte key piece are channels 4 ql .. 4 ql + 3.
          float big = 0.0f;
          uint32_t w[G::QK_STEPS][2];
#pragma unroll
          for (int ks = 0; ks < G::QK_STEPS; ++ks) {
            w[ks][0] = there ? src[ks * 8 + 2 * ql] : 0u;
            w[ks][1] = there ? src[ks * 8 + 2 * ql + 1] : 0u;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[ks][i] << 16)), fabsf(__uint_as_float(w[ks][i] & 0xffff0000u))));
          }
          big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
          big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
          const int ex = (int)(__float_as_uint(big) >> 23);  // biased exponent (0: subnormal or zero)
          const int e = ex == 255 ? 0 : min(max(ex - 127, -126), 126);
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e
          cr[hf] = c2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int ks = 0; ks < G::QK_STEPS; ++ks)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              qa[ks][2 * i + hf] = pack_f16x2(__uint_as_float(w[ks][i] << 16) * down, __uint_as_float(w[ks][i] & 0xffff0000u) * down);
        }
      }
    }

    // ---- the segment's keys
    const int32_t* table = c.table + b * c.table_stride;
    const int key0 = t0 * KW;
    const char* kbase = c.k + (int64_t)g * (DQK * G::ES);
    const char* vbase = c.v + (int64_t)g * (DV * G::ES);
    const int64_t krow = (int64_t)c.Hkv * (DQK * G::ES), vrow = (int64_t)c.Hkv * (DV * G::ES);
    const int page_mask = (1 << c.page_shift) - 1;
    // the page of key (step, lane), or -1: not there
    auto page_at = [&](int step) -> int {
      const int key = key0 + step * KW + lane;
      int pg = -1;
      if (lane < KW && step < steps && key < len) pg = table[key >> c.page_shift];
      return (unsigned)pg < (unsigned)c.num_pages ? pg : -1;
    };
    unsigned have[NS];  // which keys of each stage are there
    auto load = [&](int step, int s, int pg) {
      const unsigned vm = __ballot_sync(kFull, pg >= 0);
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i == s) have[i] = vm;
      const uint32_t sk = ring_u + s * G::STAGE, sv = sk + G::KBYTES;
      const int kb = key0 + step * KW;
#pragma unroll
      for (int i = 0; i < KW * G::KCH / 32; ++i) {
        const int idx = i * 32 + lane, r = idx / G::KCH, ch = idx % G::KCH;
        const int rp = __shfl_sync(kFull, pg, r);
        const char* src = kbase + max(rp, 0) * c.k_page + ((kb + r) & page_mask) * krow + ch * 16;
        cp_async16(sk + G::at_k(r, ch), src, rp >= 0 ? 16 : 0);
      }
#pragma unroll
      for (int i = 0; i < KW * G::VCH / 32; ++i) {
        const int idx = i * 32 + lane, r = idx / G::VCH, ch = idx % G::VCH;
        const int rp = __shfl_sync(kFull, pg, r);
        const char* src = vbase + max(rp, 0) * c.v_page + ((kb + r) & page_mask) * vrow + ch * 16;
        cp_async16(sv + G::at_v(r, ch), src, rp >= 0 ? 16 : 0);
      }
    };

    float o[DV / 8][4];
#pragma unroll
    for (int n = 0; n < DV / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    int pg = page_at(0);
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      if (s < steps) load(s, s, pg);
      cp_async_commit();
      pg = page_at(s + 1);
    }
    for (int st0 = 0; st0 < steps; st0 += NS) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int st = st0 + s;
        if (st >= steps) break;
        // the stage of step st - 1 is free: refill it, then wait for this one
        __syncwarp();
        if (st + NS - 1 < steps) load(st + NS - 1, (s + NS - 1) % NS, pg);
        cp_async_commit();
        pg = page_at(st + NS);
        cp_async_wait<NS - 1>();
        __syncwarp();
        const uint32_t sk = ring_u + s * G::STAGE, sv = sk + G::KBYTES;

        // S = Q K^T
        float sc[KW / 8][4];
#pragma unroll
        for (int n = 0; n < KW / 8; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < G::QK_STEPS; ++ks) {
          uint32_t kf[4];
          if constexpr (!FP8) {
            const int r = ((lane >> 4) << 3) + (lane & 7), ch = 2 * ks + ((lane >> 3) & 1);
            ldmatrix_x4(kf, sk + G::at_k(r, ch));
            mma_16816<false>(sc[0], qa[ks], kf[0], kf[1]);
            mma_16816<false>(sc[1], qa[ks], kf[2], kf[3]);
          } else {
            ldmatrix_x4(kf, sk + G::at_k(lane, ks));
#pragma unroll
            for (int n = 0; n < 4; ++n)
              mma_16816<true>(sc[n], qa[ks], e4m3x2_to_f16x2(kf[n]), e4m3x2_to_f16x2(kf[n] >> 16));
          }
        }
        // log2 domain, mask
        const unsigned vm = have[s];
        float mx[HF];
#pragma unroll
        for (int hf = 0; hf < HF; ++hf) {
          mx[hf] = -INFINITY;
#pragma unroll
          for (int n = 0; n < KW / 8; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& z = sc[n][2 * hf + i];
              z *= cr[hf];
              if (!((vm >> (n * 8 + 2 * ql + i)) & 1u)) z = -INFINITY;
              mx[hf] = fmaxf(mx[hf], z);
            }
        }
        // the reference moves when a score passes it by 8 (weights stay below 2^8)
        if (__any_sync(kFull, mx[0] > ref[0] + 8.0f || mx[HF - 1] > ref[HF - 1] + 8.0f)) {
          float f[2];
#pragma unroll
          for (int hf = 0; hf < HF; ++hf) {
            float m = fmaxf(mx[hf], __shfl_xor_sync(kFull, mx[hf], 1));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
            const float nref = fmaxf(ref[hf], m);
            f[hf] = (nref == -INFINITY || nref == ref[hf]) ? 1.0f : ex2_approx(ref[hf] - nref);
            ref[hf] = nref;
            l[hf] *= f[hf];
          }
          if (SMALL) f[1] = f[0];  // the low parts of the same heads
#pragma unroll
          for (int n = 0; n < DV / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] *= f[i >> 1];
        }
        uint32_t pa[KW / 16][4];
#pragma unroll
        for (int hf = 0; hf < HF; ++hf) {
          const float nb = ref[hf] == -INFINITY ? 0.0f : ref[hf];
#pragma unroll
          for (int n = 0; n < KW / 8; ++n) {
            const float p0 = ex2_approx(sc[n][2 * hf] - nb), p1 = ex2_approx(sc[n][2 * hf + 1] - nb);
            l[hf] += p0 + p1;
            const uint32_t w = FP8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
            pa[n / 2][(n & 1) * 2 + hf] = w;
            if constexpr (SMALL && !FP8)
              pa[n / 2][(n & 1) * 2 + 1] = pack_bf16x2(p0 - __uint_as_float(w << 16), p1 - __uint_as_float(w & 0xffff0000u));
            else if constexpr (SMALL)
              pa[n / 2][(n & 1) * 2 + 1] = 0u;
          }
        }
        // O += P V
        if constexpr (!FP8) {
#pragma unroll
          for (int cp = 0; cp < G::VCH / 2; ++cp) {
            uint32_t vf[4];
            const int r = ((lane >> 3) & 1) * 8 + (lane & 7), ch = 2 * cp + (lane >> 4);
            ldmatrix_x4_trans(vf, sv + G::at_v(r, ch));
            mma_16816<false>(o[2 * cp], pa[0], vf[0], vf[1]);
            mma_16816<false>(o[2 * cp + 1], pa[0], vf[2], vf[3]);
          }
        } else {
          // a 16-bit element of the transposed load is two channels of a key:
          // the even ones go to product 2 ch, the odd ones to 2 ch + 1
#pragma unroll
          for (int ch = 0; ch < G::VCH; ++ch) {
            uint32_t vf[4];
            ldmatrix_x4_trans(vf, sv + G::at_v(lane, ch));
#pragma unroll
            for (int i = 0; i < 4; ++i) vf[i] = prmt(vf[i], 0u, 0x3120u);
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
              mma_16816<true>(o[2 * ch], pa[k2], e4m3x2_to_f16x2(vf[2 * k2]), e4m3x2_to_f16x2(vf[2 * k2 + 1]));
              mma_16816<true>(o[2 * ch + 1], pa[k2], e4m3x2_to_f16x2(vf[2 * k2] >> 16), e4m3x2_to_f16x2(vf[2 * k2 + 1] >> 16));
            }
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- the segment's end: to the output, or to this piece's slot
    const bool begins = t0 == 0, ends = t0 + steps == tiles;
    const float vds = FP8 && c.v_descale ? c.v_descale[c.descale_per_head ? g : 0] : 1.0f;
    float* const slot = p.part + ((int64_t)piece * 2 + (begins ? 1 : 0)) * kSlot;
#pragma unroll
    for (int hf = 0; hf < HF; ++hf) {
      l[hf] += __shfl_xor_sync(kFull, l[hf], 1);
      l[hf] += __shfl_xor_sync(kFull, l[hf], 2);
      if (SMALL && !FP8) {
#pragma unroll
        for (int n = 0; n < DV / 8; ++n) {
          o[n][0] += o[n][2];
          o[n][1] += o[n][3];
        }
      }
      const int r = quad + hf * 8;
      if (r >= rows) continue;
      if (begins && ends) {
        const int64_t row = (int64_t)b * p.Hq + h0 + r;
        // no key was there (l = 0): 0 and -inf; NaN stays NaN
        const bool empty = l[hf] == 0.0f;
        const float inv = vds / l[hf];
        auto two = [&](float a, float z) { return empty ? 0u : pack_bf16x2(a * inv, z * inv); };
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * DV);
        if constexpr (!FP8) {
#pragma unroll
          for (int n = 0; n < DV / 8; ++n) dst[n * 4 + ql] = two(o[n][2 * hf], o[n][2 * hf + 1]);
        } else {
#pragma unroll
          for (int ch = 0; ch < DV / 16; ++ch)
            reinterpret_cast<uint2*>(dst)[ch * 4 + ql] =
                make_uint2(two(o[2 * ch][2 * hf], o[2 * ch + 1][2 * hf]), two(o[2 * ch][2 * hf + 1], o[2 * ch + 1][2 * hf + 1]));
        }
        if (p.lse && ql == 0) p.lse[row] = empty ? -INFINITY : (ref[hf] + log2f(l[hf])) * 0.6931471805599453f;
      } else {
        float* dst = slot + r * DV;
        if constexpr (!FP8) {
#pragma unroll
          for (int n = 0; n < DV / 8; ++n)
            *reinterpret_cast<float2*>(dst + n * 8 + 2 * ql) = make_float2(o[n][2 * hf], o[n][2 * hf + 1]);
        } else {
#pragma unroll
          for (int ch = 0; ch < DV / 16; ++ch)
            *reinterpret_cast<float4*>(dst + ch * 16 + 4 * ql) =
                make_float4(o[2 * ch][2 * hf], o[2 * ch + 1][2 * hf], o[2 * ch][2 * hf + 1], o[2 * ch + 1][2 * hf + 1]);
        }
        if (ql == 0) *reinterpret_cast<float2*>(slot + kRows * DV + 2 * r) = make_float2(ref[hf], l[hf]);
      }
    }
    if (begins && !ends) {
      // its parts: this piece's and those up to the one of its last place.
      // The piece of place y is the largest j with floor(line * j / pieces) <= y.
      const int64_t j = ((start + span) * pieces - 1) / line;
      cut = make_int4(b, fh, (int)(j - piece) + 1, 0);
    }
    __syncwarp();
  }
  if (lane == 0) p.cut[piece] = cut;
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

// Joins the parts of the segments that were cut; blockIdx.y is the query head
// in the head tile.  A warp joins the few parts of its own piece's segment
// alone; the parts of a segment with many are shared by the block's warps.
__global__ void __launch_bounds__(kJoinWarps * 32) decode_join_kernel(const DecodeParams p, int pieces) {
  constexpr int DV = 128;
  __shared__ float4 acc_s[kJoinWarps][32];
  __shared__ float2 stat_s[kJoinWarps];
  __shared__ int4 cut_s[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y;
  const int mine = blockIdx.x * kJoinWarps + warp;
  wait_previous_kernel();
  // slot 1 of the piece that begins the segment, slot 0 of those after it
  auto read = [&](Part& t, int piece, int first, int step, int parts) {
#pragma unroll 4
    for (int j = first; j < parts; j += step) {
      const float* s = p.part + ((int64_t)(piece + j) * 2 + (j == 0 ? 1 : 0)) * kSlot;
      t.add(*reinterpret_cast<const float2*>(s + kRows * DV + 2 * r), reinterpret_cast<const float4*>(s + r * DV)[lane]);
    }
  };
  auto write = [&](const Part& t, int4 d) {
    const int g = d.y / p.head_tiles, ht = d.y % p.head_tiles;
    const bool empty = t.l == 0.0f;
    const float vds = p.c.dtype == 1 && p.c.v_descale ? p.c.v_descale[p.c.descale_per_head ? g : 0] : 1.0f;
    const float inv = vds / t.l;
    const int64_t row = (int64_t)d.x * p.Hq + g * p.group + ht * kRows + r;
    reinterpret_cast<uint2*>(p.out + row * DV)[lane] =
        empty ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(t.a.x * inv, t.a.y * inv), pack_bf16x2(t.a.z * inv, t.a.w * inv));
    if (p.lse && lane == 0) p.lse[row] = empty ? -INFINITY : (t.m + log2f(t.l)) * 0.6931471805599453f;
  };
  int4 d = mine < pieces ? p.cut[mine] : make_int4(0, 0, 0, 0);
  if (r >= min(kRows, p.group - (d.y % p.head_tiles) * kRows)) d.z = 0;
  if (d.z > 0 && d.z <= kJoinAlone) {
    Part t;
    read(t, mine, 0, 1, d.z);
    write(t, d);
  }
  if (lane == 0) cut_s[warp] = d;
  __syncthreads();
  for (int w = 0; w < kJoinWarps; ++w) {
    const int4 e = cut_s[w];
    if (e.z <= kJoinAlone) continue;
    Part t;
    read(t, blockIdx.x * kJoinWarps + w, warp, kJoinWarps, e.z);
    acc_s[warp][lane] = t.a;
    if (lane == 0) stat_s[warp] = make_float2(t.m, t.l);
    __syncthreads();
    if (warp == 0) {
      Part all;
#pragma unroll
      for (int v = 0; v < kJoinWarps; ++v) all.add(stat_s[v], acc_s[v][lane]);
      write(all, e);
    }
    __syncthreads();
  }
}

template <int DQK, int FP8, int SMALL>
cudaError_t launch_kernel(const DecodeParams& p, cudaStream_t st, int grid) {
  using G = DecGeo<DQK, FP8>;
  auto kern = decode_kernel<DQK, FP8, SMALL>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<grid, kDecThreads, G::SMEM, st>>>(p);
  return cudaGetLastError();
}

template <int DQK, int FP8>
cudaError_t launch_variant(const DecodeParams& p, cudaStream_t st, int grid) {
  return p.group <= 8 ? launch_kernel<DQK, FP8, 1>(p, st, grid) : launch_kernel<DQK, FP8, 0>(p, st, grid);
}

constexpr size_t kCutBytes = (size_t)kMaxPieces * 16;

}  // namespace

size_t decode_workspace_bytes() { return kCutBytes + (size_t)kMaxPieces * 2 * kSlot * 4; }

cudaError_t launch_decode(const DecodeLaunch& a, cudaStream_t st, int num_sms) {
  DecodeParams p;
  p.c = a.c;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.scale = a.softmax_scale;
  p.Hq = a.Hq;
  p.group = a.Hq / a.c.Hkv;
  p.head_tiles = (p.group + kRows - 1) / kRows;
  p.cut = static_cast<int4*>(a.workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kCutBytes);
  const int grid = num_sms * kCtasPerSm < kMaxCtas ? num_sms * kCtasPerSm : kMaxCtas;
  cudaError_t e;
  if (a.c.dtype == 1)
    e = a.c.dqk == 128 ? launch_variant<128, 1>(p, st, grid) : launch_variant<192, 1>(p, st, grid);
  else
    e = a.c.dqk == 128 ? launch_variant<128, 0>(p, st, grid) : launch_variant<192, 0>(p, st, grid);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int pieces = grid * kDecWarps;
  cfg.gridDim = dim3((unsigned)((pieces + kJoinWarps - 1) / kJoinWarps), (unsigned)(p.group < kRows ? p.group : kRows));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_join_kernel, p, pieces);
}

}  // namespace zq
