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
//     pairs form one line that is cut into equal pieces, one per CTA, so
//     ragged lengths cost no balance.  A piece that holds a whole (sequence,
//     head) writes the output; a cut one writes (m, l, O) to the workspace and
//     decode_join_kernel joins the parts: M = max m_j, l = sum l_j 2^(m_j - M),
//     o = sum O_j 2^(m_j - M) / l.  The order is fixed, so runs repeat bit for
//     bit.
//   * Inside a CTA every warp streams its own keys through its own ring of
//     cp.async stages (no block-wide barrier in the loop), with its own
//     running maximum and sum; the four warps are joined at a segment's end.
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
constexpr int kMaxCtas = 512;  // pieces the workspace has room for
constexpr int kCtasPerSm = 2;

struct DecodeParams {
  PagedKV c;
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* out;
  float* lse;
  float scale;
  int Hq, group, head_tiles;
  // workspace: who cuts what, then the parts
  int4* cut;     // [grid] {sequence, flat head tile, parts, 0} of the segment this CTA starts and does not finish
  float* part;   // [grid][2][kRows * dv + 2 * kRows]: slot 0 a segment begun by an earlier CTA, slot 1 one left to later CTAs
};

template <int DQK, int FP8>
struct DecGeo {
  static constexpr int DV = 128;
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int KW = FP8 ? 32 : 16;              // keys per warp and step
  static constexpr int TK = KW * kDecWarps;             // keys per tile of the line
  static constexpr int KCH = DQK * ES / 16;             // 16-byte pieces per key row
  static constexpr int VCH = DV * ES / 16;
  static constexpr int KBYTES = KW * KCH * 16;
  static constexpr int VBYTES = KW * VCH * 16;
  static constexpr int STAGE = KBYTES + VBYTES;
  static constexpr int NS = DQK == 128 ? 3 : 2;         // stages that fit 113 KB (two CTAs per SM)
  static constexpr int RING = NS * STAGE;               // bytes per warp
  static constexpr int JOIN = kRows * DV * 4;           // a warp's O at a segment's end, over its ring
  static constexpr int SMEM = kDecWarps * RING + kDecWarps * kRows * 8;
  static constexpr int QK_STEPS = DQK / 16;
  static_assert(RING >= JOIN, "O fits the ring");
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

template <int DQK, int FP8>
__global__ void __launch_bounds__(kDecThreads, kCtasPerSm) decode_kernel(const DecodeParams p) {
  using G = DecGeo<DQK, FP8>;
  constexpr int DV = G::DV, KW = G::KW, NS = G::NS;
  constexpr unsigned kFull = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan[kDecWarps + 1];
  __shared__ int64_t first_off;
  __shared__ int first_b;
  const PagedKV& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, ql = lane & 3;
  const int heads = c.Hkv * p.head_tiles;
  launch_dependents();

  // ---- this CTA's piece [x, x1) of the line: b outermost, then the flat head tile, then the key tile
  int64_t x, x1, line;
  int pieces;
  {
    const int per = (c.B + kDecThreads - 1) / kDecThreads;
    const int b0 = min((int)threadIdx.x * per, c.B), b1 = min(b0 + per, c.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += (keys_of(c, b) + G::TK - 1) / G::TK;
    mine *= heads;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) scan[warp] = sum;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    // no more pieces than tiles, so that none is empty
    pieces = (int)min((int64_t)gridDim.x, total);
    line = total;
    x = x1 = 0;
    if ((int)blockIdx.x < pieces) {
      x = total * blockIdx.x / pieces;
      x1 = total * (blockIdx.x + 1) / pieces;
    }
    int64_t at = before + sum - mine;  // line position of this thread's first sequence
    if (x < x1 && x >= at && x < at + mine) {
      int b = b0;
      for (;; ++b) {
        const int64_t n = (int64_t)((keys_of(c, b) + G::TK - 1) / G::TK) * heads;
        if (x < at + n) break;
        at += n;
      }
      first_b = b;
      first_off = x - at;
    }
    __syncthreads();
  }
  // sequences without keys: 0 and -inf
  for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
    if (keys_of(c, b) > 0) continue;
    for (int i = threadIdx.x; i < p.Hq * DV / 2; i += kDecThreads)
      reinterpret_cast<uint32_t*>(p.out + (int64_t)b * p.Hq * DV)[i] = 0u;
    if (p.lse)
      for (int i = threadIdx.x; i < p.Hq; i += kDecThreads) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
  }

  uint8_t* const ring = smem + warp * G::RING;
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  float2* const stats = reinterpret_cast<float2*>(smem + kDecWarps * G::RING);  // [warp][row] (m, l)
  bool cut = false;  // a segment of this piece is left to later CTAs

  int b = x < x1 ? first_b : 0;
  int64_t off = x < x1 ? first_off : 0;
  while (x < x1) {
    const int len = keys_of(c, b);
    const int tiles = (len + G::TK - 1) / G::TK;
    if (off >= (int64_t)tiles * heads) {
      off -= (int64_t)tiles * heads;
      ++b;
      continue;
    }
    const int fh = (int)(off / tiles), t0 = (int)(off % tiles);
    const int steps = (int)min((int64_t)(tiles - t0), x1 - x);
    const int g = fh / p.head_tiles, ht = fh % p.head_tiles;
    const int h0 = g * p.group + ht * kRows;          // first query head of the tile
    const int rows = min(kRows, p.group - ht * kRows);  // query heads in it

    // ---- queries as A fragments: rows quad and quad + 8
    uint32_t qa[G::QK_STEPS][4];
    const float c2 = p.scale * (FP8 && c.k_descale ? c.k_descale[c.descale_per_head ? g : 0] : 1.0f) * 1.4426950408889634f;
    float cr[2] = {c2, c2};
    {
      const __nv_bfloat16* qrow = p.q + b * p.q_stride + (int64_t)h0 * DQK;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
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

    // ---- the segment's keys: warp w takes keys [w KW, (w + 1) KW) of every tile
    const int32_t* table = c.table + b * c.table_stride;
    const int key0 = t0 * G::TK + warp * KW;
    const char* kbase = c.k + (int64_t)g * (DQK * G::ES);
    const char* vbase = c.v + (int64_t)g * (DV * G::ES);
    const int64_t krow = (int64_t)c.Hkv * (DQK * G::ES), vrow = (int64_t)c.Hkv * (DV * G::ES);
    const int page_mask = (1 << c.page_shift) - 1;
    // the page of key (step, lane), or -1: not there
    auto page_at = [&](int step) -> int {
      const int key = key0 + step * G::TK + lane;
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
      const int kb = key0 + step * G::TK;
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
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < KW / 8; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[n][i] *= cr[i >> 1];
            if (!((vm >> (n * 8 + 2 * ql + (i & 1))) & 1u)) sc[n][i] = -INFINITY;
            mx[i >> 1] = fmaxf(mx[i >> 1], sc[n][i]);
          }
        // the reference moves when a score passes it by 8 (weights stay below 2^8)
        if (__any_sync(kFull, mx[0] > ref[0] + 8.0f || mx[1] > ref[1] + 8.0f)) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float m = fmaxf(mx[hf], __shfl_xor_sync(kFull, mx[hf], 1));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
            const float nref = fmaxf(ref[hf], m);
            const float f = (nref == -INFINITY || nref == ref[hf]) ? 1.0f : ex2_approx(ref[hf] - nref);
            ref[hf] = nref;
            l[hf] *= f;
#pragma unroll
            for (int n = 0; n < DV / 8; ++n) {
              o[n][2 * hf] *= f;
              o[n][2 * hf + 1] *= f;
            }
          }
        }
        const float nb[2] = {ref[0] == -INFINITY ? 0.0f : ref[0], ref[1] == -INFINITY ? 0.0f : ref[1]};
        uint32_t pa[KW / 16][4];
#pragma unroll
        for (int n = 0; n < KW / 8; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[n][i] = ex2_approx(sc[n][i] - nb[i >> 1]);
            l[i >> 1] += sc[n][i];
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            pa[n / 2][(n & 1) * 2 + hf] = FP8 ? pack_f16x2(sc[n][2 * hf], sc[n][2 * hf + 1]) : pack_bf16x2(sc[n][2 * hf], sc[n][2 * hf + 1]);
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

    // ---- join the warps: every warp's O (and m, l) through its own ring
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      l[hf] += __shfl_xor_sync(kFull, l[hf], 1);
      l[hf] += __shfl_xor_sync(kFull, l[hf], 2);
      const int r = quad + hf * 8;
      if (r < rows) {
        if (ql == 0) stats[warp * kRows + r] = make_float2(ref[hf], l[hf]);
        float* dst = reinterpret_cast<float*>(ring) + r * DV;
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
      }
    }
    __syncthreads();
    const bool begins = t0 == 0, ends = t0 + steps == tiles;
    const float vds = FP8 && c.v_descale ? c.v_descale[c.descale_per_head ? g : 0] : 1.0f;
    float* slot = p.part + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * (kRows * DV + 2 * kRows);
    for (int r = 0; r < rows; ++r) {
      float2 st[kDecWarps];
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        st[w] = stats[w * kRows + r];
        m = fmaxf(m, st[w].x);
      }
      const float mb = m == -INFINITY ? 0.0f : m;
      float acc = 0.0f, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float f = ex2_approx(st[w].x - mb);
        sum += st[w].y * f;
        acc += reinterpret_cast<const float*>(smem + w * G::RING)[r * DV + threadIdx.x] * f;
      }
      if (begins && ends) {
        const int64_t row = (int64_t)b * p.Hq + h0 + r;
        // no key was there (l = 0): 0 and -inf; NaN stays NaN
        const bool empty = sum == 0.0f;
        p.out[row * DV + threadIdx.x] = __float2bfloat16(empty ? 0.0f : acc * (vds / sum));
        if (p.lse && threadIdx.x == 0) p.lse[row] = empty ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
      } else {
        slot[r * DV + threadIdx.x] = acc;
        if (threadIdx.x == 0) {
          slot[kRows * DV + 2 * r] = m;
          slot[kRows * DV + 2 * r + 1] = sum;
        }
      }
    }
    if (begins && !ends) {
      cut = true;
      if (threadIdx.x == 0) {
        // its parts: this CTA's and those up to the one that holds its last tile
        const int64_t last = x + tiles - 1;
        // the CTA of position y: the largest j with floor(line * j / pieces) <= y
        const int64_t j = ((last + 1) * pieces - 1) / line;
        p.cut[blockIdx.x] = make_int4(b, fh, (int)(j - blockIdx.x) + 1, 0);
      }
    }
    __syncthreads();  // the rings may be filled again
    x += steps;
    off += steps;
  }
  if (!cut && threadIdx.x == 0) p.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
}

// Joins the parts of the (sequence, head tile) that CTA blockIdx.x began and
// did not finish; blockIdx.y is the query head in it.  Warp w takes parts w,
// w + 4, ...; a lane holds four channels.
__global__ void __launch_bounds__(kDecThreads) decode_join_kernel(const DecodeParams p) {
  constexpr int DV = 128;
  constexpr int SLOT = kRows * DV + 2 * kRows;
  __shared__ float4 acc_s[kDecWarps][32];
  __shared__ float2 stat_s[kDecWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y;
  wait_previous_kernel();
  const int4 d = p.cut[blockIdx.x];
  if (d.z == 0) return;
  const int b = d.x, g = d.y / p.head_tiles, ht = d.y % p.head_tiles;
  if (r >= min(kRows, p.group - ht * kRows)) return;
  auto slot = [&](int j) {  // part j: the beginning is in slot 1 of this CTA, the rest in slot 0 of those after it
    return p.part + ((int64_t)(blockIdx.x + j) * 2 + (j == 0 ? 1 : 0)) * SLOT;
  };
  float m = -INFINITY, l = 0.0f;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j = warp; j < d.z; j += kDecWarps) {
    const float* s = slot(j);
    const float2 st = *reinterpret_cast<const float2*>(s + kRows * DV + 2 * r);
    const float4 v = reinterpret_cast<const float4*>(s + r * DV)[lane];
    const float nm = fmaxf(m, st.x), nb = nm == -INFINITY ? 0.0f : nm;
    const float fa = ex2_approx(m - nb), fb = ex2_approx(st.x - nb);
    l = l * fa + st.y * fb;
    a.x = a.x * fa + v.x * fb;
    a.y = a.y * fa + v.y * fb;
    a.z = a.z * fa + v.z * fb;
    a.w = a.w * fa + v.w * fb;
    m = nm;
  }
  acc_s[warp][lane] = a;
  if (lane == 0) stat_s[warp] = make_float2(m, l);
  __syncthreads();
  if (warp != 0) return;
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, stat_s[w].x);
  const float mb = M == -INFINITY ? 0.0f : M;
  float L = 0.0f;
  a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    const float f = ex2_approx(stat_s[w].x - mb);
    const float4 v = acc_s[w][lane];
    L += stat_s[w].y * f;
    a.x += v.x * f;
    a.y += v.y * f;
    a.z += v.z * f;
    a.w += v.w * f;
  }
  const bool empty = L == 0.0f;
  const float vds = p.c.dtype == 1 && p.c.v_descale ? p.c.v_descale[p.c.descale_per_head ? g : 0] : 1.0f;
  const float inv = empty ? 0.0f : vds / L;
  const int64_t row = (int64_t)b * p.Hq + g * p.group + ht * kRows + r;
  uint2 w2 = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  if (empty) w2 = make_uint2(0u, 0u);
  reinterpret_cast<uint2*>(p.out + row * DV)[lane] = w2;
  if (p.lse && lane == 0) p.lse[row] = empty ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <int DQK, int FP8>
cudaError_t launch_variant(DecodeParams& p, cudaStream_t st, int grid) {
  using G = DecGeo<DQK, FP8>;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<DQK, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  decode_kernel<DQK, FP8><<<grid, kDecThreads, G::SMEM, st>>>(p);
  return cudaGetLastError();
}

constexpr size_t kCutBytes = (size_t)kMaxCtas * 16;

}  // namespace

size_t decode_workspace_bytes() { return kCutBytes + (size_t)kMaxCtas * 2 * (kRows * 128 + 2 * kRows) * 4; }

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
  cfg.gridDim = dim3((unsigned)grid, (unsigned)(p.group < kRows ? p.group : kRows));
  cfg.blockDim = dim3(kDecThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_join_kernel, p);
}

}  // namespace zq
