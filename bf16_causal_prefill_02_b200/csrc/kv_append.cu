// kv_append.cu -- new keys and values into a paged cache, as they are (bf16)
// or rounded to e4m3 with the cache's scales.
//
// A warp per share of a token: it finds the token's sequence (a 32-ary search of the
// sequence offsets), looks up the page its position falls in, and moves the
// share of the key and value rows, 16 bytes a lane at a time.  The rows are on
// their way from memory while the place is looked up.  Bound by memory: 2
// bytes read and 2 (bf16) or 1 (e4m3) written per element (15739 tokens of 8
// heads to e4m3, 97 MB: 19.1 us); a step of one token each is bound by the
// chain of loads (64 sequences: 2.6 us).
#include "paged.cuh"

namespace zq {

namespace {

constexpr int kAppendWarps = 8;

// The sequence whose tokens [cu[b], cu[b + 1]) hold t: the number of offsets
// cu[0..B] that are <= t, minus 1 (B or -1: no sequence holds it).  All lanes
// of the warp take part.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ cu, int B, int64_t t, int lane) {
  int lo = 0, n = B + 1;  // offsets lo .. lo + n - 1 are undecided; those before lo are <= t
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lo + min((lane + 1) * step, n) - 1;  // the last offset of this lane's piece
    const bool mine = lane * step < n;
    const unsigned le = __ballot_sync(0xffffffffu, mine && cu[at] <= t);
    const int full = __popc(le);  // pieces that lie wholly at or below t (offsets ascend)
    lo += min(full * step, n);
    n = min(step, n - min(full * step, n));
    if (step == 1) break;
    n = max(n - 1, 0);  // the last offset of the piece is above t
  }
  return lo - 1;
}

// 16 bytes (8 bf16) to 8 e4m3 codes: rne_satfinite(fl32(x * inv)).
__device__ __forceinline__ uint2 to_e4m3(uint4 x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16) * inv;
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
  }
  return make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
}

// A scale of 0 stands for a head whose values were all 0: its codes are 0.  The
// reciprocal of a scale below 2^-128 passes fp32's range; it is cut there, so
// that a value of 0 does not become NaN.
__device__ __forceinline__ float inverse_scale(const float* ds, int per_head, int h) {
  const float s = ds ? ds[per_head ? h : 0] : 1.0f;
  return s == 0.0f ? 0.0f : fminf(__frcp_rn(s), 3.40282347e+38f);
}

// Pieces of a key and of a value row that a lane has on their way before it
// knows their place; a warp's share of a token is 32 times as many of each.
// (1 / 2 / 4, e4m3: 8 heads 23.4 / 20.2 / 21.6 us, 32 heads 79 / 63 / 64 us.)
constexpr int kAhead = 2;

template <int FP8, int D>
__device__ __forceinline__ void store_piece(char* row, int x, uint4 w, const float* ds, int per_head) {
  if (FP8)
    reinterpret_cast<uint2*>(row)[x] = to_e4m3(w, inverse_scale(ds, per_head, x / (D / 8)));
  else
    reinterpret_cast<uint4*>(row)[x] = w;
}

template <int FP8, int DQK>
__global__ void __launch_bounds__(kAppendWarps * 32) kv_append_kernel(const AppendLaunch a) {
  constexpr int DV = 128;
  const int lane = threadIdx.x & 31;
  const int64_t share = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int64_t t = share / a.shares;
  launch_dependents();
  wait_previous_kernel();
  if (t >= a.T) return;
  const PagedKV& c = a.c;
  const int nk = c.Hkv * (DQK / 8), nv = c.Hkv * (DV / 8);  // pieces of 8 elements
  const int x0 = (int)(share % a.shares) * (32 * kAhead) + lane;
  const uint4* sk = reinterpret_cast<const uint4*>(a.k + t * a.k_stride);
  const uint4* sv = reinterpret_cast<const uint4*>(a.v + t * a.v_stride);
  uint4 wk[kAhead], wv[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    if (x0 + 32 * i < nk) wk[i] = __ldcs(sk + x0 + 32 * i);
    if (x0 + 32 * i < nv) wv[i] = __ldcs(sv + x0 + 32 * i);
  }
  int b = (int)t;
  int64_t i0 = 0;
  if (a.cu) {
    b = find_sequence(a.cu, c.B, t, lane);
    if (b < 0 || b >= c.B) return;  // not a token of any sequence
    i0 = t - a.cu[b];
  }
  const int have = c.seqlens[b];
  const int64_t pos = have + i0;
  const int64_t page_at = pos >> c.page_shift;
  // no room: the token is dropped (i0 < 0: the offsets do not ascend)
  if (have < 0 || i0 < 0 || page_at >= c.table_width) return;
  const int page = c.table[b * c.table_stride + page_at];
  if (page < 0 || page >= c.num_pages) return;
  const int64_t row = pos & ((1 << c.page_shift) - 1);
  constexpr int ES = FP8 ? 1 : 2;
  char* dk = c.k + page * c.k_page + row * c.Hkv * (DQK * ES);
  char* dv = c.v + page * c.v_page + row * c.Hkv * (DV * ES);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    if (x0 + 32 * i < nk) store_piece<FP8, DQK>(dk, x0 + 32 * i, wk[i], c.k_descale, c.descale_per_head);
    if (x0 + 32 * i < nv) store_piece<FP8, DV>(dv, x0 + 32 * i, wv[i], c.v_descale, c.descale_per_head);
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendLaunch& a0, cudaStream_t st) {
  AppendLaunch a = a0;
  if (a.T <= 0) return cudaSuccess;
  a.shares = (a.c.Hkv * (a.c.dqk / 8) + 32 * kAhead - 1) / (32 * kAhead);  // (d_qk >= d_v)
  const int64_t blocks = (a.T * a.shares + kAppendWarps - 1) / kAppendWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto kern = a.c.dtype == 1 ? (a.c.dqk == 128 ? kv_append_kernel<1, 128> : kv_append_kernel<1, 192>)
                             : (a.c.dqk == 128 ? kv_append_kernel<0, 128> : kv_append_kernel<0, 192>);
  return launch_overlapped(kern, dim3((unsigned)blocks), dim3(kAppendWarps * 32), 0, st, a);
}

}  // namespace zq
