// serving.h -- launch structures, and the host's choices of a schedule, of the
// packed-prompt and paged-cache operators (internal; not part of the public
// interface).  The fixed-batch kernels do not include it.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "schedule.h"

namespace zq {

// A launch whose blocks may become resident while the stream's previous kernel
// still runs.  The kernel calls griddepcontrol.wait before it touches memory,
// which returns once that kernel's writes are visible; nothing else changes in
// the stream's order.
template <class... P, class... A>
inline cudaError_t launch_overlapped_cluster(void (*kern)(P...), unsigned cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                             const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}
template <class... P, class... A>
inline cudaError_t launch_overlapped(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A&... args) {
  return launch_overlapped_cluster(kern, 1, grid, block, smem, st, args...);
}

// Attention over packed prompts.
struct VarlenParams {
  void* out;   // (Tq, Hq, d_v) bfloat16
  float* lse;  // (Hq, Tq) or nullptr
  const int32_t* cu_q;  // B + 1 row offsets
  const int32_t* cu_k;
  const float* q_descale;
  const float* k_descale;
  const float* v_descale;
  int* status;
  int descale_per_kv;  // entry b * Hkv + kv head, as in AttnParams
  int B, Tq, Tk, Hq, Hkv, group;
  int max_tiles;   // bound on the 128-row query tiles of all sequences
  int head_group;  // query heads whose units are interleaved; divides Hq
  int causal;
  int headroom_T;
  float scale_log2;  // softmax scale times log2(e)
  uint64_t timeout_ns;
  // Test hook, else 0: arrivals that the barriers of P expect and nobody makes,
  // so that the issuers wait for P until their limit and all others for them.
  // (A test in the issuers' loops cost the two-tile kernel 1 to 2%.)
  int withhold;
};
struct VarlenLaunch {
  const void* q;
  const void* k;
  const void* v;
  VarlenParams p;
  int dqk, dtype, mode, block_scale;
  bool pairs;  // two query tiles per CTA (BF16, d = 128)
};
cudaError_t launch_attention_varlen(const VarlenLaunch& a, cudaStream_t st);
cudaError_t launch_attention_varlen_pp(const VarlenLaunch& a, cudaStream_t st);

// A paged cache as the kernels address it: key c of sequence b is row
// c & (page_size - 1) of page block_table[b * table_stride + (c >> page_shift)].
// Strides in bytes.
struct PagedKV {
  char* k;
  char* v;
  int64_t k_page, v_page;
  const int32_t* table;
  const int32_t* seqlens;
  const float* k_descale;  // 1 or Hkv fp32, or nullptr (1.0)
  const float* v_descale;
  int64_t table_stride;
  int descale_per_head;
  int B, Hkv, num_pages, page_shift, table_width;
  int dqk, dv, dtype;
};
struct AppendLaunch {
  PagedKV c;
  const char* k;
  const char* v;
  int64_t k_stride, v_stride;  // bytes between tokens
  const int32_t* cu;           // B + 1 token offsets, or nullptr (token t is sequence t's)
  int64_t T;
  int shares;  // warps per token (set by the launcher)
};
cudaError_t launch_kv_append(const AppendLaunch& a, cudaStream_t st);
struct DecodeLaunch {
  PagedKV c;
  const void* q;
  int64_t q_stride;  // elements between sequences
  int Hq;
  float scale_log2;
  void* out;
  float* lse;
  void* workspace;
};
cudaError_t launch_decode(const DecodeLaunch& a, cudaStream_t st, int num_sms);
size_t decode_workspace_bytes();

// Packed prompts: a bound on the query tiles of `rows` rows, which the host
// knows without the offsets.
inline int varlen_tiles(int64_t Tq, int64_t B, int rows) {
  return Tq > 0 ? (int)((Tq + (rows - 1) * B) / rows) : 0;
}

// Packed prompts, BF16 at d = 128: two tiles per CTA (attn_varlen_pp.cu) where
// there are enough units to keep the SMs even, and sequences long enough to
// fill both tiles.  Measured against one tile per CTA (us, one / two):
//   units of 256 rows  192: 29.8 / 31.9   376: 252 / 257   416: 87 / 90
//   472: 44.4 / 46.7   512: 237 / 232     640: 197 / 190   1024: 469 / 449
//   41 sequences of 100 rows, 32 heads: 34.5 / 43.5.
inline bool use_varlen_pairs(int64_t Tq, int64_t B, int Hq, int num_sms) {
  return 3 * (int64_t)varlen_tiles(Tq, B, 2 * kTile) * Hq >= 10 * (int64_t)num_sms && Tq >= 2 * kTile * B;
}

// Packed prompts: heads whose units are interleaved.  All of them, which
// balances best, while the K and V of all heads are below 256 MB; else the
// query heads of as many kv heads as stay below.  (All heads against 4 at a
// time: 32/8 heads, 4096 rows bf16 137 against 163 us, FP8 112 against 151;
// MLA, 16 heads, 16384 rows and 168 MB of K and V 1418 against 1498 us.)
inline int choose_varlen_head_group(int Hq, int Hkv, int64_t Tk, int d_qk, int d_v, int elem_bytes) {
  const double one = (double)Tk * (d_qk + d_v) * elem_bytes;
  int kv = Hkv;
  while (kv > 1 && (Hkv % kv != 0 || kv * one > 256.0 * 1024 * 1024)) --kv;
  return Hq / Hkv * kv;
}

}  // namespace zq
