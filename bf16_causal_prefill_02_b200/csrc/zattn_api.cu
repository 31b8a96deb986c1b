// zattn_api.cu -- the C ABI declared in include/zattn.h: argument
// validation, device checks and kernel launches.  No allocation, no
// synchronisation, no state kept between calls.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "zattn.h"

#include "schedule.h"
#include "serving.h"
#include "zq_internal.h"

namespace {

constexpr int kVersion = 200;  // 0.2.0
constexpr uint64_t kTimeoutNs = 2000000000ull;  // bound on any single device-side wait
constexpr uint64_t kDebugTimeoutNs = 100000000ull;  // the same in a packed call that is made to give up
constexpr int64_t kMaxGroupedSlots = 65535;      // grouped quantiser: slots are grid.y

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Current device must be sm_100 (B200 class).  Returns the SM count through
// `num_sms` when non-null.
int check_device(int* num_sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZQ_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return ZQ_ERR_CUDA;
  if (major != 10 || minor != 0) return ZQ_ERR_ARCH;
  if (num_sms &&
      cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return ZQ_ERR_CUDA;
  return ZQ_OK;
}

// Head dims, element type, FP8 options and scale, which zq_attn_args and
// zq_varlen_args name alike.
template <class Args>
int validate_options(const Args* a) {
  if (!((a->d_qk == 128 && a->d_v == 128) || (a->d_qk == 192 && a->d_v == 128)))
    return ZQ_ERR_UNSUPPORTED;
  if (a->dtype != ZQ_DTYPE_BF16 && a->dtype != ZQ_DTYPE_FP8_E4M3) return ZQ_ERR_UNSUPPORTED;
  if (a->dtype == ZQ_DTYPE_FP8_E4M3) {
    if (a->softmax_mode != ZQ_SOFTMAX_EXACT && a->softmax_mode != ZQ_SOFTMAX_LEANP)
      return ZQ_ERR_UNSUPPORTED;
    if (a->block_scale != 0 && a->block_scale != 1) return ZQ_ERR_UNSUPPORTED;
    if (a->headroom_T < 0 || a->headroom_T > 8) return ZQ_ERR_UNSUPPORTED;
    if (a->descale_layout != ZQ_DESCALE_PER_TENSOR && a->descale_layout != ZQ_DESCALE_PER_KV_HEAD)
      return ZQ_ERR_UNSUPPORTED;
  }
  if (!(std::isfinite(a->softmax_scale))) return ZQ_ERR_SHAPE;
  return ZQ_OK;
}

int validate_attn(const zq_attn_args* a) {
  if (!a) return ZQ_ERR_NULL;
  if (!a->q || !a->k || !a->v || !a->out) return ZQ_ERR_NULL;
  if (a->B <= 0 || a->Sq <= 0 || a->Sk <= 0 || a->Hq <= 0 || a->Hkv <= 0) return ZQ_ERR_SHAPE;
  if (a->Hq % a->Hkv != 0) return ZQ_ERR_SHAPE;
  const int rc = validate_options(a);
  if (rc != ZQ_OK) return rc;
  // units = n_qtiles * B * Hq stay in int range, with room above the last
  // unit for the persistent CTAs' zigzag walk (it computes indices up to
  // two rounds of CTAs past the last unit); TMA element counts and strides
  const int64_t ntiles = (a->Sq + 127) / 128;
  if (ntiles * a->B * (int64_t)a->Hq > 0x7FFF0000ll) return ZQ_ERR_SHAPE;
  const int es = a->dtype == ZQ_DTYPE_BF16 ? 2 : 1;
  const int64_t qbytes = (int64_t)a->B * a->Sq * a->Hq * a->d_qk * es;
  const int64_t kbytes = (int64_t)a->B * a->Sk * a->Hkv * a->d_qk * es;
  if (qbytes >= (1ll << 40) || kbytes >= (1ll << 40)) return ZQ_ERR_SHAPE;
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->out) ||
      (a->lse && !aligned16(a->lse)))
    return ZQ_ERR_ALIGN;
  return ZQ_OK;
}

// The score scale in the log2 domain (softmax_scale <= 0: 1/sqrt(d_qk)), rounded once.
float scale_log2(float softmax_scale, int d_qk) {
  return (float)((softmax_scale > 0.0f ? (double)softmax_scale : 1.0 / std::sqrt((double)d_qk)) * 1.4426950408889634);
}

}  // namespace

extern "C" {

int zq_version(void) { return kVersion; }

const char* zq_status_string(int s) {
  switch (s) {
    case ZQ_OK: return "ok";
    case ZQ_ERR_NULL: return "a required pointer is NULL";
    case ZQ_ERR_SHAPE: return "invalid shape (size <= 0, Hq % Hkv != 0 or too large)";
    case ZQ_ERR_UNSUPPORTED: return "unsupported head dims, dtype, mode or option";
    case ZQ_ERR_ALIGN: return "pointer not aligned (16 bytes; 4 for tables, lengths, offsets and scales)";
    case ZQ_ERR_ARCH: return "current device is not sm_100 (B200)";
    case ZQ_ERR_CUDA: return "CUDA call failed";
    case ZQ_ERR_TIMEOUT: return "a device-side wait timed out";
    default: return "unknown status";
  }
}

// Launch description of a validated call (no device access).
static zq::AttnLaunch make_launch(const zq_attn_args* a) {
  zq::AttnLaunch L;
  L.q = a->q;
  L.k = a->k;
  L.v = a->v;
  L.dqk = a->d_qk;
  L.dv = a->d_v;
  L.dtype = a->dtype;
  L.mode = a->softmax_mode;
  L.block_scale = a->block_scale;
  L.p.out = a->out;
  L.p.lse = a->lse;
  L.p.q_descale = a->q_descale;
  L.p.k_descale = a->k_descale;
  L.p.v_descale = a->v_descale;
  L.p.descale_per_kv =
      a->dtype == ZQ_DTYPE_FP8_E4M3 && a->descale_layout == ZQ_DESCALE_PER_KV_HEAD ? 1 : 0;
  L.p.status = a->status;
  L.p.B = a->B;
  L.p.Sq = a->Sq;
  L.p.Sk = a->Sk;
  L.p.Hq = a->Hq;
  L.p.Hkv = a->Hkv;
  L.p.n_qtiles = (a->Sq + zq::kTile - 1) / zq::kTile;
  L.p.head_group = zq::choose_head_group(a->B, a->Hq, a->Hkv, a->Sq, a->Sk, a->d_qk, a->d_v,
                                         a->dtype == ZQ_DTYPE_FP8_E4M3 ? 1 : 2);
  L.p.causal = a->causal ? 1 : 0;
  L.p.headroom_T = a->dtype == ZQ_DTYPE_FP8_E4M3 ? a->headroom_T : 8;
  L.p.softmax_scale =
      a->softmax_scale > 0.0f ? a->softmax_scale : (float)(1.0 / std::sqrt((double)a->d_qk));
  L.p.timeout_ns = kTimeoutNs;
  L.p.dbg = nullptr;
  L.p.dbg_bh = 0;
  L.p.dbg_t = 0;
  L.p.dbg_flags = 0;
  return L;
}

static int attn_impl(const zq_attn_args* a, void* dbg, int dbg_bh, int dbg_t, int dbg_flags,
                     void* stream) {
  int rc = validate_attn(a);
  if (rc != ZQ_OK) return rc;
  rc = check_device(nullptr);
  if (rc != ZQ_OK) return rc;
  zq::AttnLaunch L = make_launch(a);
  L.p.dbg = dbg;
  L.p.dbg_bh = dbg_bh;
  L.p.dbg_t = dbg_t;
  L.p.dbg_flags = dbg_flags;
  cudaError_t e = zq::launch_attention(L, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

int zq_attn_fwd_ex(const zq_attn_args* a, void* stream) {
  return attn_impl(a, nullptr, 0, 0, 0, stream);
}

int zq_attn_plan_launch(const zq_attn_args* a, int num_sms, zq_attn_plan* plan,
                        int32_t* unit_tile, int32_t* unit_bh, int32_t* unit_nkv,
                        int32_t* unit_cta, int32_t* unit_round) {
  if (!plan) return ZQ_ERR_NULL;
  int rc = validate_attn(a);
  if (rc != ZQ_OK) return rc;
  if (num_sms <= 0) {
    rc = check_device(&num_sms);
    if (rc != ZQ_OK) return rc;
  }
  const zq::AttnLaunch L = make_launch(a);
  const zq::AttnParams& p = L.p;
  // the kernel launch_attention picks: pairs of query tiles with 64-key
  // tiles (BF16, d = 128, more than 64 query tiles), else single query
  // tiles with 128-key tiles
  const bool pair = zq::use_pair_kernel(L.dtype, L.dqk, p.n_qtiles);
  const long long n_units = (long long)(pair ? zq::n_pairs_of(p.n_qtiles) : p.n_qtiles) * p.B * p.Hq;
  const long long grid = zq::grid_size(p.n_qtiles, n_units, num_sms);
  plan->n_units = n_units;
  plan->grid = grid;
  plan->persistent = zq::use_persistent(p.n_qtiles) ? 1 : 0;
  plan->head_group = p.head_group;
  plan->smem_bytes = pair ? zq::attn_pp_smem_bytes() : zq::attn_smem_bytes(a->dtype, a->d_qk);
  plan->threads = pair ? zq::attn_pp_threads() : zq::attn_threads();
  plan->rows_per_unit = pair ? 2 * zq::kTile : zq::kTile;
  plan->keys_per_tile = pair ? zq::kPairKeyTile : zq::kTile;
  if (!unit_tile && !unit_bh && !unit_nkv && !unit_cta && !unit_round) return ZQ_OK;
  for (long long u = 0; u < n_units; ++u) {
    int t, bh, nkv;
    if (pair) {
      const zq::PairUnit w = zq::pair_of(p, (int)u);
      t = w.tp, bh = w.bh, nkv = w.n_kv_max;
    } else {
      const zq::Unit w = zq::unit_of(p, (int)u);
      t = w.t, bh = w.bh, nkv = w.n_kv;
    }
    if (unit_tile) unit_tile[u] = t;
    if (unit_bh) unit_bh[u] = bh;
    if (unit_nkv) unit_nkv[u] = nkv;
  }
  if (unit_cta || unit_round) {
    // walk every CTA's sequence exactly as the kernel does
    for (long long c = 0; c < grid; ++c) {
      for (int k = 0;; ++k) {
        const long long u = zq::unit_at(k, (int)grid, (int)c);
        if (u >= n_units || (k > 0 && !plan->persistent)) break;
        if (unit_cta) unit_cta[u] = (int32_t)c;
        if (unit_round) unit_round[u] = k;
      }
    }
  }
  return ZQ_OK;
}

int zq_attn_fwd_debug(const zq_attn_args* a, void* dbg, int dbg_bh, int dbg_qtile, int flags,
                      void* stream) {
  if (!dbg) return ZQ_ERR_NULL;
  if (flags & ~1) return ZQ_ERR_UNSUPPORTED;
  return attn_impl(a, dbg, dbg_bh, dbg_qtile, flags, stream);
}

int zq_attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B,
                int Sq, int Sk, int Hq, int Hkv, int d_qk, int d_v, float softmax_scale,
                int causal, int dtype, const float* q_descale, const float* k_descale,
                const float* v_descale, void* stream) {
  zq_attn_args a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.B = B;
  a.Sq = Sq;
  a.Sk = Sk;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d_qk = d_qk;
  a.d_v = d_v;
  a.softmax_scale = softmax_scale;
  a.causal = causal;
  a.dtype = dtype;
  a.q_descale = q_descale;
  a.k_descale = k_descale;
  a.v_descale = v_descale;
  a.softmax_mode = ZQ_SOFTMAX_LEANP;
  a.block_scale = 1;
  a.headroom_T = 8;
  a.status = nullptr;
  a.descale_layout = ZQ_DESCALE_PER_TENSOR;
  return zq_attn_fwd_ex(&a, stream);
}

size_t zq_quantize_workspace_bytes(void) { return 256; }

int zq_quantize_fp8(const void* x, int x_dtype, int64_t n_vec, int d, int hadamard,
                    void* x_fp8, float* descale, void* workspace, void* stream) {
  if (!descale || !workspace) return ZQ_ERR_NULL;
  if (n_vec < 0 || d <= 0) return ZQ_ERR_SHAPE;
  if (n_vec > 0 && (!x || !x_fp8)) return ZQ_ERR_NULL;
  if (x_dtype != ZQ_X_F32 && x_dtype != ZQ_X_BF16) return ZQ_ERR_UNSUPPORTED;
  if (d % 8 != 0 || (hadamard && d % 128 != 0 && d != 192)) return ZQ_ERR_UNSUPPORTED;
  if (n_vec > (int64_t)1 << 40 || n_vec * (int64_t)d > ((int64_t)1 << 40)) return ZQ_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(x_fp8) || !aligned16(workspace)) return ZQ_ERR_ALIGN;
  int sms = 0;
  int rc = check_device(&sms);
  if (rc != ZQ_OK) return rc;
  cudaError_t e = zq::launch_quantize(x, x_dtype == ZQ_X_BF16, n_vec * (int64_t)d,
                                      hadamard ? (d % 128 == 0 ? 1 : 2) : 0, x_fp8, descale, workspace,
                                      static_cast<cudaStream_t>(stream), sms);
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

size_t zq_quantize_multi_workspace_bytes(void) { return 256; }

int zq_quantize_fp8_multi(const zq_quant_tensor* t, int count, void* workspace, void* stream) {
  if (!t || !workspace) return ZQ_ERR_NULL;
  if (count < 1 || count > zq::kMaxQuantItems) return ZQ_ERR_SHAPE;
  zq::QuantItems Q = {};
  for (int i = 0; i < count; ++i) {
    const zq_quant_tensor& a = t[i];
    if (!a.descale) return ZQ_ERR_NULL;
    if (a.n_vec < 0 || a.d <= 0) return ZQ_ERR_SHAPE;
    if (a.n_vec > 0 && (!a.x || !a.x_fp8)) return ZQ_ERR_NULL;
    if (a.x_dtype != ZQ_X_F32 && a.x_dtype != ZQ_X_BF16) return ZQ_ERR_UNSUPPORTED;
    if (a.d % 8 != 0 || (a.hadamard && a.d % 128 != 0 && a.d != 192)) return ZQ_ERR_UNSUPPORTED;
    if (a.n_vec > (int64_t)1 << 40 || a.n_vec * (int64_t)a.d > ((int64_t)1 << 40)) return ZQ_ERR_SHAPE;
    if (!aligned16(a.x) || !aligned16(a.x_fp8)) return ZQ_ERR_ALIGN;
    Q.it[i].x = a.x;
    Q.it[i].out = static_cast<uint8_t*>(a.x_fp8);
    Q.it[i].descale = a.descale;
    Q.it[i].n = a.n_vec * (int64_t)a.d;
    Q.it[i].bf16 = a.x_dtype == ZQ_X_BF16 ? 1 : 0;
    Q.it[i].had = a.hadamard ? (a.d % 128 == 0 ? 1 : 2) : 0;
  }
  if (!aligned16(workspace)) return ZQ_ERR_ALIGN;
  int sms = 0;
  int rc = check_device(&sms);
  if (rc != ZQ_OK) return rc;
  cudaError_t e = zq::launch_quantize_multi(Q, count, workspace, static_cast<cudaStream_t>(stream), sms);
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

int zq_quantize_fp8_noalloc(const void* x, int x_dtype, int64_t n_vec, int d, int hadamard,
                            void* x_fp8, float* descale, void* stream) {
  if (!descale) return ZQ_ERR_NULL;
  if (n_vec < 0 || d <= 0) return ZQ_ERR_SHAPE;
  if (n_vec > 0 && (!x || !x_fp8)) return ZQ_ERR_NULL;
  if (x_dtype != ZQ_X_F32 && x_dtype != ZQ_X_BF16) return ZQ_ERR_UNSUPPORTED;
  if (d % 8 != 0 || (hadamard && d % 128 != 0 && d != 192)) return ZQ_ERR_UNSUPPORTED;
  if (n_vec > (int64_t)1 << 40 || n_vec * (int64_t)d > ((int64_t)1 << 40)) return ZQ_ERR_SHAPE;
  // the scratch this call needs must fit the fixed device array
  if (zq_quantize_workspace_bytes() > zq::noalloc_scratch_capacity()) return ZQ_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(x_fp8)) return ZQ_ERR_ALIGN;
  int sms = 0;
  int rc = check_device(&sms);
  if (rc != ZQ_OK) return rc;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZQ_ERR_CUDA;
  void* scratch = zq::noalloc_scratch_for_device(dev);
  if (!scratch) return ZQ_ERR_CUDA;
  cudaError_t e = zq::launch_quantize(x, x_dtype == ZQ_X_BF16, n_vec * (int64_t)d,
                                      hadamard ? (d % 128 == 0 ? 1 : 2) : 0, x_fp8, descale, scratch,
                                      static_cast<cudaStream_t>(stream), sms);
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

size_t zq_quantize_noalloc_scratch_bytes(void) { return zq::noalloc_scratch_capacity(); }

size_t zq_quantize_grouped_workspace_bytes(int B, int H, int heads_per_scale) {
  if (B <= 0 || H <= 0 || heads_per_scale <= 0 || H % heads_per_scale != 0) return 0;
  const int64_t slots = (int64_t)B * (H / heads_per_scale);
  if (slots > kMaxGroupedSlots) return 0;
  return (size_t)((slots * 4 + 15) / 16 * 16);
}

int zq_quantize_fp8_grouped(const void* x, int x_dtype, int B, int64_t S, int H, int d,
                            int heads_per_scale, int hadamard, void* x_fp8, float* descale,
                            void* workspace, void* stream) {
  if (!descale || !workspace) return ZQ_ERR_NULL;
  if (B <= 0 || H <= 0 || S < 0 || d <= 0 || heads_per_scale <= 0) return ZQ_ERR_SHAPE;
  if (H % heads_per_scale != 0) return ZQ_ERR_SHAPE;
  if ((int64_t)B * (H / heads_per_scale) > kMaxGroupedSlots) return ZQ_ERR_SHAPE;
  if (S > 0 && (!x || !x_fp8)) return ZQ_ERR_NULL;
  if (x_dtype != ZQ_X_F32 && x_dtype != ZQ_X_BF16) return ZQ_ERR_UNSUPPORTED;
  if (d % 8 != 0 || (hadamard && d % 128 != 0 && d != 192)) return ZQ_ERR_UNSUPPORTED;
  if (S > ((int64_t)1 << 40) || (int64_t)H * d > ((int64_t)1 << 24) ||
      (int64_t)B * S > ((int64_t)1 << 40) / ((int64_t)H * d))
    return ZQ_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(x_fp8) || !aligned16(workspace)) return ZQ_ERR_ALIGN;
  int sms = 0;
  int rc = check_device(&sms);
  if (rc != ZQ_OK) return rc;
  cudaError_t e = zq::launch_quantize_grouped(
      x, x_dtype == ZQ_X_BF16, B, S, H, d, heads_per_scale,
      hadamard ? (d % 128 == 0 ? 1 : 2) : 0, x_fp8, descale, workspace,
      static_cast<cudaStream_t>(stream), sms);
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

static int varlen_impl(const zq_varlen_args* a, int flags, void* stream) {
  if (!a) return ZQ_ERR_NULL;
  if (!a->cu_seqlens_q || !a->cu_seqlens_k) return ZQ_ERR_NULL;
  if (a->B <= 0 || a->B > 65535 || a->total_q < 0 || a->total_k < 0 || a->Hq <= 0 || a->Hkv <= 0 || a->Hq > 4096)
    return ZQ_ERR_SHAPE;
  if ((a->total_q > 0 && (!a->q || !a->out)) || (a->total_k > 0 && (!a->k || !a->v))) return ZQ_ERR_NULL;
  if (a->Hq % a->Hkv != 0) return ZQ_ERR_SHAPE;
  int rc = validate_options(a);
  if (rc != ZQ_OK) return rc;
  // the grid (a bound on the query tiles, times Hq) stays in 31 bits
  const int64_t max_tiles = zq::varlen_tiles(a->total_q, a->B, zq::kTile);
  if (max_tiles * a->Hq > 0x7FFF0000ll) return ZQ_ERR_SHAPE;
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->out) || !aligned16(a->lse)) return ZQ_ERR_ALIGN;
  if (!aligned4(a->cu_seqlens_q) || !aligned4(a->cu_seqlens_k) || !aligned4(a->status)) return ZQ_ERR_ALIGN;
  if (a->dtype == ZQ_DTYPE_FP8_E4M3 && (!aligned4(a->q_descale) || !aligned4(a->k_descale) || !aligned4(a->v_descale))) return ZQ_ERR_ALIGN;
  int sms = 0;
  rc = check_device(&sms);
  if (rc != ZQ_OK) return rc;
  zq::VarlenLaunch L;
  L.q = a->q;
  // without any key the tensor maps of k and v are never loaded from
  L.k = a->total_k > 0 ? a->k : a->q;
  L.v = a->total_k > 0 ? a->v : a->q;
  L.dqk = a->d_qk;
  L.dtype = a->dtype;
  L.mode = a->softmax_mode;
  L.block_scale = a->block_scale;
  L.pairs = a->dtype == ZQ_DTYPE_BF16 && a->d_qk == 128 && zq::use_varlen_pairs(a->total_q, a->B, a->Hq, sms);
  const bool fp8 = a->dtype == ZQ_DTYPE_FP8_E4M3;
  zq::VarlenParams& p = L.p;
  p.out = a->out;
  p.lse = a->lse;
  p.cu_q = a->cu_seqlens_q;
  p.cu_k = a->cu_seqlens_k;
  p.q_descale = a->q_descale;
  p.k_descale = a->k_descale;
  p.v_descale = a->v_descale;
  p.status = a->status;
  p.descale_per_kv = fp8 && a->descale_layout == ZQ_DESCALE_PER_KV_HEAD ? 1 : 0;
  p.B = a->B;
  p.Tq = a->total_q;
  p.Tk = a->total_k;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.group = a->Hq / a->Hkv;
  p.max_tiles = (int)max_tiles;
  p.head_group = zq::choose_varlen_head_group(a->Hq, a->Hkv, a->total_k, a->d_qk, a->d_v, fp8 ? 1 : 2);
  p.causal = a->causal ? 1 : 0;
  p.headroom_T = fp8 ? a->headroom_T : 8;
  p.scale_log2 = scale_log2(a->softmax_scale, a->d_qk);
  p.timeout_ns = flags ? kDebugTimeoutNs : kTimeoutNs;
  p.withhold = flags;
  cudaError_t e = zq::launch_attention_varlen(L, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

int zq_attn_varlen_fwd(const zq_varlen_args* a, void* stream) { return varlen_impl(a, 0, stream); }

int zq_attn_varlen_debug(const zq_varlen_args* a, int flags, void* stream) {
  if (flags & ~1) return ZQ_ERR_UNSUPPORTED;
  return varlen_impl(a, flags, stream);
}

// The cache as the kernels address it, after validation.
static int paged_cache(const zq_paged_kv* a, zq::PagedKV* c) {
  if (!a) return ZQ_ERR_NULL;
  if (!a->k_cache || !a->v_cache || !a->block_table || !a->cache_seqlens) return ZQ_ERR_NULL;
  if (a->B <= 0 || a->Hkv <= 0 || a->num_pages <= 0 || a->table_width <= 0) return ZQ_ERR_SHAPE;
  if (a->page_size <= 0 || a->page_size > 65536 || (a->page_size & (a->page_size - 1)) != 0) return ZQ_ERR_SHAPE;
  if (!((a->d_qk == 128 && a->d_v == 128) || (a->d_qk == 192 && a->d_v == 128))) return ZQ_ERR_UNSUPPORTED;
  if (a->dtype != ZQ_DTYPE_BF16 && a->dtype != ZQ_DTYPE_FP8_E4M3) return ZQ_ERR_UNSUPPORTED;
  if (a->descale_per_head != 0 && a->descale_per_head != 1) return ZQ_ERR_UNSUPPORTED;
  if ((int64_t)a->table_width * a->page_size > ((int64_t)1 << 30) || a->Hkv > 4096 || a->B > 65535) return ZQ_ERR_SHAPE;
  if (a->table_stride != 0 && (a->table_stride < a->table_width || a->table_stride > ((int64_t)1 << 40))) return ZQ_ERR_SHAPE;
  const int es = a->dtype == ZQ_DTYPE_BF16 ? 2 : 1;
  const int64_t kp = (int64_t)a->page_size * a->Hkv * a->d_qk, vp = (int64_t)a->page_size * a->Hkv * a->d_v;
  const int64_t ks = a->k_page_stride ? a->k_page_stride : kp, vs = a->v_page_stride ? a->v_page_stride : vp;
  if (ks < kp || vs < vp || ks > ((int64_t)1 << 40) || vs > ((int64_t)1 << 40)) return ZQ_ERR_SHAPE;
  if (!aligned16(a->k_cache) || !aligned16(a->v_cache) || (ks * es) % 16 != 0 || (vs * es) % 16 != 0) return ZQ_ERR_ALIGN;
  if (!aligned4(a->block_table) || !aligned4(a->cache_seqlens)) return ZQ_ERR_ALIGN;
  if (a->dtype == ZQ_DTYPE_FP8_E4M3 && (!aligned4(a->k_descale) || !aligned4(a->v_descale))) return ZQ_ERR_ALIGN;
  c->k = static_cast<char*>(a->k_cache);
  c->v = static_cast<char*>(a->v_cache);
  c->k_page = ks * es;
  c->v_page = vs * es;
  c->table = a->block_table;
  c->seqlens = a->cache_seqlens;
  c->k_descale = a->dtype == ZQ_DTYPE_FP8_E4M3 ? a->k_descale : nullptr;
  c->v_descale = a->dtype == ZQ_DTYPE_FP8_E4M3 ? a->v_descale : nullptr;
  c->table_stride = a->table_stride ? a->table_stride : a->table_width;
  c->descale_per_head = a->descale_per_head;
  c->B = a->B;
  c->Hkv = a->Hkv;
  c->num_pages = a->num_pages;
  c->page_shift = 0;
  while ((1 << c->page_shift) < a->page_size) ++c->page_shift;
  c->table_width = a->table_width;
  c->dqk = a->d_qk;
  c->dv = a->d_v;
  c->dtype = a->dtype;
  return ZQ_OK;
}

int zq_kv_append(const zq_paged_kv* cache, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                 const int32_t* cu_seqlens, int64_t T, void* stream) {
  zq::AppendLaunch L;
  int rc = paged_cache(cache, &L.c);
  if (rc != ZQ_OK) return rc;
  if (T < 0 || T > 0x7fffffffLL || (!cu_seqlens && T != cache->B)) return ZQ_ERR_SHAPE;
  if (T > 0 && (!k || !v)) return ZQ_ERR_NULL;
  const int64_t kr = (int64_t)cache->Hkv * cache->d_qk, vr = (int64_t)cache->Hkv * cache->d_v;
  const int64_t ks = k_stride ? k_stride : kr, vs = v_stride ? v_stride : vr;
  if (ks < kr || vs < vr || ks > ((int64_t)1 << 31) || vs > ((int64_t)1 << 31)) return ZQ_ERR_SHAPE;
  if (!aligned16(k) || !aligned16(v) || !aligned4(cu_seqlens) || ks % 8 != 0 || vs % 8 != 0) return ZQ_ERR_ALIGN;
  rc = check_device(nullptr);
  if (rc != ZQ_OK) return rc;
  L.k = static_cast<const char*>(k);
  L.v = static_cast<const char*>(v);
  L.k_stride = ks * 2;
  L.v_stride = vs * 2;
  L.cu = cu_seqlens;
  L.T = T;
  cudaError_t e = zq::launch_kv_append(L, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

size_t zq_decode_workspace_bytes(void) { return zq::decode_workspace_bytes(); }

int zq_attn_decode(const zq_paged_kv* cache, const void* q, int64_t q_stride, int Hq, float softmax_scale,
                   void* out, float* lse, void* workspace, void* stream) {
  zq::DecodeLaunch L;
  int rc = paged_cache(cache, &L.c);
  if (rc != ZQ_OK) return rc;
  if (!q || !out || !workspace) return ZQ_ERR_NULL;
  if (Hq <= 0 || Hq > 4096 || Hq % cache->Hkv != 0) return ZQ_ERR_SHAPE;
  if (!std::isfinite(softmax_scale)) return ZQ_ERR_SHAPE;
  const int64_t qr = (int64_t)Hq * cache->d_qk, qs = q_stride ? q_stride : qr;
  if (qs < qr || qs > ((int64_t)1 << 31)) return ZQ_ERR_SHAPE;
  // The line of key tiles (at most a 16th of the keys of all heads, and 5 a
  // sequence and head) times its pieces (at most 1280) stays in 63 bits.
  if ((int64_t)cache->B * Hq > ((int64_t)1 << 53) / ((int64_t)cache->table_width * cache->page_size)) return ZQ_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || (lse && !aligned16(lse)) || qs % 8 != 0)
    return ZQ_ERR_ALIGN;
  int sms = 0;
  rc = check_device(&sms);
  if (rc != ZQ_OK) return rc;
  L.q = q;
  L.q_stride = qs;
  L.Hq = Hq;
  L.scale_log2 = scale_log2(softmax_scale, cache->d_qk);
  L.out = out;
  L.lse = lse;
  L.workspace = workspace;
  cudaError_t e = zq::launch_decode(L, static_cast<cudaStream_t>(stream), sms);
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

int zq_debug_exp2(const float* x, float* y, int64_t n, int degree, void* stream) {
  if (n < 0) return ZQ_ERR_SHAPE;
  if (n > 0 && (!x || !y)) return ZQ_ERR_NULL;
  if (degree != 3 && degree != 4 && degree != 5 && degree != 0 && degree != -1) return ZQ_ERR_UNSUPPORTED;
  int rc = check_device(nullptr);
  if (rc != ZQ_OK) return rc;
  cudaError_t e = zq::launch_exp2_check(x, y, n, degree, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

}  // extern "C"
