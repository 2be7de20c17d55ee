// C ABI entry points: host-side argument checks, launch-shape choice and
// launch. Every check runs before the first HIP call, so a rejected call
// enqueues nothing and touches no output.
#include <algorithm>
#include <cmath>
#include <mutex>

#include <hip/hip_runtime.h>

#include "qgemm.h"
#include "launch.h"

namespace {

constexpr int kMaxDevices = 64;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

qg_status check_tensor(const qg_tensor* t, int rank, qg_dtype dt) {
  if (!t) return QG_ERR_NULL;
  if (t->rank != rank) return QG_ERR_RANK;
  if (t->dtype != dt) return QG_ERR_DTYPE;
  int64_t n = 1;
  for (int i = 0; i < rank; ++i) {
    if (t->shape[i] < 0) return QG_ERR_SHAPE;
    n *= t->shape[i];
  }
  if (n > 0) {
    if (!t->data) return QG_ERR_NULL;
    if (!aligned16(t->data)) return QG_ERR_ALIGN;
  }
  return QG_OK;
}

int device_cus() {
  static int cache[kMaxDevices] = {0};
  static std::mutex mu;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
  std::lock_guard<std::mutex> lk(mu);
  if (cache[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cache[dev] = n;
  }
  return cache[dev];
}

qg_status launch_status(hipError_t e) {
  if (e == hipErrorNotSupported) return QG_ERR_UNSUPPORTED;
  return e == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

}  // namespace

extern "C" {

const char* qg_status_string(qg_status s) {
  switch (s) {
    case QG_OK: return "ok";
    case QG_ERR_NULL: return "a required pointer is NULL";
    case QG_ERR_RANK: return "a tensor has the wrong rank";
    case QG_ERR_DTYPE: return "a tensor has the wrong dtype";
    case QG_ERR_SHAPE: return "tensor shapes are inconsistent";
    case QG_ERR_ALIGN: return "a base pointer or row length is not 16-byte aligned";
    case QG_ERR_UNSUPPORTED: return "configuration not supported by this build";
    case QG_ERR_INVALID_ARG: return "a scalar argument is out of range";
    case QG_ERR_LAUNCH: return "HIP launch failed";
  }
  return "unknown status";
}

int32_t qg_version(void) { return 100; }

// Epilogue operands of a product Y [M, N] (gated output [M, N / 2]): bias has
// the output type and shape [N] (E == 0) or one row per expert [E, N]; residual
// is shaped like the output.
static qg_status check_epilogue(int32_t epilogue, const qg_tensor* bias, const qg_tensor* residual, qg_dtype act,
                                int64_t E, int64_t M, int64_t N, qg::Epilogue* out) {
  qg_status st;
  const int64_t N_out = (epilogue & QG_EPI_SILU_GATE) ? N / 2 : N;
  out->flags = epilogue;
  if (epilogue & QG_EPI_BIAS) {
    if (!bias) return QG_ERR_NULL;
    const int rank = E == 0 ? 1 : 2;
    if (bias->rank != rank) return QG_ERR_RANK;
    if ((st = check_tensor(bias, rank, act)) != QG_OK) return st;
    if (E == 0 ? bias->shape[0] != N : (bias->shape[0] != E || bias->shape[1] != N)) return QG_ERR_SHAPE;
    out->bias = static_cast<const uint16_t*>(bias->data);
  }
  if (epilogue & QG_EPI_RESIDUAL) {
    if (!residual) return QG_ERR_NULL;
    if (residual->rank != 2) return QG_ERR_RANK;
    if ((st = check_tensor(residual, 2, act)) != QG_OK) return st;
    if (residual->shape[0] != M || residual->shape[1] != N_out) return QG_ERR_SHAPE;
    out->residual = static_cast<const uint16_t*>(residual->data);
  }
  return QG_OK;
}

// nk: B is [N, K/8] and the scales [N, K/group_size] (no epilogue)
static qg_status qgemm_w4_impl(const qg_tensor* c, const qg_tensor* a, const qg_tensor* b_packed,
                               const qg_tensor* scales, int32_t group_size, int32_t pack_factor,
                               int32_t epilogue, const qg_tensor* bias, const qg_tensor* residual,
                               hipStream_t stream, bool nk = false) {
  if (!c || !a || !b_packed || !scales) return QG_ERR_NULL;
  // rank-2 requirement first: the page's only stated error condition
  if (c->rank != 2 || a->rank != 2 || b_packed->rank != 2 || scales->rank != 2) return QG_ERR_RANK;
  qg_status st;
  // activations, scales and output are all fp16 or all bf16 (the page's a_type
  // and c_type parameters)
  const qg_dtype act = a->dtype == QG_BF16 ? QG_BF16 : QG_F16;
  if ((st = check_tensor(c, 2, act)) != QG_OK) return st;
  if ((st = check_tensor(a, 2, act)) != QG_OK) return st;
  if ((st = check_tensor(b_packed, 2, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(scales, 2, act)) != QG_OK) return st;
  if (pack_factor != 8) return QG_ERR_UNSUPPORTED;
  if (group_size <= 0) return QG_ERR_INVALID_ARG;
  if (epilogue & ~(QG_EPI_BIAS | QG_EPI_RESIDUAL | QG_EPI_SILU_GATE)) return QG_ERR_INVALID_ARG;
  const int64_t M = a->shape[0], K = a->shape[1], N = b_packed->shape[nk ? 0 : 1];
  const bool gate = (epilogue & QG_EPI_SILU_GATE) != 0;
  if (gate && N % 16 != 0) return QG_ERR_ALIGN;   // (gate, up) pairs, and an 8-aligned output
  const int64_t N_out = gate ? N / 2 : N;
  if (c->shape[0] != M || c->shape[1] != N_out) return QG_ERR_SHAPE;
  if (K % group_size != 0) return QG_ERR_SHAPE;
  if (b_packed->shape[nk ? 1 : 0] * pack_factor != K) return QG_ERR_SHAPE;
  if (nk ? (scales->shape[0] != N || scales->shape[1] != K / group_size)
         : (scales->shape[0] != K / group_size || scales->shape[1] != N))
    return QG_ERR_SHAPE;
  if (group_size % 32 != 0 || group_size > 256 || (group_size & (group_size - 1)) != 0)
    return QG_ERR_UNSUPPORTED;
  if (N % 8 != 0) return QG_ERR_ALIGN;
  qg::Epilogue epi;
  if ((st = check_epilogue(epilogue, bias, residual, act, 0, M, N, &epi)) != QG_OK) return st;
  if (M > INT32_MAX / 2 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return QG_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return QG_OK;
  if (K == 0) return QG_ERR_UNSUPPORTED;  // would need a zero fill of C
  qg::W4Args p{static_cast<uint16_t*>(c->data), static_cast<const uint16_t*>(a->data),
               static_cast<const uint32_t*>(b_packed->data), static_cast<const uint16_t*>(scales->data),
               M, N, K, group_size, act == QG_BF16 ? 1 : 0, epi};
  p.nk = nk ? 1 : 0;
  if (M <= 16) return launch_status(qg::launch_w4_decode(p, stream));
  // the tiled kernel addresses 128 rows of A and eight packed rows of B (from a
  // stage's first packed row) with 32-bit buffer offsets
  if (K >= (1LL << 24) || N >= (1LL << 27)) return QG_ERR_UNSUPPORTED;
  return launch_status(qg::launch_w4_prefill(p, device_cus(), stream));
}

qg_status qgemm_w4_nk(const qg_tensor* c, const qg_tensor* a, const qg_tensor* b_packed,
                      const qg_tensor* scales, int32_t group_size, int32_t pack_factor,
                      hipStream_t stream) {
  return qgemm_w4_impl(c, a, b_packed, scales, group_size, pack_factor, 0, nullptr, nullptr, stream, true);
}

qg_status qgemm_w4(const qg_tensor* c, const qg_tensor* a, const qg_tensor* b_packed,
                   const qg_tensor* scales, int32_t group_size, int32_t pack_factor,
                   hipStream_t stream) {
  return qgemm_w4_impl(c, a, b_packed, scales, group_size, pack_factor, 0, nullptr, nullptr, stream);
}

qg_status qgemm_w4_epilogue(const qg_tensor* c, const qg_tensor* a, const qg_tensor* b_packed,
                            const qg_tensor* scales, int32_t group_size, int32_t pack_factor,
                            int32_t epilogue, const qg_tensor* bias, const qg_tensor* residual,
                            hipStream_t stream) {
  return qgemm_w4_impl(c, a, b_packed, scales, group_size, pack_factor, epilogue, bias, residual, stream);
}

static qg_status grouped_gemm_impl(const qg_tensor* c, const qg_tensor* a, const qg_tensor* a_offsets,
                                   const qg_tensor* b, const qg_tensor* expert_ids,
                                   const uint32_t* expert_usage_stats_host, int32_t transpose_b,
                                   const int32_t* a_plane_splits, int32_t epilogue, const qg_tensor* bias,
                                   const qg_tensor* residual, hipStream_t stream) {
  if (!c || !a || !a_offsets || !b || !expert_ids || !expert_usage_stats_host) return QG_ERR_NULL;
  if (c->rank != 2 || a->rank != 2 || a_offsets->rank != 1 || b->rank != 3 || expert_ids->rank != 1)
    return QG_ERR_RANK;
  qg_status st;
  if ((st = check_tensor(c, 2, QG_BF16)) != QG_OK) return st;
  if ((st = check_tensor(a, 2, QG_BF16)) != QG_OK) return st;
  if ((st = check_tensor(a_offsets, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(b, 3, QG_BF16)) != QG_OK) return st;
  if ((st = check_tensor(expert_ids, 1, QG_I32)) != QG_OK) return st;
  const int64_t T = c->shape[0], K = a->shape[1];
  const int64_t E = b->shape[0];
  const int64_t N = transpose_b ? b->shape[1] : b->shape[2];
  const int64_t Kb = transpose_b ? b->shape[2] : b->shape[1];
  const int64_t G = expert_ids->shape[0];
  // planes of A (fused LoRA QKV): splits (s0, s1) != (0, 0) cut the columns into
  // [0, s0), [s0, s0 + s1), [s0 + s1, N), read from three planes of T rows of A
  const int64_t s0 = a_plane_splits ? a_plane_splits[0] : 0, s1 = a_plane_splits ? a_plane_splits[1] : 0;
  const bool planes = s0 != 0 || s1 != 0;
  if (s0 < 0 || s1 < 0 || s0 + s1 > N) return QG_ERR_SHAPE;
  if (s0 % 8 != 0 || s1 % 8 != 0) return QG_ERR_ALIGN;   // 8-aligned like N; gate pairs stay in one plane
  if (a->shape[0] != (planes ? 3 * T : T)) return QG_ERR_SHAPE;
  if (epilogue & ~(QG_EPI_BIAS | QG_EPI_RESIDUAL | QG_EPI_SILU_GATE)) return QG_ERR_INVALID_ARG;
  const bool gate = (epilogue & QG_EPI_SILU_GATE) != 0;
  if (gate && N % 16 != 0) return QG_ERR_ALIGN;   // (gate, up) pairs, and an 8-aligned output
  const int64_t N_out = gate ? N / 2 : N;
  if (c->shape[1] != N_out || Kb != K) return QG_ERR_SHAPE;
  if (a_offsets->shape[0] != G + 1) return QG_ERR_SHAPE;
  const uint32_t num_active = expert_usage_stats_host[1];
  if ((int64_t)num_active > G) return QG_ERR_INVALID_ARG;
  if (K % 8 != 0 || N % 8 != 0) return QG_ERR_ALIGN;
  qg::Epilogue epi;
  if ((st = check_epilogue(epilogue, bias, residual, QG_BF16, E, T, N, &epi)) != QG_OK) return st;
  if (3 * T > INT32_MAX / 2 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return QG_ERR_UNSUPPORTED;
  if (N * K * 2 > 0xFFFFFFFFLL) return QG_ERR_UNSUPPORTED;   // 32-bit buffer offsets within an expert
  if (num_active == 0 || T == 0 || N == 0 || E == 0) return QG_OK;
  if (K == 0) return QG_ERR_UNSUPPORTED;
  qg::GroupedArgs p{static_cast<uint16_t*>(c->data), static_cast<const uint16_t*>(a->data),
                    static_cast<const uint32_t*>(a_offsets->data), static_cast<const uint16_t*>(b->data),
                    static_cast<const int32_t*>(expert_ids->data), T, N, K, E, (int)num_active,
                    (int)expert_usage_stats_host[0], device_cus(), transpose_b ? 1 : 0, epi};
  p.planes = planes ? qg::Planes{(int)s0, (int)(s0 + s1), (int)T} : qg::Planes{(int)N, (int)N, 0};
  return launch_status(qg::launch_grouped_bf16(p, stream));
}

qg_status grouped_gemm(const qg_tensor* c, const qg_tensor* a, const qg_tensor* a_offsets,
                       const qg_tensor* b, const qg_tensor* expert_ids,
                       const uint32_t* expert_usage_stats_host, int32_t transpose_b,
                       const int32_t* a_plane_splits_host, hipStream_t stream) {
  return grouped_gemm_impl(c, a, a_offsets, b, expert_ids, expert_usage_stats_host, transpose_b,
                           a_plane_splits_host, 0, nullptr, nullptr, stream);
}

qg_status grouped_gemm_epilogue(const qg_tensor* c, const qg_tensor* a, const qg_tensor* a_offsets,
                                const qg_tensor* b, const qg_tensor* expert_ids,
                                const uint32_t* expert_usage_stats_host, int32_t transpose_b,
                                const int32_t* a_plane_splits_host, int32_t epilogue, const qg_tensor* bias,
                                const qg_tensor* residual, hipStream_t stream) {
  return grouped_gemm_impl(c, a, a_offsets, b, expert_ids, expert_usage_stats_host, transpose_b,
                           a_plane_splits_host, epilogue, bias, residual, stream);
}

static qg_status grouped_gemm_w4_impl(const qg_tensor* c, const qg_tensor* a, const qg_tensor* a_offsets,
                                      const qg_tensor* b_packed, const qg_tensor* scales,
                                      const qg_tensor* expert_ids, const uint32_t* expert_usage_stats_host,
                                      int32_t group_size, int32_t pack_factor, int32_t epilogue,
                                      const qg_tensor* bias, const qg_tensor* residual, hipStream_t stream) {
  if (!c || !a || !a_offsets || !b_packed || !scales || !expert_ids || !expert_usage_stats_host)
    return QG_ERR_NULL;
  if (c->rank != 2 || a->rank != 2 || a_offsets->rank != 1 || b_packed->rank != 3 || scales->rank != 3 ||
      expert_ids->rank != 1)
    return QG_ERR_RANK;
  qg_status st;
  // a, scales and c (and bias, residual) share one type, fp16 or bf16
  const qg_dtype act = a->dtype == QG_BF16 ? QG_BF16 : QG_F16;
  if ((st = check_tensor(c, 2, act)) != QG_OK) return st;
  if ((st = check_tensor(a, 2, act)) != QG_OK) return st;
  if ((st = check_tensor(a_offsets, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(b_packed, 3, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(scales, 3, act)) != QG_OK) return st;
  if ((st = check_tensor(expert_ids, 1, QG_I32)) != QG_OK) return st;
  if (pack_factor != 8) return QG_ERR_UNSUPPORTED;
  if (group_size <= 0) return QG_ERR_INVALID_ARG;
  if (epilogue & ~(QG_EPI_BIAS | QG_EPI_RESIDUAL | QG_EPI_SILU_GATE)) return QG_ERR_INVALID_ARG;
  const int64_t T = a->shape[0], K = a->shape[1], N = b_packed->shape[2];
  const int64_t E = b_packed->shape[0], G = expert_ids->shape[0];
  const bool gate = (epilogue & QG_EPI_SILU_GATE) != 0;
  if (gate && N % 16 != 0) return QG_ERR_ALIGN;   // (gate, up) pairs, and an 8-aligned output
  if (c->shape[0] != T || c->shape[1] != (gate ? N / 2 : N)) return QG_ERR_SHAPE;
  if (K % group_size != 0) return QG_ERR_SHAPE;
  if (b_packed->shape[1] * pack_factor != K) return QG_ERR_SHAPE;
  if (scales->shape[0] != E || scales->shape[1] != K / group_size || scales->shape[2] != N) return QG_ERR_SHAPE;
  if (a_offsets->shape[0] != G + 1) return QG_ERR_SHAPE;
  if (group_size % 32 != 0 || group_size > 256 || (group_size & (group_size - 1)) != 0)
    return QG_ERR_UNSUPPORTED;
  if (N % 8 != 0) return QG_ERR_ALIGN;
  const uint32_t num_active = expert_usage_stats_host[1];
  if ((int64_t)num_active > G) return QG_ERR_INVALID_ARG;
  qg::Epilogue epi;
  if ((st = check_epilogue(epilogue, bias, residual, act, E, T, N, &epi)) != QG_OK) return st;
  if (T > INT32_MAX / 2 || N > INT32_MAX / 2 || K > INT32_MAX / 2 || E > INT32_MAX / 2) return QG_ERR_UNSUPPORTED;
  // the tiled kernel addresses a tile's rows of A and eight packed rows of an
  // expert's B with 32-bit buffer offsets
  if (K >= (1LL << 24) || N >= (1LL << 27)) return QG_ERR_UNSUPPORTED;
  if (T == 0 || N == 0 || num_active == 0) return QG_OK;
  if (K == 0) return QG_ERR_UNSUPPORTED;  // would need a zero fill of the routed rows
  qg::W4GroupedArgs p{static_cast<uint16_t*>(c->data), static_cast<const uint16_t*>(a->data),
                      static_cast<const uint32_t*>(a_offsets->data), static_cast<const uint32_t*>(b_packed->data),
                      static_cast<const uint16_t*>(scales->data), static_cast<const int32_t*>(expert_ids->data),
                      T, N, K, E, group_size, (int)num_active, epi};
  p.bf16 = act == QG_BF16 ? 1 : 0;
  return launch_status(qg::launch_w4_grouped(p, stream));
}

qg_status grouped_gemm_w4(const qg_tensor* c, const qg_tensor* a, const qg_tensor* a_offsets,
                          const qg_tensor* b_packed, const qg_tensor* scales, const qg_tensor* expert_ids,
                          const uint32_t* expert_usage_stats_host, int32_t group_size, int32_t pack_factor,
                          hipStream_t stream) {
  return grouped_gemm_w4_impl(c, a, a_offsets, b_packed, scales, expert_ids, expert_usage_stats_host, group_size,
                              pack_factor, 0, nullptr, nullptr, stream);
}

qg_status grouped_gemm_w4_epilogue(const qg_tensor* c, const qg_tensor* a, const qg_tensor* a_offsets,
                                   const qg_tensor* b_packed, const qg_tensor* scales,
                                   const qg_tensor* expert_ids, const uint32_t* expert_usage_stats_host,
                                   int32_t group_size, int32_t pack_factor, int32_t epilogue,
                                   const qg_tensor* bias, const qg_tensor* residual, hipStream_t stream) {
  return grouped_gemm_w4_impl(c, a, a_offsets, b_packed, scales, expert_ids, expert_usage_stats_host, group_size,
                              pack_factor, epilogue, bias, residual, stream);
}

// Granularity and scales of an e4m3 cache.
static qg_status check_cache_scales(const qg_paged_kv* kv) {
  const int64_t* bs = kv->blocks.shape;
  const int64_t G = kv->quantization_granularity;
  if (G != 32 && G != 64 && G != 128) return QG_ERR_UNSUPPORTED;
  if (bs[5] % G != 0) return QG_ERR_UNSUPPORTED;
  if (kv->scales.rank != 6) return QG_ERR_RANK;
  const qg_status st = check_tensor(&kv->scales, 6, QG_F32);
  if (st != QG_OK) return st;
  const int64_t* ss = kv->scales.shape;
  for (int i = 0; i < 5; ++i)
    if (ss[i] != bs[i]) return QG_ERR_SHAPE;
  return ss[5] == bs[5] / G ? QG_OK : QG_ERR_SHAPE;
}

// planes: 1 (keys only) or 2 (weight columns = [W_k | W_v])
static qg_status kv_proj_impl(const qg_tensor* hidden, const qg_tensor* input_row_offsets,
                              const qg_tensor* weight, const qg_tensor* input_scale,
                              const qg_tensor* weight_scale, const int32_t* scales_granularity_mnk,
                              const qg_paged_kv* kv, uint32_t layer_idx, int planes, hipStream_t stream) {
  if (!hidden || !input_row_offsets || !weight || !input_scale || !weight_scale ||
      !scales_granularity_mnk || !kv)
    return QG_ERR_NULL;
  if (hidden->rank != 2 || input_row_offsets->rank != 1 || weight->rank != 2 || input_scale->rank != 2 ||
      weight_scale->rank != 2 || kv->blocks.rank != 6)
    return QG_ERR_RANK;
  qg_status st;
  const bool hidden_fp8 = hidden->dtype == QG_FP8_E4M3;   // the page's dtype parameter: bf16 or e4m3
  if ((st = check_tensor(hidden, 2, hidden_fp8 ? QG_FP8_E4M3 : QG_BF16)) != QG_OK) return st;
  if ((st = check_tensor(input_row_offsets, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(weight, 2, QG_FP8_E4M3)) != QG_OK) return st;
  if ((st = check_tensor(input_scale, 2, QG_F32)) != QG_OK) return st;
  if ((st = check_tensor(weight_scale, 2, QG_F32)) != QG_OK) return st;
  const bool fp8 = kv->blocks.dtype == QG_FP8_E4M3;   // quantized cache
  if ((st = check_tensor(&kv->blocks, 6, fp8 ? QG_FP8_E4M3 : QG_BF16)) != QG_OK) return st;
  if (scales_granularity_mnk[0] != 1 || scales_granularity_mnk[1] != 128 || scales_granularity_mnk[2] != 128)
    return QG_ERR_UNSUPPORTED;
  const int64_t T = hidden->shape[0], Kh = hidden->shape[1];
  const int64_t N = weight->shape[1];
  const int64_t B = input_row_offsets->shape[0] - 1;
  const int64_t* bs = kv->blocks.shape;
  const int64_t L = bs[0], P = bs[2], S = bs[3], Hkv = bs[4], D = bs[5];
  if (B < 0) return QG_ERR_SHAPE;
  if (weight->shape[0] != Kh) return QG_ERR_SHAPE;
  if (Kh % 128 != 0 || N % 128 != 0) return QG_ERR_SHAPE;
  if (input_scale->shape[0] != T || input_scale->shape[1] != Kh / 128) return QG_ERR_SHAPE;
  if (weight_scale->shape[0] != Kh / 128 || weight_scale->shape[1] != N / 128) return QG_ERR_SHAPE;
  if (bs[1] != 2 || Hkv * D * planes != N) return QG_ERR_SHAPE;
  if (planes > 1 && (Hkv * D) % 128 != 0) return QG_ERR_SHAPE;   // each 128-column tile in one plane
  const int64_t G = fp8 ? kv->quantization_granularity : 0;
  if (fp8 && (st = check_cache_scales(kv)) != QG_OK) return st;
  if ((int64_t)layer_idx >= L) return QG_ERR_INVALID_ARG;
  if (kv->max_pages_per_seq <= 0 && T > 0) return QG_ERR_INVALID_ARG;
  if (B > 0 && T > 0 && (!kv->cache_lengths || !kv->page_table)) return QG_ERR_NULL;
  if (T > INT32_MAX / 2 || Kh > INT32_MAX / 2 || N > INT32_MAX / 2) return QG_ERR_UNSUPPORTED;
  if (T == 0 || B == 0 || N == 0) return QG_OK;
  if (Kh == 0) return QG_ERR_UNSUPPORTED;
  qg::KProjArgs p{static_cast<const uint16_t*>(hidden->data),
                  static_cast<const uint32_t*>(input_row_offsets->data),
                  static_cast<const uint8_t*>(weight->data),
                  static_cast<const float*>(input_scale->data),
                  static_cast<const float*>(weight_scale->data),
                  kv->blocks.data,
                  kv->cache_lengths, kv->page_table,
                  T, Kh, N, B, kv->max_pages_per_seq, L, P, S, layer_idx, device_cus()};
  p.n_plane = Hkv * D;
  p.fp8 = fp8 ? 1 : 0;
  p.kv_scales = fp8 ? static_cast<float*>(kv->scales.data) : nullptr;
  p.qgran = (int)G;
  p.hidden_fp8 = hidden_fp8 ? 1 : 0;
  return launch_status(qg::launch_kproj_fp8(p, stream));
}

qg_status k_matmul_ragged_paged_scale(const qg_tensor* hidden, const qg_tensor* input_row_offsets,
                                      const qg_tensor* weight, const qg_tensor* input_scale,
                                      const qg_tensor* weight_scale,
                                      const int32_t* scales_granularity_mnk,
                                      const qg_paged_kv* kv, uint32_t layer_idx,
                                      hipStream_t stream) {
  return kv_proj_impl(hidden, input_row_offsets, weight, input_scale, weight_scale, scales_granularity_mnk, kv,
                      layer_idx, 1, stream);
}

qg_status kv_matmul_ragged_paged_scale(const qg_tensor* hidden, const qg_tensor* input_row_offsets,
                                       const qg_tensor* weight, const qg_tensor* input_scale,
                                       const qg_tensor* weight_scale,
                                       const int32_t* scales_granularity_mnk,
                                       const qg_paged_kv* kv, uint32_t layer_idx,
                                       hipStream_t stream) {
  return kv_proj_impl(hidden, input_row_offsets, weight, input_scale, weight_scale, scales_granularity_mnk, kv,
                      layer_idx, 2, stream);
}

qg_status tables_ragged_paged(const qg_tensor* input_row_offsets, const qg_tensor* slot_map,
                              const qg_tensor* page_table, const qg_tensor* result,
                              const qg_tensor* cache_lengths, const qg_tensor* new_lengths,
                              const qg_tensor* free_pages, const qg_tensor* free_count, int32_t page_size,
                              hipStream_t stream) {
  if (!input_row_offsets || !page_table || !result || !cache_lengths || !new_lengths || !free_pages || !free_count)
    return QG_ERR_NULL;
  qg_status st;
  if ((st = check_tensor(input_row_offsets, 1, QG_U32)) != QG_OK) return st;
  if (slot_map && (st = check_tensor(slot_map, 1, QG_I32)) != QG_OK) return st;
  if ((st = check_tensor(page_table, 2, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(result, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(cache_lengths, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(new_lengths, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(free_pages, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(free_count, 1, QG_U32)) != QG_OK) return st;
  const int64_t B = cache_lengths->shape[0], W = page_table->shape[1];
  if (new_lengths->shape[0] != B || page_table->shape[0] != B || input_row_offsets->shape[0] != B + 1)
    return QG_ERR_SHAPE;
  if (result->shape[0] != 2 || free_count->shape[0] != 1) return QG_ERR_SHAPE;
  if (page_size <= 0) return QG_ERR_INVALID_ARG;
  const int64_t F = free_pages->shape[0], T = slot_map ? slot_map->shape[0] : 0;
  if (B > qg::kTablesMaxBatch || W >= INT32_MAX / page_size || F > INT32_MAX || T > INT32_MAX) return QG_ERR_UNSUPPORTED;
  if (B == 0) return QG_OK;
  // a slot map without elements still bounds the number of tokens
  static int32_t none;
  qg::TablesArgs p{static_cast<uint32_t*>(input_row_offsets->data),
                   !slot_map ? nullptr : T > 0 ? static_cast<int32_t*>(slot_map->data) : &none,
                   static_cast<uint32_t*>(page_table->data), static_cast<uint32_t*>(result->data),
                   static_cast<const uint32_t*>(cache_lengths->data), static_cast<const uint32_t*>(new_lengths->data),
                   static_cast<const uint32_t*>(free_pages->data), static_cast<const uint32_t*>(free_count->data),
                   (int)B, (int)W, F, T, page_size, device_cus()};
  return launch_status(qg::launch_tables_ragged(p, stream));
}

static bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return a_bytes > 0 && b_bytes > 0 && x < y + b_bytes && y < x + a_bytes;
}

qg_status release_ragged_paged(const qg_tensor* free_pages, const qg_tensor* result, const qg_tensor* page_table,
                               const qg_tensor* held_lengths, const qg_tensor* kept_lengths,
                               const qg_tensor* free_count, int32_t page_size, hipStream_t stream) {
  if (!free_pages || !result || !page_table || !held_lengths || !kept_lengths || !free_count) return QG_ERR_NULL;
  qg_status st;
  if ((st = check_tensor(free_pages, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(result, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(page_table, 2, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(held_lengths, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(kept_lengths, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(free_count, 1, QG_U32)) != QG_OK) return st;
  const int64_t B = held_lengths->shape[0], W = page_table->shape[1], F = free_pages->shape[0];
  if (kept_lengths->shape[0] != B || page_table->shape[0] != B) return QG_ERR_SHAPE;
  if (result->shape[0] != 2 || free_count->shape[0] != 1) return QG_ERR_SHAPE;
  if (page_size <= 0) return QG_ERR_INVALID_ARG;
  if (overlap(result->data, 8, free_count->data, 4)) return QG_ERR_INVALID_ARG;
  if (B > qg::kTablesMaxBatch || W >= INT32_MAX / page_size || F > INT32_MAX) return QG_ERR_UNSUPPORTED;
  if (B == 0) return QG_OK;
  qg::ReleaseArgs p{static_cast<uint32_t*>(free_pages->data), static_cast<uint32_t*>(result->data),
                    static_cast<const uint32_t*>(page_table->data), static_cast<const uint32_t*>(held_lengths->data),
                    static_cast<const uint32_t*>(kept_lengths->data), static_cast<const uint32_t*>(free_count->data),
                    (int)B, (int)W, F, page_size, device_cus()};
  return launch_status(qg::launch_release_ragged(p, stream));
}

// The cache of a call for B sequences: its form first, then, where rows are to be moved,
// what they are reached by.
static qg_status check_cache(const qg_paged_kv* kv) {
  if (kv->blocks.rank != 6) return QG_ERR_RANK;
  const bool fp8 = kv->blocks.dtype == QG_FP8_E4M3;
  qg_status st;
  if ((st = check_tensor(&kv->blocks, 6, fp8 ? QG_FP8_E4M3 : QG_BF16)) != QG_OK) return st;
  if (kv->blocks.shape[1] != 2) return QG_ERR_SHAPE;
  if (kv->blocks.shape[5] % 8 != 0) return QG_ERR_ALIGN;
  return fp8 ? check_cache_scales(kv) : QG_OK;
}
static qg_status cache_args(const qg_paged_kv* kv, int64_t B, bool lengths, qg::CacheArgs* out) {
  const int64_t* bs = kv->blocks.shape;
  if (bs[2] == 0 || bs[3] == 0 || kv->max_pages_per_seq <= 0) return QG_ERR_INVALID_ARG;
  if ((lengths && !kv->cache_lengths) || !kv->page_table) return QG_ERR_NULL;
  // positions of a sequence are counted in 32 bits
  if (B > INT32_MAX / 2 || bs[3] > INT32_MAX / 2 || kv->max_pages_per_seq > (INT32_MAX / 2) / bs[3]) return QG_ERR_UNSUPPORTED;
  if (bs[4] > (1 << 26) / bs[5]) return QG_ERR_UNSUPPORTED;   // a cache row's bytes too
  const bool fp8 = kv->blocks.dtype == QG_FP8_E4M3;
  out->blocks = kv->blocks.data;
  out->scales = fp8 ? static_cast<float*>(kv->scales.data) : nullptr;
  out->cache_len = kv->cache_lengths;
  out->page_table = kv->page_table;
  out->layers = bs[0];
  out->pages = bs[2];
  out->max_pages = kv->max_pages_per_seq;
  out->batch = (int)B;
  out->page_size = (int)bs[3];
  out->hkv = (int)bs[4];
  out->d = (int)bs[5];
  out->gran = fp8 ? (int)kv->quantization_granularity : 0;
  out->fp8 = fp8 ? 1 : 0;
  return QG_OK;
}
constexpr int64_t kMostRows = 1 << 24;   // tokens, rows or sequences of a call: a launch has less than 2^32 threads

// One of rope_ragged_paged's inputs [T, H, D], whose rows are `stride` elements apart.
static qg_status check_rows(const qg_tensor* t, int64_t T, int64_t H, int64_t D, int64_t stride) {
  if (t->shape[0] != T || t->shape[1] != H || t->shape[2] != D) return QG_ERR_SHAPE;
  if (stride < H * D) return QG_ERR_SHAPE;
  return stride % 8 == 0 ? QG_OK : QG_ERR_ALIGN;
}

qg_status rope_ragged_paged(const qg_tensor* q_out, const qg_tensor* q, const qg_tensor* k, const qg_tensor* v,
                            const int64_t* row_strides_host, const qg_tensor* input_row_offsets,
                            const qg_paged_kv* kv, uint32_t layer_idx, const qg_tensor* inv_freq,
                            const qg_tensor* positions, int32_t interleaved, float amplitude, hipStream_t stream) {
  if ((!q && !k) || !q != !q_out || !k != !v || !input_row_offsets || !kv || !inv_freq) return QG_ERR_NULL;
  qg_status st;
  for (const qg_tensor* t : {q_out, q, k, v})
    if (t && (st = check_tensor(t, 3, QG_BF16)) != QG_OK) return st;
  if ((st = check_tensor(input_row_offsets, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_tensor(inv_freq, 1, QG_F32)) != QG_OK) return st;
  if (positions && (st = check_tensor(positions, 1, QG_I32)) != QG_OK) return st;
  if ((st = check_cache(kv)) != QG_OK) return st;
  const int64_t* bs = kv->blocks.shape;
  const int64_t T = (q ? q : k)->shape[0], Hq = q ? q->shape[1] : 0, Hkv = bs[4], D = bs[5];
  const int64_t B = input_row_offsets->shape[0] - 1;
  if (B < 0) return QG_ERR_SHAPE;
  const int64_t qs = row_strides_host && q ? row_strides_host[0] : Hq * D;
  const int64_t ks = row_strides_host && k ? row_strides_host[1] : Hkv * D;
  const int64_t vs = row_strides_host && v ? row_strides_host[2] : Hkv * D;
  if (q && (st = check_rows(q, T, Hq, D, qs)) != QG_OK) return st;
  if (q && (st = check_rows(q_out, T, Hq, D, Hq * D)) != QG_OK) return st;
  if (k && (st = check_rows(k, T, Hkv, D, ks)) != QG_OK) return st;
  if (k && (st = check_rows(v, T, Hkv, D, vs)) != QG_OK) return st;
  if (2 * inv_freq->shape[0] > D) return QG_ERR_SHAPE;
  if (positions && positions->shape[0] != T) return QG_ERR_SHAPE;
  if ((int64_t)layer_idx >= bs[0]) return QG_ERR_INVALID_ARG;
  if (!std::isfinite(amplitude)) return QG_ERR_INVALID_ARG;
  if (D > 1024 || T > kMostRows || Hq > (1 << 26) / (D > 0 ? D : 1)) return QG_ERR_UNSUPPORTED;
  if (T == 0 || B == 0 || D == 0 || (Hq == 0 && (!k || Hkv == 0))) return QG_OK;
  // a workgroup's threads read what others of it turn: not in place
  auto bytes = [&](int64_t H, int64_t stride) { return H > 0 ? 2 * ((T - 1) * std::min<int64_t>(stride, 1ll << 36) + H * D) : 0; };
  if (q && (overlap(q_out->data, bytes(Hq, Hq * D), q->data, bytes(Hq, qs)) ||
            (k && (overlap(q_out->data, bytes(Hq, Hq * D), k->data, bytes(Hkv, ks)) ||
                   overlap(q_out->data, bytes(Hq, Hq * D), v->data, bytes(Hkv, vs))))))
    return QG_ERR_INVALID_ARG;
  qg::RopeArgs p{};
  if ((st = cache_args(kv, B, true, &p.kv)) != QG_OK) return st;
  if (q && Hq > 0) {
    p.q_out = static_cast<uint16_t*>(q_out->data);
    p.q = static_cast<const uint16_t*>(q->data);
  }
  if (k && Hkv > 0) {
    p.k = static_cast<const uint16_t*>(k->data);
    p.v = static_cast<const uint16_t*>(v->data);
  }
  p.q_stride = qs;
  p.k_stride = ks;
  p.v_stride = vs;
  p.offs = static_cast<const uint32_t*>(input_row_offsets->data);
  p.inv_freq = static_cast<const float*>(inv_freq->data);
  p.positions = positions ? static_cast<const int32_t*>(positions->data) : nullptr;
  p.T = T;
  p.hq = (int)Hq;
  p.layer = (int)layer_idx;
  p.half = (int)inv_freq->shape[0];
  p.interleaved = interleaved ? 1 : 0;
  p.num_cus = device_cus();
  p.amplitude = amplitude;
  return launch_status(qg::launch_rope_paged(p, stream));
}

qg_status kv_read_ragged_paged(const qg_tensor* k_out, const qg_tensor* v_out, const qg_tensor* output_row_offsets,
                               const qg_tensor* first_positions, const qg_paged_kv* kv, uint32_t layer_idx,
                               hipStream_t stream) {
  if ((!k_out && !v_out) || !output_row_offsets || !kv) return QG_ERR_NULL;
  qg_status st;
  const qg_tensor* one = k_out ? k_out : v_out;
  const qg_dtype type = one->dtype == QG_F32 ? QG_F32 : QG_BF16;
  for (const qg_tensor* t : {k_out, v_out})
    if (t && (st = check_tensor(t, 3, type)) != QG_OK) return st;
  if ((st = check_tensor(output_row_offsets, 1, QG_U32)) != QG_OK) return st;
  if (first_positions && (st = check_tensor(first_positions, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_cache(kv)) != QG_OK) return st;
  const int64_t* bs = kv->blocks.shape;
  const int64_t T = one->shape[0], Hkv = bs[4], D = bs[5], B = output_row_offsets->shape[0] - 1;
  if (B < 0) return QG_ERR_SHAPE;
  for (const qg_tensor* t : {k_out, v_out})
    if (t && (t->shape[0] != T || t->shape[1] != Hkv || t->shape[2] != D)) return QG_ERR_SHAPE;
  if (first_positions && first_positions->shape[0] != B) return QG_ERR_SHAPE;
  if ((int64_t)layer_idx >= bs[0]) return QG_ERR_INVALID_ARG;
  if (T > kMostRows) return QG_ERR_UNSUPPORTED;
  if (T == 0 || B == 0 || Hkv == 0 || D == 0) return QG_OK;
  qg::KvReadArgs p{};
  if ((st = cache_args(kv, B, false, &p.kv)) != QG_OK) return st;
  p.out[0] = k_out ? k_out->data : nullptr;
  p.out[1] = v_out ? v_out->data : nullptr;
  p.offs = static_cast<const uint32_t*>(output_row_offsets->data);
  p.first = first_positions ? static_cast<const uint32_t*>(first_positions->data) : nullptr;
  p.T = T;
  p.layer = (int)layer_idx;
  p.f32 = type == QG_F32 ? 1 : 0;
  p.num_cus = device_cus();
  return launch_status(qg::launch_kv_read(p, stream));
}

qg_status kv_keep_ragged_paged(const qg_tensor* path, const qg_tensor* kept, const qg_paged_kv* kv,
                               hipStream_t stream) {
  if (!path || !kept || !kv) return QG_ERR_NULL;
  qg_status st;
  if ((st = check_tensor(path, 2, QG_I32)) != QG_OK) return st;
  if ((st = check_tensor(kept, 1, QG_U32)) != QG_OK) return st;
  if ((st = check_cache(kv)) != QG_OK) return st;
  const int64_t* bs = kv->blocks.shape;
  const int64_t B = kept->shape[0], M = path->shape[1];
  if (path->shape[0] != B) return QG_ERR_SHAPE;
  if (B > kMostRows / 4 || M > INT32_MAX / 2 || bs[0] > INT32_MAX / 2) return QG_ERR_UNSUPPORTED;
  if (B == 0 || M == 0 || bs[0] == 0 || bs[4] == 0 || bs[5] == 0) return QG_OK;
  qg::KvKeepArgs p{};
  if ((st = cache_args(kv, B, true, &p.kv)) != QG_OK) return st;
  p.path = static_cast<const int32_t*>(path->data);
  p.kept = static_cast<const uint32_t*>(kept->data);
  p.width = M;
  p.num_cus = device_cus();
  return launch_status(qg::launch_kv_keep(p, stream));
}

int64_t attention_ragged_paged_workspace(int64_t T, int64_t batch, int64_t num_q_heads, int64_t num_kv_heads,
                                         int64_t head_dim) {
  if (T <= 0 || batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0) return 0;
  return qg::attention_paged_workspace(T, batch, num_q_heads, num_kv_heads, head_dim);
}

// tree: with tree_mask (then causal is 0)
static qg_status attention_impl(const qg_tensor* out, const qg_tensor* q, const qg_tensor* input_row_offsets,
                                const qg_tensor* tree_mask, const qg_paged_kv* kv, uint32_t layer_idx, float scale,
                                int32_t causal, int32_t window, const qg_tensor* workspace, bool tree,
                                hipStream_t stream) {
  if (!out || !q || !input_row_offsets || !kv || !workspace || (tree && !tree_mask)) return QG_ERR_NULL;
  if (out->rank != 3 || q->rank != 3 || input_row_offsets->rank != 1 || kv->blocks.rank != 6 || workspace->rank != 1)
    return QG_ERR_RANK;
  qg_status st;
  if ((st = check_tensor(out, 3, QG_BF16)) != QG_OK) return st;
  if ((st = check_tensor(q, 3, QG_BF16)) != QG_OK) return st;
  if ((st = check_tensor(input_row_offsets, 1, QG_U32)) != QG_OK) return st;
  const bool fp8 = kv->blocks.dtype == QG_FP8_E4M3;   // quantized cache
  if ((st = check_tensor(&kv->blocks, 6, fp8 ? QG_FP8_E4M3 : QG_BF16)) != QG_OK) return st;
  if ((st = check_tensor(workspace, 1, QG_F32)) != QG_OK) return st;
  if (tree && (st = check_tensor(tree_mask, 2, QG_U32)) != QG_OK) return st;
  const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t B = input_row_offsets->shape[0] - 1;
  const int64_t* bs = kv->blocks.shape;
  const int64_t L = bs[0], P = bs[2], S = bs[3], Hkv = bs[4];
  if (B < 0 || out->shape[0] != T || out->shape[1] != Hq || out->shape[2] != D) return QG_ERR_SHAPE;
  if (bs[1] != 2 || bs[5] != D) return QG_ERR_SHAPE;
  if (Hkv == 0 ? Hq != 0 : Hq % Hkv != 0) return QG_ERR_SHAPE;
  if (tree && (tree_mask->shape[0] != T || tree_mask->shape[1] < 1)) return QG_ERR_SHAPE;
  if (D % 8 != 0) return QG_ERR_ALIGN;
  if (fp8 && (st = check_cache_scales(kv)) != QG_OK) return st;
  if ((int64_t)layer_idx >= L) return QG_ERR_INVALID_ARG;
  // (log2 e: the kernels' exponents have base 2)
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f) || window < 0) return QG_ERR_INVALID_ARG;
  if (window > 0 && !causal && !tree) return QG_ERR_UNSUPPORTED;
  if (D > 256) return QG_ERR_UNSUPPORTED;
  if (T == 0 || B == 0 || Hq == 0 || D == 0) return QG_OK;
  if (P == 0 || S == 0 || kv->max_pages_per_seq <= 0) return QG_ERR_INVALID_ARG;
  if (!kv->cache_lengths || !kv->page_table) return QG_ERR_NULL;
  if (workspace->shape[0] < qg::attention_paged_workspace(T, B, Hq, Hkv, D)) return QG_ERR_SHAPE;
  // rows of a key/value head and positions of a sequence are counted in 32 bits
  if (B > INT32_MAX / 2 || S > INT32_MAX / 2 || Hq > INT32_MAX / 2 || T > (INT32_MAX / 2) / (Hq / Hkv) ||
      kv->max_pages_per_seq > (INT32_MAX / 2) / S)
    return QG_ERR_UNSUPPORTED;
  if (tree && tree_mask->shape[1] > (1 << 24)) return QG_ERR_UNSUPPORTED;   // a row's bits are counted in 32 bits
  if (Hkv > (1 << 26) / D) return QG_ERR_UNSUPPORTED;   // offsets within 16 cache rows are 32-bit
  qg::AttnArgs p{};
  p.out = static_cast<uint16_t*>(out->data);
  p.q = static_cast<const uint16_t*>(q->data);
  p.offs = static_cast<const uint32_t*>(input_row_offsets->data);
  p.blocks = kv->blocks.data;
  p.scales = fp8 ? static_cast<const float*>(kv->scales.data) : nullptr;
  p.cache_len = kv->cache_lengths;
  p.page_table = kv->page_table;
  p.workspace = static_cast<float*>(workspace->data);
  p.T = T;
  p.max_pages = kv->max_pages_per_seq;
  p.pages = P;
  p.batch = (int)B;
  p.hq = (int)Hq;
  p.hkv = (int)Hkv;
  p.group = (int)(Hq / Hkv);
  p.d = (int)D;
  p.page_size = (int)S;
  p.layer = (int)layer_idx;
  p.gran = fp8 ? (int)kv->quantization_granularity : 0;
  p.causal = causal ? 1 : 0;
  p.window = window;
  p.fp8 = fp8 ? 1 : 0;
  p.num_cus = device_cus();
  p.scale = scale;
  if (tree) {
    p.tree = static_cast<const uint32_t*>(tree_mask->data);
    p.tree_words = (int)tree_mask->shape[1];
  }
  return launch_status(qg::launch_attention_paged(p, stream));
}

qg_status attention_ragged_paged(const qg_tensor* out, const qg_tensor* q, const qg_tensor* input_row_offsets,
                                 const qg_paged_kv* kv, uint32_t layer_idx, float scale, int32_t causal,
                                 int32_t window, const qg_tensor* workspace, hipStream_t stream) {
  return attention_impl(out, q, input_row_offsets, nullptr, kv, layer_idx, scale, causal, window, workspace, false, stream);
}

qg_status attention_tree_ragged_paged(const qg_tensor* out, const qg_tensor* q, const qg_tensor* input_row_offsets,
                                      const qg_tensor* tree_mask, const qg_paged_kv* kv, uint32_t layer_idx,
                                      float scale, int32_t window, const qg_tensor* workspace, hipStream_t stream) {
  return attention_impl(out, q, input_row_offsets, tree_mask, kv, layer_idx, scale, 0, window, workspace, true, stream);
}

}  // extern "C"
