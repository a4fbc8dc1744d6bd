// Host half of the C ABI: status strings, the thread-local error, offline
// preparation, packing and size queries.  No HIP calls here.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>

#include "common.h"
#include "cross_layout.h"
#include "fp8_layout.h"
#include "host_prepare.h"
#include "kv4_layout.h"
#include "layout.h"
#include "moe_layout.h"

namespace svdq {

static thread_local char g_last_error[512] = "";

svdq_status_t fail(svdq_status_t s, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

static bool shape_ok(int N, int K, int rank, const char *who, svdq_status_t *st) {
  if (N < 1 || K < 1) {
    *st = fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: N=%d K=%d must be >= 1", who, N, K);
    return false;
  }
  if (K % kGroup != 0) {
    *st = fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: K=%d is not a multiple of 64", who, K);
    return false;
  }
  if (rank < 0 || rank > N || rank > K || rank > SVDQ_MAX_RANK) {
    *st = fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: rank=%d outside [0, min(N=%d, K=%d, %d)]", who,
               rank, N, K, SVDQ_MAX_RANK);
    return false;
  }
  if ((int64_t)N * K > (int64_t)1 << 31) {
    *st = fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: N*K=%lld exceeds 2^31", who,
               (long long)N * K);
    return false;
  }
  return true;
}

static bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

static void copy_unless_same(void *dst, const void *src, size_t bytes) {
  if (dst != src && bytes) std::memmove(dst, src, bytes);
}

// Shared checks and the factor merge of svdq_merge_lora / svdq_mx_merge_lora.
template <typename HW>
static svdq_status_t merge_lora_checked(const HW *in, const uint16_t *A, const uint16_t *B, int r2,
                                        float alpha, HW *out, const char *who) {
  svdq_status_t st;
  if (!in || !out) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL weights", who);
  if (r2 < 0) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: lora_rank=%d < 0", who, r2);
  if (r2 > 0 && (!A || !B)) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL LoRA factor", who);
  const int N = in->N, K = in->K, r = in->rank;
  if (!shape_ok(N, K, r, who, &st)) return st;
  if (r + r2 > SVDQ_MAX_RANK || r + r2 > N || r + r2 > K)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: merged rank %d + %d outside [0, min(N=%d, K=%d, %d)]",
                who, r, r2, N, K, SVDQ_MAX_RANK);
  if (!in->inv_lambda || !in->qweight || !in->wscales || !in->bias || (r > 0 && (!in->l1s || !in->l2)))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL input buffer", who);
  const int rt = r + r2;
  if (!out->inv_lambda || !out->qweight || !out->wscales || !out->bias ||
      (rt > 0 && (!out->l1s || !out->l2)))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL output buffer", who);
  const size_t f_in = 2 * (size_t)K * r, u_in = 2 * (size_t)r * N;
  const size_t f_out = 2 * (size_t)K * rt, u_out = 2 * (size_t)rt * N;
  if (overlaps(out->l1s, f_out, in->l1s, f_in) || overlaps(out->l1s, f_out, in->l2, u_in) ||
      overlaps(out->l2, u_out, in->l1s, f_in) || overlaps(out->l2, u_out, in->l2, u_in) ||
      overlaps(out->l1s, f_out, out->l2, u_out))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: output factors overlap the input factors", who);
  st = merge_lora_factors(N, K, r, in->l1s, in->l2, A, B, r2, alpha, out->l1s, out->l2);
  if (st != SVDQ_OK) return st;
  copy_unless_same(out->inv_lambda, in->inv_lambda, sizeof(float) * (size_t)K);
  copy_unless_same(out->bias, in->bias, sizeof(float) * (size_t)N);
  copy_unless_same(out->qweight, in->qweight, (size_t)N * K / 2);
  out->N = N;
  out->K = K;
  out->rank = rt;
  return SVDQ_OK;
}

}  // namespace svdq

using namespace svdq;

extern "C" {

int svdq_abi_version(void) { return SVDQ_ABI_VERSION; }

const char *svdq_status_string(svdq_status_t s) {
  switch (s) {
    case SVDQ_OK: return "ok";
    case SVDQ_ERR_INVALID_ARGUMENT: return "invalid argument";
    case SVDQ_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case SVDQ_ERR_NO_DEVICE: return "no HIP device";
    case SVDQ_ERR_UNSUPPORTED_DEVICE: return "unsupported device (gfx950 required)";
    case SVDQ_ERR_WORKSPACE_TOO_SMALL: return "workspace or buffer too small";
    case SVDQ_ERR_NUMERICAL: return "non-finite input";
    case SVDQ_ERR_HIP: return "HIP runtime error";
  }
  return "unknown status";
}

const char *svdq_last_error(void) { return g_last_error; }

svdq_status_t svdq_host_weights_sizes(int N, int K, int rank, size_t sizes_out[6]) {
  svdq_status_t st;
  if (!sizes_out) return fail(SVDQ_ERR_INVALID_ARGUMENT, "sizes_out is NULL");
  if (!shape_ok(N, K, rank, "svdq_host_weights_sizes", &st)) return st;
  sizes_out[0] = sizeof(float) * (size_t)K;
  sizes_out[1] = 2 * (size_t)K * rank;
  sizes_out[2] = 2 * (size_t)rank * N;
  sizes_out[3] = (size_t)N * K / 2;
  sizes_out[4] = sizeof(float) * (size_t)N * (K / kGroup);
  sizes_out[5] = sizeof(float) * (size_t)N;
  return SVDQ_OK;
}

svdq_status_t svdq_calibration_absmax(const uint16_t *X, int rows, int K, float *absmax) {
  if (!X || !absmax) return fail(SVDQ_ERR_INVALID_ARGUMENT, "NULL pointer");
  if (rows < 1 || K < 1) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "rows=%d K=%d", rows, K);
  for (int k = 0; k < K; ++k) absmax[k] = 0.0f;
  for (int64_t i = 0; i < rows; ++i)
    for (int k = 0; k < K; ++k) {
      const float v = std::fabs(bf16_to_f32(X[i * K + k]));
      if (!std::isfinite(v)) return fail(SVDQ_ERR_NUMERICAL, "non-finite calibration value");
      if (v > absmax[k]) absmax[k] = v;
    }
  return SVDQ_OK;
}

svdq_status_t svdq_prepare_weights(const uint16_t *W, int N, int K, const float *act_absmax,
                                   const uint16_t *bias, int rank, int group_size,
                                   svdq_host_weights_t *out) {
  svdq_status_t st;
  if (!W || !out) return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_prepare_weights: NULL pointer");
  if (group_size != kGroup)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "group_size=%d (only 64 is supported)", group_size);
  if (!shape_ok(N, K, rank, "svdq_prepare_weights", &st)) return st;
  if (!out->inv_lambda || !out->qweight || !out->wscales || !out->bias ||
      (rank > 0 && (!out->l1s || !out->l2)))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_prepare_weights: NULL output buffer");
  return prepare_weights(W, N, K, act_absmax, bias, rank, out);
}

size_t svdq_device_weights_bytes(int N, int K, int rank) {
  svdq_status_t st;
  if (!shape_ok(N, K, rank, "svdq_device_weights_bytes", &st)) return 0;
  return (size_t)WeightLayout(N, K, rank).total;
}

svdq_status_t svdq_pack_device_weights(const svdq_host_weights_t *in, void *blob, size_t bytes) {
  svdq_status_t st;
  if (!in || !blob) return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_pack_device_weights: NULL");
  if (!shape_ok(in->N, in->K, in->rank, "svdq_pack_device_weights", &st)) return st;
  if (in->group_size != kGroup) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "group_size must be 64");
  if (!in->inv_lambda || !in->qweight || !in->wscales || !in->bias ||
      (in->rank > 0 && (!in->l1s || !in->l2)))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_pack_device_weights: NULL input buffer");
  return pack_device_weights(in, blob, bytes);
}

svdq_status_t svdq_merge_lora(const svdq_host_weights_t *in, const uint16_t *lora_down_bf16,
                              const uint16_t *lora_up_bf16, int lora_rank, float alpha,
                              svdq_host_weights_t *out) {
  if (in && in->group_size != kGroup)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_merge_lora: group_size=%d (64 only)", in->group_size);
  const svdq_status_t st = merge_lora_checked(in, lora_down_bf16, lora_up_bf16, lora_rank, alpha,
                                              out, "svdq_merge_lora");
  if (st != SVDQ_OK) return st;
  copy_unless_same(out->wscales, in->wscales, sizeof(float) * (size_t)in->N * (in->K / kGroup));
  out->group_size = kGroup;
  return SVDQ_OK;
}

svdq_status_t svdq_mx_host_weights_sizes(int N, int K, int rank, size_t sizes_out[6]) {
  svdq_status_t st;
  if (!sizes_out) return fail(SVDQ_ERR_INVALID_ARGUMENT, "sizes_out is NULL");
  if (!shape_ok(N, K, rank, "svdq_mx_host_weights_sizes", &st)) return st;
  sizes_out[0] = sizeof(float) * (size_t)K;
  sizes_out[1] = 2 * (size_t)K * rank;
  sizes_out[2] = 2 * (size_t)rank * N;
  sizes_out[3] = (size_t)N * K / 2;
  sizes_out[4] = (size_t)N * (K / kMxBlock);
  sizes_out[5] = sizeof(float) * (size_t)N;
  return SVDQ_OK;
}

svdq_status_t svdq_mx_prepare_weights(const uint16_t *W, int N, int K, const float *act_absmax,
                                      const uint16_t *bias, int rank, svdq_mx_host_weights_t *out) {
  svdq_status_t st;
  if (!W || !out) return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_mx_prepare_weights: NULL pointer");
  if (!shape_ok(N, K, rank, "svdq_mx_prepare_weights", &st)) return st;
  if (!out->inv_lambda || !out->qweight || !out->wscales || !out->bias ||
      (rank > 0 && (!out->l1s || !out->l2)))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_mx_prepare_weights: NULL output buffer");
  return prepare_weights_mx(W, N, K, act_absmax, bias, rank, out);
}

size_t svdq_mx_device_weights_bytes(int N, int K, int rank) {
  svdq_status_t st;
  if (!shape_ok(N, K, rank, "svdq_mx_device_weights_bytes", &st)) return 0;
  return (size_t)MxWeightLayout(N, K, rank).total;
}

svdq_status_t svdq_mx_pack_device_weights(const svdq_mx_host_weights_t *in, void *blob, size_t bytes) {
  svdq_status_t st;
  if (!in || !blob) return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_mx_pack_device_weights: NULL");
  if (!shape_ok(in->N, in->K, in->rank, "svdq_mx_pack_device_weights", &st)) return st;
  if (!in->inv_lambda || !in->qweight || !in->wscales || !in->bias ||
      (in->rank > 0 && (!in->l1s || !in->l2)))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_mx_pack_device_weights: NULL input buffer");
  return pack_device_weights_mx(in, blob, bytes);
}

svdq_status_t svdq_mx_merge_lora(const svdq_mx_host_weights_t *in, const uint16_t *lora_down_bf16,
                                 const uint16_t *lora_up_bf16, int lora_rank, float alpha,
                                 svdq_mx_host_weights_t *out) {
  const svdq_status_t st = merge_lora_checked(in, lora_down_bf16, lora_up_bf16, lora_rank, alpha,
                                              out, "svdq_mx_merge_lora");
  if (st != SVDQ_OK) return st;
  copy_unless_same(out->wscales, in->wscales, (size_t)in->N * (in->K / kMxBlock));
  return SVDQ_OK;
}

size_t svdq_mx_workspace_bytes(int M, int N, int K, int rank) {
  svdq_status_t st;
  if (M < 1 || !shape_ok(N, K, rank, "svdq_mx_workspace_bytes", &st)) return 0;
  return (size_t)MxWorkLayout(M, K, rank).total;
}

size_t svdq_workspace_bytes(int M, int N, int K, int rank) {
  svdq_status_t st;
  if (M < 1 || !shape_ok(N, K, rank, "svdq_workspace_bytes", &st)) return 0;
  return (size_t)(WorkLayout(M, K, rank).total + k2_split_bytes(M, N, K));
}

svdq_status_t awq_quantize_weights(const uint16_t *W, int N, int K, int group_size, uint8_t *q,
                                   uint16_t *s, uint16_t *z) {
  svdq_status_t st;
  if (!W || !q || !s || !z) return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_quantize_weights: NULL");
  if (group_size != kGroup) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "group_size must be 64");
  if (!shape_ok(N, K, 0, "awq_quantize_weights", &st)) return st;
  return awq_quantize(W, N, K, q, s, z);
}

size_t awq_device_weights_bytes(int N, int K) {
  svdq_status_t st;
  if (!shape_ok(N, K, 0, "awq_device_weights_bytes", &st)) return 0;
  return (size_t)AwqLayout(N, K).total;
}

svdq_status_t awq_pack_device_weights(const uint8_t *q, const uint16_t *s, const uint16_t *z,
                                      int N, int K, void *blob, size_t bytes) {
  svdq_status_t st;
  if (!q || !s || !z || !blob) return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_pack: NULL");
  if (!shape_ok(N, K, 0, "awq_pack_device_weights", &st)) return st;
  return awq_pack(q, s, z, N, K, blob, bytes);
}

size_t svdq_kv4_cache_bytes(int num_pages, int page_size, int kv_heads, int head_dim) {
  if (!kv4_shape_ok(num_pages, page_size, kv_heads, head_dim)) {
    fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_cache_bytes: %d pages of %d tokens, %d heads of %d channels", num_pages,
         page_size, kv_heads, head_dim);
    return 0;
  }
  return (size_t)Kv4Layout(num_pages, page_size, kv_heads, head_dim).total();
}

size_t svdq_kv4_attention_workspace_bytes(int B, int Q, int Hq, int kv_heads, int head_dim) {
  if (!kv4_shape_ok(1, 16, kv_heads, head_dim) || !kv4_query_ok(B, Q, Hq, kv_heads)) {
    fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_attention_workspace_bytes: B=%d Q=%d Hq=%d over %d heads of %d channels",
         B, Q, Hq, kv_heads, head_dim);
    return 0;
  }
  return (size_t)kv4_workspace_bytes(Q, Hq, kv_heads, head_dim);
}

size_t svdq_fp8_device_weights_bytes(int N, int K) {
  if (!fp8_weights_ok(N, K)) {
    fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_fp8_device_weights_bytes: N=%d K=%d", N, K);
    return 0;
  }
  return (size_t)fp8_w_bytes(N, K);
}

size_t svdq_fp8_workspace_bytes(int M, int N, int K) {
  if (!fp8_weights_ok(N, K) || !fp8_call_ok(M, N) || !fp8_call_ok(M, K)) {
    fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_fp8_workspace_bytes: M=%d N=%d K=%d", M, N, K);
    return 0;
  }
  const size_t n = M > 0 ? (size_t)fp8_plan(M, N, K).total : 0;
  return n > 0 ? n : 1;        // 0 is for errors
}

svdq_status_t svdq_fp8_quantize_weights(const float *W, int N, int K, uint8_t *codes, float *scales) {
  const char *who = "svdq_fp8_quantize_weights";
  if (!W || !codes || !scales) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL pointer", who);
  if (!fp8_weights_ok(N, K)) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: N=%d K=%d", who, N, K);
  try {
    return fp8_quantize(W, N, K, codes, scales);
  } catch (const std::exception &e) {       // the thread pool could not start
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: %s", who, e.what());
  }
}

svdq_status_t svdq_rotary_plan(int head_dim, const int32_t *widths, int axes, double theta, int interleaved,
                               int per_axis, svdq_rotary_t *plan) {
  const char *who = "svdq_rotary_plan";
  if (!widths || !plan) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL pointer", who);
  if (head_dim < 8 || head_dim % 8 != 0 || head_dim > 2 * SVDQ_ROTARY_MAX_PAIRS || axes < 1 || axes > SVDQ_ROTARY_MAX_AXES)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: head_dim=%d with %d axes", who, head_dim, axes);
  if (!(theta > 0.0) || !std::isfinite(theta)) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: theta=%g", who, theta);
  int64_t turned = 0;
  for (int a = 0; a < axes; ++a) {
    if (widths[a] < 2 || widths[a] % 2 != 0)
      return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: axis %d of %d channels", who, a, widths[a]);
    turned += widths[a];
  }
  if (turned > head_dim)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: axes of %lld channels in %d", who, (long long)turned, head_dim);
  *plan = svdq_rotary_t{};
  plan->head_dim = head_dim;
  plan->axes = axes;
  plan->interleaved = interleaved != 0;
  int j = 0;
  for (int a = 0; a < axes; ++a)
    for (int i = 0; i < widths[a] / 2; ++i, ++j) {
      plan->axis[j] = (uint8_t)a;
      plan->freq[j] = std::pow(theta, per_axis ? -2.0 * i / widths[a] : -2.0 * j / (double)turned);
      if (!std::isfinite(plan->freq[j])) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: theta=%g", who, theta);
    }
  plan->pairs = j;
  return SVDQ_OK;
}

size_t svdq_cross_attention_workspace_bytes(int B, int Lq, int Lk, int Hq, int Hkv, int D, int masked) {
  if (!cross_shape_ok(B, Lq, Lk, Hq, Hkv, D)) {
    fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_cross_attention_workspace_bytes: B=%d Lq=%d Lk=%d, %d heads over %d of %d channels",
         B, Lq, Lk, Hq, Hkv, D);
    return 0;
  }
  const size_t n = (size_t)cross_plan(B, Lq, Lk, Hq, Hkv, D, masked != 0).total;
  return n > 0 ? n : 1;        // 0 is for errors
}

size_t svdq_moe_route_workspace_bytes(int T, int E) {
  if (!moe_route_ok(T, E, 8, 1)) {
    fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_moe_route_workspace_bytes: T=%d E=%d", T, E);
    return 0;
  }
  return (size_t)round_up((T > 0 ? T : 1) * (int64_t)E * 8, kAlign);
}

size_t awq_moe_workspace_bytes(int T, int top_k, int K, int I) {
  if (!moe_weights_ok(1, K, I) || !moe_call_ok(T, top_k)) {
    fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "awq_moe_workspace_bytes: T=%d top_k=%d K=%d I=%d", T, top_k, K, I);
    return 0;
  }
  return (size_t)MoeWork(T > 0 ? T : 1, top_k, K, I).total;
}

static bool moe_linear_ok(int E, int N, int K, const char *who) {
  if (E >= 1 && E <= MOE_MAX_EXPERTS && N >= kGroup && N % kGroup == 0 && K >= kGroup && K % kGroup == 0 &&
      (int64_t)N * K <= (int64_t)1 << 31)
    return true;
  fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: E=%d N=%d K=%d (E in 1..%d, N and K multiples of 64)", who, E, N, K,
       MOE_MAX_EXPERTS);
  return false;
}

size_t awq_moe_device_weights_bytes(int E, int N, int K) {
  return moe_linear_ok(E, N, K, "awq_moe_device_weights_bytes") ? (size_t)(E * MoeWeightLayout(N, K).total) : 0;
}

svdq_status_t awq_moe_pack_device_weights(const uint8_t *q, const uint16_t *s, const uint16_t *z, int E, int N, int K,
                                          void *host_blob, size_t bytes) {
  if (!q || !s || !z || !host_blob) return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_pack_device_weights: NULL");
  if (!moe_linear_ok(E, N, K, "awq_moe_pack_device_weights")) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  try {
    return awq_moe_pack(q, s, z, E, N, K, host_blob, bytes);
  } catch (const std::exception &e) {       // the thread pool could not start
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_pack_device_weights: %s", e.what());
  }
}

}  // extern "C"
