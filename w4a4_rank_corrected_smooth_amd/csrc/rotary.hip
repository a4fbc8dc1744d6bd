// Rotary positions with several axes.
//
//  rotary_kernel    query and key rows turned by their tokens' positions
//
// A workgroup takes a few tokens.  It first finds the sine and cosine of every
// (token, pair), each once, in LDS, and then turns all heads of these tokens by them:
// the float64 angles cost a pair's 40 instructions once for all its heads.
// Bound by memory where a lane takes 16 bytes: every value is read and written once (32760 tokens of 24 heads of 128,
// 403 MB: 80 us as neighbours, 82 as halves, 5.0 TB/s; a plain copy 4.95).  Halves whose pairs are no multiple of 8
// go by 8 bytes (28 pairs of 128 channels, the same rows: 112 us) or, if none of 4, by single channels
// (18 pairs of 72 channels in 48 heads, 453 MB: 328 us, where a copy takes 92).  A decode step's launch (8 tokens, 40 heads) takes 3.2 us.
#include <hip/hip_runtime.h>

#include "common.h"
#include "device_util.h"

using namespace svdq;

namespace {

constexpr int kRotaryTable = 1024;     // (token, pair) entries of a workgroup at most

struct RotaryRows {
  const uint16_t *in;
  uint16_t *out;
  int64_t in_row, in_head, out_row, out_head;
};
struct RotaryArgs {
  RotaryRows q, k;
  const void *positions;
  int T, tokens;                       // rows; rows of a workgroup
  int q_heads, heads;                  // query heads; all heads
  int heads_part;                      // heads of a workgroup (blockIdx.y counts the parts)
  int pairs, axes, items;              // items: pieces of V channels (or pairs) of a row
  double turns[SVDQ_ROTARY_MAX_PAIRS]; // freq / 2 pi
  uint8_t axis[SVDQ_ROTARY_MAX_PAIRS];
};

// (cos, sin) of `t` turns: the nearest quarter is taken off in float64, which is exact, and the rest, at
// most pi / 4, goes through the Taylor series (their next terms are below 2^-28).
__device__ __forceinline__ float2 cos_sin(double t) {
  const double r = t - rint(t);                      // [-1/2, 1/2]
  const double quarter = rint(4.0 * r);
  const float x = (float)((r - 0.25 * quarter) * 6.283185307179586476925);
  const float z = x * x;
  float s = __builtin_fmaf(z, 2.75573192e-6f, -1.98412698e-4f);
  s = __builtin_fmaf(z, s, 8.33333333e-3f);
  s = __builtin_fmaf(z, s, -1.66666667e-1f);
  s = __builtin_fmaf(x * z, s, x);
  float c = __builtin_fmaf(z, -2.75573192e-7f, 2.48015873e-5f);
  c = __builtin_fmaf(z, c, -1.38888889e-3f);
  c = __builtin_fmaf(z, c, 4.16666667e-2f);
  c = __builtin_fmaf(z, c, -0.5f);
  c = __builtin_fmaf(z, c, 1.0f);
  const int n = (int)quarter & 3;                    // NaN and infinite positions leave NaN in x
  const float a = n & 1 ? s : c, b = n & 1 ? c : s;
  return make_float2(n == 1 || n == 2 ? -a : a, n >= 2 ? -b : b);
}

template <bool F16>
__device__ __forceinline__ float widen(uint32_t h) {
  if constexpr (F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  else return __uint_as_float(h << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t narrow(float f) {
  if constexpr (F16) return __builtin_bit_cast(uint16_t, (_Float16)f);
  else return __builtin_bit_cast(uint16_t, (__bf16)f);
}

template <int V>
struct Piece { uint16_t h[V]; };
template <>
struct alignas(16) Piece<8> { uint16_t h[8]; };
template <>
struct alignas(8) Piece<4> { uint16_t h[4]; };

template <bool F16>
__device__ __forceinline__ void turn(uint16_t &a, uint16_t &b, float2 cs) {
  const float x = widen<F16>(a), y = widen<F16>(b);
  a = narrow<F16>(__builtin_fmaf(x, cs.x, -(y * cs.y)));
  b = narrow<F16>(__builtin_fmaf(x, cs.y, y * cs.x));
}

// V: channels that a lane reads at a time.  Neighbouring pairs: items of 8
// channels, 8 always.  Halves: items of V pairs, V channels from each half, and behind
// them items of V channels that stay; V = 8, 4 or 1 as it divides the pairs.
template <bool F16, bool PAIRED, int V, bool FLOATS>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryArgs a) {
  __shared__ float2 table[kRotaryTable];
  const int t0 = blockIdx.x * a.tokens, tokens = min(a.tokens, a.T - t0);
  for (int i = threadIdx.x; i < tokens * a.pairs; i += 256) {
    const int t = i / a.pairs, j = i - t * a.pairs;
    const int64_t at = (int64_t)(t0 + t) * a.axes + a.axis[j];
    const double p = FLOATS ? (double)static_cast<const float *>(a.positions)[at]
                            : (double)static_cast<const int *>(a.positions)[at];
    table[i] = cos_sin(p * a.turns[j]);
  }
  __syncthreads();
  const int h0 = blockIdx.y * a.heads_part, heads = min(a.heads_part, a.heads - h0);
  const int turned = PAIRED ? (2 * a.pairs + 7) / 8 : a.pairs / V;
  const int rows = tokens * heads;
  for (int i = threadIdx.x; i < rows * a.items; i += 256) {
    const int r = (int)((uint32_t)i / (uint32_t)a.items), c = i - r * a.items;
    const int t = (int)((uint32_t)r / (uint32_t)heads), h = h0 + r - t * heads;
    const bool is_q = h < a.q_heads;
    const int hh = is_q ? h : h - a.q_heads;
    const uint16_t *in = (is_q ? a.q.in : a.k.in) + (int64_t)(t0 + t) * (is_q ? a.q.in_row : a.k.in_row) +
                         hh * (is_q ? a.q.in_head : a.k.in_head);
    uint16_t *out = (is_q ? a.q.out : a.k.out) + (int64_t)(t0 + t) * (is_q ? a.q.out_row : a.k.out_row) +
                    hh * (is_q ? a.q.out_head : a.k.out_head);
    const float2 *cs = table + t * a.pairs;
    typedef Piece<V> P;
    if constexpr (PAIRED) {
      P p = *reinterpret_cast<const P *>(in + V * c);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const int j = V / 2 * c + e;
        if (j < a.pairs) turn<F16>(p.h[2 * e], p.h[2 * e + 1], cs[j]);
      }
      *reinterpret_cast<P *>(out + V * c) = p;
    } else if (c < turned) {
      P p = *reinterpret_cast<const P *>(in + V * c), o = *reinterpret_cast<const P *>(in + a.pairs + V * c);
#pragma unroll
      for (int e = 0; e < V; ++e) turn<F16>(p.h[e], o.h[e], cs[V * c + e]);
      *reinterpret_cast<P *>(out + V * c) = p;
      *reinterpret_cast<P *>(out + a.pairs + V * c) = o;
    } else {
      const int at = 2 * a.pairs + V * (c - turned);
      *reinterpret_cast<P *>(out + at) = *reinterpret_cast<const P *>(in + at);
    }
  }
}

}  // namespace

extern "C" {

svdq_status_t svdq_rotary_apply(const svdq_rotary_t *plan, const void *q, int64_t q_row, int64_t q_head, int q_heads,
                                void *q_out, int64_t q_out_row, int64_t q_out_head, const void *k, int64_t k_row,
                                int64_t k_head, int k_heads, void *k_out, int64_t k_out_row, int64_t k_out_head,
                                svdq_dtype_t dtype, const void *positions, int float_positions, int T,
                                void *hip_stream) {
  const char *who = "svdq_rotary_apply";
  if (!plan) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL plan", who);
  const int D = plan->head_dim, pairs = plan->pairs;
  if (D < 8 || D > 2 * SVDQ_ROTARY_MAX_PAIRS || D % 8 != 0 || pairs < 1 || 2 * pairs > D || plan->axes < 1 ||
      plan->axes > SVDQ_ROTARY_MAX_AXES)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: plan of %d pairs in %d channels, %d axes", who, pairs, D, plan->axes);
  for (int j = 0; j < pairs; ++j)
    if (plan->axis[j] >= plan->axes || !__builtin_isfinite(plan->freq[j]))
      return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: pair %d has axis %d of %d and frequency %g", who, j, plan->axis[j],
                  plan->axes, plan->freq[j]);
  if (dtype != SVDQ_BF16 && dtype != SVDQ_FP16)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: dtype must be SVDQ_BF16 or SVDQ_FP16", who);
  if (T < 0 || q_heads < 0 || k_heads < 0 || (int64_t)q_heads + k_heads > 65536 ||
      (int64_t)T * (q_heads + k_heads) * D > (int64_t)1 << 34)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: T=%d with %d and %d heads of %d channels", who, T, q_heads, k_heads, D);
  const int heads = q_heads + k_heads;
  if (T == 0 || heads == 0) return SVDQ_OK;
  if ((q_heads && (!q || !q_out)) || (k_heads && (!k || !k_out)) || !positions)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL pointer", who);
  RotaryArgs a{};
  if (q_heads) a.q = {static_cast<const uint16_t *>(q), static_cast<uint16_t *>(q_out), q_row, q_head, q_out_row, q_out_head};
  if (k_heads) a.k = {static_cast<const uint16_t *>(k), static_cast<uint16_t *>(k_out), k_row, k_head, k_out_row, k_out_head};
  for (const RotaryRows *r : {&a.q, &a.k})
    for (int64_t s : {r->in_row, r->in_head, r->out_row, r->out_head})
      if (s < 0 || s % 8 != 0 || !aligned16(r->in) || !aligned16(r->out))
        return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: misaligned pointer, or a stride that is not a multiple of 8", who);
  if ((uintptr_t)positions & 3u) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: misaligned positions", who);
  svdq_status_t st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  const bool paired = plan->interleaved != 0;
  const int V = paired || pairs % 8 == 0 ? 8 : pairs % 4 == 0 ? 4 : 1;
  a.positions = positions;
  a.T = T;
  a.q_heads = q_heads;
  a.heads = heads;
  a.pairs = pairs;
  a.axes = plan->axes;
  a.items = paired ? D / 8 : pairs / V + (D - 2 * pairs) / V;
  for (int j = 0; j < pairs; ++j) {
    a.turns[j] = plan->freq[j] * 0.15915494309189533577;
    a.axis[j] = plan->axis[j];
  }
  // as many tokens as give every lane an angle, and more where the heads are few
  const int64_t token_items = (int64_t)heads * a.items;
  int tokens = (256 + pairs - 1) / pairs;
  while (tokens * token_items < 1024 && 2 * tokens * pairs <= kRotaryTable) tokens *= 2;
  if (tokens > T) tokens = T;
  const int64_t tiles = ((int64_t)T + tokens - 1) / tokens;
  // few tokens: the heads in parts, so that the work is on many CUs (a workgroup's items then are below 2^28)
  int parts = 1;
  while (tiles * parts < 512 && heads / (2 * parts) >= 1 && (int64_t)tokens * (heads / (2 * parts)) * a.items >= 256) parts *= 2;
  a.tokens = tokens;
  a.heads_part = (heads + parts - 1) / parts;
  const dim3 grid((unsigned)tiles, (unsigned)((heads + a.heads_part - 1) / a.heads_part));
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
#define ROTARY_GO(FF, PP, VV)                                                                                   \
  do {                                                                                                          \
    if (float_positions) hipLaunchKernelGGL((rotary_kernel<FF, PP, VV, true>), grid, dim3(256), 0, stream, a);  \
    else hipLaunchKernelGGL((rotary_kernel<FF, PP, VV, false>), grid, dim3(256), 0, stream, a);                 \
  } while (0)
#define ROTARY_TYPE(FF)                    \
  do {                                     \
    if (paired) ROTARY_GO(FF, true, 8);    \
    else if (V == 8) ROTARY_GO(FF, false, 8); \
    else if (V == 4) ROTARY_GO(FF, false, 4); \
    else ROTARY_GO(FF, false, 1);          \
  } while (0)
  if (dtype == SVDQ_FP16) ROTARY_TYPE(true);
  else ROTARY_TYPE(false);
#undef ROTARY_TYPE
#undef ROTARY_GO
  return launch_status("rotary launch");
}

}  // extern "C"
