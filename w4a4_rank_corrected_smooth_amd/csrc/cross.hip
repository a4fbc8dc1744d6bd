// Cross attention: queries over an encoder's states of another length.
//
//  cross_list_kernel     the visible states of each batch row, where there is a mask
//  cross_attend_kernel   attention of a tile of rows over a piece of the states
//  cross_join_kernel     joins the pieces of a row
//
// One pass over the states with a running maximum m and sum l (float32, in units
// of log2): S^T = K Q^T on 32x32x16 matrix instructions, P^T = 2^(c S^T - m),
// O^T += V^T P^T.  A lane's column of all three is one row (a query of a head),
// so maximum, sum and rescaling are one value a lane, shared with the
// lane 32 further, which holds the column's other half; and the 16 scores of a
// block of 32 states are, in the lane that has them, the contraction slots
// that the second product wants there: slots 0..7 of half u of the block in lane
// half h are the states 16 u + 4 h + [0, 4) and 16 u + 8 + 4 h + [0, 4).  P never
// leaves the registers.
//
// K and V tiles are copied into LDS as they lie in memory (rows of 16-byte
// chunks, global_load_lds), the chunks of a row permuted so that no read meets
// a bank twice: K rows are read as operand rows, V columns through the
// transposing read (ds_read_b64_tr_b16: lane i of 16 gets column i of 4 rows).
// Rows behind the last state repeat it; their scores are set to -inf and their V
// rows in LDS to zero.  With a mask, rows are fetched through the list of the
// visible ones, so nothing else in the kernel knows of it.
#include <hip/hip_runtime.h>

#include "common.h"
#include "cross_layout.h"
#include "device_util.h"

using namespace svdq;

namespace {

typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef short v4i16 __attribute__((ext_vector_type(4)));

constexpr float kLowest = -3.0e38f;      // the maximum of a row that has met no score above -inf
// How far (log2) scores may pass the running maximum before the sums are
// rescaled: 2^8 more is no loss in float32, and nearly all tiles go without.
constexpr float kSlack = 8.0f;
// float16 weights are p 2^7, at most 2^15 with the slack: the type's smallest step is then at most
// 2^-31 of the largest weight, so that many small ones do not vanish.
constexpr float kShift16 = 7.0f;

struct CrossArgs {
  const uint16_t *q, *k, *v;
  int64_t q_b, q_i, q_h, k_b, k_t, k_h, v_b, v_t, v_h;
  const int *lens;                       // visible states of a batch row (or NULL: all)
  const int *index;                      // [B, Lk] their numbers, where there is a mask
  uint16_t *out;
  float *ml, *o;                         // pieces: [piece][B Hkv][row] (m, l), and [..][D]
  int B, Lq, Lk, Hq, Hkv, group, D, rows, tiles, parts;
  int64_t work, per_xcd;
  float c;
  uint32_t flip;
};

template <bool F16>
__device__ __forceinline__ v16f mma(v4u a, v4u b, v16f c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (F16) {
    const v2h h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
  } else {
    const v2b h = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, h);
  }
}
// the value and that of the lane 32 further, both halves alike
__device__ __forceinline__ float half_max(float x) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// The tiles' place in LDS, for blocks of 32 channels DB: rows of SLOTS chunks of 16 bytes.
template <int DB, int KEYS>
struct Tile {
  static constexpr int SLOTS = DB <= 2 ? 8 : DB <= 4 ? 16 : 32;
  static constexpr int ROW = SLOTS * 16, HALF = KEYS * ROW, BYTES = 2 * HALF;   // K, then V
  static constexpr int COPY_ROWS = 64 / SLOTS;                                  // rows of one copy
  // A chunk's slot is the chunk xor this.  K: 8 or 16 neighbouring rows are read
  // at the same chunk.  V: 4 neighbouring rows at 4 neighbouring chunks.
  static __device__ __forceinline__ int k_swap(int row) { return SLOTS == 8 ? row >> 1 & 7 : SLOTS == 16 ? row & 15 : row & 7; }
  static __device__ __forceinline__ int v_swap(int row) { return SLOTS == 8 ? (row >> 1 & 1) << 2 : (row & 3) << 2; }
};

// DB: blocks of 32 channels.  KEYS: states of a tile.  OWN: the four wavefronts
// share 32 rows and take tiles of their own, in LDS of their own, without barriers;
// otherwise each has 32 rows and all read the same tiles.
template <int DB, int KEYS, bool OWN, bool F16, bool LIST>
__global__ __launch_bounds__(256, OWN && DB > 2 ? 1 : 2) void cross_attend_kernel(const CrossArgs a) {
  typedef Tile<DB, KEYS> L;
  constexpr int KB = KEYS / 32, STEPS = 2 * DB;
  constexpr int COPIES = KEYS / L::COPY_ROWS / (OWN ? 1 : 4);     // copies of K (and of V) that a wavefront makes for a tile
  __shared__ __attribute__((aligned(1024))) uint8_t lds[(OWN ? 4 : 1) * 2 * L::BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Neighbouring pieces of work, which read the same states, go to one XCD (workgroups
  // are dealt out to the eight in turn).
  const int64_t id = (int64_t)(blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
  if (id >= a.work) return;
  const int tile_row = (int)(id % a.tiles), part = (int)(id / a.tiles % a.parts);
  const int64_t bh = id / a.tiles / a.parts;
  const int b = (int)(bh / a.Hkv), hk = (int)(bh - (int64_t)b * a.Hkv);
  int n = a.lens ? min(max(a.lens[b], 0), a.Lk) : a.Lk;
  const int all = (n + KEYS - 1) / KEYS;                           // tiles
  int t0 = (int)((int64_t)all * part / a.parts), t1 = (int)((int64_t)all * (part + 1) / a.parts);
  if constexpr (OWN) t0 += w;
  constexpr int STRIDE = OWN ? 4 : 1;

  // this lane's row and the queries' operand
  const int m = lane & 31, h = lane >> 5;
  const int row = tile_row * (OWN ? 32 : 128) + (OWN ? 0 : 32 * w) + m;
  const int rr = min(row, a.rows - 1), qi = rr / a.group, hq = hk * a.group + rr - qi * a.group;
  v4u q[STEPS];
  {
    const uint16_t *src = a.q + (int64_t)b * a.q_b + qi * a.q_i + hq * a.q_h;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int at = 16 * s + 8 * h;
      q[s] = at < a.D ? *reinterpret_cast<const v4u *>(src + at) : v4u{0u, 0u, 0u, 0u};
      q[s] ^= a.flip;
    }
  }

  uint8_t *mine = lds + (OWN ? w * 2 * L::BYTES : 0);
  const uint32_t lds_at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)mine);
  // chunks past D are never copied: zeros from the start
  if (a.D < 32 * DB) {
    for (int i = threadIdx.x * 16; i < (int)sizeof(lds); i += 256 * 16) *reinterpret_cast<uint4 *>(lds + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }

  const uint8_t *kb = reinterpret_cast<const uint8_t *>(a.k + (int64_t)b * a.k_b + hk * a.k_h);
  const uint8_t *vb = reinterpret_cast<const uint8_t *>(a.v + (int64_t)b * a.v_b + hk * a.v_h);
  const int *index = LIST ? a.index + (int64_t)b * a.Lk : nullptr;
  const int chunks = a.D / 8, slot = lane & (L::SLOTS - 1);
  // Copies tile t's rows into buffer `buf`.
  auto fetch = [&](int t, int buf) {
    const bool whole = !LIST && (t + 1) * KEYS <= n;
#pragma unroll
    for (int j = 0; j < COPIES; ++j) {
      const int base = (OWN ? j : 4 * j + w) * L::COPY_ROWS, r = base + lane / L::SLOTS;
      const int kc = slot ^ L::k_swap(r), vc = slot ^ L::v_swap(r);
      const uint32_t to = lds_at + buf * L::BYTES + base * L::ROW;
      if (whole) {
        const int64_t first = (int64_t)t * KEYS + base;
        if (kc < chunks) lds_dma16_s(kb + 2 * first * a.k_t, (uint32_t)(lane / L::SLOTS) * (uint32_t)(2 * a.k_t) + 16 * kc, to);
        if (vc < chunks) lds_dma16_s(vb + 2 * first * a.v_t, (uint32_t)(lane / L::SLOTS) * (uint32_t)(2 * a.v_t) + 16 * vc, to + L::HALF);
      } else {
        int key = min(t * KEYS + r, n - 1);
        if constexpr (LIST) key = index[key];
        if (kc < chunks) lds_dma16(kb + 2 * (int64_t)key * a.k_t + 16 * kc, to);
        if (vc < chunks) lds_dma16(vb + 2 * (int64_t)key * a.v_t + 16 * vc, to + L::HALF);
      }
    }
  };

  v16f o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float top = kLowest, sum = 0.0f;       // of this lane's half: the halves' sums are added at the end

  const int k_lane = m * L::ROW, k_x = h ^ L::k_swap(m);
  // the transposing read: row 4 h + (lane % 16) / 4 of a block of 16 states, channels 16 (lane / 16 % 2) + 4 (lane % 4)
  const int v_row = 4 * h + (lane >> 2 & 3), v_z = L::v_swap(v_row) >> 2;
  const int v_lane = L::HALF + v_row * L::ROW + (2 * (lane >> 4 & 1) + (lane >> 1 & 1)) * 16 + (lane & 1) * 8;

  if (t0 < t1) fetch(t0, 0);
  int buf = 0;
  for (int t = t0; t < t1; t += STRIDE, buf ^= 1) {
    vmcnt_wait0();
    if constexpr (!OWN) __syncthreads();
    const bool last = (t + 1) * KEYS > n;
    uint8_t *st = mine + buf * L::BYTES;
    if (last) {                            // V rows behind the last state: zero, whatever the last one holds
      const int from = n - t * KEYS;
      for (int i = from * L::ROW + (OWN ? lane : (int)threadIdx.x) * 16; i < L::HALF; i += (OWN ? 64 : 256) * 16)
        *reinterpret_cast<uint4 *>(st + L::HALF + i) = make_uint4(0, 0, 0, 0);
      if constexpr (OWN) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      else __syncthreads();
    }
    if (t + STRIDE < t1) {
      if constexpr (OWN) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the other buffer has been read
      fetch(t + STRIDE, buf ^ 1);
    }

    v16f s[KB];
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[k][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const v4u x = *reinterpret_cast<const v4u *>(st + 32 * k * L::ROW + k_lane + ((k_x ^ (2 * i)) << 4));
        s[k] = mma<F16>(x, q[i], s[k]);
      }
    if (last) {
      const int left = n - t * KEYS - 4 * h;
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * k + 8 * (i / 4) + i % 4 >= left) s[k][i] = -__builtin_inff();
    }
    float best = s[0][0];
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) best = fmaxf(best, s[k][i]);
    best = half_max(best) * a.c;
    if (__any(best > top + kSlack)) {
      const float to = best > top + kSlack ? best : top;
      const float r = __builtin_amdgcn_exp2f(top - to);
      top = to;
      sum *= r;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= r;
    }
    const float off = (F16 ? kShift16 : 0.0f) - top;
#pragma unroll
    for (int k = 0; k < KB; ++k) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[k][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][i], a.c, off));
        sum += s[k][i];
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        v4u p;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = pack2<F16>(s[k][8 * u + 2 * i], s[k][8 * u + 2 * i + 1]);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          typedef __attribute__((address_space(3))) v4i16 *Read;
          const uint8_t *at = st + (32 * k + 16 * u) * L::ROW + v_lane + ((d ^ v_z) << 6);
          const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Read)(uint8_t *)at);
          const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Read)(uint8_t *)(at + 8 * L::ROW));
          const uint2 x = __builtin_bit_cast(uint2, lo), y = __builtin_bit_cast(uint2, hi);
          o[d] = mma<F16>(v4u{x.x, x.y, y.x, y.y}, p, o[d]);
        }
      }
    }
  }

  sum = half_sum(sum);
  if (row >= a.rows) return;
  if (a.ml) {
    const int64_t piece = OWN ? 4 * part + w : part;
    const int64_t at = (piece * a.B * a.Hkv + bh) * a.rows + row;
    if (h == 0) {
      a.ml[2 * at] = top;
      a.ml[2 * at + 1] = t0 < t1 ? sum : -1.0f;      // -1: a piece without states
    }
    if (t0 < t1) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int ch = 32 * d + 8 * j + 4 * h;
          if (ch < a.D)
            *reinterpret_cast<v4f *>(a.o + at * a.D + ch) = v4f{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
        }
    }
    return;
  }
  const float inv = n > 0 ? 1.0f / sum : 0.0f;
  uint16_t *dst = a.out + (((int64_t)b * a.Lq + qi) * a.Hq + hq) * a.D;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int ch = 32 * d + 8 * j + 4 * h;
      if (ch < a.D)
        *reinterpret_cast<uint2 *>(dst + ch) = make_uint2(pack2<F16>(o[d][4 * j] * inv, o[d][4 * j + 1] * inv),
                                                          pack2<F16>(o[d][4 * j + 2] * inv, o[d][4 * j + 3] * inv));
    }
}

// A wavefront joins a row's pieces: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
template <bool F16>
__global__ __launch_bounds__(256) void cross_join_kernel(const CrossArgs a, int pieces) {
  const int lane = threadIdx.x & 63;
  const int64_t heads = (int64_t)a.B * a.Hkv, all = heads * a.rows, at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (at >= all) return;
  float top = kLowest;
  for (int i = lane; i < pieces; i += 64)
    if (a.ml[2 * (i * all + at) + 1] != -1.0f) top = fmaxf(top, a.ml[2 * (i * all + at)]);
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
  const int ch = 4 * lane;
  float sum = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  bool some = false;
  for (int i = 0; i < pieces; ++i) {
    const float l = a.ml[2 * (i * all + at) + 1];
    if (l == -1.0f) continue;
    some = true;
    const float f = __builtin_amdgcn_exp2f(a.ml[2 * (i * all + at)] - top);
    sum = __builtin_fmaf(f, l, sum);
    if (ch < a.D) {
      const v4f x = *reinterpret_cast<const v4f *>(a.o + (i * all + at) * a.D + ch);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(f, x[e], o[e]);
    }
  }
  if (ch >= a.D) return;
  const float inv = some ? 1.0f / sum : 0.0f;
  const int64_t bh = at / a.rows;
  const int row = (int)(at - bh * a.rows), qi = row / a.group, b = (int)(bh / a.Hkv);
  const int hq = (int)(bh - (int64_t)b * a.Hkv) * a.group + row - qi * a.group;
  *reinterpret_cast<uint2 *>(a.out + (((int64_t)b * a.Lq + qi) * a.Hq + hq) * a.D + ch) =
      make_uint2(pack2<F16>(o[0] * inv, o[1] * inv), pack2<F16>(o[2] * inv, o[3] * inv));
}

// The numbers of each batch row's visible states in order, and how many.  A
// thread counts a run of neighbouring states and writes it behind the runs before.
__global__ __launch_bounds__(1024) void cross_list_kernel(const uint8_t *__restrict__ mask, const int *__restrict__ lens,
                                                          int Lk, int *__restrict__ index, int *__restrict__ count) {
  __shared__ int sums[16];
  const int b = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n = lens ? min(max(lens[b], 0), Lk) : Lk;
  const uint8_t *seen = mask + (int64_t)b * Lk;
  int *out = index + (int64_t)b * Lk;
  const int run = (n + 1023) / 1024;
  const int from = min((int64_t)threadIdx.x * run, (int64_t)n), to = min(from + run, n);
  int mine = 0;
  for (int t = from; t < to; ++t) mine += seen[t] != 0;
  int upto = mine;                                   // of this lane and those before it
  for (int x = 1; x < 64; x <<= 1) {
    const int y = __shfl_up(upto, x);
    if (lane >= x) upto += y;
  }
  if (lane == 63) sums[w] = upto;
  __syncthreads();
  int at = upto - mine;
  for (int i = 0; i < w; ++i) at += sums[i];
  for (int t = from; t < to; ++t)
    if (seen[t] != 0) out[at++] = t;
  if (threadIdx.x == 1023) count[b] = at;
}

}  // namespace

extern "C" {

svdq_status_t svdq_cross_attention(const void *q, int64_t q_batch, int64_t q_token, int64_t q_head, const void *k,
                                   int64_t k_batch, int64_t k_token, int64_t k_head, const void *v, int64_t v_batch,
                                   int64_t v_token, int64_t v_head, svdq_dtype_t dtype, int B, int Lq, int Lk, int Hq,
                                   int Hkv, int D, const int32_t *key_lens, const uint8_t *mask, float scale,
                                   void *out, void *workspace, size_t ws_bytes, void *hip_stream) {
  const char *who = "svdq_cross_attention";
  if (dtype != SVDQ_BF16 && dtype != SVDQ_FP16)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: dtype must be SVDQ_BF16 or SVDQ_FP16", who);
  if (!cross_shape_ok(B, Lq, Lk, Hq, Hkv, D))
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: B=%d Lq=%d Lk=%d, %d heads over %d of %d channels", who, B, Lq, Lk, Hq, Hkv, D);
  if (B == 0 || Lq == 0) return SVDQ_OK;
  const CrossPlan p = cross_plan(B, Lq, Lk, Hq, Hkv, D, mask != nullptr);
  if (!q || !out || (!workspace && p.total > 0) || (Lk > 0 && (!k || !v))) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL pointer", who);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(workspace) || ((uintptr_t)key_lens & 3u))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", who);
  for (int64_t s : {q_batch, q_token, q_head, k_batch, k_token, k_head, v_batch, v_token, v_head})
    if (s < 0 || s % 8 != 0) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: stride %lld is not a multiple of 8", who, (long long)s);
  if (k_token >= 1 << 24 || v_token >= 1 << 24)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: states %lld and %lld elements apart", who, (long long)k_token, (long long)v_token);
  if (!(fabsf(scale) < 0x1p127f)) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: scale is not a number below 2^127", who);
  if (ws_bytes < (size_t)p.total)
    return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %lld bytes, got %zu", who, (long long)p.total, ws_bytes);
  svdq_status_t st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  CrossArgs a{};
  a.q = static_cast<const uint16_t *>(q);
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  a.q_b = q_batch; a.q_i = q_token; a.q_h = q_head;
  a.k_b = k_batch; a.k_t = k_token; a.k_h = k_head;
  a.v_b = v_batch; a.v_t = v_token; a.v_h = v_head;
  a.out = static_cast<uint16_t *>(out);
  a.B = B; a.Lq = Lq; a.Lk = Lk; a.Hq = Hq; a.Hkv = Hkv; a.group = Hq / Hkv; a.D = D;
  a.rows = (int)p.rows; a.tiles = (int)p.tiles; a.parts = p.parts;
  if (p.pieces > 1) {
    a.ml = reinterpret_cast<float *>(ws + p.ml_off);
    a.o = reinterpret_cast<float *>(ws + p.o_off);
  }
  a.lens = key_lens;
  const bool list = mask && Lk > 0;
  if (list) {
    int *index = reinterpret_cast<int *>(ws), *count = reinterpret_cast<int *>(ws + p.count_off);
    hipLaunchKernelGGL(cross_list_kernel, dim3(B), dim3(1024), 0, stream, mask, key_lens, Lk, index, count);
    st = launch_status("cross attention list launch");
    if (st != SVDQ_OK) return st;
    a.index = index;
    a.lens = count;
  }
  // Maxima are taken of the bare products, so the scale's sign goes to the queries, and
  // a scale of zero becomes one that still hides the rows behind the last state.
  a.c = fmaxf((float)(fabs((double)scale) * 1.4426950408889634), 1e-37f);
  a.flip = scale < 0.0f ? 0x80008000u : 0u;
  a.work = (int64_t)B * Hkv * p.tiles * p.parts;
  a.per_xcd = (a.work + 7) / 8;
  const dim3 grid((unsigned)(8 * a.per_xcd));
#define CROSS_GO(DB, KEYS, OWN, FF, LL) \
  hipLaunchKernelGGL((cross_attend_kernel<DB, KEYS, OWN, FF, LL>), grid, dim3(256), 0, stream, a)
#define CROSS_TYPE(DB, KEYS, OWN)                             \
  do {                                                        \
    if (dtype == SVDQ_FP16) {                                 \
      if (list) CROSS_GO(DB, KEYS, OWN, true, true);          \
      else CROSS_GO(DB, KEYS, OWN, true, false);              \
    } else {                                                  \
      if (list) CROSS_GO(DB, KEYS, OWN, false, true);         \
      else CROSS_GO(DB, KEYS, OWN, false, false);             \
    }                                                         \
  } while (0)
#define CROSS_FORM(DB, KEYS) do { if (p.own) CROSS_TYPE(DB, 32, true); else CROSS_TYPE(DB, KEYS, false); } while (0)
  switch (p.blocks) {
    case 2: CROSS_FORM(2, 64); break;
    case 3: CROSS_FORM(3, 64); break;
    case 4: CROSS_FORM(4, 64); break;
    case 5: CROSS_TYPE(5, 32, false); break;
    default: CROSS_TYPE(8, 32, false); break;
  }
#undef CROSS_FORM
#undef CROSS_TYPE
#undef CROSS_GO
  st = launch_status("cross attention launch");
  if (st != SVDQ_OK || p.pieces == 1) return st;
  const dim3 joins((unsigned)(((int64_t)B * Hkv * p.rows + 3) / 4));
  if (dtype == SVDQ_FP16) hipLaunchKernelGGL(cross_join_kernel<true>, joins, dim3(256), 0, stream, a, p.pieces);
  else hipLaunchKernelGGL(cross_join_kernel<false>, joins, dim3(256), 0, stream, a, p.pieces);
  return launch_status("cross attention join launch");
}

}  // extern "C"
