// Key/value cache in MXFP4 and the attention of new tokens over it.
//
//  kv4_append_kernel    16-bit key and value rows -> cache slots
//  kv4_read_kernel      cache slots -> values
//  kv4_attend_kernel    attention of a few new tokens over paged sequences
//  kv4_join_kernel      joins the pieces of a sequence that several
//                       workgroups attended to
//
// Cache layout.  A page holds page_size tokens (a power of two, 16..256) of
// every key/value head; the rows of one (page, head) are cut into units of 16
// tokens, 17 D bytes each:
//   [0, 8 D)          key codes:   lane l (token l % 16, quarter c = l / 16),
//                     word b = the eight codes of channels 32 b + 8 c + [0, 8)
//   [8 D, 16 D)       value codes: lane l (r = l % 16, c = l / 16), word b,
//                     byte i = token 4 c + i, channel 32 b + r in the low
//                     nibble and 32 b + 16 + r in the high one
//   [16 D, 16.5 D)    key scales   [token][D / 32], E8M0
//   [16.5 D, 17 D)    value scales [token][D / 32], E8M0
// with lane l's D / 32 words next to each other, so that a wavefront reads a
// unit's keys, or its values, as one contiguous piece that is already in the
// order of a 16x16x32 matrix operand (keys: a row per token; values: a row
// per channel, the tokens along the contraction).  A unit is the smallest
// thing that has this form, so pages as small as 16 tokens cost nothing.
#include <hip/hip_runtime.h>

#include "common.h"
#include "device_util.h"
#include "kv4_layout.h"

using namespace svdq;

namespace {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// the 16-bit value `h` of either type as float
template <bool F16>
__device__ __forceinline__ float wide(uint32_t h) {
  if constexpr (F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  else return __uint_as_float(h << 16);
}

// ---------------------------------------------------------------- append, read
// One thread per (row, keys or values, head, block of 32 channels).  With
// a = max |v| and E its biased exponent field, e = E - 129 clamped at -127
// (E = 0: -127); v 2^-e is exact and below 8, and the packed conversion
// rounds it to the nearest E2M1 value, ties to the even code, 6 the largest.
// A block with an infinity or a NaN gets the scale byte 255, for which every
// value reads as NaN.  Codes that round to zero are +0.
__device__ __forceinline__ uint32_t encode_block(const float (&v)[32], uint32_t (&w)[4]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const int E = (int)(top >> 23);
  const int e = E == 0 ? -127 : max(E - 129, -127);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t d = 0u;
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, __fmul_rn(v[8 * j], inv), __fmul_rn(v[8 * j + 1], inv), 1.0f, 0);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, __fmul_rn(v[8 * j + 2], inv), __fmul_rn(v[8 * j + 3], inv), 1.0f, 1);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, __fmul_rn(v[8 * j + 4], inv), __fmul_rn(v[8 * j + 5], inv), 1.0f, 2);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, __fmul_rn(v[8 * j + 6], inv), __fmul_rn(v[8 * j + 7], inv), 1.0f, 3);
    const uint32_t mag = d & 0x77777777u;
    const uint32_t nz = (mag | (mag >> 1) | (mag >> 2)) & 0x11111111u;
    w[j] = E == 255 ? 0u : mag | (d & (nz << 3));
  }
  return E == 255 ? 255u : (uint32_t)(e + 127);
}

template <bool F16>
__global__ __launch_bounds__(256) void kv4_append_kernel(uint8_t *__restrict__ data, Kv4Layout L,
                                                         const uint16_t *__restrict__ k, int64_t k_row,
                                                         int64_t k_head, const uint16_t *__restrict__ v,
                                                         int64_t v_row, int64_t v_head,
                                                         const int *__restrict__ slots, int T) {
  const int blocks = L.D / 32;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int b = (int)(idx % blocks), h = (int)(idx / blocks % L.H);
  const int64_t rest = idx / blocks / L.H;
  const int t = (int)(rest >> 1), is_v = (int)(rest & 1);
  if (t >= T) return;
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= (int64_t)L.pages << L.page_shift) return;
  const uint16_t *src = is_v ? v + t * v_row + h * v_head : k + t * k_row + h * k_head;
  float x[32];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 u = *reinterpret_cast<const uint4 *>(src + 32 * b + 8 * j);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[8 * j + 2 * c] = wide<F16>(w[c] & 0xFFFFu);
      x[8 * j + 2 * c + 1] = wide<F16>(w[c] >> 16);
    }
  }
  uint32_t w[4];
  const uint32_t scale = encode_block(x, w);
  uint8_t *unit = data + L.unit(slot >> L.page_shift, h, (int)(slot & (L.page_size() - 1)) >> 4);
  const int token = (int)(slot & 15);
  if (!is_v) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      reinterpret_cast<uint32_t *>(unit)[(16 * c + token) * blocks + b] = w[c];
    unit[L.k_scales() + token * blocks + b] = (uint8_t)scale;
  } else {
    uint8_t *vals = unit + L.v_codes();
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const uint32_t low = w[r / 8] >> (4 * (r % 8)) & 15u, high = w[2 + r / 8] >> (4 * (r % 8)) & 15u;
      vals[((token / 4 * 16 + r) * blocks + b) * 4 + token % 4] = (uint8_t)(low | high << 4);
    }
    unit[L.v_scales() + token * blocks + b] = (uint8_t)scale;
  }
}

// One thread per (row, keys or values, head, block of 32 channels): the
// values of a slot, as bf16 (exact: two significant bits) or float32; slots
// outside the cache read as zeros.
template <bool F32>
__global__ __launch_bounds__(256) void kv4_read_kernel(const uint8_t *__restrict__ data, Kv4Layout L,
                                                       const int *__restrict__ slots, int T,
                                                       void *__restrict__ k, void *__restrict__ v) {
  const int blocks = L.D / 32;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int b = (int)(idx % blocks), h = (int)(idx / blocks % L.H);
  const int64_t rest = idx / blocks / L.H;
  const int t = (int)(rest >> 1), is_v = (int)(rest & 1);
  if (t >= T) return;
  const int64_t slot = slots[t];
  uint32_t w[4] = {0u, 0u, 0u, 0u}, scale = 0;
  if (slot >= 0 && slot < (int64_t)L.pages << L.page_shift) {
    const uint8_t *unit = data + L.unit(slot >> L.page_shift, h, (int)(slot & (L.page_size() - 1)) >> 4);
    const int token = (int)(slot & 15);
    if (!is_v) {
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = reinterpret_cast<const uint32_t *>(unit)[(16 * c + token) * blocks + b];
      scale = unit[L.k_scales() + token * blocks + b];
    } else {
      const uint8_t *vals = unit + L.v_codes();
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t byte = vals[((token / 4 * 16 + r) * blocks + b) * 4 + token % 4];
        w[r / 8] |= (byte & 15u) << (4 * (r % 8));
        w[2 + r / 8] |= (byte >> 4) << (4 * (r % 8));
      }
      scale = unit[L.v_scales() + token * blocks + b];
    }
  }
  const float s = __uint_as_float(scale << 23);
  const int64_t at = ((int64_t)t * L.H + h) * L.D + 32 * b;
  uint32_t pairs[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    pairs[4 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 0));
    pairs[4 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 1));
    pairs[4 * j + 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 2));
    pairs[4 * j + 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 3));
  }
  if constexpr (F32) {
    float4 *out = reinterpret_cast<float4 *>(static_cast<float *>(is_v ? v : k) + at);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      out[j] = make_float4(bf16_lo(pairs[2 * j]), bf16_hi(pairs[2 * j]), bf16_lo(pairs[2 * j + 1]),
                           bf16_hi(pairs[2 * j + 1]));
  } else {
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(is_v ? v : k) + at);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      out[j] = make_uint4(pairs[4 * j], pairs[4 * j + 1], pairs[4 * j + 2], pairs[4 * j + 3]);
  }
}

// ------------------------------------------------------------------- attention
// out[b, i, h] = sum_t p_t v_t / sum_t p_t, p_t = exp(scale q . k_t - m), over
// the tokens t < len - Q + i + 1 of sequence b, one pass with the running
// maximum m and sum; a row that sees no token is zero.
//
// The g = Hq / Hkv query heads that share a key/value head, times the Q new
// tokens, are the columns of 16-wide matrix tiles (NT of them):
//   S^T [16 tokens, 16 rows] = K [16, D] Q^T      (D / 32 matrix steps)
//   O^T [16 channels, 16 rows] += V^T [16, 32 tokens] P^T
// In S^T a lane (row l % 16, quarter c = l / 16) holds tokens 4 c + [0, 4) of
// a unit, and the same lane enters those of two units as the eight
// contraction slots of P^T, so the weights go from one product to the next
// in registers; the order of the tokens along the contraction is free, and
// the cache's value words follow this one.  The row's maximum, sum and
// rescaling factor are then one value a lane.
// Keys and values become bf16 exactly with the packed scaled conversion (two
// significant bits times a power of two).  fp16 queries enter as two bf16
// pieces (exact), the weights p as two bf16 pieces (16 significant bits):
// what is rounded is p, at 2^-17, and the output.
//
// Work split: the tokens of each (sequence, head, block of rows) are cut
// into chunks of 128 (32 for each wavefront at a time); all chunks of the
// call form one line, of which each workgroup takes an equal piece, so short
// and long sequences share the machine evenly.  A workgroup that holds all
// chunks of a (sequence, head) writes the output, otherwise its running
// state, which kv4_join_kernel joins in order.
struct AttendArgs {
  const uint8_t *data;
  Kv4Layout L;
  const uint16_t *q;
  int64_t q_b, q_i, q_h;        // strides in elements
  const int *table;
  int width;                    // entries of a page-table row
  const int *lens;
  int B, Q, group, rows, row_blocks, block_rows;   // block_rows = min(rows, 16 NT)
  float scale;                  // softmax scale times log2(e)
  uint16_t *out;
  float *part;                  // [2 W][block_rows][D], then [2 W][block_rows][2]
  int W;
};

constexpr int kChunk = 128;

__device__ __forceinline__ int seq_len(const AttendArgs &a, int b) {
  return min(max(a.lens[b], 0), (int)min((int64_t)a.width << a.L.page_shift, (int64_t)1 << 30));
}
__device__ __forceinline__ int seq_chunks(int len) { return max(1, (len + kChunk - 1) / kChunk); }

// sum of x over the wavefront, and over lanes 0..lane
__device__ __forceinline__ int64_t wave_sum(int64_t x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ __forceinline__ int64_t wave_scan(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// chunks of all sequences before `b` (times 1), and of all
__device__ __forceinline__ void chunks_before(const AttendArgs &a, int b, int lane, int64_t &before, int64_t &all) {
  int64_t x = 0, y = 0;
  for (int i = lane; i < a.B; i += 64) {
    const int n = seq_chunks(seq_len(a, i));
    y += n;
    if (i < b) x += n;
  }
  before = wave_sum(x);
  all = wave_sum(y);
}

template <int D>
struct Tile {                       // two units of 16 tokens
  uint32_t k[2][D / 32], v[2][D / 32], ks[2][(D + 127) / 128], vs[2][D / 32];
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    w[0] = u.x; w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

// The unit of tokens [t, t + 16) of sequence b; `ok` is false where the page
// table has no valid page for it (page 0 is read in its place).
template <int D>
__device__ __forceinline__ void load_unit(const AttendArgs &a, const int *row, int h, int t, int lane,
                                          Tile<D> &x, int u, bool &ok) {
  const int at = t >> a.L.page_shift;
  int page = row[min(at, a.width - 1)];
  ok = at < a.width && page >= 0 && page < a.L.pages;
  page = __builtin_amdgcn_readfirstlane(ok ? page : 0);
  const uint8_t *unit = a.data + a.L.unit(page, h, (t & (a.L.page_size() - 1)) >> 4);
  load_words(x.k[u], unit + lane * (D / 8));
  load_words(x.v[u], unit + 8 * D + lane * (D / 8));
  if constexpr (D == 64) x.ks[u][0] = *reinterpret_cast<const uint16_t *>(unit + 16 * D + (lane & 15) * 2);
  else load_words(x.ks[u], unit + 16 * D + (lane & 15) * (D / 32));
  load_words(x.vs[u], unit + 16 * D + D / 2 + (lane >> 4) * (D / 8));
}

// Byte i of `w` as the power of two it stands for.  The conversion reads
// only the exponent field of its scale, so the neighbouring bytes that the
// shift leaves in the sign and mantissa fields do not matter.
__device__ __forceinline__ float scale_of(uint32_t w, int i) {
  return __uint_as_float(i == 0 ? w << 23 : i == 1 ? w << 15 : i == 2 ? w << 7 : w >> 1);
}
template <int I>
__device__ __forceinline__ uint32_t two_values(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, I));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, v2bf{(__bf16)a, (__bf16)b});
}

template <int D, int NT, bool F16>
__global__ __launch_bounds__(256) void kv4_attend_kernel(AttendArgs a) {
  constexpr int NB = D / 32;                       // blocks of 32 channels
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, c4 = lane >> 4;
  __shared__ float sm[4][NT * 16], sl[4][NT * 16];
  __shared__ v4f so[2][NT * 2 * NB][64];

  const int HR = a.L.H * a.row_blocks;
  int64_t before, all;
  chunks_before(a, 0, lane, before, all);
  const int64_t per = (all * HR + a.W - 1) / a.W;
  const int64_t u0 = blockIdx.x * per, u1 = min(u0 + per, all * HR);
  if (u0 >= u1) return;
  // the sequence that holds chunk u0, and the chunks before it
  int b = 0;
  int64_t start = 0;
  for (int base = 0; base < a.B; base += 64) {
    const int64_t n = base + lane < a.B ? (int64_t)HR * seq_chunks(seq_len(a, base + lane)) : 0;
    const int64_t upto = start + wave_scan(n, lane);
    const uint64_t past = __ballot(upto > u0);
    if (past) {
      const int i = __builtin_ctzll(past);
      b = base + i;
      start = __shfl(upto - n, i);
      break;
    }
    start = __shfl(upto, 63);
  }

  int64_t u = u0;
  while (u < u1) {
    b = __builtin_amdgcn_readfirstlane(b);
    const int len = __builtin_amdgcn_readfirstlane(seq_len(a, b));
    const int n = seq_chunks(len);
    const int hr = __builtin_amdgcn_readfirstlane((int)((u - start) / n));
    const int ch0 = __builtin_amdgcn_readfirstlane((int)((u - start) % n));
    const int ch1 = __builtin_amdgcn_readfirstlane((int)min((int64_t)n, ch0 + (u1 - u)));
    const int h = hr / a.row_blocks, r0 = hr % a.row_blocks * (16 * NT);
    const int *table = a.table + (int64_t)b * a.width;

    // queries: row r = i * group + j is new token i, head h * group + j
    v8bf qh[NT][NB], ql[NT][F16 ? NB : 1];
    int limit[NT];                                 // tokens that the lane's row sees
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      const int r = r0 + 16 * x + col;
      const bool real = r < a.rows;
      const int i = real ? r / a.group : 0, j = real ? r % a.group : 0;
      limit[x] = min(len, len - a.Q + i + 1);
      const uint16_t *src = a.q + b * a.q_b + i * a.q_i + (int64_t)(h * a.group + j) * a.q_h + 8 * c4;
#pragma unroll
      for (int s = 0; s < NB; ++s) {
        uint4 v = real ? *reinterpret_cast<const uint4 *>(src + 32 * s) : make_uint4(0, 0, 0, 0);
        if constexpr (F16) {
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f0 = wide<true>(in[e] & 0xFFFFu), f1 = wide<true>(in[e] >> 16);
            hi[e] = pack_bf16(f0, f1);
            const float g0 = f0 - bf16_lo(hi[e]), g1 = f1 - bf16_hi(hi[e]);
            lo[e] = pack_bf16(__builtin_isfinite(f0) ? g0 : 0.0f, __builtin_isfinite(f1) ? g1 : 0.0f);
          }
          qh[x][s] = as_v8bf(make_uint4(hi[0], hi[1], hi[2], hi[3]));
          ql[x][s] = as_v8bf(make_uint4(lo[0], lo[1], lo[2], lo[3]));
        } else {
          qh[x][s] = as_v8bf(v);
        }
      }
    }

    float m[NT], l[NT];
    v4f o[NT][2 * NB];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      m[x] = -__builtin_inff();
      l[x] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i) o[x][i] = v4f{};
    }

    const int t1 = min(ch1 * kChunk, len);
    const int whole = len - a.Q + 1;               // tokens that every row sees
    int t = ch0 * kChunk + 32 * w;
    Tile<D> cur;
    bool ok[2] = {true, true};
    if (t < t1) {
      load_unit<D>(a, table, h, t, lane, cur, 0, ok[0]);
      load_unit<D>(a, table, h, t + 16, lane, cur, 1, ok[1]);
    }
    while (t < t1) {
      Tile<D> nxt;
      bool nok[2] = {true, true};
      if (t + kChunk < t1) {
        load_unit<D>(a, table, h, t + kChunk, lane, nxt, 0, nok[0]);
        load_unit<D>(a, table, h, t + kChunk + 16, lane, nxt, 1, nok[1]);
      }
      const bool edge = t + 32 > whole || !ok[0] || !ok[1];
      v4f s[NT][2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int x = 0; x < NT; ++x) s[x][g] = v4f{};
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          const float sc = scale_of(cur.ks[g][k / 4], k % 4);
          const uint32_t kw = cur.k[g][k];
          const v8bf ka = as_v8bf(make_uint4(two_values<0>(kw, sc), two_values<1>(kw, sc), two_values<2>(kw, sc),
                                             two_values<3>(kw, sc)));
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            s[x][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, qh[x][k], s[x][g], 0, 0, 0);
            if constexpr (F16) s[x][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, ql[x][k], s[x][g], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[x][g][i] *= a.scale;
      if (edge) {
        // after the scale, which may be negative or zero: rows' own limits, and units without a page
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = t + 16 * g + 4 * c4 + i;
#pragma unroll
            for (int x = 0; x < NT; ++x)
              if (!ok[g] || tok >= limit[x]) s[x][g][i] = -__builtin_inff();
          }
          // what stands in the cache past the end may be anything, and zero
          // times it must be zero: such tokens' codes and scales are cleared
          uint32_t keep = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (ok[g] && t + 16 * g + 4 * c4 + i < len) keep |= 0xFFu << (8 * i);
#pragma unroll
          for (int k = 0; k < NB; ++k) cur.v[g][k] &= keep;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < NB; ++k)
              if (!(keep >> (8 * i) & 1u)) cur.vs[g][(i * NB + k) / 4] &= ~(0xFFu << (8 * ((i * NB + k) % 4)));
        }
      }
      // running maximum and weights
      v8bf ph[NT], pl[NT];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        float top = -__builtin_inff();
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, s[x][g][i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float now = fmaxf(m[x], top);
        const float ref = now == -__builtin_inff() ? 0.0f : now;
        if (__ballot(now > m[x])) {
          const float f = __builtin_amdgcn_exp2f(m[x] - ref);
          l[x] *= f;
#pragma unroll
          for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[x][i][e] *= f;
          m[x] = now;
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = __builtin_amdgcn_exp2f(s[x][g][2 * i] - ref);
            const float p1 = __builtin_amdgcn_exp2f(s[x][g][2 * i + 1] - ref);
            l[x] += p0 + p1;
            const uint32_t pk = pack_bf16(p0, p1);
            hi[2 * g + i] = pk;
            lo[2 * g + i] = pack_bf16(p0 - bf16_lo(pk), p1 - bf16_hi(pk));
          }
        ph[x] = as_v8bf(make_uint4(hi[0], hi[1], hi[2], hi[3]));
        pl[x] = as_v8bf(make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t lo[4], hi[4];                     // channels 32 k + col, and 16 above
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t vw = cur.v[g][k];
          const uint32_t x0 = two_values<0>(vw, scale_of(cur.vs[g][k / 4], k % 4));
          const uint32_t x1 = two_values<1>(vw, scale_of(cur.vs[g][(NB + k) / 4], (NB + k) % 4));
          const uint32_t x2 = two_values<2>(vw, scale_of(cur.vs[g][(2 * NB + k) / 4], (2 * NB + k) % 4));
          const uint32_t x3 = two_values<3>(vw, scale_of(cur.vs[g][(3 * NB + k) / 4], (3 * NB + k) % 4));
          lo[2 * g] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
          hi[2 * g] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
          lo[2 * g + 1] = __builtin_amdgcn_perm(x3, x2, 0x05040100u);
          hi[2 * g + 1] = __builtin_amdgcn_perm(x3, x2, 0x07060302u);
        }
        const v8bf va = as_v8bf(make_uint4(lo[0], lo[1], lo[2], lo[3]));
        const v8bf vb = as_v8bf(make_uint4(hi[0], hi[1], hi[2], hi[3]));
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          o[x][2 * k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, ph[x], o[x][2 * k], 0, 0, 0);
          o[x][2 * k + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, ph[x], o[x][2 * k + 1], 0, 0, 0);
          o[x][2 * k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, pl[x], o[x][2 * k], 0, 0, 0);
          o[x][2 * k + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, pl[x], o[x][2 * k + 1], 0, 0, 0);
        }
      }
      cur = nxt;
      ok[0] = nok[0];
      ok[1] = nok[1];
      t += kChunk;
    }

    // the four wavefronts' states meet: everything relative to the largest
    // maximum, then wavefronts 2 and 3 into 0 and 1, and 1 into 0
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      l[x] += __shfl_xor(l[x], 16);
      l[x] += __shfl_xor(l[x], 32);
      if (c4 == 0) {
        sm[w][16 * x + col] = m[x];
        sl[w][16 * x + col] = l[x];
      }
    }
    __syncthreads();
    float mall[NT], lall[NT];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      const int i = 16 * x + col;
      mall[x] = fmaxf(fmaxf(sm[0][i], sm[1][i]), fmaxf(sm[2][i], sm[3][i]));
      const float ref = mall[x] == -__builtin_inff() ? 0.0f : mall[x];
      lall[x] = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) lall[x] += sl[k][i] * __builtin_amdgcn_exp2f(sm[k][i] - ref);
      const float f = __builtin_amdgcn_exp2f(m[x] - ref);
#pragma unroll
      for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][k][e] *= f;
    }
    if (w >= 2) {
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) so[w - 2][x * 2 * NB + k][lane] = o[x][k];
    }
    __syncthreads();
    if (w < 2) {
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) {
          const v4f y = so[w][x * 2 * NB + k][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[x][k][e] += y[e];
          if (w == 1) so[1][x * 2 * NB + k][lane] = o[x][k];
        }
    }
    __syncthreads();
    if (w == 0) {
      const bool done = ch0 == 0 && ch1 == n;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (u > u0 ? 1 : 0);
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const int r = r0 + 16 * x + col;
        const int i = r / a.group, j = r % a.group;
        const float inv = lall[x] > 0.0f || lall[x] != lall[x] ? 1.0f / lall[x] : 0.0f;
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) {
          const v4f y = so[1][x * 2 * NB + k][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[x][k][e] += y[e];
          const int d = 16 * k + 4 * c4;
          if (r < a.rows) {
            if (done) {
              uint2 out;
              if constexpr (F16) {
                out.x = __builtin_bit_cast(uint32_t, v2h{(_Float16)(o[x][k][0] * inv), (_Float16)(o[x][k][1] * inv)});
                out.y = __builtin_bit_cast(uint32_t, v2h{(_Float16)(o[x][k][2] * inv), (_Float16)(o[x][k][3] * inv)});
              } else {
                out.x = pack_bf16(o[x][k][0] * inv, o[x][k][1] * inv);
                out.y = pack_bf16(o[x][k][2] * inv, o[x][k][3] * inv);
              }
              *reinterpret_cast<uint2 *>(
                  a.out + (((int64_t)b * a.Q + i) * (a.L.H * a.group) + h * a.group + j) * D + d) = out;
            } else {
              *reinterpret_cast<v4f *>(a.part + (slot * a.block_rows + 16 * x + col) * D + d) = o[x][k];
            }
          }
        }
        if (!done && r < a.rows && c4 == 0) {
          float *ml = a.part + 2 * (int64_t)a.W * a.block_rows * D + (slot * a.block_rows + 16 * x + col) * 2;
          ml[0] = mall[x];
          ml[1] = lall[x];
        }
      }
    }
    __syncthreads();
    u += ch1 - ch0;
    if (u >= start + (int64_t)HR * n) {
      start += (int64_t)HR * n;
      ++b;
    }
  }
}

// One workgroup per (sequence, new token, query head) whose chunks went to
// more than one workgroup: the pieces' states, in order, relative to their
// largest maximum.  Wavefront w takes pieces w, w + 4, ...; a lane holds
// D / 64 channels.
template <int D, bool F16>
__global__ __launch_bounds__(256) void kv4_join_kernel(AttendArgs a) {
  constexpr int V = D / 64;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int Hq = a.L.H * a.group;
  const int hq = blockIdx.x % Hq;
  const int i = blockIdx.x / Hq % a.Q, b = blockIdx.x / Hq / a.Q;
  const int h = hq / a.group, r = i * a.group + hq % a.group;
  const int HR = a.L.H * a.row_blocks;
  int64_t before, all;
  chunks_before(a, b, lane, before, all);
  const int n = seq_chunks(seq_len(a, b));
  const int64_t per = (all * HR + a.W - 1) / a.W;
  const int64_t first = before * HR + (int64_t)(h * a.row_blocks + r / a.block_rows) * n;
  const int64_t g0 = first / per, g1 = (first + n - 1) / per;
  if (g0 == g1) return;
  const int pieces = (int)(g1 - g0 + 1);
  const int rb = r % a.block_rows;
  const float *ml = a.part + 2 * (int64_t)a.W * a.block_rows * D;
  auto slot = [&](int p) { return 2 * (g0 + p) + (p == 0 && first > g0 * per ? 1 : 0); };
  float top = -__builtin_inff();
  for (int p = lane; p < pieces; p += 64) top = fmaxf(top, ml[(slot(p) * a.block_rows + rb) * 2]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float ref = top == -__builtin_inff() ? 0.0f : top;
  float acc[V] = {}, l = 0.0f;
  for (int p = w; p < pieces; p += 4) {
    const int64_t at = slot(p) * a.block_rows + rb;
    const float f = __builtin_amdgcn_exp2f(ml[at * 2] - ref);
    l = __builtin_fmaf(ml[at * 2 + 1], f, l);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = __builtin_fmaf(a.part[at * D + lane * V + e], f, acc[e]);
  }
  __shared__ float so[4][D], sl[4];
#pragma unroll
  for (int e = 0; e < V; ++e) so[w][lane * V + e] = acc[e];
  if (lane == 0) sl[w] = l;
  __syncthreads();
  const int d = threadIdx.x;
  if (d < D) {
    const float sum = (sl[0] + sl[1]) + (sl[2] + sl[3]);
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    const float y = ((so[0][d] + so[1][d]) + (so[2][d] + so[3][d])) * inv;
    const int64_t at = (((int64_t)b * a.Q + i) * Hq + hq) * D + d;
    a.out[at] = F16 ? __builtin_bit_cast(uint16_t, (_Float16)y) : __builtin_bit_cast(uint16_t, (__bf16)y);
  }
}

// ------------------------------------------------------------------- host side
svdq_status_t validate_cache(const svdq_kv4_cache_t *c, const char *who, Kv4Layout *L) {
  if (!c || !c->data) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL cache", who);
  if (!aligned16(c->data)) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: misaligned cache", who);
  if (!kv4_shape_ok(c->num_pages, c->page_size, c->kv_heads, c->head_dim))
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: cache of %d pages of %d tokens, %d heads of %d channels", who,
                c->num_pages, c->page_size, c->kv_heads, c->head_dim);
  *L = Kv4Layout(c->num_pages, c->page_size, c->kv_heads, c->head_dim);
  return SVDQ_OK;
}

bool strides_ok(const int64_t *s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] < 0 || s[i] % 8 != 0) return false;
  return true;
}

}  // namespace

extern "C" {

svdq_status_t svdq_kv4_append(const svdq_kv4_cache_t *cache, const void *k, int64_t k_row, int64_t k_head,
                              const void *v, int64_t v_row, int64_t v_head, svdq_dtype_t dtype, int T,
                              const int32_t *slots, void *hip_stream) {
  Kv4Layout L;
  svdq_status_t st = validate_cache(cache, "svdq_kv4_append", &L);
  if (st != SVDQ_OK) return st;
  if (T < 0) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_append: T=%d", T);
  if (dtype != SVDQ_BF16 && dtype != SVDQ_FP16)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_append: dtype must be SVDQ_BF16 or SVDQ_FP16");
  if (T == 0) return SVDQ_OK;
  if (!k || !v || !slots) return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_append: NULL pointer");
  const int64_t strides[4] = {k_row, k_head, v_row, v_head};
  if (!aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 3u) || !strides_ok(strides, 4))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_append: misaligned pointer, or a stride that is not a multiple of 8");
  const int64_t threads = (int64_t)T * L.H * 2 * (L.D / 32);
  if (threads > (int64_t)1 << 38) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_append: T=%d", T);
  st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  const dim3 grid((unsigned)((threads + 255) / 256));
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  uint8_t *data = static_cast<uint8_t *>(cache->data);
  const uint16_t *kp = static_cast<const uint16_t *>(k), *vp = static_cast<const uint16_t *>(v);
  if (dtype == SVDQ_FP16)
    hipLaunchKernelGGL((kv4_append_kernel<true>), grid, dim3(256), 0, stream, data, L, kp, k_row, k_head, vp, v_row,
                       v_head, slots, T);
  else
    hipLaunchKernelGGL((kv4_append_kernel<false>), grid, dim3(256), 0, stream, data, L, kp, k_row, k_head, vp, v_row,
                       v_head, slots, T);
  return launch_status("cache append launch");
}

svdq_status_t svdq_kv4_read(const svdq_kv4_cache_t *cache, const int32_t *slots, int T, void *k, void *v,
                            svdq_dtype_t dtype, void *hip_stream) {
  Kv4Layout L;
  svdq_status_t st = validate_cache(cache, "svdq_kv4_read", &L);
  if (st != SVDQ_OK) return st;
  if (T < 0) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_read: T=%d", T);
  if (dtype != SVDQ_BF16 && dtype != SVDQ_FP32)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_read: dtype must be SVDQ_BF16 or SVDQ_FP32");
  if (T == 0) return SVDQ_OK;
  if (!k || !v || !slots) return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_read: NULL pointer");
  if (!aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 3u))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_read: misaligned pointer");
  const int64_t threads = (int64_t)T * L.H * 2 * (L.D / 32);
  if (threads > (int64_t)1 << 38) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_read: T=%d", T);
  st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  const dim3 grid((unsigned)((threads + 255) / 256));
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const uint8_t *data = static_cast<const uint8_t *>(cache->data);
  if (dtype == SVDQ_FP32)
    hipLaunchKernelGGL((kv4_read_kernel<true>), grid, dim3(256), 0, stream, data, L, slots, T, k, v);
  else
    hipLaunchKernelGGL((kv4_read_kernel<false>), grid, dim3(256), 0, stream, data, L, slots, T, k, v);
  return launch_status("cache read launch");
}

svdq_status_t svdq_kv4_attention(const svdq_kv4_cache_t *cache, const void *q, int64_t q_batch, int64_t q_token,
                                 int64_t q_head, svdq_dtype_t dtype, int B, int Q, int Hq,
                                 const int32_t *page_table, int table_width, const int32_t *seq_lens, float scale,
                                 void *out, void *workspace, size_t ws_bytes, void *hip_stream) {
  Kv4Layout L;
  svdq_status_t st = validate_cache(cache, "svdq_kv4_attention", &L);
  if (st != SVDQ_OK) return st;
  if (dtype != SVDQ_BF16 && dtype != SVDQ_FP16)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_attention: dtype must be SVDQ_BF16 or SVDQ_FP16");
  if (!kv4_query_ok(B, Q, Hq, L.H) || table_width < 1)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_attention: B=%d Q=%d Hq=%d over %d heads, page table of %d columns",
                B, Q, Hq, L.H, table_width);
  if (B == 0) return SVDQ_OK;
  if (!q || !page_table || !seq_lens || !out || !workspace)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_attention: NULL pointer");
  const int64_t strides[3] = {q_batch, q_token, q_head};
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || ((uintptr_t)page_table & 3u) ||
      ((uintptr_t)seq_lens & 3u) || !strides_ok(strides, 3))
    return fail(SVDQ_ERR_INVALID_ARGUMENT,
                "svdq_kv4_attention: misaligned pointer, or a stride that is not a multiple of 8");
  if (!__builtin_isfinite(scale)) return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_attention: scale is not finite");
  const size_t need = svdq_kv4_attention_workspace_bytes(B, Q, Hq, L.H, L.D);
  if (ws_bytes < need)
    return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "svdq_kv4_attention: workspace needs %zu bytes, got %zu", need, ws_bytes);
  st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  AttendArgs a{};
  a.data = static_cast<const uint8_t *>(cache->data);
  a.L = L;
  a.q = static_cast<const uint16_t *>(q);
  a.q_b = q_batch;
  a.q_i = q_token;
  a.q_h = q_head;
  a.table = page_table;
  a.width = table_width;
  a.lens = seq_lens;
  a.B = B;
  a.Q = Q;
  a.group = Hq / L.H;
  a.rows = a.group * Q;
  const int nt = a.rows > 16 ? 2 : 1;
  a.row_blocks = (a.rows + 16 * nt - 1) / (16 * nt);
  a.block_rows = a.rows < 16 * nt ? a.rows : 16 * nt;
  a.scale = (float)((double)scale * 1.4426950408889634);
  a.out = static_cast<uint16_t *>(out);
  a.part = static_cast<float *>(workspace);
  // no more workgroups than there can be chunks
  const int64_t most = (((int64_t)table_width << L.page_shift) + kChunk - 1) / kChunk * B * L.H * a.row_blocks;
  a.W = (int)(most < kKv4Groups ? most : kKv4Groups);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const dim3 join_grid((unsigned)((int64_t)B * Q * Hq));
#define KV4_GO(DD, NN, FF)                                                                      \
  do {                                                                                          \
    hipLaunchKernelGGL((kv4_attend_kernel<DD, NN, FF>), dim3(a.W), dim3(256), 0, stream, a);    \
    hipLaunchKernelGGL((kv4_join_kernel<DD, FF>), join_grid, dim3(256), 0, stream, a);          \
  } while (0)
#define KV4_ROWS(DD, FF) do { if (nt == 1) KV4_GO(DD, 1, FF); else KV4_GO(DD, 2, FF); } while (0)
#define KV4_TYPE(DD) do { if (dtype == SVDQ_FP16) KV4_ROWS(DD, true); else KV4_ROWS(DD, false); } while (0)
  if (L.D == 64) KV4_TYPE(64);
  else if (L.D == 128) KV4_TYPE(128);
  else KV4_TYPE(256);
#undef KV4_TYPE
#undef KV4_ROWS
#undef KV4_GO
  return launch_status("cache attention launch");
}

}  // extern "C"
