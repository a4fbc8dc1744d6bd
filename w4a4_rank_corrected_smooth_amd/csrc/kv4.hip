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
// One thread per (row, keys or values, head, block of 32 channels): with
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

// A thread's place: row, keys or values, head and block of 32 channels, four
// neighbouring rows in neighbouring lanes and 16 rows of a head next to each
// other, so that a wavefront of consecutive slots covers whole units.
struct Item {
  int t, h, b, is_v, i;
  __device__ __forceinline__ explicit Item(uint32_t idx, const Kv4Layout &L) {
    const int shift = L.D == 64 ? 1 : L.D == 128 ? 2 : 3;        // blocks of a row: 2, 4 or 8
    i = idx & 3;
    b = idx >> 2 & ((1 << shift) - 1);
    const uint32_t r = idx >> (2 + shift), u = r >> 3, tile = u / (uint32_t)L.H;
    is_v = r >> 2 & 1;
    h = u - tile * L.H;
    t = tile * 16 + 4 * (r & 3) + i;
  }
};
// Whether the four lanes of a row quad hold tokens 4 c .. 4 c + 3 of a unit:
// then a word of value codes, four tokens' bytes, is read or written whole.
__device__ __forceinline__ bool whole_quad(int64_t slot, bool in, int i) {
  const int first = __builtin_amdgcn_update_dpp(0, (int)slot, 0x00, 0xF, 0xF, true);    // quad_perm 0,0,0,0
  const uint64_t ok = __ballot(in && (first & 3) == 0 && (int)slot == first + i);
  return (ok >> (threadIdx.x & 60) & 15) == 15;
}
// four words of bytes, transposed: byte k of word j becomes byte j of word k
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t c = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  w[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
  w[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
  w[3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
}

template <bool F16>
__global__ __launch_bounds__(256) void kv4_append_kernel(uint8_t *__restrict__ data, Kv4Layout L,
                                                         const uint16_t *__restrict__ k, int64_t k_row,
                                                         int64_t k_head, const uint16_t *__restrict__ v,
                                                         int64_t v_row, int64_t v_head,
                                                         const int *__restrict__ slots, int T) {
  __shared__ uint32_t swap[256][4];
  const int blocks = L.D / 32;
  const Item it(blockIdx.x * 256 + threadIdx.x, L);
  const int64_t slot = it.t < T ? slots[it.t] : -1;
  const bool in = slot >= 0 && slot < (int64_t)L.pages << L.page_shift;
  uint32_t w[4] = {0u, 0u, 0u, 0u}, scale = 0;
  uint8_t *unit = data;
  if (in) {
    const uint16_t *src = it.is_v ? v + it.t * v_row + it.h * v_head : k + it.t * k_row + it.h * k_head;
    float x[32];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 u = *reinterpret_cast<const uint4 *>(src + 32 * it.b + 8 * j);
      const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[8 * j + 2 * c] = wide<F16>(uw[c] & 0xFFFFu);
        x[8 * j + 2 * c + 1] = wide<F16>(uw[c] >> 16);
      }
    }
    scale = encode_block(x, w);
    unit += L.unit(slot >> L.page_shift, it.h, (int)(slot & (L.page_size() - 1)) >> 4);
  }
  const int token = (int)(slot & 15);
  const bool quad = whole_quad(slot, in, it.i);
  // value bytes r = 4 q .. 4 q + 3 of this token: channels r low, 16 + r high
  uint32_t bytes[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t lo = w[q / 2] >> (16 * (q % 2)) & 0xFFFFu, hi = w[2 + q / 2] >> (16 * (q % 2)) & 0xFFFFu;
    lo = (lo | lo << 8) & 0x00FF00FFu;
    hi = (hi | hi << 8) & 0x00FF00FFu;
    bytes[q] = ((lo | lo << 4) & 0x0F0F0F0Fu) | ((hi | hi << 4) & 0x0F0F0F0Fu) << 4;
  }
  *reinterpret_cast<uint4 *>(swap[threadIdx.x]) = make_uint4(bytes[0], bytes[1], bytes[2], bytes[3]);
  __syncthreads();
  if (!in) return;
  if (!it.is_v) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      reinterpret_cast<uint32_t *>(unit)[(16 * c + token) * blocks + it.b] = w[c];
    unit[L.k_scales() + token * blocks + it.b] = (uint8_t)scale;
  } else {
    if (quad) {                          // this lane writes words r = 4 i .. 4 i + 3
      uint32_t m[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) m[n] = swap[(threadIdx.x & ~3) + n][it.i];
      transpose4(m);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        reinterpret_cast<uint32_t *>(unit + L.v_codes())[(token / 4 * 16 + 4 * it.i + n) * blocks + it.b] = m[n];
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        unit[L.v_codes() + ((token / 4 * 16 + r) * blocks + it.b) * 4 + token % 4] = (uint8_t)(bytes[r / 4] >> (8 * (r % 4)));
    }
    unit[L.v_scales() + token * blocks + it.b] = (uint8_t)scale;
  }
}

// The values of a slot, as bf16 (exact: two significant bits) or float32;
// slots outside the cache read as zeros.
template <bool F32>
__global__ __launch_bounds__(256) void kv4_read_kernel(const uint8_t *__restrict__ data, Kv4Layout L,
                                                       const int *__restrict__ slots, int T,
                                                       void *__restrict__ k, void *__restrict__ v) {
  __shared__ uint32_t swap[256][4];
  __shared__ uint4 out[256][5];
  const int blocks = L.D / 32;
  const Item it(blockIdx.x * 256 + threadIdx.x, L);
  const int64_t slot = it.t < T ? slots[it.t] : -1;
  const bool in = slot >= 0 && slot < (int64_t)L.pages << L.page_shift;
  const int token = (int)(slot & 15);
  const bool quad = whole_quad(slot, in, it.i);
  uint32_t w[4] = {0u, 0u, 0u, 0u}, scale = 0;
  if (in) {
    const uint8_t *unit = data + L.unit(slot >> L.page_shift, it.h, (int)(slot & (L.page_size() - 1)) >> 4);
    if (!it.is_v) {
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = reinterpret_cast<const uint32_t *>(unit)[(16 * c + token) * blocks + it.b];
      scale = unit[L.k_scales() + token * blocks + it.b];
    } else {
      if (quad) {                        // words r = 4 i .. 4 i + 3, a byte of each token
        uint32_t m[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          m[n] = reinterpret_cast<const uint32_t *>(unit + L.v_codes())[(token / 4 * 16 + 4 * it.i + n) * blocks + it.b];
        transpose4(m);
#pragma unroll
        for (int n = 0; n < 4; ++n) swap[(threadIdx.x & ~3) + n][it.i] = m[n];
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t m = 0;
#pragma unroll
          for (int n = 0; n < 4; ++n)
            m |= (uint32_t)unit[L.v_codes() + ((token / 4 * 16 + 4 * q + n) * blocks + it.b) * 4 + token % 4] << (8 * n);
          swap[threadIdx.x][q] = m;
        }
      }
      scale = unit[L.v_scales() + token * blocks + it.b];
    }
  }
  __syncthreads();
  if (in && it.is_v) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {        // bytes r = 4 q .. 4 q + 3 back to nibbles of channels r and 16 + r
      const uint32_t m = swap[threadIdx.x][q];
      uint32_t lo = m & 0x0F0F0F0Fu, hi = m >> 4 & 0x0F0F0F0Fu;
      lo = (lo | lo >> 4) & 0x00FF00FFu;
      hi = (hi | hi >> 4) & 0x00FF00FFu;
      w[q / 2] |= ((lo | lo >> 8) & 0xFFFFu) << (16 * (q % 2));
      w[2 + q / 2] |= ((hi | hi >> 8) & 0xFFFFu) << (16 * (q % 2));
    }
  }
  const float s = __uint_as_float(scale << 23);
  uint32_t pairs[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    pairs[4 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 0));
    pairs[4 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 1));
    pairs[4 * j + 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 2));
    pairs[4 * j + 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 3));
  }
  // through LDS, so that neighbouring lanes store neighbouring 16-byte pieces
  // of a row (a block is four; 8190 rows of 8 heads of 128 took 15 us without)
#pragma unroll
  for (int j = 0; j < 4; ++j)
    out[threadIdx.x][j] = make_uint4(pairs[4 * j], pairs[4 * j + 1], pairs[4 * j + 2], pairs[4 * j + 3]);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int piece = threadIdx.x + 256 * j, off = piece & (4 * blocks - 1);
    const int seg = piece >> (L.D == 64 ? 3 : L.D == 128 ? 4 : 5);
    const int item = ((seg >> 2) * blocks + (off >> 2)) * 4 + (seg & 3);
    const Item to(blockIdx.x * 256 + item, L);
    if (to.t >= T) continue;
    const uint4 u = out[item][off % 4];
    const int64_t at = ((int64_t)to.t * L.H + to.h) * L.D + 8 * off;
    if constexpr (F32) {
      float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(to.is_v ? v : k) + at);
      f[0] = make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
      f[1] = make_float4(bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w));
    } else {
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(to.is_v ? v : k) + at) = u;
    }
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
// and long sequences share the machine evenly.  Beginning and ending a
// (sequence, head) takes about as long as kKv4Start chunks, which stand on the
// line before its first one.  A workgroup that holds all chunks of a
// (sequence, head) writes the output, otherwise its running state, which
// kv4_join_kernel joins in order.
struct AttendArgs {
  const uint8_t *data;
  Kv4Layout L;
  const uint16_t *q;
  int64_t q_b, q_i, q_h;        // strides in elements
  const int *table;
  int width;                    // entries of a page-table row
  const int *lens;
  int B, Q, group, rows, row_blocks, block_rows;   // block_rows = min(rows, ROWS)
  float scale;                  // |softmax scale| log2(e), positive
  uint32_t flip;                // sign bits of the queries to turn, for a negative scale
  uint16_t *out;
  float *part;                  // [2 W][block_rows][D], then [2 W][block_rows][2]
  int W;
};

__device__ __forceinline__ int seq_len(const AttendArgs &a, int b) {
  return min(max(a.lens[b], 0), a.width << a.L.page_shift);
}
__device__ __forceinline__ int seq_chunks(int len) { return max(1, (len + kKv4Chunk - 1) / kKv4Chunk); }

// sum of x over lanes 0..lane, within the vector unit (16 lanes at a time,
// then the last lane of a row into the next rows)
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);    // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);    // row_bcast:15
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);    // row_bcast:31
  return x;
}

// The line of a call, for one key/value head and block of rows: a sequence
// takes its chunks and kKv4Start.  The wavefront looks at 64 sequences at a
// time: their lengths in tokens, and where their parts of the line end.
struct Line {
  int base = -64, len = 0, upto = 0;
  // sequences base.., the line before them being `before` long; returns its length after them
  __device__ __forceinline__ int look(const AttendArgs &a, int base_, int before, int lane) {
    base = base_;
    len = base + lane < a.B ? seq_len(a, base + lane) : 0;
    upto = before + wave_scan(base + lane < a.B ? seq_chunks(len) + kKv4Start : 0);
    return __builtin_amdgcn_readlane(upto, 63);
  }
};
// The whole line's length; `line` is left at the last sequences.
__device__ __forceinline__ int line_length(const AttendArgs &a, Line &line, int lane) {
  int all = 0;
  for (int base = 0; base < a.B; base += 64) all = line.look(a, base, all, lane);
  return all;
}

template <int D>
struct Keys { uint32_t k[2][D / 32], s[2][(D + 127) / 128]; };     // two units of 16 tokens
template <int D>
struct Values { uint32_t v[2][D / 32], s[2][D / 32]; };

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const v4u u = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(p) + i);
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    w[0] = u.x; w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

// The pages of a sequence, 64 entries of its page-table row at a time in the
// lanes of a register, so that a tile's page costs no trip to memory.
struct Pages {
  const int *row;
  int width, pages, first, lanes;   // entries [first, first + 64)
  // The load is waited for here: left to its use, where the paths with and
  // without it meet, the wait would also hold up the tiles being copied.
  __device__ __forceinline__ void load(int at, int lane) {
    first = at;
    lanes = row[min(at + lane, width - 1)];
    __builtin_amdgcn_s_waitcnt(0x0F70);     // vmcnt(0)
  }
  // entry `at` (the same in every lane), -1 if it names no page
  __device__ __forceinline__ int get(int at, int lane) {
    if (at >= first + 64) load(at, lane);
    const int p = __builtin_amdgcn_readlane(lanes, at - first);
    return at < width && p >= 0 && p < pages ? p : -1;
  }
};

// The units of tokens [t, t + 16) and [t + 16, t + 32) of a sequence, and
// whether they have a page (page 0 is read in the place of one that has none).
struct Place { const uint8_t *unit[2]; bool ok[2]; };
template <int D>
__device__ __forceinline__ Place locate(const AttendArgs &a, Pages &pages, int h, int t, int lane) {
  Place p;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int page = pages.get((t + 16 * u) >> a.L.page_shift, lane);
    p.ok[u] = page >= 0;
    p.unit[u] = a.data + a.L.unit(max(page, 0), h, ((t + 16 * u) & (a.L.page_size() - 1)) >> 4);
  }
  return p;
}
template <int D>
__device__ __forceinline__ void load_keys(const Place &p, int lane, Keys<D> &x) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    load_words(x.k[u], p.unit[u] + lane * (D / 8));
    if constexpr (D == 64) x.s[u][0] = *reinterpret_cast<const uint16_t *>(p.unit[u] + 16 * D + (lane & 15) * 2);
    else load_words(x.s[u], p.unit[u] + 16 * D + (lane & 15) * (D / 32));
  }
}
template <int D>
__device__ __forceinline__ void load_values(const Place &p, int lane, Values<D> &x) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    load_words(x.v[u], p.unit[u] + 8 * D + lane * (D / 8));
    load_words(x.s[u], p.unit[u] + 16 * D + D / 2 + (lane >> 4) * (D / 8));
  }
}

// Byte i of `w` as the power of two it stands for.  The conversion reads
// only the exponent field of its scale, so the neighbouring bytes that the
// shift leaves in the sign and mantissa fields do not matter.
__device__ __forceinline__ float scale_of(uint32_t w, int i) {
  return __uint_as_float(i == 0 ? w << 23 : i == 1 ? w << 15 : i == 2 ? w << 7 : w >> 1);
}
// 0x80 in the bytes of `w` that are 255 (without those bits they are the scale 1)
__device__ __forceinline__ uint32_t bytes_255(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u; }
template <int I>
__device__ __forceinline__ uint32_t two_values(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, I));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, v2bf{(__bf16)a, (__bf16)b});
}

// the lane 8 columns on, of the same quarter
__device__ __forceinline__ float other_half(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x128, 0xF, 0xF, true));
}
// the largest x of the four lanes of a column (l % 16)
__device__ __forceinline__ float column_max(float x) {
  const uint32_t u = __float_as_uint(x);
  auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const uint32_t v = __float_as_uint(x);
  r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

constexpr float kLargest = 3.402823466e38f;        // of the float32 numbers
// 1 / the sum of a row's weights; zero for a row that has no maximum, since it saw no token
__device__ __forceinline__ float inverse_of(float sum, float top) {
  return sum > 0.0f || sum != sum ? 1.0f / sum : top == -__builtin_inff() ? 0.0f : __builtin_nanf("");
}

// Registers: two or more wavefronts a SIMD keep the matrix accumulators in
// ordinary registers; with all 512 of one, the compiler moves them to and from
// the accumulation registers around every tile.  Heads of 256 with 32 rows run that
// way all the same (128 accumulators and up to 128 words of queries a lane; two
// wavefronts would spill them).  There, and in two fp16 forms of 16 rows, a few registers
// that the loop over tiles does not use go to scratch memory, up to 60 bytes a lane.
// ROWS: rows of a block at most, 8, 16 or 32.  Eight rows leave half of a
// tile's columns free: columns 8..15 then take the second pieces of the same
// rows (of fp16 queries, and of the weights), which halves the products of
// those; a lane's two column halves are added where they meet (rotating a row
// of 16 lanes by 8).
// MANY: several new tokens, so that rows see different tokens.  (One new token, without
// what that takes: 48 ragged sequences 26.1 us against 26.6 with it, 16 x 4000 tokens of
// 8 heads of 256 with 32 rows 62.7 and 64.5.)
template <int D, int ROWS, bool F16, bool MANY>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(kv4_waves(D, ROWS)))) void kv4_attend_kernel(AttendArgs a) {
  constexpr int NB = D / 32;                       // blocks of 32 channels
  constexpr int NT = ROWS == 32 ? 2 : 1;           // 16-column tiles
  constexpr bool HALF = ROWS == 8;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, c4 = lane >> 4;
  const bool second = HALF && col >= 8;            // a lane of the second pieces
  __shared__ float sm[4][ROWS], sl[4][ROWS];
  __shared__ __attribute__((aligned(16))) float so[4][ROWS][D + 4];    // + 4: columns on different banks

  const int HR = a.L.H * a.row_blocks;
  Line line;
  const int all = line_length(a, line, lane) * HR;
  const int per = (all + a.W - 1) / a.W;
  const int u0 = blockIdx.x * per, u1 = min(u0 + per, all);
  if (u0 >= u1) return;
  // the sequence that u0 falls into, and where it begins
  int b = 0, start = 0;
  for (int base = 0, before = 0;; base += 64) {
    if (line.base != base) line.look(a, base, before, lane);
    const uint64_t past = __ballot(line.upto * HR > u0);
    before = __builtin_amdgcn_readlane(line.upto, 63);
    if (past) {
      const int i = __builtin_ctzll(past);
      b = base + i;
      start = (__builtin_amdgcn_readlane(line.upto, i) - kKv4Start -
               seq_chunks(__builtin_amdgcn_readlane(line.len, i))) * HR;
      break;
    }
  }

  // the lane's rows of the first block of rows
  int row_i[NT], row_j[NT];
  bool row_in[NT];
#pragma unroll
  for (int x = 0; x < NT; ++x) {
    const int r = HALF ? col & 7 : 16 * x + col;
    row_in[x] = r < a.rows;
    row_i[x] = row_in[x] ? r / a.group : 0;
    row_j[x] = row_in[x] ? r % a.group : 0;
  }

  int u = u0;
  while (u < u1) {
    if (b - line.base >= 64) line.look(a, line.base + 64, 0, lane);
    const int len = __builtin_amdgcn_readlane(line.len, b - line.base);
    const int n = seq_chunks(len), span = n + kKv4Start;
    const int hr = __builtin_amdgcn_readfirstlane((u - start) / span);
    const int at = u - start - hr * span;                 // place in this (sequence, head)
    const int ch0 = max(at - kKv4Start, 0), ch1 = min(at - kKv4Start + u1 - u, n);
    const int next = start + (hr + 1) * span;
    const int next_b = hr + 1 == HR ? b + 1 : b, next_start = hr + 1 == HR ? next : start;
    if (ch1 <= 0) break;                                  // the line ends before the first chunk
    const int h = hr / a.row_blocks, r0 = hr % a.row_blocks * ROWS;
    // queries: row r = i * group + j is new token i, head h * group + j
    // (asked for before the pages, which are waited for)
    uint4 qv[NT][NB];
    int limit[NT];                                 // tokens that the lane's row sees
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      int i = row_i[x], j = row_j[x];
      bool real = row_in[x];
      if (a.row_blocks > 1) {
        const int r = r0 + (HALF ? col & 7 : 16 * x + col);
        real = r < a.rows;
        i = real ? r / a.group : 0;
        j = real ? r % a.group : 0;
      }
      limit[x] = min(len, len - a.Q + i + 1);
      const uint16_t *src = a.q + b * a.q_b + i * a.q_i + (int64_t)(h * a.group + j) * a.q_h + 8 * c4;
#pragma unroll
      for (int s = 0; s < NB; ++s)
        qv[x][s] = real ? *reinterpret_cast<const uint4 *>(src + 32 * s) : make_uint4(0, 0, 0, 0);
    }
    Pages pages{a.table + (int64_t)b * a.width, a.width, a.L.pages, 0, 0};
    pages.load(ch0 * kKv4Chunk >> a.L.page_shift, lane);
    v8bf qh[NT][NB], ql[NT][F16 && !HALF ? NB : 1];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int s = 0; s < NB; ++s) {
        const uint4 v = make_uint4(qv[x][s].x ^ a.flip, qv[x][s].y ^ a.flip, qv[x][s].z ^ a.flip, qv[x][s].w ^ a.flip);
        if constexpr (F16) {
          // the upper 16 bits of the value as float32, and the rest (a value that is
          // not finite leaves a row that is not, either way)
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t f0 = __float_as_uint(wide<true>(in[e] & 0xFFFFu)), f1 = __float_as_uint(wide<true>(in[e] >> 16));
            hi[e] = __builtin_amdgcn_perm(f1, f0, 0x07060302u);
            lo[e] = pack_bf16(__uint_as_float(f0) - bf16_hi(f0), __uint_as_float(f1) - bf16_hi(f1));
          }
          if constexpr (HALF) {
            qh[x][s] = as_v8bf(second ? make_uint4(lo[0], lo[1], lo[2], lo[3]) : make_uint4(hi[0], hi[1], hi[2], hi[3]));
          } else {
            qh[x][s] = as_v8bf(make_uint4(hi[0], hi[1], hi[2], hi[3]));
            ql[x][s] = as_v8bf(make_uint4(lo[0], lo[1], lo[2], lo[3]));
          }
        } else {
          qh[x][s] = as_v8bf(v);
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

    const int t1 = min(ch1 * kKv4Chunk, len);
    const int whole = len - a.Q + 1;               // tokens that every row sees
    // One tile's keys and one tile's values are in registers; the next ones
    // are asked for as soon as these are used up, so the keys arrive while
    // the weights and the values are worked on, the values while the keys
    // are.  The loads are unconditional (past the end, one line of the last
    // tile), so that the number outstanding is known at every wait.
    const int tw = ch0 * kKv4Chunk + 32 * w;
    const int last = tw + (t1 - 1 - tw) / kKv4Chunk * kKv4Chunk;
    Keys<D> keys;
    Values<D> vals;
    Place place;
    uint64_t not_finite = 0;
    if (tw < t1) {
      place = locate<D>(a, pages, h, tw, lane);
      load_keys<D>(place, lane, keys);
      load_values<D>(place, lane, vals);
    }
    for (int t = tw; t < t1; t += kKv4Chunk) {
      const Place next = locate<D>(a, pages, h, min(t + kKv4Chunk, last), lane);
      const int nlane = t < last ? lane : 0;
      v4f s[NT][2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int x = 0; x < NT; ++x) s[x][g] = v4f{};
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          const float sc = scale_of(keys.s[g][k / 4], k % 4);
          const uint32_t kw = keys.k[g][k];
          const v8bf ka = as_v8bf(make_uint4(two_values<0>(kw, sc), two_values<1>(kw, sc), two_values<2>(kw, sc),
                                             two_values<3>(kw, sc)));
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            s[x][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, qh[x][k], s[x][g], 0, 0, 0);
            if constexpr (F16 && !HALF) s[x][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, ql[x][k], s[x][g], 0, 0, 0);
          }
        }
      }
      load_keys<D>(next, nlane, keys);
      if constexpr (F16 && HALF) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[0][g][i] += other_half(s[0][g][i]);
      }
      if (t + 32 > whole || !place.ok[0] || !place.ok[1]) {
        // rows' own limits, and units without a page
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = t + 16 * g + 4 * c4 + i;
#pragma unroll
            for (int x = 0; x < NT; ++x)
              if (!place.ok[g] || tok >= limit[x]) s[x][g][i] = -__builtin_inff();
          }
          // what stands in the cache past the end may be anything, and zero
          // times it must be zero: such tokens' codes and scales are cleared
          uint32_t keep = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (place.ok[g] && t + 16 * g + 4 * c4 + i < len) keep |= 0xFFu << (8 * i);
#pragma unroll
          for (int k = 0; k < NB; ++k) vals.v[g][k] &= keep;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < NB; ++k)
              if (!(keep >> (8 * i) & 1u)) vals.s[g][(i * NB + k) / 4] &= ~(0xFFu << (8 * ((i * NB + k) % 4)));
        }
        // Where rows see different tokens, a block of values that is not finite (scale
        // byte 255) must not meet the zero weights of the rows that do not see its
        // token: it gets another scale, and the rows that do become NaN after the last tile.
        if constexpr (MANY) {
          uint32_t any = 0;
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              const uint32_t bytes = bytes_255(vals.s[g][i]);
              vals.s[g][i] &= ~bytes;
              any |= bytes;
            }
          not_finite |= __ballot(any != 0);
        }
      }
      // running maximum (of the bare products) and weights
      v8bf ph[NT], pl[NT];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const v4f s0 = s[x][0], s1 = s[x][1];
        const float top = column_max(fmaxf(fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s0[2], s0[3])),
                                           fmaxf(fmaxf(s1[0], s1[1]), fmaxf(s1[2], s1[3]))));
        if (__ballot(top > m[x])) {
          const float now = fmaxf(m[x], top);
          const float f = __builtin_amdgcn_exp2f((m[x] - now) * a.scale);
          m[x] = now;
          // a row that has seen no token yet keeps nothing (f is not a number there)
          const float g = now == -__builtin_inff() ? 0.0f : f;
          l[x] *= g;
#pragma unroll
          for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[x][i][e] *= g;
        }
        // Differences are taken of the bare products: of scaled ones a fused product would hold
        // the rounding of the maximum, many units of the exponent where scores are far from zero.
        const float ref = m[x] == -__builtin_inff() ? 0.0f : m[x];
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = __builtin_amdgcn_exp2f((s[x][g][2 * i] - ref) * a.scale);
            const float p1 = __builtin_amdgcn_exp2f((s[x][g][2 * i + 1] - ref) * a.scale);
            l[x] += p0 + p1;
            const uint32_t pk = pack_bf16(p0, p1);
            hi[2 * g + i] = pk;
            lo[2 * g + i] = pack_bf16(p0 - bf16_lo(pk), p1 - bf16_hi(pk));
          }
        if constexpr (HALF) {
          ph[x] = as_v8bf(second ? make_uint4(lo[0], lo[1], lo[2], lo[3]) : make_uint4(hi[0], hi[1], hi[2], hi[3]));
        } else {
          ph[x] = as_v8bf(make_uint4(hi[0], hi[1], hi[2], hi[3]));
          pl[x] = as_v8bf(make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t lo[4], hi[4];                     // channels 32 k + col, and 16 above
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t vw = vals.v[g][k];
          const uint32_t x0 = two_values<0>(vw, scale_of(vals.s[g][k / 4], k % 4));
          const uint32_t x1 = two_values<1>(vw, scale_of(vals.s[g][(NB + k) / 4], (NB + k) % 4));
          const uint32_t x2 = two_values<2>(vw, scale_of(vals.s[g][(2 * NB + k) / 4], (2 * NB + k) % 4));
          const uint32_t x3 = two_values<3>(vw, scale_of(vals.s[g][(3 * NB + k) / 4], (3 * NB + k) % 4));
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
          if constexpr (!HALF) {
            o[x][2 * k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, pl[x], o[x][2 * k], 0, 0, 0);
            o[x][2 * k + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, pl[x], o[x][2 * k + 1], 0, 0, 0);
          }
        }
      }
      load_values<D>(next, nlane, vals);
      place = next;
    }

    if (MANY && __builtin_expect(not_finite != 0, 0)) {
      // the rows that see a block of values that is not finite (the scales are read again,
      // so that nothing is kept for this in the loop's registers)
      for (int t = tw; t < t1; t += kKv4Chunk) {
        if (t + 32 <= whole) continue;
        pages.load(t >> a.L.page_shift, lane);
        const Place p = locate<D>(a, pages, h, t, lane);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (!p.ok[g]) continue;
          uint32_t sc[NB];
          load_words(sc, p.unit[g] + 16 * D + D / 2 + c4 * (D / 8));
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              bool sees = false;                   // one of the lane's four tokens
#pragma unroll
              for (int i = 0; i < 4; ++i)
                sees |= (bytes_255(sc[(i * NB + k) / 4]) >> (8 * ((i * NB + k) % 4)) & 0x80u) != 0 &&
                        t + 16 * g + 4 * c4 + i < limit[x];
              uint64_t rows = __ballot(sees);      // of a column's four lanes
              rows |= rows >> 32;
              rows |= rows >> 16;
              if (rows >> col & 1) o[x][2 * k] = o[x][2 * k + 1] = v4f{} + __builtin_nanf("");
            }
        }
      }
    }

    // A row whose scores are all minus infinity is 0 / 0, and one that sees no token is
    // zero.  Both have no maximum yet; the first gets the lowest number for one.
#pragma unroll
    for (int x = 0; x < NT; ++x)
      if (__builtin_expect(__ballot(m[x] == -__builtin_inff()) != 0, 0))
        for (int t = tw; t < t1; t += kKv4Chunk) {
          pages.load(t >> a.L.page_shift, lane);
          const Place p = locate<D>(a, pages, h, t, lane);
          if (m[x] == -__builtin_inff() && ((p.ok[0] && t < limit[x]) || (p.ok[1] && t + 16 < limit[x]))) m[x] = -kLargest;
        }

    // The four wavefronts' states meet: all of them into LDS, then every
    // thread takes some channels of one row, relative to the row's largest
    // maximum, and writes them.
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      l[x] += __shfl_xor(l[x], 16);
      l[x] += __shfl_xor(l[x], 32);
      const bool mine = !second;
      if (mine && c4 == 0) {
        sm[w][16 * x + col] = m[x];
        sl[w][16 * x + col] = l[x];
      }
#pragma unroll
      for (int k = 0; k < 2 * NB; ++k) {
        if constexpr (HALF) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[x][k][e] += other_half(o[x][k][e]);
        }
        if (mine) *reinterpret_cast<v4f *>(&so[w][16 * x + col][16 * k + 4 * c4]) = o[x][k];
      }
    }
    __syncthreads();
    {
      constexpr int THREADS = 256 / ROWS, EACH = D / THREADS, U = EACH < 4 ? EACH : 4;
      const int c = threadIdx.x / THREADS, first = threadIdx.x % THREADS * U;
      const int r = r0 + c;
      float f[4], top = fmaxf(fmaxf(sm[0][c], sm[1][c]), fmaxf(sm[2][c], sm[3][c])), sum = 0.0f;
      const float ref = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[k] = __builtin_amdgcn_exp2f((sm[k][c] - ref) * a.scale);
        sum = __builtin_fmaf(sl[k][c], f[k], sum);
      }
      const bool done = ch0 == 0 && ch1 == n;
      const float inv = done ? inverse_of(sum, top) : 1.0f;
      const int i = r / a.group, j = r % a.group;
      uint16_t *out = a.out + (((int64_t)b * a.Q + i) * (a.L.H * a.group) + h * a.group + j) * D;
      const int64_t slot = (2 * (int64_t)blockIdx.x + (u > u0 ? 1 : 0)) * a.block_rows + c;
      if (r < a.rows) {
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += THREADS * U) {
          const int d = d0 + first;
          float y[U];
#pragma unroll
          for (int e = 0; e < U; ++e) {
            y[e] = so[0][c][d + e] * f[0];
#pragma unroll
            for (int k = 1; k < 4; ++k) y[e] = __builtin_fmaf(so[k][c][d + e], f[k], y[e]);
            y[e] *= inv;
          }
#pragma unroll
          for (int e = 0; e < U; e += 2) {
            if (done) {
              if constexpr (F16)
                *reinterpret_cast<v2h *>(out + d + e) = v2h{(_Float16)y[e], (_Float16)y[e + 1]};
              else
                *reinterpret_cast<uint32_t *>(out + d + e) = pack_bf16(y[e], y[e + 1]);
            } else {
              *reinterpret_cast<float2 *>(a.part + slot * D + d + e) = make_float2(y[e], y[e + 1]);
            }
          }
        }
        if (!done && first == 0) {
          float *ml = a.part + 2 * (int64_t)a.W * a.block_rows * D + slot * 2;
          ml[0] = top;
          ml[1] = sum;
        }
      }
    }
    __syncthreads();
    u = next;
    b = next_b;
    start = next_start;
  }
}

// One wavefront (WIDE: four, a workgroup) per (sequence, new token, query
// head) whose chunks went to more than one workgroup: the pieces' states,
// relative to their largest maximum, added in order.  A lane holds D / 64
// channels; with four wavefronts, w takes pieces w, w + 4, ...
template <int D, bool F16, bool WIDE>
__global__ __launch_bounds__(256) void kv4_join_kernel(AttendArgs a) {
  constexpr int V = D / 64, STEP = WIDE ? 4 : 1;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int Hq = a.L.H * a.group;
  const int row = WIDE ? blockIdx.x : blockIdx.x * 4 + w;
  if (row >= a.B * a.Q * Hq) return;
  const int hq = row % Hq, i = row / Hq % a.Q, b = row / Hq / a.Q;
  const int h = hq / a.group, r = i * a.group + hq % a.group;
  const int HR = a.L.H * a.row_blocks;
  Line line;
  int all = 0, n = 0, first = 0;
  for (int base = 0; base < a.B; base += 64) {
    all = line.look(a, base, all, lane);
    if (b >= base && b < base + 64) {
      n = seq_chunks(__builtin_amdgcn_readlane(line.len, b - base));
      first = (__builtin_amdgcn_readlane(line.upto, b - base) - n - kKv4Start) * HR;
    }
  }
  const int per = (all * HR + a.W - 1) / a.W;
  // the line's place of the first chunk, and the workgroups with a chunk
  first += (h * a.row_blocks + r / a.block_rows) * (n + kKv4Start);
  const int g0 = (first + kKv4Start) / per, g1 = (first + kKv4Start + n - 1) / per;
  if (g0 == g1) return;
  const int pieces = g1 - g0 + 1;
  const int rb = r % a.block_rows;
  const float *ml = a.part + 2 * (int64_t)a.W * a.block_rows * D;
  auto place = [&](int p) {
    return (int64_t)(2 * (g0 + p) + (p == 0 && first > g0 * per ? 1 : 0)) * a.block_rows + rb;
  };
  float top = -__builtin_inff();
  for (int p = lane; p < pieces; p += 64) top = fmaxf(top, ml[place(p) * 2]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float ref = top == -__builtin_inff() ? 0.0f : top;
  float acc[V] = {}, l = 0.0f;
#pragma unroll 4
  for (int p = WIDE ? w : 0; p < pieces; p += STEP) {
    const int64_t at = place(p);
    const float f = __builtin_amdgcn_exp2f((ml[at * 2] - ref) * a.scale);
    l = __builtin_fmaf(ml[at * 2 + 1], f, l);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = __builtin_fmaf(a.part[at * D + lane * V + e], f, acc[e]);
  }
  if constexpr (WIDE) {
    __shared__ float so[3][D], sl[3];
    if (w > 0) {
#pragma unroll
      for (int e = 0; e < V; ++e) so[w - 1][lane * V + e] = acc[e];
      if (lane == 0) sl[w - 1] = l;
    }
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      l += sl[k];
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += so[k][lane * V + e];
    }
  }
  const float inv = inverse_of(l, top);
  const int64_t at = (((int64_t)b * a.Q + i) * Hq + hq) * D + lane * V;
#pragma unroll
  for (int e = 0; e < V; ++e)
    a.out[at + e] = F16 ? __builtin_bit_cast(uint16_t, (_Float16)(acc[e] * inv))
                        : __builtin_bit_cast(uint16_t, (__bf16)(acc[e] * inv));
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
  const int64_t threads = ((int64_t)T + 15) / 16 * 16 * L.H * 2 * (L.D / 32);
  if (threads > (int64_t)1 << 31) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_append: T=%d", T);
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
  const int64_t threads = ((int64_t)T + 15) / 16 * 16 * L.H * 2 * (L.D / 32);
  if (threads > (int64_t)1 << 31) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_read: T=%d", T);
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
  if (!kv4_query_ok(B, Q, Hq, L.H) || table_width < 1 || (int64_t)table_width << L.page_shift > kKv4MaxTokens)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_attention: B=%d Q=%d Hq=%d over %d heads, page table of %d columns",
                B, Q, Hq, L.H, table_width);
  const int rows = Q * (Hq / L.H), block = rows > 16 ? 32 : rows > 8 ? 16 : 8, row_blocks = (rows + block - 1) / block;
  // the chunks of the longest sequences that the table can name, on the kernels' 32-bit line
  const int64_t chunks = (((int64_t)table_width << L.page_shift) + kKv4Chunk - 1) / kKv4Chunk;
  if ((chunks + kKv4Start) * B * L.H * row_blocks + kKv4Groups > 0x7FFFFFFF)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_kv4_attention: B=%d Q=%d Hq=%d with a page table of %d columns is too much work",
                B, Q, Hq, table_width);
  if (B == 0) return SVDQ_OK;
  if (!q || !page_table || !seq_lens || !out || !workspace)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_attention: NULL pointer");
  const int64_t strides[3] = {q_batch, q_token, q_head};
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || ((uintptr_t)page_table & 3u) ||
      ((uintptr_t)seq_lens & 3u) || !strides_ok(strides, 3))
    return fail(SVDQ_ERR_INVALID_ARGUMENT,
                "svdq_kv4_attention: misaligned pointer, or a stride that is not a multiple of 8");
  if (!(fabsf(scale) < 0x1p127f))        // times log2(e) it is a float32 number
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_kv4_attention: scale is not a number below 2^127");
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
  a.rows = rows;
  a.row_blocks = row_blocks;
  a.block_rows = rows < block ? rows : block;
  // Maxima are taken of the bare products, so the scale's sign goes to the queries.
  a.scale = log2_scale(scale);
  a.flip = scale < 0.0f ? 0x80008000u : 0u;
  a.out = static_cast<uint16_t *>(out);
  a.part = static_cast<float *>(workspace);
  // no more workgroups than there can be chunks
  const int64_t most = chunks * B * L.H * row_blocks;
  const int resident = 256 * kv4_waves(L.D, block);
  a.W = (int)(most < resident ? most : resident);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  // A workgroup joins each row where there are few rows of many pieces, at most 64 rows
  // for each piece of one, and a wavefront where there are more.  With a workgroup and
  // with a wavefront (rows, pieces on average): 128 and 24 74.5 and 75.7 us; 512 and 24
  // 17.1 and 18.9; 384 and 8 41.4 and 41.7; 1024 and 16 45.1 and 45.6; 1024 and 12 23.3
  // and 23.0; 768 and 4 42.9 and 42.5; 1536 and 6 23.6 and 22.6; 2560 and 4 29.7 and 26.7.
  const int64_t all_rows = (int64_t)B * Q * Hq;
  const bool wide_join = all_rows * B * L.H * row_blocks <= 64ll * a.W;
  const dim3 join_grid((unsigned)(wide_join ? all_rows : (all_rows + 3) / 4));
#define KV4_GO(DD, NN, FF)                                                                                  \
  do {                                                                                                      \
    if (Q > 1) hipLaunchKernelGGL((kv4_attend_kernel<DD, NN, FF, true>), dim3(a.W), dim3(256), 0, stream, a); \
    else hipLaunchKernelGGL((kv4_attend_kernel<DD, NN, FF, false>), dim3(a.W), dim3(256), 0, stream, a);    \
    if (wide_join) hipLaunchKernelGGL((kv4_join_kernel<DD, FF, true>), join_grid, dim3(256), 0, stream, a); \
    else hipLaunchKernelGGL((kv4_join_kernel<DD, FF, false>), join_grid, dim3(256), 0, stream, a);          \
  } while (0)
#define KV4_ROWS(DD, FF)                       \
  do {                                         \
    if (block == 8) KV4_GO(DD, 8, FF);         \
    else if (block == 16) KV4_GO(DD, 16, FF);  \
    else KV4_GO(DD, 32, FF);                   \
  } while (0)
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
