// Cross attention: queries over an encoder's states of another length.
//
//  cross_list_kernel     the visible states of each batch row, where there is a mask over many
//  cross_many_kernel     attention of a tile of rows over a piece of the states
//  cross_near_kernel     the same over few states, all of them in LDS
//  cross_few_kernel      the same for a handful of rows
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

constexpr float kLowest = -0x1.fffffep127f;      // the maximum of a row that has met no score above -inf
// How far (log2) scores may pass the running maximum before the sums are
// rescaled: nearly all tiles go without.
constexpr float kSlack = 8.0f;
// From this maximum on (log2) what rounding to float32 takes off it, up to half a step, is kept beside it: at
// 2^24 that is one unit of the exponent, and soon more than the weights have room for.  Below it is 2^-9 at most.
constexpr float kFar = 0x1p16f;
// Weights carry 2^shift, which the result's division takes off again.  Those of bfloat16 2^-9, for
// that none passes 1, slack and a maximum's rounding included: a product with a value of V is then no larger than that
// one, as far as float32 and bfloat16 reach, and a weight is lost from 2^-117 down.  Those of float16 2^7, so at most
// 2^15: the type's smallest step is then at most 2^-31 of the largest weight, so that many small ones do not vanish.
template <bool F16>
constexpr float kShift = F16 ? 7.0f : -kSlack - 1.0f;

struct CrossArgs {
  const uint16_t *q, *k, *v;
  int64_t q_b, q_i, q_h, k_b, k_t, k_h, v_b, v_t, v_h;
  const int *lens;                       // states of a batch row (or NULL: all)
  const uint8_t *mask;                   // which of them are visible: the workgroup lists them itself; or
  const int *index, *count;              // [B, Lk] the visible ones' numbers, and how many
  uint16_t *out;
  float *ml, *o;                         // pieces: [place][row] (m, l), and [..][D]
  float *rest;                           // and what goes with an m from kFar on, elsewhere not written
  int B, Lq, Lk, Hq, Hkv, group, D, rows, tiles, parts;
  int run, work;                         // pieces of work; how many go to one XCD together
  int line, least;                       // parts of all batch rows together, shared out by their lengths (0: `parts` each); tiles of one
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

// Rows of K and V in LDS, for DB blocks of 32 channels: SLOTS chunks of 16 bytes, permuted
// so that no read meets a bank twice (64 banks of 4 bytes).  K is read 16 rows at the same chunk,
// V 4 neighbouring rows at 4 neighbouring chunks.  Where the slots are a power of two, a chunk's slot is the chunk
// xor a number that goes with the row; 12 slots are turned by a quarter of the row in K (the
// rows' starts, 48 words apart, take four places in the banks), and stay in V.
template <int DB>
struct Rows {
  static constexpr int SLOTS = DB <= 2 ? 8 : DB == 3 ? 12 : DB == 4 ? 16 : 32, ROW = SLOTS * 16;
  static constexpr bool XOR = SLOTS != 12;
  static __device__ __forceinline__ int k_swap(int row) {
    return SLOTS == 8 ? row >> 1 & 7 : SLOTS == 12 ? row >> 2 & 3 : SLOTS == 16 ? row & 15 : row & 7;
  }
  static __device__ __forceinline__ int v_swap(int row) { return SLOTS == 8 ? (row >> 1 & 1) << 2 : SLOTS == 12 ? 0 : (row & 3) << 2; }
  static __device__ __forceinline__ int k_slot(int row, int chunk) {
    const int s = chunk + k_swap(row);
    return XOR ? chunk ^ k_swap(row) : s >= 12 ? s - 12 : s;
  }
  static __device__ __forceinline__ int k_chunk(int row, int slot) {
    const int c = slot - k_swap(row);
    return XOR ? slot ^ k_swap(row) : c < 0 ? c + 12 : c;
  }
  static __device__ __forceinline__ int v_slot(int row, int chunk) { return chunk ^ v_swap(row); }
  static __device__ __forceinline__ int v_chunk(int row, int slot) { return slot ^ v_swap(row); }
};

// Numbers the visible ones of n states in order, by WAVES wavefronts, and returns how many.  Eight states
// a thread at a time, 64 WAVES apart: one trip to memory, and a ballot for each.
template <int WAVES>
__device__ __forceinline__ int list_visible(const uint8_t *seen, int n, int *out) {
  __shared__ int sums[8][WAVES];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int all = 0;
  for (int64_t from = 0; from < n; from += 8 * 64 * WAVES) {
    uint8_t flag[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = from + 64 * WAVES * i + threadIdx.x;
      flag[i] = t < n ? seen[t] : 0;
    }
    uint64_t votes[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      votes[i] = __ballot(flag[i] != 0);
      if (lane == 0) sums[i][w] = __popcll(votes[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int at = all + __popcll(votes[i] & ((1ull << lane) - 1));
#pragma unroll
      for (int v = 0; v < WAVES; ++v) {
        const int x = sums[i][v];
        at += v < w ? x : 0;
        all += x;
      }
      if (flag[i] != 0) out[at] = (int)(from + 64 * WAVES * i + threadIdx.x);
    }
    __syncthreads();
  }
  return all;
}

// The parts of a line that each of up to 64 batch rows gets, by its tiles of `keys` states: its share, rounded
// down, and one at least, together no more than line + B.  A lane holds a batch row's.
struct Shares {
  int n, tiles, parts, before;           // states, tiles, parts, parts of the batch rows before
  __device__ __forceinline__ Shares(const CrossArgs &a, int keys) {
    const int lane = threadIdx.x & 63;
    n = lane < a.B ? min(max(a.lens[lane], 0), a.Lk) : 0;
    tiles = (n + keys - 1) / keys;
    int64_t all = tiles;
#pragma unroll
    for (int i = 32; i > 0; i >>= 1) all += __shfl_xor((long long)all, i);
    parts = tiles > 0 ? max(1, min((int)((int64_t)tiles * a.line / all), tiles / a.least)) : 0;
    before = parts;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
      const int x = __shfl_up(before, i);
      if (lane >= i) before += x;
    }
    before -= parts;
  }
};

// A workgroup's piece of the work, the same in all its lanes, and its batch row's states.
struct Piece {
  int tile_row, part, b, hk, n, t0, t1;
  int place;                             // of its sums for the join
  const int *index;                      // where there is a mask
  bool any;
  // Workgroups are dealt out to the eight XCDs in turn: runs of neighbouring row tiles,
  // which read the same states, go to one XCD.
  __device__ __forceinline__ Piece(const CrossArgs &a, int keys) {
    const uint32_t x = blockIdx.x & 7, i = blockIdx.x >> 3, run = (uint32_t)a.run;
    const uint32_t id = (i / run * 8 + x) * run + i % run;
    any = id < (uint32_t)a.work;
    if (!any) return;
    const uint32_t piece = id / (uint32_t)a.tiles;
    tile_row = (int)(id - piece * (uint32_t)a.tiles);
    if (a.line) {
      const uint32_t at = piece / (uint32_t)a.Hkv;
      hk = (int)(piece - at * (uint32_t)a.Hkv);
      place = (int)piece;
      const Shares s(a, keys);
      const uint64_t mine = __ballot(s.before <= (int)at && (int)at < s.before + s.parts);
      any = mine != 0;
      if (!any) return;
      b = __builtin_amdgcn_readfirstlane(__ffsll((long long)mine) - 1);
      n = __builtin_amdgcn_readlane(s.n, b);
      part = (int)at - __builtin_amdgcn_readlane(s.before, b);
      span(__builtin_amdgcn_readlane(s.tiles, b), __builtin_amdgcn_readlane(s.parts, b));
      return;
    }
    const int bh = (int)(piece / (uint32_t)a.parts);
    part = (int)piece - bh * a.parts;
    b = (int)((uint32_t)bh / (uint32_t)a.Hkv);
    hk = bh - b * a.Hkv;
    place = part * a.B * a.Hkv + bh;
  }
  __device__ __forceinline__ void span(int all, int parts) {
    t0 = parts == 1 ? 0 : (int)((uint64_t)(uint32_t)all * (uint32_t)part / (uint32_t)parts);
    t1 = parts == 1 ? all : (int)((uint64_t)(uint32_t)all * (uint32_t)(part + 1) / (uint32_t)parts);
  }
  // The states, listed in `list` if they are not listed yet, and this piece's tiles of `keys` of them.
  template <bool LIST, int WAVES>
  __device__ __forceinline__ void cut(const CrossArgs &a, int keys, int *list) {
    if (a.line) return;                  // by its share already
    n = a.lens ? min(max(a.lens[b], 0), a.Lk) : a.Lk;
    if constexpr (LIST) {
      if (a.mask) {
        n = list_visible<WAVES>(a.mask + (int64_t)b * a.Lk, n, list);
        index = list;
      } else {
        n = a.count[b];
        index = a.index + (int64_t)b * a.Lk;
      }
    }
    span((int)((uint32_t)(n + keys - 1) / (uint32_t)keys), a.parts);
  }
};

// Where a lane's row is, and its operand of the first product.
struct Row {
  int row, qi, hq;
  __device__ __forceinline__ Row(const CrossArgs &a, const Piece &p, int row_) : row(row_) {
    const int rr = min(row, a.rows - 1);
    qi = rr / a.group;
    hq = p.hk * a.group + rr - qi * a.group;
  }
  template <int STEPS>
  __device__ __forceinline__ void load(const CrossArgs &a, const Piece &p, int h, v4u (&q)[STEPS]) const {
    const uint16_t *src = a.q + (int64_t)p.b * a.q_b + qi * a.q_i + hq * a.q_h;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int at = 16 * s + 8 * h;
      q[s] = at < a.D ? *reinterpret_cast<const v4u *>(src + at) : v4u{0u, 0u, 0u, 0u};
    }
  }
  // the scale's sign
  template <int STEPS>
  static __device__ __forceinline__ void flip(const CrossArgs &a, v4u (&q)[STEPS]) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) q[s] ^= a.flip;
  }
};

// Copies a tile's rows into LDS, K's and V's, 64 chunks at a time, by WAVES wavefronts.
template <int DB, int KEYS, int WAVES, bool LIST>
struct Copier {
  typedef Rows<DB> L;
  static constexpr int ALL = KEYS * L::SLOTS / 64, COPIES = (ALL + WAVES - 1) / WAVES;
  // A lane copies the same chunk each time where the wavefronts' rows together are a multiple of the swaps' period.
  static constexpr bool SAME = L::XOR && WAVES >= 4;
  const uint8_t *k, *v;
  const int *index;
  uint32_t k_t, v_t;                     // bytes from a state to the next, below 2^25
  int n, chunks, lane, w;
  uint32_t key[LIST ? COPIES : 1];       // the listed states of the next tile's rows, this lane's
  __device__ __forceinline__ Copier(const CrossArgs &a, const Piece &p, int lane_, int w_)
      : k(reinterpret_cast<const uint8_t *>(a.k + (int64_t)p.b * a.k_b + p.hk * a.k_h)),
        v(reinterpret_cast<const uint8_t *>(a.v + (int64_t)p.b * a.v_b + p.hk * a.v_h)), index(p.index), k_t((uint32_t)(2 * a.k_t)),
        v_t((uint32_t)(2 * a.v_t)), n(p.n), chunks(a.D / 8), lane(lane_), w(w_) {}
  __device__ __forceinline__ bool mine(int j) const { return ALL % WAVES == 0 || WAVES * j + w < ALL; }
  __device__ __forceinline__ int row(int j) const { return (64 * (WAVES * j + w) + lane) / L::SLOTS; }
  __device__ __forceinline__ int slot(int j) const { return (64 * (WAVES * j + w) + lane) % L::SLOTS; }
  // Reads tile t's part of the list, a tile ahead of its use.
  __device__ __forceinline__ void look_up(int t) {
    if constexpr (LIST) {
#pragma unroll
      for (int j = 0; j < COPIES; ++j) key[j] = (uint32_t)index[min(t * KEYS + row(j), n - 1)];
    }
  }
  // The rows of K (or of V): `chunk` of each, that of copy j.
  template <typename Chunk>
  __device__ __forceinline__ void half(int t, const uint8_t *rows, uint32_t step, const Chunk &chunk, uint32_t to) const {
    const bool whole = !LIST && (t + 1) * KEYS <= n;
    auto copy = [&](int j) __attribute__((always_inline)) {
      const uint32_t at = __builtin_amdgcn_readfirstlane(to + 1024 * (WAVES * j + w));
      if (whole) {
        // a scalar base (also where the compiler has lost sight of that) and the lane's 32-bit offset
        const int skip = L::XOR ? (WAVES * j + w) * (64 / L::SLOTS) : 0;
        const uint64_t first = reinterpret_cast<uint64_t>(rows) + (uint64_t)(uint32_t)(t * KEYS + skip) * step;
        const uint64_t base = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(first >> 32)) << 32 |
                              (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)first);
        lds_dma16_moved(reinterpret_cast<const void *>(base), (uint32_t)(row(j) - skip) * step + 16 * chunk(j), at);
      } else {                           // rows behind the last state repeat it
        const uint32_t key_at = LIST ? key[LIST ? j : 0] : (uint32_t)min(t * KEYS + row(j), n - 1);
        lds_dma16(rows + 16 * chunk(j) + (uint64_t)key_at * step, at);
      }
    };
    if (SAME && (whole && L::SLOTS == 4 * DB && chunks == 4 * DB)) {
#pragma unroll
      for (int j = 0; j < COPIES; ++j) copy(j);
    } else if constexpr (SAME) {
      if (chunk(0) < chunks) {
#pragma unroll
        for (int j = 0; j < COPIES; ++j) copy(j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < COPIES; ++j)
        if (mine(j) && chunk(j) < chunks) copy(j);
    }
  }
  __device__ __forceinline__ void both(int t, uint32_t k_to, uint32_t v_to) const {
    half(t, k, k_t, [&](int j) __attribute__((always_inline)) { return L::k_chunk(row(SAME ? 0 : j), slot(SAME ? 0 : j)); }, k_to);
    half(t, v, v_t, [&](int j) __attribute__((always_inline)) { return L::v_chunk(row(SAME ? 0 : j), slot(SAME ? 0 : j)); }, v_to);
  }
};

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)p);
}
// K's chunks from D to 32 DB channels, which no copy writes: zeros from the start.  (Queries are zero
// there, but what LDS holds may be NaN.  V's only reach results that are not stored.)
template <int DB>
__device__ __forceinline__ void clear_pads(const CrossArgs &a, uint8_t *rows, int count, int thread, int threads) {
  const int chunks = a.D / 8, pads = 4 * DB - chunks;
  for (int i = thread; i < count * pads; i += threads) {
    const int r = i / pads;
    *reinterpret_cast<uint4 *>(rows + r * Rows<DB>::ROW + Rows<DB>::k_slot(r, chunks + i - r * pads) * 16) = make_uint4(0, 0, 0, 0);
  }
}
// V's rows from `from` to `to`, behind the last state: zero, whatever that one holds.
template <int DB>
__device__ __forceinline__ void clear_rows(uint8_t *rows, int from, int to, int thread, int threads) {
  for (int i = from * Rows<DB>::ROW + thread * 16; i < to * Rows<DB>::ROW; i += threads * 16)
    *reinterpret_cast<uint4 *>(rows + i) = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ v16f zero16() {
  v16f z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}
// A lane's part of the operands: K rows m = lane % 32 (chunk 2 i + lane / 32 of step i), and through the
// transposing read V's rows 4 (lane / 32) + lane % 16 / 4 of a block of 16 states, channels 16 (lane / 16 % 2) + 4 (lane % 4).
template <int DB>
struct Reader {
  typedef Rows<DB> L;
  int k_at[L::XOR ? 1 : 2 * DB], k_x, v_at, v_z;
  __device__ __forceinline__ explicit Reader(int lane) {
    const int m = lane & 31, h = lane >> 5, v_row = 4 * h + (lane >> 2 & 3);
    k_x = h ^ L::k_swap(m);
    if constexpr (L::XOR) {
      k_at[0] = m * L::ROW;
    } else {
#pragma unroll
      for (int i = 0; i < 2 * DB; ++i) k_at[i] = m * L::ROW + L::k_slot(m, 2 * i + h) * 16;
    }
    v_z = L::v_swap(v_row) >> 2;
    v_at = v_row * L::ROW + (2 * (lane >> 4 & 1) + (lane >> 1 & 1)) * 16 + (lane & 1) * 8;
  }
  __device__ __forceinline__ v4u k(const uint8_t *block, int i) const {
    return *reinterpret_cast<const v4u *>(block + (L::XOR ? k_at[0] + ((k_x ^ (2 * i)) << 4) : k_at[L::XOR ? 0 : i]));
  }
  __device__ __forceinline__ v4u v(const uint8_t *block, int d) const {
    typedef __attribute__((address_space(3))) v4i16 *Read;
    const uint8_t *at = block + v_at + ((d ^ v_z) << 6);
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Read)(uint8_t *)at);
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Read)(uint8_t *)(at + 8 * L::ROW));
    const uint2 x = __builtin_bit_cast(uint2, lo), y = __builtin_bit_cast(uint2, hi);
    return v4u{x.x, x.y, y.x, y.y};
  }
};

// A row's running state, and its results: pieces for the join, or the output.
template <int DB, bool F16>
struct Sums {
  v16f o[DB];
  float top = kLowest, rest = 0.0f;      // the weights' reference: rest is 0 below kFar
  float sum = 0.0f;                      // of this lane's half; the halves' are added at the end
  bool far = false;                      // some row of the wavefront has a rest
  __device__ __forceinline__ Sums() {
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] = zero16();
  }
  // makes room for scores whose largest is `best` times c
  __device__ __forceinline__ void raise(float best, float c) {
    const bool up = __builtin_fmaf(best, c, -top) - rest > kSlack;
    if (__any(up)) {
      const float to = up ? best * c : top, size = fabsf(to);
      const float left = !up ? rest : size >= kFar && size < __builtin_inff() ? __builtin_fmaf(best, c, -to) : 0.0f;
      const float r = __builtin_amdgcn_exp2f((top - to) + (rest - left));
      top = to;
      rest = left;
      far = __any(rest != 0.0f);
      sum *= r;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= r;
    }
  }
  // a piece for the join
  __device__ __forceinline__ void leave(const CrossArgs &a, const Piece &p, const Row &r, int h, bool some) {
    sum = half_sum(sum);
    if (r.row >= a.rows) return;
    const int64_t at = (int64_t)p.place * a.rows + r.row;
    if (h == 0) {
      a.ml[2 * at] = top;
      a.ml[2 * at + 1] = some ? sum : -1.0f;           // -1: a piece without states
      if (fabsf(top) >= kFar) a.rest[at] = rest;
    }
    if (!some) return;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int ch = 32 * d + 8 * j + 4 * h;
        if (ch < a.D)
          *reinterpret_cast<v4f *>(a.o + at * a.D + ch) = v4f{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
      }
  }
  // The output of a lane's row.  The halves exchange pieces of four channels for eight each.
  __device__ __forceinline__ void store(const CrossArgs &a, const Piece &p, const Row &r, int h) {
    sum = half_sum(sum);
    const float inv = p.n > 0 ? 1.0f / sum : 0.0f;
    uint16_t *dst = a.out + (((int64_t)p.b * a.Lq + r.qi) * a.Hq + r.hq) * a.D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        uint32_t w[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const auto x = __builtin_amdgcn_permlane32_swap(
              pack2<F16>(o[d][4 * j + 2 * e] * inv, o[d][4 * j + 2 * e + 1] * inv),
              pack2<F16>(o[d][4 * j + 4 + 2 * e] * inv, o[d][4 * j + 5 + 2 * e] * inv), false, false);
          w[0][e] = x[0];
          w[1][e] = x[1];
        }
        const int ch = 32 * d + 8 * j + 8 * h;
        if (r.row < a.rows && ch < a.D) *reinterpret_cast<uint4 *>(dst + ch) = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
      }
  }
  // The output of 32 rows from row0 on, through a wavefront's 2048 DB bytes of LDS, so that
  // rows leave 16 bytes a lane.
  __device__ __forceinline__ void finish(const CrossArgs &a, const Piece &p, int row0, int lane, uint8_t *mine) {
    sum = half_sum(sum);
    const float inv = p.n > 0 ? 1.0f / sum : 0.0f;
    const int m = lane & 31, h = lane >> 5;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint2 *>(mine + m * 64 * DB + ((4 * d + j) ^ (m & 3)) * 16 + 8 * h) =
            make_uint2(pack2<F16>(o[d][4 * j] * inv, o[d][4 * j + 1] * inv), pack2<F16>(o[d][4 * j + 2] * inv, o[d][4 * j + 3] * inv));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    constexpr int SLOTS = Rows<DB>::XOR ? Rows<DB>::SLOTS : 16;       // lanes to a row
    const int c = lane & (SLOTS - 1);
    if (8 * c >= a.D) return;
#pragma unroll
    for (int i = 0; i < 32 * SLOTS / 64; ++i) {
      const int m2 = 64 / SLOTS * i + lane / SLOTS, row = row0 + m2;
      if (row < a.rows) {
        int qi = row, hq = p.hk;
        if (a.group > 1) {
          qi = row / a.group;
          hq = p.hk * a.group + row - qi * a.group;
        }
        *reinterpret_cast<uint4 *>(a.out + (((int64_t)p.b * a.Lq + qi) * a.Hq + hq) * a.D + 8 * c) =
            *reinterpret_cast<const uint4 *>(mine + m2 * 64 * DB + (c ^ (m2 & 3)) * 16);
      }
    }
  }
};

// sets the scores of block rows from `left` on to -inf (h: the lane's half)
__device__ __forceinline__ void hide(v16f &s, int left, int h) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (8 * (i / 4) + 4 * h + i % 4 >= left) s[i] = -__builtin_inff();
}
__device__ __forceinline__ float largest(const v16f &s) {
  float best = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) best = fmaxf(best, s[i]);
  return best;
}

// The exponentials of a block's scores, and packed as the operand of the second product (pw[u]: half u
// of the block).  (Adding up with the two-element dot product, half the instructions, was slower.)
template <bool F16>
__device__ __forceinline__ void weigh(const v16f &s, float c, float off, float &sum, v4u (&pw)[2]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * e], c, off));
    const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * e + 1], c, off));
    sum += x;
    sum += y;
    pw[e / 4][e % 4] = pack2<F16>(x, y);
  }
}

// KB blocks of 32 states, of which `left` are there: scores, weights and sums.
template <int DB, int KB, bool F16>
__device__ __forceinline__ void attend(Sums<DB, F16> &acc, const v4u (&q)[2 * DB], const Reader<DB> &read, const uint8_t *k,
                                       const uint8_t *v, int left, int h, float c) {
  v16f s[KB];
#pragma unroll
  for (int b = 0; b < KB; ++b) s[b] = zero16();
#pragma unroll
  for (int i = 0; i < 2 * DB; ++i)
#pragma unroll
    for (int b = 0; b < KB; ++b) s[b] = mma<F16>(read.k(k + 32 * b * Rows<DB>::ROW, i), q[i], s[b]);
  if (left < 32 * KB) {
#pragma unroll
    for (int b = 0; b < KB; ++b) hide(s[b], left - 32 * b, h);
  }
  float best = largest(s[0]);
#pragma unroll
  for (int b = 1; b < KB; ++b) best = fmaxf(best, largest(s[b]));
  acc.raise(half_max(best), c);
  float off = kShift<F16> - acc.top;
  if (acc.far) {                         // such rows' scores less their maximum, whose rest would be lost in `off`
    const bool apart = acc.rest != 0.0f;
    const float inv = 1.0f / c;
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = apart ? (__builtin_fmaf(s[b][i], c, -acc.top) - acc.rest) * inv : s[b][i];
    off = apart ? kShift<F16> : off;
  }
#pragma unroll
  for (int b = 0; b < KB; ++b) {
    v4u pw[2];
    weigh<F16>(s[b], c, off, acc.sum, pw);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int d = 0; d < DB; ++d) acc.o[d] = mma<F16>(read.v(v + (32 * b + 16 * u) * Rows<DB>::ROW, d), pw[u], acc.o[d]);
  }
}

// Many rows: each of the four wavefronts has 32, and all read the same tiles of
// KEYS states, two in LDS.  A block of 32 x 32 scores of 128 channels is 16 matrix instructions, 512 cycles, 80
// vector instructions, 16 of them exponentials, and 24 LDS reads, 16 KB.  In registers, two wavefronts to a SIMD
// and none waiting for another's result, the matrix instructions take 222 ns, with 64 FMAs and 16 exponentials among
// them 228, and with 16 KB from LDS besides 318; but with 128 and 256 FMAs 305 and 458, so the vector ALU is not
// free.  The kernel takes 939 cycles a block, 505 ns at the clock it runs at: the matrix core is busy for 55% of
// them and LDS for 27%.  What the units leave unused goes to each block's own order (products, maximum,
// exponentials, products), which only two wavefronts of a SIMD cover.  Ordering it by hand, the next block's
// scores between this one's exponentials, was slower than the compiler's order (564 against 539 us at
// 4096 x 16384, 16 heads).  Workgroups that go on to
// the next row tile with its queries asked for ahead were no faster (32760 rows over 512 states, 12 heads: 146 us, this 142),
// as the registers they need cost more.  4096 x 16384, 16 heads of 128: 520 us, 1.06 PFLOP/s; of 256 channels
// 4096 x 4096 268 us, of 160 190.
template <int DB, int KEYS, bool F16, bool LIST>
__global__ __launch_bounds__(256, 2) void cross_many_kernel(const CrossArgs a) {
  typedef Rows<DB> L;
  constexpr int KB = KEYS / 32, STEPS = 2 * DB, HALF = KEYS * L::ROW;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * HALF];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ int list[LIST ? kCrossOwnList : 1];
  Piece p(a, KEYS);
  if (!p.any) return;
  p.template cut<LIST, 4>(a, KEYS, list);
  const int m = lane & 31, h = lane >> 5;
  const uint32_t lds_at = lds_offset(lds);
  clear_pads<DB>(a, lds, KEYS, threadIdx.x, 256);
  clear_pads<DB>(a, lds + 2 * HALF, KEYS, threadIdx.x, 256);
  Copier<DB, KEYS, 4, LIST> copy(a, p, lane, w);
  auto fetch = [&](int t, int buf) __attribute__((always_inline)) { copy.both(t, lds_at + 2 * buf * HALF, lds_at + (2 * buf + 1) * HALF); };
  const int row0 = p.tile_row * 128 + 32 * w;
  const Row r(a, p, row0 + m);
  v4u q[STEPS];
  if (p.t0 < p.t1) {
    copy.look_up(p.t0);
    fetch(p.t0, 0);
    copy.look_up(p.t0 + 1);
  }
  r.load(a, p, h, q);
  Row::flip(a, q);

  Sums<DB, F16> acc;
  const Reader<DB> read(lane);
  int buf = 0;
  for (int t = p.t0; t < p.t1; ++t, buf ^= 1) {
    vmcnt_wait0_known();
    __syncthreads();
    const bool last = (t + 1) * KEYS > p.n;
    uint8_t *st = lds + 2 * buf * HALF;
    if (last) {
      clear_rows<DB>(st + HALF, p.n - t * KEYS, KEYS, threadIdx.x, 256);
      __syncthreads();
    }
    if (t + 1 < p.t1) {
      fetch(t + 1, buf ^ 1);
      copy.look_up(t + 2);
    }
    attend<DB, KB, F16>(acc, q, read, st, st + HALF, last ? p.n - t * KEYS : 32 * KB, h, a.c);
  }
  if (a.ml) {
    acc.leave(a, p, r, h, p.t0 < p.t1);
  } else {
    __syncthreads();
    acc.finish(a, p, row0, lane, lds + w * 2048 * DB);
  }
}

// Many rows over few states: a workgroup keeps all of a key/value head's states in LDS (up to CAP), and its
// eight wavefronts go through rows by 32, each by itself, without barriers.  2 x 4096 rows over 300 states, 16 heads of
// 72: 28 us, of which 10 do not grow with the rows (launch, the states' way into LDS, last stores); the rest is
// the order of a block's steps as above.  The tiles of four wavefronts take 37.
template <int DB, int CAP, bool F16, bool LIST>
__global__ __launch_bounds__(512, 2) void cross_near_kernel(const CrossArgs a) {
  typedef Rows<DB> L;
  constexpr int KEYS = 64;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * CAP * L::ROW];
  __shared__ int list[LIST ? CAP : 1];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m = lane & 31, h = lane >> 5;
  Piece p(a, KEYS);
  if (!p.any) return;
  p.template cut<LIST, 8>(a, KEYS, list);
  uint8_t *kl = lds, *vl = lds + CAP * L::ROW;
  const uint32_t k_at = lds_offset(kl), v_at = lds_offset(vl);
  Copier<DB, KEYS, 8, LIST> copy(a, p, lane, w);
  for (int t = 0; t < p.t1; ++t) {
    if constexpr (LIST) {
#pragma unroll
      for (int j = 0; j < copy.COPIES; ++j) copy.key[j] = (uint32_t)list[min(t * KEYS + copy.row(j), p.n - 1)];
    }
    copy.both(t, k_at + t * KEYS * L::ROW, v_at + t * KEYS * L::ROW);
  }
  clear_pads<DB>(a, kl, p.t1 * KEYS, threadIdx.x, 512);
  // this workgroup's blocks of 32 rows
  const int blocks = (a.rows + 31) / 32;
  const int b0 = (int)((int64_t)blocks * p.tile_row / a.tiles), b1 = (int)((int64_t)blocks * (p.tile_row + 1) / a.tiles);
  Row r(a, p, 32 * (b0 + w) + m);
  v4u q[2 * DB];
  r.load(a, p, h, q);
  Row::flip(a, q);
  const Reader<DB> read(lane);
  vmcnt_wait0_known();
  __syncthreads();
  if (p.n < p.t1 * KEYS) {
    clear_rows<DB>(vl, p.n, p.t1 * KEYS, threadIdx.x, 512);
    __syncthreads();
  }
  for (int i = b0 + w; i < b1; i += 8) {
    // the next rows' queries, asked for before this block's states are gone through
    const Row next(a, p, 32 * (i + 8) + m);
    v4u ahead[2 * DB];
    next.load(a, p, h, ahead);
    Sums<DB, F16> acc;
    for (int t = 0; t < p.t1; ++t)
      attend<DB, 2, F16>(acc, q, read, kl + t * KEYS * L::ROW, vl + t * KEYS * L::ROW, p.n - t * KEYS, h, a.c);
    acc.store(a, p, r, h);
    r = next;
#pragma unroll
    for (int j = 0; j < 2 * DB; ++j) q[j] = ahead[j] ^ a.flip;
  }
}

// Few rows (up to 32 of a key/value head): the wavefronts (four or eight) take tiles of 32 states of
// their own, in LDS of their own, without barriers, two tiles in flight, and add up at the end.  Bound by memory
// (8 x 20 heads of 64 over 1500 states, 61 MB: 15.6 us, 3.9 TB/s with a workgroup on 160 of the CUs; 32 rows over
// 20000 states of 8 heads of 128, 82 MB: 26 us with its join; 8 x 20 heads of 72 over 1500, 69 MB: 24).
template <int DB, int W, bool F16, bool LIST>
__global__ __launch_bounds__(64 * W, DB > 2 ? 1 : 2) void cross_few_kernel(const CrossArgs a) {
  typedef Rows<DB> L;
  constexpr int KEYS = 32, STEPS = 2 * DB, HALF = KEYS * L::ROW, PITCH = 32 * DB + 4;     // floats of a row of sums
  constexpr int TILES = W * 4 * HALF, SUMS = W * 32 * (PITCH + 3) * 4, SHARE = 2 * W;     // threads to a row
  __shared__ __attribute__((aligned(1024))) uint8_t lds[TILES > SUMS ? TILES : SUMS];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ int list[LIST ? kCrossOwnList : 1];
  Piece p(a, KEYS);
  if (!p.any) return;
  p.template cut<LIST, W>(a, KEYS, list);
  const int m = lane & 31, h = lane >> 5;
  uint8_t *mine = lds + w * 4 * HALF;
  const uint32_t lds_at = lds_offset(mine);
  clear_pads<DB>(a, mine, KEYS, lane, 64);
  clear_pads<DB>(a, mine + 2 * HALF, KEYS, lane, 64);
  Copier<DB, KEYS, 1, LIST> copy(a, p, lane, 0);
  auto fetch = [&](int t, int buf) __attribute__((always_inline)) { copy.both(t, lds_at + 2 * buf * HALF, lds_at + (2 * buf + 1) * HALF); };
  const int t0 = p.t0 + w;
  const Row r(a, p, m);
  v4u q[STEPS];
  r.load(a, p, h, q);
  if (t0 < p.t1) {
    copy.look_up(t0);
    fetch(t0, 0);
  }
  if (t0 + W < p.t1) {
    copy.look_up(t0 + W);
    fetch(t0 + W, 1);
    copy.look_up(t0 + 2 * W);
  }
  Row::flip(a, q);

  Sums<DB, F16> acc;
  const Reader<DB> read(lane);
  int buf = 0;
  for (int t = t0; t < p.t1; t += W, buf ^= 1) {
    // this tile has landed when only the next one's copies are outstanding (a list's reads are among those)
    if (!LIST && t + W < p.t1) vmcnt_wait<2 * Copier<DB, KEYS, 1, LIST>::COPIES>();
    else vmcnt_wait0();
    const bool last = (t + 1) * KEYS > p.n;
    uint8_t *st = mine + 2 * buf * HALF;
    if (last) clear_rows<DB>(st + HALF, p.n - t * KEYS, KEYS, lane, 64);
    attend<DB, 1, F16>(acc, q, read, st, st + HALF, last ? p.n - t * KEYS : KEYS, h, a.c);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");       // the tile has been read
    if (t + 2 * W < p.t1) {
      fetch(t + 2 * W, buf);
      copy.look_up(t + 3 * W);
    }
  }
  // The wavefronts' sums, [wavefront][row][channel], with their maxima, these' rests and sums behind.
  acc.sum = half_sum(acc.sum);
  __syncthreads();
  float *so = reinterpret_cast<float *>(lds), *sm = so + W * 32 * PITCH, *sr = sm + W * 32, *sl = sr + W * 32;
  if (m < a.rows) {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<v4f *>(so + (32 * w + m) * PITCH + 32 * d + 8 * j + 4 * h) =
            v4f{acc.o[d][4 * j], acc.o[d][4 * j + 1], acc.o[d][4 * j + 2], acc.o[d][4 * j + 3]};
    sm[32 * w + m] = acc.top;
    sr[32 * w + m] = acc.rest;
    sl[32 * w + m] = t0 < p.t1 ? acc.sum : -1.0f;            // -1: no states
  }
  __syncthreads();
  const int row = threadIdx.x / SHARE, part = threadIdx.x % SHARE;
  if (row >= a.rows) return;
  float top = kLowest, rest = 0.0f, sum = 0.0f, f[W];
  bool some = false;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const bool in = sl[32 * i + row] != -1.0f;
    const float x = sm[32 * i + row], y = sr[32 * i + row];
    some = some || in;
    rest = !in || x < top ? rest : x > top ? y : fmaxf(rest, y);
    if (in) top = fmaxf(top, x);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const bool in = sl[32 * i + row] != -1.0f;
    f[i] = in ? __builtin_amdgcn_exp2f((sm[32 * i + row] - top) + (sr[32 * i + row] - rest)) : 0.0f;
    sum = in ? __builtin_fmaf(f[i], sl[32 * i + row], sum) : sum;
  }
  const Row at_row(a, p, row);
  const int64_t at = (int64_t)p.place * a.rows + row;
  uint16_t *dst = a.out + (((int64_t)p.b * a.Lq + at_row.qi) * a.Hq + at_row.hq) * a.D;
  const float inv = some ? 1.0f / sum : 0.0f;
  if (a.ml && part == 0) {
    a.ml[2 * at] = top;
    a.ml[2 * at + 1] = some ? sum : -1.0f;
    if (fabsf(top) >= kFar) a.rest[at] = rest;
  }
#pragma unroll
  for (int c = 4 * part; c < 32 * DB; c += 4 * SHARE) {
    if (c >= a.D) break;
    v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const v4f x = *reinterpret_cast<const v4f *>(so + (32 * i + row) * PITCH + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(f[i], x[e], y[e]);
    }
    if (a.ml) {
      *reinterpret_cast<v4f *>(a.o + at * a.D + c) = y;
    } else {
      *reinterpret_cast<uint2 *>(dst + c) = make_uint2(pack2<F16>(y[0] * inv, y[1] * inv), pack2<F16>(y[2] * inv, y[3] * inv));
    }
  }
}

// A wavefront joins a row's pieces: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// LANES lanes hold a row's channels, four each; 64 / LANES pieces are read at a time, and four of
// those in flight (about 40 pieces of 1024 rows of 128, 21 MB, to 6144 rows: 8 us, 2.6 TB/s).
template <int LANES, bool F16>
__global__ __launch_bounds__(256) void cross_join_kernel(const CrossArgs a, int keys) {
  const int lane = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= (int64_t)a.B * a.Hkv * a.rows) return;
  // the row, and where its first piece is; the others follow `all` rows apart
  const int bh = (int)(id / a.rows), row = (int)(id - (int64_t)bh * a.rows), b = bh / a.Hkv, hk = bh - b * a.Hkv;
  int pieces = a.parts;
  int64_t at = id, all = (int64_t)a.B * a.Hkv * a.rows;
  if (a.line) {
    const Shares s(a, keys);
    pieces = __shfl(s.parts, b);
    at = ((int64_t)__shfl(s.before, b) * a.Hkv + hk) * a.rows + row;
    all = (int64_t)a.Hkv * a.rows;
  }
  constexpr int GROUPS = 64 / LANES;
  const int g = lane / LANES, ch = 4 * (lane % LANES);
  const float2 *ml = reinterpret_cast<const float2 *>(a.ml);
  float top = kLowest, rest = 0.0f, sum = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  bool some = false;
  // 64 pieces at a time, their maxima and sums a lane each
  for (int p0 = 0; p0 < pieces; p0 += 64) {
    const float2 x = p0 + lane < pieces ? ml[(p0 + lane) * all + at] : make_float2(kLowest, -1.0f);
    const bool in = x.y != -1.0f;
    float to = in ? fmaxf(top, x.x) : top, r, f;
#pragma unroll
    for (int i = 32; i > 0; i >>= 1) to = fmaxf(to, __shfl_xor(to, i));
    if (__any(in && fabsf(x.x) >= kFar) || rest != 0.0f) {
      // maxima that are alike differ in their rests
      const float mine = in && fabsf(x.x) >= kFar ? a.rest[(p0 + lane) * all + at] : 0.0f;
      float left = fmaxf(in && x.x == to ? mine : -__builtin_inff(), top == to ? rest : -__builtin_inff());
#pragma unroll
      for (int i = 32; i > 0; i >>= 1) left = fmaxf(left, __shfl_xor(left, i));
      r = __builtin_amdgcn_exp2f((top - to) + (rest - left));
      f = in ? __builtin_amdgcn_exp2f((x.x - to) + (mine - left)) : 0.0f;
      rest = left;
    } else {
      r = __builtin_amdgcn_exp2f(top - to);
      f = in ? __builtin_amdgcn_exp2f(x.x - to) : 0.0f;
    }
    some = some || __any(in);
    top = to;
    float add = in ? f * x.y : 0.0f;
#pragma unroll
    for (int i = 32; i > 0; i >>= 1) add += __shfl_xor(add, i);
    sum = __builtin_fmaf(sum, r, add);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= r;
    const uint64_t have = __ballot(in);
    const int n = min(64, pieces - p0);
    for (int i = 0; i < n; i += 4 * GROUPS) {
      v4f y[4];
      float fy[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = i + u * GROUPS + g;              // up to 63 + 3 GROUPS: the factor of a lane past 63 is not used
        const bool ok = j < n && (have >> (j & 63) & 1) != 0 && ch < a.D;
        fy[u] = __shfl(f, j & 63);
        y[u] = ok ? *reinterpret_cast<const v4f *>(a.o + ((p0 + j) * all + at) * a.D + ch) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(fy[u], y[u][e], o[e]);
    }
  }
#pragma unroll
  for (int i = LANES; i < 64; i <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], i);
  if (g != 0 || ch >= a.D) return;
  const float inv = some ? 1.0f / sum : 0.0f;
  const int qi = row / a.group, hq = hk * a.group + row - qi * a.group;
  *reinterpret_cast<uint2 *>(a.out + (((int64_t)b * a.Lq + qi) * a.Hq + hq) * a.D + ch) =
      make_uint2(pack2<F16>(o[0] * inv, o[1] * inv), pack2<F16>(o[2] * inv, o[3] * inv));
}

// The lists of all batch rows, where they are too long for a workgroup to make its own.
__global__ __launch_bounds__(1024) void cross_list_kernel(const uint8_t *__restrict__ mask, const int *__restrict__ lens,
                                                          int Lk, int *__restrict__ index, int *__restrict__ count) {
  const int b = blockIdx.x, n = lens ? min(max(lens[b], 0), Lk) : Lk;
  const int all = list_visible<16>(mask + (int64_t)b * Lk, n, index + (int64_t)b * Lk);
  if (threadIdx.x == 0) count[b] = all;
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
  // lengths that differ: the parts are shared out on the device, by length
  a.line = key_lens && !mask ? p.line : 0;
  a.least = p.least;
  if (p.parts > 1 || a.line) {
    a.ml = reinterpret_cast<float *>(ws + p.ml_off);
    a.rest = reinterpret_cast<float *>(ws + p.rest_off);
    a.o = reinterpret_cast<float *>(ws + p.o_off);
  }
  a.lens = key_lens;
  const bool list = mask && Lk > 0;
  if (list && Lk <= kCrossOwnList) {
    a.mask = mask;
  } else if (list) {
    int *index = reinterpret_cast<int *>(ws), *count = reinterpret_cast<int *>(ws + p.count_off);
    hipLaunchKernelGGL(cross_list_kernel, dim3(B), dim3(1024), 0, stream, mask, key_lens, Lk, index, count);
    st = launch_status("cross attention list launch");
    if (st != SVDQ_OK) return st;
    a.index = index;
    a.count = count;
  }
  // Maxima are taken of the bare products, so the scale's sign goes to the queries.
  a.c = log2_scale(scale);
  a.flip = scale < 0.0f ? 0x80008000u : 0u;
  a.work = (int)(Hkv * p.tiles * (a.line ? a.line + B : B * (int64_t)p.parts));      // at most 2^28 / 128 + 2^20
  // Row tiles of a head that go to one XCD together: up to 32, as far as no XCD gets a sixteenth more
  // than its share; the workgroups of the form with the states in LDS, one to a CU, singly (252 of
  // them in runs of 11, 33 to some XCDs' 32 CUs: 115 us, singly 74).
  a.run = (int)(p.near ? 1 : p.tiles < 32 ? p.tiles : 32);
  while (a.run > 1 && 16 * ((a.work + 8 * a.run - 1) / (8 * a.run) * 8ll * a.run) > 17ll * a.work) a.run = (a.run + 1) / 2;
  const dim3 grid((unsigned)((a.work + 8 * a.run - 1) / (8 * a.run) * (8 * a.run)));
#define CROSS_MANY(DB, KEYS)                                                              \
  do {                                                                                    \
    if (dtype == SVDQ_FP16) {                                                             \
      if (list) hipLaunchKernelGGL((cross_many_kernel<DB, KEYS, true, true>), grid, dim3(256), 0, stream, a);   \
      else hipLaunchKernelGGL((cross_many_kernel<DB, KEYS, true, false>), grid, dim3(256), 0, stream, a);       \
    } else {                                                                              \
      if (list) hipLaunchKernelGGL((cross_many_kernel<DB, KEYS, false, true>), grid, dim3(256), 0, stream, a);  \
      else hipLaunchKernelGGL((cross_many_kernel<DB, KEYS, false, false>), grid, dim3(256), 0, stream, a);      \
    }                                                                                     \
  } while (0)
#define CROSS_NEAR(DB)                                                                    \
  do {                                                                                    \
    constexpr int CAP = cross_near_states(DB);                                            \
    if (dtype == SVDQ_FP16) {                                                             \
      if (list) hipLaunchKernelGGL((cross_near_kernel<DB, CAP, true, true>), grid, dim3(512), 0, stream, a);   \
      else hipLaunchKernelGGL((cross_near_kernel<DB, CAP, true, false>), grid, dim3(512), 0, stream, a);       \
    } else {                                                                              \
      if (list) hipLaunchKernelGGL((cross_near_kernel<DB, CAP, false, true>), grid, dim3(512), 0, stream, a);  \
      else hipLaunchKernelGGL((cross_near_kernel<DB, CAP, false, false>), grid, dim3(512), 0, stream, a);      \
    }                                                                                     \
  } while (0)
#define CROSS_FEW(DB, W)                                                                     \
  do {                                                                                    \
    if (dtype == SVDQ_FP16) {                                                             \
      if (list) hipLaunchKernelGGL((cross_few_kernel<DB, W, true, true>), grid, dim3(64 * W), 0, stream, a);   \
      else hipLaunchKernelGGL((cross_few_kernel<DB, W, true, false>), grid, dim3(64 * W), 0, stream, a);       \
    } else {                                                                              \
      if (list) hipLaunchKernelGGL((cross_few_kernel<DB, W, false, true>), grid, dim3(64 * W), 0, stream, a);  \
      else hipLaunchKernelGGL((cross_few_kernel<DB, W, false, false>), grid, dim3(64 * W), 0, stream, a);      \
    }                                                                                     \
  } while (0)
  switch (p.blocks) {
    case 2: if (p.wide) CROSS_FEW(2, 8); else if (p.own) CROSS_FEW(2, 4); else if (p.near) CROSS_NEAR(2); else CROSS_MANY(2, 64); break;
    case 3: if (p.own) CROSS_FEW(3, 4); else if (p.near) CROSS_NEAR(3); else CROSS_MANY(3, 64); break;
    case 4: if (p.own) CROSS_FEW(4, 4); else if (p.near) CROSS_NEAR(4); else CROSS_MANY(4, 64); break;
    case 5: CROSS_MANY(5, 32); break;
    default: CROSS_MANY(8, 32); break;
  }
#undef CROSS_FEW
#undef CROSS_NEAR
#undef CROSS_MANY
  st = launch_status("cross attention launch");
  if (st != SVDQ_OK || !a.ml) return st;
  const dim3 joins((unsigned)(((int64_t)B * Hkv * p.rows + 3) / 4));
#define CROSS_JOIN(LANES)                                                                                            \
  do {                                                                                                               \
    if (dtype == SVDQ_FP16) hipLaunchKernelGGL((cross_join_kernel<LANES, true>), joins, dim3(256), 0, stream, a, p.tile_keys); \
    else hipLaunchKernelGGL((cross_join_kernel<LANES, false>), joins, dim3(256), 0, stream, a, p.tile_keys);            \
  } while (0)
  if (D <= 64) CROSS_JOIN(16);
  else if (D <= 128) CROSS_JOIN(32);
  else CROSS_JOIN(64);
#undef CROSS_JOIN
  return launch_status("cross attention join launch");
}

}  // extern "C"
