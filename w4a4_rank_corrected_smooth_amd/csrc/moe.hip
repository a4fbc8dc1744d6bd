// The expert layer of a mixture of experts for a few tokens, with AWQ W4A16
// experts, and the router that picks them.
//
//  moe_logits_kernel   x w^T in float64
//  moe_choose_kernel   scores, the best top_k of each token, their weights
//  moe_gate_up_kernel  h = act(x Gate^T) * (x Up^T) of every (token, expert)
//  moe_down_kernel     h Down^T of every (token, expert)
//  moe_sum_kernel      the weighted sum over a token's experts
#include <hip/hip_runtime.h>

#include "common.h"
#include "device_util.h"
#include "layout.h"
#include "moe_layout.h"

using namespace svdq;

namespace {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, v2bf{(__bf16)a, (__bf16)b});
}
template <bool F16>
__device__ __forceinline__ float wide(uint32_t h) {
  if constexpr (F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  else return __uint_as_float(h << 16);
}

// ---------------------------------------------------------------------- router
// Logits in float64: a product of two 16-bit values is exact in float32, and
// their sum in float64 is exact to 2^-53 of its terms, so the order of the
// sum cannot move a logit across its neighbour's and the choice does not
// depend on how the work is split.  One wavefront per expert and kTokens tokens.
constexpr int kTokens = 4;

template <bool F16>
__global__ __launch_bounds__(256) void moe_logits_kernel(const uint16_t *__restrict__ x, const uint16_t *__restrict__ wr,
                                                         int T, int E, int K, double *__restrict__ logits) {
  const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t0 = blockIdx.y * kTokens;
  if (e >= E) return;
  double acc[kTokens] = {};
  for (int k = lane * 8; k < K; k += 512) {
    const uint4 wv = *reinterpret_cast<const uint4 *>(wr + (int64_t)e * K + k);
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      const uint4 xv = *reinterpret_cast<const uint4 *>(x + (int64_t)min(t0 + t, T - 1) * K + k);
      const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[t] += (double)(wide<F16>(ww[i] & 0xFFFFu) * wide<F16>(xw[i] & 0xFFFFu));
        acc[t] += (double)(wide<F16>(ww[i] >> 16) * wide<F16>(xw[i] >> 16));
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[t] += __shfl_xor(acc[t], o);
    if (lane == 0 && t0 + t < T) logits[(int64_t)(t0 + t) * E + e] = acc[t];
  }
}

// One wavefront per token.  The order is by key, the lower index first where
// keys are equal; the key is the score plus the expert's bias, or the logit
// itself where there is no bias (the score grows with it).  A NaN key is
// taken as the smallest.  P: keys of a lane, E <= 64 P.

template <int P>
__global__ __launch_bounds__(64) void moe_choose_kernel(const double *__restrict__ logits, const float *__restrict__ bias,
                                                        int E, int top_k, int sigmoid, int normalize,
                                                        int *__restrict__ ids, float *__restrict__ weights) {
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  __shared__ double score[MOE_MAX_EXPERTS];
  double key[P];
  double top = -__builtin_inf();
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (64 * i < E) {
      const int e = 64 * i + lane;
      key[i] = e < E ? logits[t * E + e] : -__builtin_inf();
      top = fmax(top, key[i]);
    }
  for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o));
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (64 * i < E) {
      const int e = 64 * i + lane;
      if (e < E) {
        const double s = sigmoid ? 1.0 / (1.0 + exp(-key[i])) : exp(key[i] - top);
        score[e] = s;
        sum += s;
      }
    }
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  __syncthreads();
  if (bias)
  #pragma unroll
  for (int i = 0; i < P; ++i)
      if (64 * i + lane < E) key[i] = (sigmoid ? score[64 * i + lane] : score[64 * i + lane] / sum) + (double)bias[64 * i + lane];
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (64 * i < E && key[i] != key[i]) key[i] = -__builtin_inf();
  // lane j keeps the j-th choice
  int mine = 0;
  uint32_t taken = 0;
  for (int j = 0; j < top_k; ++j) {
    double best = -__builtin_inf();
    int at = MOE_MAX_EXPERTS;
  #pragma unroll
  for (int i = 0; i < P; ++i)
      if (64 * i + lane < E && !(taken >> i & 1u) && (at == MOE_MAX_EXPERTS || key[i] > best)) {
        best = key[i];
        at = 64 * i + lane;
      }
    for (int o = 32; o > 0; o >>= 1) {
      const double b = __shfl_xor(best, o);
      const int a = __shfl_xor(at, o);
      if (a != MOE_MAX_EXPERTS && (at == MOE_MAX_EXPERTS || b > best || (b == best && a < at))) {
        best = b;
        at = a;
      }
    }
    if ((at & 63) == lane) taken |= 1u << (at >> 6);
    if (lane == j) mine = at;
  }
  const double s = lane < top_k ? score[mine] : 0.0;
  double chosen = s;
  for (int o = 32; o > 0; o >>= 1) chosen += __shfl_xor(chosen, o);
  const double div = normalize ? chosen : sigmoid ? 1.0 : sum;
  if (lane < top_k) {
    ids[t * top_k + lane] = mine;
    weights[t * top_k + lane] = (float)(s / div);
  }
}

// --------------------------------------------------------------------- experts
struct MoeArgs {
  const uint8_t *gate_up, *down;      // E blobs each, one after another
  int64_t gate_up_stride, down_stride;
  int E, K, I;
  const uint16_t *x;
  int T, top_k;
  const int *ids;
  const float *weights;
  uint16_t *h_hi, *h_lo;              // [T top_k][I] bf16, h = hi + lo
  float *part;                        // [T top_k][K]
  MoePlan *plan;                      // above 64 pairs
  uint16_t *y;
};

// The rows of one expert, for a wavefront: its (token, choice) pairs.  Their
// order does not matter: a row of a matrix product does not depend on where
// it stands.  Up to 64 pairs every wavefront finds them for itself, in
// registers; above, moe_plan_kernel has sorted them.
template <bool PLAN>
struct Rows {
  int expert = -1, count = 0;
  int list = 0;                 // !PLAN: lane r holds the pair of row r
  const uint16_t *sorted = nullptr;

  // the `slot`-th expert that the ids name; false where there are fewer
  __device__ __forceinline__ bool find(const MoeArgs &a, int slot, int lane) {
    if constexpr (PLAN) {
      if (slot >= a.plan->slots) return false;
      expert = a.plan->expert[slot];
      const int first = a.plan->first[slot];
      count = a.plan->first[slot + 1] - first;
      sorted = a.plan->pairs + first;
    } else {
      const int n = a.T * a.top_k;
      const int id = lane < n ? a.ids[lane] : -1;
      uint64_t left = __ballot(id >= 0 && id < a.E), same = 0;
      do {
        if (left == 0) return false;
        expert = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        same = __ballot(id == expert);
        left &= ~same;
      } while (slot-- > 0);
      count = __builtin_popcountll(same);
      // lane i of the set goes to the lane of its rank; the others to the end
      const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
      const bool in = same >> lane & 1;
      list = __builtin_amdgcn_ds_permute(4 * (in ? rank : 63 - (lane - rank)), lane);
    }
    return true;
  }
  __device__ __forceinline__ int pair(int r) const {      // r in [0, count), any in each lane
    if constexpr (PLAN) return sorted[r];
    else return __shfl(list, r);
  }
};

// Pairs sorted by expert.  One workgroup.
__global__ __launch_bounds__(1024) void moe_plan_kernel(MoeArgs a) {
  __shared__ int count[MOE_MAX_EXPERTS], first[MOE_MAX_EXPERTS], wsum[2][16];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n = a.T * a.top_k;
  count[tid] = 0;
  __syncthreads();
  int id[kMoeMaxPairs / 1024], rank[kMoeMaxPairs / 1024];
#pragma unroll
  for (int i = 0; i < kMoeMaxPairs / 1024; ++i) {
    const int p = 1024 * i + tid;
    id[i] = p < n ? a.ids[p] : -1;
    if (id[i] >= a.E) id[i] = -1;
    if (id[i] >= 0) rank[i] = atomicAdd(&count[id[i]], 1);
  }
  __syncthreads();
  // places of the experts that have pairs, and of their pairs
  const int c = count[tid];
  int pairs = c, slots = c > 0 ? 1 : 0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int p = __shfl_up(pairs, o), q = __shfl_up(slots, o);
    if (lane >= o) {
      pairs += p;
      slots += q;
    }
  }
  if (lane == 63) {
    wsum[0][w] = pairs;
    wsum[1][w] = slots;
  }
  __syncthreads();
  int all = 0, used = 0;
  for (int i = 0; i < 16; ++i) {
    if (i < w) {
      pairs += wsum[0][i];
      slots += wsum[1][i];
    }
    all += wsum[0][i];
    used += wsum[1][i];
  }
  first[tid] = pairs - c;
  if (c > 0) {
    a.plan->expert[slots - 1] = tid;
    a.plan->first[slots - 1] = pairs - c;
  }
  if (tid == 0) {
    a.plan->slots = used;
    a.plan->first[used] = all;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMoeMaxPairs / 1024; ++i)
    if (id[i] >= 0) a.plan->pairs[first[id[i]] + rank[i]] = (uint16_t)(1024 * i + tid);
}

// Eight codes of a blob word (even channels in the low half-words) as the
// bf16 values 128 + code: 0x4300 is 128 and a code fills the last mantissa
// bits, so one shift and one and-or make a pair.  (An instruction takes one
// constant from scalar registers, so the other is put into a vector register;
// the and-or itself is left to the compiler, which then knows what the matrix
// instructions have to wait for.)
__device__ __forceinline__ uint32_t in_vector(uint32_t c) {
  uint32_t v;
  asm("v_mov_b32 %0, %1" : "=v"(v) : "s"(c));
  return v;
}
__device__ __forceinline__ v8bf codes_128(uint32_t word) {
  uint32_t o[4];
  const uint32_t magic = in_vector(0x43004300u);
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = (word >> (4 * j) & 0x000F000Fu) | magic;
  return as_v8bf(make_uint4(o[0], o[1], o[2], o[3]));
}
// Eight codes as the fp16 values code - zero, exactly: 1024 + code minus 1024 + zero.
__device__ __forceinline__ v8h codes_minus_zero(uint32_t word, _Float16 zero) {
  const _Float16 off = -((_Float16)1024.0f + zero);
  const uint32_t magic = in_vector(0x64006400u);
  v8h o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t pr = (word >> (4 * j) & 0x000F000Fu) | magic;
    const v2h v = __builtin_bit_cast(v2h, pr) + v2h{off, off};
    o[2 * j] = v.x;
    o[2 * j + 1] = v.y;
  }
  return o;
}
__device__ __forceinline__ float scale_of(uint32_t sz) { return (float)__builtin_bit_cast(_Float16, (uint16_t)sz); }
__device__ __forceinline__ _Float16 zero_of(uint32_t sz) { return __builtin_bit_cast(_Float16, (uint16_t)(sz >> 16)); }

__device__ __forceinline__ v4f mma(uint4 a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_v8bf(a), b, c, 0, 0, 0);
}

template <int N>
struct Int { static constexpr int value = N; };

// acc += the group's 64 channels: s (sum x (128 + code) - (128 + zero) sum x)
// for bf16 activations (sum x from one more product, with ones, shared by the
// columns), s sum x (code - zero) for fp16.  a0, a1: the lane's row, channels
// 16 (lane / 16) + [0, 16) of the group.
template <bool F16>
__device__ __forceinline__ void group_mma(uint4 a0, uint4 a1, v4f xsum, uint32_t w0, uint32_t w1, uint32_t sz, v4f &acc) {
  const float s = scale_of(sz);
  if constexpr (F16) {
    const _Float16 z = zero_of(sz);
    v4f p = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a0), codes_minus_zero(w0, z), v4f{}, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a1), codes_minus_zero(w1, z), p, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(p[e], s, acc[e]);
  } else {
    v4f p = mma(a0, codes_128(w0), v4f{});
    p = mma(a1, codes_128(w1), p);
    const float z = -(128.0f + (float)zero_of(sz));
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(__builtin_fmaf(z, xsum[e], p[e]), s, acc[e]);
  }
}
__device__ __forceinline__ v8bf ones() { return as_v8bf(make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u)); }

// Work of a wavefront: TP tiles of 16 output columns of one expert (gate_up:
// TP gate tiles and the TP up tiles that belong to them) over one of KS equal
// parts of the input channels; the four wavefronts of a workgroup are KS parts
// of 4 / KS neighbouring sets of tiles.  Rows go 16 R at a time.  A step is a
// pair of groups of 64 channels, one 16-byte code load for each tile; the next
// step's loads are issued before a step's products, and the last step is
// loaded once more at the end, so that every load is unconditional.
template <int TILES, int R, int H>
struct Step {
  uint4 code[TILES];
  uint2 sz[TILES];
  uint4 x[R][H][4];                     // H pieces of the rows' 2 x 16 channels
};

struct Tiles {
  const uint8_t *code;                  // the lane's 16 bytes of step 0 of tile 0
  const uint32_t *sz;                   // the lane's column's scale words of tile 0
};
__device__ __forceinline__ Tiles tiles_of(const uint8_t *blob, const AwqLayout &L, int tile, int lane) {
  return Tiles{blob + L.q + (int64_t)tile * awq_pairs(L.G) * kAwqBlockBytes + lane * 16,
               reinterpret_cast<const uint32_t *>(blob + L.sz) +
                   (int64_t)(tile * kAwqTile + (lane & 15)) * awq_g4(L.G)};
}

// this wavefront's steps
__device__ __forceinline__ void wave_steps(int G, int part, int parts, int &p0, int &p1) {
  const int P = (G + 1) / 2, each = (P + parts - 1) / parts;
  p0 = min(P, part * each);
  p1 = min(P, p0 + each);
}

// Gate and up products of R x 16 rows; acc[0]: gate, acc[1]: up.
template <bool F16, int TP, int R>
__device__ __forceinline__ void gate_up_rows(const MoeArgs &a, const Tiles (&tl)[2][TP], const uint16_t *const (&xr)[R],
                                             int G, int p0, int p1, v4f (&acc)[2][R][TP]) {
  typedef Step<2 * TP, R, 1> S;
  auto load = [&](int p, S &s) {
#pragma unroll
    for (int i = 0; i < 2 * TP; ++i) {
      const Tiles &t = tl[i / TP][i % TP];
      s.code[i] = *reinterpret_cast<const uint4 *>(t.code + (int64_t)p * kAwqBlockBytes);
      s.sz[i] = *reinterpret_cast<const uint2 *>(t.sz + 2 * p);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < 4; ++k)     // an odd last group reads the one before it, and is not used
        s.x[r][0][k] = *reinterpret_cast<const uint4 *>(xr[r] + min(2 * p + k / 2, G - 1) * kGroup + 8 * (k % 2));
  };
  auto work = [&](int p, const S &s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (2 * p + i >= G) break;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4 a0 = s.x[r][0][2 * i], a1 = s.x[r][0][2 * i + 1];
        v4f xsum = v4f{};
        if constexpr (!F16) xsum = mma(a1, ones(), mma(a0, ones(), v4f{}));
#pragma unroll
        for (int t = 0; t < 2 * TP; ++t)
          group_mma<F16>(a0, a1, xsum, i ? s.code[t].z : s.code[t].x, i ? s.code[t].w : s.code[t].y,
                         i ? s.sz[t].y : s.sz[t].x, acc[t / TP][r][t % TP]);
      }
    }
  };
  if (p0 >= p1) return;
  S x, y;
  load(p0, x);
  for (int p = p0;; p += 2) {
    load(min(p + 1, p1 - 1), y);
    work(p, x);
    if (p + 1 >= p1) break;
    load(min(p + 2, p1 - 1), x);
    work(p + 1, y);
    if (p + 2 >= p1) break;
  }
}

template <bool F16, bool GELU, int TP, int KS, bool PLAN>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3))) void moe_gate_up_kernel(MoeArgs a) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Rows<PLAN> rows;
  if (!rows.find(a, blockIdx.y, lane)) return;
  const int G = a.K / kGroup, n = a.I / kAwqTile;
  const AwqLayout L(2 * (int64_t)a.I, a.K);
  const uint8_t *blob = a.gate_up + rows.expert * a.gate_up_stride;
  const int tile0 = (blockIdx.x * (4 / KS) + w / KS) * TP;
  Tiles tl[2][TP];
#pragma unroll
  for (int t = 0; t < TP; ++t) {        // tiles past the last are worked on as the last, and not stored
    tl[0][t] = tiles_of(blob, L, min(tile0 + t, n - 1), lane);
    tl[1][t] = tiles_of(blob, L, min(tile0 + t, n - 1) + n, lane);
  }
  int p0, p1;
  wave_steps(G, w % KS, KS, p0, p1);
  __shared__ v4f red[KS > 1 ? 4 : 1][KS > 1 ? 4 * TP : 1][64];

  auto pass = [&](int r0, auto rt) {
    constexpr int R = decltype(rt)::value;
    const uint16_t *xr[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      xr[r] = a.x + (int64_t)(rows.pair(min(r0 + 16 * r + (lane & 15), rows.count - 1)) / a.top_k) * a.K + 16 * (lane >> 4);
    v4f acc[2][R][TP] = {};
    gate_up_rows<F16, TP, R>(a, tl, xr, G, p0, p1, acc);
    if constexpr (KS > 1) {             // the parts meet, in order, in the first one's wavefront
      if (w % KS != 0) {
#pragma unroll
        for (int i = 0; i < 2 * R * TP; ++i) red[w][i][lane] = acc[i / (R * TP)][i / TP % R][i % TP];
      }
      __syncthreads();
      if (w % KS == 0) {
#pragma unroll
        for (int i = 0; i < 2 * R * TP; ++i)
#pragma unroll
          for (int k = 1; k < KS; ++k) {
            const v4f y = red[w + k][i][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i / (R * TP)][i / TP % R][i % TP][e] += y[e];
          }
      }
      __syncthreads();
      if (w % KS != 0) return;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = r0 + 16 * r + 4 * (lane >> 4) + e;
        const int64_t at = (int64_t)rows.pair(min(row, rows.count - 1)) * a.I + (lane & 15);
#pragma unroll
        for (int t = 0; t < TP; ++t) {
          const float g = acc[0][r][t][e], u = acc[1][r][t][e];
          const float h = (GELU ? gelu_tanh_f32(g) : g * __builtin_amdgcn_rcpf(1.0f + __expf(-g))) * u;
          if (row < rows.count && tile0 + t < n) {
            const __bf16 hi = (__bf16)h;
            a.h_hi[at + (tile0 + t) * kAwqTile] = __builtin_bit_cast(uint16_t, hi);
            a.h_lo[at + (tile0 + t) * kAwqTile] =
                __builtin_bit_cast(uint16_t, (__bf16)(__builtin_isfinite(h) ? h - (float)hi : 0.0f));
          }
        }
      }
  };
  for (int r0 = 0; r0 < rows.count;) {
    if (rows.count - r0 > 16) {
      pass(r0, Int<2>{});
      r0 += 32;
    } else {
      pass(r0, Int<1>{});
      r0 += 16;
    }
  }
}

// h enters the down product as its two bf16 pieces (h to 2^-17, in float32's
// range).
template <int TP, int KS, bool PLAN>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3))) void moe_down_kernel(MoeArgs a) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Rows<PLAN> rows;
  if (!rows.find(a, blockIdx.y, lane)) return;
  const int G = a.I / kGroup, n = a.K / kAwqTile;
  const AwqLayout L(a.K, a.I);
  const uint8_t *blob = a.down + rows.expert * a.down_stride;
  const int tile0 = (blockIdx.x * (4 / KS) + w / KS) * TP;
  Tiles tl[TP];
#pragma unroll
  for (int t = 0; t < TP; ++t) tl[t] = tiles_of(blob, L, min(tile0 + t, n - 1), lane);
  int p0, p1;
  wave_steps(G, w % KS, KS, p0, p1);
  __shared__ v4f red[KS > 1 ? 4 : 1][KS > 1 ? TP : 1][64];

  for (int r0 = 0; r0 < rows.count; r0 += 16) {
    const int64_t at = (int64_t)rows.pair(min(r0 + (lane & 15), rows.count - 1)) * a.I + 16 * (lane >> 4);
    const uint16_t *hr[2] = {a.h_hi + at, a.h_lo + at};
    v4f acc[TP] = {};
    typedef Step<TP, 1, 2> S;
    auto load = [&](int p, S &s) {
#pragma unroll
      for (int t = 0; t < TP; ++t) {
        s.code[t] = *reinterpret_cast<const uint4 *>(tl[t].code + (int64_t)p * kAwqBlockBytes);
        s.sz[t] = *reinterpret_cast<const uint2 *>(tl[t].sz + 2 * p);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          s.x[0][h][k] = *reinterpret_cast<const uint4 *>(hr[h] + min(2 * p + k / 2, G - 1) * kGroup + 8 * (k % 2));
    };
    auto work = [&](int p, const S &s) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (2 * p + i >= G) break;
        const uint4 h0 = s.x[0][0][2 * i], h1 = s.x[0][0][2 * i + 1], l0 = s.x[0][1][2 * i], l1 = s.x[0][1][2 * i + 1];
        const v4f sum = mma(l1, ones(), mma(l0, ones(), mma(h1, ones(), mma(h0, ones(), v4f{}))));
#pragma unroll
        for (int t = 0; t < TP; ++t) {
          const v8bf b0 = codes_128(i ? s.code[t].z : s.code[t].x), b1 = codes_128(i ? s.code[t].w : s.code[t].y);
          const v4f prod = mma(l1, b1, mma(l0, b0, mma(h1, b1, mma(h0, b0, v4f{}))));
          const uint32_t sz = i ? s.sz[t].y : s.sz[t].x;
          const float z = -(128.0f + (float)zero_of(sz)), sc = scale_of(sz);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][e] = __builtin_fmaf(__builtin_fmaf(z, sum[e], prod[e]), sc, acc[t][e]);
        }
      }
    };
    if (p0 < p1) {
      S x, y;
      load(p0, x);
      for (int p = p0;; p += 2) {
        load(min(p + 1, p1 - 1), y);
        work(p, x);
        if (p + 1 >= p1) break;
        load(min(p + 2, p1 - 1), x);
        work(p + 1, y);
        if (p + 2 >= p1) break;
      }
    }
    if constexpr (KS > 1) {
      if (w % KS != 0) {
#pragma unroll
        for (int t = 0; t < TP; ++t) red[w][t][lane] = acc[t];
      }
      __syncthreads();
      if (w % KS == 0) {
#pragma unroll
        for (int t = 0; t < TP; ++t)
#pragma unroll
          for (int k = 1; k < KS; ++k) {
            const v4f y = red[w + k][t][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t][e] += y[e];
          }
      }
      __syncthreads();
      if (w % KS != 0) continue;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = r0 + 4 * (lane >> 4) + e;
      const int64_t to = (int64_t)rows.pair(min(row, rows.count - 1)) * a.K + (lane & 15);
#pragma unroll
      for (int t = 0; t < TP; ++t)
        if (row < rows.count && tile0 + t < n) a.part[to + (tile0 + t) * kAwqTile] = acc[t][e];
    }
  }
}

// y[t] = sum over the token's choices of weight times part, in order; choices
// without an expert here are left out.  One thread per 4 columns.
template <bool F16>
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeArgs a) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int quads = a.K / 4;
  const int64_t t = idx / quads;
  const int c = (int)(idx % quads) * 4;
  if (t >= a.T) return;
  v4f y = v4f{};
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t p = t * a.top_k + j;
    const int e = a.ids[p];
    if (e < 0 || e >= a.E) continue;
    const float w = a.weights[p];
    const v4f v = *reinterpret_cast<const v4f *>(a.part + p * a.K + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(w, v[i], y[i]);
  }
  uint2 out;
  if constexpr (F16) {
    out.x = __builtin_bit_cast(uint32_t, v2h{(_Float16)y[0], (_Float16)y[1]});
    out.y = __builtin_bit_cast(uint32_t, v2h{(_Float16)y[2], (_Float16)y[3]});
  } else {
    out.x = pack_bf16(y[0], y[1]);
    out.y = pack_bf16(y[2], y[3]);
  }
  *reinterpret_cast<uint2 *>(a.y + t * a.K + c) = out;
}

}  // namespace

#ifndef GTP0
#define GTP0 1
#define GKS0 4
#define GTP1 1
#define GKS1 1
#define DTP0 1
#define DKS0 2
#define DTP1 4
#define DKS1 1
#define FEWG 2048
#define FEWD 4096
#endif

extern "C" {

svdq_status_t svdq_moe_route(const void *x, const void *w_router, const float *bias, svdq_dtype_t dtype, int T, int E,
                             int K, int top_k, svdq_moe_score_t score, int normalize, int32_t *ids, float *weights,
                             void *workspace, size_t ws_bytes, void *hip_stream) {
  if (dtype != SVDQ_BF16 && dtype != SVDQ_FP16)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_moe_route: dtype must be SVDQ_BF16 or SVDQ_FP16");
  if (score != SVDQ_MOE_SOFTMAX && score != SVDQ_MOE_SIGMOID)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_moe_route: unknown score %d", (int)score);
  if (!moe_route_ok(T, E, K, top_k))
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "svdq_moe_route: T=%d E=%d K=%d top_k=%d", T, E, K, top_k);
  if (T == 0) return SVDQ_OK;
  if (!x || !w_router || !ids || !weights || !workspace)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_moe_route: NULL pointer");
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(workspace) ||
      (((uintptr_t)ids | (uintptr_t)weights | (uintptr_t)bias) & 3u))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "svdq_moe_route: misaligned pointer");
  const size_t need = svdq_moe_route_workspace_bytes(T, E);
  if (ws_bytes < need)
    return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "svdq_moe_route: workspace needs %zu bytes, got %zu", need, ws_bytes);
  const svdq_status_t st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  double *logits = static_cast<double *>(workspace);
  const uint16_t *xp = static_cast<const uint16_t *>(x), *wp = static_cast<const uint16_t *>(w_router);
  const dim3 grid((unsigned)((E + 3) / 4), (unsigned)((T + kTokens - 1) / kTokens));
  if (dtype == SVDQ_FP16)
    hipLaunchKernelGGL((moe_logits_kernel<true>), grid, dim3(256), 0, stream, xp, wp, T, E, K, logits);
  else
    hipLaunchKernelGGL((moe_logits_kernel<false>), grid, dim3(256), 0, stream, xp, wp, T, E, K, logits);
  const int sigmoid = score == SVDQ_MOE_SIGMOID ? 1 : 0;
#define MOE_CHOOSE(P) hipLaunchKernelGGL((moe_choose_kernel<P>), dim3((unsigned)T), dim3(64), 0, stream, logits, bias, E, \
                                         top_k, sigmoid, normalize, ids, weights)
  if (E <= 64) MOE_CHOOSE(1);
  else if (E <= 128) MOE_CHOOSE(2);
  else if (E <= 256) MOE_CHOOSE(4);
  else if (E <= 512) MOE_CHOOSE(8);
  else MOE_CHOOSE(16);
#undef MOE_CHOOSE
  return launch_status("router launch");
}

svdq_status_t awq_moe_forward(const awq_moe_weights_t *w, const void *x, svdq_dtype_t dtype, int T, const int32_t *ids,
                              const float *weights, int top_k, svdq_moe_act_t act, void *y, void *workspace,
                              size_t ws_bytes, void *hip_stream) {
  if (!w || !w->gate_up || !w->down) return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_forward: NULL weights");
  if (!aligned16(w->gate_up) || !aligned16(w->down))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_forward: misaligned weights");
  if (dtype != SVDQ_BF16 && dtype != SVDQ_FP16)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_forward: dtype must be SVDQ_BF16 or SVDQ_FP16");
  if (act != SVDQ_MOE_SILU && act != SVDQ_MOE_GELU_TANH)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_forward: unknown activation %d", (int)act);
  if (!moe_weights_ok(w->E, w->K, w->I) || !moe_call_ok(T, top_k))
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "awq_moe_forward: E=%d K=%d I=%d T=%d top_k=%d", w->E, w->K, w->I, T, top_k);
  if (T == 0) return SVDQ_OK;
  if (!x || !ids || !weights || !y || !workspace)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_forward: NULL pointer");
  if (!aligned16(x) || !aligned16(y) || !aligned16(workspace) || (((uintptr_t)ids | (uintptr_t)weights) & 3u))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_forward: misaligned pointer");
  const MoeWork L(T, top_k, w->K, w->I);
  if ((int64_t)ws_bytes < L.total)
    return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "awq_moe_forward: workspace needs %lld bytes, got %zu",
                (long long)L.total, ws_bytes);
  const svdq_status_t st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  MoeArgs a{};
  a.gate_up = static_cast<const uint8_t *>(w->gate_up);
  a.down = static_cast<const uint8_t *>(w->down);
  a.gate_up_stride = AwqLayout(2 * (int64_t)w->I, w->K).total;
  a.down_stride = AwqLayout(w->K, w->I).total;
  a.E = w->E;
  a.K = w->K;
  a.I = w->I;
  a.x = static_cast<const uint16_t *>(x);
  a.T = T;
  a.top_k = top_k;
  a.ids = ids;
  a.weights = weights;
  a.h_hi = reinterpret_cast<uint16_t *>(ws + L.h_hi);
  a.h_lo = reinterpret_cast<uint16_t *>(ws + L.h_lo);
  a.part = reinterpret_cast<float *>(ws + L.part);
  a.y = static_cast<uint16_t *>(y);
  a.plan = reinterpret_cast<MoePlan *>(ws + L.plan);
  const int pairs = T * top_k, slots = pairs < w->E ? pairs : w->E;
  const bool plan = pairs > 64;
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (plan) hipLaunchKernelGGL(moe_plan_kernel, dim3(1), dim3(1024), 0, stream, a);
  const int gt = w->I / kAwqTile, dt = w->K / kAwqTile;
#define MOE_GU3(F, A, TP, KS, P)                                                                        \
  hipLaunchKernelGGL((moe_gate_up_kernel<F, A, TP, KS, P>),                                             \
                     dim3((gt + TP * (4 / KS) - 1) / (TP * (4 / KS)), (unsigned)slots), dim3(256), 0, stream, a)
#define MOE_GU2(F, A, P) do { if (few) MOE_GU3(F, A, GTP0, GKS0, P); else MOE_GU3(F, A, GTP1, GKS1, P); } while (0)
#define MOE_GU(F, A) do { if (plan) MOE_GU2(F, A, true); else MOE_GU2(F, A, false); } while (0)
#define MOE_D3(TP, KS, P)                                                                               \
  hipLaunchKernelGGL((moe_down_kernel<TP, KS, P>), dim3((dt + TP * (4 / KS) - 1) / (TP * (4 / KS)), (unsigned)slots), \
                     dim3(256), 0, stream, a)
#define MOE_D2(P) do { if (few_down) MOE_D3(DTP0, DKS0, P); else MOE_D3(DTP1, DKS1, P); } while (0)
  const bool few = (int64_t)slots * gt < FEWG, few_down = (int64_t)slots * dt < FEWD;
  if (dtype == SVDQ_FP16) {
    if (act == SVDQ_MOE_GELU_TANH) MOE_GU(true, true); else MOE_GU(true, false);
  } else {
    if (act == SVDQ_MOE_GELU_TANH) MOE_GU(false, true); else MOE_GU(false, false);
  }
  if (plan) MOE_D2(true); else MOE_D2(false);
#undef MOE_D2
#undef MOE_D3
#undef MOE_GU
#undef MOE_GU2
#undef MOE_GU3
  const dim3 g3((unsigned)(((int64_t)T * (w->K / 4) + 255) / 256));
  if (dtype == SVDQ_FP16) hipLaunchKernelGGL((moe_sum_kernel<true>), g3, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((moe_sum_kernel<false>), g3, dim3(256), 0, stream, a);
  return launch_status("expert layer launch");
}

}  // extern "C"
