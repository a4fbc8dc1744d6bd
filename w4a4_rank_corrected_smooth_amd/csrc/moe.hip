// The expert layer of a mixture of experts for a few tokens, with AWQ W4A16
// experts, and the router that picks them.
//
//  moe_pack_kernel     weights to the experts' blobs, on the device
//  moe_logits_kernel   x w^T in float64
//  moe_choose_kernel   scores, the best top_k of each token, their weights
//  moe_route_kernel    both, where the matrix is small
//  moe_plan_kernel     the pairs of many, sorted by expert
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

// ------------------------------------------------------------------------ pack
// One wavefront per block of 1152 bytes.  Four canonical bytes (channel 2 j in
// the low nibble of byte j, 2 j + 1 in the high one) become a blob word (channel
// 2 j at nibble j of the low half-word, 2 j + 1 of the high one).
__device__ __forceinline__ uint32_t blob_word(uint32_t u) {
  uint32_t a = u & 0x0F0F0F0Fu, b = u >> 4 & 0x0F0F0F0Fu;
  a = (a | a >> 4) & 0x00FF00FFu;
  b = (b | b >> 4) & 0x00FF00FFu;
  return ((a | a >> 8) & 0xFFFFu) | (b | b >> 8) << 16;
}
__global__ __launch_bounds__(256) void moe_pack_kernel(const uint8_t *__restrict__ q, const uint16_t *__restrict__ s,
                                                       const uint16_t *__restrict__ z, int64_t blocks, int K, int G,
                                                       int P, uint8_t *__restrict__ blob) {
  const int lane = threadIdx.x & 63;
  const int64_t block = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);     // (expert, tile, step)
  if (block >= blocks) return;
  const int64_t tile = block / P, n = tile * kAwqTile + lane % 16;
  const int p = (int)(block % P);
  uint8_t *out = blob + block * kMoeBlockBytes;
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (2 * p + i < G) {
      const uint2 u = *reinterpret_cast<const uint2 *>(q + n * (K / 2) + (2 * p + i) * (kGroup / 2) + 8 * (lane / 16));
      w[2 * i] = blob_word(u.x);
      w[2 * i + 1] = blob_word(u.y);
    }
  *reinterpret_cast<uint4 *>(out + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  if (lane < 32) {
    const int64_t at = (tile * kAwqTile + lane / 2) * G + 2 * p + lane % 2;
    const bool in = 2 * p + lane % 2 < G;
    reinterpret_cast<uint32_t *>(out + kAwqBlockBytes)[lane] = in ? (uint32_t)s[at] | (uint32_t)z[at] << 16 : 0u;
  }
}

// ---------------------------------------------------------------------- router
// Logits in float64: a product of two 16-bit values is exact there (of bf16
// ones not in float32, whose range it can leave), and their sum is good to 2^-53
// of its terms, so the order of the sum cannot move a logit across its
// neighbour's and the choice does not depend on how the work is split.  One
// wavefront per expert and kTokens tokens.
constexpr int kTokens = 4;
// Logits of a call above which the matrix form takes over: at K = 4096 the two
// took 15.5 and 20.4 us for 64 x 256 logits (router in all), 23.5 and 21.5 for
// 128 x 256, 37.4 and 22.1 for 250 x 256.
constexpr int kTileLogits = 24576;

template <bool F16>
__global__ __launch_bounds__(256) void moe_logits_kernel(const uint16_t *__restrict__ x, const uint16_t *__restrict__ wr,
                                                         int T, int E, int K, double *__restrict__ logits) {
  const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t0 = blockIdx.y * kTokens;
  if (e >= E) return;
  double acc[kTokens] = {};
  // two turns of 512 channels at a time, all their loads in flight
  for (int k0 = lane * 8; k0 < K + lane * 8; k0 += 1024) {
    uint4 wv[2], xv[2][kTokens];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = min(k0 + 512 * i, K - 8);
      wv[i] = *reinterpret_cast<const uint4 *>(wr + (int64_t)e * K + k);
#pragma unroll
      for (int t = 0; t < kTokens; ++t)
        xv[i][t] = *reinterpret_cast<const uint4 *>(x + (int64_t)min(t0 + t, T - 1) * K + k);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (k0 + 512 * i >= K) break;
      const uint32_t ww[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
#pragma unroll
      for (int t = 0; t < kTokens; ++t) {
        const uint32_t xw[4] = {xv[i][t].x, xv[i][t].y, xv[i][t].z, xv[i][t].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[t] = __builtin_fma((double)wide<F16>(ww[j] & 0xFFFFu), (double)wide<F16>(xw[j] & 0xFFFFu), acc[t]);
          acc[t] = __builtin_fma((double)wide<F16>(ww[j] >> 16), (double)wide<F16>(xw[j] >> 16), acc[t]);
        }
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

// The same for more tokens: 16 x 16 logits a workgroup on the float64 matrix
// instruction, its eight wavefronts an eighth of K each (in turns of 32
// channels), met in LDS in order.  A lane holds row (token, expert) l % 16 and
// channels 8 (l / 16) + [0, 8) of a turn, one for each of eight products; the
// channels' order does not matter as long as both operands agree.  Both
// operands are used by 16 rows of the other, where the form above converts
// every product.
typedef double v4d __attribute__((ext_vector_type(4)));

template <bool F16>
__global__ __launch_bounds__(512) void moe_logits_tile_kernel(const uint16_t *__restrict__ x,
                                                              const uint16_t *__restrict__ wr, int T, int E, int K,
                                                              double *__restrict__ logits) {
  __shared__ v4d red[8][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = 8 * (lane >> 4);
  const int t0 = blockIdx.y * 16, e0 = blockIdx.x * 16;
  const uint16_t *xr = x + (int64_t)min(t0 + (lane & 15), T - 1) * K;
  const uint16_t *er = wr + (int64_t)min(e0 + (lane & 15), E - 1) * K;
  v4d acc = v4d{};
  const int turns = (K + 31) / 32;
  auto load = [&](int i, uint4 &a, uint4 &b) {
    const int k = min(32 * i + c, K - 8);
    a = *reinterpret_cast<const uint4 *>(xr + k);
    b = *reinterpret_cast<const uint4 *>(er + k);
  };
  constexpr int AHEAD = 4;
  uint4 a[AHEAD], b[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load(min(w + 8 * i, turns - 1), a[i], b[i]);
  for (int i0 = w; i0 < turns; i0 += 8 * AHEAD) {
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      const int i = i0 + 8 * n;
      if (i >= turns) break;
      if (32 * i + 32 > K && 32 * i + c >= K) a[n] = b[n] = make_uint4(0, 0, 0, 0);     // the last turn may end inside
      const uint32_t aw[4] = {a[n].x, a[n].y, a[n].z, a[n].w}, bw[4] = {b[n].x, b[n].y, b[n].z, b[n].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double a0 = (double)wide<F16>(aw[j] & 0xFFFFu), a1 = (double)wide<F16>(aw[j] >> 16);
        const double b0 = (double)wide<F16>(bw[j] & 0xFFFFu), b1 = (double)wide<F16>(bw[j] >> 16);
        acc = __builtin_amdgcn_mfma_f64_16x16x4f64(a0, b0, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f64_16x16x4f64(a1, b1, acc, 0, 0, 0);
      }
      load(min(i + 8 * AHEAD, turns - 1), a[n], b[n]);
    }
  }
  red[w][lane] = acc;
  __syncthreads();
  // wavefronts 0..3 take one element of each lane: token 4 e + lane / 16, expert lane % 16
  if (w >= 4) return;
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += red[k][lane][w];
  const int t = t0 + 4 * w + (lane >> 4), e = e0 + (lane & 15);
  if (t < T && e < E) logits[(int64_t)t * E + e] = s;
}

// Reductions over the wavefront within the vector unit: lanes of a row of 16,
// then the rows' last lanes into the next; the result stands in lane 63.
template <typename Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t x, uint32_t none, Op op) {
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, 0x111, 0xF, 0xF, false));   // row_shr:1
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, 0x112, 0xF, 0xF, false));
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, 0x114, 0xF, 0xF, false));
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, 0x118, 0xF, 0xF, false));
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, 0x142, 0xA, 0xF, false));   // row_bcast:15
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, 0x143, 0xC, 0xF, false));   // row_bcast:31
  return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  return wave_reduce(x, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint32_t wave_min(uint32_t x) {
  return wave_reduce(x, ~0u, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_f64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double x) {
  x = add_dpp<0x111, 0xF>(x);
  x = add_dpp<0x112, 0xF>(x);
  x = add_dpp<0x114, 0xF>(x);
  x = add_dpp<0x118, 0xF>(x);
  x = add_dpp<0x142, 0xA>(x);
  x = add_dpp<0x143, 0xC>(x);
  return lane_f64(x, 63);
}
// sum of x over lanes 0..lane
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
  return x;
}
// A number's place in the order of numbers, as an unsigned integer; NaN is the
// smallest, and the two zeros are equal.
__device__ __forceinline__ uint64_t order_of(double x) {
  if (x != x) return 0;
  const int64_t u = __builtin_bit_cast(int64_t, x + 0.0);
  return (uint64_t)(u < 0 ? ~u : u | (int64_t)1 << 63);
}

// One wavefront per token.  The order is by key, the lower index first where
// keys are equal; the key is the score plus the expert's bias, or the logit
// itself where there is no bias (the score grows with it).  A NaN key is
// taken as the smallest.  A choice is the largest upper half of a key, and
// only where several lanes have it, the largest lower half, then the lowest
// index.  P: keys of a lane, E <= 64 P.
template <int P>
__device__ __forceinline__ void choose(const double *logits, const float *__restrict__ bias, int E, int top_k, int sigmoid,
                                       int normalize, int64_t t, int lane, int *__restrict__ ids,
                                       float *__restrict__ weights) {
  double logit[P], score[P], top = -__builtin_inf();
  uint64_t key[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = 64 * i + lane;
    logit[i] = e < E ? logits[e] : -__builtin_inf();
    top = fmax(top, logit[i]);
  }
  if (!sigmoid) {
    const uint64_t u = order_of(top);
    const uint32_t hi = wave_max((uint32_t)(u >> 32));
    const uint32_t lo = wave_max((uint32_t)(u >> 32) == hi ? (uint32_t)u : 0u);
    // back from the order: the largest logit
    const uint64_t m = (uint64_t)hi << 32 | lo;
    top = __builtin_bit_cast(double, m >> 63 ? m & ~(1ull << 63) : ~m);
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const bool real = 64 * i + lane < E;
    score[i] = !real ? 0.0 : sigmoid ? 1.0 / (1.0 + exp(-logit[i])) : exp(logit[i] - top);
    sum += score[i];
  }
  const bool whole = !sigmoid && (bias || !normalize);      // the softmax's own denominator is needed
  sum = whole ? wave_sum(sum) : 1.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = 64 * i + lane;
    key[i] = e < E ? order_of(bias ? score[i] / sum + (double)bias[e] : logit[i]) : 0;
  }
  // lane j keeps the j-th choice
  int mine = 0;
  double mine_score = 0.0;
  uint32_t taken = 0;
  for (int j = 0; j < top_k; ++j) {
    uint64_t best = 0;
    uint32_t at = ~0u;                                      // an expert of this lane, if any is left
    double sc = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint32_t e = 64 * i + lane;
      if ((int)e < E && !(taken >> i & 1u) && (at == ~0u || key[i] > best)) {
        best = key[i];
        at = e;
        sc = score[i];
      }
    }
    const uint32_t hi = wave_max((uint32_t)(best >> 32));
    uint64_t in = __ballot(at != ~0u && (uint32_t)(best >> 32) == hi);
    if (in & (in - 1)) {
      const uint32_t lo = wave_max(in >> lane & 1 ? (uint32_t)best : 0u);
      in &= __ballot((uint32_t)best == lo);
      if (in & (in - 1)) {
        const uint32_t e = wave_min(in >> lane & 1 ? at : ~0u);
        in = __ballot(at == e);
      }
    }
    const int who = __builtin_ctzll(in);
    const int e = __builtin_amdgcn_readlane((int)at, who);
    const double s = lane_f64(sc, who);
    if (lane == who) taken |= 1u << (e >> 6);
    if (lane == j) {
      mine = e;
      mine_score = s;
    }
  }
  const double div = normalize ? wave_sum(mine_score) : sum;
  if (lane < top_k) {
    ids[t * top_k + lane] = mine;
    weights[t * top_k + lane] = (float)(mine_score / div);
  }
}
template <int P>
__global__ __launch_bounds__(64) void moe_choose_kernel(const double *__restrict__ logits, const float *__restrict__ bias,
                                                        int E, int top_k, int sigmoid, int normalize,
                                                        int *__restrict__ ids, float *__restrict__ weights) {
  const int64_t t = blockIdx.x;
  choose<P>(logits + t * E, bias, E, top_k, sigmoid, normalize, t, threadIdx.x, ids, weights);
}

// Both in one kernel, a workgroup per token, where each can read the router's
// whole matrix: its sixteen wavefronts take four experts each at a time, 1024
// channels a turn, and the first one chooses.  A launch less is 2.2 us less of a call
// from the host (14.0 against 11.8), and a turn is 2 us in a graph, where the two
// kernels need not wait for the host: up to two turns it costs at most what it saves.
// In one kernel and in two, 1 and 250 tokens: 64 experts of 512 (one turn) 4.7 and 5.6, 5.3
// and 7.7 us; 64 of 1536 (two) 6.6 and 6.3, 7.6 and 9.6; 64 of 2048 7.4 and 6.5, 8.8 and
// 10.5; 128 of 1024 8.5 and 6.3, 9.7 and 9.6; but 64 of 2560 (three) 8.5 and 7.2, 9.7 and
// 12.0; 192 of 1024 12.2 and 7.4, 13.6 and 10.5; 32 of 4096 (four) 11.2 and 8.1, 12.6 and
// 12.2.  With 600 tokens, more than there are CUs, 64 of 2048 take 15.6 and 12.1.
constexpr int kSmallTurns = 2;
constexpr int64_t route_turns(int E, int K) { return (int64_t)((E + 63) / 64) * ((K + 1023) / 1024); }
template <bool F16, int P>
__global__ __launch_bounds__(1024) void moe_route_kernel(const uint16_t *__restrict__ x, const uint16_t *__restrict__ wr,
                                                         const float *__restrict__ bias, int E, int K, int top_k,
                                                         int sigmoid, int normalize, int *__restrict__ ids,
                                                         float *__restrict__ weights) {
  __shared__ double logits[64 * P];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  const uint16_t *xr = x + t * K;
  for (int e0 = w; e0 < E; e0 += 64) {
    double acc[4] = {};
    for (int k0 = lane * 8; k0 < K + lane * 8; k0 += 1024) {
      uint4 wv[2][4], xv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = min(k0 + 512 * i, K - 8);
        xv[i] = *reinterpret_cast<const uint4 *>(xr + k);
#pragma unroll
        for (int n = 0; n < 4; ++n)
          wv[i][n] = *reinterpret_cast<const uint4 *>(wr + (int64_t)min(e0 + 16 * n, E - 1) * K + k);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (k0 + 512 * i >= K) break;
        const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t ww[4] = {wv[i][n].x, wv[i][n].y, wv[i][n].z, wv[i][n].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[n] = __builtin_fma((double)wide<F16>(ww[j] & 0xFFFFu), (double)wide<F16>(xw[j] & 0xFFFFu), acc[n]);
            acc[n] = __builtin_fma((double)wide<F16>(ww[j] >> 16), (double)wide<F16>(xw[j] >> 16), acc[n]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const double sum = wave_sum(acc[n]);
      if (lane == 0 && e0 + 16 * n < E) logits[e0 + 16 * n] = sum;
    }
  }
  __syncthreads();
  if (w == 0) choose<P>(logits, bias, E, top_k, sigmoid, normalize, t, lane, ids, weights);
}

// --------------------------------------------------------------------- experts
// With s and z the scale and zero point of an output channel and group of 64
// input channels, q the codes: an expert's product is sum_g s sum_k x (q - z).
// bf16 rows take the codes as the bf16 values c (128 + q) (one and-or a pair,
// exact) and c sum_k x from one more product, with c in the place of the code:
//   c sum_k x (q - z) = sum_k x c (128 + q) - (128 + z) sum_k x c,
// in float32 (the terms are about 30 times the result's, so 2^-19 of it, and less
// of a row with a common offset).  c = 2^-14: 64 terms of up to 143 c |x| each
// stay in float32's range for any x, and 1 / c is taken off at the end, exactly.
// fp16 rows take q - z exactly (1024 + q minus 1024 + z).  The gated product
// h = act(gate) up goes on as two bf16 pieces, which hold it to 2^-17 in
// float32's range (an fp16 h would overflow where y does not).
// What bounds it: the experts' bytes, each read once.  128 tokens with 8 of 128
// experts of 2048 x 768 (341 MB) take 84 us: gate and up 47 (227 MB, 4.8 TB/s; the
// weights' stream alone 41, the products alone 28), down 33 (113 MB; 24 and 20),
// the sum 4.
struct MoeArgs {
  const uint8_t *gate_up, *down;      // E blobs each, one after another
  int64_t gate_up_stride, down_stride;
  int E, K, I;
  const uint16_t *x;
  int T, top_k;
  const int *ids;
  const float *weights;
  uint16_t *h;                        // [T top_k][I / 64][2][64] bf16: h = first piece + second
  float *part;                        // [T top_k][K]
  MoePlan *plan;                      // above kLocalPairs pairs
  uint16_t *y;
};

// The rows of one expert are its (token, choice) pairs.  Their order does not
// matter: a row of a matrix product does not depend on where it stands.

// Up to 64 pairs, for a wavefront by itself, in registers.
struct WaveRows {
  int expert = -1, count = 0;
  int list = 0;                 // lane r holds the pair of row r

  // the `slot`-th expert that the ids name; false where there are fewer
  __device__ __forceinline__ bool find(const MoeArgs &a, int slot, int lane) {
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
    return true;
  }
  __device__ __forceinline__ int pair(int r) const { return __shfl(list, r); }     // r in [0, count)
};

// Up to kLocalPairs pairs, for a workgroup by itself, in LDS: which experts the
// ids name is a set of bits, of which the `slot`-th is this one's.  (A kernel
// that sorts them once costs 3.5 us more: 56.0 against 52.5 for 72 pairs, 85.9
// against 84.0 for 1024.)  Up to 64, each wavefront finds them as above and
// writes the list itself, the same as the others do: no barrier, 1 us less.
constexpr int kLocalPairs = 1024;
template <int WAVES>
struct LocalRows {
  static constexpr int LDS_BYTES = 2 * kLocalPairs + MOE_MAX_EXPERTS / 8 + 16;
  int expert = -1, count = 0;
  const uint16_t *sorted = nullptr;

  __device__ __forceinline__ bool find(const MoeArgs &a, int slot, uint8_t *lds, int lane) {
    uint16_t *list = reinterpret_cast<uint16_t *>(lds);
    uint32_t *named = reinterpret_cast<uint32_t *>(lds + 2 * kLocalPairs);
    int *used = reinterpret_cast<int *>(named + MOE_MAX_EXPERTS / 32);
    constexpr int EACH = kLocalPairs / (WAVES * 64), WORDS = MOE_MAX_EXPERTS / 32;
    const int tid = threadIdx.x, n = a.T * a.top_k;
    sorted = list;
    if (n <= 64) {
      WaveRows own;
      if (!own.find(a, slot, lane)) return false;
      expert = own.expert;
      count = own.count;
      if (lane < count) list[lane] = (uint16_t)own.list;
      return true;
    }
    int id[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int p = WAVES * 64 * i + tid;
      id[i] = p < n ? a.ids[p] : -1;
    }
    if (tid <= WORDS) (tid < WORDS ? (int *)named + tid : used)[0] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EACH; ++i)
      if (id[i] >= 0 && id[i] < a.E) atomicOr(&named[id[i] / 32], 1u << (id[i] % 32));
    __syncthreads();
    uint32_t word = lane < WORDS ? named[lane] : 0u;
    const int own = __builtin_popcount(word);
    const int upto = wave_scan(own);
    const uint64_t past = __ballot(upto > slot);
    if (past == 0) return false;
    const int at = __builtin_ctzll(past);
    uint32_t bits = __builtin_amdgcn_readlane((int)word, at);
    for (int i = slot - (__builtin_amdgcn_readlane(upto, at) - __builtin_popcount(bits)); i > 0; --i) bits &= bits - 1;
    expert = 32 * at + __builtin_ctz(bits);
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const uint64_t in = __ballot(id[i] == expert);
      if (in) {
        int first = 0;
        if (lane == 0) first = atomicAdd(used, __builtin_popcountll(in));
        first = __builtin_amdgcn_readfirstlane(first);
        if (in >> lane & 1) list[first + __builtin_popcountll(in & ((1ull << lane) - 1))] = (uint16_t)(WAVES * 64 * i + tid);
      }
    }
    __syncthreads();
    count = __builtin_amdgcn_readfirstlane(*used);
    return true;
  }
  __device__ __forceinline__ int one(int r) const { return __builtin_amdgcn_readfirstlane(sorted[r]); }   // the same r in all lanes
  __device__ __forceinline__ int pair(int r) const { return sorted[r]; }
};

// More: moe_plan_kernel has sorted them, in 4 us, where every thread of the form
// above would look at up to 16 ids.
struct PlanRows {
  static constexpr int LDS_BYTES = 16;
  int expert = -1, count = 0;
  const uint16_t *sorted = nullptr;

  __device__ __forceinline__ bool find(const MoeArgs &a, int slot, uint8_t *, int) {
    if (slot >= a.plan->slots) return false;
    expert = __builtin_amdgcn_readfirstlane(a.plan->expert[slot]);
    const int first = __builtin_amdgcn_readfirstlane(a.plan->first[slot]);
    count = __builtin_amdgcn_readfirstlane(a.plan->first[slot + 1]) - first;
    sorted = a.plan->pairs + first;
    return true;
  }
  __device__ __forceinline__ int one(int r) const { return __builtin_amdgcn_readfirstlane(sorted[r]); }
  __device__ __forceinline__ int pair(int r) const { return sorted[r]; }
};
template <bool PLAN, int WAVES> struct RowsOf { typedef LocalRows<WAVES> type; };
template <int WAVES> struct RowsOf<true, WAVES> { typedef PlanRows type; };

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
// bf16 values 2^-14 (128 + code): 0x3C00 is 2^-14 128 and a code fills the last
// mantissa bits, so one shift and one and-or make a pair.  (An instruction takes one
// constant from scalar registers, so the other is put into a vector register;
// the and-or itself is left to the compiler, which then knows what the matrix
// instructions have to wait for.)
__device__ __forceinline__ uint32_t in_vector(uint32_t c) {
  uint32_t v;
  asm("v_mov_b32 %0, %1" : "=v"(v) : "s"(c));
  return v;
}
constexpr float kCodeUnit = 0x1p-14f;
__device__ __forceinline__ v8bf codes_128(uint32_t word) {
  uint32_t o[4];
  const uint32_t magic = in_vector(0x3C003C00u);
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

// acc += the group's 64 channels: s c (sum x (128 + code) - (128 + zero) sum x)
// for bf16 activations (c sum x from one more product, shared by the columns; c is
// kCodeUnit), s sum x (code - zero) for fp16.  a0, a1: the lane's row, channels
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
__device__ __forceinline__ v8bf units() { return as_v8bf(make_uint4(0x38803880u, 0x38803880u, 0x38803880u, 0x38803880u)); }   // kCodeUnit
// 1 / c of the sums of group_mma
template <bool F16>
__device__ __forceinline__ float whole(float sum) { return F16 ? sum : sum * (1.0f / kCodeUnit); }
// The two bf16 pieces of a gated product.  The largest numbers, for which the
// first piece would round to infinity, get the largest one that does not.
__device__ __forceinline__ void split_h(float h, uint16_t &first, uint16_t &second) {
  __bf16 hi = (__bf16)h;
  if (__builtin_isfinite(h) && !__builtin_isfinite((float)hi)) hi = __builtin_bit_cast(__bf16, (uint16_t)(h > 0.0f ? 0x7F7F : 0xFF7F));
  first = __builtin_bit_cast(uint16_t, hi);
  second = __builtin_bit_cast(uint16_t, (__bf16)(__builtin_isfinite(h) ? h - (float)hi : 0.0f));
}

// One expert's product for a block of rows, the form both products share.
//
// Work of a wavefront: TILES tiles of 16 output columns over one of KS equal
// parts of the input channels; a workgroup's WAVES wavefronts are KS parts
// of WAVES / KS neighbouring sets of tiles.  A step is a pair of groups of
// 64 channels.
// Weights: each wavefront streams its tiles from memory into a ring of RING
// steps of registers; a step's place is filled anew as soon as it is used up.
// Rows: through LDS, CHUNK steps of every part at a time, shared by the
// wavefronts; a chunk is fetched to registers while the one before is worked
// on and then written to the other buffer.  (Loads are waited for in the
// order in which they are issued, so rows loaded straight into operands would
// hold up the weights asked for after them.)
// Rows come in one 16-bit piece (x) or in two (h): FORM 1: one piece, 16 R rows;
// 2: two pieces, 16 R rows, a product of each; 3: two pieces, 8 R rows, the second
// pieces in the tile's upper eight rows, so that one product takes both (and
// the two halves of the sums are added at the end).
// A row's chunk is WAVES x 16 pieces of 16 bytes, 16 for each (part, step,
// piece); 16-byte piece p of tile row r is at place p ^ (r % 16) of its 16, so
// that the operand reads, one row a lane, fall on different banks.
// Every load is unconditional: past the end a wavefront reads its last step
// again, and rows past the last repeat it.
template <int TILES, int FORM, int KS, int R, int WAVES>
struct Product {
  static constexpr int PIECES = FORM == 2 ? 2 : 1;       // products of a tile row
  static constexpr int ROWS = (FORM == 3 ? 8 : 16) * R;  // rows of a block
  static constexpr int CHUNK = WAVES / (KS * PIECES), RING = TILES <= 2 ? 4 : 2;
  static constexpr int UNROLL = CHUNK > RING ? CHUNK : RING;
  static_assert(CHUNK >= 1 && UNROLL % CHUNK == 0 && UNROLL % RING == 0, "whole chunks and rings");
  static constexpr int ROW_BYTES = WAVES * 256, BUFFER = 16 * R * ROW_BYTES, LDS_BYTES = 2 * BUFFER;
  static constexpr int WPR = WAVES / 4;              // wavefronts that fetch a row

  // (addresses are kept as a base that the wavefront shares, in scalar
  // registers, and a lane's own 32-bit offset)
  const uint8_t *w[TILES];            // the tiles' step 0
  const uint16_t *src;                // rows of ld elements; with two pieces, 64 of one and 64 of the other in turn
  int64_t ld;
  int G, P, each, p0, p1;             // groups, steps, steps of a part, this wavefront's steps

  uint4 code[RING][TILES];
  uint2 sz[RING][TILES];
  uint4 stage[4 * R];

  __device__ __forceinline__ void init(const uint8_t *blob, const MoeWeightLayout &L, const int (&tile)[TILES],
                                       int wave) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) w[t] = blob + L.block(tile[t], 0);
    G = (int)L.G;
    P = (int)L.P;
    each = (P + KS - 1) / KS;
    p0 = min(P, wave % KS * each);
    p1 = min(P, p0 + each);
  }
  // tile row of the j-th 16-byte piece that the wavefront fetches, and its row of the block
  static __device__ __forceinline__ int tile_row(int wave, int j) { return wave / WPR + 4 * j; }
  static __device__ __forceinline__ int block_row(int wave, int j) {
    const int r = tile_row(wave, j);
    return FORM == 3 ? r / 16 * 8 + r % 8 : r;
  }
  __device__ __forceinline__ void load_step(int i, int p, int lane) {
    p = max(min(min(p, p1 - 1), P - 1), 0);
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const uint8_t *block = w[t] + (int64_t)p * kMoeBlockBytes;
      const v4u c = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(block + (uint32_t)lane * 16));
      code[i][t] = make_uint4(c.x, c.y, c.z, c.w);
      sz[i][t] = *reinterpret_cast<const uint2 *>(block + (kAwqBlockBytes + (uint32_t)(lane & 15) * 8));
    }
  }
  // chunk c of the rows into registers; row[j]: the place in src of block row block_row(wave, j)
  __device__ __forceinline__ void fetch(int c, const int (&row)[4 * R], int wave, int lane) {
    const int s = wave % WPR * 4 + lane / 16, step = s / PIECES % CHUNK, part = s / PIECES / CHUNK;
    const int p = min(min(part * each + c * CHUNK + step, part * each + each - 1), P - 1);
    const int group = min(2 * p + lane % 16 / 8, G - 1);      // an odd last step has one group
#pragma unroll
    for (int j = 0; j < 4 * R; ++j) {
      const int piece = FORM == 2 ? s % 2 : FORM == 3 ? j / 2 % 2 : 0;
      const uint32_t at = (uint32_t)((group * (FORM == 1 ? 1 : 2) + piece) * kGroup + lane % 8 * 8) * 2;
      stage[j] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(src + row[j] * ld) + at);
    }
  }
  __device__ __forceinline__ void put(uint8_t *lds, int wave, int lane) const {
#pragma unroll
    for (int j = 0; j < 4 * R; ++j) {
      const int r = tile_row(wave, j);
      *reinterpret_cast<uint4 *>(lds + r * ROW_BYTES + (wave % WPR * 4 + lane / 16) * 256 + ((lane ^ r) % 16) * 16) = stage[j];
    }
  }
  __device__ __forceinline__ uint4 operand(const uint8_t *lds, int r, int s, int k, int lane) const {
    const int row = 16 * r + lane % 16, piece = 8 * (k / 2) + 2 * (lane / 16) + k % 2;
    return *reinterpret_cast<const uint4 *>(lds + row * ROW_BYTES + s * 256 + ((piece ^ row) % 16) * 16);
  }
  // all steps; `group(g, ring place, operands of each piece, r)` adds a group
  template <typename Group>
  __device__ __forceinline__ void run(uint8_t *lds, const int (&row)[4 * R], int wave, int lane, Group group) {
    const int chunks = (each + CHUNK - 1) / CHUNK;
    fetch(0, row, wave, lane);
#pragma unroll
    for (int i = 0; i < RING; ++i) load_step(i, p0 + i, lane);
    put(lds, wave, lane);
    __syncthreads();
    uint8_t *cur = lds, *other = lds + BUFFER;
    for (int c = 0; c < chunks; c += UNROLL / CHUNK) {
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) {
        if (i % CHUNK == 0) {
          if (i > 0 && c + i / CHUNK >= chunks) break;
          fetch(c + i / CHUNK + 1, row, wave, lane);
        }
        const int p = p0 + c * CHUNK + i;
        if (p < p1) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (2 * p + g >= G) break;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              uint4 a[PIECES][2];
#pragma unroll
              for (int h = 0; h < PIECES; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  a[h][k] = operand(cur, r, (wave % KS * CHUNK + i % CHUNK) * PIECES + h, 2 * g + k, lane);
              group(g, i % RING, a, r);
            }
          }
        }
        load_step(i % RING, p + RING, lane);
        if (i % CHUNK == CHUNK - 1) {
          put(other, wave, lane);
          __syncthreads();
          uint8_t *x = cur;
          cur = other;
          other = x;
        }
      }
    }
  }
};

// The KS parts' sums meet, in order, in the first part's wavefront.
template <int N, int KS>
__device__ __forceinline__ void meet(v4f (&acc)[N], uint8_t *lds, int w, int lane) {
  if constexpr (KS > 1) {
    v4f (*red)[N][64] = reinterpret_cast<v4f (*)[N][64]>(lds);
    if (w % KS != 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[w][i][lane] = acc[i];
    }
    __syncthreads();
    if (w % KS == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 1; k < KS; ++k) {
          const v4f y = red[w + k][i][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] += y[e];
        }
    }
    __syncthreads();
  }
}

// h = act(gate) * up of 16 columns a wavefront (tiles: the gate's and the up's).
template <bool F16, bool GELU, int KS, int R, bool PLAN, int WAVES>
__global__ __launch_bounds__(WAVES * 64) __attribute__((amdgpu_waves_per_eu(2))) void moe_gate_up_kernel(MoeArgs a) {
  typedef Product<2, 1, KS, R, WAVES> Pr;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Pr::LDS_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typedef typename RowsOf<PLAN, WAVES>::type Rows;
  __shared__ __attribute__((aligned(16))) uint8_t plan[Rows::LDS_BYTES];
  Rows rows;
  if (!rows.find(a, blockIdx.y, plan, lane)) return;
  const int n = a.I / kAwqTile, tile = blockIdx.x * (WAVES / KS) + w / KS;
  Pr pr;
  const int tiles[2] = {min(tile, n - 1), min(tile, n - 1) + n};
  pr.init(a.gate_up + rows.expert * a.gate_up_stride, MoeWeightLayout(2 * (int64_t)a.I, a.K), tiles, w);
  pr.src = a.x;
  pr.ld = a.K;
  for (int r0 = 0; r0 < rows.count; r0 += 16 * R) {
    int row[4 * R];
#pragma unroll
    for (int j = 0; j < 4 * R; ++j) row[j] = rows.one(min(r0 + Pr::block_row(w, j), rows.count - 1)) / a.top_k;
    v4f acc[2 * R] = {};
    pr.run(lds, row, w, lane, [&](int g, int i, const uint4 (&x)[1][2], int r) {
      v4f xsum = v4f{};
      if constexpr (!F16) xsum = mma(x[0][1], units(), mma(x[0][0], units(), v4f{}));
#pragma unroll
      for (int t = 0; t < 2; ++t)
        group_mma<F16>(x[0][0], x[0][1], xsum, g ? pr.code[i][t].z : pr.code[i][t].x,
                       g ? pr.code[i][t].w : pr.code[i][t].y, g ? pr.sz[i][t].y : pr.sz[i][t].x, acc[2 * r + t]);
    });
    meet<2 * R, KS>(acc, lds, w, lane);
    if (w % KS != 0) continue;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at_row = r0 + 16 * r + 4 * (lane >> 4) + e;
        const int64_t at = (int64_t)rows.pair(min(at_row, rows.count - 1)) * (2 * a.I) + tile / 4 * 128 +
                           tile % 4 * kAwqTile + (lane & 15);
        const float g = whole<F16>(acc[2 * r][e]), u = whole<F16>(acc[2 * r + 1][e]);
        const float h = (GELU ? gelu_tanh_f32(g) : g * __builtin_amdgcn_rcpf(1.0f + __expf(-g))) * u;
        if (at_row < rows.count && tile < n) split_h(h, a.h[at], a.h[at + kGroup]);
      }
  }
}

// TILES tiles of 16 columns of h Down^T a wavefront; h enters as its two bf16
// pieces (h to 2^-17, in float32's range).
template <int TILES, int FORM, int KS, int R, bool PLAN, int WAVES>
__global__ __launch_bounds__(WAVES * 64) __attribute__((amdgpu_waves_per_eu(2))) void moe_down_kernel(MoeArgs a) {
  typedef Product<TILES, FORM, KS, R, WAVES> Pr;
  __shared__ __attribute__((aligned(16))) uint8_t lds[Pr::LDS_BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typedef typename RowsOf<PLAN, WAVES>::type Rows;
  __shared__ __attribute__((aligned(16))) uint8_t plan[Rows::LDS_BYTES];
  Rows rows;
  if (!rows.find(a, blockIdx.y, plan, lane)) return;
  const int n = a.K / kAwqTile, tile0 = (blockIdx.x * (WAVES / KS) + w / KS) * TILES;
  Pr pr;
  int tiles[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) tiles[t] = min(tile0 + t, n - 1);
  pr.init(a.down + rows.expert * a.down_stride, MoeWeightLayout(a.K, a.I), tiles, w);
  pr.src = a.h;
  pr.ld = 2 * a.I;
  for (int r0 = 0; r0 < rows.count; r0 += Pr::ROWS) {
    int row[4 * R];
#pragma unroll
    for (int j = 0; j < 4 * R; ++j) row[j] = rows.one(min(r0 + Pr::block_row(w, j), rows.count - 1));
    v4f acc[TILES * R] = {};
    pr.run(lds, row, w, lane, [&](int g, int i, const uint4 (&h)[Pr::PIECES][2], int r) {
      v4f sum = v4f{};
#pragma unroll
      for (int k = 0; k < 2 * Pr::PIECES; ++k) sum = mma(h[k / 2][k % 2], units(), sum);
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const v8bf b0 = codes_128(g ? pr.code[i][t].z : pr.code[i][t].x);
        const v8bf b1 = codes_128(g ? pr.code[i][t].w : pr.code[i][t].y);
        v4f prod = v4f{};
#pragma unroll
        for (int k = 0; k < 2 * Pr::PIECES; ++k) prod = mma(h[k / 2][k % 2], k % 2 ? b1 : b0, prod);
        const uint32_t sz = g ? pr.sz[i][t].y : pr.sz[i][t].x;
        const float z = -(128.0f + (float)zero_of(sz)), sc = scale_of(sz);
        v4f &o = acc[TILES * r + t];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(__builtin_fmaf(z, sum[e], prod[e]), sc, o[e]);
      }
    });
    meet<TILES * R, KS>(acc, lds, w, lane);
    if (w % KS != 0) continue;
    if constexpr (FORM == 3) {            // the second pieces' sums stand 32 lanes on
#pragma unroll
      for (int i = 0; i < TILES * R; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] += __shfl_xor(acc[i][e], 32);
      if (lane >= 32) continue;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at_row = r0 + (FORM == 3 ? 8 : 16) * r + 4 * (lane >> 4) + e;
        const int64_t to = (int64_t)rows.pair(min(at_row, rows.count - 1)) * a.K + (lane & 15);
#pragma unroll
        for (int t = 0; t < TILES; ++t)
          if (at_row < rows.count && tile0 + t < n) a.part[to + (tile0 + t) * kAwqTile] = whole<false>(acc[TILES * r + t][e]);
      }
  }
}

// ------------------------------------------------- a handful of pairs
// A step of one or two sequences: up to kMoeFewPairs (token, choice) pairs of up
// to kFewExperts experts.  The layer is two kernels and all latency: each
// wavefront holds all its loads in flight, rows come straight into operands
// (there are few, so they share lines), and the down product's workgroups own
// their columns of y, so the sum over the choices needs no kernel of its own.
// One token with 8 of 64 experts of 2048 x 768: 15.4 us against 17.0 in the form
// above (21 MB of weights, 3.4 us at the rate of a long read; the two kernels'
// launches and the chain ids, rows and weights, product, meeting make up the rest).
// A workgroup's weights of down are (experts) x I / 128 steps, and every 256
// column tiles are a turn of the machine's CUs; at most kFewSteps steps in all
// turns: 64 steps (2 experts of 4096 x 4096) 21.4 against 29.5, 128 (8 of 2048 x
// 2048) 25.9 and 23.6, 224 (8 of 4096 x 3584) 64 and 44; two turns of 64 (4 of
// 7168 x 2048) 38.6 and 33.7.  With more experts the other form's workgroups
// are enough: 12 tokens with one of 32 experts of 2048 x 512 17.2 and 16.1, 8 with
// one of 64 of 2048 x 768 15.3 and 16.3.
// kMoeFewPairs is the rows of its tile; with 16 pairs of 8 experts of 2048 x 768
// 16.1 and 16.8 us, of 4 experts 13.2 and 15.0.
constexpr int kFewSteps = 64, kFewExperts = 8;
constexpr int kFewGateParts = 4, kFewDownWaves = 8;     // wavefronts a workgroup (8 and 16: 19.9 and 16.6 us)
template <int TILES>
struct FewWeights {
  uint4 code[TILES];
  uint2 sz[TILES];
  __device__ __forceinline__ void load(const uint8_t *const (&w)[TILES], int p, int lane) {
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const uint8_t *block = w[t] + (int64_t)p * kMoeBlockBytes;
      code[t] = *reinterpret_cast<const uint4 *>(block + (uint32_t)lane * 16);
      sz[t] = *reinterpret_cast<const uint2 *>(block + (kAwqBlockBytes + (uint32_t)(lane & 15) * 8));
    }
  }
};
template <int PIECES>
struct FewRows {
  uint4 x[PIECES][4];
  __device__ __forceinline__ void load(const uint16_t *row, int p, int G, int lane) {
#pragma unroll
    for (int h = 0; h < PIECES; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[h][k] = *reinterpret_cast<const uint4 *>(row + (min(2 * p + k / 2, G - 1) * PIECES + h) * kGroup +
                                                   16 * (lane >> 4) + 8 * (k % 2));
  }
};

template <bool F16, bool GELU, int KS>
__global__ __launch_bounds__(KS * 64) __attribute__((amdgpu_waves_per_eu(2))) void moe_gate_up_few_kernel(MoeArgs a) {
  __shared__ v4f red[KS][2][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  WaveRows rows;
  if (!rows.find(a, blockIdx.y, lane)) return;
  const int n = a.I / kAwqTile, tile = blockIdx.x;
  const MoeWeightLayout L(2 * (int64_t)a.I, a.K);
  const uint8_t *blob = a.gate_up + rows.expert * a.gate_up_stride;
  const uint8_t *const tiles[2] = {blob + L.block(tile, 0), blob + L.block(tile + n, 0)};
  const uint16_t *x = a.x + (int64_t)(rows.pair(min(lane & 15, rows.count - 1)) / a.top_k) * a.K;
  const int G = (int)L.G, P = (int)L.P, each = (P + KS - 1) / KS;
  const int p0 = min(P, w * each), p1 = min(P, p0 + each);
  v4f acc[2] = {};
  constexpr int AHEAD = 4;
  FewWeights<2> s[AHEAD];
  FewRows<1> r[AHEAD];
  for (int p = p0; p < p1; p += AHEAD) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) s[i].load(tiles, min(p + i, p1 - 1), lane);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) r[i].load(x, min(p + i, p1 - 1), G, lane);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (p + i >= p1) break;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (2 * (p + i) + g >= G) break;
        const uint4 a0 = r[i].x[0][2 * g], a1 = r[i].x[0][2 * g + 1];
        v4f xsum = v4f{};
        if constexpr (!F16) xsum = mma(a1, units(), mma(a0, units(), v4f{}));
#pragma unroll
        for (int t = 0; t < 2; ++t)
          group_mma<F16>(a0, a1, xsum, g ? s[i].code[t].z : s[i].code[t].x, g ? s[i].code[t].w : s[i].code[t].y,
                         g ? s[i].sz[t].y : s[i].sz[t].x, acc[t]);
      }
    }
  }
  red[w][0][lane] = acc[0];
  red[w][1][lane] = acc[1];
  __syncthreads();
  // one element a thread of the first four wavefronts: row 4 (lane / 16) + w
  if (w >= 4) return;
  float g = 0.0f, u = 0.0f;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    g += red[k][0][lane][w];
    u += red[k][1][lane][w];
  }
  g = whole<F16>(g);
  u = whole<F16>(u);
  const float h = (GELU ? gelu_tanh_f32(g) : g * __builtin_amdgcn_rcpf(1.0f + __expf(-g))) * u;
  const int row = 4 * (lane >> 4) + w;
  const int64_t at = (int64_t)rows.pair(min(row, rows.count - 1)) * (2 * a.I) + tile / 4 * 128 + tile % 4 * kAwqTile + (lane & 15);
  if (row < rows.count) split_h(h, a.h[at], a.h[at + kGroup]);
}

// y's 16 columns of one workgroup.  The (expert, step) items of all experts
// form one line, of which each wavefront takes an equal piece.  Row t of the
// tile is token t's; a token that did not choose the expert gets another's
// row, and its product is not taken.  A token that names an expert twice
// counts it with both weights.
template <bool F16, int WAVES>
__global__ __launch_bounds__(WAVES * 64) __attribute__((amdgpu_waves_per_eu(WAVES / 4))) void moe_down_few_kernel(MoeArgs a) {
  __shared__ v4f red[WAVES][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = a.T * a.top_k;
  const int id = lane < n ? a.ids[lane] : -1;
  const float wt = lane < n ? a.weights[lane] : 0.0f;
  const MoeWeightLayout L(a.K, a.I);
  const int G = (int)L.G, P = (int)L.P;
  uint64_t left = __ballot(id >= 0 && id < a.E);
  // the experts: lane i is the first of its expert's pairs if no lower one has the same id
  bool first = false;
  {
    uint64_t rest = left;
    while (rest) {
      const int f = __builtin_ctzll(rest);
      rest &= ~__ballot(id == __builtin_amdgcn_readlane(id, f));
      if (lane == f) first = true;
    }
  }
  uint64_t firsts = __ballot(first);
  const int items = __builtin_popcountll(firsts) * P, each = (items + WAVES - 1) / WAVES;
  int at = min(items, w * each);
  const int end = min(items, at + each);
  v4f y = v4f{};
  for (int slot = 0; at < end; ++slot, firsts &= firsts - 1) {
    if (at >= (slot + 1) * P) continue;
    const int expert = __builtin_amdgcn_readlane(id, __builtin_ctzll(firsts));
    const uint64_t same = __ballot(id == expert);
    // the pairs of token lane % 16, and its weight
    const int t0 = (lane & 15) * a.top_k;
    const uint64_t mine = t0 < 64 ? same >> t0 & ((2ull << (a.top_k - 1)) - 1) : 0;
    const int pair = mine ? t0 + __builtin_ctzll(mine) : __builtin_ctzll(same);
    float weight = 0.0f;
    for (uint64_t any = __ballot(mine != 0), m = mine; any; any = __ballot(m != 0)) {
      const float x = __shfl(wt, m ? t0 + __builtin_ctzll(m) : 0);
      if (m) weight += x;
      m &= m - 1;
    }
    const uint8_t *const tile[1] = {a.down + expert * a.down_stride + L.block(blockIdx.x, 0)};
    const uint16_t *h = a.h + (int64_t)pair * (2 * a.I);
    const int p1 = min(P, end - slot * P);
    v4f acc = v4f{};
    // weights eight steps ahead, rows (from the cache) two
    constexpr int AHEAD = 8, RA = 2;
    FewWeights<1> s[AHEAD];
    FewRows<2> r[RA];
    for (int p = at - slot * P; p < p1; p += AHEAD) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) s[i].load(tile, min(p + i, p1 - 1), lane);
#pragma unroll
      for (int i = 0; i < RA; ++i) r[i].load(h, min(p + i, p1 - 1), G, lane);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (p + i >= p1) break;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (2 * (p + i) + g >= G) break;
          const uint4 h0 = r[i % RA].x[0][2 * g], h1 = r[i % RA].x[0][2 * g + 1];
          const uint4 l0 = r[i % RA].x[1][2 * g], l1 = r[i % RA].x[1][2 * g + 1];
          const v8bf b0 = codes_128(g ? s[i].code[0].z : s[i].code[0].x), b1 = codes_128(g ? s[i].code[0].w : s[i].code[0].y);
          const v4f sum = mma(l1, units(), mma(l0, units(), mma(h1, units(), mma(h0, units(), v4f{}))));
          const v4f prod = mma(l1, b1, mma(l0, b0, mma(h1, b1, mma(h0, b0, v4f{}))));
          const uint32_t sz = g ? s[i].sz[0].y : s[i].sz[0].x;
          const float z = -(128.0f + (float)zero_of(sz)), sc = scale_of(sz);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(__builtin_fmaf(z, sum[e], prod[e]), sc, acc[e]);
        }
        if (i + RA < AHEAD) r[i % RA].load(h, min(p + i + RA, p1 - 1), G, lane);
      }
    }
    const uint64_t chose = __ballot(mine != 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 4 * (lane >> 4) + e;
      const float x = __shfl(weight, t);
      if (chose >> t & 1) y[e] = __builtin_fmaf(x, whole<false>(acc[e]), y[e]);
    }
    at = slot * P + p1;
  }
  red[w][lane] = y;
  __syncthreads();
  if (w >= 4) return;
  const int t = 4 * (lane >> 4) + w;
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < WAVES; ++k) v += red[k][lane][w];
  if (t < a.T)
    a.y[(int64_t)t * a.K + blockIdx.x * kAwqTile + (lane & 15)] =
        F16 ? __builtin_bit_cast(uint16_t, (_Float16)v) : __builtin_bit_cast(uint16_t, (__bf16)v);
}

// y[t] = sum over the token's choices of weight times part, in order; choices
// without an expert here are left out.  One thread per 4 columns of a token.
template <bool F16>
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeArgs a) {
  const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (c >= a.K) return;
  const int *ids = a.ids + (int64_t)t * a.top_k;
  const float *weights = a.weights + (int64_t)t * a.top_k;
  const float *part = a.part + (int64_t)t * a.top_k * a.K + c;
  v4f y = v4f{};
  for (int j0 = 0; j0 < a.top_k; j0 += 4) {      // four rows' loads in flight
    v4f v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const v4f *>(part + (int64_t)min(j0 + k, a.top_k - 1) * a.K);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (j0 + k >= a.top_k) break;
      const int e = ids[j0 + k];
      const float w = weights[j0 + k];
      if (e >= 0 && e < a.E) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(w, v[k][i], y[i]);
      }
    }
  }
  uint2 out;
  if constexpr (F16) {
    out.x = __builtin_bit_cast(uint32_t, v2h{(_Float16)y[0], (_Float16)y[1]});
    out.y = __builtin_bit_cast(uint32_t, v2h{(_Float16)y[2], (_Float16)y[3]});
  } else {
    out.x = pack_bf16(y[0], y[1]);
    out.y = pack_bf16(y[2], y[3]);
  }
  *reinterpret_cast<uint2 *>(a.y + (int64_t)t * a.K + c) = out;
}

}  // namespace

extern "C" {

svdq_status_t awq_moe_pack_on_device(const uint8_t *q, const uint16_t *s, const uint16_t *z, int E, int N, int K,
                                     void *blob, size_t bytes, void *hip_stream) {
  if (!q || !s || !z || !blob) return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_pack_on_device: NULL");
  if (!aligned16(q) || !aligned16(blob) || (((uintptr_t)s | (uintptr_t)z) & 1u))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "awq_moe_pack_on_device: misaligned pointer");
  const size_t need = awq_moe_device_weights_bytes(E, N, K);
  if (need == 0) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (bytes < need)
    return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "awq_moe_pack_on_device: blob needs %zu bytes, got %zu", need, bytes);
  const svdq_status_t st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  const MoeWeightLayout L(N, K);
  const int64_t blocks = (int64_t)E * (N / kAwqTile) * L.P;
  hipLaunchKernelGGL(moe_pack_kernel, dim3((unsigned)((blocks + 3) / 4)), dim3(256), 0, static_cast<hipStream_t>(hip_stream),
                     q, s, z, blocks, K, (int)L.G, (int)L.P, static_cast<uint8_t *>(blob));
  return launch_status("expert weight packing launch");
}

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
  const int sigmoid = score == SVDQ_MOE_SIGMOID ? 1 : 0;
  if (route_turns(E, K) <= kSmallTurns && T <= 256) {
#define MOE_ROUTE(F, P) hipLaunchKernelGGL((moe_route_kernel<F, P>), dim3((unsigned)T), dim3(1024), 0, stream, xp, wp, bias, E, \
                                           K, top_k, sigmoid, normalize, ids, weights)
    if (dtype == SVDQ_FP16) {
      if (E <= 64) MOE_ROUTE(true, 1); else MOE_ROUTE(true, 2);
    } else {
      if (E <= 64) MOE_ROUTE(false, 1); else MOE_ROUTE(false, 2);
    }
#undef MOE_ROUTE
    return launch_status("router launch");
  }
  if ((int64_t)T * E > kTileLogits) {
    const dim3 grid((unsigned)((E + 15) / 16), (unsigned)((T + 15) / 16));
    if (dtype == SVDQ_FP16)
      hipLaunchKernelGGL((moe_logits_tile_kernel<true>), grid, dim3(512), 0, stream, xp, wp, T, E, K, logits);
    else
      hipLaunchKernelGGL((moe_logits_tile_kernel<false>), grid, dim3(512), 0, stream, xp, wp, T, E, K, logits);
  } else {
    const dim3 grid((unsigned)((E + 3) / 4), (unsigned)((T + kTokens - 1) / kTokens));
    if (dtype == SVDQ_FP16)
      hipLaunchKernelGGL((moe_logits_kernel<true>), grid, dim3(256), 0, stream, xp, wp, T, E, K, logits);
    else
      hipLaunchKernelGGL((moe_logits_kernel<false>), grid, dim3(256), 0, stream, xp, wp, T, E, K, logits);
  }
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
  a.gate_up_stride = MoeWeightLayout(2 * (int64_t)w->I, w->K).total;
  a.down_stride = MoeWeightLayout(w->K, w->I).total;
  a.E = w->E;
  a.K = w->K;
  a.I = w->I;
  a.x = static_cast<const uint16_t *>(x);
  a.T = T;
  a.top_k = top_k;
  a.ids = ids;
  a.weights = weights;
  a.h = reinterpret_cast<uint16_t *>(ws + L.h);
  a.part = reinterpret_cast<float *>(ws + L.part);
  a.y = static_cast<uint16_t *>(y);
  a.plan = reinterpret_cast<MoePlan *>(ws + L.plan);
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const int pairs = T * top_k, slots = pairs < w->E ? pairs : w->E;       // experts in use at most
  const int gt = w->I / kAwqTile, dt = w->K / kAwqTile;
  const bool gelu = act == SVDQ_MOE_GELU_TANH;
  const int64_t few_steps = (int64_t)slots * ((w->I + 127) / 128) * ((dt + 255) / 256);
  if (pairs <= kMoeFewPairs && slots <= kFewExperts && few_steps <= kFewSteps) {
#define MOE_FEW(F, A)                                                                                            \
  hipLaunchKernelGGL((moe_gate_up_few_kernel<F, A, kFewGateParts>), dim3((unsigned)gt, (unsigned)slots),         \
                     dim3(kFewGateParts * 64), 0, stream, a)
#define MOE_FEW_DOWN(F)                                                                                          \
  hipLaunchKernelGGL((moe_down_few_kernel<F, kFewDownWaves>), dim3((unsigned)dt), dim3(kFewDownWaves * 64), 0, stream, a)
    if (dtype == SVDQ_FP16) {
      if (gelu) MOE_FEW(true, true); else MOE_FEW(true, false);
      MOE_FEW_DOWN(true);
    } else {
      if (gelu) MOE_FEW(false, true); else MOE_FEW(false, false);
      MOE_FEW_DOWN(false);
    }
#undef MOE_FEW_DOWN
#undef MOE_FEW
    return launch_status("expert layer launch");
  }
  // Blocks of 32 rows from 12 pairs an expert on: an expert of more than 16 rows
  // then reads its weights once, not twice.  16 experts of 2048 x 704, blocks of 16
  // and of 32: 10 pairs an expert 23.9 and 29.7 us, 12 30.9 and 30.0, 14 31.6 and 30.3, 16
  // 36.2 and 30.6; 8 of 4096 x 3584: 10 49.9 and 65.0, 12 61.4 and 66.2, 16 84.0 and 67.5.
  const bool many = pairs > 12 * slots;
  // Up to 5 pairs an expert, both pieces of h in one tile: 12 tokens with 6 of 64
  // experts took 57.3 us against 62.6, 8 with 2 of 8 45 against 51; at 8 pairs an
  // expert, where four experts in ten have more than 8 rows, 108 against 92.  (The
  // rule knows the average only: an expert's down weights are read once per 8
  // of its rows however many those are.  128 tokens that all choose the same one of
  // 128 experts of 2048 x 768 take 186 us, 132 in the other form.)
  const bool packed = pairs <= 5 * slots;
  // Few tiles: K in parts for the wavefronts of a workgroup.  With 256 and 512
  // tiles of gate and up 16.2 and 26.5 us in four parts, 20.2 and 31.5 in one;
  // layers with 768 tiles 29.6 us in two parts (24.3 and 26.1 with 1024), 36.8 in
  // one (24.7, 26.9), 29.7 in four (28.8, 30.9); with 1280 tiles of 32 steps 51.9
  // in two, 55.1 in one, 57.6 in four; with 1792, 59.1, 55.5 and 67.3.
  // Down, as two parts of two tiles and as four tiles: layers of 2048 tiles 20.8 and
  // 23.0 us (11 steps 27.3 and 30.6), 2560 23.0 and 23.9 (30.8, 31.7), 2816 23.3 and 24.5,
  // 12 x 256 24.8 and 25.4 (32.9, 33.1), 3328 29.5 and 28.0 (37.0, 36.6), 4096 32.4 and 29.5,
  // 8192 51.0 and 45.8.
  const int64_t gate_tiles = (int64_t)slots * gt;
  const int gate_parts = gate_tiles < 640 ? 4 : gate_tiles < 1536 ? 2 : 1;
  const int64_t down_tiles = (int64_t)slots * dt;
  const bool few_down = down_tiles <= 12 * 256;
  const bool plan = pairs > kLocalPairs;
  if (plan) hipLaunchKernelGGL(moe_plan_kernel, dim3(1), dim3(1024), 0, stream, a);
  // Wavefronts a workgroup: eight share a row's chunk, twice as long, where a
  // product has many steps and few tiles; with more tiles, or few steps, smaller
  // workgroups fill the machine more evenly.  Layer of 8 experts of 4096 x 3584
  // (1792 tiles of gate and up): 52.7 us with eight, 55.4 with four; of 32 experts
  // of 4096 x 1536 72.9 and 62.3; gate and up of 16 steps 51.7 and 47.3; down of 20
  // steps 50.9 and 46.0.  Layers whose down has 28 or 32 steps, with eight (two parts) and
  // with four wavefronts as four tiles: 3328 tiles 72.8 and 74.6, 84.7 and 89.7; 4096
  // tiles 89.5 and 88.7.
  const bool large_gate = w->K >= 24 * 2 * kGroup && gate_tiles < 2560;
  const bool large_down = w->I >= 24 * 2 * kGroup && down_tiles < 4096;
#define MOE_GU(F, A, KS, R, P, W)                                                                                \
  hipLaunchKernelGGL((moe_gate_up_kernel<F, A, KS, R, P, W>), dim3((gt + W / KS - 1) / (W / KS), (unsigned)slots), \
                     dim3(W * 64), 0, stream, a)
#define MOE_GU_R(F, A, KS, W)                       \
  do {                                              \
    if (many && plan) MOE_GU(F, A, KS, 2, true, W); \
    else if (many) MOE_GU(F, A, KS, 2, false, W);   \
    else if (plan) MOE_GU(F, A, KS, 1, true, W);    \
    else MOE_GU(F, A, KS, 1, false, W);             \
  } while (0)
#define MOE_GU_K(F, A)                              \
  do {                                              \
    if (gate_parts == 4) MOE_GU_R(F, A, 4, 4);      \
    else if (gate_parts == 2) MOE_GU_R(F, A, 2, 4); \
    else if (large_gate) MOE_GU_R(F, A, 1, 8);      \
    else MOE_GU_R(F, A, 1, 4);                      \
  } while (0)
#define MOE_DN(TT, FM, KS, R, P, W)                                                                              \
  hipLaunchKernelGGL((moe_down_kernel<TT, FM, KS, R, P, W>),                                                     \
                     dim3((dt + TT * (W / KS) - 1) / (TT * (W / KS)), (unsigned)slots), dim3(W * 64), 0, stream, a)
#define MOE_DN_R(TT, KS, W)                                  \
  do {                                                       \
    if (many && plan) MOE_DN(TT, 2, KS, 2, true, W);         \
    else if (many) MOE_DN(TT, 2, KS, 2, false, W);           \
    else if (packed && plan) MOE_DN(TT, 3, KS, 1, true, W);  \
    else if (packed) MOE_DN(TT, 3, KS, 1, false, W);         \
    else if (plan) MOE_DN(TT, 2, KS, 1, true, W);            \
    else MOE_DN(TT, 2, KS, 1, false, W);                     \
  } while (0)
  if (dtype == SVDQ_FP16) {
    if (gelu) MOE_GU_K(true, true); else MOE_GU_K(true, false);
  } else {
    if (gelu) MOE_GU_K(false, true); else MOE_GU_K(false, false);
  }
  if (large_down) MOE_DN_R(2, 2, 8);
  else if (few_down) MOE_DN_R(2, 2, 4);
  else MOE_DN_R(4, 1, 4);
#undef MOE_DN_R
#undef MOE_DN
#undef MOE_GU_K
#undef MOE_GU_R
#undef MOE_GU
  const dim3 g3((unsigned)((w->K / 4 + 255) / 256), (unsigned)T);
  if (dtype == SVDQ_FP16) hipLaunchKernelGGL((moe_sum_kernel<true>), g3, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((moe_sum_kernel<false>), g3, dim3(256), 0, stream, a);
  return launch_status("expert layer launch");
}

}  // extern "C"
