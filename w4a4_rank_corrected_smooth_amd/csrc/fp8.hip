// Linear in 8-bit floating point with a scale for each block of 128.
//
//  fp8_pack_kernel       canonical codes and scales -> operand blocks
//  fp8_quantize_kernel   16-bit rows -> operand blocks, or canonical codes
//  fp8_tile_kernel       the product, a tile of rows by channels to a workgroup
//  fp8_rows_kernel       the product for up to 96 rows: one stream of the weights
//  fp8_few_kernel        the same for up to 16 rows
//
// A block of 128 channels is two 32x32x64 block-scaled matrix instructions
// (e4m3, operands in fp8_layout.h's order), with the rows' power-of-two scales as the
// instruction's own E8M0 scales.  The weights' float32 scale, the same for a whole tile, is
// m 2^e: 2^e is the instruction's other scale, so that no sum leaves float32's range before the
// result does, and m in [1, 2) is applied by one FMA an element and block on the way into the sums:
//   P = sum_{k in block} (sx a) (2^e w),   acc = fma(P, m, acc).
// W is the A operand and X the B operand, so a lane's 16 results are of one row m
// = lane % 32, channels n = 8 j + 4 (lane / 32) + [0, 4) of the tile.
#include <hip/hip_runtime.h>

#include "common.h"
#include "device_util.h"
#include "fp8_layout.h"

using namespace svdq;

namespace {

struct Fp8Args {
  const uint8_t *w, *x;          // blocks
  const uint8_t *ws, *xs;        // their scales
  const float *bias;
  uint16_t *out;
  int M, N, blocks_k;
  int m_blocks, n_blocks;        // of 32
  int tiles_m, tiles_n;
  int gelu;
  // the forms for few rows that quantise them themselves
  const uint16_t *rows;
  int64_t rows_stride;
  int K;
};

template <bool F16>
__device__ __forceinline__ float widen(uint32_t h) {
  if constexpr (F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  else return __uint_as_float(h << 16);
}

// ---------------------------------------------------------------- quantiser
// Sixteen channels of a row (zeros past the end) to codes; the eight lanes of a block of 128
// are neighbours.  With a = max |x| = 1.f 2^(E - 127), 448 = 1.75 2^8: the smallest e
// with a <= 448 2^e is E - 135, or one more where f > 0.75, and at least -127.
// x 2^-e is exact (16-bit values are multiples of 2^-133, bfloat16's smallest, and 2^-e is 2^127 at most) and at most 448.
template <bool F16>
__device__ __forceinline__ uint32_t quantize16(const uint16_t *src, int k, int K, v4u &codes) {
  uint32_t in[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const v4u u = k + 8 * i < K ? *reinterpret_cast<const v4u *>(src + k + 8 * i) : v4u{0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 4; ++j) in[4 * i + j] = u[j];
  }
  float x[16];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = widen<F16>(in[i / 2] >> (16 * (i & 1)) & 0xFFFFu);
    top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, s));
  if (top >= 0x7F800000u) {
    codes = v4u{0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
    return 127u;
  }
  const int scale = max((int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u), 0);
  const float inv = __uint_as_float((uint32_t)(254 - scale) << 23);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int d = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * j] * inv, x[4 * j + 1] * inv, 0, false);
    d = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * j + 2] * inv, x[4 * j + 3] * inv, d, true);
    codes[j] = (uint32_t)d;
  }
  return (uint32_t)scale;
}

// A workgroup: 32 rows by one block.  Bound by memory (4095 x 4608: 56 MB in 10.6 us, 5.3 TB/s).  CANON: codes [M, K] and scales [M, blocks] instead of operand blocks.
template <bool F16, bool CANON>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(const uint16_t *__restrict__ x, int64_t x_row, int M, int K,
                                                           int blocks_k, uint8_t *__restrict__ out,
                                                           uint8_t *__restrict__ scales) {
  const int mb = blockIdx.x / blocks_k, kb = blockIdx.x - mb * blocks_k;
  const int u = threadIdx.x & 7, r = threadIdx.x >> 3, m = 32 * mb + r;
  if (m >= M) return;
  v4u codes;
  const int k = 128 * kb + 16 * u;
  const uint32_t s = quantize16<F16>(x + (int64_t)m * x_row, k, K, codes);
  if constexpr (CANON) {
    uint8_t *to = out + (int64_t)m * K + k;
    if (k < K) *reinterpret_cast<uint2 *>(to) = make_uint2(codes[0], codes[1]);
    if (k + 8 < K) *reinterpret_cast<uint2 *>(to + 8) = make_uint2(codes[2], codes[3]);
    if (u == 0) scales[(int64_t)m * blocks_k + kb] = (uint8_t)s;
  } else {
    *reinterpret_cast<v4u *>(out + (int64_t)blockIdx.x * kFp8Block + (u >> 1) * 1024 + (u & 1) * 512 + 16 * r) = codes;
    if (u == 0) scales[(int64_t)blockIdx.x * kFp8XScales + r] = (uint8_t)s;
  }
}

__global__ __launch_bounds__(256) void fp8_pack_kernel(const uint8_t *__restrict__ codes, const float *__restrict__ scales,
                                                       int N, int K, int blocks_k, uint8_t *__restrict__ blob) {
  const int nb = blockIdx.x / blocks_k, kb = blockIdx.x - nb * blocks_k;
  const int u = threadIdx.x & 7, r = threadIdx.x >> 3, n = 32 * nb + r, k = 128 * kb + 16 * u;
  const uint8_t *src = codes + (int64_t)n * K + k;
  uint2 lo = make_uint2(0, 0), hi = lo;
  if (n < N && k < K) lo = *reinterpret_cast<const uint2 *>(src);
  if (n < N && k + 8 < K) hi = *reinterpret_cast<const uint2 *>(src + 8);
  *reinterpret_cast<uint4 *>(blob + (int64_t)blockIdx.x * kFp8Block + (u >> 1) * 1024 + (u & 1) * 512 + 16 * r) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  if (threadIdx.x == 0) {
    const float sw = scales[(int64_t)(nb / 4) * blocks_k + kb];
    const uint32_t e = max(__float_as_uint(sw) >> 23 & 255u, 1u);
    // 2^(e - 127) with e from 1 (a subnormal scale's m is below 1) to 254
    const float m = ldexpf(sw, 127 - (int)e);
    *reinterpret_cast<uint2 *>(blob + (int64_t)gridDim.x * kFp8Block + (int64_t)blockIdx.x * kFp8WScales) =
        make_uint2(__float_as_uint(m), e);
  }
}

// ------------------------------------------------------------------ product
// One half (64 channels) of a tile's product with a block of K.
__device__ __forceinline__ v16f mma_half(const v4u &w0, const v4u &w1, int we, const v4u &x0, const v4u &x1, int sx, v16f p) {
  const v8i a = {(int)w0[0], (int)w0[1], (int)w0[2], (int)w0[3], (int)w1[0], (int)w1[1], (int)w1[2], (int)w1[3]};
  const v8i b = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, p, 0, 0, 0, we, 0, sx);
}
__device__ __forceinline__ v16f zero16() {
  v16f p;
#pragma unroll
  for (int i = 0; i < 16; ++i) p[i] = 0.0f;
  return p;
}
__device__ __forceinline__ v16f mma(const v4u (&w)[4], int we, const v4u (&x)[4], int sx) {
  return mma_half(w[2], w[3], we, x[2], x[3], sx, mma_half(w[0], w[1], we, x[0], x[1], sx, zero16()));
}

// OUT: svdq_dtype_t of the result
template <int OUT>
__device__ __forceinline__ uint16_t narrow(float y) {
  if constexpr (OUT == SVDQ_FP16) return __builtin_bit_cast(uint16_t, (_Float16)y);
  else return __builtin_bit_cast(uint16_t, (__bf16)y);
}
template <int OUT>
__device__ __forceinline__ uint32_t pair_of(float a, float b) {
  if constexpr (OUT == SVDQ_FP16) {
    const v2h h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
  } else {
    typedef __bf16 v2b __attribute__((ext_vector_type(2)));
    const v2b h = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, h);
  }
}

// The epilogue of four results of one row, channels n .. n + 3.
__device__ __forceinline__ v4f finish(const Fp8Args &a, v4f bias, v4f y) {
  y += bias;
  if (a.gelu) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = gelu_tanh_f32(y[e]);
  }
  return y;
}

// A wavefront's tile is TM blocks of rows by TN blocks of channels, a workgroup's
// WM by WN of those; ST stages of one block of K in LDS.
//
// The matrix core and the vector ALU work side by side only where the code lets them: the two
// instructions of a tile are followed by the 16 FMAs of the tile before, eight to each
// (alone, such an instruction takes 27 ns, with eight FMAs 31, and FMAs that wait for their own
// tile's result cost their full 15 ns for eight).  Operands of the next block of K are read from LDS during the last row of
// tiles, so that the barrier before it, which frees the stage just read for the
// next copy, costs no read of its own.  4608 x 16384 x 4096 in tiles of 256 x 256: 305 to 330 us with the quantiser and GELU,
// by the card's clock under load, 2.0 PFLOP/s (with zeros for values 254 us); bound by the matrix core.
template <int TM, int TN, int WM, int WN, int ST, int OUT>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tile_kernel(const Fp8Args a) {
  constexpr int XB = TM * WM, WB = TN * WN, WAVES = WM * WN, COPIES = (XB + WB + WAVES - 1) / WAVES;
  // a stage: the blocks of X and W, then their scales, 256 bytes to each (what a copy writes)
  constexpr int W_AT = XB * kFp8Block, XS_AT = W_AT + WB * kFp8Block, WS_AT = XS_AT + XB * 256;
  constexpr int STAGE = WS_AT + WB * 256;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[ST * STAGE];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w % WM, wn = w / WM;
  // Workgroups are dealt out to the eight XCDs in turn: each XCD gets a contiguous
  // run of tiles, eight rows of tiles high, so that its L2 holds few rows and channels.
  const int tiles = a.tiles_m * a.tiles_n, per = (tiles + 7) / 8;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= tiles) return;
  const int band = id / (8 * a.tiles_n), high = min(8, a.tiles_m - 8 * band), in = id - band * 8 * a.tiles_n;
  const int tm = 8 * band + in % high, tn = in / high;

  const uint32_t lds_at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds);
  // the blocks that this wavefront copies (the last one more than once where they do not come out even)
  auto block_of = [&](int c) { return (XB + WB) % WAVES == 0 ? w + WAVES * c : min(w + WAVES * c, XB + WB - 1); };
  const uint8_t *from[COPIES], *scale[COPIES];
  uint32_t scale_lane[COPIES];
  int scale_step[COPIES];
#pragma unroll
  for (int c = 0; c < COPIES; ++c) {
    const int i = block_of(c);
    const bool is_x = i < XB;
    const int64_t at = (int64_t)(is_x ? min(tm * XB + i, a.m_blocks - 1) : min(tn * WB + i - XB, a.n_blocks - 1)) * a.blocks_k;
    from[c] = (is_x ? a.x : a.w) + at * kFp8Block;
    scale_step[c] = is_x ? kFp8XScales : kFp8WScales;
    scale[c] = (is_x ? a.xs : a.ws) + at * scale_step[c];
    scale_lane[c] = min(4 * lane, scale_step[c] - 4);
  }
  // The next block of K, five copies for each of its blocks, one at a time; behind the last one
  // it is copied again, so that the loop has no branch for the compiler to move its work across.
  constexpr int FETCHES = 5 * COPIES;
  int fetched = 0;
  auto fetch1 = [&](int stage, int f) {
    const int c = f / 5, j = f % 5, i = block_of(c);
    const uint32_t at = lds_at + stage * STAGE;
    if (j < 4) {
      lds_dma16_s(from[c] + 1024 * j, 16 * lane, at + i * kFp8Block + 1024 * j);
    } else {
      lds_dma4_s(scale[c], scale_lane[c], at + XS_AT + i * 256);
      if (c + 1 == COPIES) ++fetched;
      const int more = c + 1 == COPIES ? fetched < a.blocks_k : fetched + 1 < a.blocks_k;
      from[c] += more * kFp8Block;
      scale[c] += more * scale_step[c];
    }
  };
  auto fetch = [&](int stage) {
#pragma unroll
    for (int f = 0; f < FETCHES; ++f) fetch1(stage, f);
  };

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  v4u wf[TN][4], xf[4];
  uint2 sw[TN];
  int sx;
  auto read_w = [&](const uint8_t *st, int j, int half) {
#pragma unroll
    for (int q = 2 * half; q < 2 * half + 2; ++q)
      wf[j][q] = *reinterpret_cast<const v4u *>(st + W_AT + (wn * TN + j) * kFp8Block + 1024 * q + 16 * lane);
    if (half == 1) sw[j] = *reinterpret_cast<const uint2 *>(st + WS_AT + (wn * TN + j) * 256);
  };
  auto read_x = [&](const uint8_t *st, int i, int half) {
    if (half == 0) sx = st[XS_AT + (wm * TM + i) * 256 + (lane & 31)];
#pragma unroll
    for (int q = 2 * half; q < 2 * half + 2; ++q)
      xf[q] = *reinterpret_cast<const v4u *>(st + (wm * TM + i) * kFp8Block + 1024 * q + 16 * lane);
  };

#pragma unroll
  for (int s = 0; s < ST; ++s) fetch(s);
  vmcnt_wait<(ST - 1) * FETCHES>();
  __syncthreads();
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int j = 0; j < TN; ++j) read_w(lds, j, half);
    read_x(lds, 0, half);
  }
  // the product before, not yet added, and its m: its tile is the last one
  v16f p[2] = {zero16(), zero16()};
  float m = 0.0f;
  int stage = 0;
  for (int kb = 0; kb < a.blocks_k; ++kb) {
    const uint8_t *st = lds + stage * STAGE;
    const int next = stage + 1 == ST ? 0 : stage + 1;
    const uint8_t *ahead = lds + next * STAGE;        // behind the last block: bytes that are read and not used
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const bool last = i + 1 == TM;
      if (last) {
        // All reads of this stage are done, and the next one has landed when only the
        // copies of those after it are outstanding.
        vmcnt_wait<(ST - 2) * FETCHES>();
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int s = i * TN + j;
        const float m_now = __uint_as_float(sw[j].x);
        const int we = (int)sw[j].y, scale_x = sx;
        v16f &sum = s == 0 ? acc[TM - 1][TN - 1] : acc[(s - 1) / TN][(s - 1) % TN];
        const v16f &before = p[~s & 1];
        v16f now = zero16();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          __builtin_amdgcn_s_setprio(1);
          now = mma_half(wf[j][2 * half], wf[j][2 * half + 1], we, xf[2 * half], xf[2 * half + 1], scale_x, now);
          __builtin_amdgcn_s_setprio(0);
          // operands that this was the last to use make room for their successors
          if (last) {
            read_w(ahead, j, half);
#pragma unroll
            for (int f = (2 * j + half) * FETCHES / (2 * TN); f < (2 * j + half + 1) * FETCHES / (2 * TN); ++f) fetch1(stage, f);
          }
          if (j + 1 == TN) read_x(last ? ahead : st, last ? 0 : i + 1, half);
#pragma unroll
          for (int e = 8 * half; e < 8 * half + 8; ++e) sum[e] = __builtin_fmaf(before[e], m, sum[e]);
          __builtin_amdgcn_sched_barrier(0);
        }
        p[s & 1] = now;
        m = m_now;
      }
    }
    if constexpr (TM * TN & 1) p[1] = p[0];
    stage = next;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[TM - 1][TN - 1][e] = __builtin_fmaf(p[1][e], m, acc[TM - 1][TN - 1][e]);

  // Results go through LDS, 32 rows at a time, so that a row's channels leave in whole
  // lines: 8 bytes a lane to 32 rows took a quarter of the kernel's time.
  constexpr int PITCH = 64 * TN + 16;                  // bytes of a row in LDS
  static_assert(WAVES * 32 * PITCH <= ST * STAGE, "LDS");
  vmcnt_wait0();
  __syncthreads();
  const int h = lane >> 5, n0 = 32 * (tn * WB + wn * TN);
  uint8_t *mine = lds + w * 32 * PITCH;
  const bool whole = (a.N & 7) == 0;
  v4f bias[TN][4];
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) bias[j][q][e] = a.bias ? a.bias[min(n0 + 32 * j + 8 * q + 4 * h + e, a.N - 1)] : 0.0f;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m0 = 32ll * ((int64_t)tm * XB + wm * TM + i);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v4f y = finish(a, bias[j][q], v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]});
        *reinterpret_cast<uint2 *>(mine + (lane & 31) * PITCH + 64 * j + 16 * q + 8 * h) =
            make_uint2(pair_of<OUT>(y[0], y[1]), pair_of<OUT>(y[2], y[3]));
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    constexpr int LANES = 4 * TN, ROWS = 64 / LANES;   // lanes of 16 bytes to a row
#pragma unroll
    for (int r = lane / LANES; r < 32; r += ROWS) {
      const uint4 y = *reinterpret_cast<const uint4 *>(mine + r * PITCH + (lane % LANES) * 16);
      const int n = n0 + (lane % LANES) * 8;
      if (m0 + r < a.M && n < a.N) {
        uint16_t *dst = a.out + (m0 + r) * a.N + n;
        if (whole) {
          *reinterpret_cast<uint4 *>(dst) = y;
        } else {
          const uint32_t words[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < a.N) dst[e] = (uint16_t)(words[e / 2] >> (16 * (e & 1)));
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// All rows, quantised into LDS by a workgroup of kFp8RowsWaves wavefronts: unit u of block kb of row m at ((8 kb + u)
// M + m) 16, its scale at kb M + m.  (Row, block) pairs, eight lanes to each.
constexpr int kFp8RowsWaves = 8, kFp8Ahead = 4;
template <bool F16>
__device__ __forceinline__ void quantize_rows(const Fp8Args &a, uint8_t *xl, uint8_t *xs) {
  for (int i = threadIdx.x >> 3; i < a.M * a.blocks_k; i += 8 * kFp8RowsWaves) {
    const int kb = i / a.M, m = i - kb * a.M, u = threadIdx.x & 7;
    v4u codes;
    const uint32_t s = quantize16<F16>(a.rows + m * a.rows_stride, 128 * kb + 16 * u, a.K, codes);
    *reinterpret_cast<v4u *>(xl + ((kb * 8 + u) * a.M + m) * 16) = codes;
    if (u == 0) xs[i] = (uint8_t)s;
  }
}

// Few rows.  A workgroup has 32 output channels; its eight wavefronts deal out
// the blocks of K among themselves and add up in LDS.  Weights go from memory
// straight into operands, AHEAD blocks of a wavefront in flight (one row of 6144 x 4096: 7.0 us, 3.7 TB/s, most of the
// rest the launch and the rows' quantising; 8 rows 10.3, 64 12.9, 96 14.9; 77 of 2121 x 1160: 9.1 with the quantiser's launch).  OWN: the
// workgroup quantises the rows itself, into LDS (one block of 32 rows, up to 24576 values in all).
template <int XB, bool OWN, bool F16, int OUT>
__global__ __launch_bounds__(64 * kFp8RowsWaves) void fp8_rows_kernel(const Fp8Args a) {
  constexpr int RED = kFp8RowsWaves * XB * 16 * 65 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[RED];
  __shared__ __attribute__((aligned(16))) uint8_t xl[OWN ? 24576 : 16];
  __shared__ uint8_t xs[OWN ? 192 : 1];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 31;
  const int nb = blockIdx.x;
  const uint8_t *wp = a.w + (int64_t)nb * a.blocks_k * kFp8Block, *wsp = a.ws + (int64_t)nb * a.blocks_k * kFp8WScales;

  v4u wf[kFp8Ahead][4];
  uint2 sw[kFp8Ahead];
  auto load = [&](int slot, int kb) {
    kb = min(kb, a.blocks_k - 1);
    const uint8_t *b = wp + (int64_t)kb * kFp8Block;
#pragma unroll
    for (int q = 0; q < 4; ++q) wf[slot][q] = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(b + 1024 * q + 16 * lane));
    sw[slot] = *reinterpret_cast<const uint2 *>(wsp + (int64_t)kb * kFp8WScales);
  };
#pragma unroll
  for (int i = 0; i < kFp8Ahead; ++i) load(i, w + kFp8RowsWaves * i);

  if constexpr (OWN) {
    quantize_rows<F16>(a, xl, xs);
    __syncthreads();
  }

  v16f acc[XB];
#pragma unroll
  for (int x = 0; x < XB; ++x)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[x][e] = 0.0f;
  for (int base = w; base < a.blocks_k; base += kFp8RowsWaves * kFp8Ahead) {
#pragma unroll
    for (int i = 0; i < kFp8Ahead; ++i) {
      const int kb = base + kFp8RowsWaves * i;
      if (kb >= a.blocks_k) break;
#pragma unroll
      for (int x = 0; x < XB; ++x) {
        v4u xf[4];
        int sx;
        if constexpr (OWN) {
          const bool in = r < a.M;
          const int rr = in ? r : 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            xf[q] = *reinterpret_cast<const v4u *>(xl + ((kb * 8 + 2 * q + (lane >> 5)) * a.M + rr) * 16);
            if (!in) xf[q] = v4u{0u, 0u, 0u, 0u};
          }
          sx = xs[kb * a.M + rr];
        } else {
          const int64_t at = (int64_t)min(x, a.m_blocks - 1) * a.blocks_k + kb;
          const uint8_t *b = a.x + at * kFp8Block;
#pragma unroll
          for (int q = 0; q < 4; ++q) xf[q] = *reinterpret_cast<const v4u *>(b + 1024 * q + 16 * lane);
          sx = a.xs[at * kFp8XScales + r];
        }
        const v16f p = mma(wf[i], (int)sw[i].y, xf, sx);
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[x][e] = __builtin_fmaf(p[e], __uint_as_float(sw[i].x), acc[x][e]);
      }
      if (kb + kFp8RowsWaves * kFp8Ahead < a.blocks_k) load(i, kb + kFp8RowsWaves * kFp8Ahead);
    }
  }
  float *red = reinterpret_cast<float *>(lds);      // [wavefront][block][register][65]
#pragma unroll
  for (int x = 0; x < XB; ++x)
#pragma unroll
    for (int e = 0; e < 16; ++e) red[((w * XB + x) * 16 + e) * 65 + lane] = acc[x][e];
  __syncthreads();
  const int rows = min(a.M, 32 * XB);
  for (int i = threadIdx.x; i < 32 * rows; i += 64 * kFp8RowsWaves) {
    const int c = i & 31, m = i >> 5, n = 32 * nb + c;
    if (n >= a.N) continue;
    const int e = (c >> 3) * 4 + (c & 3), l = (c >> 2 & 1) * 32 + (m & 31), x = m >> 5;
    float y = 0.0f;
#pragma unroll
    for (int v = 0; v < kFp8RowsWaves; ++v) y += red[((v * XB + x) * 16 + e) * 65 + l];
    if (a.bias) y += a.bias[n];
    if (a.gelu) y = gelu_tanh_f32(y);
    a.out[(int64_t)m * a.N + n] = narrow<OUT>(y);
  }
}

// Up to 16 rows.  As above, with 16 output channels to a workgroup, so that few channels make more
// workgroups, and more of a wavefront's part of K in flight (one row of 4096 x 14336, 59 MB: 15.3 us, 3.8 TB/s).  The
// instruction takes a whole block of 128: lane l holds units 2 (l / 16) and 2 (l / 16) + 1 of channel (of row) l % 16,
// and its results are of row l % 16, channels 4 (l / 16) + [0, 4).
constexpr int kFp8FewAhead = 8;
template <bool OWN, bool F16, int OUT>
__global__ __launch_bounds__(64 * kFp8RowsWaves) void fp8_few_kernel(const Fp8Args a) {
  __shared__ float red[kFp8RowsWaves][4][65];
  __shared__ __attribute__((aligned(16))) uint8_t xl[OWN ? 24576 : 16];
  __shared__ uint8_t xs[OWN ? 192 : 1];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int64_t first = (int64_t)(blockIdx.x >> 1) * a.blocks_k;
  const uint8_t *wp = a.w + first * kFp8Block + (blockIdx.x & 1) * 256 + g * 1024 + 16 * r, *wsp = a.ws + first * kFp8WScales;

  v4u wf[kFp8FewAhead][2];
  uint2 sw[kFp8FewAhead];
  auto load = [&](int slot, int kb) {
    kb = min(kb, a.blocks_k - 1);
    const uint8_t *b = wp + (int64_t)kb * kFp8Block;
#pragma unroll
    for (int q = 0; q < 2; ++q) wf[slot][q] = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(b + 512 * q));
    sw[slot] = *reinterpret_cast<const uint2 *>(wsp + (int64_t)kb * kFp8WScales);
  };
#pragma unroll
  for (int i = 0; i < kFp8FewAhead; ++i) load(i, w + kFp8RowsWaves * i);
  if constexpr (OWN) {
    quantize_rows<F16>(a, xl, xs);
    __syncthreads();
  }

  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool in = r < a.M;
  const int rr = in ? r : 0;
  for (int base = w; base < a.blocks_k; base += kFp8RowsWaves * kFp8FewAhead) {
#pragma unroll
    for (int i = 0; i < kFp8FewAhead; ++i) {
      const int kb = base + kFp8RowsWaves * i;
      if (kb >= a.blocks_k) break;
      v4u xf[2];
      int sx;
      if constexpr (OWN) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          xf[q] = *reinterpret_cast<const v4u *>(xl + ((kb * 8 + 2 * g + q) * a.M + rr) * 16);
          if (!in) xf[q] = v4u{0u, 0u, 0u, 0u};
        }
        sx = xs[kb * a.M + rr];
      } else {
        const uint8_t *b = a.x + (int64_t)kb * kFp8Block + g * 1024 + 16 * r;
#pragma unroll
        for (int q = 0; q < 2; ++q) xf[q] = *reinterpret_cast<const v4u *>(b + 512 * q);
        sx = a.xs[(int64_t)kb * kFp8XScales + r];
      }
      const v8i wa = {(int)wf[i][0][0], (int)wf[i][0][1], (int)wf[i][0][2], (int)wf[i][0][3],
                      (int)wf[i][1][0], (int)wf[i][1][1], (int)wf[i][1][2], (int)wf[i][1][3]};
      const v8i xb = {(int)xf[0][0], (int)xf[0][1], (int)xf[0][2], (int)xf[0][3],
                      (int)xf[1][0], (int)xf[1][1], (int)xf[1][2], (int)xf[1][3]};
      const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, (int)sw[i].y, 0, sx);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(p[e], __uint_as_float(sw[i].x), acc[e]);
      if (kb + kFp8RowsWaves * kFp8FewAhead < a.blocks_k) load(i, kb + kFp8RowsWaves * kFp8FewAhead);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[w][e][lane] = acc[e];
  __syncthreads();
  const int c = threadIdx.x & 15, m = threadIdx.x >> 4, n = 16 * blockIdx.x + c;
  if (m >= a.M || n >= a.N) return;
  float y = 0.0f;
#pragma unroll
  for (int v = 0; v < kFp8RowsWaves; ++v) y += red[v][c & 3][16 * (c >> 2) + m];
  if (a.bias) y += a.bias[n];
  if (a.gelu) y = gelu_tanh_f32(y);
  a.out[(int64_t)m * a.N + n] = narrow<OUT>(y);
}

template <int TM, int TN, int WM, int WN, int ST, int OUT>
void launch_tiles(Fp8Args &a, hipStream_t stream) {
  a.tiles_m = (a.M + 32 * TM * WM - 1) / (32 * TM * WM);
  a.tiles_n = (a.N + 32 * TN * WN - 1) / (32 * TN * WN);
  const dim3 grid((unsigned)((a.tiles_m * a.tiles_n + 7) / 8 * 8));
  hipLaunchKernelGGL((fp8_tile_kernel<TM, TN, WM, WN, ST, OUT>), grid, dim3(64 * WM * WN), 0, stream, a);
}

template <int OUT>
void launch_product(const Fp8Plan &p, Fp8Args &a, bool f16, hipStream_t stream) {
  if (p.form == FP8_FEW) {
    const dim3 grid((unsigned)(2 * a.n_blocks)), block(64 * kFp8RowsWaves);
    if (p.inline_x && f16) hipLaunchKernelGGL((fp8_few_kernel<true, true, OUT>), grid, block, 0, stream, a);
    else if (p.inline_x) hipLaunchKernelGGL((fp8_few_kernel<true, false, OUT>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((fp8_few_kernel<false, false, OUT>), grid, block, 0, stream, a);
    return;
  }
  if (p.form == FP8_ROWS) {
    const dim3 grid((unsigned)a.n_blocks), block(64 * kFp8RowsWaves);
    if (p.inline_x && f16) hipLaunchKernelGGL((fp8_rows_kernel<1, true, true, OUT>), grid, block, 0, stream, a);
    else if (p.inline_x) hipLaunchKernelGGL((fp8_rows_kernel<1, true, false, OUT>), grid, block, 0, stream, a);
    else if (p.x_blocks == 1) hipLaunchKernelGGL((fp8_rows_kernel<1, false, false, OUT>), grid, block, 0, stream, a);
    else if (p.x_blocks == 2) hipLaunchKernelGGL((fp8_rows_kernel<2, false, false, OUT>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((fp8_rows_kernel<3, false, false, OUT>), grid, block, 0, stream, a);
    return;
  }
  switch (p.form) {
    case FP8_256: launch_tiles<4, 2, 2, 4, 2, OUT>(a, stream); break;
    case FP8_192: launch_tiles<1, 2, 6, 2, 3, OUT>(a, stream); break;
    case FP8_128_DEEP: launch_tiles<2, 1, 2, 4, 4, OUT>(a, stream); break;
    case FP8_128: launch_tiles<2, 2, 2, 2, 2, OUT>(a, stream); break;
    default: launch_tiles<1, 1, 2, 2, 4, OUT>(a, stream); break;
  }
}

svdq_status_t rows_ok(const char *who, const void *x, int64_t x_row, svdq_dtype_t dtype) {
  if (dtype != SVDQ_BF16 && dtype != SVDQ_FP16)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: x must be SVDQ_BF16 or SVDQ_FP16", who);
  if (!aligned16(x) || x_row < 0 || x_row % 8 != 0)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: misaligned x, or a row stride that is not a multiple of 8", who);
  return SVDQ_OK;
}

void launch_quantize(const void *x, int64_t x_row, svdq_dtype_t dtype, int M, int K, void *out, uint8_t *scales,
                     bool canon, hipStream_t stream) {
  const int blocks_k = (K + 127) / 128;
  const dim3 grid((unsigned)((int64_t)((M + 31) / 32) * blocks_k));
  const uint16_t *xp = static_cast<const uint16_t *>(x);
  uint8_t *to = static_cast<uint8_t *>(out);
#define FP8_QUANTIZE(FF, CC) \
  hipLaunchKernelGGL((fp8_quantize_kernel<FF, CC>), grid, dim3(256), 0, stream, xp, x_row, M, K, blocks_k, to, scales)
  if (dtype == SVDQ_FP16) {
    if (canon) FP8_QUANTIZE(true, true);
    else FP8_QUANTIZE(true, false);
  } else {
    if (canon) FP8_QUANTIZE(false, true);
    else FP8_QUANTIZE(false, false);
  }
#undef FP8_QUANTIZE
}

}  // namespace

extern "C" {

svdq_status_t svdq_fp8_pack_on_device(const uint8_t *codes, const float *scales, int N, int K, void *blob, size_t bytes,
                                      void *hip_stream) {
  const char *who = "svdq_fp8_pack_on_device";
  if (!fp8_weights_ok(N, K)) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: N=%d K=%d", who, N, K);
  if (!codes || !scales || !blob) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL pointer", who);
  if (!aligned16(codes) || !aligned16(blob) || ((uintptr_t)scales & 3u))
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", who);
  if (bytes < (size_t)fp8_w_bytes(N, K))
    return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "%s: blob needs %lld bytes, got %zu", who, (long long)fp8_w_bytes(N, K), bytes);
  svdq_status_t st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  const int blocks_k = (K + 127) / 128;
  hipLaunchKernelGGL(fp8_pack_kernel, dim3((unsigned)((int64_t)((N + 31) / 32) * blocks_k)), dim3(256), 0,
                     static_cast<hipStream_t>(hip_stream), codes, scales, N, K, blocks_k, static_cast<uint8_t *>(blob));
  return launch_status("fp8 pack launch");
}

svdq_status_t svdq_fp8_quantize_activations(const void *x, int64_t x_row, svdq_dtype_t dtype, int M, int K,
                                            uint8_t *codes, uint8_t *scales, void *hip_stream) {
  const char *who = "svdq_fp8_quantize_activations";
  if (!fp8_weights_ok(1, K) || !fp8_call_ok(M, K)) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: M=%d K=%d", who, M, K);
  if (M == 0) return SVDQ_OK;
  if (!x || !codes || !scales) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL pointer", who);
  svdq_status_t st = rows_ok(who, x, x_row, dtype);
  if (st != SVDQ_OK) return st;
  if (!aligned16(codes)) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: misaligned codes", who);
  st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  launch_quantize(x, x_row, dtype, M, K, codes, scales, true, static_cast<hipStream_t>(hip_stream));
  return launch_status("fp8 quantize launch");
}

svdq_status_t svdq_fp8_linear_forward(const svdq_fp8_weights_t *w, const void *x, int64_t x_row, svdq_dtype_t x_dtype,
                                      int M, void *out, svdq_dtype_t out_dtype, svdq_epilogue_t epilogue,
                                      void *workspace, size_t ws_bytes, void *hip_stream) {
  const char *who = "svdq_fp8_linear_forward";
  if (!w || !w->blob) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL weights", who);
  if (!aligned16(w->blob) || ((uintptr_t)w->bias & 3u)) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: misaligned weights", who);
  if (!fp8_weights_ok(w->N, w->K) || !fp8_call_ok(M, w->N) || !fp8_call_ok(M, w->K))
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s: M=%d N=%d K=%d", who, M, w->N, w->K);
  if (epilogue != SVDQ_EPILOGUE_NONE && epilogue != SVDQ_EPILOGUE_GELU_TANH)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: epilogue %d", who, (int)epilogue);
  if (out_dtype != SVDQ_BF16 && out_dtype != SVDQ_FP16)
    return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: out must be SVDQ_BF16 or SVDQ_FP16", who);
  svdq_status_t st = rows_ok(who, x, x_row, x_dtype);
  if (st != SVDQ_OK) return st;
  if (M == 0) return SVDQ_OK;
  const Fp8Plan p = fp8_plan(M, w->N, w->K);
  if (!x || !out || (!workspace && p.total > 0)) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: NULL pointer", who);
  if (!aligned16(out) || !aligned16(workspace)) return fail(SVDQ_ERR_INVALID_ARGUMENT, "%s: misaligned pointer", who);
  if (ws_bytes < (size_t)p.total)
    return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "%s: workspace needs %lld bytes, got %zu", who, (long long)p.total, ws_bytes);
  st = svdq_device_check();
  if (st != SVDQ_OK) return st;
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  Fp8Args a{};
  a.w = static_cast<const uint8_t *>(w->blob);
  a.x = static_cast<const uint8_t *>(workspace);
  a.ws = a.w + fp8_blocks(w->N, w->K) * kFp8Block;
  a.xs = a.x + fp8_blocks(M, w->K) * kFp8Block;
  a.bias = w->bias;
  a.out = static_cast<uint16_t *>(out);
  a.M = M;
  a.N = w->N;
  a.K = w->K;
  a.blocks_k = (w->K + 127) / 128;
  a.m_blocks = (M + 31) / 32;
  a.n_blocks = (w->N + 31) / 32;
  a.gelu = epilogue == SVDQ_EPILOGUE_GELU_TANH;
  a.rows = static_cast<const uint16_t *>(x);
  a.rows_stride = x_row;
  if (!p.inline_x) {
    launch_quantize(x, x_row, x_dtype, M, w->K, workspace, const_cast<uint8_t *>(a.xs), false, stream);
    st = launch_status("fp8 quantize launch");
    if (st != SVDQ_OK) return st;
  }
  const bool f16 = x_dtype == SVDQ_FP16;
  if (out_dtype == SVDQ_FP16) launch_product<SVDQ_FP16>(p, a, f16, stream);
  else launch_product<SVDQ_BF16>(p, a, f16, stream);
  return launch_status("fp8 product launch");
}

}  // extern "C"
