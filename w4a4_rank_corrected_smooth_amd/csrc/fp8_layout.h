// Layout, limits and workspace of the 8-bit floating point linear, shared by the
// host's size queries and the device kernels.
#pragma once

#include <stdint.h>

namespace svdq {

// Codes are kept in blocks of 32 rows (of X, or of W: output channels) by 128
// channels, 4096 bytes in the order of the matrix operand: channel c of row r is byte c
// % 16 of unit q = c / 16, and unit q of row r stands at
//   (q / 2) 1024 + (q % 2) 512 + 16 r,
// so that lane l = 32 (q % 2) + r of a wavefront reads its two 32-byte operands of
// a 32x32x64 instruction as four contiguous kilobytes.  The blocks of 32 rows follow each
// other along K.  Rows and channels past the end are zeros in W; X's channels too, and its rows
// are never looked at.  Behind all codes stand the scales, in the blocks' order: X's as 32
// bytes E8M0 a block, one a row; W's as m 2^(e - 127) of the 128 x 128 block, m
// float32 and e an int32.
constexpr int kFp8Block = 4096;
constexpr int kFp8XScales = 32, kFp8WScales = 8;    // bytes a block

constexpr bool fp8_weights_ok(int64_t N, int64_t K) {
  return N >= 1 && N <= (1 << 20) && K >= 8 && K <= (1 << 20) && K % 8 == 0 && N * K <= (int64_t)1 << 33;
}
constexpr bool fp8_call_ok(int64_t M, int64_t N) { return M >= 0 && M <= (1 << 22) && M * N <= (int64_t)1 << 34; }

constexpr int64_t fp8_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
constexpr int64_t fp8_blocks(int64_t rows, int64_t K) { return fp8_up(rows, 32) / 32 * (fp8_up(K, 128) / 128); }
constexpr int64_t fp8_w_bytes(int64_t N, int64_t K) { return fp8_blocks(N, K) * (kFp8Block + kFp8WScales); }
constexpr int64_t fp8_x_bytes(int64_t M, int64_t K) { return fp8_up(fp8_blocks(M, K) * (kFp8Block + kFp8XScales), 256); }

// Which kernel multiplies: few rows, or tiles of 64, 128 or 256 rows and channels, or of 192 rows by 128.
// No form cuts K over workgroups, so few channels or few tiles of a long K leave CUs idle (6144 x 4096 with 128 rows 15.2 us, 256 19.5,
// 512 23, 1024 38, 2048 61; 128 x 512 x 8192, 16 tiles, 22.6; 4608 x 64 x 8192, 72 tiles, 44).
// FP8_128_DEEP: four stages of the tiles in LDS, a workgroup to a CU, where FP8_128 has two and two.
enum Fp8Form { FP8_FEW, FP8_ROWS, FP8_64, FP8_128_DEEP, FP8_192, FP8_128, FP8_256 };
struct Fp8Plan {
  Fp8Form form = FP8_ROWS;
  bool inline_x = false;       // FP8_FEW, FP8_ROWS: each workgroup quantises the rows for itself
  int x_blocks = 1;            // FP8_ROWS: blocks of 32 rows
  int64_t total = 0;           // bytes of workspace: the rows' blocks
};

inline Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K) {
  Fp8Plan p;
  const int64_t kb = (K + 127) / 128;
  if (M <= 32) {
    // up to 24576 values each workgroup quantises the rows itself (rows of 4096, both ways: 1: 7.1 and 9.5 us, 4: 9.4
    // and 10.0, 6: 9.8 and 10.1, 8: 10.6 and 10.3)
    p.inline_x = M * kb * 128 <= 24576;
    // 16 channels to a workgroup where that makes no more than one round of them (one row of 4096 x 14336: 15.3 us, by 32
    // channels 17.5; of 1152 x 4608: 6.0 and 6.6; of 6144 x 4096: 9.1 and 7.1)
    if (M <= 16 && N <= 4096) p.form = FP8_FEW;
  } else if (M <= 64 || (M <= 96 && N <= 8192)) {
    // a round of workgroups of 32 channels (96 x 6144 x 4096 14.6 us, in 64 x 64 tiles 16.2; at 128 rows 16.4 and 16.0, at
    // 128 x 16384 x 4096 30 and 25)
    p.x_blocks = (int)((M + 31) / 32);
  } else {
    const int64_t t128 = (M + 127) / 128 * ((N + 127) / 128), t256 = (M + 255) / 256 * ((N + 255) / 256);
    // Tiles of 256 x 256, a workgroup to a CU, take 1.4 times as long a round as tiles of 128 x 128 two to a CU
    // (4096 x 4096 x 4096: 74 us in 1 round, 85 in 2; 2048 x 6144 x 4096: 64 and 70; 4096 x 2048 x 8192: 106 and 87).
    // Those keep four stages, one to a CU, where that makes one round (1024 x 4096 x 4096: 28.4 us, two stages 32.4,
    // 64 x 64 tiles 41; 4095 x 1152 x 4608, 288 tiles: 49, 45 and 53), and are 192 high where that makes one round of them
    // (twelve wavefronts, three stages; 4095 x 1152 x 4608: 45.6, two of 128 to a CU 48.3; 2304 x 2048 x 4096: 35.7 and
    // 40.0; 160 or 256 high, and other shares of the wavefronts, were no better).  Tiles of 64 x 64 fill the CUs where
    // those do not (256 x 6144 x 4096, 96 tiles: 20.3 us, 128 x 128 21.6).
    const int64_t t192 = (M + 191) / 192 * ((N + 127) / 128);
    p.form = (t256 + 255) / 256 * 5120 <= 7 * t128 ? FP8_256 : t128 < 128 ? FP8_64 : t128 <= 256 ? FP8_128_DEEP
             : t192 <= 256 ? FP8_192 : FP8_128;
  }
  p.total = p.inline_x ? 0 : fp8_x_bytes(M, K);
  return p;
}

}  // namespace svdq
