// Layout and limits of the MXFP4 key/value cache, shared by the host's size
// queries and the device kernels (kv4.hip describes a unit's bytes).
#pragma once

#include <stdint.h>

namespace svdq {

// Wavefronts a SIMD (workgroups a CU) that the attention kernel is built for,
// by head_dim and rows: what its registers allow.  At D = 128 with up to 8 rows
// 524k tokens of 8 heads take 74.0, 73.8 and 85.8 us with 2, 3 and 4 (128 registers,
// some of them spilled), 48 ragged sequences 27.1, 26.0 and 31.8; at D = 64, 3 and 4
// are alike; at D = 256 with 8 rows 16 x 16000 tokens of 8 heads take 106 us with 1
// and 101 with 2, with 32 rows 16 x 4000 tokens 57 and 71.
constexpr int kv4_waves(int D, int rows) {
  return D == 64 ? (rows <= 16 ? 4 : 2) : D == 128 ? (rows <= 16 ? 3 : 2) : rows <= 16 ? 2 : 1;
}
// Workgroups of an attention call at most (256 CUs), which sizes its workspace.
constexpr int kKv4Groups = 256 * 4;
// Tokens that a workgroup takes at a time, and the cost of beginning and ending
// a (sequence, head), in such chunks (with 1, 2, 3 and 4, 48 ragged sequences
// take 28.2, 26.0, 26.5 and 26.5 us, 16 sequences of 5 new tokens 15.6, 14.9,
// 15.5 and 15.4).
constexpr int kKv4Chunk = 128;
constexpr int kKv4Start = 2;
// Tokens that a row of a page table names at most: token numbers, and those up to two
// chunks on, are 32-bit integers.
constexpr int64_t kKv4MaxTokens = (int64_t)1 << 30;
// Rows (new tokens times query heads of one key/value head) at most.
constexpr int kKv4MaxRows = 1024;

constexpr bool kv4_shape_ok(int64_t pages, int page_size, int H, int D) {
  return pages >= 1 && page_size >= 16 && page_size <= 256 && (page_size & (page_size - 1)) == 0 && H >= 1 &&
         H <= 1024 && (D == 64 || D == 128 || D == 256) && pages * page_size <= 0x7FFFFFFF;
}
constexpr bool kv4_query_ok(int64_t B, int64_t Q, int64_t Hq, int64_t H) {
  return B >= 0 && B <= 65536 && Q >= 1 && Hq >= 1 && Hq % H == 0 && Q * (Hq / H) <= kKv4MaxRows &&
         B * Q * Hq <= (1 << 24);
}

// bytes of an attention call's workspace: two running states for each workgroup
constexpr int64_t kv4_workspace_bytes(int64_t Q, int64_t Hq, int64_t H, int64_t D) {
  const int64_t rows = Q * (Hq / H), block = rows < 32 ? rows : 32;
  return 2 * (int64_t)kKv4Groups * block * (D + 2) * 4;
}

struct Kv4Layout {
  int pages = 0, page_shift = 0, H = 0, D = 0;
  constexpr Kv4Layout() = default;
  constexpr Kv4Layout(int pages_, int page_size_, int H_, int D_) : pages(pages_), H(H_), D(D_) {
    for (page_shift = 4; (1 << page_shift) < page_size_;) ++page_shift;
  }
  constexpr int page_size() const { return 1 << page_shift; }
  constexpr int64_t unit_bytes() const { return 17 * (int64_t)D; }
  // byte offset of unit u (16 tokens) of head h in a page
  constexpr int64_t unit(int64_t page, int h, int u) const {
    return (((page * H + h) << (page_shift - 4)) + u) * unit_bytes();
  }
  constexpr int v_codes() const { return 8 * D; }
  constexpr int k_scales() const { return 16 * D; }
  constexpr int v_scales() const { return 16 * D + D / 2; }
  constexpr int64_t total() const { return unit(pages, 0, 0); }
};

}  // namespace svdq
