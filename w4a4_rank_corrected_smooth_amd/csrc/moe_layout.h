// Limits and the workspace of the expert layer, shared by the host's size
// queries and the device side.
#pragma once

#include <stdint.h>

#include "layout.h"

#define MOE_MAX_EXPERTS 1024

namespace svdq {

constexpr int kMoeMaxTopK = 32;
constexpr int kMoeMaxPairs = 4096;     // tokens times choices of one call

constexpr int kMoeFewPairs = 16;       // the form for a handful of pairs
constexpr bool moe_route_ok(int64_t T, int E, int K, int top_k) {
  return T >= 0 && E >= 1 && E <= MOE_MAX_EXPERTS && K >= 8 && K % 8 == 0 && K <= (1 << 20) && top_k >= 1 &&
         top_k <= E && top_k <= kMoeMaxTopK && T <= 65535;
}
constexpr bool moe_weights_ok(int E, int K, int I) {
  return E >= 1 && E <= MOE_MAX_EXPERTS && K >= 64 && K % kGroup == 0 && I >= 64 && I % kGroup == 0 &&
         (int64_t)2 * I * K <= (int64_t)1 << 31;
}
constexpr bool moe_call_ok(int64_t T, int top_k) {
  return T >= 0 && top_k >= 1 && top_k <= kMoeMaxTopK && T * top_k <= kMoeMaxPairs;
}

// Weights of one expert's linear [N, K], N a multiple of 16: for each tile of
// 16 output channels and each step (pair of groups of 64 input channels), the
// 1024 code bytes of an AWQ block (layout.h) and then, for each of the 16
// channels, its two groups' scale words (fp16 scale | fp16 zero << 16), so
// that a step's weights are one contiguous piece.  (With the scales in an
// array of their own, as in the linear layer's blob, their loads touched 16
// lines for 128 bytes, and the gate and up products of 128 tokens took 77 us
// against 51 without them.)  The second group of an odd last step is zero.
constexpr int kMoeBlockBytes = kAwqBlockBytes + kAwqTile * 8;
struct MoeWeightLayout {
  int64_t N = 0, K = 0, G = 0, P = 0, total = 0;
  constexpr MoeWeightLayout(int64_t N_, int64_t K_) : N(N_), K(K_), G(K_ / kGroup), P((K_ / kGroup + 1) / 2) {
    total = N / kAwqTile * P * kMoeBlockBytes;
  }
  constexpr int64_t block(int64_t tile, int64_t step) const { return (tile * P + step) * kMoeBlockBytes; }
};

// (token, choice) pairs sorted by expert: the experts that have any, where
// their pairs begin (and, after the last, end), and the pairs
struct MoePlan {
  int slots, expert[MOE_MAX_EXPERTS], first[MOE_MAX_EXPERTS + 1];
  uint16_t pairs[kMoeMaxPairs];
};

// the gated products h as two bf16 pieces, each pair's output row, the plan
struct MoeWork {
  int64_t h = 0, part = 0, plan = 0, total = 0;
  constexpr MoeWork(int64_t T, int64_t top_k, int64_t K, int64_t I) {
    const int64_t n = T * top_k;
    int64_t o = 0;
    h = o;     o = round_up(o + n * I * 4, kAlign);
    part = o;  o = round_up(o + n * K * 4, kAlign);
    plan = o;  o = round_up(o + (int64_t)sizeof(MoePlan), kAlign);
    total = o;
  }
};

}  // namespace svdq
