// Limits and the workspace of the expert layer, shared by the host's size
// queries and the device side.
#pragma once

#include <stdint.h>

#include "layout.h"

#define MOE_MAX_EXPERTS 1024

namespace svdq {

constexpr int kMoeMaxTopK = 32;
constexpr int kMoeMaxPairs = 4096;     // tokens times choices of one call

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

// (token, choice) pairs sorted by expert: the experts that have any, where
// their pairs begin (and, after the last, end), and the pairs
struct MoePlan {
  int slots, expert[MOE_MAX_EXPERTS], first[MOE_MAX_EXPERTS + 1];
  uint16_t pairs[kMoeMaxPairs];
};

// the gated products h as two bf16 pieces, each pair's output row, the plan
struct MoeWork {
  int64_t h_hi = 0, h_lo = 0, part = 0, plan = 0, total = 0;
  constexpr MoeWork(int64_t T, int64_t top_k, int64_t K, int64_t I) {
    const int64_t n = T * top_k;
    int64_t o = 0;
    h_hi = o;  o = round_up(o + n * I * 2, kAlign);
    h_lo = o;  o = round_up(o + n * I * 2, kAlign);
    part = o;  o = round_up(o + n * K * 4, kAlign);
    plan = o;  o = round_up(o + (n > 64 ? (int64_t)sizeof(MoePlan) : 0), kAlign);
    total = o;
  }
};

}  // namespace svdq
