// Limits, forms and workspace of the cross attention, shared by the host's size
// query and the device kernels.
#pragma once

#include <stdint.h>

namespace svdq {

constexpr bool cross_shape_ok(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t D) {
  return B >= 0 && B <= 65536 && Lq >= 0 && Lk >= 0 && Lk <= (1 << 30) && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && D >= 8 &&
         D <= 256 && D % 8 == 0 && B * Hkv <= (1 << 20) && Lq * Hq <= (1 << 28) && B * (Lq * Hq) <= (1 << 28);
}

// States of a batch row that a workgroup lists for itself, in LDS, where there is a
// mask; longer rows are listed by a kernel of their own.
constexpr int kCrossOwnList = 2048;

// States that the form that keeps them all in LDS is built for, by blocks of 32 channels: what fits there, 64 at a
// time, beside their list.
constexpr int cross_near_states(int blocks) { return blocks == 2 ? 576 : blocks == 3 ? 384 : blocks == 4 ? 256 : 0; }

// How a call is cut up.  Rows: the Lq queries of the g heads that share a key/value head.
struct CrossPlan {
  int64_t rows = 0;       // of a (batch row, key/value head)
  int blocks = 0;         // blocks of 32 channels that the kernel is built for
  bool near = false;      // all states in LDS, many rows
  bool own = false;       // each wavefront has states of its own (few rows), not rows of its own
  bool wide = false;      // own: eight wavefronts, not four
  int least = 1;          // tiles of a part, for that the parts' sums are not most of the work
  int tile_keys = 0;      // states that a workgroup (own: a wavefront) takes at a time
  int64_t tiles = 0;      // workgroups that share the rows of a (batch row, key/value head)
  int parts = 1;          // pieces that the states are cut into, over workgroups; or, where the lengths differ,
  int line = 0;           // pieces of all batch rows, shared out by their lengths (0: `parts` each)
  int64_t index_off = 0, count_off = 0, ml_off = 0, rest_off = 0, o_off = 0, total = 0;
};

constexpr int64_t cross_up(int64_t x) { return (x + 255) / 256 * 256; }

inline CrossPlan cross_plan(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t D, bool masked) {
  CrossPlan p;
  p.rows = Lq * (Hq / Hkv);
  p.blocks = D <= 64 ? 2 : D <= 96 ? 3 : D <= 128 ? 4 : D <= 160 ? 5 : 8;
  p.own = p.rows <= 32 && p.blocks <= 4;    // wider states: four pairs of tiles are more than the LDS
  p.tile_keys = p.own || p.blocks > 4 ? 32 : 64;
  p.least = p.own ? 4 : 6;
  const int64_t heads = B * Hkv, blocks32 = (p.rows + 31) / 32;
  p.near = !p.own && Lk <= cross_near_states(p.blocks) && heads * blocks32 >= 8 * 256;
  if (p.near) {
    // a workgroup to a CU, eight blocks of 32 rows to each at least (a number of heads that is no part of 256 leaves CUs
    // idle: 8 x 4096 rows over 77 states of 64 channels take 78 us for 20 heads, 160 workgroups, and 88 for 32, 256)
    p.tiles = heads < 256 ? 256 / heads : 1;
    if (p.tiles > (blocks32 + 7) / 8) p.tiles = (blocks32 + 7) / 8;
  } else {
    p.tiles = p.own ? 1 : (p.rows + 127) / 128;
  }
  const int64_t work = heads * p.tiles;
  const int64_t key_tiles = (Lk + p.tile_keys - 1) / p.tile_keys;
  // The states in parts where there is less work than places for workgroups (one to a CU where
  // the form for few rows needs most of the LDS, two elsewhere): as many as fit in one round, of `least` tiles
  // (many rows: 256 over 1500 states, 16 heads of 64, with 4, 6, 8 and 12 take 14.7, 15.3, 17.1 and 19.4 us, 512 over 4096, 8
  // heads of 64, 22.9, 21.4, 19.2 and 21.8; 256 rows over 15804 states of 6 batch rows 33.4, 32.5, 32.3 and 41.8).
  // Few rows of 64 channels or less: eight wavefronts, and no join, where a workgroup to a head nearly fills the CUs
  // (160 heads over 1500 states 15.1 us, two workgroups of four to a CU and a join 16.7; 240 18.6 and 21.5, with a mask
  // 21.5 and 24.5; 256 over 448 7.5 and 11.0; but 80 over 1500 11.9 and 11.4, 320 28.8 and 25.3).  Longer states are
  // shared out by their lengths.  From a round of workgroups on states are whole, also where the last round is part
  // empty (over 16384 states of 128 channels: 4096 rows of 16 heads, 512 workgroups, 520 us; 4500 rows, 576, 762;
  // 4608 of 24 heads, 864, 973).
  p.wide = p.own && p.blocks == 2 && work > 128 && work <= 256 && Lk <= 2048;
  const int64_t places = p.wide || (p.own && p.blocks > 2) ? 256 : 512;
  if (!p.near && work > 0 && work < places) {
    const int64_t want = places / work, most = key_tiles / p.least;
    p.parts = (int)(want < most ? want : most);
    if (p.parts < 1) p.parts = 1;
    // up to 64 batch rows, with two pieces each on average
    const int64_t line = places / (Hkv * p.tiles);
    if (B > 1 && B <= 64 && most > 1 && line >= 2 * B) p.line = (int)(line < B * most ? line : B * most);
  }
  const bool lists = masked && Lk > kCrossOwnList;
  p.count_off = lists ? cross_up(4 * B * Lk) : 0;
  const int64_t even = p.parts > 1 ? p.parts * heads : 0, shared = p.line ? (p.line + B) * Hkv : 0, pieces = even > shared ? even : shared;
  p.ml_off = p.count_off + (lists ? cross_up(4 * B) : 0);
  p.rest_off = p.ml_off + (pieces > 0 ? cross_up(8 * pieces * p.rows) : 0);
  p.o_off = p.rest_off + (pieces > 0 ? cross_up(4 * pieces * p.rows) : 0);
  p.total = p.o_off + (pieces > 0 ? cross_up(4 * pieces * p.rows * D) : 0);
  return p;
}

}  // namespace svdq
