#pragma once
// The choice of a 16-bit fused or grouped product's tile and slices of K (host code alone).
#include <stdlib.h>

#include "internal.h"

namespace gb300 {

inline void fused_plan(FusedArgs& a) {
  // The tile and slices of K with the least estimated time, in ns: rounds of units over
  // the GPU x the greater of the main loop -- K steps x what one takes, 330 ns on pairs of
  // 256 x 256, else the bytes that it brings into a block's shared memory at 126 a ns --
  // and the epilogue, which runs under the next unit's main loop; + start and the last
  // epilogue; and with slices their sums' way through memory and a second kernel.
  // Measured, us: 512 x 5632 x 2048 pairs 17.7, 128 x 128 22.3, 128 x 64 28.5; 512 x 2048 x
  // 5632 (residual) pairs 33.6, in four slices 22.4, 128 x 128 28.4, in two 21.8.  Where
  // one row of tiles takes all rows, each column of B comes from memory once, and a step
  // takes at least its bytes' share of 6.6 TB/s, and as long as the ring's bytes of B take
  // at 2.2 us from request to arrival (32 rows of 64 groups, 24 with rows, 1408 x 2048: 128
  // x 128 30.6, 128 x 64 41.0, 128 x 192 36.8, pairs 35.5).  The host does not know the
  // groups' sizes: rows spread evenly over groups.
  const struct { int bm, bn, slots, fixed, epilogue, stages; } shape[FUSED_TILES] = {
      {256, 256, a.num_sms / 2, 6000, 2500, 5}, {128, 192, a.num_sms, 5500, 2000, 4},
      {128, 128, a.num_sms, 5000, 1500, 6}, {128, 64, a.num_sms, 5000, 1000, 8}};
  static const int forced = [] {
    const char* e = getenv("GEMM_GB300_FUSED_TILE");
    return e ? atoi(e) : -1;
  }();
  static const int forced_splits = [] {
    const char* e = getenv("GEMM_GB300_FUSED_SPLITS");
    return e ? atoi(e) : 0;
  }();
  const bool rows = a.kind == FUSED_ROWS, inner = a.kind == FUSED_INNER;
  int64_t live = 1;  // groups with rows, if these are spread evenly (one where there are none)
  if (rows && a.M > 0) live = a.groups < a.M ? a.groups : a.M;
  const int64_t per = ((int64_t)a.M + live - 1) / live;
  const int64_t kk = inner ? ((int64_t)a.K + a.groups - 1) / a.groups : a.K;
  const int64_t steps = (kk + 63) / 64;
  const bool a_rows = !a.transA && !inner;
  double least = 0;
  a.tile = -1;
  a.splits = 1;
  for (int i = 0; i < FUSED_TILES; ++i) {
    if (forced >= 0 && forced < FUSED_TILES && i != forced) continue;
    const int64_t tm = (per + shape[i].bm - 1) / shape[i].bm;
    const int64_t tiles = live * tm * (((int64_t)a.N + shape[i].bn - 1) / shape[i].bn) *
                          (inner ? a.groups : 1);
    // bytes of a step: rows of A in boxes of 32, B's columns (half of them a block of a pair)
    const int64_t rows_in = a_rows && per < 128 ? (per + 31) / 32 * 32 : 128;
    const double ns = i == FUSED_TILE_PAIR ? 330.0 : (double)(rows_in + shape[i].bn) * 128 / 126;
    for (int s = 1; s <= FUSED_MAX_SPLITS; ++s) {
      const int64_t each = (steps + s - 1) / s;
      if (s > 1 && (a.kind != FUSED_DENSE || (s - 1) * each >= steps || each < 4)) continue;
      if (forced_splits > 0 && a.kind == FUSED_DENSE && s != forced_splits && (s > 1 || steps >= 4 * forced_splits))
        continue;
      const int64_t rounds = (tiles * s + shape[i].slots - 1) / shape[i].slots;
      double step = ns;
      if (!inner && tm == 1) {
        const int blocks = i == FUSED_TILE_PAIR ? 2 : 1;  // of a unit, each with bn / blocks columns
        const int64_t units = tiles * s < shape[i].slots ? tiles * s : shape[i].slots;
        const double bytes = (double)shape[i].bn / blocks * 128;
        const double share = bytes * (double)(units * blocks) / 6600, wait = 2200.0 / shape[i].stages;
        step = step > share ? step : share;
        step = step > wait ? step : wait;
      }
      const double loop = (double)each * step, epi = (double)shape[i].epilogue;
      double cost = (double)rounds * (loop > epi ? loop : epi) + shape[i].fixed;
      if (s > 1) cost += 2500 + (double)a.M * a.N * 8 * s / 6000;
      if (a.tile < 0 || cost < least) {
        least = cost;
        a.tile = i;
        a.splits = s;
      }
    }
  }
  if (a.tile < 0) a.tile = forced >= 0 && forced < FUSED_TILES ? forced : FUSED_TILE_128;
}

}  // namespace gb300
