#pragma once
// Products grouped by expert: where a group's rows are, and which group a row tile
// belongs to, from the offsets in device memory (groups + 1 of them, ascending).
#include "common.cuh"

namespace gb300 {
namespace {

// Rows [lo, lo + n) of group g, within 0 .. rows whatever the offsets hold.
__device__ __forceinline__ void group_span(const int* offsets, int g, int rows, int& lo, int& n) {
  lo = min(max(offsets[g], 0), rows);
  n = min(max(offsets[g + 1], lo), rows) - lo;
}

// One warp looks all offsets over and sets STATUS_BAD_OFFSETS where they do not
// ascend within 0 .. rows.
__device__ __forceinline__ void check_offsets(const int* offsets, int groups, int rows,
                                              unsigned int* status, int lane) {
  bool bad = false;
  for (int g = lane; g < groups; g += 32) {
    const int lo = offsets[g], hi = offsets[g + 1];
    bad |= lo < 0 || hi < lo || hi > rows;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(status, (unsigned int)STATUS_BAD_OFFSETS);
}

// Row tiles of BMT rows, counted group by group: a warp holds 32 groups at a time,
// lane l group g0 + l and the row tiles up to and with it.  Tiles are asked for in
// ascending order, so it never looks back.
template <int BMT>
struct RowTiles {
  int64_t base;  // tiles of the groups before g0
  int g0, lo, n, upto;

  __device__ __forceinline__ void load(const int* offsets, int groups, int rows, int lane) {
    lo = n = 0;
    if (g0 + lane < groups) group_span(offsets, g0 + lane, rows, lo, n);
    upto = (n + BMT - 1) / BMT;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
  }
  __device__ __forceinline__ void init(const int* offsets, int groups, int rows, int lane) {
    base = 0;
    g0 = 0;
    load(offsets, groups, rows, lane);
  }
  // Tile t of `columns` tiles a row tile: its group, that group's rows, and the
  // tile's number within the group.  The whole warp asks; false past the last tile.
  __device__ __forceinline__ bool find(const int* offsets, int groups, int rows, int columns,
                                       int64_t t, int lane, int& g, int& g_lo, int& g_n, int& loc) {
    for (;;) {
      const int64_t here = (int64_t)__shfl_sync(0xffffffffu, upto, 31) * columns;
      if (t < base + here) break;
      base += here;
      if (groups - g0 <= 32) return false;
      g0 += 32;
      load(offsets, groups, rows, lane);
    }
    const int64_t in = t - base;
    const int l = __ffs((int)__ballot_sync(0xffffffffu, (int64_t)upto * columns > in)) - 1;
    g = g0 + l;
    g_lo = __shfl_sync(0xffffffffu, lo, l);
    g_n = __shfl_sync(0xffffffffu, n, l);
    const int rt = (g_n + BMT - 1) / BMT;
    loc = (int)(in - (int64_t)(__shfl_sync(0xffffffffu, upto, l) - rt) * columns);
    return true;
  }
};

}  // namespace
}  // namespace gb300
