// fp16 instantiation of the fused and grouped products (fused_tcgen05.cuh), and the
// choice of their tile.
#include <stdlib.h>

#include "fused_tcgen05.cuh"

namespace gb300 {

int fused_pick(const FusedArgs& a) {
  static const int forced = [] {
    const char* e = getenv("GEMM_GB300_FUSED_TILE");
    return e ? atoi(e) : -1;
  }();
  if (forced >= 0 && forced < FUSED_TILES) return forced;
  // The tile with the least estimated time: rounds of tiles over the GPU x (K steps x
  // the bytes a block moves for one + a tile's start and epilogue, as bytes).  The
  // host does not know the groups' sizes: rows spread evenly over groups.
  const struct { int bm, bn, slots, kib, fixed; } shape[FUSED_TILES] = {
      {256, 256, a.num_sms / 2, 40, 160}, {128, 128, a.num_sms, 32, 100}, {128, 64, a.num_sms, 24, 80}};
  const bool rows = a.kind == FUSED_ROWS, inner = a.kind == FUSED_INNER;
  const int64_t live = rows ? (a.groups < a.M ? a.groups : a.M) : 1;
  const int64_t per = ((int64_t)a.M + live - 1) / live;
  const int64_t kk = inner ? ((int64_t)a.K + a.groups - 1) / a.groups : a.K;
  const int64_t steps = (kk + 63) / 64;
  int best = 0;
  double least = 0;
  for (int i = 0; i < FUSED_TILES; ++i) {
    const int64_t tiles = live * ((per + shape[i].bm - 1) / shape[i].bm) *
                          (((int64_t)a.N + shape[i].bn - 1) / shape[i].bn) *
                          (inner ? a.groups : 1);
    const int64_t rounds = (tiles + shape[i].slots - 1) / shape[i].slots;
    const double cost = (double)rounds * ((double)steps * shape[i].kib + shape[i].fixed);
    if (i == 0 || cost < least) {
      least = cost;
      best = i;
    }
  }
  return best;
}

cudaError_t launch_fused(const FusedArgs& a, LaunchCtx& ctx) {
  return a.dtype == 2 ? launch_fused_bf16(a, ctx) : launch_fused_t<__half>(a, ctx);
}

}  // namespace gb300
