// The converted product (mx_mixed.cuh) for fp16, and its plan.
#include <stdlib.h>

#include "mx_mixed.cuh"

namespace gb300 {

// Form of a converted product: the one with the least estimated time, in units
// of a stage's loads: rounds of tiles x (stages of a block + what a tile costs
// beside them).
MixedPlan mixed_plan(int M, int N, int K, int num_sms) {
  static const int forced = [] {
    const char* e = getenv("GEMM_GB300_MX_MIXED");
    return e ? atoi(e) : -1;
  }();
  const int64_t steps = ((int64_t)K + 63) / 64;
  const int64_t n128 = ((int64_t)N + 127) / 128;
  MixedPlan pl;
  pl.mt = M <= 32 ? 32 : M <= 64 ? 64 : 128;
  // single: as many slices of K as leave every cluster resident (an SM a block;
  // clusters of up to 8 leave some SMs of a GPC over)
  const int64_t tiles = n128 * (((int64_t)M + pl.mt - 1) / pl.mt);
  int64_t s = tiles > 0 ? (int64_t)num_sms * 7 / 8 / tiles : 1;
  if (s > 8) s = 8;
  if (s > steps) s = steps;
  if (s < 1) s = 1;
  pl.splits = (int)s;
  const int64_t rounds1 = (tiles * s + num_sms - 1) / num_sms;
  const double t1 = (double)rounds1 * ((double)((steps + s - 1) / s) + (s > 1 ? 14 : 10));
  const int64_t pairs = ((N + 255) / 256) * (int64_t)(((int64_t)M + 255) / 256);
  const int64_t rounds2 = (pairs + num_sms / 2 - 1) / (num_sms / 2);
  const double t2 = (double)rounds2 * (double)steps * 1.05 + 20;
  pl.pair = M > 128 && t2 < t1;
  if (forced == 0) pl.pair = true;
  if (forced > 0) {
    pl.pair = false;
    pl.splits = forced < 8 ? forced : 8;
  }
  return pl;
}

cudaError_t launch_mx_mixed_f16(const MxStreamArgs& a, LaunchCtx& ctx) {
  return launch_mixed_t<__half>(a, ctx);
}

cudaError_t launch_mx_mixed(const MxStreamArgs& a, LaunchCtx& ctx) {
  return a.out == 1 ? launch_mx_mixed_f16(a, ctx) : launch_mx_mixed_bf16(a, ctx);
}

}  // namespace gb300
