// The converted product (mx_mixed.cuh) for fp16, and its plan.
#include <stdlib.h>

#include "mx_mixed.cuh"

namespace gb300 {

// Rows of C a tile covers, and as many slices of K as leave every cluster
// resident (an SM a block; at most 6: clusters of 8 leave too many SMs of a GPC
// over, 33 x 2048 x 2048 14.0 us with 8, 7.8 with 6, 8.0 with 4); and whether that is estimated to take less time than expanding the operand
// and multiplying with the 16-bit kernel: rounds of blocks x stages x 0.4 us
// against the operand's bytes (read, written, read: 5 a value) and the products
// at 1.5 PFLOP/s.  Measured, us, converted against expanded, fp4 (nt but where
// said):  33 x 2048 x 2048 8.0 / 16.1;  64 x 8192 x 8192 33 / 61;  128 x 8192 x
// 8192 32 / 61;  256 x 8192 x 8192 56 / 73;  nn 1 x 8192 x 8192 28 / 64;  nn 512 x
// 2048 x 5632 24 / 25;  512 x 5632 x 2048 34 / 20;  1000 x 3000 x 777 24 / 15;
// 4096^3 205 / 86.
MixedPlan mixed_plan(int M, int N, int K, int num_sms) {
  static const int forced = [] {
    const char* e = getenv("GEMM_GB300_MX_MIXED");
    return e ? atoi(e) : -1;
  }();
  const int64_t steps = ((int64_t)K + 63) / 64;
  MixedPlan pl;
  pl.mt = M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const int64_t tiles = ((int64_t)N + 127) / 128 * (((int64_t)M + pl.mt - 1) / pl.mt);
  int64_t s = forced > 0 ? forced : (int64_t)num_sms * 7 / 8 / (tiles > 0 ? tiles : 1);
  s = forced > 0 ? (s < 8 ? s : 8) : s < 6 ? s : 6;
  s = s < steps ? s : steps;
  s = s > 1 ? s : 1;
  pl.splits = (int)s;
  const int64_t rounds = (tiles * s + num_sms - 1) / num_sms;
  const double convert = 6 + 0.4 * (double)rounds * (double)((steps + s - 1) / s);
  const double nk = (double)N * K;
  const double expand = 8 + 5 * nk / 6.8e6 + 2 * nk * M / 1.5e9;
  pl.convert = forced == 0 ? false : forced > 0 || convert < expand;
  return pl;
}

bool mx_mixed_takes(int format, int transA, int transB, int M, int N, int K, int num_sms) {
  if (format == MX_INT8 ? !(transA && !transB) : transA != 0) return false;
  const MixedPlan pl = mixed_plan(M, N, K, num_sms);
  const int64_t tiles = ((int64_t)M + pl.mt - 1) / pl.mt * (((int64_t)N + 127) / 128);
  return pl.convert && tiles <= 65535;
}

cudaError_t launch_mx_mixed_f16(const MxStreamArgs& a, LaunchCtx& ctx) {
  return launch_mixed_t<__half>(a, ctx);
}

cudaError_t launch_mx_mixed(const MxStreamArgs& a, LaunchCtx& ctx) {
  return a.out == 1 ? launch_mx_mixed_f16(a, ctx) : launch_mx_mixed_bf16(a, ctx);
}

}  // namespace gb300
