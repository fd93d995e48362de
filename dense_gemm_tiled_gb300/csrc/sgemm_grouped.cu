// fp32 products grouped by expert on the CUDA cores: the cp.async kernel of
// sgemm_ffma.cuh with a block a tile, over the groups' rows (raw products, which
// fused_elementwise.cu finishes) or over each group's range of K.  The host does not
// know the groups' sizes, so the grid over rows has a row tile more a group than the
// rows alone need; blocks past the last tile leave at once.  Where tiles are fewer than
// the SMs, K is cut into slices on grid.z, whose raw sums fused_elementwise.cu adds up
// (455 rows of 9 groups, 258 x 1332: 146 us whole; a K step of 64 is 2 us of a tile).
#include "sgemm_ffma.cuh"

namespace gb300 {

int sgemm_grouped_splits(const FusedArgs& a) {
  using TL = TileWide;
  const bool inner = a.kind == FUSED_INNER;
  const int64_t live = inner ? a.groups : (a.groups < a.M ? a.groups : a.M);
  const int64_t per = inner ? a.M : ((int64_t)a.M + live - 1) / live;
  const int64_t tiles = live * ((per + TL::BM - 1) / TL::BM) * (((int64_t)a.N + TL::BN - 1) / TL::BN);
  const int64_t k = inner ? ((int64_t)a.K + a.groups - 1) / a.groups : a.K;
  const int64_t steps = (k + TL::BK - 1) / TL::BK;
  int64_t s = a.num_sms / (tiles > 0 ? tiles : 1);
  if (s > FUSED_MAX_SPLITS_F32) s = FUSED_MAX_SPLITS_F32;
  if (s > steps) s = steps;
  return s > 1 ? (int)s : 1;
}

cudaError_t launch_sgemm_grouped(const FusedArgs& a, float* P, int64_t ldp, LaunchCtx& ctx) {
  using TL = TileWide;
  const bool inner = a.kind == FUSED_INNER;
  Params p = {};
  p.A = static_cast<const float*>(a.A);
  p.B = static_cast<const float*>(a.B);
  const bool direct = inner && a.splits == 1;  // (else raw sums)
  p.C = direct ? static_cast<float*>(a.Y) : P;
  p.lda = a.lda;
  p.ldb = a.ldb;
  p.ldc = direct ? a.ldy : ldp;
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.k_slice = ((a.K + TL::BK - 1) / TL::BK + a.splits - 1) / a.splits * TL::BK;
  p.stride_z = (int64_t)a.M * (inner ? a.groups : 1) * ldp;
  p.tiles_m = (a.M + TL::BM - 1) / TL::BM;
  p.tiles_n = (a.N + TL::BN - 1) / TL::BN;
  p.group_m = p.tiles_m < 8 ? (p.tiles_m > 0 ? p.tiles_m : 1) : 8;
  p.alpha = direct ? a.alpha : 1.f;
  p.beta = direct ? a.beta : 0.f;
  p.stride_b = inner ? 0 : a.stride_b;
  p.stride_c = direct ? a.stride_y : inner ? (int64_t)a.M * ldp : 0;
  p.offsets = a.offsets;
  p.groups = a.groups;
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  auto aligned = [](const void* q, int64_t ld) { return ((uintptr_t)q & 15u) == 0 && ld % 4 == 0; };
  const bool vec = aligned(a.A, a.lda) && aligned(a.B, a.ldb) && p.stride_b % 4 == 0;
  p.c_vec = aligned(p.C, p.ldc) && p.stride_c % 4 == 0;
  const int64_t tiles = inner ? (int64_t)p.tiles_m * p.tiles_n
                              : ((int64_t)p.tiles_m + (a.groups < a.M ? a.groups : a.M)) * p.tiles_n;
  if (tiles >= (1ll << 31) || a.groups > 65535) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)tiles, inner ? (unsigned)a.groups : 1u, (unsigned)a.splits);
  cudaError_t e;
  if (inner)
    e = vec ? launch_one<TL, false, false, true, KIND_INNER>(p, grid, ctx.stream)
            : launch_one<TL, false, false, false, KIND_INNER>(p, grid, ctx.stream);
  else if (a.transB)
    e = vec ? launch_one<TL, true, true, true, KIND_ROWS>(p, grid, ctx.stream)
            : launch_one<TL, true, true, false, KIND_ROWS>(p, grid, ctx.stream);
  else
    e = vec ? launch_one<TL, true, false, true, KIND_ROWS>(p, grid, ctx.stream)
            : launch_one<TL, true, false, false, KIND_ROWS>(p, grid, ctx.stream);
  ctx.grid = (int)(grid.x * grid.y * grid.z);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

}  // namespace gb300
