// What fused products do outside their main kernel: the epilogue of fp32 products
// (bias, activation or its slope, residual, column sums, over raw sums in memory),
// and the join of the column sums of either type.
//
// fp32 products spend 2 K / 72 ps a value on the CUDA cores (K = 2048: 57 ps); a pass
// over the values in memory costs 2 to 4 ps, so it is not worth an epilogue of its
// own in each of their five kernels.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gelu.cuh"
#include "groups.cuh"
#include "internal.h"

namespace gb300 {
namespace {

struct FinishParams {
  int M, N, groups;
  const int* offsets;  // null: one group of all rows
  const float* P;
  int64_t ldp;
  float alpha, beta;
  const float* bias;
  int act, mode;
  const float* in;
  int64_t ld_in;
  float* U;
  int64_t ldu;
  float* Y;
  int64_t ldy;
  float* part;
  int chunks;  // of 256 columns
  int64_t units;
};

// A slot of 32 rows (group g's begin at o[g] / 32 + g) x 256 columns a block, a
// column a thread.
__global__ void __launch_bounds__(256) fused_finish_kernel(const FinishParams p) {
  pdl_wait();
  pdl_trigger();
  for (int64_t unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
    const int slot = (int)(unit / p.chunks);
    const int n = (int)(unit - (int64_t)slot * p.chunks) * 256 + (int)threadIdx.x;
    int g = 0, lo = 0, len = p.M;
    if (p.offsets) {
      // the last group whose first slot is not past this one
      int a = 0, b = p.groups - 1;
      while (a < b) {
        const int m = a + (b - a + 1) / 2;
        group_span(p.offsets, m, p.M, lo, len);
        if ((lo >> 5) + m <= slot) a = m;
        else b = m - 1;
      }
      g = a;
      group_span(p.offsets, g, p.M, lo, len);
    }
    const int r0 = (slot - (lo >> 5) - g) * 32;
    const int rows = r0 < 0 ? 0 : min(32, len - r0);
    if (rows <= 0 || n >= p.N) continue;
    const int64_t m0 = (int64_t)lo + r0;
    const float bias = p.bias ? __ldg(p.bias + (int64_t)g * p.N + n) : 0.f;
    float sum = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < rows; i0 += 8) {
      float v[8], f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = i0 + i < rows;
        v[i] = in ? p.P[(m0 + i0 + i) * p.ldp + n] : 0.f;
        f[i] = in && p.mode != FUSED_NONE ? p.in[(m0 + i0 + i) * p.ld_in + n] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = p.alpha * v[i] + bias;
        if (p.U && i0 + i < rows) p.U[(m0 + i0 + i) * p.ldu + n] = v[i];
      }
      if (p.mode == FUSED_SLOPE) {
        slope_of<float>(v, f, p.act);
      } else {
        act_of<float>(v, p.act);
        if (p.mode == FUSED_ADD) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __fmaf_rn(p.beta, f[i], v[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < rows) {
          p.Y[(m0 + i0 + i) * p.ldy + n] = v[i];
          sum += v[i];
        }
    }
    if (p.part) p.part[(int64_t)slot * p.N + n] = sum;
  }
}

// dbias[g][j] = the sum of group g's slots: 32 columns a block, eight warps taking
// the slots in turn, their sums joined in warp order.
__global__ void __launch_bounds__(256) fused_dbias_kernel(const float* __restrict__ part,
                                                          const int* offsets, int M, int N,
                                                          int chunks, int64_t units,
                                                          float* __restrict__ dbias) {
  pdl_wait();
  pdl_trigger();
  __shared__ float join[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int g = (int)(unit / chunks), n = (int)(unit - (int64_t)g * chunks) * 32 + lane;
    int lo = 0, len = M;
    if (offsets) group_span(offsets, g, M, lo, len);
    const int slots = (len + 31) / 32;
    const float* src = part + ((int64_t)(lo >> 5) + g) * N + n;
    float sum = 0.f;
    if (n < N) {
#pragma unroll 8
      for (int s = warp; s < slots; s += 8) sum += src[(int64_t)s * N];
    }
    __syncthreads();  // (the last unit's sums are read)
    join[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && n < N) {
#pragma unroll
      for (int w = 1; w < 8; ++w) sum += join[w][lane];
      dbias[(int64_t)g * N + n] = sum;
    }
  }
}

}  // namespace

cudaError_t launch_fused_finish(const FusedArgs& a, const float* P, int64_t ldp, LaunchCtx& ctx) {
  FinishParams p;
  p.M = a.M; p.N = a.N;
  p.groups = a.groups;
  p.offsets = a.kind == FUSED_DENSE ? nullptr : a.offsets;
  p.P = P;
  p.ldp = ldp;
  p.alpha = a.alpha; p.beta = a.beta;
  p.bias = static_cast<const float*>(a.bias);
  p.act = a.act; p.mode = a.mode;
  p.in = static_cast<const float*>(a.in);
  p.ld_in = a.ld_in;
  p.U = static_cast<float*>(a.U);
  p.ldu = a.ldu;
  p.Y = static_cast<float*>(a.Y);
  p.ldy = a.ldy;
  p.part = a.part;
  p.chunks = (a.N + 255) / 256;
  p.units = (a.M / 32 + a.groups + 1) * (int64_t)p.chunks;
  const int64_t most = (int64_t)a.num_sms * 64;
  const cudaError_t e = launch_kernel(fused_finish_kernel, dim3((unsigned)(p.units < most ? p.units : most)),
                                      dim3(256), 0, ctx.stream, 1, p);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

cudaError_t launch_fused_dbias(const FusedArgs& a, float* dbias, LaunchCtx& ctx) {
  const int chunks = (a.N + 31) / 32;
  const int64_t units = (int64_t)a.groups * chunks, most = (int64_t)a.num_sms * 64;
  const cudaError_t e =
      launch_kernel(fused_dbias_kernel, dim3((unsigned)(units < most ? units : most)), dim3(256), 0,
                    ctx.stream, 1, (const float*)a.part,
                    a.kind == FUSED_DENSE ? (const int*)nullptr : a.offsets, a.M, a.N, chunks, units,
                    dbias);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

}  // namespace gb300
