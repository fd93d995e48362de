// What fused products do outside their main kernel: the epilogue over raw sums in
// memory, and the join of the column sums.
//
// The raw sums are fp32 products -- 2 K / 72 ps a value on the CUDA cores (K = 2048: 57
// ps), where a pass over the values in memory costs 2 to 4 ps (1000 x 3001 x 777 with
// relu and a residual: 125 us; with the residual read in the products' own epilogue, which
// nothing there hides, 141) -- or the slices of K of a 16-bit
// product with few tiles (512 x 2048 x 5632: four of 64 tiles instead of 64 for 152 SMs).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gelu.cuh"
#include "groups.cuh"
#include "internal.h"

namespace gb300 {
namespace {

struct FinishParams {
  int M, N, groups;
  const int* offsets;  // null: one group of all rows
  const float* P;      // [splits][M][ldp]
  int64_t ldp;
  int splits;
  float alpha, beta;
  const void* bias;
  int act, mode;
  const void* in;
  int64_t ld_in;
  void* U;
  int64_t ldu;
  void* Y;
  int64_t ldy;
  float* part;
  int chunks;  // of FIN_COLS columns
  int64_t units;
};

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// four values of a row, aligned
template <typename T>
struct alignas(sizeof(T) * 4) Vec4 {
  T v[4];
};

// A slot of 32 rows (group g's begin at o[g] / 32 + g) x 256 columns a block: a thread has
// four columns of four rows, and asks for those of all slices (up to S of them) at once.
// PACKED: the four follow one another, where every matrix has aligned rows of whole
// fours; else they are 64 apart, so that a warp still reads what lies together.
constexpr int FIN_THREADS = 512, FIN_COLS = 256;
template <typename T, bool PACKED, int S>
__global__ void __launch_bounds__(FIN_THREADS) fused_finish_kernel(const FinishParams p) {
  __shared__ float join[8][FIN_COLS];
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  for (int64_t unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
    const int slot = (int)(unit / p.chunks);
    const int n0 = (int)(unit - (int64_t)slot * p.chunks) * FIN_COLS;
    const int at = PACKED ? 4 * tx : tx;  // its columns: n0 + at + step j
    constexpr int step = PACKED ? 1 : 64;
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
    if (rows <= 0) continue;  // (the whole block)
    const int n = n0 + at;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    const int i0 = 4 * ty;
    if (n < p.N && i0 < rows) {
      auto get = [&](const auto* row, auto& x) {  // four of a row from column 0 on
        if constexpr (PACKED) {
          x = *reinterpret_cast<const std::decay_t<decltype(x)>*>(row + n);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + step * j < p.N) x.v[j] = row[n + step * j];
        }
      };
      float v[16], f[16];
      Vec4<float> x[S][4];
      Vec4<T> y[4], b;
      if (p.bias) get(static_cast<const T*>(p.bias) + (int64_t)g * p.N, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = (int64_t)lo + r0 + min(i0 + i, rows - 1);
        if (p.mode != FUSED_NONE) get(static_cast<const T*>(p.in) + m * p.ld_in, y[i]);
#pragma unroll
        for (int s = 0; s < S; ++s)
          if (s < p.splits) get(p.P + ((int64_t)s * p.M + m) * p.ldp, x[s][i]);
      }
      // (slices past S, in order: fp32 alone has so many)
      if constexpr (sizeof(T) == 4 && S > 1) {
        for (int s0 = S; s0 < p.splits; s0 += S - 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int s = 1; s < S; ++s) x[0][i].v[j] += x[s][i].v[j];
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t m = (int64_t)lo + r0 + min(i0 + i, rows - 1);
#pragma unroll
            for (int s = 1; s < S; ++s) {
              x[s][i] = Vec4<float>{{0.f, 0.f, 0.f, 0.f}};
              if (s0 + s - 1 < p.splits) get(p.P + ((int64_t)(s0 + s - 1) * p.M + m) * p.ldp, x[s][i]);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] = x[0][i / 4].v[i % 4];
        f[i] = p.mode != FUSED_NONE ? to_f(y[i / 4].v[i % 4]) : 0.f;
#pragma unroll
        for (int s = 1; s < S; ++s)
          if (s < p.splits) v[i] += x[s][i / 4].v[i % 4];
        v[i] = p.alpha * v[i] + (p.bias ? to_f(b.v[i % 4]) : 0.f);
      }
      auto put = [&](void* to, int64_t ld) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i0 + i >= rows) continue;
          T* const row = static_cast<T*>(to) + ((int64_t)lo + r0 + i0 + i) * ld + n;
          if constexpr (PACKED) {
            Vec4<T> o;
#pragma unroll
            for (int j = 0; j < 4; ++j) o.v[j] = from_f<T>(v[4 * i + j]);
            *reinterpret_cast<Vec4<T>*>(row) = o;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (n + step * j < p.N) row[step * j] = from_f<T>(v[4 * i + j]);
          }
        }
      };
      if (p.U) put(p.U, p.ldu);
      if (p.mode == FUSED_SLOPE) {
        slope_of<T>(v, f, p.act);
      } else {
        act_of<T>(v, p.act);
        if (p.mode == FUSED_ADD) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __fmaf_rn(p.beta, f[i], v[i]);
        }
      }
      put(p.Y, p.ldy);
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i % 4] += i0 + i / 4 < rows ? v[i] : 0.f;
    }
    if (p.part) {
      __syncthreads();  // (the last unit's sums are read)
#pragma unroll
      for (int j = 0; j < 4; ++j) join[ty][at + step * j] = sum[j];
      __syncthreads();
      if ((int)threadIdx.x < FIN_COLS && n0 + (int)threadIdx.x < p.N) {
        float all = join[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < 8; ++w) all += join[w][threadIdx.x];
        p.part[(int64_t)slot * p.N + n0 + threadIdx.x] = all;
      }
    }
  }
}

// dbias[g][j] = the sum of group g's slots: 32 columns a block, its warps taking the
// slots in turn, their sums joined in warp order.  Thirty-two warps where a group has
// many slots (one of 512: 8 us with eight, the call 258 -> 244), eight elsewhere (64 of
// 16 slots on average: 4 us less).
template <int DB_WARPS>
__global__ void __launch_bounds__(32 * DB_WARPS)
    fused_dbias_kernel(const float* __restrict__ part, const int* offsets, int M, int N, int chunks,
                       int64_t units, float* __restrict__ dbias) {
  pdl_wait();
  pdl_trigger();
  __shared__ float join[DB_WARPS][32];
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
      for (int s = warp; s < slots; s += DB_WARPS) sum += src[(int64_t)s * N];
    }
    __syncthreads();  // (the last unit's sums are read)
    join[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && n < N) {
#pragma unroll
      for (int w = 1; w < DB_WARPS; ++w) sum += join[w][lane];
      dbias[(int64_t)g * N + n] = sum;
    }
  }
}

}  // namespace

template <typename T>
static cudaError_t launch_finish(const FusedArgs& a, const float* P, int64_t ldp, LaunchCtx& ctx) {
  FinishParams p;
  p.M = a.M; p.N = a.N;
  p.groups = a.groups;
  p.offsets = a.kind == FUSED_DENSE ? nullptr : a.offsets;
  p.P = P;
  p.ldp = ldp;
  p.splits = a.splits;
  p.alpha = a.alpha; p.beta = a.beta;
  p.bias = a.bias;
  p.act = a.act; p.mode = a.mode;
  p.in = a.in;
  p.ld_in = a.ld_in;
  p.U = a.U;
  p.ldu = a.ldu;
  p.Y = a.Y;
  p.ldy = a.ldy;
  p.part = a.part;
  auto four = [](const void* q, int64_t ld, size_t e) {
    return !q || (((uintptr_t)q % (4 * e)) == 0 && ld % 4 == 0);
  };
  const bool packed = a.N % 4 == 0 && four(P, ldp, 4) && four(a.Y, a.ldy, sizeof(T)) &&
                      four(a.U, a.ldu, sizeof(T)) && four(a.bias, a.N, sizeof(T)) &&
                      (a.mode == FUSED_NONE || four(a.in, a.ld_in, sizeof(T)));
  p.chunks = (a.N + FIN_COLS - 1) / FIN_COLS;
  p.units = (a.M / 32 + a.groups + 1) * (int64_t)p.chunks;
  const int64_t most = (int64_t)a.num_sms * 64;
  const dim3 grid((unsigned)(p.units < most ? p.units : most));
  constexpr int S = FUSED_MAX_SPLITS;
  auto kern = packed ? (a.splits == 1 ? fused_finish_kernel<T, true, 1> : fused_finish_kernel<T, true, S>)
                     : (a.splits == 1 ? fused_finish_kernel<T, false, 1> : fused_finish_kernel<T, false, S>);
  const cudaError_t e = launch_kernel(kern, grid, dim3(FIN_THREADS), 0, ctx.stream, 1, p);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

cudaError_t launch_fused_finish(const FusedArgs& a, const float* P, int64_t ldp, LaunchCtx& ctx) {
  switch (a.dtype) {
    case 0: return launch_finish<float>(a, P, ldp, ctx);
    case 1: return launch_finish<__half>(a, P, ldp, ctx);
    default: return launch_finish<__nv_bfloat16>(a, P, ldp, ctx);
  }
}

cudaError_t launch_fused_dbias(const FusedArgs& a, float* dbias, LaunchCtx& ctx) {
  const int chunks = (a.N + 31) / 32;
  const int64_t units = (int64_t)a.groups * chunks, most = (int64_t)a.num_sms * 64;
  const bool many = a.M / 32 >= 128ll * a.groups;
  const cudaError_t e = launch_kernel(
      many ? fused_dbias_kernel<32> : fused_dbias_kernel<8>,
      dim3((unsigned)(units < most ? units : most)), dim3(many ? 1024 : 256), 0, ctx.stream, 1,
      (const float*)a.part, a.kind == FUSED_DENSE ? (const int*)nullptr : a.offsets, a.M, a.N, chunks,
      units, dbias);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

}  // namespace gb300
