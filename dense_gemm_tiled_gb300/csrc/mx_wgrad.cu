// Gradient of a low-rank adapter from an 8-bit checkpoint,
//
//   C[m, n] = act(alpha * sum_t A[t, m] s[t, n/32] q[t, n] + beta * C + bias[n]),
//
// A [T, M] fp16 or bf16 with M up to 32 columns, q the checkpoint of the
// layer's input, [T, N] (the tn product of "Metal GEMM Kernels for LoRA Training
// on Apple Silicon", section 5, with its right operand stored in 8 bits).
// The bytes of the checkpoint, each read once, are its floor: 32 x 8192 x 8192 fp16
// takes 25.8 us, 2.7 TB/s, where 70 MB at HBM's rate would be 10.4.  Of that, start
// and join without a K loop 4.2; with its loads but no products 18.3; all but the
// finishing of C 23.9.  So the loads, at two blocks an SM, come first (DRAM 31 % busy),
// then turning codes into operands, which they hide in part only (1.7 instructions
// a cycle of 4).
//
// A block takes 128 columns of the checkpoint and a slice of T; a cluster's
// blocks share the columns and split T.  A producer warp brings 64 rows of q (128-
// byte swizzle), their scale tile and the same rows of A into a ring by TMA.
// Eight warps: four quarters of the columns, two halves of each stage's rows.
// The warp MMA (m16n8k16) wants pairs of t for one column: a lane reads 4 bytes
// of four rows and interleaves them with byte permutes, so one pass makes the
// operands of four 8-column tiles (column 4g + j of the quarter in tile j).  A
// comes through ldmatrix.trans.
//   Every row has a scale of its own, so a pair of rows needs both scales side by
// side: one more warp makes these once a stage (32 row pairs x 4 blocks) for all
// the others, which otherwise spent a third of their instructions on them (28.3
// -> 25.8 us at the size above; two blocks of ten warps an SM: three, at 64
// registers a thread, 31.3; the loading warp making them as well, 36).
//   A code becomes fp16 by putting its byte into 1024's fraction (1024 + q + 128,
// exact); one FMA by the scale takes 1152 times the scale away, exactly while
// the scale is a power of two between 2^-14 and 2.  Other scales, and bf16, go
// through fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mx_format.cuh"
#include "per_device.h"
#include "tensor_map.h"

namespace gb300 {
namespace {

constexpr int COLS = 128;   // columns of the checkpoint a block takes
constexpr int TSTEP = 64;   // rows of it a stage holds
constexpr int WG_WARPS = 8;
constexpr int WG_THREADS = 32 * (WG_WARPS + 2);  // and a producer, and the scales' warp
constexpr int WG_RING = 4;
constexpr int WG_PITCH = COLS + 4;  // of the sums (a row's start moves by 16 bytes of a bank row)
constexpr int WG_SPLIT = 8;

template <int MT>
struct GCfg {
  static constexpr int Q_BYTES = TSTEP * 128;
  static constexpr int A_BYTES = TSTEP * 32 * MT;
  static constexpr int S_BYTES = 512;       // one scale tile
  static constexpr int P_BYTES = 128 * 8;   // and the row pairs' scales made from it
  static constexpr int PAD = 512;           // (a stage is whole swizzle periods)
  static constexpr int STAGE = Q_BYTES + A_BYTES + S_BYTES + P_BYTES + PAD;
  static constexpr uint32_t TX = Q_BYTES + A_BYTES + S_BYTES;
  static constexpr int SUMS = 16 * MT * WG_PITCH * 4;
  static constexpr int smem(int ring) { return ring * STAGE + SUMS + 1024 + 256; }
};

struct GParams {
  int M, N, K;
  int stages, per, ring;
  void* C;
  int64_t ldc;
  float alpha, beta;
  Epilogue ep;
  unsigned int* status;
  uint64_t timeout_ns;
  int fault_injection;
};

template <typename T>
__device__ __forceinline__ void mma_16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// What a pair of rows' scale bytes become for code_pairs: two words.
//   fp16, both between 2^-14 and 2 (activations below 254; they and 1152 times
//   them are normal fp16 numbers): the scales as a half2, then -1152 times them
//   otherwise: the scales in fp32, the first one's sign (scales are positive)
//   telling the fp16 form so
template <typename T>
__device__ __forceinline__ uint2 pair_scales(uint32_t s0, uint32_t s1) {
  if constexpr (std::is_same<T, __half>::value) {
    const uint32_t t = s0 | (s1 << 16);
    if (((t - 0x00710071u) & 0xFFF0FFF0u) == 0u) {
      const uint32_t sbits = (t - 0x00700070u) << 10;
      const __half2 off =
          __hmul2(*reinterpret_cast<const __half2*>(&sbits), __float2half2_rn(-1152.f));
      return make_uint2(sbits, *reinterpret_cast<const uint32_t*>(&off));
    }
    return make_uint2(__float_as_uint(e8m0_value(s0)) | 0x80000000u, __float_as_uint(e8m0_value(s1)));
  } else {
    return make_uint2(__float_as_uint(e8m0_value(s0)), __float_as_uint(e8m0_value(s1)));
  }
}

// Pairs (row 0, row 1) of four columns' values as 16-bit operands: a, b the two
// rows' codes (each offset by 128), sc their pair_scales.
template <typename T>
__device__ __forceinline__ void code_pairs(uint32_t a, uint32_t b, uint2 sc, uint32_t (&out)[4]) {
  if constexpr (std::is_same<T, __half>::value) {
    if ((int32_t)sc.x >= 0) {
      const __half2 s = *reinterpret_cast<const __half2*>(&sc.x);
      const __half2 off = *reinterpret_cast<const __half2*>(&sc.y);
      const uint32_t lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = __byte_perm(j < 2 ? lo : hi, 0x64646464u, (j & 1) ? 0x4342 : 0x4140);
        const __half2 x = __hfma2(*reinterpret_cast<const __half2*>(&v), s, off);
        out[j] = *reinterpret_cast<const uint32_t*>(&x);
      }
      return;
    }
  }
  // code + 128 in the fraction of 2^23, less 2^23 + 128: the code; times its
  // scale: exact in fp32 and, within its range, in the 16-bit type
  const float f0 = __uint_as_float(sc.x & 0x7FFFFFFFu), f1 = __uint_as_float(sc.y);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x = __uint_as_float(__byte_perm(a, 0x4B000000u, 0x7540 + j)) - 8388736.f;
    const float y = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7540 + j)) - 8388736.f;
    out[j] = pack2<T>(x * f0, y * f1);
  }
}

template <typename T, int MT>
__global__ void __launch_bounds__(WG_THREADS)
    mx_wgrad_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmS,
                    const __grid_constant__ CUtensorMap tmA, const GParams p) {
  using C_ = GCfg<MT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t sums = base + (uint32_t)(p.ring * C_::STAGE);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(base_ptr + p.ring * C_::STAGE + C_::SUMS);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(WG_RING + s); };
  auto scale_bar = [&](int s) { return bar0 + 8u * (uint32_t)(2 * WG_RING + s); };
  volatile uint32_t* const abort_flag = reinterpret_cast<uint32_t*>(bars + 3 * WG_RING);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = (int)gridDim.x, rank = (int)blockIdx.x;
  const int n0 = (int)blockIdx.y * COLS;
  const int k_lo = rank * p.per, k_hi = min(p.stages, k_lo + p.per);
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), WG_WARPS);
      mbar_init(scale_bar(s), 1);
    }
    *abort_flag = 0u;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{p.status, abort_flag, p.timeout_ns};

  float acc[MT][4][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
  const int g = lane >> 2, c = lane & 3;
  const int quarter = warp & 3, part = warp >> 2;  // columns 32 quarter ..; rows 32 part .. of a stage

  if (warp == WG_WARPS) {
    // ------------------------------------------------------------ producer
    {
      const bool leader = elect_one();
      int stage = 0;
      uint32_t phase = 0, pending = 0, pend_phase = 0;
      for (int k = k_lo; k < k_hi; ++k) {
        if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, wc))) break;
        const bool skip = p.fault_injection == 1 && k == k_lo;
        if (!skip) {
          pending |= 1u << stage;
          pend_phase = (pend_phase & ~(1u << stage)) | (phase << stage);
        }
        if (!skip && leader) {
          const uint32_t q = base + (uint32_t)(stage * C_::STAGE), a = q + C_::Q_BYTES;
          const uint32_t bar = full_bar(stage);
          mbar_arrive_expect_tx(bar, C_::TX);
          tma_load_3d(q, &tmQ, n0, k * TSTEP, 0, bar);
          tma_load_3d(a, &tmA, 0, k * TSTEP, 0, bar);
          tma_load_3d(a + C_::A_BYTES, &tmS, 0, (int)blockIdx.y, (k * TSTEP) >> 7, bar);
        }
        __syncwarp();
        if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      }
      for (int s = 0; s < p.ring; ++s)
        if (pending & (1u << s))
          mbar_wait_drain(full_bar(s), (pend_phase >> s) & 1u, p.timeout_ns);
    }
  } else if (warp > WG_WARPS) {
    // ------------------------------------------------------------ scales of row pairs
    int stage = 0;
    uint32_t phase = 0;
    for (int k = k_lo; k < k_hi; ++k) {
      if (!__all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, wc))) break;
      const uint32_t tile =
          base + (uint32_t)(stage * C_::STAGE + C_::Q_BYTES + C_::A_BYTES);
      // entry 4 pair + block; rows 2 pair and 2 pair + 1 of the stage, which starts
      // in the middle of its scale tile every other time
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = 32 * i + lane, t = ((k * TSTEP) & 127) + 2 * (at >> 2);
        const uint32_t from = tile + (uint32_t)((t & 31) * 16 + (t >> 5) * 4 + (at & 3));
        const uint2 v = pair_scales<T>(lds8(from), lds8(from + 16u));
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(
                         tile + (uint32_t)(C_::S_BYTES + at * 8)),
                     "r"(v.x), "r"(v.y)
                     : "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(scale_bar(stage));
      if (++stage == p.ring) { stage = 0; phase ^= 1u; }
    }
  } else {
    // ------------------------------------------------------------ products
    // this lane's places within a stage: rows 2 c + (i & 1) + 8 (i >> 1) of a
    // 16-row step (the swizzle goes by the row's last three bits: the same for
    // every step)
    uint32_t at_q[2], at_a[MT];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * c + i;
      at_q[i] = (uint32_t)(t * 128 + (((2 * quarter + (g >> 2)) ^ t) * 16) + 4 * (g & 3) + part * 4096);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      // 8 x 8 blocks (rows t, columns m): t half by lane bit 4, m half by bit 3
      const int t = (lane & 7) + ((lane >> 4) << 3);
      const int ch = 2 * i + ((lane >> 3) & 1);  // 16-byte chunk of A's row
      // (the swizzle of a row of 32 MT bytes)
      const int sw = MT == 2 ? ((t >> 1) & 3) : ((t >> 2) & 1);
      at_a[i] = (uint32_t)(C_::Q_BYTES + (t + part * 32) * 32 * MT + ((ch ^ sw) * 16));
    }
    // (row pair 16 part + c of the stage's 32, this quarter's block)
    const uint32_t at_s = (uint32_t)(C_::Q_BYTES + C_::A_BYTES + C_::S_BYTES +
                                     ((16 * part + c) * 4 + quarter) * 8);
    int stage = 0;
    uint32_t phase = 0;
    for (int k = k_lo; k < k_hi; ++k) {
      bool ok = false;
      // (the codes' own barrier too: it is the scales' warp that has seen it)
      if (lane == 0)
        ok = mbar_wait(scale_bar(stage), phase, wc) && mbar_wait(full_bar(stage), phase, wc);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      const uint32_t q = base + (uint32_t)(stage * C_::STAGE);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {  // rows 32 part + 16 kk .. + 15 of the stage
        uint32_t am[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
          ldmatrix_x4_trans(q + at_a[i] + (uint32_t)(kk * 16 * 32 * MT), am[i]);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = lds32(q + at_q[i & 1] + (uint32_t)(kk * 16 + 8 * (i >> 1)) * 128u) ^ 0x80808080u;
        // rows 2c, 2c + 1 and 8 further on: pairs 8 kk + c and 4 further on
        const uint2 s0 = lds64(q + at_s + (uint32_t)(kk * 8 * 32));
        const uint2 s1 = lds64(q + at_s + (uint32_t)((kk * 8 + 4) * 32));
        uint32_t lo[4], hi[4];
        code_pairs<T>(w[0], w[1], s0, lo);
        code_pairs<T>(w[2], w[3], s1, hi);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i) mma_16<T>(acc[i][j], am[i], lo[j], hi[j]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(stage));
      if (++stage == p.ring) { stage = 0; phase ^= 1u; }
    }
  }
  // ------------------------------------------------------------ join
  // the two row halves' sums, then the slices' (element (i, j, e) of the warp's
  // tiles is row 16 i + g + 8 (e / 2), column 32 quarter + 4 (2 c + e % 2) + j)
  for (int turn = 1; turn >= 0; --turn) {
    if (warp < WG_WARPS && part == turn) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = 16 * i + g + 8 * (e >> 1), n = 32 * quarter + 4 * (2 * c + (e & 1));
          const uint32_t at = sums + (uint32_t)((m * WG_PITCH + n) * 4);
          float v[4] = {acc[i][0][e], acc[i][1][e], acc[i][2][e], acc[i][3][e]};
          if (turn == 0) {
            float o[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3])
                         : "r"(at));
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += o[j];
          }
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v[0]), "f"(v[1]),
                       "f"(v[2]), "f"(v[3]));
        }
    }
    if (turn == 1) __syncthreads();
  }
  cluster_sync();
  // (a block finishes its share of the 128 columns, four a thread)
  const int q_lo = rank * (COLS / 4) / splits, q_cnt = (rank + 1) * (COLS / 4) / splits - q_lo;
  for (int i = threadIdx.x; i < q_cnt * p.M; i += WG_THREADS) {
    const int m = i / q_cnt, n = 4 * (q_lo + i % q_cnt);
    if (n0 + n >= p.N) continue;
    const float4 sum = cluster_sum4(sums + (uint32_t)((m * WG_PITCH + n) * 4), splits);
    const float v4[4] = {sum.x, sum.y, sum.z, sum.w};
    T* const dst = static_cast<T*>(p.C) + (int64_t)m * p.ldc + n0 + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n0 + n + e >= p.N) break;
      float v = p.alpha * v4[e];
      if (p.beta != 0.f) v = __fmaf_rn(p.beta, MxIo<T>::to(dst[e]), v);
      dst[e] = MxIo<T>::from(apply_epilogue<T>(v, p.ep, n0 + n + e));
    }
  }
  cluster_sync();
}

template <typename T, int MT>
cudaError_t launch_wgrad(const MxStreamArgs& a, LaunchCtx& ctx) {
  using C_ = GCfg<MT>;
  auto kern = mx_wgrad_kernel<T, MT>;
  static OncePerDevice set;
  const cudaError_t attr = set.run(call_device(), cudaSuccess, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C_::smem(WG_RING));
  });
  if (attr != cudaSuccess) return attr;
  GParams p;
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.stages = (a.K + TSTEP - 1) / TSTEP;
  const int64_t cb = ((int64_t)a.N + COLS - 1) / COLS;
  if (cb > 65535) return cudaErrorNotSupported;
  // the most slices of T whose clusters are all resident at once (queried once
  // for each cluster and ring size, and device)
  int splits = 1;
  p.per = p.stages;
  for (int s = WG_SPLIT; s > 1; --s) {
    const int per = (p.stages + s - 1) / s, n = (p.stages + per - 1) / per;
    const int ring = per < WG_RING ? per : WG_RING;
    static CountPerDevice slots[WG_SPLIT + 1][WG_RING + 1];
    const int have = slots[n][ring].get(call_device(), [kern, n, ring] {
      return resident_clusters((const void*)kern, n, WG_THREADS, (size_t)C_::smem(ring));
    });
    if (cb <= have) {
      splits = n;
      p.per = per;
      break;
    }
  }
  p.ring = p.per < WG_RING ? p.per : WG_RING;
  p.C = a.C; p.ldc = a.ldc;
  p.alpha = a.alpha; p.beta = a.beta;
  p.ep = a.ep;
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  p.fault_injection = a.fault_injection;
  const int64_t tiles = mx_scale_tiles(MX_INT8, a.N);
  CUtensorMap mQ, mS, mA;
  const CUtensorMapSwizzle sw = MT == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  const CUtensorMapDataType ty = std::is_same<T, __half>::value
                                     ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!make_map(&mQ, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, a.K, a.N, a.ldb, 128, TSTEP,
                CU_TENSOR_MAP_SWIZZLE_128B, 1, 0, 1) ||
      !make_map(&mS, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.Bs, tiles, 128, 128, 128, 1,
                CU_TENSOR_MAP_SWIZZLE_NONE, ((int64_t)a.K + 127) / 128, tiles * 128, 4) ||
      !make_map(&mA, ty, a.A, a.K, a.M, a.lda, 16 * MT, TSTEP, sw))
    return cudaErrorNotSupported;
  ctx.grid = (int)(splits * cb);
  const cudaError_t e = launch_kernel(kern, dim3((unsigned)splits, (unsigned)cb), dim3(WG_THREADS),
                                      (size_t)C_::smem(p.ring), ctx.stream, splits, mQ, mS, mA, p);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

template <typename T>
cudaError_t launch_wgrad_t(const MxStreamArgs& a, LaunchCtx& ctx) {
  if (a.M <= 16) return launch_wgrad<T, 1>(a, ctx);
  return launch_wgrad<T, 2>(a, ctx);
}

}  // namespace

cudaError_t launch_mx_wgrad(const MxStreamArgs& a, LaunchCtx& ctx) {
  return a.out == 1 ? launch_wgrad_t<__half>(a, ctx) : launch_wgrad_t<__nv_bfloat16>(a, ctx);
}

}  // namespace gb300
