// Products of a few rows with a large 4-bit stored operand,
//
//   C[m, n] = act(alpha * sum_k A[m, k] sb[n, k/b] qb[n, k] + beta * C + bias[n]),
//
// B stored [N, K]: one new token, or a small serving batch, through a
// projection.  Bound by the bytes of B, each read once.
//
// A block takes 128 rows of B and a slice of K; the blocks of a cluster share
// the rows and split K, so that a weight of a few dozen row ranges still keeps
// every SM loading.  A producer warp brings 128 x 256 codes, their scale tiles
// and the matching columns of A into a ring of stages by TMA; eight warps
// multiply 16 rows each with m16n8k16 warp MMAs, the codes as the 16-row operand.  The
// K order within a 32-code group is the loads': lane c of a quad holds codes 8c
// .. 8c + 7 (one word) and the same eight columns of A (one 16-byte load).
//   Power-of-two scales are applied to the fp32 sums of a 32-code group, which
// are exact products of codes and A, where A is fp16 or stored.  Other scales go
// to the codes: e4m3 ones in fp16 (a 4-bit significand times a 2-bit one: exact),
// since a group spans two of their blocks; powers of two, for a bf16 A, as bf16
// (exact: it has fp32's exponents), since a sum of bf16 values times unscaled codes
// may leave fp32 where the product does not.
//   The slices' fp32 sums are joined through distributed shared memory in rank
// order, so a result does not depend on timing.
//   tcgen05 would use 8 to 32 of its 128 rows here and take 16-bit operands from
// shared memory, which the codes would have to be written to first; the warp MMAs
// take them from registers and are nowhere near a limit.
//   Measured in a graph, us, and of that: start and join without a K loop; with
// the loop's loads but no products; all but the finishing of C
//   8 x 8192 x 8192 fp4_e4m3 bf16   16.8     3.6   10.3   15.2   (5.6 by its bytes)
//   8 x 8192 x 8192 fp4 fp16        15.2     3.6   10.0   13.5
//   32 x 8192 x 8192 fp4 fp16       22.9     3.7   11.4   20.6
//   1 x 5632 x 2048 fp4 fp16         5.6     2.4    3.8    4.7
// so no one part bounds it: with four stages a block, making operands of codes
// takes about as long again as waiting for them, and neither hides the other (2.0
// instructions a cycle of 4, DRAM at 24 %; barriers are the largest stall).
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

constexpr int ROWS = 128;          // rows of B a block takes
constexpr int KSTEP = 256;         // codes of K a stage holds
constexpr int WARPS = 8;            // 16 rows of B each
constexpr int ST_THREADS = 32 * (WARPS + 1);
// Two stages a block: small blocks, several an SM, keep more loads in flight than
// deeper rings (32 x 8192 x 8192 fp4 29.6 us with three, 22.5 with two; 8 rows
// 15.2 / 14.6)
constexpr int RING = 2;
constexpr int SUM_PITCH = ROWS + 4;  // (a quad's four columns in different banks)
constexpr int MAX_SPLIT = 8;       // blocks of a cluster (the portable limit)

// A's type: fp16, bf16, or codes of B's format
enum { X_F16 = 1, X_BF16 = 2, X_FP4 = 3 };

template <int FMT, int XT, int NT>
struct SCfg {
  static constexpr int TPS = KSTEP / mx_block(FMT) / 4;
  static constexpr int W_BYTES = ROWS * 128;
  static constexpr int X_BYTES = XT == X_FP4 ? 8 * NT * 128 : 8 * NT * KSTEP * 2;
  static constexpr int S_BYTES = TPS * 512;
  static constexpr int XS_BYTES = XT == X_FP4 ? TPS * 512 : 0;
  static constexpr int STAGE = W_BYTES + X_BYTES + S_BYTES + XS_BYTES;
  static constexpr int SUMS = SUM_PITCH * 8 * NT * 4;
  static constexpr int smem(int ring) { return ring * STAGE + SUMS + 1024 + 256; }
};

struct SParams {
  int M, N, K;
  int stages;       // K stages in all
  int per;          // and of a block
  int ring;
  void* C;
  int64_t ldc;
  int out;          // element type of C and bias
  float alpha, beta;
  Epilogue ep;
  unsigned int* status;
  uint64_t timeout_ns;
  int fault_injection;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_to_bf162(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t h, __half2 s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&h), s);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bf162_mul(uint32_t h, __nv_bfloat162 s) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&h), s);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// a power-of-two scale twice as bf16, which has fp32's exponents: 2^-127 is a
// subnormal, 255 NaN
__device__ __forceinline__ __nv_bfloat162 e8m0_bf162(uint32_t byte) {
  const uint32_t v = (byte == 255u ? 0x7FC0u : byte == 0u ? 0x0040u : byte << 7) * 0x10001u;
  return *reinterpret_cast<const __nv_bfloat162*>(&v);
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ __half2 e4m3_half2(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
  return __half2half2(__half(h));
}

template <typename T>
__device__ __forceinline__ void finish4(const SParams& p, int m, int n, const float4& sum) {
  T* const c = static_cast<T*>(p.C) + (int64_t)m * p.ldc + n;
  const float v4[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= p.N) break;
    float v = p.alpha * v4[e];
    if (p.beta != 0.f) v = __fmaf_rn(p.beta, MxIo<T>::to(c[e]), v);
    c[e] = MxIo<T>::from(apply_epilogue<T>(v, p.ep, n + e));
  }
}

template <int FMT, int XT, int NT>
__global__ void __launch_bounds__(ST_THREADS)
    mx_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
                     const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ CUtensorMap tmXS, const SParams p) {
  using C_ = SCfg<FMT, XT, NT>;
  constexpr int TPS = C_::TPS;
  // power-of-two scales multiply the sums of a 32-code group (others the codes)
  constexpr bool SUMS_SCALED = FMT == MX_FP4 && XT != X_BF16;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t sums = base + (uint32_t)(p.ring * C_::STAGE);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(base_ptr + p.ring * C_::STAGE + C_::SUMS);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(RING + s); };
  volatile uint32_t* const abort_flag = reinterpret_cast<uint32_t*>(bars + 2 * RING);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = (int)gridDim.x, rank = (int)blockIdx.x;  // a cluster is a row of the grid
  const int n0 = (int)blockIdx.y * ROWS;
  const int k_lo = rank * p.per, k_hi = min(p.stages, k_lo + p.per);
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), WARPS);
    }
    *abort_flag = 0u;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{p.status, abort_flag, p.timeout_ns};

  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

  if (warp == WARPS) {
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
          const uint32_t w = base + (uint32_t)(stage * C_::STAGE), x = w + C_::W_BYTES;
          const uint32_t s = x + C_::X_BYTES, xs = s + C_::S_BYTES;
          const uint32_t bar = full_bar(stage);
          mbar_arrive_expect_tx(bar, (uint32_t)C_::STAGE);
          tma_load_3d(w, &tmW, k * 128, n0, 0, bar);
          tma_load_3d(s, &tmS, 0, k * TPS, n0 >> 7, bar);
          if constexpr (XT == X_FP4) {
            tma_load_3d(x, &tmX, k * 128, 0, 0, bar);
            tma_load_3d(xs, &tmXS, 0, k * TPS, 0, bar);
          } else {
            // 32 columns a box: [group][row][64 bytes]
#pragma unroll
            for (int b = 0; b < KSTEP / 32; ++b)
              tma_load_3d(x + (uint32_t)(b * 8 * NT * 64), &tmX, k * KSTEP + 32 * b, 0, 0, bar);
          }
        }
        __syncwarp();
        if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      }
      // every load issued lands before the block's shared memory is released
      for (int s = 0; s < p.ring; ++s)
        if (pending & (1u << s))
          mbar_wait_drain(full_bar(s), (pend_phase >> s) & 1u, p.timeout_ns);
    }
  } else {
    // ------------------------------------------------------------ products
    const int g = lane >> 2, c = lane & 3;
    // this lane's places in a stage: row 16 warp + g of the codes (the 128-byte
    // swizzle goes by g), its scale word
    const uint32_t w_at = (uint32_t)((16 * warp + g) * 128 + 4 * c);
    const uint32_t s_at = (uint32_t)(((16 * warp + g) & 31) * 16 + (warp >> 1) * 4);
    int stage = 0;
    uint32_t phase = 0;
    for (int k = k_lo; k < k_hi; ++k) {
      bool ok = false;
      if (lane == 0) ok = mbar_wait(full_bar(stage), phase, wc);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      const uint32_t w = base + (uint32_t)(stage * C_::STAGE), x = w + C_::W_BYTES;
      const uint32_t s = x + C_::X_BYTES, xs = s + C_::S_BYTES;
      // scale words of rows g and g + 8 of the warp's 16
      uint32_t sw[TPS][2];
#pragma unroll
      for (int t = 0; t < TPS; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          sw[t][i] = lds32(s + s_at + (uint32_t)(t * 512 + i * 128));
      // Two power-of-two scales: A's first, then B's.  A sum of code products, a
      // multiple of 1/4 below 2^11, times a scale below 2^113 is exact and within
      // fp32; where A has a greater one, the lesser of each two scales comes first
      // (2^120 and 2^-120 would leave fp32 on their way to 1).
      bool far = false;
      if constexpr (FMT == MX_FP4 && XT == X_FP4) {
        uint32_t top = 0;  // (bytes of 0xF0 and more)
#pragma unroll
        for (int i = lane; i < 8 * NT * TPS; i += 32) {
          const uint32_t word =
              lds32(xs + (uint32_t)(i / (8 * NT) * 512 + i % (8 * NT) * 16));
          top |= word & (word >> 1) & (word >> 2) & (word >> 3) & 0x10101010u;
        }
        far = __any_sync(0xffffffffu, top != 0u);
      }
      const auto products = [&](auto far_scales) {
        [[maybe_unused]] constexpr bool FAR = decltype(far_scales)::value;
#pragma unroll
        for (int b = 0; b < KSTEP / 32; ++b) {
          // B's codes: rows g and g + 8, eight a lane
          uint32_t wa[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v = lds32(w + w_at + (uint32_t)(i * 1024) + (uint32_t)((b ^ g) * 16));
            e2m1_halves(v, wa[i]);
            if constexpr (FMT == MX_FP4_E4M3) {
              const int blk = 2 * b + (c >> 1);  // of the stage's 16
              const __half2 sc = e4m3_half2((sw[b / 2][i] >> (8 * (blk & 3))) & 255u);
#pragma unroll
              for (int j = 0; j < 4; ++j) wa[i][j] = half2_mul(wa[i][j], sc);
            }
            if constexpr (XT == X_BF16) {
#pragma unroll
              for (int j = 0; j < 4; ++j) wa[i][j] = half2_to_bf162(wa[i][j]);
              if constexpr (FMT == MX_FP4) {
                const __nv_bfloat162 sc = e8m0_bf162((sw[b / 4][i] >> (8 * (b & 3))) & 255u);
#pragma unroll
                for (int j = 0; j < 4; ++j) wa[i][j] = bf162_mul(wa[i][j], sc);
              }
            }
          }
          const uint32_t a0[4] = {wa[0][0], wa[1][0], wa[0][1], wa[1][1]};
          const uint32_t a1[4] = {wa[0][2], wa[1][2], wa[0][3], wa[1][3]};
          [[maybe_unused]] float sc[2];
          if constexpr (SUMS_SCALED) {
#pragma unroll
            for (int i = 0; i < 2; ++i) sc[i] = e8m0_value((sw[b / 4][i] >> (8 * (b & 3))) & 255u);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint32_t xb[4];
            if constexpr (XT == X_FP4) {
              const int r = 8 * j + g;
              e2m1_halves(lds32(x + (uint32_t)(r * 128 + ((b ^ g) * 16) + 4 * c)), xb);
              if constexpr (FMT == MX_FP4_E4M3) {
                const int blk = 2 * b + (c >> 1);
                const uint32_t word = lds32(xs + (uint32_t)((blk >> 2) * 512 + r * 16));
                const __half2 xsc = e4m3_half2((word >> (8 * (blk & 3))) & 255u);
#pragma unroll
                for (int e = 0; e < 4; ++e) xb[e] = half2_mul(xb[e], xsc);
              }
            } else {
              const uint4 v = lds128(x + (uint32_t)((b * 8 * NT + 8 * j + g) * 64 + 16 * c));
              xb[0] = v.x; xb[1] = v.y; xb[2] = v.z; xb[3] = v.w;
            }
            if constexpr (SUMS_SCALED) {
              float part[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(part, a0, xb[0], xb[1]);
              mma_f16(part, a1, xb[2], xb[3]);
              if constexpr (XT == X_FP4) {
                // the scales of A's rows 2c and 2c + 1 of this tile
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t word =
                      lds32(xs + (uint32_t)((b >> 2) * 512 + (8 * j + 2 * c + e) * 16));
                  const uint32_t xb8 = (word >> (8 * (b & 3))) & 255u;
                  if constexpr (!FAR) {
                    const float xsc = e8m0_value(xb8);
                    part[e] *= xsc;
                    part[2 + e] *= xsc;
                  } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {  // (255, NaN, is the greater)
                      const uint32_t wb8 = (sw[b / 4][i] >> (8 * (b & 3))) & 255u;
                      part[2 * i + e] *= e8m0_value(min(xb8, wb8));
                      part[2 * i + e] *= e8m0_value(max(xb8, wb8));
                    }
                  }
                }
              }
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[j][e] = __fmaf_rn(part[e], FAR ? 1.f : sc[e >> 1], acc[j][e]);
            } else {
              if constexpr (XT == X_BF16) {
                mma_bf16(acc[j], a0, xb[0], xb[1]);
                mma_bf16(acc[j], a1, xb[2], xb[3]);
              } else {
                mma_f16(acc[j], a0, xb[0], xb[1]);
                mma_f16(acc[j], a1, xb[2], xb[3]);
              }
            }
          }
        }
      };
      if (far) products(std::true_type{});
      else products(std::false_type{});
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(stage));
      if (++stage == p.ring) { stage = 0; phase ^= 1u; }
    }
    // this block's sums: [row of C][row of B]
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = 16 * warp + g + 8 * (e >> 1), m = 8 * j + 2 * c + (e & 1);
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(sums + (uint32_t)((m * SUM_PITCH + n) * 4)),
                     "f"(acc[j][e]));
      }
  }
  // ------------------------------------------------------------ join
  // (a block alone is a cluster of one: the barriers then are the block's)
  cluster_sync();
  // (a block finishes its share of the 128 columns, four a thread)
  const int q_lo = rank * (ROWS / 4) / splits, q_cnt = (rank + 1) * (ROWS / 4) / splits - q_lo;
  for (int i = threadIdx.x; i < q_cnt * p.M; i += ST_THREADS) {
    const int m = i / q_cnt, n = 4 * (q_lo + i % q_cnt);
    if (n0 + n >= p.N) continue;
    const float4 v = cluster_sum4(sums + (uint32_t)((m * SUM_PITCH + n) * 4), splits);
    if (p.out == 0) finish4<float>(p, m, n0 + n, v);
    else if (p.out == 1) finish4<__half>(p, m, n0 + n, v);
    else finish4<__nv_bfloat16>(p, m, n0 + n, v);
  }
  cluster_sync();  // no block leaves while another reads its sums
}

// ---------------------------------------------------------------- host side
template <int FMT, int XT, int NT>
cudaError_t launch_stream(const MxStreamArgs& a, LaunchCtx& ctx) {
  using C_ = SCfg<FMT, XT, NT>;
  auto kern = mx_stream_kernel<FMT, XT, NT>;
  static OncePerDevice set;
  const cudaError_t attr = set.run(call_device(), cudaSuccess, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C_::smem(RING));
  });
  if (attr != cudaSuccess) return attr;
  SParams p;
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.stages = (a.K + KSTEP - 1) / KSTEP;
  const int64_t rb = ((int64_t)a.N + ROWS - 1) / ROWS;
  if (rb > 65535) return cudaErrorNotSupported;
  // The most slices of K whose clusters are all resident at once (a slice's
  // stages, up to the ring, are its block's loads in flight); one where no split
  // is.
  int splits = 1;
  p.per = p.stages;
  for (int s = MAX_SPLIT; s > 1; --s) {
    const int per = (p.stages + s - 1) / s, n = (p.stages + per - 1) / per;
    const int ring = per < RING ? per : RING;
    // (queried once for each cluster and ring size, and device)
    static CountPerDevice slots[MAX_SPLIT + 1][RING + 1];
    const int have = slots[n][ring].get(call_device(), [kern, n, ring] {
      return resident_clusters((const void*)kern, n, ST_THREADS, (size_t)C_::smem(ring));
    });
    // (blocks of one stage only where blocks of two would leave SMs without one: 1 x
    // 5632 x 2048 6.3 us in 352 blocks, 5.3 in 176)
    if (per == 1 && rb * ((p.stages + 1) / 2) >= a.num_sms) continue;
    if (rb <= have) {
      splits = n;
      p.per = per;
      break;
    }
  }
  p.ring = p.per < RING ? p.per : RING;
  p.C = a.C; p.ldc = a.ldc; p.out = a.out;
  p.alpha = a.alpha; p.beta = a.beta;
  p.ep = a.ep;
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  p.fault_injection = a.fault_injection;
  const int64_t kbytes = ((int64_t)a.K + 1) / 2;
  const int64_t tiles = mx_scale_tiles(FMT, a.K);
  CUtensorMap mW, mS, mX, mXS;
  memset(&mXS, 0, sizeof(mXS));
  const CUtensorMapDataType U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  auto scales = [&](CUtensorMap* m, const void* s, int64_t rows) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, s, tiles, 128, 128, 128, C_::TPS,
                    CU_TENSOR_MAP_SWIZZLE_NONE, (rows + 127) / 128, tiles * 128, 4);
  };
  bool ok = make_map(&mW, U8, a.B, a.N, kbytes, a.ldb, 128, ROWS, CU_TENSOR_MAP_SWIZZLE_128B, 1, 0, 1) &&
            scales(&mS, a.Bs, a.N);
  if constexpr (XT == X_FP4)
    ok = ok && make_map(&mX, U8, a.A, a.M, kbytes, a.lda, 128, 8 * NT, CU_TENSOR_MAP_SWIZZLE_128B, 1, 0, 1) &&
         scales(&mXS, a.As, a.M);
  else
    ok = ok && make_map(&mX, XT == X_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        a.A, a.M, a.K, a.lda, 32, 8 * NT, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (!ok) return cudaErrorNotSupported;
  ctx.grid = (int)(splits * rb);
  const cudaError_t e =
      launch_kernel(kern, dim3((unsigned)splits, (unsigned)rb), dim3(ST_THREADS),
                    (size_t)C_::smem(p.ring), ctx.stream, splits, mW, mS, mX, mXS, p);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

template <int FMT, int XT>
cudaError_t launch_stream_nt(const MxStreamArgs& a, LaunchCtx& ctx) {
  if (a.M <= 8) return launch_stream<FMT, XT, 1>(a, ctx);
  if (a.M <= 16) return launch_stream<FMT, XT, 2>(a, ctx);
  // (M is at most 32)
  return launch_stream<FMT, XT, 4>(a, ctx);
}
template <int FMT>
cudaError_t launch_stream_x(const MxStreamArgs& a, LaunchCtx& ctx) {
  if (a.As) return launch_stream_nt<FMT, X_FP4>(a, ctx);
  if (a.out == 1) return launch_stream_nt<FMT, X_F16>(a, ctx);
  return launch_stream_nt<FMT, X_BF16>(a, ctx);
}

}  // namespace

cudaError_t launch_mx_stream(const MxStreamArgs& a, LaunchCtx& ctx) {
  return a.format == MX_FP4 ? launch_stream_x<MX_FP4>(a, ctx)
                            : launch_stream_x<MX_FP4_E4M3>(a, ctx);
}

}  // namespace gb300
