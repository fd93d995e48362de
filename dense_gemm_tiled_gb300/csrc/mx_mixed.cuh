#pragma once
// Product of a 16-bit operand with a stored one on the 5th-generation tensor
// cores, the stored operand converted on its way:
//
//   C[m, n] = act(alpha * sum_k A[m, k] w[n, k] + beta * C + bias[n]),
//
// w[n, k] = code * scale, stored [N, K] (nt) or [K, N] (nn, tn), A fp16 or bf16.
// This header holds the kernel; mx_mixed_f16.cu and mx_mixed_bf16.cu
// instantiate it.
//
// The tensor core's 16-bit kinds take both operands in A's type, so the codes
// become that type in shared memory.  The stored operand is the MMA's 128-row
// side: a block converts 128 of its rows (or columns) once for up to 128 rows of
// A (256 with a pair), and the accumulator is C transposed: lanes are columns of
// C, so a warp's stores cover 32 of them in a row.
//   warp 0        producer: TMA of A's tile (128-byte swizzle), the codes and
//                 their scale tiles, into one ring of stages of 64 k
//   warp 1        tensor memory, MMA issue
//   warps 2-5     epilogue
//   warps 6-13    converters: 32 codes a thread and stage, written in the
//                 swizzled K-major (nt) or MN-major (nn, tn) operand layout
// Two forms:
//   pairs   256 columns x 256 rows of C, 2-SM MMAs (each block converts its own
//           128 columns and loads half of A's rows), persistent, two
//           accumulators: large products, bound by the MMAs and L2's rate
//   single  128 columns x 32, 64 or 128 rows, K split over a cluster whose blocks
//           join their fp32 sums through distributed shared memory in rank order:
//           small and skinny products, bound by the codes' bytes or latency
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <type_traits>

#include "hgemm_tcgen05.cuh"
#include "mx_format.cuh"

namespace gb300 {
namespace {

constexpr int MM_K = 64;          // k of a stage: a 128-byte row of 16-bit values
constexpr int MM_CONV = 8;        // converter warps
constexpr int MM_EPI = 4;
constexpr int MM_THREADS = 32 * (2 + MM_EPI + MM_CONV);
constexpr int MM_W_BYTES = 128 * 128;
constexpr int MM_S_BYTES = 1024;  // up to two scale tiles
constexpr int MM_MAX_STAGES = 6;
constexpr int MM_FIXED = 1024 + 512;

template <int FMT>
__host__ __device__ constexpr int mm_code_bytes() { return FMT == MX_INT8 ? 128 * MM_K : 64 * MM_K; }
// scale tiles of a stage: along K (w stored [N, K]) one; along N (stored [K, N])
// 128 columns are four blocks of 32, or eight of 16
template <int FMT, bool W_MN>
__host__ __device__ constexpr int mm_scale_tiles() { return W_MN && FMT == MX_FP4_E4M3 ? 2 : 1; }

struct MixedParams {
  int M, N, K;
  int mt;              // rows of C a tile covers (pairs: 256)
  int x_bytes;         // A's tile in a block's stage
  int ring;            // stages
  int steps;           // k stages in all
  int per;             // of a block (its slice)
  int tiles_m, tiles_n, tiles;
  void* C;
  int64_t ldc;
  float alpha, beta;
  Epilogue ep;
  unsigned int* status;
  uint64_t timeout_ns;
  int fault_injection;
};

// acquire at cluster scope: arrivals may come from the pair's other block, with
// shared memory it wrote
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  if (!mbar_wait(bar, parity, w)) return false;
  return mbar_try_wait_cluster(bar, parity);  // (the phase is complete: returns at once)
}

// 32 codes of one row -> 16 words of T values.  `codes`: 16 bytes of e2m1 pairs
// or 32 signed bytes; b0, b1 the scale bytes of its first and second 16 (equal
// for 32-wide blocks).  One rounding, to T, and that exact but where T's range
// ends.
template <typename T, int FMT>
__device__ __forceinline__ void convert32(const uint32_t (&codes)[FMT == MX_INT8 ? 8 : 4],
                                          uint32_t b0, uint32_t b1, uint32_t (&out)[16]) {
  constexpr bool HALF = std::is_same<T, __half>::value;
  if constexpr (FMT == MX_INT8) {
    // fp16, scale 2^-14 .. 2: (1024 + 128 + code) s - 1152 s in one exact FMA
    if (HALF && b0 - 113u < 16u) {
      const uint32_t sb = (b0 - 112u) << 10, s2 = sb | (sb << 16);
      const __half2 s = *reinterpret_cast<const __half2*>(&s2);
      const __half2 off = __hmul2(s, __float2half2_rn(-1152.f));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w = codes[i] ^ 0x80808080u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t v = __byte_perm(w, 0x64646464u, j ? 0x4342 : 0x4140);
          const __half2 x = __hfma2(*reinterpret_cast<const __half2*>(&v), s, off);
          out[2 * i + j] = *reinterpret_cast<const uint32_t*>(&x);
        }
      }
      return;
    }
  } else if (HALF) {
    // fp16: e4m3 scales, and powers of two 2^-14 .. 2^15, are fp16 numbers, and
    // the product has at most six significant bits
    if (FMT == MX_FP4_E4M3 || b0 - 113u < 30u) {
      uint32_t s0, s1;
      if (FMT == MX_FP4_E4M3) {
        const __half_raw h0 = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b0, __NV_E4M3);
        const __half_raw h1 = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b1, __NV_E4M3);
        s0 = h0.x * 0x10001u;
        s1 = h1.x * 0x10001u;
      } else {
        s0 = s1 = ((b0 - 112u) << 10) * 0x10001u;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h[4];
        e2m1_halves(codes[i], h);
        const uint32_t sw = i < 2 ? s0 : s1;
        const __half2 s = *reinterpret_cast<const __half2*>(&sw);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&h[j]), s);
          out[4 * i + j] = *reinterpret_cast<const uint32_t*>(&x);
        }
      }
      return;
    }
  }
  // bf16, and scales that are no normal fp16 number: through fp32
  const float s0 = mx_scale_value<FMT>(b0), s1 = mx_scale_value<FMT>(b1);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    MxCodes<FMT> c;
#pragma unroll
    for (int i = 0; i < MxCodes<FMT>::WORDS; ++i) c.w[i] = codes[h * MxCodes<FMT>::WORDS + i];
    float v[16];
    mx_decode16<FMT>(c, h ? s1 : s0, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const typename Elem<T>::T2 p = Elem<T>::pack(v[2 * i], v[2 * i + 1]);
      out[8 * h + i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
}

// W_MN: the codes are stored [K, N]; X_MN: A is stored [K, M]
template <typename T, int FMT, bool W_MN, bool X_MN, bool PAIR>
__global__ void __launch_bounds__(MM_THREADS, 1)
    mx_mixed_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmS, const MixedParams p) {
  constexpr int CODE_BYTES = mm_code_bytes<FMT>();
  constexpr int STILES = mm_scale_tiles<FMT, W_MN>();
  const int stage_bytes = MM_W_BYTES + p.x_bytes + CODE_BYTES + MM_S_BYTES;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;       // block of a pair
  const int slice = PAIR ? 0 : (int)blockIdx.x;             // block of a split cluster
  const int splits = PAIR ? 1 : (int)gridDim.x;
  const int worker = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.y;
  const int workers = PAIR ? (int)(gridDim.x >> 1) : p.tiles;  // (single: one tile a cluster)
  const int k_lo = slice * p.per, k_hi = min(p.steps, k_lo + p.per);
  const int nk = k_hi - k_lo;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - smem_u32(smem_raw));
  uint64_t* const bars = reinterpret_cast<uint64_t*>(base_ptr + p.ring * stage_bytes);
  const uint32_t bar0 = smem_u32(bars);
  // this block's codes and scales landed; A's tile landed (pairs: both blocks',
  // on the even block); codes converted (pairs: both blocks', there too); the
  // MMAs that read the stage finished
  auto code_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto x_bar = [&](int s) { return bar0 + 8u * (uint32_t)(MM_MAX_STAGES + s); };
  auto conv_bar = [&](int s) { return bar0 + 8u * (uint32_t)(2 * MM_MAX_STAGES + s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(3 * MM_MAX_STAGES + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (uint32_t)(4 * MM_MAX_STAGES + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (uint32_t)(4 * MM_MAX_STAGES + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (uint32_t)(4 * MM_MAX_STAGES + 4);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * MM_MAX_STAGES + 5);
  volatile uint32_t* const abort_flag = tmem_slot + 1;
  static_assert(8 * (4 * MM_MAX_STAGES + 6) <= 512, "barrier area");
  auto w_at = [&](int s) { return base + (uint32_t)(s * stage_bytes); };
  auto x_at = [&](int s) { return w_at(s) + (uint32_t)MM_W_BYTES; };
  auto c_at = [&](int s) { return x_at(s) + (uint32_t)p.x_bytes; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem_cols = PAIR ? 512u : (uint32_t)p.mt;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(code_bar(s), 1);
      mbar_init(x_bar(s), 1);
      mbar_init(conv_bar(s), (PAIR ? 2 : 1) * MM_CONV);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), (PAIR ? 2 : 1) * 32 * MM_EPI);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), tmem_cols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), tmem_cols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{p.status, abort_flag, p.timeout_ns};

  // tile t: columns n0 of this block, rows m0 (row tiles innermost: the blocks
  // that run together read few columns' codes and all of A)
  auto origin = [&](int t, int& n0, int& m0) {
    const int tn = t / p.tiles_m;
    n0 = (PAIR ? 2 * tn + rank : tn) * 128;
    m0 = (t - tn * p.tiles_m) * p.mt;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmX);
      tma_prefetch_desc(&tmW);
      tma_prefetch_desc(&tmS);
      int stage = 0;
      uint32_t phase = 0, pending = 0, pend_phase = 0;
      bool ok = true, first = true;
      for (int t = worker; ok && t < p.tiles; t += workers) {
        int n0, m0;
        origin(t, n0, m0);
        for (int k = k_lo; k < k_hi; ++k) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, wc)) { ok = false; break; }
          const bool skip = first && p.fault_injection == 1;
          first = false;
          if (skip) {
            pending &= ~(1u << stage);
          } else {
            const uint32_t x = x_at(stage), c = c_at(stage), s = c + (uint32_t)CODE_BYTES;
            const uint32_t cb = code_bar(stage);
            mbar_arrive_expect_tx(cb, (uint32_t)(CODE_BYTES + STILES * 512));
            if constexpr (W_MN) {
              tma_load_3d(c, &tmW, FMT == MX_INT8 ? n0 : n0 / 2, k * MM_K, 0, cb);
              tma_load_3d(s, &tmS, 0, (n0 >> 7) * STILES, (k * MM_K) >> 7, cb);
            } else {
              tma_load_3d(c, &tmW, FMT == MX_INT8 ? k * MM_K : k * MM_K / 2, n0, 0, cb);
              tma_load_3d(s, &tmS, 0, k * MM_K / (4 * mx_block(FMT)), n0 >> 7, cb);
            }
            const int mx = m0 + (PAIR ? rank * 128 : 0);
            if constexpr (PAIR) {
              const uint32_t xb = mapa_shared(x_bar(stage), 0u);
              if (rank == 0) mbar_arrive_expect_tx(x_bar(stage), 2u * (uint32_t)p.x_bytes);
              if constexpr (X_MN) {
                tma_load_3d_pair(x, &tmX, mx, k * MM_K, 0, xb);
                tma_load_3d_pair(x + 8192u, &tmX, mx + 64, k * MM_K, 0, xb);
              } else {
                tma_load_3d_pair(x, &tmX, k * MM_K, mx, 0, xb);
              }
            } else {
              const uint32_t xb = x_bar(stage);
              mbar_arrive_expect_tx(xb, (uint32_t)p.x_bytes);
              if constexpr (X_MN) {
                for (int h = 0; h < p.x_bytes / 8192; ++h)
                  tma_load_3d(x + (uint32_t)(h * 8192), &tmX, mx + 64 * h, k * MM_K, 0, xb);
              } else {
                tma_load_3d(x, &tmX, k * MM_K, mx, 0, xb);
              }
            }
            pending |= 1u << stage;
            pend_phase = (pend_phase & ~(1u << stage)) | (phase << stage);
          }
          if (++stage == p.ring) { stage = 0; phase ^= 1u; }
        }
      }
      // every load issued lands before shared memory is released
      for (int s = 0; s < p.ring; ++s)
        if (pending & (1u << s)) {
          mbar_wait_drain(code_bar(s), (pend_phase >> s) & 1u, p.timeout_ns);
          if (rank == 0) mbar_wait_drain(x_bar(s), (pend_phase >> s) & 1u, p.timeout_ns);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // (the warp stays converged; see mx4_tcgen05.cu on uniform operands)
    if (rank == 0) {
      uint32_t lead;
      asm volatile(
          "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(lead));
      const bool leader = lead != 0;
      // D fp32, A and B of T, majors, N = mt, M = 128 or 256
      const uint32_t idesc = (1u << 4) | (Elem<T>::FMT << 7) | (Elem<T>::FMT << 10) |
                             ((W_MN ? 1u : 0u) << 15) | ((X_MN ? 1u : 0u) << 16) |
                             ((uint32_t)(p.mt >> 3) << 17) | ((PAIR ? 16u : 8u) << 24);
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int t = worker; ok && t < p.tiles; t += workers, ++it) {
        const int buf = it & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(acce_bar(buf), ((uint32_t)(it >> 1) & 1u) ^ 1u, wc));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(PAIR ? buf * 256 : 0);
        for (int k = 0; k < nk; ++k) {
          ok = __all_sync(0xffffffffu, mbar_wait(x_bar(stage), phase, wc) &&
                                           mbar_wait_cluster(conv_bar(stage), phase, wc));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint32_t w = w_at(stage), x = x_at(stage);
#pragma unroll
            for (int kk = 0; kk < MM_K / 16; ++kk) {
              const uint64_t ad = W_MN ? make_sdesc(w + (uint32_t)kk * 2048u, 8192u, 1024u)
                                       : make_sdesc(w + (uint32_t)kk * 32u, 16u, 1024u);
              const uint64_t bd = X_MN ? make_sdesc(x + (uint32_t)kk * 2048u, 8192u, 1024u)
                                       : make_sdesc(x + (uint32_t)kk * 32u, 16u, 1024u);
              const uint32_t acc = (k | kk) != 0 ? 1u : 0u;
              if constexpr (PAIR) tc_mma_f16_pair(d, ad, bd, idesc, acc);
              else tc_mma_f16(d, ad, bd, idesc, acc);
            }
            if constexpr (PAIR) tc_commit_pair_mc(empty_bar(stage), (uint16_t)3u);
            else tc_commit(empty_bar(stage));
          }
          __syncwarp();
          if (++stage == p.ring) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (leader) {
          if constexpr (PAIR) tc_commit_pair_mc(accf_bar(buf), (uint16_t)3u);
          else tc_commit(accf_bar(buf));
        }
        __syncwarp();
      }
      if (leader) {
        if constexpr (PAIR) tc_commit_pair_mc(drain_bar, (uint16_t)1u);
        else tc_commit(drain_bar);
        mbar_wait_drain(drain_bar, 0u, p.timeout_ns);
      }
      __syncwarp();
    }
  } else if (warp < 2 + MM_EPI) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    int it = 0;
    for (int t = worker; t < p.tiles; t += workers, ++it) {
      int n0, m0;
      origin(t, n0, m0);
      const int buf = it & 1;
      bool got = false;
      if (lane == 0) got = mbar_wait(accf_bar(buf), (uint32_t)(it >> 1) & 1u, wc);
      got = __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
      if (!got) break;
      tc_fence_after();
      const uint32_t row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(PAIR ? buf * 256 : 0);
      const int n = n0 + 32 * q + lane;  // this lane's column of C
      const int chunks = min(p.mt, p.M - m0 + 31) / 32;
      T* const col = static_cast<T*>(p.C) + n;
      float bias = 0.f;
      if (p.ep.bias != nullptr && n < p.N) bias = bias_value(static_cast<const T*>(p.ep.bias), n);
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(row + (uint32_t)(c * 32), r);
        tmem_ld_wait();
        if (splits > 1) {
          // fp32 sums [row of C][column], in the ring: every stage was consumed
#pragma unroll
          for (int j = 0; j < 32; ++j)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(
                             base + (uint32_t)(((c * 32 + j) * 128 + 32 * q + lane) * 4)),
                         "r"(r[j])
                         : "memory");
          continue;
        }
        const int mc = min(32, p.M - m0 - c * 32);
        if (n < p.N) {
          T* dst = col + (int64_t)(m0 + c * 32) * p.ldc;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (j < mc) {
              float v = p.alpha * __uint_as_float(r[j]);
              if (p.beta != 0.f) v = __fmaf_rn(p.beta, Elem<T>::to(*dst), v);
              *dst = Elem<T>::from(apply_act(v + bias, p.ep.act));
            }
            dst += p.ldc;
          }
        }
      }
      tc_fence_before();
      if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(acce_bar(buf), 0u));
      else mbar_arrive(acce_bar(buf));
    }
  } else {
    // ------------------------------------------------------------ converters
    const int ct = threadIdx.x - 32 * (2 + MM_EPI);  // 0 .. 255
    // stored [N, K]: row ct / 2, 32 codes of K from 32 (ct & 1);
    // stored [K, N]: k row (ct % 128) / 2, 32 columns from 32 seg
    const int r = W_MN ? (ct & 127) >> 1 : ct >> 1;
    const int seg = W_MN ? 2 * (ct >> 7) + (ct & 1) : (ct & 1);
    constexpr int B32 = FMT == MX_INT8 ? 32 : 16;  // bytes of 32 codes
    const uint32_t from = (uint32_t)(r * (W_MN ? 4 : 2) * B32 + seg * B32);
    const uint32_t to = W_MN ? (uint32_t)((seg >> 1) * 8192 + r * 128) : (uint32_t)(r * 128);
    const int chunk0 = W_MN ? 4 * (seg & 1) : 4 * seg;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = worker; ok && t < p.tiles; t += workers) {
      for (int k = k_lo; k < k_hi; ++k) {
        ok = false;
        if (lane == 0) ok = mbar_wait(code_bar(stage), phase, wc);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        const uint32_t c = c_at(stage), s = c + (uint32_t)CODE_BYTES;
        uint32_t codes[FMT == MX_INT8 ? 8 : 4];
#pragma unroll
        for (int i = 0; i < B32 / 16; ++i)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(codes[4 * i]), "=r"(codes[4 * i + 1]), "=r"(codes[4 * i + 2]),
                         "=r"(codes[4 * i + 3])
                       : "r"(c + from + (uint32_t)(16 * i)));
        // the block of this thread's codes (two of 16), and the row, in the tiles
        const int tr = W_MN ? ((k * MM_K) & 127) + r : r;
        const int blk = FMT == MX_FP4_E4M3 ? 2 * seg
                        : W_MN             ? seg
                                           : ((k * MM_K) >> 5 & 3) + seg;
        uint32_t word;
        asm volatile("ld.shared.b32 %0, [%1];"
                     : "=r"(word)
                     : "r"(s + (uint32_t)((blk >> 2) * 512 + (tr & 31) * 16 + (tr >> 5) * 4)));
        const uint32_t b0 = (word >> (8 * (blk & 3))) & 255u;
        const uint32_t b1 = FMT == MX_FP4_E4M3 ? (word >> (8 * (blk & 3) + 8)) & 255u : b0;
        uint32_t out[16];
        convert32<T, FMT>(codes, b0, b1, out);
        const uint32_t w = w_at(stage) + to;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           w + (uint32_t)(((chunk0 + j) ^ (r & 7)) * 16)),
                       "r"(out[4 * j]), "r"(out[4 * j + 1]), "r"(out[4 * j + 2]),
                       "r"(out[4 * j + 3])
                       : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(conv_bar(stage), 0u));
          else mbar_arrive(conv_bar(stage));
        }
        if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      }
    }
  }

  tc_fence_before();
  // a pair leaves together; a split cluster joins its sums
  cluster_sync();
  if (!PAIR && splits > 1) {
    int n0, m0;
    origin(worker, n0, m0);
    const int q_lo = slice * 32 / splits, q_cnt = (slice + 1) * 32 / splits - q_lo;
    const int mc = min(p.mt, p.M - m0);
    for (int i = threadIdx.x; i < q_cnt * mc; i += MM_THREADS) {
      const int m = i / q_cnt, n = 4 * (q_lo + i % q_cnt);
      if (n0 + n >= p.N) continue;
      const float4 sum = cluster_sum4(base + (uint32_t)((m * 128 + n) * 4), splits);
      const float v4[4] = {sum.x, sum.y, sum.z, sum.w};
      T* const dst = static_cast<T*>(p.C) + (int64_t)(m0 + m) * p.ldc + n0 + n;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (n0 + n + e >= p.N) break;
        float v = p.alpha * v4[e];
        if (p.beta != 0.f) v = __fmaf_rn(p.beta, Elem<T>::to(dst[e]), v);
        dst[e] = Elem<T>::from(apply_epilogue<T>(v, p.ep, n0 + n + e));
      }
    }
    cluster_sync();  // no block leaves while its sums are read
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, tmem_cols);
    else tmem_dealloc(tmem_base, tmem_cols);
  }
}

// ---------------------------------------------------------------- host side
template <typename T, int FMT, bool W_MN, bool X_MN, bool PAIR>
cudaError_t launch_mixed_form(const MxStreamArgs& a, int mt, int want_splits, LaunchCtx& ctx) {
  auto kern = mx_mixed_kernel<T, FMT, W_MN, X_MN, PAIR>;
  constexpr int CODE_BYTES = mm_code_bytes<FMT>();
  MixedParams p;
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.mt = mt;
  const int x_rows = PAIR ? 128 : mt;
  p.x_bytes = X_MN ? (x_rows + 63) / 64 * 8192 : x_rows * 128;
  const int stage = MM_W_BYTES + p.x_bytes + CODE_BYTES + MM_S_BYTES;
  p.ring = (SMEM_LIMIT - MM_FIXED) / stage;
  if (p.ring > MM_MAX_STAGES) p.ring = MM_MAX_STAGES;
  p.steps = (a.K + MM_K - 1) / MM_K;
  p.per = (p.steps + want_splits - 1) / want_splits;
  const int splits = (p.steps + p.per - 1) / p.per;
  const int bn = PAIR ? 256 : 128;
  p.tiles_n = (int)(((int64_t)a.N + bn - 1) / bn);
  p.tiles_m = (int)(((int64_t)a.M + mt - 1) / mt);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > (PAIR ? (1 << 30) : 65535)) return cudaErrorNotSupported;
  p.tiles = (int)tiles;
  p.C = a.C; p.ldc = a.ldc;
  p.alpha = a.alpha; p.beta = a.beta;
  p.ep = a.ep;
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  p.fault_injection = a.fault_injection;
  const size_t smem = (size_t)p.ring * stage + MM_FIXED;
  static const cudaError_t attr =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT);
  if (attr != cudaSuccess) return attr;
  CUtensorMap mX, mW, mS;
  const CUtensorMapDataType U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapSwizzle NONE = CU_TENSOR_MAP_SWIZZLE_NONE;
  const int64_t wr = W_MN ? a.K : a.N, wc = W_MN ? a.N : a.K;
  const int64_t wbytes = FMT == MX_INT8 ? wc : (wc + 1) / 2;
  const int64_t stiles = mx_scale_tiles(FMT, (int)wc);
  const int row_codes = W_MN ? 128 : MM_K;  // codes of a box row
  bool ok = X_MN ? make_map(&mX, Elem<T>::TMA, a.A, a.K, a.M, a.lda, 64, MM_K)
                 : make_map(&mX, Elem<T>::TMA, a.A, a.M, a.K, a.lda, MM_K, x_rows);
  ok = ok && make_map(&mW, U8, a.B, wr, wbytes, a.ldb, FMT == MX_INT8 ? row_codes : row_codes / 2,
                      W_MN ? MM_K : 128, NONE, 1, 0, 1);
  ok = ok && make_map(&mS, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.Bs, stiles, 128, 128, 128,
                      mm_scale_tiles<FMT, W_MN>(), NONE, (wr + 127) / 128, stiles * 128, 4);
  if (!ok) return cudaErrorNotSupported;
  cudaError_t e;
  if (PAIR) {
    static std::atomic<int> pairs{0};
    int have = pairs.load(std::memory_order_relaxed);
    if (have == 0) {
      have = resident_clusters((const void*)kern, 2, MM_THREADS, smem);
      if (have <= 0) have = a.num_sms / 2;
      pairs.store(have, std::memory_order_relaxed);
    }
    const int workers = have < p.tiles ? have : p.tiles;
    ctx.grid = 2 * workers;
    e = launch_kernel(kern, dim3((unsigned)ctx.grid), dim3(MM_THREADS), smem, ctx.stream, 2, mX, mW,
                      mS, p);
  } else {
    ctx.grid = splits * p.tiles;
    e = launch_kernel(kern, dim3((unsigned)splits, (unsigned)p.tiles), dim3(MM_THREADS), smem,
                      ctx.stream, splits, mX, mW, mS, p);
  }
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

template <typename T, int FMT, bool W_MN, bool X_MN>
cudaError_t launch_mixed_v(const MxStreamArgs& a, LaunchCtx& ctx) {
  const MixedPlan pl = mixed_plan(a.M, a.N, a.K, a.num_sms);
  return pl.pair ? launch_mixed_form<T, FMT, W_MN, X_MN, true>(a, 256, 1, ctx)
                 : launch_mixed_form<T, FMT, W_MN, X_MN, false>(a, pl.mt, pl.splits, ctx);
}

template <typename T>
cudaError_t launch_mixed_t(const MxStreamArgs& a, LaunchCtx& ctx) {
  const bool fp4 = a.format == MX_FP4;
  if (a.format == MX_INT8)
    return a.transA && !a.transB ? launch_mixed_v<T, MX_INT8, true, true>(a, ctx)
                                 : cudaErrorNotSupported;
  if (a.transA) return cudaErrorNotSupported;
  if (a.transB)
    return fp4 ? launch_mixed_v<T, MX_FP4, false, false>(a, ctx)
               : launch_mixed_v<T, MX_FP4_E4M3, false, false>(a, ctx);
  return fp4 ? launch_mixed_v<T, MX_FP4, true, false>(a, ctx)
             : launch_mixed_v<T, MX_FP4_E4M3, true, false>(a, ctx);
}

}  // namespace
}  // namespace gb300
