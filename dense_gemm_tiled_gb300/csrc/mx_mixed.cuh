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
// A, and the accumulator is C transposed: lanes are columns of C, so a warp's
// stores cover 32 of them in a row.
//   warp 0        producer: TMA of A's tile (128-byte swizzle), the codes and
//                 their scale tiles, into a ring of stages of 64 k
//   warp 1        tensor memory, MMA issue
//   warps 2-5     epilogue
//   warps 6-15    converters: codes to 16-bit values in the swizzled K-major (nt)
//                 or MN-major (nn, tn) operand layout, in a ring of tiles of its
//                 own.  Five groups of two warps take the stages in turn, each
//                 with a tile of its own
// What bounds it is the chain of a stage: convert, fence to the tensor core's
// proxy, barrier, MMA, commit, barrier, about 2 us, of which five overlap: 0.4 us
// a stage (0.19 without conversion and MMAs).  Eight tiles for the five groups,
// with fewer stages of loads, measured the same to 20 % slower, all warps on each
// stage the same.
// One tile of C a cluster, K split over its blocks, which join their fp32 sums
// through distributed shared memory in rank order.  For up to a few hundred rows
// of A, where expanding the stored operand into scratch for the 16-bit kernels
// would move 4.5 times its bytes.  (For large products that expansion costs a few
// per cent and the 16-bit kernel's pairs of blocks feed the MMAs better: a form
// of this kernel on pairs reached 0.97 PFLOP/s at 4096^3 against 1.59.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "hgemm_tcgen05.cuh"
#include "mx_format.cuh"

namespace gb300 {
namespace {

constexpr int MM_K = 64;          // k of a stage: a 128-byte row of 16-bit values
constexpr int MM_CONV = 10;       // converter warps, in groups of
constexpr int MM_GROUP = 2;       // two: a group converts every fifth stage
constexpr int MM_GROUPS = MM_CONV / MM_GROUP;
constexpr int MM_EPI = 4;
constexpr int MM_THREADS = 32 * (2 + MM_EPI + MM_CONV);
constexpr int MM_W_BYTES = 128 * 128;
constexpr int MM_S_BYTES = 1024;  // up to two scale tiles
constexpr int MM_MAX_STAGES = 12;
constexpr int MM_TILES = MM_GROUPS;   // converted tiles
constexpr int MM_FIXED = 1024 + 512;

template <int FMT>
__host__ __device__ constexpr int mm_code_bytes() { return FMT == MX_INT8 ? 128 * MM_K : 64 * MM_K; }
// scale tiles of a stage: along K (w stored [N, K]) one; along N (stored [K, N])
// 128 columns are four blocks of 32, or eight of 16
template <int FMT, bool W_MN>
__host__ __device__ constexpr int mm_scale_tiles() { return W_MN && FMT == MX_FP4_E4M3 ? 2 : 1; }

struct MixedParams {
  int M, N, K;
  int mt;              // rows of C a tile covers
  int x_bytes;         // A's tile in a block's stage
  int ring;            // stages of loads
  int steps;           // k stages in all
  int per;             // of a block (its slice)
  int tiles_m;
  void* C;
  int64_t ldc;
  float alpha, beta;
  Epilogue ep;
  unsigned int* status;
  uint64_t timeout_ns;
  int fault_injection;
};

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
template <typename T, int FMT, bool W_MN, bool X_MN>
__global__ void __launch_bounds__(MM_THREADS, 1)
    mx_mixed_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmS, const MixedParams p) {
  constexpr int CODE_BYTES = mm_code_bytes<FMT>();
  constexpr int STILES = mm_scale_tiles<FMT, W_MN>();
  const int stage_bytes = p.x_bytes + CODE_BYTES + MM_S_BYTES;
  const int slice = (int)blockIdx.x, splits = (int)gridDim.x;  // a cluster is a row of the grid
  const int k_lo = slice * p.per, k_hi = min(p.steps, k_lo + p.per);
  const int nk = k_hi - k_lo;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - smem_u32(smem_raw));
  uint64_t* const bars =
      reinterpret_cast<uint64_t*>(base_ptr + MM_TILES * MM_W_BYTES + p.ring * stage_bytes);
  const uint32_t bar0 = smem_u32(bars);
  // codes and scales landed; A's tile landed; the MMAs that read the stage
  // finished; codes converted; the MMAs that read the converted tile finished
  auto code_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto x_bar = [&](int s) { return bar0 + 8u * (uint32_t)(MM_MAX_STAGES + s); };
  auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(2 * MM_MAX_STAGES + s); };
  constexpr int B1 = 3 * MM_MAX_STAGES;
  auto conv_bar = [&](int w) { return bar0 + 8u * (uint32_t)(B1 + w); };
  auto free_bar = [&](int w) { return bar0 + 8u * (uint32_t)(B1 + MM_TILES + w); };
  constexpr int B2 = B1 + 2 * MM_TILES;
  const uint32_t acc_bar = bar0 + 8u * (uint32_t)B2;
  const uint32_t drain_bar = bar0 + 8u * (uint32_t)(B2 + 1);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + B2 + 2);
  volatile uint32_t* const abort_flag = tmem_slot + 1;
  static_assert(8 * (B2 + 3) <= 512, "barrier area");
  auto w_at = [&](int w) { return base + (uint32_t)(w * MM_W_BYTES); };
  auto x_at = [&](int s) {
    return base + (uint32_t)(MM_TILES * MM_W_BYTES) + (uint32_t)(s * stage_bytes);
  };
  auto c_at = [&](int s) { return x_at(s) + (uint32_t)p.x_bytes; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem_cols = (uint32_t)p.mt;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(code_bar(s), 1);
      mbar_init(x_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int w = 0; w < MM_TILES; ++w) {
      mbar_init(conv_bar(w), MM_GROUP);
      mbar_init(free_bar(w), 1);
    }
    mbar_init(acc_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{p.status, abort_flag, p.timeout_ns};

  // the cluster's tile: columns n0, rows m0 (row tiles innermost: the blocks that
  // run together read few columns' codes and all of A)
  const int n0 = (int)blockIdx.y / p.tiles_m * 128, m0 = (int)blockIdx.y % p.tiles_m * p.mt;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    {
      const bool leader = elect_one();
      if (leader) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmS);
      }
      __syncwarp();
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
          const uint32_t x = x_at(stage), c = c_at(stage), s = c + (uint32_t)CODE_BYTES;
          const uint32_t cb = code_bar(stage), xb = x_bar(stage);
          mbar_arrive_expect_tx(cb, (uint32_t)(CODE_BYTES + STILES * 512));
          if constexpr (W_MN) {
            tma_load_3d(c, &tmW, FMT == MX_INT8 ? n0 : n0 / 2, k * MM_K, 0, cb);
            tma_load_3d(s, &tmS, 0, (n0 >> 7) * STILES, (k * MM_K) >> 7, cb);
          } else {
            tma_load_3d(c, &tmW, FMT == MX_INT8 ? k * MM_K : k * MM_K / 2, n0, 0, cb);
            tma_load_3d(s, &tmS, 0, k * MM_K / (4 * mx_block(FMT)), n0 >> 7, cb);
          }
          mbar_arrive_expect_tx(xb, (uint32_t)p.x_bytes);
          if constexpr (X_MN) {
            for (int h = 0; h < p.x_bytes / 8192; ++h)
              tma_load_3d(x + (uint32_t)(h * 8192), &tmX, m0 + 64 * h, k * MM_K, 0, xb);
          } else {
            tma_load_3d(x, &tmX, k * MM_K, m0, 0, xb);
          }
        }
        __syncwarp();
        if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      }
      // every load issued lands before shared memory is released
      for (int s = 0; s < p.ring; ++s)
        if (pending & (1u << s)) {
          mbar_wait_drain(code_bar(s), (pend_phase >> s) & 1u, p.timeout_ns);
          mbar_wait_drain(x_bar(s), (pend_phase >> s) & 1u, p.timeout_ns);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    // D fp32, A and B of T, majors, N = mt, M = 128
    const uint32_t idesc = (1u << 4) | (Elem<T>::FMT << 7) | (Elem<T>::FMT << 10) |
                           ((W_MN ? 1u : 0u) << 15) | ((X_MN ? 1u : 0u) << 16) |
                           ((uint32_t)(p.mt >> 3) << 17) | (8u << 24);
    int stage = 0, slot = 0;
    uint32_t phase = 0, wphase = 0;
    bool ok = true;
    for (int k = 0; k < nk; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(x_bar(stage), phase, wc) &&
                                       mbar_wait(conv_bar(slot), wphase, wc));
      if (!ok) break;
      tc_fence_after();
      if (leader) {
        const uint32_t w = w_at(slot), x = x_at(stage);
#pragma unroll
        for (int kk = 0; kk < MM_K / 16; ++kk) {
          const uint64_t ad = W_MN ? make_sdesc(w + (uint32_t)kk * 2048u, 8192u, 1024u)
                                   : make_sdesc(w + (uint32_t)kk * 32u, 16u, 1024u);
          const uint64_t bd = X_MN ? make_sdesc(x + (uint32_t)kk * 2048u, 8192u, 1024u)
                                   : make_sdesc(x + (uint32_t)kk * 32u, 16u, 1024u);
          tc_mma_f16(tmem_base, ad, bd, idesc, (k | kk) != 0 ? 1u : 0u);
        }
        tc_commit(free_bar(slot));
        tc_commit(empty_bar(stage));
      }
      __syncwarp();
      if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      if (++slot == MM_TILES) { slot = 0; wphase ^= 1u; }
    }
    if (leader) {
      if (ok) tc_commit(acc_bar);
      tc_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0u, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp < 2 + MM_EPI) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    bool got = false;
    if (lane == 0) got = mbar_wait(acc_bar, 0u, wc);
    got = __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
    if (got) {
      tc_fence_after();
      const uint32_t row = tmem_base + ((uint32_t)(q * 32) << 16);
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
          // fp32 sums [row of C][column], over the converted tiles: the MMAs are done
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
    }
  } else {
    // ------------------------------------------------------------ converters
    // A thread of a group of 64 takes four runs of 32 codes of a stage:
    //   stored [N, K]: rows r, r + 32, r + 64, r + 96, 32 codes of K from 32 seg
    //   stored [K, N]: k rows r, r + 32, 32 columns from 32 seg and 32 (seg + 2)
    const int ct = (threadIdx.x - 32 * (2 + MM_EPI)) & (32 * MM_GROUP - 1);
    const int group = (warp - 2 - MM_EPI) / MM_GROUP;
    const int r = ct >> 1, seg = ct & 1;
    constexpr int B32 = FMT == MX_INT8 ? 32 : 16;  // bytes of 32 codes
    constexpr int ROW = (W_MN ? 4 : 2) * B32;      // of a row of codes
    const uint32_t from = (uint32_t)(r * ROW + seg * B32);
    const uint32_t to = (uint32_t)(r * 128);
    int stage = 0, turn = 0;
    uint32_t phase = 0, wphase = 1;
    for (int k = k_lo; k < k_hi; ++k) {
      const int st = stage;
      const uint32_t ph = phase;
      if (++stage == p.ring) { stage = 0; phase ^= 1u; }
      const bool mine = turn == group;
      if (++turn == MM_GROUPS) turn = 0;
      if (!mine) continue;
      // (the tile first: with the MMAs of the stage before this group's done, the
      // codes of that stage and of all before it have landed, so that the load
      // barrier is at most one phase behind, the ring having at least as many
      // stages as there are groups)
      bool ok = false;
      if (lane == 0) ok = mbar_wait(free_bar(group), wphase, wc) && mbar_wait(code_bar(st), ph, wc);
      wphase ^= 1u;
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      const uint32_t c = c_at(st), s = c + (uint32_t)CODE_BYTES;
      uint32_t codes[4][FMT == MX_INT8 ? 8 : 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = c + from +
                            (uint32_t)(W_MN ? (i & 1) * 32 * ROW + (i >> 1) * 2 * B32 : i * 32 * ROW);
#pragma unroll
        for (int h = 0; h < B32 / 16; ++h)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(codes[i][4 * h]), "=r"(codes[i][4 * h + 1]),
                         "=r"(codes[i][4 * h + 2]), "=r"(codes[i][4 * h + 3])
                       : "r"(at + (uint32_t)(16 * h)));
      }
      // the runs' scale words: rows 32 apart are neighbours in a scale tile
      uint32_t word[4];
      if constexpr (W_MN) {
        const uint32_t at = s + (uint32_t)(r * 16 + ((k * MM_K) & 127) / 32 * 4);
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(word[0]), "=r"(word[1]) : "r"(at));
        word[2] = word[0];
        word[3] = word[1];
        if constexpr (STILES == 2)
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                       : "=r"(word[2]), "=r"(word[3])
                       : "r"(at + 512u));
      } else {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(word[0]), "=r"(word[1]), "=r"(word[2]), "=r"(word[3])
                     : "r"(s + (uint32_t)(r * 16)));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the run's block (the first of two 16-wide ones) within its word
        const int blk = FMT == MX_FP4_E4M3 ? 2 * seg
                        : W_MN             ? seg + 2 * (i >> 1)
                                           : ((k * MM_K) >> 5 & 3) + seg;
        const uint32_t b0 = (word[i] >> (8 * blk)) & 255u;
        const uint32_t b1 = FMT == MX_FP4_E4M3 ? (word[i] >> (8 * blk + 8)) & 255u : b0;
        uint32_t out[16];
        convert32<T, FMT>(codes[i], b0, b1, out);
        const uint32_t w = w_at(group) + to +
                           (uint32_t)(W_MN ? (i >> 1) * 8192 + (i & 1) * 32 * 128 : i * 32 * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           w + (uint32_t)(((4 * seg + j) ^ (r & 7)) * 16)),
                       "r"(out[4 * j]), "r"(out[4 * j + 1]), "r"(out[4 * j + 2]),
                       "r"(out[4 * j + 3])
                       : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(conv_bar(group));
    }
  }

  tc_fence_before();
  cluster_sync();
  if (splits > 1) {  // join the slices' sums
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
    tmem_dealloc(tmem_base, tmem_cols);
  }
}

// ---------------------------------------------------------------- host side
template <typename T, int FMT, bool W_MN, bool X_MN>
cudaError_t launch_mixed_v(const MxStreamArgs& a, LaunchCtx& ctx) {
  auto kern = mx_mixed_kernel<T, FMT, W_MN, X_MN>;
  constexpr int CODE_BYTES = mm_code_bytes<FMT>();
  const MixedPlan pl = mixed_plan(a.M, a.N, a.K, a.num_sms);
  MixedParams p;
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.mt = pl.mt;
  p.x_bytes = X_MN ? (pl.mt + 63) / 64 * 8192 : pl.mt * 128;
  const int stage = p.x_bytes + CODE_BYTES + MM_S_BYTES;
  p.ring = (SMEM_LIMIT - MM_FIXED - MM_TILES * MM_W_BYTES) / stage;
  if (p.ring > MM_MAX_STAGES) p.ring = MM_MAX_STAGES;
  static_assert((SMEM_LIMIT - MM_FIXED - MM_TILES * MM_W_BYTES) /
                        (128 * 128 + CODE_BYTES + MM_S_BYTES) >= MM_GROUPS,
                "a ring of as many stages as there are groups, at the most rows");
  p.steps = (a.K + MM_K - 1) / MM_K;
  p.per = (p.steps + pl.splits - 1) / pl.splits;
  const int splits = (p.steps + p.per - 1) / p.per;
  p.tiles_m = (int)(((int64_t)a.M + pl.mt - 1) / pl.mt);
  const int64_t tiles = (int64_t)p.tiles_m * (((int64_t)a.N + 127) / 128);
  p.C = a.C; p.ldc = a.ldc;
  p.alpha = a.alpha; p.beta = a.beta;
  p.ep = a.ep;
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  p.fault_injection = a.fault_injection;
  const size_t smem = (size_t)MM_TILES * MM_W_BYTES + (size_t)p.ring * stage + MM_FIXED;
  static OncePerDevice set;
  const cudaError_t attr = set.run(call_device(), cudaSuccess, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT);
  });
  if (attr != cudaSuccess) return attr;
  CUtensorMap mX, mW, mS;
  const CUtensorMapDataType U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapSwizzle NONE = CU_TENSOR_MAP_SWIZZLE_NONE;
  const int64_t wr = W_MN ? a.K : a.N, wc = W_MN ? a.N : a.K;
  const int64_t wbytes = FMT == MX_INT8 ? wc : (wc + 1) / 2;
  const int64_t stiles = mx_scale_tiles(FMT, (int)wc);
  const int row_codes = W_MN ? 128 : MM_K;  // codes of a box row
  bool ok = X_MN ? make_map(&mX, Elem<T>::TMA, a.A, a.K, a.M, a.lda, 64, MM_K)
                 : make_map(&mX, Elem<T>::TMA, a.A, a.M, a.K, a.lda, MM_K, pl.mt);
  ok = ok && make_map(&mW, U8, a.B, wr, wbytes, a.ldb, FMT == MX_INT8 ? row_codes : row_codes / 2,
                      W_MN ? MM_K : 128, NONE, 1, 0, 1);
  ok = ok && make_map(&mS, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.Bs, stiles, 128, 128, 128,
                      mm_scale_tiles<FMT, W_MN>(), NONE, (wr + 127) / 128, stiles * 128, 4);
  if (!ok) return cudaErrorNotSupported;
  ctx.grid = (int)(splits * tiles);
  const cudaError_t e = launch_kernel(kern, dim3((unsigned)splits, (unsigned)tiles),
                                      dim3(MM_THREADS), smem, ctx.stream, splits, mX, mW, mS, p);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

template <typename T>
cudaError_t launch_mixed_t(const MxStreamArgs& a, LaunchCtx& ctx) {
  if (a.format == MX_INT8) return launch_mixed_v<T, MX_INT8, true, true>(a, ctx);
  const bool fp4 = a.format == MX_FP4;
  if (a.transB)
    return fp4 ? launch_mixed_v<T, MX_FP4, false, false>(a, ctx)
               : launch_mixed_v<T, MX_FP4_E4M3, false, false>(a, ctx);
  return fp4 ? launch_mixed_v<T, MX_FP4, true, false>(a, ctx)
             : launch_mixed_v<T, MX_FP4_E4M3, true, false>(a, ctx);
}

}  // namespace
}  // namespace gb300
