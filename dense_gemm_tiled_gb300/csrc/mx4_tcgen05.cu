// Product of two 4-bit microscaled operands on the 5th-generation tensor cores
// (block-scaled tcgen05.mma, accumulators in tensor memory):
//
//   C = act(alpha * A B^T + beta * C + bias),
//   (A B^T)_mn = sum_k sa[m, k/b] sb[n, k/b] qa[m, k] qb[n, k]
//
// with e2m1 codes q and b = 32 (power-of-two scales, kind::mxf4) or 16 (e4m3
// scales, kind::mxf4nvf4).  The tensor core multiplies each product of codes
// by both scales and accumulates in fp32, so a 4-bit product costs the same
// bytes of shared memory per instruction as a 16-bit one and does four times
// the multiply-adds.
//
// Structure (per block; the 16-bit kernel's, hgemm_tcgen05.cuh, with the
// scales added):
//   warp 0     producer: TMA tiles of codes (128 bytes = 256 codes a row, 128-
//              byte swizzle) and the scale tiles that go with them, as they lie
//              in memory, into one ring of stages
//   warp 1     tensor-memory allocation; per stage copies the scale tiles to
//              tensor memory (tcgen05.cp: 32 rows x 16 bytes onto 32 lanes x 4
//              columns, repeated to all four lane quarters) and issues the MMAs
//   warps 2..  epilogue
// Measured: 8192^3 fp4 to bf16 170 us (6.5 PFLOP/s) on pairs of 256 x 256, tensor
// pipe 75 % of SM-active cycles; the MMAs and scale copies without loads take 144.
// Two 128 x 128 or 256 x 128 tiles' accumulators fit beside the scales, one of 256
// x 256: its epilogue empties it into registers first, about 1 us a tile.
// The storage's scale tile is that copy's source as it lies in memory.  Each
// ring stage has scale columns of its own in tensor memory: a stage is refilled
// only after the MMAs that read it completed, so its columns are free then too.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include "hgemm_tcgen05.cuh"
#include "mx_format.cuh"

namespace gb300 {
namespace {

constexpr int KSTAGE = 256;   // codes of K a stage holds: one 128-byte swizzle row
constexpr int KMMA = 64;      // codes of K an MMA takes
constexpr int EPI = 8;        // epilogue warps: two per lane quarter, half of the columns each
constexpr int MX_THREADS = 64 + 32 * EPI;

template <int FMT, int BN, bool PAIR>
struct MxCfg {
  static constexpr int TPS = KSTAGE / mx_block(FMT) / 4;  // scale tiles of a stage and 128 rows
  static constexpr int NBLK = (BN + 127) / 128;           // 128-row ranges of B
  static constexpr int HALVES = BN >= 128 ? 2 : 1;        // epilogue warps in use per quarter
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = (PAIR ? BN / 2 : BN) * 128;
  static constexpr int SFA_BYTES = TPS * 512;
  static constexpr int SFB_BYTES = NBLK * TPS * 512;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int SF_BYTES = SFA_BYTES + SFB_BYTES;
  static constexpr int STAGING_BYTES = 4 * HALVES * 4096;
  static constexpr int FIXED = 1024 + 512;
  static constexpr int RAW = (SMEM_LIMIT - FIXED - STAGING_BYTES) / (STAGE_BYTES + SF_BYTES);
  static constexpr int SF_COLS = TPS * 4 * (1 + NBLK);    // tensor-memory columns of a stage
  // Accumulators: two, so that a tile's epilogue runs under the next tile's
  // main loop; one where two of 256 columns would leave no room for the scales
  // (the epilogue then takes the whole accumulator into registers first).
  static constexpr int NACC = BN == 256 ? 1 : 2;
  static constexpr int FIT = (512 - NACC * BN) / SF_COLS;
  static constexpr int STAGES = RAW < FIT ? (RAW < 8 ? RAW : 8) : (FIT < 8 ? FIT : 8);
  static_assert(STAGES >= 3, "ring");
  static constexpr int SMEM_BYTES = STAGES * (STAGE_BYTES + SF_BYTES) + STAGING_BYTES + FIXED;
};

struct MxTcParams {
  HParams h;           // sizes, schedule, C and epilogue (whole tiles only)
  int s_tiles;         // scale tiles of a 128-row range
  int stages_k;        // K stages of a tile
};

// Shared-memory descriptors as (low word, constant high word): the low word
// holds the address >> 4, so a step along K or a ring stage is an addition.
//   codes: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart
//   scale tile: no swizzle, 8-row groups 128 bytes apart
constexpr uint32_t CODES_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t SCALES_HI = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (1u << 16);
}

// 32 rows x 16 bytes of a scale tile -> 32 lanes x 4 columns, in each lane quarter
template <bool PAIR>
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint32_t lo) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(lo), "n"(SCALES_HI)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(lo), "n"(SCALES_HI)
        : "memory");
}

#define GB300_MX_MMA(GROUP, KIND)                                                       \
  asm volatile(                                                                         \
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"                                     \
      "setp.ne.b32 p, %4, 0;\n\t"                                                       \
      "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"                              \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND                                    \
      " [%0], da, db, %3, [%5], [%6], p;\n\t}" ::"r"(d),                                \
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb), "n"(CODES_HI)     \
      : "memory")
template <int FMT, bool PAIR>
__device__ __forceinline__ void tc_mma_mx4(uint32_t d, uint32_t a_lo, uint32_t b_lo,
                                           uint32_t idesc, uint32_t acc, uint32_t sfa,
                                           uint32_t sfb) {
  if constexpr (FMT == MX_FP4) {
    if constexpr (PAIR) GB300_MX_MMA("2", "mxf4.block_scale.scale_vec::2X");
    else GB300_MX_MMA("1", "mxf4.block_scale.scale_vec::2X");
  } else {
    if constexpr (PAIR) GB300_MX_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else GB300_MX_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  }
}
#undef GB300_MX_MMA

// Instruction descriptor of the block-scaled 4-bit kinds: scale-byte index of
// B (bits 4-5) and A (29-30) within the columns' words, A and B format (bits
// 7-9, 10-11: 1 = e2m1), N >> 3 (17-22), scale type (23: 1 = e8m0), M >> 4
// (24-28).
template <int FMT, int BN, int M_ROWS>
__device__ __forceinline__ constexpr uint32_t mx_idesc(uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
         ((FMT == MX_FP4 ? 1u : 0u) << 23) | ((uint32_t)(M_ROWS >> 4) << 24) | (sf_id << 29);
}

// One block-scaled product, 128 x BN a block or 256 x BN a pair of blocks
// (cta_group::2: each block holds its 128 rows of A and half of the B tile, and
// the scales of all of it).
template <typename T, int FMT, int BN, bool PAIR>
__global__ void __launch_bounds__(MX_THREADS, 1)
    mx4_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmSA,
                  const __grid_constant__ CUtensorMap tmSB,
                  const __grid_constant__ CUtensorMap tmC, const MxTcParams mp) {
  using C_ = MxCfg<FMT, BN, PAIR>;
  // bytes that complete a stage (a pair's: both blocks', on the even block's barrier)
  constexpr uint32_t STAGE_TX = (uint32_t)(C_::STAGE_BYTES + C_::SF_BYTES) * (PAIR ? 2u : 1u);
  constexpr int STAGES = C_::STAGES, TPS = C_::TPS, NBLK = C_::NBLK, NACC = C_::NACC;
  const HParams& p = mp.h;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;
  const int worker = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int workers = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t tiles_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* const tiles_ptr = smem_raw + (tiles_addr - raw_addr);
  const uint32_t staging_addr = tiles_addr + (uint32_t)(STAGES * C_::STAGE_BYTES);
  const uint32_t sf_addr = staging_addr + (uint32_t)C_::STAGING_BYTES;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(
      tiles_ptr + STAGES * (C_::STAGE_BYTES + C_::SF_BYTES) + C_::STAGING_BYTES);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(STAGES + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + NACC + b); };
  const uint32_t drain_bar = bar0 + 8u * (uint32_t)(2 * STAGES + 2 * NACC);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 2 * NACC + 1);
  volatile uint32_t* const abort_flag = tmem_slot + 1;
  static_assert(8 * (2 * STAGES + 2 * NACC + 2) <= 512, "barrier area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < NACC; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), (PAIR ? 2 : 1) * 32 * 4 * C_::HALVES);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), 512u);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512u);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t sf_tmem = tmem_base + (uint32_t)(NACC * BN);
  pdl_wait();
  pdl_trigger();

  const WaitCtl wc{p.status, abort_flag, p.timeout_ns};

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    {
      const bool leader = elect_one();
      if (leader) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSA);
        tma_prefetch_desc(&tmSB);
      }
      __syncwarp();
      int stage = 0;
      uint32_t phase = 0;
      uint32_t pending = 0, pend_phase = 0;
      bool ok = true, first = true;
      for (int t = worker; ok && t < p.tiles; t += workers) {
        int m0, n0, bz;
        tile_origin<PAIR, BN>(p, t, rank, m0, n0, bz);
        for (int kb = 0; kb < mp.stages_k; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, wc));
          if (!ok) break;
          const bool skip = first && p.fault_injection == 1;
          first = false;
          if (!skip) {
            const uint32_t sa = tiles_addr + (uint32_t)(stage * C_::STAGE_BYTES);
            const uint32_t sb = sa + (uint32_t)C_::A_BYTES;
            const uint32_t fa = sf_addr + (uint32_t)(stage * C_::SF_BYTES);
            const uint32_t fb = fa + (uint32_t)C_::SFA_BYTES;
            // scale tiles past a row's end, and rows past the last range, read
            // as zero
            const int t0 = kb * TPS, ra = m0 >> 7, rb = n0 >> 7;
            if (!leader) {
            } else if constexpr (PAIR) {
              const uint32_t bar = mapa_shared(full_bar(stage), 0u);
              if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), STAGE_TX);
              tma_load_3d_pair(sa, &tmA, kb * 128, m0, 0, bar);
              tma_load_3d_pair(sb, &tmB, kb * 128, n0 + rank * (BN / 2), 0, bar);
              tma_load_3d_pair(fa, &tmSA, 0, t0, ra, bar);
#pragma unroll
              for (int i = 0; i < NBLK; ++i)
                tma_load_3d_pair(fb + (uint32_t)(i * TPS * 512), &tmSB, 0, t0, rb + i, bar);
            } else {
              const uint32_t bar = full_bar(stage);
              mbar_arrive_expect_tx(bar, STAGE_TX);
              tma_load_3d(sa, &tmA, kb * 128, m0, 0, bar);
              tma_load_3d(sb, &tmB, kb * 128, n0, 0, bar);
              tma_load_3d(fa, &tmSA, 0, t0, ra, bar);
#pragma unroll
              for (int i = 0; i < NBLK; ++i)
                tma_load_3d(fb + (uint32_t)(i * TPS * 512), &tmSB, 0, t0, rb + i, bar);
            }
            pending |= 1u << stage;
            pend_phase = (pend_phase & ~(1u << stage)) | (phase << stage);
          } else {
            pending &= ~(1u << stage);
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // every load issued must land before the block can exit (a pair's land
      // on the even block's barriers, and the pair leaves together)
      if (rank == 0)
        for (int s = 0; s < STAGES; ++s)
          if (pending & (1u << s))
            mbar_wait_drain(full_bar(s), (pend_phase >> s) & 1u, p.timeout_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      const bool leader = elect_one();
      const uint32_t a_lo0 = desc_lo(tiles_addr), b_lo0 = desc_lo(tiles_addr + C_::A_BYTES);
      const uint32_t fa_lo0 = desc_lo(sf_addr), fb_lo0 = desc_lo(sf_addr + C_::SFA_BYTES);
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int t = worker; ok && t < p.tiles; t += workers, ++it) {
        const int buf = it % NACC;
        const uint32_t acc_phase = (uint32_t)(it / NACC) & 1u;
        ok = __all_sync(0xffffffffu, mbar_wait(acce_bar(buf), acc_phase ^ 1u, wc));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(buf * BN);
        // a 64-column tile may start in the middle of a 128-row range: its scale
        // columns start two words on
        int m0, n0, bz;
        tile_origin<PAIR, BN>(p, t, rank, m0, n0, bz);
        const uint32_t tb_off = (uint32_t)((n0 & 127) / 32);
        for (int kb = 0; kb < mp.stages_k; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, wc));
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_lo = a_lo0 + (uint32_t)(stage * (C_::STAGE_BYTES >> 4));
          const uint32_t b_lo = b_lo0 + (uint32_t)(stage * (C_::STAGE_BYTES >> 4));
          const uint32_t fa_lo = fa_lo0 + (uint32_t)(stage * (C_::SF_BYTES >> 4));
          const uint32_t fb_lo = fb_lo0 + (uint32_t)(stage * (C_::SF_BYTES >> 4));
          const uint32_t ta = sf_tmem + (uint32_t)(stage * C_::SF_COLS);
          const uint32_t tb = ta + (uint32_t)(TPS * 4);
          // tiles and MMAs past the end of K are left out (their scales do not exist)
          const int nt = mp.s_tiles - kb * TPS;
          const int nm = (p.K - kb * KSTAGE + KMMA - 1) / KMMA;
          if (leader) {
#pragma unroll
            for (int i = 0; i < TPS; ++i) {
              if (i >= nt) break;
              tc_cp_scales<PAIR>(ta + (uint32_t)(4 * i), fa_lo + (uint32_t)(32 * i));
#pragma unroll
              for (int r = 0; r < NBLK; ++r)
                tc_cp_scales<PAIR>(tb + (uint32_t)(4 * (i * NBLK + r)),
                                   fb_lo + (uint32_t)(32 * (r * TPS + i)));
            }
#pragma unroll
            for (int kk = 0; kk < KSTAGE / KMMA; ++kk) {
              if (kk >= nm) break;
              const int tile = kk * TPS / (KSTAGE / KMMA);             // its scale tile
              const uint32_t id = FMT == MX_FP4 ? 2u * (kk & 1) : 0u;  // and byte within the words
              tc_mma_mx4<FMT, PAIR>(d_tmem, a_lo + (uint32_t)(2 * kk), b_lo + (uint32_t)(2 * kk),
                                    mx_idesc<FMT, BN, PAIR ? 256 : 128>(id),
                                    (kb | kk) != 0 ? 1u : 0u, ta + (uint32_t)(4 * tile),
                                    tb + tb_off + (uint32_t)(4 * NBLK * tile));
            }
            if constexpr (PAIR) tc_commit_pair_mc(empty_bar(stage), (uint16_t)3u);
            else tc_commit(empty_bar(stage));
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
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
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;   // tensor-memory lanes 32q .. 32q + 31
    const int ew = warp - 2;
    const int hh = ew / 4;    // its share of the columns
    constexpr int CW = BN / C_::HALVES;        // columns of a share
    constexpr int KBOX = 128 / (int)sizeof(T);  // columns of a store box (128 bytes a row)
    const uint32_t sbuf = staging_addr + (uint32_t)(ew * 4096);
    auto release_acc = [&](int buf) {
      tc_fence_before();
      if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(acce_bar(buf), 0u));
      else mbar_arrive(acce_bar(buf));
    };
    const bool epi = p.ep.bias != nullptr || p.ep.act != 0;
    int it = 0;
    for (int t = worker; hh < C_::HALVES && t < p.tiles; t += workers, ++it) {
      int m0, n0, bz;
      tile_origin<PAIR, BN>(p, t, rank, m0, n0, bz);
      const int buf = it % NACC;
      const uint32_t acc_phase = (uint32_t)(it / NACC) & 1u;
      bool got = false;
      if (lane == 0) got = mbar_wait(accf_bar(buf), acc_phase, wc);
      got = __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
      if (!got) break;
      tc_fence_after();
      const int gn0 = n0 + hh * CW, gm0 = m0 + q * 32;
      const uint32_t t_row =
          tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN + hh * CW);
      if (p.c_tma && p.beta == 0.f) {
        // The share into registers, finished and rounded; the accumulator is
        // free from there on.
        uint32_t o[CW * (int)sizeof(T) / 4];
#pragma unroll
        for (int c = 0; c < CW / 32; ++c) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld_32x32b_x32(t_row + (uint32_t)(c * 32), r);
          tmem_ld_wait();
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = p.alpha * __uint_as_float(r[j]);
          if (epi) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (gn0 + c * 32 + j < p.N) v[j] = apply_epilogue<T>(v[j], p.ep, gn0 + c * 32 + j);
          }
          if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[c * 32 + j] = __float_as_uint(v[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const typename Elem<T>::T2 h = Elem<T>::pack(v[2 * j], v[2 * j + 1]);
              o[c * 16 + j] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
        }
        release_acc(buf);
        // 32-row boxes through this warp's staging buffer (128-byte swizzle:
        // 16-byte chunk w of row l at chunk w ^ (l & 7))
#pragma unroll
        for (int b = 0; b < CW / KBOX; ++b) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int w = 0; w < 8; ++w)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             sbuf + (uint32_t)(lane * 128 + ((w ^ (lane & 7)) * 16))),
                         "r"(o[b * 32 + 4 * w]), "r"(o[b * 32 + 4 * w + 1]),
                         "r"(o[b * 32 + 4 * w + 2]), "r"(o[b * 32 + 4 * w + 3])
                         : "memory");
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && gm0 < p.M && gn0 + b * KBOX < p.N) {
            tma_store_3d(&tmC, gn0 + b * KBOX, gm0, 0, sbuf);
            bulk_commit();
          }
        }
        continue;
      }
      // C read (beta), or rows off 16-byte alignment
      const int gm = gm0 + lane;
#pragma unroll 1
      for (int c = 0; c < CW / 32; ++c) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(t_row + (uint32_t)(c * 32), r);
        tmem_ld_wait();
        if (c == CW / 32 - 1) release_acc(buf);
        if (!p.c_vec_ok) {
          if (gm0 < p.M) store_c32_staged<T>(p, 0, gm0, gn0 + c * 32, sbuf, r, lane);
          continue;
        }
        if (gm >= p.M) continue;
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        store_c32<T>(p, 0, gm, gn0 + c * 32, v);
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  if constexpr (PAIR) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, 512u);
    else tmem_dealloc(tmem_base, 512u);
  }
}

// ---------------------------------------------------------------- host side
// Scale tiles as [128-row range][tile][128 words], loaded `box` tiles at a time.
bool scale_map(CUtensorMap* m, const void* s, int64_t rows, int64_t tiles, int box) {
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, s, tiles, 128, 128, 128, box,
                  CU_TENSOR_MAP_SWIZZLE_NONE, (rows + 127) / 128, tiles * 128, 4);
}

// Blocks (or pairs) resident at once: an SM each (pairs: as many as the GPU's
// clusters of two allow, queried once a device).
template <typename T, int FMT, int BN, bool PAIR>
int mx4_slots(int num_sms) {
  if (!PAIR) return num_sms;
  static CountPerDevice slots;
  const int n = slots.get(call_device(), [num_sms] {
    return resident_clusters((const void*)mx4_tc_kernel<T, FMT, BN, PAIR>, 2, MX_THREADS,
                             MxCfg<FMT, BN, PAIR>::SMEM_BYTES, dim3(2 * (num_sms / 2)));
  });
  return n > 0 ? n : num_sms / 2;
}

template <typename T, int FMT, int BN, bool PAIR>
cudaError_t launch_mx4_cfg(const Mx4Args& a, LaunchCtx& ctx) {
  using C_ = MxCfg<FMT, BN, PAIR>;
  auto kern = mx4_tc_kernel<T, FMT, BN, PAIR>;
  static OncePerDevice set;
  const cudaError_t attr = set.run(call_device(), cudaSuccess, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C_::SMEM_BYTES);
  });
  if (attr != cudaSuccess) return attr;
  MxTcParams mp;
  memset(&mp, 0, sizeof(mp));
  HParams& p = mp.h;
  p.C = a.C; p.ldc = a.ldc;
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.tiles_m = (a.M + 127) / 128;
  p.tiles_n = (a.N + BN - 1) / BN;
  const int64_t tiles = (int64_t)(PAIR ? (p.tiles_m + 1) / 2 : p.tiles_m) * p.tiles_n;
  if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  p.tiles = (int)tiles;
  p.alpha = a.alpha; p.beta = a.beta;
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  p.fault_injection = a.fault_injection;
  constexpr int VEC = 16 / (int)sizeof(T);
  p.c_vec_ok = ((uintptr_t)a.C & 15u) == 0 && (a.ldc % VEC) == 0;
  p.batch = 1;
  p.ep = a.ep;
  p.c_tma = p.c_vec_ok;
  mp.s_tiles = (int)mx_scale_tiles(FMT, a.K);
  mp.stages_k = (a.K + KSTAGE - 1) / KSTAGE;
  const int64_t kbytes = ((int64_t)a.K + 1) / 2;
  CUtensorMap mA, mB, mSA, mSB, mC;
  memset(&mC, 0, sizeof(mC));
  const CUtensorMapSwizzle SW = CU_TENSOR_MAP_SWIZZLE_128B;
  const CUtensorMapDataType U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!make_map(&mA, U8, a.A, a.M, kbytes, a.lda, 128, 128, SW, 1, 0, 1) ||
      !make_map(&mB, U8, a.B, a.N, kbytes, a.ldb, 128, PAIR ? BN / 2 : BN, SW, 1, 0, 1) ||
      !scale_map(&mSA, a.As, a.M, mp.s_tiles, C_::TPS) ||
      !scale_map(&mSB, a.Bs, a.N, mp.s_tiles, C_::TPS) ||
      (p.c_tma && !make_map(&mC, Elem<T>::TMA, a.C, a.M, a.N, a.ldc, 128 / (int)sizeof(T), 32, SW, 1,
                            0, (int)sizeof(T))))
    return cudaErrorNotSupported;
  const int workers = (int)min((int64_t)mx4_slots<T, FMT, BN, PAIR>(a.num_sms), tiles);
  ctx.grid = PAIR ? 2 * workers : workers;
  const cudaError_t e = launch_kernel(kern, dim3(ctx.grid), dim3(MX_THREADS), C_::SMEM_BYTES,
                                      ctx.stream, PAIR ? 2 : 1, mA, mB, mSA, mSB, mC, mp);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

// Tile: the one with the least estimated time, rounds of tiles x (K stages x
// the bytes a block loads for a stage + the time of a tile's epilogue and start,
// as bytes).
enum { TILE_256_PAIR, TILE_128_PAIR, TILE_128, TILE_64, TILES };
int mx4_pick(int M, int N, int K, int num_sms) {
  static const int forced = [] {
    const char* e = getenv("GEMM_GB300_MX_TILE");
    return e ? atoi(e) : -1;
  }();
  if (forced >= 0 && forced < TILES) return forced;
  const struct { int bm, bn, slots, kib, fixed; } shape[TILES] = {
      {256, 256, num_sms / 2, 35, 140}, {256, 128, num_sms / 2, 26, 80},
      {128, 128, num_sms, 34, 80}, {128, 64, num_sms, 26, 60}};
  const int64_t stages = ((int64_t)K + KSTAGE - 1) / KSTAGE;
  int best = 0;
  double least = 0;
  for (int i = 0; i < TILES; ++i) {
    const int64_t tiles = (((int64_t)M + shape[i].bm - 1) / shape[i].bm) *
                          (((int64_t)N + shape[i].bn - 1) / shape[i].bn);
    const int64_t rounds = (tiles + shape[i].slots - 1) / shape[i].slots;
    const double cost = (double)rounds * ((double)stages * shape[i].kib + shape[i].fixed);
    if (i == 0 || cost < least) {
      least = cost;
      best = i;
    }
  }
  return best;
}

template <typename T, int FMT>
cudaError_t launch_mx4_f(const Mx4Args& a, LaunchCtx& ctx) {
  switch (mx4_pick(a.M, a.N, a.K, a.num_sms)) {
    case TILE_256_PAIR: return launch_mx4_cfg<T, FMT, 256, true>(a, ctx);
    case TILE_128_PAIR: return launch_mx4_cfg<T, FMT, 128, true>(a, ctx);
    case TILE_128: return launch_mx4_cfg<T, FMT, 128, false>(a, ctx);
    default: return launch_mx4_cfg<T, FMT, 64, false>(a, ctx);
  }
}
template <typename T>
cudaError_t launch_mx4_t(const Mx4Args& a, LaunchCtx& ctx) {
  return a.format == MX_FP4 ? launch_mx4_f<T, MX_FP4>(a, ctx)
                            : launch_mx4_f<T, MX_FP4_E4M3>(a, ctx);
}

}  // namespace

cudaError_t launch_mx4(const Mx4Args& a, LaunchCtx& ctx) {
  switch (a.out) {
    case 0: return launch_mx4_t<float>(a, ctx);
    case 1: return launch_mx4_t<__half>(a, ctx);
    case 2: return launch_mx4_t<__nv_bfloat16>(a, ctx);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gb300
