#pragma once
// Products whose epilogue does all that an MLP layer needs, of one matrix or
// grouped by expert, 16-bit operands on the 5th-generation tensor cores:
//
//   forward     U = alpha op(A) op(B) + bias,  Y = act(U) + beta R
//   backward    dX = (alpha op(A) op(B)) act'(U),  dbias = column sums of dX
//   weights     C_g = alpha A_g^T B_g + beta C_g
//
// In a grouped product the offsets o lie in device memory and cut the rows:
// group g's rows o[g] .. o[g+1] of A meet matrix g of B (FUSED_ROWS), or are the
// inner dimension of C_g's product (FUSED_INNER).
//
// The block is that of the 4-bit product (mx4_tcgen05.cu): a TMA producer warp, a
// warp that issues the MMAs, epilogue warps; persistent workers (blocks, or
// pairs of blocks on 2-SM MMAs) walk the tiles.  What the groups change:
//  * A tile's place follows from the offsets alone, so every role finds it by
//    itself: a warp looks at 32 groups at once (tile counts by lane, their running
//    sum by shuffles), and since a worker's tiles ascend it never looks back.  No
//    list of tiles is made beforehand and the host never waits for the offsets.
//  * Groups begin and end at any row, tiles at multiples of 64 or 32 of them.  Rows
//    of another group that a tile of A, R or U takes along do no harm: an accumulator
//    row depends on its own row alone, and those past the group's end are left out of
//    sums and results (a box of the result that the end cuts is stored row by row).
//    Where rows are the inner dimension they would: there the operands' maps describe
//    the rows twice over, [start row][64 rows][columns] with the row pitch for both
//    outer dimensions, and the last box of a group's n < 64 rows from row r on starts
//    at (x, n - 64, r): it ends with those n rows, in both operands alike, and what
//    lies ahead of them is out of range and reads as zero.  One map bounds every
//    group, with nothing masked in shared memory.
//  * Eight or sixteen epilogue warps (see fu_threads) work on boxes of 32 rows x 64
//    columns.  R or U comes by TMA, ahead of the accumulator, into the staging buffer
//    that the result then leaves from; column sums are taken from registers, 32 rows at
//    a time, by a transposing shuffle reduction, and joined by fused_dbias_kernel in the
//    order of the rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "gelu.cuh"
#include "groups.cuh"
#include "hgemm_tcgen05.cuh"

namespace gb300 {
namespace {

// W: epilogue warps.  Their boxes' steps are chains of dependent instructions, so what a
// tile's epilogue costs goes by warps and by registers, which let the steps of several
// values run side by side: 256 x 256 pairs take sixteen warps of 96 registers, but eight
// of 168 for the slope of an activation (us, eight / sixteen: 16384 x 5632 x 2048
// backward 250 / 271, 32768 rows of 64 groups backward 193 / 203; 4000 rows of 8 groups
// forward 85.6 / 82.7, their weights' gradients 103 / 93).
constexpr int fu_threads(int W) { return 64 + 32 * W; }

template <int BN, bool PAIR>
struct FuCfg {
  static constexpr int SHARES = BN / 64;  // boxes of a tile's 32 rows
  static constexpr int B_BYTES = (PAIR ? BN / 2 : BN) * 128;
  static constexpr int STAGE_BYTES = A_TILE_BYTES + B_BYTES;
  static constexpr int STAGING_BYTES = 4 * SHARES * 4096;
  static constexpr int FIXED = 1024 + 512;
  static constexpr int RAW = (SMEM_LIMIT - FIXED - STAGING_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = RAW < 8 ? RAW : 8;
  static constexpr int TMEM_COLS = BN == 192 ? 512 : 2 * BN;  // two accumulators (a power of two)
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STAGING_BYTES + FIXED;
};

enum { U_NONE, U_SECTORS, U_HALVES, U_ROWS };

struct FuParams {
  int kind;
  int M, N, K;         // rows of all groups (FUSED_INNER: of C_g), columns, inner size (of all groups)
  int groups;
  const int* offsets;  // groups + 1 (grouped kinds)
  int b_mask;          // 0: one matrix of B for all groups, else -1
  int tiles_m, tiles_n;
  int64_t tiles;       // (FUSED_ROWS: the most that ascending offsets can have)
  // slices of K (FUSED_DENSE): a unit is a tile's slice of k_slice columns, whose raw sums
  // go to P [splits][M][ldp]; 1: none
  int splits, k_slice;
  float* P;
  int64_t ldp;
  float alpha, beta;
  const void* bias;    // [groups][N], or null
  int bias_vec;        // its rows 16-byte aligned
  int act;
  int mode;            // what `in` is: FUSED_NONE, FUSED_ADD (R), FUSED_SLOPE (U)
  const void* in;
  int64_t ld_in;
  void* U;             // stored pre-activation, or null
  int64_t ldu;
  void* Y;
  int64_t ldy, stride_y;
  int tma_in, tma_y;  // 16-byte aligned rows: through the tensor-memory-access unit
  int u_way;          // U's rows: U_SECTORS 32-byte aligned, U_HALVES 16-byte, U_ROWS neither
  float* part;         // column sums of each 32 rows of a group, [rows / 32 + groups + 1][N]
  unsigned int* status;
  uint64_t timeout_ns;
  int fault_injection;
};

// A worker's tile: this block's first row m0 (of all rows; FUSED_INNER: of C_g) and
// the end of its rows, the tile's first column, its group, and the range of the
// inner dimension.
struct FuTile {
  int m0, row_end, n0, g, g_lo, k_lo, k_len, slice;
};

// A worker's tiles, asked for in ascending order by every role of the block (whole
// warps).
template <int BMT, int BN>
struct FuWalk {
  RowTiles<BMT> rows;

  __device__ __forceinline__ void init(const FuParams& p, int lane) {
    if (p.kind == FUSED_ROWS) rows.init(p.offsets, p.groups, p.M, lane);
  }
  __device__ __forceinline__ bool find(const FuParams& p, int64_t t, int rank, int lane, FuTile& u) {
    int rt = p.tiles_m, loc = (int)t;
    u.g = u.g_lo = 0;
    u.row_end = p.M;
    u.k_lo = 0;
    u.k_len = p.K;
    u.slice = 0;
    if (p.kind == FUSED_ROWS) {
      int n;
      // (offsets that do not ascend may hold the same rows many times over: no more tiles
      // than ascending ones can have)
      if (t >= p.tiles) return false;
      if (!rows.find(p.offsets, p.groups, p.M, p.tiles_n, t, lane, u.g, u.g_lo, n, loc)) return false;
      u.row_end = u.g_lo + n;
      rt = (n + BMT - 1) / BMT;
    } else if (t >= p.tiles * p.splits) {
      return false;
    } else if (p.kind == FUSED_INNER) {
      const unsigned int per = (unsigned int)rt * (unsigned int)p.tiles_n;
      u.g = (int)((unsigned int)t / per);
      loc = (int)((unsigned int)t - (unsigned int)u.g * per);
      group_span(p.offsets, u.g, p.K, u.k_lo, u.k_len);
    } else if (p.splits > 1) {
      // (a tile's slices side by side)
      loc = (int)t / p.splits;
      u.slice = (int)t - loc * p.splits;
      u.k_lo = u.slice * p.k_slice;
      u.k_len = min(p.K - u.k_lo, p.k_slice);
    }
    // bands of GROUP_M row tiles, column by column
    const int per_band = GROUP_M * p.tiles_n;
    const int fm = loc / per_band * GROUP_M, in_band = loc % per_band;
    const int height = min(rt - fm, GROUP_M);
    u.m0 = u.g_lo + (fm + in_band % height) * BMT + rank * BM;
    u.n0 = in_band / height * BN;
    return true;
  }
};

// descriptors as (low word, constant high word), as in mx4_tcgen05.cu: 128-byte
// swizzle, 8-row groups 1024 bytes apart; an MN-major operand's 64-wide atoms are
// 8192 bytes apart
constexpr uint32_t FU_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
template <bool MN>
__device__ __forceinline__ uint32_t fu_desc_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((MN ? 8192u >> 4 : 1u) << 16);
}
template <bool PAIR>
__device__ __forceinline__ void fu_mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t acc) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(FU_DESC_HI)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(FU_DESC_HI)
        : "memory");
}

// Column sums of 16 columns over the warp's 32 rows, in a fixed order: each step sends
// half of the columns to the lane across and adds those received to the other half.
// Lanes l and l ^ 1 get the sum of column l / 2.
__device__ __forceinline__ float warp_column_sum(float (&v)[16], int lane) {
#pragma unroll
  for (int d = 8; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < d; ++i) {
      const bool up = (lane & (2 * d)) != 0;
      const float give = up ? v[i] : v[i + d], keep = up ? v[i + d] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * d);
    }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// Byte offset of column c (of 64) of row r in a staging buffer: 16-byte chunks in
// the 128-byte swizzle.
__device__ __forceinline__ uint32_t fu_at(int r, int c) {
  return (uint32_t)(r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2);
}
// A box's rows between memory and its staging buffer, row by row: a row's 64 columns at
// a time, by the whole warp (rows off 16-byte alignment, or that a group's end cuts; rows
// and columns past the ends excepted).  Off alignment, a row a lane would touch 32 rows
// at every access (2000 x 4001 x 2048 with R and U: 130 us, this way 48).
template <typename T>
__device__ __forceinline__ void fu_rows_in(const T* src, int64_t ld, int rows, int cols,
                                           uint32_t sbuf, int lane) {
  const uint16_t* s = reinterpret_cast<const uint16_t*>(src);
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 8) {
    uint16_t v[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[i][h] = (r0 + i < rows && lane + 32 * h < cols) ? s[(int64_t)(r0 + i) * ld + lane + 32 * h]
                                                          : (uint16_t)0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(sbuf + fu_at(r0 + i, lane + 32 * h)),
                     "h"(v[i][h])
                     : "memory");
  }
  __syncwarp();
}
// (vec: 16-byte aligned rows, eight lanes a row)
template <typename T>
__device__ __forceinline__ void fu_rows_out(T* dst, int64_t ld, int rows, int cols, bool vec,
                                            uint32_t sbuf, int lane) {
  uint16_t* d = reinterpret_cast<uint16_t*>(dst);
  if (vec && cols % 8 == 0) {
    const int c = (lane & 7) * 8;
    if (c < cols)
      for (int r = lane >> 3; r < rows; r += 4) {
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(sbuf + fu_at(r, c))
                     : "memory");
        *reinterpret_cast<uint4*>(d + (int64_t)r * ld + c) = v;
      }
    __syncwarp();
    return;
  }
#pragma unroll 4
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (lane + 32 * h >= cols) continue;
      uint16_t v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(sbuf + fu_at(r, lane + 32 * h)) : "memory");
      d[(int64_t)r * ld + lane + 32 * h] = v;
    }
}

template <typename T, int BN, bool A_MN, bool B_MN, bool PAIR, int W>
__global__ void __launch_bounds__(fu_threads(W), 1)
    fused_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                    const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmI, const __grid_constant__ CUtensorMap tmY,
                    const FuParams p) {
  using C_ = FuCfg<BN, PAIR>;
  using E = Elem<T>;
  constexpr int STAGES = C_::STAGES;
  constexpr int BMT = PAIR ? 2 * BM : BM;
  // warps of a lane quarter with boxes: box b is warp b % BOX_WARPS's
  constexpr int BOX_WARPS = W / 4 < C_::SHARES ? W / 4 : C_::SHARES;
  constexpr uint32_t STAGE_TX = (uint32_t)C_::STAGE_BYTES * (PAIR ? 2u : 1u);
  const int rank = PAIR ? (int)cluster_ctarank() : 0;
  const int worker = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int workers = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t tiles_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* const tiles_ptr = smem_raw + (tiles_addr - raw_addr);
  const uint32_t staging_addr = tiles_addr + (uint32_t)(STAGES * C_::STAGE_BYTES);
  uint64_t* const bars =
      reinterpret_cast<uint64_t*>(tiles_ptr + STAGES * C_::STAGE_BYTES + C_::STAGING_BYTES);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(STAGES + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (uint32_t)(2 * STAGES + 4);
  auto in_bar = [&](int w) { return bar0 + 8u * (uint32_t)(2 * STAGES + 5 + w); };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5 + 4 * C_::SHARES);
  volatile uint32_t* const abort_flag = tmem_slot + 1;
  static_assert(8 * (2 * STAGES + 6 + 4 * C_::SHARES) <= 512, "barrier area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), (PAIR ? 2 : 1) * 32 * 4 * BOX_WARPS);
    }
    mbar_init(drain_bar, 1);
    for (int w = 0; w < 4 * C_::SHARES; ++w) mbar_init(in_bar(w), 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), (uint32_t)C_::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), (uint32_t)C_::TMEM_COLS);
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
  FuWalk<BMT, BN> walk;
  walk.init(p, lane);
  FuTile u;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    if (leader && p.K > 0) {  // (else there are no maps)
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmB);
    }
    __syncwarp();
    int stage = 0;
    uint32_t phase = 0, pending = 0, pend_phase = 0;
    bool ok = true, first = true;
    for (int64_t t = worker; ok && walk.find(p, t, rank, lane, u); t += workers) {
      const int nkb = (u.k_len + BK - 1) / BK;
      for (int kb = 0; kb < nkb; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, wc));
        if (!ok) break;
        const bool skip = first && p.fault_injection == 1;
        first = false;
        if (!skip) {
          const uint32_t sa = tiles_addr + (uint32_t)(stage * C_::STAGE_BYTES);
          const uint32_t sb = sa + (uint32_t)A_TILE_BYTES;
          const int k0 = kb * BK;
          // operands stored by k: rows of groups from k_lo on (see above), or all rows
          const int ky = p.kind == FUSED_INNER ? min(u.k_len - k0 - BK, 0) : u.k_lo + k0;
          const int kz = p.kind == FUSED_INNER ? u.k_lo + k0 : 0;
          if (leader) {
            auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
              if constexpr (PAIR) tma_load_3d_pair(dst, map, x, y, z, bar);
              else tma_load_3d(dst, map, x, y, z, bar);
            };
            const uint32_t bar = PAIR ? mapa_shared(full_bar(stage), 0u) : full_bar(stage);
            // 64-column atoms past the last column are not loaded (what they would add
            // to is not stored)
            constexpr int ATOMS = BN / 64 / (PAIR ? 2 : 1);
            // nor are rows of A past the group's last, 32 at a time (a box of 128 where
            // there are more than 96)
            auto a_boxes = [&](int from) { return min(max((u.row_end - from + 31) / 32, 0), 4); };
            if (rank == 0) {
              uint32_t bytes = STAGE_TX;
              if constexpr (A_MN) {
                const int have = min(max((p.M - u.m0 + 63) / 64, 0), BMT / 64);
                bytes -= (uint32_t)(BMT / 64 - have) * 8192u;
              } else {
                bytes -= (uint32_t)(4 - a_boxes(u.m0)) * 4096u;
                if constexpr (PAIR) bytes -= (uint32_t)(4 - a_boxes(u.m0 + BM)) * 4096u;
              }
              if constexpr (B_MN) {
                const int have = min((p.N - u.n0 + 63) / 64, BN / 64);
                bytes -= (uint32_t)(BN / 64 - have) * 8192u;
              }
              mbar_arrive_expect_tx(full_bar(stage), bytes);
            }
            if constexpr (A_MN) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (u.m0 + 64 * h < p.M)
                  load(sa + (uint32_t)h * 8192u, &tmA, u.m0 + 64 * h, ky, kz, bar);
            } else {
              const int boxes = a_boxes(u.m0);
              if (boxes == 4) load(sa, &tmA, u.k_lo + k0, u.m0, 0, bar);
              else
                for (int h = 0; h < boxes; ++h)
                  load(sa + (uint32_t)h * 4096u, &tmA32, u.k_lo + k0, u.m0 + 32 * h, 0, bar);
            }
            if constexpr (B_MN) {
#pragma unroll
              for (int h = 0; h < ATOMS; ++h) {
                const int x = u.n0 + 64 * (rank * ATOMS + h);
                if (x < p.N)
                  load(sb + (uint32_t)h * 8192u, &tmB, x, ky,
                       p.kind == FUSED_INNER ? kz : u.g & p.b_mask, bar);
              }
            } else {
              // (the odd block's box may lie wholly past the last column: zeros)
              load(sb, &tmB, u.k_lo + k0, u.n0 + rank * (BN / 2), u.g & p.b_mask, bar);
            }
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
    if (worker == 0 && rank == 0 && p.kind != FUSED_DENSE)
      check_offsets(p.offsets, p.groups, p.kind == FUSED_ROWS ? p.M : p.K, p.status, lane);
    // every load issued must land before the block can exit (a pair's land on the
    // even block's barriers, and the pair leaves together)
    if (rank == 0)
      for (int s = 0; s < STAGES; ++s)
        if (pending & (1u << s))
          mbar_wait_drain(full_bar(s), (pend_phase >> s) & 1u, p.timeout_ns);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      const bool leader = elect_one();
      constexpr uint32_t idesc = make_idesc<BN, A_MN, B_MN, BMT, E::FMT>();
      const uint32_t a_lo0 = fu_desc_lo<A_MN>(tiles_addr);
      const uint32_t b_lo0 = fu_desc_lo<B_MN>(tiles_addr + A_TILE_BYTES);
      constexpr uint32_t A_STEP = A_MN ? 2048u >> 4 : 32u >> 4, B_STEP = B_MN ? 2048u >> 4 : 32u >> 4;
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int64_t t = worker; ok && walk.find(p, t, rank, lane, u); t += workers, ++it) {
        const int nkb = (u.k_len + BK - 1) / BK;
        const int buf = it & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(acce_bar(buf), ((uint32_t)(it >> 1) & 1u) ^ 1u, wc));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(buf * BN);
        for (int kb = 0; kb < nkb; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, wc));
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_lo = a_lo0 + (uint32_t)(stage * (C_::STAGE_BYTES >> 4));
          const uint32_t b_lo = b_lo0 + (uint32_t)(stage * (C_::STAGE_BYTES >> 4));
          // (16 of K that are zero in both operands are left out: ahead of a group's
          // last rows, or past the end)
          const int kn = min(u.k_len - kb * BK, BK);
          const int lo = p.kind == FUSED_INNER ? (BK - kn) / 16 : 0;
          const int hi = p.kind == FUSED_INNER ? BK / 16 : (kn + 15) / 16;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              if (kk < lo || kk >= hi) continue;
              fu_mma<PAIR>(d_tmem, a_lo + (uint32_t)kk * A_STEP, b_lo + (uint32_t)kk * B_STEP, idesc,
                           kb != 0 || kk != lo ? 1u : 0u);
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
    const int hh = ew / 4;    // of the warps of its quarter
    auto release_acc = [&](int buf) {
      tc_fence_before();
      if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(acce_bar(buf), 0u));
      else mbar_arrive(acce_bar(buf));
    };
    uint32_t in_phase = 0, in_flight = 0;  // loads of `in` by box: parity, under way (lane 0)
    int it = 0;
    for (int64_t t = worker; hh < BOX_WARPS && walk.find(p, t, rank, lane, u); t += workers, ++it) {
      const int buf = it & 1;
      const int gm = u.m0 + q * 32;  // the warp's rows
      const int rows = min(max(u.row_end - gm, 0), 32);
      // boxes of the tile with something in them
      const int boxes = rows > 0 ? min((p.N - u.n0 + 63) / 64, C_::SHARES) : 0;
      const int64_t gy = p.kind == FUSED_INNER ? (int64_t)u.g * p.stride_y : 0;
      auto sbuf_of = [&](int b) { return staging_addr + (uint32_t)((4 * b + q) * 4096); };
      // R, U or C: the boxes into their staging buffers, once the last stores have read
      // those
      const bool in_box = p.mode != FUSED_NONE && p.tma_in;
      if (in_box && lane == 0 && hh < boxes) {
        bulk_wait_read<0>();
        for (int b = hh; b < boxes; b += BOX_WARPS) {
          mbar_arrive_expect_tx(in_bar(4 * b + q), 4096u);
          tma_load_3d(sbuf_of(b), &tmI, u.n0 + 64 * b, gm, p.kind == FUSED_INNER ? u.g : 0,
                      in_bar(4 * b + q));
          in_flight |= 1u << b;
        }
      }
      bool got = false;
      if (lane == 0) got = mbar_wait(accf_bar(buf), (uint32_t)(it >> 1) & 1u, wc);
      got = warp_got(got);
      if (!got) break;
      tc_fence_after();
      if (hh >= boxes) {
        release_acc(buf);
        continue;
      }
#pragma unroll 1
      for (int b = hh; b < boxes; b += BOX_WARPS) {
        const uint32_t sbuf = sbuf_of(b);
        const int gn = u.n0 + 64 * b, cols = min(p.N - gn, 64);
        const uint32_t t_row = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN + 64 * b);
        got = true;
        if (lane == 0) {
          if (in_box) {
            got = mbar_wait(in_bar(4 * b + q), (in_phase >> b) & 1u, wc);
            if (got) {
              in_phase ^= 1u << b;
              in_flight &= ~(1u << b);
            }
          } else {
            bulk_wait_read<0>();  // the last store has read the buffer
          }
        }
        got = warp_got(got);
        if (!got) break;
        // sixteen columns' accumulators, and U in fp32
        auto sums_of = [&](int c, uint32_t (&r)[16]) {
          tmem_ld_32x32b_x16(t_row + (uint32_t)(16 * c), r);
          tmem_ld_wait();
        };
        auto linear = [&](int col, const uint32_t (&r)[16], float (&v)[16]) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(r[e]);
          if (p.alpha != 1.f) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= p.alpha;
          }
          if (u.k_len == 0) {  // (no product was added up)
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
          }
          if (p.bias) {
            const T* b = static_cast<const T*>(p.bias) + (int64_t)u.g * p.N + col;
            if (p.bias_vec && col + 15 < p.N) {
              uint4 bv[2] = {__ldg(reinterpret_cast<const uint4*>(b)),
                             __ldg(reinterpret_cast<const uint4*>(b) + 1)};
              const typename E::T2* b2 = reinterpret_cast<const typename E::T2*>(bv);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 f = E::unpack(b2[e]);
                v[2 * e] += f.x;
                v[2 * e + 1] += f.y;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (col + e < p.N) v[e] += E::to(b[e]);
            }
          }
        };
        auto place = [&](int c, int w) {  // the lane's 16-byte chunk 2c + w of its row
          return sbuf + (uint32_t)(lane * 128 + (((2 * c + w) ^ (lane & 7)) * 16));
        };
        auto pack = [&](const float (&v)[16], uint4 (&o)[2]) {
          typename E::T2* oh = reinterpret_cast<typename E::T2*>(o);
#pragma unroll
          for (int e = 0; e < 8; ++e) oh[e] = E::pack(v[2 * e], v[2 * e + 1]);
        };
        auto put = [&](int c, const uint4 (&o)[2]) {
#pragma unroll
          for (int w = 0; w < 2; ++w)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place(c, w)), "r"(o[w].x),
                         "r"(o[w].y), "r"(o[w].z), "r"(o[w].w)
                         : "memory");
        };
        if (p.u_way == U_ROWS) {
          // U through the staging buffer, ahead of the rest
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t r[16];
            float v[16];
            uint4 o[2];
            sums_of(c, r);
            linear(gn + 16 * c, r, v);
            pack(v, o);
            put(c, o);
            __syncwarp();
          }
          fu_rows_out(static_cast<T*>(p.U) + (int64_t)gm * p.ldu + gn, p.ldu, rows, cols, false, sbuf,
                      lane);
          __syncwarp();
        }
        if (p.mode != FUSED_NONE && !in_box)
          fu_rows_in(static_cast<const T*>(p.in) + gy + (int64_t)gm * p.ld_in + gn, p.ld_in, rows, cols,
                     sbuf, lane);
        // Sixteen columns at a time.  (Not unrolled: the code that one call takes of all
        // that is here then stays in the instruction cache; unrolled over 64 columns,
        // steps that a call does not take slowed it as well: wgrad of 4000 rows of 8
        // groups 140 us, 117 without the slope's code in the kernel.)
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int col = gn + 16 * c;
          uint32_t r[16];
          sums_of(c, r);
          if (c == 3 && b + BOX_WARPS >= boxes) release_acc(buf);
          if (p.splits > 1) {
            // raw sums of the slice: 64 bytes of this lane's row of P (whose rows are whole)
            if (lane < rows && col < p.ldp) {
              float* const d = p.P + ((int64_t)u.slice * p.M + gm + lane) * p.ldp + col;
#pragma unroll
              for (int e = 0; e < 16; e += 8)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d + e),
                             "r"(r[e]), "r"(r[e + 1]), "r"(r[e + 2]), "r"(r[e + 3]), "r"(r[e + 4]),
                             "r"(r[e + 5]), "r"(r[e + 6]), "r"(r[e + 7])
                             : "memory");
            }
            __syncwarp();
            continue;
          }
          float v[16];
          linear(col, r, v);
          uint4 o[2];
          if ((p.u_way == U_SECTORS || p.u_way == U_HALVES) && lane < rows) {
            pack(v, o);
            T* const dst = static_cast<T*>(p.U) + (int64_t)(gm + lane) * p.ldu + col;
            if (col + 15 >= p.N) {
              const uint32_t* w = reinterpret_cast<const uint32_t*>(o);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (col + e < p.N)
                  reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
            } else if (p.u_way == U_SECTORS) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
                           "r"(o[0].x), "r"(o[0].y), "r"(o[0].z), "r"(o[0].w), "r"(o[1].x), "r"(o[1].y),
                           "r"(o[1].z), "r"(o[1].w)
                           : "memory");
            } else {
              reinterpret_cast<uint4*>(dst)[0] = o[0];
              reinterpret_cast<uint4*>(dst)[1] = o[1];
            }
          }
          if (p.mode != FUSED_SLOPE) act_of<T>(v, p.act);
          if (p.mode != FUSED_NONE) {
            uint4 in[2];
#pragma unroll
            for (int w = 0; w < 2; ++w)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(in[w].x), "=r"(in[w].y), "=r"(in[w].z), "=r"(in[w].w)
                           : "r"(place(c, w))
                           : "memory");
            const typename E::T2* c2 = reinterpret_cast<const typename E::T2*>(in);
            float f[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 x = E::unpack(c2[e]);
              f[2 * e] = x.x;
              f[2 * e + 1] = x.y;
            }
            if (p.mode == FUSED_SLOPE) {
              slope_of<T>(v, f, p.act);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __fmaf_rn(p.beta, f[e], v[e]);
            }
          }
          pack(v, o);
          put(c, o);
          if (p.part) {
            if (lane >= rows) {
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = 0.f;
            }
            const float sum = warp_column_sum(v, lane);
            const int64_t slot = (int64_t)(u.g_lo >> 5) + u.g + ((gm - u.g_lo) >> 5);
            if ((lane & 1) == 0 && col + (lane >> 1) < p.N) p.part[slot * p.N + col + (lane >> 1)] = sum;
          }
          __syncwarp();  // (the tensor-memory loads are the warp's together)
        }
        if (p.splits > 1) continue;
        // a box that the group's end cuts is stored row by row, as are rows off alignment and
        // a last box that ends within 16 bytes (tma_store_3d would fill those)
        if (!p.tma_y || cols % 8 != 0 || (p.kind == FUSED_ROWS && rows < 32)) {
          fu_rows_out(static_cast<T*>(p.Y) + gy + (int64_t)gm * p.ldy + gn, p.ldy, rows, cols, p.tma_y,
                      sbuf, lane);
          // (the next tile's `in` comes into the buffer by TMA: after what was read and
          // written here)
          if (in_box) fence_proxy_async_smem();
          __syncwarp();
        } else {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmY, gn, gm, p.kind == FUSED_INNER ? u.g : 0, sbuf);
            bulk_commit();
          }
        }
      }
      if (!got) break;
    }
    if (lane == 0) {
      bulk_wait_all();
      // (after an abort: a load still in flight lands before shared memory is released)
      for (int b = 0; b < C_::SHARES; ++b)
        if ((in_flight >> b) & 1u)
          mbar_wait_drain(in_bar(4 * b + q), (in_phase >> b) & 1u, p.timeout_ns);
    }
  }

  tc_fence_before();
  if constexpr (PAIR) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, (uint32_t)C_::TMEM_COLS);
    else tmem_dealloc(tmem_base, (uint32_t)C_::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side
// The rows of a matrix twice over, [rows][64 rows][cols] with the row pitch for both
// outer dimensions (see above).  A box of this use lies within the rows but for what
// is out of range.
bool rows_map(CUtensorMap* m, CUtensorMapDataType type, const void* p, int64_t rows, int64_t cols,
              int64_t ld) {
  return make_map(m, type, p, BK, cols, ld, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B, rows, ld, 2);
}

// Pairs resident at once (fewer than half the SMs where a GPC's do not all pair up)
template <typename T, int BN, bool A_MN, bool B_MN, bool PAIR, int W>
int fused_slots(int num_sms) {
  if (!PAIR) return num_sms;
  static CountPerDevice slots;
  const int n = slots.get(call_device(), [num_sms] {
    return resident_clusters((const void*)fused_tc_kernel<T, BN, A_MN, B_MN, PAIR, W>, 2, fu_threads(W),
                             FuCfg<BN, PAIR>::SMEM_BYTES, dim3(2 * (num_sms / 2)));
  });
  return n > 0 ? n : num_sms / 2;
}

template <typename T, int BN, bool A_MN, bool B_MN, bool PAIR, int W>
cudaError_t launch_fused_cfg(const FusedArgs& a, LaunchCtx& ctx) {
  using C_ = FuCfg<BN, PAIR>;
  constexpr int BMT = PAIR ? 2 * BM : BM;
  auto kern = fused_tc_kernel<T, BN, A_MN, B_MN, PAIR, W>;
  static OncePerDevice set;
  const cudaError_t attr = set.run(call_device(), cudaSuccess, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C_::SMEM_BYTES);
  });
  if (attr != cudaSuccess) return attr;
  const bool rows = a.kind == FUSED_ROWS, inner = a.kind == FUSED_INNER;
  FuParams p;
  memset(&p, 0, sizeof(p));
  p.kind = a.kind;
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.groups = a.groups;
  p.offsets = a.offsets;
  p.tiles_m = (a.M + BMT - 1) / BMT;
  p.tiles_n = (a.N + BN - 1) / BN;
  const int64_t most = (int64_t)(p.tiles_m + (rows ? (a.groups < a.M ? a.groups : a.M) : 0)) *
                       p.tiles_n * (inner ? a.groups : 1);
  p.tiles = most;
  // (slices of whole K steps, none of them empty: fused_plan)
  p.splits = a.splits;
  const int steps = (a.K + BK - 1) / BK;
  p.k_slice = (steps + a.splits - 1) / a.splits * BK;
  if (a.splits > 1 && (a.kind != FUSED_DENSE || !a.P || (int64_t)(a.splits - 1) * p.k_slice >= a.K))
    return cudaErrorInvalidValue;
  p.P = a.P;
  p.ldp = a.ldp;
  p.alpha = a.alpha; p.beta = a.beta;
  p.bias = a.bias;
  p.bias_vec = ((uintptr_t)a.bias & 15u) == 0 && a.N % 8 == 0;
  p.act = a.act;
  p.mode = a.splits > 1 ? FUSED_NONE : a.mode;
  p.in = a.in; p.ld_in = a.ld_in;
  p.U = a.U; p.ldu = a.ldu;
  p.Y = a.Y; p.ldy = a.ldy; p.stride_y = inner ? a.stride_y : 0;
  auto aligned = [](const void* q, int64_t ld) { return ((uintptr_t)q & 15u) == 0 && ld % 8 == 0; };
  p.tma_y = aligned(a.Y, a.ldy) && (!inner || a.groups == 1 || a.stride_y % 8 == 0);
  p.u_way = !a.U || a.splits > 1                                   ? U_NONE
            : ((uintptr_t)a.U & 31u) == 0 && a.ldu % 16 == 0 ? U_SECTORS
            : aligned(a.U, a.ldu)                            ? U_HALVES
                                                             : U_ROWS;
  // (U on its way through the staging buffer leaves no room for a box asked for ahead)
  p.tma_in = p.mode != FUSED_NONE && aligned(a.in, a.ld_in) && (!inner || p.tma_y) && p.u_way != U_ROWS;
  p.part = a.part;
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  p.fault_injection = a.fault_injection;
  constexpr CUtensorMapDataType TY = Elem<T>::TMA;
  const CUtensorMapSwizzle SW = CU_TENSOR_MAP_SWIZZLE_128B;
  CUtensorMap mA, mA32, mB, mI, mY;
  memset(&mA32, 0, sizeof(mA32));
  memset(&mI, 0, sizeof(mI));
  memset(&mY, 0, sizeof(mY));
  // (a stride of 0: one matrix)
  const int64_t matrices = a.stride_b != 0 ? a.groups : 1;
  p.b_mask = a.stride_b != 0 ? -1 : 0;
  bool ok = true;
  if (a.K > 0) {
    if (inner) ok = rows_map(&mA, TY, a.A, a.K, a.M, a.lda) && rows_map(&mB, TY, a.B, a.K, a.N, a.ldb);
    else {
      if (A_MN) ok = make_map(&mA, TY, a.A, a.K, a.M, a.lda, 64, 64);
      else ok = make_map(&mA, TY, a.A, a.M, a.K, a.lda, 64, BM) &&
                make_map(&mA32, TY, a.A, a.M, a.K, a.lda, 64, 32);
      if (B_MN) ok = ok && make_map(&mB, TY, a.B, a.K, a.N, a.ldb, 64, 64, SW, matrices, a.stride_b, 2);
      else ok = ok && make_map(&mB, TY, a.B, a.N, a.K, a.ldb, 64, PAIR ? BN / 2 : BN, SW, matrices, a.stride_b, 2);
    }
  } else {  // (no load is made)
    memset(&mA, 0, sizeof(mA));
    memset(&mB, 0, sizeof(mB));
  }
  if (p.tma_y)
    ok = ok && (inner ? make_map(&mY, TY, a.Y, a.M, a.N, a.ldy, 64, 32, SW, a.groups, a.stride_y, 2)
                      : make_map(&mY, TY, a.Y, a.M, a.N, a.ldy, 64, 32));
  if (inner) mI = mY;  // (C itself)
  else if (p.tma_in) ok = ok && make_map(&mI, TY, a.in, a.M, a.N, a.ld_in, 64, 32);
  if (!ok) return cudaErrorNotSupported;
  const int slots = fused_slots<T, BN, A_MN, B_MN, PAIR, W>(a.num_sms);
  const int64_t units = most * a.splits;
  if (units >= (1ll << 31)) return cudaErrorNotSupported;
  const int workers = (int)(units < slots ? units : slots);
  ctx.grid = PAIR ? 2 * workers : workers;
  const cudaError_t e = launch_kernel(kern, dim3(ctx.grid), dim3(fu_threads(W)), C_::SMEM_BYTES,
                                      ctx.stream, PAIR ? 2 : 1, mA, mA32, mB, mI, mY, p);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

template <typename T, bool A_MN, bool B_MN>
cudaError_t launch_fused_l(const FusedArgs& a, LaunchCtx& ctx) {
  switch (a.tile) {
    case FUSED_TILE_PAIR:
      return a.mode == FUSED_SLOPE && a.splits == 1 ? launch_fused_cfg<T, 256, A_MN, B_MN, true, 8>(a, ctx)
                                                    : launch_fused_cfg<T, 256, A_MN, B_MN, true, 16>(a, ctx);
    case FUSED_TILE_192: return launch_fused_cfg<T, 192, A_MN, B_MN, false, 12>(a, ctx);
    case FUSED_TILE_128: return launch_fused_cfg<T, 128, A_MN, B_MN, false, 8>(a, ctx);
    default: return launch_fused_cfg<T, 64, A_MN, B_MN, false, 4>(a, ctx);
  }
}
template <typename T>
cudaError_t launch_fused_t(const FusedArgs& a, LaunchCtx& ctx) {
  if (a.transA)
    return a.transB ? launch_fused_l<T, true, false>(a, ctx) : launch_fused_l<T, true, true>(a, ctx);
  return a.transB ? launch_fused_l<T, false, false>(a, ctx) : launch_fused_l<T, false, true>(a, ctx);
}

}  // namespace
}  // namespace gb300
