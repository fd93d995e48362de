// Fused and grouped products of a few rows: one new token, or a small serving batch,
// through a projection or through the experts that its tokens chose,
//
//   U = alpha A B_g^T + bias,  Y = act(U) + beta R      on the rows of each group g,
//
// B_g stored [N, K].  Bound by the bytes of the matrices whose groups have rows, each
// read once.
//
// A unit is sixteen rows of one B_g: eight warps share its K, 64 columns at a time in
// turn, and join their sums through shared memory in warp order.  B is the 16-row
// operand of m16n8k16 warp MMAs, A's rows the columns, eight at a time; a lane holds
// eight consecutive values of a row of each as one half of two operands (the order of
// K within a chunk is the loads', in both alike).  Blocks take the units of all groups
// with rows in turn; there are at most as many of these groups as rows, and each block
// lists them from the offsets.  Each warp brings its own 16 x 64 boxes of B by TMA,
// DEPTH ahead and across the units' ends, and waits for nothing but those; A stays in
// the L1 cache from one unit to the next.  (Copies by every lane cost the instructions
// that bound it, 8 x 8192 x 8192 38 us; teams of one, two or four warps for a unit
// gained nothing.)  The 16-bit tensor-core kernel would read the same bytes through
// tiles of 128 rows: 5632 x 2048 for one row is 44 or 88 tiles for 152 SMs there and
// 352 units here.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "gelu.cuh"
#include "groups.cuh"
#include "internal.h"
#include "per_device.h"
#include "tensor_map.h"

namespace gb300 {
namespace {

constexpr int FS_WARPS = 8, FS_THREADS = 32 * FS_WARPS;
constexpr int UNIT_ROWS = 16;    // rows of B a unit has
constexpr int CHUNK = 64;        // columns of K a warp takes at a time: a 128-byte row
constexpr int BOX = UNIT_ROWS * CHUNK * 2;
constexpr int FS_BLOCKS = 2;     // blocks of an SM
static_assert(FUSED_FEW_ROWS <= 16, "two operands of eight rows, the list of groups with rows");

// Chunks on their way: as many as two blocks' shared memory holds -- and so many that a
// third block never fits: blocks have equal shares of the units, and an SM with three
// while another has one is late (8192 x 8192, one row: 36 us with four chunks, 29 with
// six).
template <int NB>
struct FsCfg {
  static constexpr int DEPTH = 6;
  static constexpr int RING = FS_WARPS * DEPTH * BOX;
  static constexpr int SUMS = FS_WARPS * 8 * NB * UNIT_ROWS * 4;
  static constexpr int SMEM_BYTES = 1024 + RING + SUMS;
  static_assert(3 * (SMEM_BYTES + 1024) > 228 * 1024 && 2 * (SMEM_BYTES + 2048) <= 228 * 1024,
                "two blocks an SM");
};

struct FsParams {
  int M, N, K;
  int groups;
  const int* offsets;  // null: one group of all rows
  const void* A;
  int64_t lda;
  int b_mask;          // 0: one matrix of B for all groups, else -1
  float alpha, beta;
  const void* bias;
  int act;
  const void* R;       // residual, or null
  int64_t ldr;
  void* U;             // pre-activation to store, or null
  int64_t ldu;
  void* Y;
  int64_t ldy;
  int units_n;         // units of a group
  unsigned int* status;
  uint64_t timeout_ns;
  int fault_injection;
};

template <typename T>
struct Fs;
template <>
struct Fs<__half> {
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from(float f) { return __float2half_rn(f); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Fs<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float f) { return __float2bfloat16_rn(f); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// Eight 16-bit values of a 16-byte aligned row from column k on; with `end` those past
// K are zero and are not read.
__device__ __forceinline__ uint4 row8(const uint16_t* p, int k, int K, bool end) {
  if (!end || k + 8 <= K) return *reinterpret_cast<const uint4*>(p + k);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (k + e < K) w[e / 2] |= (uint32_t)p[k + e] << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// NB: groups of eight rows of A that a group may have
template <typename T, int NB>
__global__ void __launch_bounds__(FS_THREADS, FS_BLOCKS)
    fused_stream_kernel(const __grid_constant__ CUtensorMap tmB, const FsParams p) {
  using C_ = FsCfg<NB>;
  constexpr int DEPTH = C_::DEPTH;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[FS_WARPS * DEPTH];
  __shared__ uint32_t abort_word;
  __shared__ int list[FUSED_FEW_ROWS][3];  // groups with rows: number, first row, rows
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;  // (the swizzle's pattern)
  float* const sums =
      reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) + C_::RING);
  // sums[warp][row of A][row of the unit]
  auto sum_at = [&](int w, int m, int n) -> float* {
    return sums + ((w * 8 * NB + m) * UNIT_ROWS + n);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < FS_WARPS * DEPTH; ++i) mbar_init(smem_u32(bars + i), 1);
    abort_word = 0u;
    fence_mbar_init();
    if (p.K > 0) tma_prefetch_desc(&tmB);  // (else there is no map)
  }
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;  // row of B's and A's operands, place in a row

  int live = 1;
  if (p.offsets) {
    live = 0;
    for (int g = 0; g < p.groups; g += 32) {
      int lo = 0, n = 0;
      if (g + lane < p.groups) group_span(p.offsets, g + lane, p.M, lo, n);
      const unsigned int mask = __ballot_sync(0xffffffffu, n > 0);
      const int at = live + __popc(mask & ((1u << lane) - 1u));
      // (offsets that do not ascend may give more groups than rows: the first ones)
      if (warp == 0 && n > 0 && at < FUSED_FEW_ROWS) {
        list[at][0] = g + lane;
        list[at][1] = lo;
        list[at][2] = n;
      }
      live += __popc(mask);
    }
    live = min(live, FUSED_FEW_ROWS);
    if (blockIdx.x == 0 && warp == 0) check_offsets(p.offsets, p.groups, p.M, p.status, lane);
  } else if (threadIdx.x == 0) {
    list[0][0] = list[0][1] = 0;
    list[0][2] = p.M;
  }
  __syncthreads();
  // This block's units: every gridDim.x-th, so that each block has its share of the
  // groups with more rows, which cost more.
  const unsigned int units = (unsigned int)live * (unsigned int)p.units_n;
  unsigned int t = blockIdx.x;
  if (t >= units) return;
  auto unit = [&](unsigned int t_, int& at_, int& n0_) {
    at_ = (int)(t_ / (unsigned int)p.units_n);  // in the list
    n0_ = (int)(t_ - (unsigned int)at_ * (unsigned int)p.units_n) * UNIT_ROWS;
  };
  int at, n0;
  unit(t, at, n0);

  const int chunks = (p.K + CHUNK - 1) / CHUNK;
  const int mine = chunks > warp ? (chunks - 1 - warp) / FS_WARPS + 1 : 0;  // of each unit
  const int depth = min(mine, DEPTH);
  const uint32_t ring = base + (uint32_t)(warp * DEPTH * BOX);
  const uint32_t bar = smem_u32(bars + warp * DEPTH);
  const WaitCtl wc{p.status, &abort_word, p.timeout_ns};
  const bool leader = elect_one();
  // the box of a unit's chunk, into an entry of the ring (rows and columns past the
  // matrix read as zero)
  int asked = 0, taken = 0;  // boxes so far
  int to = 0;                // entry of the next one asked for
  auto ask = [&](int at_, int n0_, int chunk) {
    if (leader && !(p.fault_injection == 1 && asked == 0)) {
      mbar_arrive_expect_tx(bar + 8u * (uint32_t)to, (uint32_t)BOX);
      tma_load_3d(ring + (uint32_t)(to * BOX), &tmB, (chunk * FS_WARPS + warp) * CHUNK, n0_,
                  list[at_][0] & p.b_mask, bar + 8u * (uint32_t)to);
    }
    to = to + 1 == DEPTH ? 0 : to + 1;
    ++asked;
  };
  for (int d = 0; d < depth; ++d) ask(at, n0, d);
  __syncwarp();
  // this lane's places in a box: rows r and r + 8, 16-byte chunks c and 4 + c
  const uint32_t place[2] = {(uint32_t)(r * 128 + ((c ^ r) * 16)),
                             (uint32_t)(r * 128 + (((4 + c) ^ r) * 16))};
  bool ok = true;
  int entry = 0;       // of the next box, and its barrier's parity
  uint32_t phase = 0;
  for (; t < units; t += gridDim.x) {
    const bool more = t + gridDim.x < units;
    int at_next = 0, n0_next = 0;
    if (more) unit(t + gridDim.x, at_next, n0_next);
    const int g = list[at][0], lo = list[at][1], rows = min(list[at][2], 8 * NB);
    float acc[NB][4];
    const uint16_t* a_row[NB];
#pragma unroll
    for (int m = 0; m < NB; ++m) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][e] = 0.f;
      // (rows past the group's: its last one, whose sums there are not used)
      a_row[m] = static_cast<const uint16_t*>(p.A) + (int64_t)(lo + min(8 * m + r, rows - 1)) * p.lda;
    }
#pragma unroll 1
    for (int i = 0; ok && i < mine; ++i) {
      const int k0 = (i * FS_WARPS + warp) * CHUNK, k = k0 + 8 * c;
      const bool end = k0 + CHUNK > p.K;
      uint4 a[NB][2];
#pragma unroll
      for (int m = 0; m < NB; ++m) {
        if (8 * m >= rows) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) a[m][h] = row8(a_row[m], k + 32 * h, p.K, end);
      }
      const uint32_t box = ring + (uint32_t)(entry * BOX);
      ok = __all_sync(0xffffffffu, mbar_wait(bar + 8u * (uint32_t)entry, phase, wc));
      if (!ok) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 b[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(b[q].x), "=r"(b[q].y), "=r"(b[q].z), "=r"(b[q].w)
                       : "r"(box + place[h] + (uint32_t)(q * 1024))
                       : "memory");
        const uint32_t b0[4] = {b[0].x, b[1].x, b[0].y, b[1].y};
        const uint32_t b1[4] = {b[0].z, b[1].z, b[0].w, b[1].w};
#pragma unroll
        for (int m = 0; m < NB; ++m) {
          if (8 * m >= rows) continue;
          Fs<T>::mma(acc[m], b0, a[m][h].x, a[m][h].y);
          Fs<T>::mma(acc[m], b1, a[m][h].z, a[m][h].w);
        }
      }
      if (++entry == DEPTH) {
        entry = 0;
        phase ^= 1u;
      }
      ++taken;
      __syncwarp();  // (every lane has read the box)
      // the chunk `depth` ahead, of this unit or the next
      if (i + depth < mine) ask(at, n0, i + depth);
      else if (more) ask(at_next, n0_next, i + depth - mine);
    }
    // sums: rows r and r + 8 of the unit, rows 2c and 2c + 1 of A
    __syncthreads();  // (the last unit's are read)
#pragma unroll
    for (int m = 0; m < NB; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *sum_at(warp, 8 * m + 2 * c + (e & 1), r + 8 * (e >> 1)) = acc[m][e];
    __syncthreads();
    const int m = threadIdx.x / 8, n = n0 + 2 * (threadIdx.x & 7);
    if (m < rows && n < p.N) {
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < FS_WARPS; ++w) {
        const float2 s = *reinterpret_cast<const float2*>(sum_at(w, m, 2 * (threadIdx.x & 7)));
        v[0] += s.x;
        v[1] += s.y;
      }
      const bool two = n + 1 < p.N;
      const int64_t out = lo + m;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[e] *= p.alpha;
        if (p.bias && (e == 0 || two))
          v[e] += Fs<T>::to(static_cast<const T*>(p.bias)[(int64_t)g * p.N + n + e]);
      }
      if (p.U) {
        T* const d = static_cast<T*>(p.U) + out * p.ldu + n;
        d[0] = Fs<T>::from(v[0]);
        if (two) d[1] = Fs<T>::from(v[1]);
      }
      act_of<T>(v, p.act);
      if (p.R) {
        const T* const s = static_cast<const T*>(p.R) + out * p.ldr + n;
        v[0] = __fmaf_rn(p.beta, Fs<T>::to(s[0]), v[0]);
        if (two) v[1] = __fmaf_rn(p.beta, Fs<T>::to(s[1]), v[1]);
      }
      T* const d = static_cast<T*>(p.Y) + out * p.ldy + n;
      d[0] = Fs<T>::from(v[0]);
      if (two) d[1] = Fs<T>::from(v[1]);
    }
    at = at_next;
    n0 = n0_next;
  }
  // (after a wait that ran out: boxes on their way land before shared memory is released)
  for (; taken < asked; ++taken) {
    mbar_wait_drain(bar + 8u * (uint32_t)entry, phase, p.timeout_ns);
    if (++entry == DEPTH) {
      entry = 0;
      phase ^= 1u;
    }
  }
}

template <typename T, int NB>
cudaError_t launch_stream(const FusedArgs& a, LaunchCtx& ctx) {
  FsParams p;
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.groups = a.groups;
  p.offsets = a.kind == FUSED_DENSE ? nullptr : a.offsets;
  p.A = a.A; p.lda = a.lda;
  p.b_mask = a.stride_b != 0 ? -1 : 0;
  p.alpha = a.alpha; p.beta = a.beta;
  p.bias = a.bias;
  p.act = a.act;
  p.R = a.mode == FUSED_ADD ? a.in : nullptr;
  p.ldr = a.ld_in;
  p.U = a.U; p.ldu = a.ldu;
  p.Y = a.Y; p.ldy = a.ldy;
  p.units_n = (a.N + UNIT_ROWS - 1) / UNIT_ROWS;
  p.status = ctx.status;
  p.timeout_ns = ctx.timeout_ns;
  p.fault_injection = a.fault_injection;
  const int64_t most = (int64_t)p.units_n * (a.groups < a.M ? a.groups : a.M);
  if (most >= (1ll << 31)) return cudaErrorNotSupported;
  CUtensorMap mB;
  memset(&mB, 0, sizeof(mB));
  if (a.K > 0 && !make_map(&mB, a.dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           a.B, a.N, a.K, a.ldb, CHUNK, UNIT_ROWS, CU_TENSOR_MAP_SWIZZLE_128B,
                           a.stride_b != 0 ? a.groups : 1, a.stride_b, 2))
    return cudaErrorNotSupported;
  auto kern = fused_stream_kernel<T, NB>;
  static OncePerDevice set;
  const cudaError_t attr = set.run(call_device(), cudaSuccess, [kern] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                FsCfg<NB>::SMEM_BYTES);
  });
  if (attr != cudaSuccess) return attr;
  const int64_t slots = (int64_t)a.num_sms * FS_BLOCKS;
  ctx.grid = (int)(most < slots ? most : slots);
  const cudaError_t e = launch_kernel(kern, dim3((unsigned)ctx.grid), dim3(FS_THREADS),
                                      FsCfg<NB>::SMEM_BYTES, ctx.stream, 1, mB, p);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

template <typename T>
cudaError_t launch_stream_t(const FusedArgs& a, LaunchCtx& ctx) {
  return a.M <= 8 ? launch_stream<T, 1>(a, ctx) : launch_stream<T, 2>(a, ctx);
}

}  // namespace

cudaError_t launch_fused_stream(const FusedArgs& a, LaunchCtx& ctx) {
  if (a.M > FUSED_FEW_ROWS) return cudaErrorInvalidValue;
  return a.dtype == 1 ? launch_stream_t<__half>(a, ctx) : launch_stream_t<__nv_bfloat16>(a, ctx);
}

}  // namespace gb300
