#pragma once
// Microscaled storage, the elementwise side: quantisation of a matrix (with
// the activation of the forward pass in the same read), its inverse, and the
// activation's backward pass from an 8-bit checkpoint.
//
//   scale  s_rb = scale of max over the block |mult * x|        (mx_format.cuh)
//   code   q_rc = nearest code to mult * x_rc / s_rb, ties to even
//   Y      y_rc = act(x_rc)
//   dX     dx_rc = dy_rc * act'(q_rc s_rb),   dbias_c = sum_r dx_rc
//
// All are bound by HBM: each element is read once and written once.  Measured at
// 16384 x 5632 bf16: gelu with its checkpoint 91 us and the backward pass 92 (5.1
// TB/s together); 8192 x 8192 fp16 transposed to fp4_e4m3 41 us, read back 27 (6.4
// TB/s).  The gelu kernels issue 2.4 to 2.7 instructions a cycle of 4 at 57 % of
// DRAM's rate; the transposed one 2.4 at 48 %, with a tile's loads held in registers
// and none under way while it is encoded.  A thread keeps one unit of 16 columns
// and walks down the rows, two units (two 32-byte loads of a 16-bit type) in
// flight; 8 threads a row cover 128 columns, and a block of 8 warps 64 rows x 128
// columns at a time.  The grid is the column strips times as many blocks a strip as
// fill the GPU, so that a strip's column sums stay in registers until its blocks
// join them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "common.cuh"
#include "internal.h"
#include "mx_format.cuh"

namespace gb300 {
namespace {

constexpr int STRIP = 128;    // columns of a block
constexpr int UNITS = 2;      // units of a thread in flight
constexpr int TILE_ROWS = 32 * UNITS;
constexpr int THREADS = 256;
constexpr int BLOCKS_PER_SM = 4;
// The kernels come in two: for 16-byte aligned rows (and mult 1), and a general
// one with the staging of unaligned rows, whose registers would cost the first
// its fourth block an SM (16384 x 5632 bf16 gelu, both passes: 181 -> 236 us).
constexpr int BLOCKS_PER_SM_GENERAL = 3;
constexpr int blocks_per_sm(bool general) { return general ? BLOCKS_PER_SM_GENERAL : BLOCKS_PER_SM; }

struct QuantParams {
  const void* X;
  int64_t ldx;
  int rows, cols;
  float mult;
  void* Y;  // act(X), or null
  int64_t ldy;
  uint8_t* q;
  int64_t ldq;
  uint8_t* s;
  int64_t s_tiles;   // scale tiles of a 128-row range
  int64_t tiles_m;   // row tiles (the last 128-row range in full: its padding is written)
  int64_t tiles_n, tiles;  // (transposed form)
  int vec_x, vec_y;
};

// Rows off 16-byte alignment, four of them at once by a whole warp through its
// shared-memory buffer, so that a warp's accesses still cover consecutive
// elements of a row: element by element from the threads' own units, each of a
// warp's accesses touched 32 sectors (gelu forward and backward 12800 x 495 bf16
// 92 us).  `rows` of the four and `cols` of the strip's 128 exist; absent
// elements read as 0.  v: this thread's unit (row lane / 8, columns 16 (lane % 8)).
constexpr int STAGE_PITCH = STRIP + 8;
template <typename T>
__device__ __forceinline__ void warp_load_rows(const T* p, int64_t ld, int rows, int cols, T* buf,
                                               int lane, MxRow16<T>& v) {
  __syncwarp();
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = i * 32 + lane;
      buf[r * STAGE_PITCH + c] = r < rows && c < cols ? p[r * ld + c] : MxIo<T>::from(0.f);
    }
  __syncwarp();
  memcpy(&v, buf + (lane >> 3) * STAGE_PITCH + (lane & 7) * 16, sizeof(v));
}
template <typename T>
__device__ __forceinline__ void warp_store_rows(T* p, int64_t ld, int rows, int cols, T* buf,
                                                int lane, const float (&x)[16]) {
  T e[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) e[i] = MxIo<T>::from(x[i]);
  __syncwarp();
  memcpy(buf + (lane >> 3) * STAGE_PITCH + (lane & 7) * 16, e, sizeof(e));
  __syncwarp();
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = i * 32 + lane;
      if (r < rows && c < cols) p[r * ld + c] = buf[r * STAGE_PITCH + c];
    }
}
// (rows of the four from r0 on, columns of the strip)
__device__ __forceinline__ int left_of(int64_t end, int64_t from, int most) {
  return (int)max((int64_t)0, min((int64_t)most, end - from));
}

// bits of |mult| * (a magnitude given by its bits), with a NaN's kept a NaN's
__device__ __forceinline__ uint32_t scale_bits(uint32_t m, float mult) {
  return __float_as_uint(__uint_as_float(m) * mult) & 0x7FFFFFFFu;
}
__device__ __forceinline__ uint32_t max_abs_bits(const float (&x)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}

// 16-bit types.  For a pair x, given as n = -|x|: c = erfc(|x| / sqrt 2) / 2 =
// Phi(-|x|) and e = exp(-x^2 / 2), which the gelu and its derivative share:
//   erfc(z) = t (a1 + t (a2 + ... )) exp(-z^2),  t = 1 / (1 + p z),
// within 1.5e-7 (M. Abramowitz and I. Stegun, "Handbook of Mathematical
// Functions", 7.1.26), which the rounding to 16 bits covers but in the far tail:
// 0.3 % of gelu(-5.7) = -3e-8, 1.2 % of gelu(-8.5) = -8e-17.  A value costs an
// exponential, a reciprocal and five paired operations; with erff and expf, the
// forward and backward pass at 16384 x 5632 bf16 took 465 us against 232 with
// scalar operations of this form.
__device__ __forceinline__ f32x2 normal_tail2(f32x2 n, f32x2& e) {
  float a, b;
  unpair(fma2(n, pair(-0.3275911f * 0.70710678f), pair(1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  const f32x2 t = pair(a, b);
  unpair(mul2(mul2(n, n), pair(-0.72134752f)), a, b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  e = pair(a, b);
  f32x2 c = fma2(t, pair(0.5f * 1.061405429f), pair(0.5f * -1.453152027f));
  c = fma2(t, c, pair(0.5f * 1.421413741f));
  c = fma2(t, c, pair(0.5f * -0.284496736f));
  c = fma2(t, c, pair(0.5f * 0.254829592f));
  return mul2(mul2(t, c), e);
}
// -|x|, not below -64 (where c and e are 0 already), so that an infinity meets no
// 0; a NaN stays one
__device__ __forceinline__ float minus_abs(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(-fabsf(x)), "f"(-64.f));
  return r;
}
// x Phi(x) = max(x, 0) - |x| Phi(-|x|); fp32 results within a few ulp, from
// normcdff (both tails keep their relative accuracy; the rational form's error
// would be several ulp between -3.5 and -0.5).  That costs time: forward and
// backward pass at 16384 x 5632 fp32 542 us, 298 with the rational form, 245 by
// their bytes.
template <typename T, int ACT>
__device__ __forceinline__ void act_values(const float (&x)[16], float (&y)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float m0 = x[i] > 0.f ? x[i] : 0.f, m1 = x[i + 1] > 0.f ? x[i + 1] : 0.f;
    if constexpr (ACT == 2 && sizeof(T) == 4) {
      const float n0 = minus_abs(x[i]), n1 = minus_abs(x[i + 1]);
      y[i] = __fmaf_rn(n0, normcdff(n0), m0);
      y[i + 1] = __fmaf_rn(n1, normcdff(n1), m1);
    } else if constexpr (ACT == 2) {
      const f32x2 n = pair(minus_abs(x[i]), minus_abs(x[i + 1]));
      f32x2 e;
      const f32x2 c = normal_tail2(n, e);
      unpair(fma2(n, c, pair(m0, m1)), y[i], y[i + 1]);
    } else {
      y[i] = ACT == 1 ? m0 : x[i];
      y[i + 1] = ACT == 1 ? m1 : x[i + 1];
    }
  }
}

// ACT: the activation of Y, or -1 without Y
template <typename T, int FMT, int ACT, bool GENERAL>
__global__ void __launch_bounds__(THREADS, blocks_per_sm(GENERAL))
    mx_quantize_kernel(const QuantParams p) {
  __shared__ __align__(16) T stage[GENERAL ? THREADS / 32 : 1][GENERAL ? 4 * STAGE_PITCH : 16];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = lane & 7;
  const int64_t c0 = (int64_t)blockIdx.x * STRIP + u * 16;
  const int n = (int)min((int64_t)16, max((int64_t)0, (int64_t)p.cols - c0));
  const int64_t qcol = c0 / 16 * mx_bytes16<FMT>();
  const bool has_codes = qcol < mx_row_bytes(FMT, p.cols);
  const int64_t st = c0 / (4 * mx_block(FMT));
  // the lane that writes a scale word
  const bool has_word = (mx_block(FMT) == 32 ? u == 0 : (u & 3) == 0) && st < p.s_tiles;
  for (int64_t tm = blockIdx.y; tm < p.tiles_m; tm += gridDim.y) {
    const int64_t r0 = tm * TILE_ROWS + warp * 4 * UNITS + (lane >> 3);
    MxRow16<T> in[UNITS];
    int64_t row[UNITS];
#pragma unroll
    for (int j = 0; j < UNITS; ++j)
      row[j] = min(r0 + 4 * j, (int64_t)p.rows - 1) * p.ldx;  // (rows past the end: not stored)
    if (!GENERAL || p.vec_x != MX_SCALAR)
      mx_load_units<T, UNITS>(static_cast<const T*>(p.X) + c0, row, n, p.vec_x, in);
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      const int64_t r = r0 + 4 * j, w0 = r - (lane >> 3);  // (the warp's first of four rows)
      const bool real = r < p.rows;
      if (GENERAL && p.vec_x == MX_SCALAR)
        warp_load_rows<T>(static_cast<const T*>(p.X) + w0 * p.ldx + (c0 - u * 16), p.ldx,
                          left_of(p.rows, w0, 4), left_of(p.cols, c0 - u * 16, STRIP), stage[warp],
                          lane, in[j]);
      float x[16];
      mx_unpack16<T>(in[j], x);
      if constexpr (ACT >= 0) {
        float y[16];
        act_values<T, ACT>(x, y);
        if (GENERAL && p.vec_y == MX_SCALAR)
          warp_store_rows<T>(static_cast<T*>(p.Y) + w0 * p.ldy + (c0 - u * 16), p.ldy,
                             left_of(p.rows, w0, 4), left_of(p.cols, c0 - u * 16, STRIP),
                             stage[warp], lane, y);
        else if (real)
          mx_store16<T>(static_cast<T*>(p.Y) + r * p.ldy + c0, n, p.vec_y, y);
      }
      // (the largest of |mult x| is |mult| times the largest |x|: rounding keeps order)
      uint32_t m = mx_max_abs16<T>(in[j]);
      if (GENERAL) {  // (otherwise mult is 1)
        m = scale_bits(m, p.mult);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= p.mult;
        if (n < 16) {  // (absent columns stay 0: the code of -1 * 0 is another)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (i >= n) x[i] = 0.f;
        }
      }
      if (mx_block(FMT) == 32) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      uint32_t byte = mx_scale_byte<FMT>(__uint_as_float(m));
      MxCodes<FMT> c;
      mx_encode16<FMT>(x, byte, __uint_as_float(m), c);
      // (codes of absent columns up to the row's 16-byte unit are written as 0)
      if (real && has_codes) mx_store_codes<FMT>(p.q + r * p.ldq + qcol, c);
      // four blocks' scale bytes as a word; absent rows and blocks 0 (of a 32-
      // column block's two units only the second may be absent)
      uint32_t w;
      if (mx_block(FMT) == 32) {
        w = real && n > 0 && (u & 1) == 0 ? byte << (4 * u) : 0u;
        w |= __shfl_xor_sync(0xffffffffu, w, 2);
        w |= __shfl_xor_sync(0xffffffffu, w, 4);
      } else {
        w = real && n > 0 ? byte << (8 * (u & 3)) : 0u;
        w |= __shfl_xor_sync(0xffffffffu, w, 1);
        w |= __shfl_xor_sync(0xffffffffu, w, 2);
      }
      if (has_word)
        *reinterpret_cast<uint32_t*>(p.s + mx_scale_word(r, st, p.s_tiles)) = w;
    }
  }
}

// The transposed form: X is stored [cols, rows], so a block of a stored-to row
// runs down a column of X.  A thread takes two adjacent op(X) rows (one 4- or
// 8-byte load from each stored row, 32 of them in flight) and 32 columns;
// codes and scale bytes go through shared memory, so that they leave in whole
// row segments.
constexpr int TT_ROWS = 64, TT_COLS = 128, TT_THREADS = 128;

template <typename T, int FMT, bool MULT>
__global__ void __launch_bounds__(TT_THREADS) mx_quantize_t_kernel(const QuantParams p) {
  constexpr int ROW_BYTES = TT_COLS / 16 * mx_bytes16<FMT>();
  constexpr int PITCH = ROW_BYTES + 16;  // (rows two apart in different banks)
  constexpr int NB = TT_COLS / mx_block(FMT);
  __shared__ __align__(16) uint8_t codes[TT_ROWS * PITCH];
  __shared__ __align__(16) uint8_t scales[TT_ROWS * NB];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x) {
    const int64_t tm = t / p.tiles_n;
    const int64_t r0 = tm * TT_ROWS, cc0 = (t - tm * p.tiles_n) * TT_COLS;
    const int64_t r = r0 + 2 * lane;
    const int64_t c0 = cc0 + 32 * warp;
    const int nr = (int)min((int64_t)2, max((int64_t)0, (int64_t)p.rows - r));
    const int nc = (int)min((int64_t)32, max((int64_t)0, (int64_t)p.cols - c0));
    const T* src = static_cast<const T*>(p.X) + c0 * p.ldx + r;
    struct alignas(2 * sizeof(T)) Two { T a, b; };
    Two in[32];
    // (the paths apart, so that a whole tile's loads are issued together)
    if (p.vec_x && nr == 2 && nc == 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i) in[i] = *reinterpret_cast<const Two*>(src + i * p.ldx);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        in[i].a = in[i].b = MxIo<T>::from(0.f);
        if (i < nc && nr > 0) in[i].a = src[i * p.ldx];
        if (i < nc && nr > 1) in[i].b = src[i * p.ldx + 1];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float lo[16], hi[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        lo[i] = MxIo<T>::to(h ? in[i].b : in[i].a);
        hi[i] = MxIo<T>::to(h ? in[16 + i].b : in[16 + i].a);
        if (MULT) {
          lo[i] *= p.mult;
          hi[i] *= p.mult;
        }
      }
      if (MULT && nc < 32) {  // (absent columns stay 0: the code of -1 * 0 is another)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (i >= nc) lo[i] = 0.f;
          if (16 + i >= nc) hi[i] = 0.f;
        }
      }
      uint32_t ml = max_abs_bits(lo), mh = max_abs_bits(hi);
      if (mx_block(FMT) == 32) ml = mh = max(ml, mh);
      const uint32_t bl = mx_scale_byte<FMT>(__uint_as_float(ml));
      const uint32_t bh = mx_scale_byte<FMT>(__uint_as_float(mh));
      MxCodes<FMT> c;
      uint8_t* dst = codes + (2 * lane + h) * PITCH + 2 * warp * mx_bytes16<FMT>();
      mx_encode16<FMT>(lo, bl, __uint_as_float(ml), c);
      mx_store_codes<FMT>(dst, c);
      mx_encode16<FMT>(hi, bh, __uint_as_float(mh), c);
      mx_store_codes<FMT>(dst + mx_bytes16<FMT>(), c);
      uint8_t* sb = scales + (2 * lane + h) * NB;
      if (mx_block(FMT) == 32) {
        sb[warp] = (uint8_t)(nr > h && nc > 0 ? bl : 0u);
      } else {
        sb[2 * warp] = (uint8_t)(nr > h && nc > 0 ? bl : 0u);
        sb[2 * warp + 1] = (uint8_t)(nr > h && nc > 16 ? bh : 0u);
      }
    }
    __syncthreads();
    constexpr int CH = ROW_BYTES / 16;  // 16-byte chunks of a tile row
    for (int i = threadIdx.x; i < TT_ROWS * CH; i += TT_THREADS) {
      const int rr = i / CH, ch = i % CH;
      const int64_t at = cc0 / 16 * mx_bytes16<FMT>() + ch * 16;
      if (r0 + rr < p.rows && at < mx_row_bytes(FMT, p.cols))
        *reinterpret_cast<uint4*>(p.q + (r0 + rr) * p.ldq + at) =
            *reinterpret_cast<const uint4*>(codes + rr * PITCH + ch * 16);
    }
    for (int i = threadIdx.x; i < TT_ROWS * NB / 4; i += TT_THREADS) {
      const int rr = i / (NB / 4), w = i % (NB / 4);
      const int64_t st = cc0 / TT_COLS * (NB / 4) + w;
      if (st < p.s_tiles)
        *reinterpret_cast<uint32_t*>(p.s + mx_scale_word(r0 + rr, st, p.s_tiles)) =
            *reinterpret_cast<const uint32_t*>(scales + rr * NB + 4 * w);
    }
    __syncthreads();
  }
}

struct DequantParams {
  const uint8_t* q;
  int64_t ldq;
  const uint8_t* s;
  int64_t s_tiles;
  int rows, cols;
  void* Y;
  int64_t ldy;
  int64_t tiles_m;
  int vec_y;
};

template <typename T, int FMT, bool GENERAL>
__global__ void __launch_bounds__(THREADS, blocks_per_sm(GENERAL))
    mx_dequantize_kernel(const DequantParams p) {
  __shared__ __align__(16) T stage[GENERAL ? THREADS / 32 : 1][GENERAL ? 4 * STAGE_PITCH : 16];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t cc0 = (int64_t)blockIdx.x * STRIP, c0 = cc0 + (lane & 7) * 16;
  const int n = left_of(p.cols, c0, 16);
  const uint8_t* const q = p.q + c0 / 16 * mx_bytes16<FMT>();
  const int64_t b = c0 / mx_block(FMT);
  for (int64_t tm = blockIdx.y; (GENERAL || n > 0) && tm < p.tiles_m; tm += gridDim.y) {
    const int64_t r0 = tm * TILE_ROWS + warp * 4 * UNITS + (lane >> 3);
    MxCodes<FMT> c[UNITS];
    uint32_t byte[UNITS];
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      const int64_t r = min(r0 + 4 * j, (int64_t)p.rows - 1);
      if (!GENERAL || n > 0) {
        c[j] = mx_load_codes<FMT>(q + r * p.ldq);
        byte[j] = p.s[mx_scale_word(r, b >> 2, p.s_tiles) + (b & 3)];
      } else {
        c[j] = {};
        byte[j] = 0;
      }
    }
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      const int64_t r = r0 + 4 * j, w0 = r - (lane >> 3);
      if (!GENERAL && r >= p.rows) continue;
      float x[16];
      mx_decode16<FMT>(c[j], mx_scale_value<FMT>(byte[j]), x);
      if (GENERAL && p.vec_y == MX_SCALAR)
        warp_store_rows<T>(static_cast<T*>(p.Y) + w0 * p.ldy + cc0, p.ldy, left_of(p.rows, w0, 4),
                           left_of(p.cols, cc0, STRIP), stage[warp], lane, x);
      else if (r < p.rows && n > 0)
        mx_store16<T>(static_cast<T*>(p.Y) + r * p.ldy + c0, n, p.vec_y, x);
    }
  }
}

struct ActBwdParams {
  const void* dY;
  int64_t lddy;
  const uint8_t* q;
  int64_t ldq;
  const uint8_t* s;
  int64_t s_tiles;
  int rows, cols;
  void* dX;
  int64_t lddx;
  float* part;  // [blocks of a strip][cols] column sums, or null
  float* dbias; // the sums themselves, where a strip's blocks are a cluster
  int64_t tiles_m;
  int vec_in, vec_out;
};

// dy act'(x): relu 1 where x > 0; gelu Phi(x) + x phi(x), the derivative of x
// Phi(x), which is h = Phi(-|x|) - |x| phi(x) where x < 0 and 1 - h elsewhere.
template <typename T, int ACT>
__device__ __forceinline__ void act_gradients(const float (&x)[16], float (&dy)[16]) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    if constexpr (ACT == 1) {
      dy[i] *= x[i] > 0.f ? 1.f : 0.f;
      dy[i + 1] *= x[i + 1] > 0.f ? 1.f : 0.f;
    } else if constexpr (ACT == 2 && sizeof(T) == 4) {
#pragma unroll
      for (int k = i; k < i + 2; ++k) {
        const float n = minus_abs(x[k]);
        const float h = __fmaf_rn(n * 0.39894228f, expf(-0.5f * n * n), normcdff(n));
        dy[k] *= x[k] < 0.f ? h : 1.f - h;
      }
    } else if constexpr (ACT == 2) {
      const f32x2 n = pair(minus_abs(x[i]), minus_abs(x[i + 1]));
      f32x2 e;
      const f32x2 c = normal_tail2(n, e);
      const f32x2 h = fma2(mul2(n, pair(0.39894228f)), e, c);
      float h0, h1, g0, g1;
      unpair(h, h0, h1);
      unpair(fma2(h, pair(-1.f), pair(1.f)), g0, g1);
      const f32x2 s = pair(x[i] < 0.f ? h0 : g0, x[i + 1] < 0.f ? h1 : g1);
      unpair(mul2(pair(dy[i], dy[i + 1]), s), dy[i], dy[i + 1]);
    }
  }
}

// JOINED: a strip's blocks are a cluster (grid: blocks x strips), which joins
// their column sums; otherwise (grid: strips x blocks) they go to `part`.
template <typename T, int ACT, bool JOINED, bool GENERAL>
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM - 1 - (GENERAL ? 1 : 0))
    mx_act_backward_kernel(const ActBwdParams p) {
  __shared__ __align__(16) float colsum[8][STRIP];
  __shared__ __align__(16) T stage[GENERAL ? THREADS / 32 : 1][GENERAL ? 4 * STAGE_PITCH : 16];
  const unsigned strip = JOINED ? blockIdx.y : blockIdx.x;
  const unsigned first = JOINED ? blockIdx.x : blockIdx.y;
  const unsigned step = JOINED ? gridDim.x : gridDim.y;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = lane & 7;
  const int64_t cc0 = (int64_t)strip * STRIP, c0 = cc0 + u * 16;
  const int n = (int)min((int64_t)16, max((int64_t)0, (int64_t)p.cols - c0));
  const int64_t b = c0 / 32;
  f32x2 sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0ull;
  // (the general kernel moves rows with whole warps: its threads without columns
  // stay)
  for (int64_t tm = first; (GENERAL || n > 0) && tm < p.tiles_m; tm += step) {
    const int64_t r0 = tm * TILE_ROWS + warp * 4 * UNITS + (lane >> 3);
    MxRow16<T> in[UNITS];
    MxCodes<MX_INT8> c[UNITS];
    uint32_t byte[UNITS];
    int64_t row[UNITS];
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      const int64_t r = min(r0 + 4 * j, (int64_t)p.rows - 1);
      row[j] = r * p.lddy;
      if (!GENERAL || n > 0) {
        c[j] = mx_load_codes<MX_INT8>(p.q + r * p.ldq + c0);
        byte[j] = p.s[mx_scale_word(r, b >> 2, p.s_tiles) + (b & 3)];
      } else {
        c[j] = {};
        byte[j] = 0;
      }
    }
    if (!GENERAL || p.vec_in != MX_SCALAR)
      mx_load_units<T, UNITS>(static_cast<const T*>(p.dY) + c0, row, n, p.vec_in, in);
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      const int64_t r = r0 + 4 * j, w0 = r - (lane >> 3);
      if (!GENERAL && r >= p.rows) continue;
      const int rows4 = left_of(p.rows, w0, 4), cols = left_of(p.cols, cc0, STRIP);
      if (GENERAL && p.vec_in == MX_SCALAR)
        warp_load_rows<T>(static_cast<const T*>(p.dY) + w0 * p.lddy + cc0, p.lddy, rows4, cols,
                          stage[warp], lane, in[j]);
      float dy[16], x[16];
      mx_unpack16<T>(in[j], dy);  // (absent columns 0)
      mx_decode16<MX_INT8>(c[j], e8m0_value(byte[j]), x);
      act_gradients<T, ACT>(x, dy);
      if (!GENERAL || r < p.rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = add2(sum[i], pair(dy[2 * i], dy[2 * i + 1]));
      }
      if (GENERAL && p.vec_out == MX_SCALAR)
        warp_store_rows<T>(static_cast<T*>(p.dX) + w0 * p.lddx + cc0, p.lddx, rows4, cols,
                           stage[warp], lane, dy);
      else if (!GENERAL || (r < p.rows && n > 0))
        mx_store16<T>(static_cast<T*>(p.dX) + r * p.lddx + c0, n, p.vec_out, dy);
    }
  }
  if (JOINED || p.part) {
    // the warp's rows, then the block's, in a fixed order
    float v16[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) unpair(sum[i], v16[2 * i], v16[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v16[i] += __shfl_xor_sync(0xffffffffu, v16[i], 8);
      v16[i] += __shfl_xor_sync(0xffffffffu, v16[i], 16);
      if (lane < 8) colsum[warp][u * 16 + i] = v16[i];
    }
    __syncthreads();
    float v = 0.f;
    if (threadIdx.x < STRIP) {
#pragma unroll
      for (int w = 0; w < 8; ++w) v += colsum[w][threadIdx.x];
    }
    if constexpr (JOINED) {
      __syncthreads();
      if (threadIdx.x < STRIP) colsum[0][threadIdx.x] = v;
      cluster_sync();
      if (first == 0 && threadIdx.x < STRIP / 4) {
        const int64_t c = cc0 + 4 * threadIdx.x;
        const float4 s = cluster_sum4(smem_u32(&colsum[0][4 * threadIdx.x]), (int)step);
        if (c < p.cols) p.dbias[c] = s.x;
        if (c + 1 < p.cols) p.dbias[c + 1] = s.y;
        if (c + 2 < p.cols) p.dbias[c + 2] = s.z;
        if (c + 3 < p.cols) p.dbias[c + 3] = s.w;
      }
      cluster_sync();  // no block leaves while its sums are read
    } else if (threadIdx.x < STRIP && cc0 + threadIdx.x < p.cols) {
      p.part[first * (int64_t)p.cols + cc0 + threadIdx.x] = v;
    }
  }
}

// out[c] = sum of the blocks' column sums, in order
__global__ void mx_column_sum_kernel(const float* part, int blocks, int cols, float* out) {
  pdl_wait();
  pdl_trigger();
  const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= cols) return;
  float v = 0.f;
#pragma unroll 8
  for (int t = 0; t < blocks; ++t) v += part[(int64_t)t * cols + c];
  out[c] = v;
}

inline int vec_of(const void* p, int64_t ld, int64_t es) {
  if (((uintptr_t)p % 32) == 0 && (ld * es) % 32 == 0) return MX_VEC32;
  if (((uintptr_t)p % 16) == 0 && (ld * es) % 16 == 0) return MX_VEC16;
  return MX_SCALAR;
}
inline unsigned grid_of(int64_t tiles) {
  return (unsigned)(tiles < (1ll << 30) ? tiles : (1ll << 30));
}
// Column strips x blocks a strip: one row tile a block while that fits the GPU
// `per_sm` blocks deep, else equal numbers of row tiles in no more blocks than
// are resident at once (a few blocks more would run alone after the others).
dim3 strip_grid(int64_t cols, int64_t tiles_m, int sms, int per_sm) {
  const int64_t strips = (cols + STRIP - 1) / STRIP;
  int64_t most = (int64_t)sms * per_sm / strips;
  most = most < 1 ? 1 : most < tiles_m ? most : tiles_m;
  const int64_t iters = (tiles_m + most - 1) / most;
  return dim3((unsigned)strips, (unsigned)((tiles_m + iters - 1) / iters));
}

template <typename T, int FMT>
cudaError_t quantize_t(const MxQuantArgs& a, LaunchCtx& ctx) {
  QuantParams p;
  p.X = a.X; p.ldx = a.ldx;
  p.rows = a.rows; p.cols = a.cols;
  p.mult = a.mult;
  p.Y = a.Y; p.ldy = a.ldy;
  p.q = static_cast<uint8_t*>(a.q); p.ldq = a.ldq;
  p.s = static_cast<uint8_t*>(a.s);
  p.s_tiles = mx_scale_tiles(FMT, a.cols);
  p.vec_y = a.Y ? vec_of(a.Y, a.ldy, sizeof(T)) : MX_SCALAR;
  const int64_t rows128 = ((int64_t)a.rows + 127) / 128;
  cudaError_t e;
  if (a.transX) {
    p.vec_x = ((uintptr_t)a.X % (2 * sizeof(T))) == 0 && a.ldx % 2 == 0;
    p.tiles_n = ((int64_t)a.cols + TT_COLS - 1) / TT_COLS;
    p.tiles = rows128 * (128 / TT_ROWS) * p.tiles_n;
    ctx.grid = (int)grid_of(p.tiles);
    auto kern = a.mult == 1.f ? mx_quantize_t_kernel<T, FMT, false>
                              : mx_quantize_t_kernel<T, FMT, true>;
    e = launch_kernel(kern, dim3(ctx.grid), dim3(TT_THREADS), 0, ctx.stream, 1, p);
  } else {
    p.vec_x = vec_of(a.X, a.ldx, sizeof(T));
    p.tiles_m = rows128 * (128 / TILE_ROWS);
    const bool general =
        a.mult != 1.f || p.vec_x == MX_SCALAR || (a.Y && p.vec_y == MX_SCALAR);
    const dim3 grid = strip_grid(a.cols, p.tiles_m, a.num_sms, blocks_per_sm(general));
    ctx.grid = (int)(grid.x * grid.y);
    const int act = a.Y ? a.act : -1;
    auto kern = !general ? (act == 2   ? mx_quantize_kernel<T, FMT, 2, false>
                            : act == 1 ? mx_quantize_kernel<T, FMT, 1, false>
                            : act == 0 ? mx_quantize_kernel<T, FMT, 0, false>
                                       : mx_quantize_kernel<T, FMT, -1, false>)
                         : (act == 2   ? mx_quantize_kernel<T, FMT, 2, true>
                            : act == 1 ? mx_quantize_kernel<T, FMT, 1, true>
                            : act == 0 ? mx_quantize_kernel<T, FMT, 0, true>
                                       : mx_quantize_kernel<T, FMT, -1, true>);
    e = launch_kernel(kern, grid, dim3(THREADS), 0, ctx.stream, 1, p);
  }
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

template <typename T, int FMT>
cudaError_t dequantize_t(const MxDequantArgs& a, LaunchCtx& ctx) {
  DequantParams p;
  p.q = static_cast<const uint8_t*>(a.q); p.ldq = a.ldq;
  p.s = static_cast<const uint8_t*>(a.s);
  p.s_tiles = mx_scale_tiles(FMT, a.cols);
  p.rows = a.rows; p.cols = a.cols;
  p.Y = a.Y; p.ldy = a.ldy;
  p.vec_y = vec_of(a.Y, a.ldy, sizeof(T));
  p.tiles_m = ((int64_t)a.rows + TILE_ROWS - 1) / TILE_ROWS;
  const bool general = p.vec_y == MX_SCALAR;
  const dim3 grid = strip_grid(a.cols, p.tiles_m, a.num_sms, 2 * blocks_per_sm(general));
  ctx.grid = (int)(grid.x * grid.y);
  auto kern = general ? mx_dequantize_kernel<T, FMT, true> : mx_dequantize_kernel<T, FMT, false>;
  const cudaError_t e = launch_kernel(kern, grid, dim3(THREADS), 0, ctx.stream, 1, p);
  if (e == cudaSuccess) ctx.launches++;
  return e;
}

// Up to 8 blocks a strip (the portable cluster) join their column sums
// themselves; more leave them for a second kernel (512 x 5632, 8 blocks a strip:
// two launches for the forward and backward pass instead of three).
inline bool act_joined(const dim3& grid) { return grid.y <= 8 && grid.x <= 65535; }
inline int64_t act_tiles(int rows) { return ((int64_t)rows + TILE_ROWS - 1) / TILE_ROWS; }

using ActKernel = void (*)(const ActBwdParams);
template <typename T, bool JOINED>
ActKernel act_kernel(int act, bool general) {
  if (general)
    return act == 2   ? mx_act_backward_kernel<T, 2, JOINED, true>
           : act == 1 ? mx_act_backward_kernel<T, 1, JOINED, true>
                      : mx_act_backward_kernel<T, 0, JOINED, true>;
  return act == 2   ? mx_act_backward_kernel<T, 2, JOINED, false>
         : act == 1 ? mx_act_backward_kernel<T, 1, JOINED, false>
                    : mx_act_backward_kernel<T, 0, JOINED, false>;
}

template <typename T>
cudaError_t act_backward_t(const MxActBwdArgs& a, LaunchCtx& ctx) {
  ActBwdParams p;
  p.dY = a.dY; p.lddy = a.lddy;
  p.q = static_cast<const uint8_t*>(a.q); p.ldq = a.ldq;
  p.s = static_cast<const uint8_t*>(a.s);
  p.s_tiles = mx_scale_tiles(MX_INT8, a.cols);
  p.rows = a.rows; p.cols = a.cols;
  p.dX = a.dX; p.lddx = a.lddx;
  p.part = a.dbias ? a.part : nullptr;
  p.dbias = a.dbias;
  p.vec_in = vec_of(a.dY, a.lddy, sizeof(T));
  p.vec_out = vec_of(a.dX, a.lddx, sizeof(T));
  p.tiles_m = act_tiles(a.rows);
  const dim3 grid = strip_grid(a.cols, p.tiles_m, a.num_sms, BLOCKS_PER_SM - 1);
  ctx.grid = (int)(grid.x * grid.y);
  const bool general = p.vec_in == MX_SCALAR || p.vec_out == MX_SCALAR;
  if (a.dbias && act_joined(grid)) {
    auto kern = act_kernel<T, true>(a.act, general);
    const cudaError_t e =
        launch_kernel(kern, dim3(grid.y, grid.x), dim3(THREADS), 0, ctx.stream, (int)grid.y, p);
    if (e == cudaSuccess) ctx.launches++;
    return e;
  }
  cudaError_t e = launch_kernel(act_kernel<T, false>(a.act, general), grid, dim3(THREADS), 0,
                                ctx.stream, 1, p);
  if (e == cudaSuccess) ctx.launches++;
  if (e == cudaSuccess && a.dbias) {
    e = launch_kernel(mx_column_sum_kernel, dim3((unsigned)(((int64_t)a.cols + 63) / 64)), dim3(64), 0,
                      ctx.stream, 1, (const float*)a.part, (int)grid.y, a.cols, a.dbias);
    if (e == cudaSuccess) ctx.launches++;
  }
  return e;
}

// The three launchers for one element type; mx_elementwise.cu holds the dispatch
// over types, and fp32's, mx_elementwise_f16.cu and _bf16.cu the others'.
template <typename T>
cudaError_t quantize_of(const MxQuantArgs& a, LaunchCtx& ctx) {
  switch (a.format) {
    case MX_FP4: return quantize_t<T, MX_FP4>(a, ctx);
    case MX_FP4_E4M3: return quantize_t<T, MX_FP4_E4M3>(a, ctx);
    default: return quantize_t<T, MX_INT8>(a, ctx);
  }
}
template <typename T>
cudaError_t dequantize_of(const MxDequantArgs& a, LaunchCtx& ctx) {
  switch (a.format) {
    case MX_FP4: return dequantize_t<T, MX_FP4>(a, ctx);
    case MX_FP4_E4M3: return dequantize_t<T, MX_FP4_E4M3>(a, ctx);
    default: return dequantize_t<T, MX_INT8>(a, ctx);
  }
}

}  // namespace

cudaError_t mx_quantize_f16(const MxQuantArgs& a, LaunchCtx& ctx);
cudaError_t mx_quantize_bf16(const MxQuantArgs& a, LaunchCtx& ctx);
cudaError_t mx_dequantize_f16(const MxDequantArgs& a, LaunchCtx& ctx);
cudaError_t mx_dequantize_bf16(const MxDequantArgs& a, LaunchCtx& ctx);
cudaError_t mx_act_backward_f16(const MxActBwdArgs& a, LaunchCtx& ctx);
cudaError_t mx_act_backward_bf16(const MxActBwdArgs& a, LaunchCtx& ctx);
}  // namespace gb300
