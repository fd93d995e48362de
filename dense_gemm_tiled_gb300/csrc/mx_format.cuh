// Microscaled storage: device helpers shared by the kernels that write and
// read it (layout: include/gemm.h, gemm_mx_format_t).
//
// A block's scale is a power of two 2^(byte - 127) (e8m0, byte 255 = NaN) or
// an e4m3 number; its elements are e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and
// their negatives), two a byte, or signed bytes.  A power of two makes x /
// scale, and code * scale, exact in fp32, so the one rounding of a stored
// value is the one to its code.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gb300 {

// gemm_mx_format_t
enum { MX_FP4 = 0, MX_FP4_E4M3 = 1, MX_INT8 = 2 };

__host__ __device__ constexpr int mx_block(int fmt) { return fmt == MX_FP4_E4M3 ? 16 : 32; }
__host__ __device__ constexpr int mx_blocks(int fmt, int cols) {
  return (int)(((int64_t)cols + mx_block(fmt) - 1) / mx_block(fmt));
}
// bytes of a row of codes, in whole 16-byte units
__host__ __device__ constexpr int64_t mx_row_bytes(int fmt, int64_t cols) {
  const int64_t b = fmt == MX_INT8 ? cols : (cols + 1) / 2;
  return (b + 15) / 16 * 16;
}
// Scale tiles: 128 rows x 4 blocks of bytes, 512 bytes each, tiles of a row
// range in block order.  Row r, block b of a tile lies at (r % 32) * 16 +
// (r / 32) * 4 + b: 32 rows of four 4-byte words, the form in which the tensor
// core's scale operand is copied into tensor memory (a row of the tile is a
// lane, a word a column), so that a product's scales need no re-laying.
__host__ __device__ constexpr int64_t mx_scale_tiles(int fmt, int cols) {
  return ((int64_t)mx_blocks(fmt, cols) + 3) / 4;
}
__host__ __device__ constexpr int64_t mx_scale_bytes(int fmt, int64_t rows, int cols) {
  return (rows + 127) / 128 * mx_scale_tiles(fmt, cols) * 512;
}
// byte offset of the word that holds row r's scales of blocks 4t .. 4t + 3
__host__ __device__ constexpr int64_t mx_scale_word(int64_t r, int64_t t, int64_t tiles) {
  return ((r >> 7) * tiles + t) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// ---------------------------------------------------------------- scales
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  // 2^-127 is an fp32 subnormal; 255 is NaN
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
  return __half2float(__half(h));
}
template <int FMT>
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return FMT == MX_FP4_E4M3 ? e4m3_value(byte) : e8m0_value(byte);
}
// The scale byte of a block whose largest magnitude is `amax` (which is not
// finite if the block holds a NaN or an infinity: the scale is then NaN).
//   e8m0: floor(log2 amax) - emax, emax the exponent of the largest code (6 =
//   1.5 * 2^2; 127 = 1.98 * 2^6): fp32's exponent field less emax, at least 0.
//   e4m3: amax / 6 rounded to nearest even, at most 448.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  if (FMT == MX_FP4_E4M3) {
    if (bits >= 0x7F800000u) return 0x7Fu;
    return (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.0f), __NV_SATFINITE, __NV_E4M3);
  }
  if (bits >= 0x7F800000u) return 255u;
  const int e = (int)(bits >> 23) - (FMT == MX_FP4 ? 2 : 6);
  return e > 0 ? (uint32_t)e : 0u;
}

// ---------------------------------------------------------------- pairs of fp32
// Two IEEE fp32 operations an instruction; the elementwise kernels issue more than
// half of what an SM can, so they work on pairs throughout.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 pair(float v) { return pair(v, v); }
__device__ __forceinline__ void unpair(f32x2 p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// ---------------------------------------------------------------- elements
// eight fp32 values -> eight e2m1 codes, the first in the lowest half byte
// (nearest, ties to even, at most 6)
__device__ __forceinline__ uint32_t e2m1_word(const float* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}
// a word's eight e2m1 codes -> eight fp16 values, in pairs (exact)
__device__ __forceinline__ void e2m1_halves(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 16 elements' codes: 8 bytes of e2m1 pairs or 16 signed bytes.
template <int FMT>
struct MxCodes {
  static constexpr int WORDS = FMT == MX_INT8 ? 4 : 2;
  uint32_t w[WORDS];
};

// Codes of x / scale, the scale's byte already chosen from the block; `amax`
// the block's largest magnitude.  Whole warps.
template <int FMT>
__device__ __forceinline__ void mx_encode16(const float (&x)[16], uint32_t byte, float amax,
                                            MxCodes<FMT>& c) {
  if constexpr (FMT == MX_FP4_E4M3) {
    // The correctly rounded quotient (a tie between two codes only where x /
    // scale is one) from the correctly rounded reciprocal r of the block's
    // scale: y0 = rn(x r), y = rn(y0 + r (x - y0 s)) with the residual exact in
    // an FMA (P. Markstein, "Computation of elementary functions on the IBM RISC
    // System/6000 processor", 1990).  |x| is at most a few times 6 s, or 448 is
    // s, so nothing overflows; where the residual is inexact (x below 2^-100) y
    // is far below every code.  Computed negated, and the codes' signs turned
    // back: a residual of 0 times -r is -0, to which a zero quotient of either
    // sign adds without losing its own.
    float y[16];
    const float s = e4m3_value(byte);
    if (byte == 0u) {  // every code 0, with its element's sign
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = copysignf(0.f, -x[i]);
    } else {
      const float r = __frcp_rn(s);
      const f32x2 r2 = pair(-r), s2 = pair(s);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const f32x2 v = pair(x[i], x[i + 1]), y0 = mul2(v, r2);
        unpair(fma2(fma2(y0, s2, v), r2, y0), y[i], y[i + 1]);
      }
    }
    c.w[0] = e2m1_word(y) ^ 0x88888888u;
    c.w[1] = e2m1_word(y + 8) ^ 0x88888888u;
    if (byte == 0x7Fu) c.w[0] = c.w[1] = 0u;
  } else {
    // times 2^(127 - byte), a normal number for every byte up to 253: exact
    // (but where the product is far below every code)
    const float inv = __uint_as_float((254u - byte) << 23);
    if constexpr (FMT == MX_INT8) {
      // x inv + 1.5 * 2^23 rounds to the nearest whole number (even on a tie),
      // two's complement in the low byte; only a block whose amax lies within
      // half a step of 128 can round to +-128, which saturates
      constexpr float ROUND = 12582912.f;
      const f32x2 inv2 = pair(inv), round2 = pair(ROUND);
      float f[16];
#pragma unroll
      for (int i = 0; i < 16; i += 2)
        unpair(fma2(pair(x[i], x[i + 1]), inv2, round2), f[i], f[i + 1]);
      if (__any_sync(0xffffffffu, amax * inv >= 127.5f)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = fminf(fmaxf(f[i], ROUND - 127.f), ROUND + 127.f);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c.w[i] = __byte_perm(
            __byte_perm(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), 0x0040),
            __byte_perm(__float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]), 0x0040),
            0x5410);
      if (byte == 255u) c.w[0] = c.w[1] = c.w[2] = c.w[3] = 0u;
    } else {
      float y[16];
      const f32x2 inv2 = pair(inv);
#pragma unroll
      for (int i = 0; i < 16; i += 2) unpair(mul2(pair(x[i], x[i + 1]), inv2), y[i], y[i + 1]);
      c.w[0] = e2m1_word(y);
      c.w[1] = e2m1_word(y + 8);
      if (byte == 255u) c.w[0] = c.w[1] = 0u;
    }
  }
}

template <int FMT>
__device__ __forceinline__ void mx_decode16(const MxCodes<FMT>& c, float scale, float (&x)[16]) {
  if constexpr (FMT == MX_INT8) {
    // code + 128 as the low byte of 2^23 is an fp32 number; less 2^23 + 128 it is
    // the code
    const f32x2 base2 = pair(-8388736.f), s2 = pair(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = c.w[i] ^ 0x80808080u;
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        unpair(mul2(add2(pair(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + j)),
                              __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7541 + j))),
                         base2),
                    s2),
               x[4 * i + j], x[4 * i + j + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h[4];
      e2m1_halves(c.w[i], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        unpair(mul2(pair(f.x, f.y), pair(scale)), x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
      }
    }
  }
}

// ---------------------------------------------------------------- 16 values of a row
// Loads and stores of 16 consecutive elements as fp32: 32- or 16-byte accesses
// where the rows allow, otherwise (or at a row's end) element by element, absent
// elements 0.
template <typename T>
struct MxIo;
template <>
struct MxIo<float> {
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
};
template <>
struct MxIo<__half> {
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
};
template <>
struct MxIo<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};

template <typename T>
struct MxRow16 {
  static constexpr int VECS = 16 * (int)sizeof(T) / 16;
  uint4 v[VECS];
};

// How a row's 16-element units may be accessed: 32 bytes at a time, 16, or
// element by element.
enum { MX_SCALAR = 0, MX_VEC16 = 1, MX_VEC32 = 2 };

__device__ __forceinline__ void mx_ld32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                 "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ void mx_st32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
// U units of 16 elements, `step` elements apart (n elements of each exist);
// with the loads of a vector path issued together.
template <typename T, int U>
__device__ __forceinline__ void mx_load_units(const T* p, const int64_t (&row)[U], int n, int vec,
                                              MxRow16<T> (&in)[U]) {
  if (n == 16 && vec == MX_VEC32) {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < MxRow16<T>::VECS; i += 2)
        mx_ld32(p + row[j] + i * (16 / (int)sizeof(T)), in[j].v[i], in[j].v[i + 1]);
  } else if (n == 16 && vec == MX_VEC16) {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < MxRow16<T>::VECS; ++i)
        in[j].v[i] = reinterpret_cast<const uint4*>(p + row[j])[i];
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      T e[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) e[i] = i < n ? p[row[j] + i] : MxIo<T>::from(0.f);
      memcpy(&in[j], e, sizeof(in[j]));
    }
  }
}

// Largest magnitude of 16 loaded values, as fp32 bits: a NaN counts above
// infinity, infinity above all numbers.  16-bit types two at a time.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b, __half*) {
  const __half2 r = __hmax2_nan(__habs2(*reinterpret_cast<const __half2*>(&a)),
                                __habs2(*reinterpret_cast<const __half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b, __nv_bfloat16*) {
  const __nv_bfloat162 r = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t mx_max_abs16(const MxRow16<T>& r) {
  uint32_t m = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < MxRow16<T>::VECS; ++i)
      m = max(max(max(m, r.v[i].x & 0x7FFFFFFFu), r.v[i].y & 0x7FFFFFFFu),
              max(r.v[i].z & 0x7FFFFFFFu, r.v[i].w & 0x7FFFFFFFu));
    return m;
  } else {
#pragma unroll
    for (int i = 0; i < MxRow16<T>::VECS; ++i) {
      m = max_abs2(m, r.v[i].x, (T*)nullptr);
      m = max_abs2(m, r.v[i].y, (T*)nullptr);
      m = max_abs2(m, r.v[i].z, (T*)nullptr);
      m = max_abs2(m, r.v[i].w, (T*)nullptr);
    }
    // (as bits: a NaN's above infinity's)
    const unsigned short h = (unsigned short)max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
    T e;
    memcpy(&e, &h, 2);
    return __float_as_uint(MxIo<T>::to(e)) & 0x7FFFFFFFu;
  }
}
template <typename T>
__device__ __forceinline__ void mx_unpack16(const MxRow16<T>& r, float (&x)[16]) {
  T e[16];
  memcpy(e, &r, sizeof(r));
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = MxIo<T>::to(e[i]);
}
template <typename T>
__device__ __forceinline__ void mx_store16(T* p, int n, int vec, const float (&x)[16]) {
  T e[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) e[i] = MxIo<T>::from(x[i]);
  MxRow16<T> r;
  memcpy(&r, e, sizeof(r));
  if (n == 16 && vec == MX_VEC32) {
#pragma unroll
    for (int i = 0; i < MxRow16<T>::VECS; i += 2)
      mx_st32(p + i * (16 / (int)sizeof(T)), r.v[i], r.v[i + 1]);
  } else if (n == 16 && vec == MX_VEC16) {
#pragma unroll
    for (int i = 0; i < MxRow16<T>::VECS; ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = e[i];
  }
}
template <int FMT>
__device__ __forceinline__ MxCodes<FMT> mx_load_codes(const uint8_t* p) {
  MxCodes<FMT> c;
  if constexpr (FMT == MX_INT8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    c.w[0] = v.x; c.w[1] = v.y; c.w[2] = v.z; c.w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    c.w[0] = v.x; c.w[1] = v.y;
  }
  return c;
}
template <int FMT>
__device__ __forceinline__ void mx_store_codes(uint8_t* p, const MxCodes<FMT>& c) {
  if constexpr (FMT == MX_INT8)
    *reinterpret_cast<uint4*>(p) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(c.w[0], c.w[1]);
}
// bytes of 16 codes
template <int FMT>
__host__ __device__ constexpr int mx_bytes16() { return FMT == MX_INT8 ? 16 : 8; }

}  // namespace gb300
