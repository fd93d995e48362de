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

// ---------------------------------------------------------------- elements
// two fp32 values -> two e2m1 codes, lo in the low half (nearest, ties to
// even, at most 6)
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
      "cvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}
// the low byte's two e2m1 codes -> two fp16 values (exact)
__device__ __forceinline__ uint32_t e2m1_half2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.u8.u32 t, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(byte));
  return r;
}

// 16 elements' codes: 8 bytes of e2m1 pairs or 16 signed bytes.
template <int FMT>
struct MxCodes {
  static constexpr int WORDS = FMT == MX_INT8 ? 4 : 2;
  uint32_t w[WORDS];
};

// y = x / scale, with the scale's byte already chosen from the block
template <int FMT>
__device__ __forceinline__ void mx_encode16(const float (&x)[16], uint32_t byte,
                                            MxCodes<FMT>& c) {
  float y[16];
  if constexpr (FMT == MX_FP4_E4M3) {
    // a correctly rounded quotient: it is a tie between two codes only where
    // x / scale is one
    const float s = e4m3_value(byte);
    // (a scale of 0: every code 0, with its element's sign)
    const bool some = byte != 0u && byte != 0x7Fu;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      y[i] = some ? __fdiv_rn(x[i], s) : byte == 0u ? copysignf(0.f, x[i]) : 0.f;
  } else {
    // times 2^(127 - byte), a normal number for every byte up to 253
    const float inv = __uint_as_float((254u - byte) << 23);
    const bool some = byte != 255u;
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = some ? x[i] * inv : 0.f;
  }
  if constexpr (FMT == MX_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        int q = __float2int_rn(y[4 * i + j]);
        q = q > 127 ? 127 : q < -127 ? -127 : q;
        v |= (uint32_t)(q & 255) << (8 * j);
      }
      c.w[i] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) v |= e2m1_pair(y[8 * i + 2 * j], y[8 * i + 2 * j + 1]) << (8 * j);
      c.w[i] = v;
    }
  }
}

template <int FMT>
__device__ __forceinline__ void mx_decode16(const MxCodes<FMT>& c, float scale, float (&x)[16]) {
  if constexpr (FMT == MX_INT8) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      x[i] = (float)(int8_t)((c.w[i >> 2] >> (8 * (i & 3))) & 255u) * scale;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t h = e2m1_half2((c.w[i >> 2] >> (8 * (i & 3))) & 255u);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[2 * i] = f.x * scale;
      x[2 * i + 1] = f.y * scale;
    }
  }
}

// ---------------------------------------------------------------- 16 values of a row
// Loads and stores of 16 consecutive elements as fp32: 16-byte accesses where
// the rows allow, otherwise (or at a row's end) element by element, absent
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

template <typename T>
__device__ __forceinline__ MxRow16<T> mx_load16(const T* p, int n, bool vec) {
  MxRow16<T> r;
  if (vec && n >= 16) {
#pragma unroll
    for (int i = 0; i < MxRow16<T>::VECS; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    T e[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) e[i] = i < n ? p[i] : MxIo<T>::from(0.f);
    memcpy(&r, e, sizeof(r));
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void mx_unpack16(const MxRow16<T>& r, float (&x)[16]) {
  T e[16];
  memcpy(e, &r, sizeof(r));
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = MxIo<T>::to(e[i]);
}
template <typename T>
__device__ __forceinline__ void mx_store16(T* p, int n, bool vec, const float (&x)[16]) {
  T e[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) e[i] = MxIo<T>::from(x[i]);
  if (vec && n >= 16) {
    MxRow16<T> r;
    memcpy(&r, e, sizeof(r));
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
