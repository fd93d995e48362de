// C entry points of the microscaled operands (include/gemm.h): argument
// checks, choice of kernel, scratch, launch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/gemm.h"
#include "internal.h"
#include "mx_format.cuh"

using namespace gb300;

static_assert((int)GEMM_MX_FP4 == (int)MX_FP4 && (int)GEMM_MX_FP4_E4M3 == (int)MX_FP4_E4M3 &&
                  (int)GEMM_MX_INT8 == (int)MX_INT8,
              "format codes");

namespace {

constexpr int64_t LIM = (int64_t)1 << 31;
// Products' sizes end earlier: the kernels and the copies around them count
// stages, tiles and a grid's strides (up to 2^17 elements past an end) in 32 bits.
constexpr int64_t PRODUCT_LIM = LIM - ((int64_t)1 << 18);

// Rows (columns of A, in the tn product) up to which the streaming kernels take a
// product: as many as they hold.  In a graph, us, at 32 of them, streamed against
// converted (expanded: 61, 18, 20; int8 66, 19, 20):
//                       8192 x 8192    5632 x 2048    2048 x 5632  (N x K)
//   nt fp4 fp16         23.0 / 28.0     9.2 /  9.6    11.0 / 11.1
//   nt fp4 bf16         24.3 / 32.9     9.6 / 10.5    11.4 / 12.2
//   nt fp4_e4m3 fp16    19.3 / 28.6     8.2 /  9.3     9.8 / 11.0
//   tn int8 fp16        26.0 / 35.0     9.5 / 10.9    11.7 / 12.7
//   tn int8 bf16        31.4 / 35.0    10.3 / 10.7    13.6 / 12.6
// Two stored operands take the same bound, where the 4-bit tensor-core kernel
// would be level or faster from one row on with fp4 (8192 x 8192: 8 rows 20.4 /
// 18.4, 32 rows 46.0 / 12.3) and from 16 on with fp4_e4m3 (8 rows 15.9 / 19.2, 16
// rows 20.0 / 18.8, 32 rows 29.0 / 13.3).
constexpr int64_t WGRAD_ROWS = 32;
constexpr int64_t STREAM_ROWS = 32;

inline bool known_format(int f) { return f >= GEMM_MX_FP4 && f <= GEMM_MX_INT8; }
inline bool known_type(int d) {
  return d == GEMM_F32 || d == GEMM_F16_F32ACC || d == GEMM_BF16_F32ACC;
}
inline bool known_act(int a) {
  return a == GEMM_ACT_NONE || a == GEMM_ACT_RELU || a == GEMM_ACT_GELU;
}
inline int64_t type_bytes(int d) { return d == GEMM_F32 ? 4 : 2; }

struct Span {
  uintptr_t lo, hi;
};
// bytes [rows, cols] of `e`-byte elements at pitch ld covers
inline Span span_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t e) {
  const uintptr_t b = (uintptr_t)p;
  if (!p || rows <= 0 || cols <= 0) return {0, 0};
  return {b, b + (uintptr_t)(((rows - 1) * ld + cols) * e)};
}
inline bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// a plain matrix: pitch, pointer and element alignment
int check_plain(const void* p, int64_t cols, int64_t ld, int64_t e) {
  if (ld < (cols > 1 ? cols : 1)) return GEMM_ERR_INVALID_ARG;
  if (!p || ((uintptr_t)p % (uintptr_t)e) != 0) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}
// a stored matrix: codes in 16-byte rows, scale tiles 16-byte aligned
int check_stored(int format, const void* q, int64_t ldq, const void* s, int64_t cols) {
  if (ldq < mx_row_bytes(format, cols) || ldq % 16 != 0) return GEMM_ERR_INVALID_ARG;
  if (!q || !s || ((uintptr_t)q % 16) != 0 || ((uintptr_t)s % 16) != 0)
    return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}
inline Span span_q(int format, const void* q, int64_t ldq, int64_t rows, int64_t cols) {
  return span_of(q, rows, mx_row_bytes(format, cols), ldq, 1);
}
inline Span span_s(int format, const void* s, int64_t rows, int64_t cols) {
  const uintptr_t b = (uintptr_t)s;
  return {b, b + (uintptr_t)mx_scale_bytes(format, rows, (int)cols)};
}

struct Scratch {
  void* ptr = nullptr;
  cudaStream_t stream = nullptr;
  ~Scratch() { api_scratch_free(ptr, stream); }
  cudaError_t get(size_t bytes, cudaStream_t s) {
    stream = s;
    return api_scratch(&ptr, bytes, s);
  }
};

// shared by the products: sizes, C, bias, activation
int check_product(int64_t M, int64_t N, int64_t K, int dtype, const void* C, int64_t ldc,
                  const void* bias, int act) {
  if (!known_type(dtype) || !known_act(act)) return GEMM_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (M > PRODUCT_LIM || N > PRODUCT_LIM || K > PRODUCT_LIM) return GEMM_ERR_UNSUPPORTED;
  if (ldc < (N > 1 ? N : 1)) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  const int64_t e = type_bytes(dtype);
  int rc = check_plain(C, N, ldc, e);
  if (rc != GEMM_OK) return rc;
  if (bias && ((uintptr_t)bias % (uintptr_t)e) != 0) return GEMM_ERR_INVALID_ARG;
  if (bias && meet(span_of(C, M, N, ldc, e), span_of(bias, 1, N, N, e))) return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

}  // namespace

extern "C" {

int64_t gemm_mx_row_bytes(int format, int64_t cols) {
  return known_format(format) && cols >= 0 && cols < LIM ? mx_row_bytes(format, cols) : -1;
}

int64_t gemm_mx_scale_bytes(int format, int64_t rows, int64_t cols) {
  if (!known_format(format) || rows < 0 || cols < 0 || rows >= LIM || cols >= LIM) return -1;
  return mx_scale_bytes(format, rows, (int)cols);
}

int gemm_mx_quantize(int format, int transX, int64_t rows, int64_t cols, int dtype, float mult,
                     const void* X, int64_t ldx, int act, void* Y, int64_t ldy, void* q,
                     int64_t ldq, void* scales, gemm_stream_t stream) {
  api_reset();
  if (!known_format(format) || (transX != 0 && transX != 1) || !known_type(dtype) ||
      !known_act(act) || !isfinite(mult))
    return GEMM_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0) return GEMM_ERR_INVALID_ARG;
  if (rows >= LIM || cols >= LIM) return GEMM_ERR_UNSUPPORTED;
  if (!Y && act != GEMM_ACT_NONE) return GEMM_ERR_INVALID_ARG;
  if (Y && transX) return GEMM_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return GEMM_OK;
  const int64_t e = type_bytes(dtype);
  const int64_t xr = transX ? cols : rows, xc = transX ? rows : cols;
  int rc = check_plain(X, xc, ldx, e);
  if (rc == GEMM_OK && Y) rc = check_plain(Y, cols, ldy, e);
  if (rc == GEMM_OK) rc = check_stored(format, q, ldq, scales, cols);
  if (rc != GEMM_OK) return rc;
  const Span sx = span_of(X, xr, xc, ldx, e), sy = span_of(Y, rows, cols, ldy, e);
  const Span sq = span_q(format, q, ldq, rows, cols), ss = span_s(format, scales, rows, cols);
  // (Y may be X itself: every element is read before it is written)
  if (meet(sq, sx) || meet(ss, sx) || meet(sq, ss) || meet(sq, sy) || meet(ss, sy) ||
      (meet(sx, sy) && !(X == Y && ldx == ldy)))
    return GEMM_ERR_ALIAS;
  ApiState st;
  rc = api_state(&st);
  if (rc != GEMM_OK) return rc;
  LaunchCtx ctx{(cudaStream_t)stream, st.status, st.timeout_ns, 0};
  MxQuantArgs a{format, dtype, transX, (int)rows, (int)cols, mult, X, ldx, Y, ldy, act, q, ldq,
                scales, st.sms};
  return api_done(GEMM_PATH_MX, ctx, launch_mx_quantize(a, ctx));
}

int gemm_mx_dequantize(int format, int64_t rows, int64_t cols, const void* q, int64_t ldq,
                       const void* scales, int dtype, void* Y, int64_t ldy,
                       gemm_stream_t stream) {
  api_reset();
  if (!known_format(format) || !known_type(dtype)) return GEMM_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0) return GEMM_ERR_INVALID_ARG;
  if (rows >= LIM || cols >= LIM) return GEMM_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return GEMM_OK;
  int rc = check_plain(Y, cols, ldy, type_bytes(dtype));
  if (rc == GEMM_OK) rc = check_stored(format, q, ldq, scales, cols);
  if (rc != GEMM_OK) return rc;
  const Span sy = span_of(Y, rows, cols, ldy, type_bytes(dtype));
  if (meet(sy, span_q(format, q, ldq, rows, cols)) || meet(sy, span_s(format, scales, rows, cols)))
    return GEMM_ERR_ALIAS;
  ApiState st;
  rc = api_state(&st);
  if (rc != GEMM_OK) return rc;
  LaunchCtx ctx{(cudaStream_t)stream, st.status, st.timeout_ns, 0};
  MxDequantArgs a{format, dtype, (int)rows, (int)cols, q, ldq, scales, Y, ldy, st.sms};
  return api_done(GEMM_PATH_MX, ctx, launch_mx_dequantize(a, ctx));
}

int gemm_mx_act_backward(int64_t rows, int64_t cols, int dtype, int act, const void* dY,
                         int64_t lddy, const void* q, int64_t ldq, const void* scales, void* dX,
                         int64_t lddx, float* dbias, gemm_stream_t stream) {
  api_reset();
  if (!known_type(dtype) || !known_act(act)) return GEMM_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0) return GEMM_ERR_INVALID_ARG;
  if (rows >= LIM || cols >= LIM) return GEMM_ERR_UNSUPPORTED;
  const int64_t e = type_bytes(dtype);
  if (dbias && ((uintptr_t)dbias % 4) != 0) return GEMM_ERR_INVALID_ARG;
  if (cols == 0) return GEMM_OK;
  ApiState st;
  if (rows == 0) {  // an empty sum
    if (!dbias) return GEMM_OK;
    int rc = api_state(&st);
    if (rc != GEMM_OK) return rc;
    LaunchCtx ctx{(cudaStream_t)stream, st.status, st.timeout_ns, 0};
    return api_done(GEMM_PATH_MX, ctx,
                    cudaMemsetAsync(dbias, 0, (size_t)cols * 4, (cudaStream_t)stream));
  }
  int rc = check_plain(dY, cols, lddy, e);
  if (rc == GEMM_OK) rc = check_plain(dX, cols, lddx, e);
  if (rc == GEMM_OK) rc = check_stored(GEMM_MX_INT8, q, ldq, scales, cols);
  if (rc != GEMM_OK) return rc;
  const Span sy = span_of(dY, rows, cols, lddy, e), sx = span_of(dX, rows, cols, lddx, e);
  const Span sq = span_q(GEMM_MX_INT8, q, ldq, rows, cols);
  const Span ss = span_s(GEMM_MX_INT8, scales, rows, cols);
  const Span sd = span_of(dbias, 1, cols, cols, 4);
  // (dX may be dY itself: every element is read before it is written)
  if (meet(sx, sq) || meet(sx, ss) || meet(sd, sx) || meet(sd, sy) || meet(sd, sq) ||
      meet(sd, ss) || (meet(sx, sy) && !(dX == dY && lddx == lddy)))
    return GEMM_ERR_ALIAS;
  rc = api_state(&st);
  if (rc != GEMM_OK) return rc;
  LaunchCtx ctx{(cudaStream_t)stream, st.status, st.timeout_ns, 0};
  MxActBwdArgs a{dtype, (int)rows, (int)cols, act, dY, lddy, q, ldq, scales, dX, lddx, dbias,
                 nullptr, st.sms};
  Scratch ws;
  const size_t need = dbias ? mx_act_backward_scratch(a.rows, a.cols, st.sms) : 0;
  if (need > 0) {
    const cudaError_t ce = ws.get(need, ctx.stream);
    if (ce != cudaSuccess) return api_done(GEMM_PATH_NONE, ctx, ce);
    a.part = static_cast<float*>(ws.ptr);
  }
  return api_done(GEMM_PATH_MX, ctx, launch_mx_act_backward(a, ctx));
}

int gemm_mx4(int format, int64_t M, int64_t N, int64_t K, int dtype, float alpha, float beta,
             const void* A, int64_t lda, const void* As, const void* B, int64_t ldb,
             const void* Bs, void* C, int64_t ldc, const void* bias, int act,
             gemm_stream_t stream) {
  api_reset();
  if (!known_format(format)) return GEMM_ERR_INVALID_ARG;
  if (format == GEMM_MX_INT8) return GEMM_ERR_UNSUPPORTED;
  int rc = check_product(M, N, K, dtype, C, ldc, bias, act);
  if (rc != GEMM_OK || M == 0 || N == 0) return rc;
  const int64_t e = type_bytes(dtype);
  Epilogue ep;
  ep.bias = bias;
  ep.act = act;
  ApiState st;
  if (K > 0) {
    rc = check_stored(format, A, lda, As, K);
    if (rc == GEMM_OK) rc = check_stored(format, B, ldb, Bs, K);
    if (rc != GEMM_OK) return rc;
    const Span sc = span_of(C, M, N, ldc, e);
    if (meet(sc, span_q(format, A, lda, M, K)) || meet(sc, span_s(format, As, M, K)) ||
        meet(sc, span_q(format, B, ldb, N, K)) || meet(sc, span_s(format, Bs, N, K)))
      return GEMM_ERR_ALIAS;
  }
  rc = api_state(&st);
  if (rc != GEMM_OK) return rc;
  LaunchCtx ctx{(cudaStream_t)stream, st.status, st.timeout_ns, 0};
  if (K == 0)
    return api_done(GEMM_PATH_SCALE, ctx,
                    launch_scale(dtype, (int)M, (int)N, C, ldc, beta, ctx, ep));
  if (M <= STREAM_ROWS) {
    MxStreamArgs a{format, dtype, (int)M, (int)N, (int)K, A, lda, As, B, ldb, Bs, C, ldc, alpha,
                   beta, ep, st.sms, st.fault_injection};
    const cudaError_t ce = launch_mx_stream(a, ctx);
    if (ce != cudaErrorNotSupported) return api_done(GEMM_PATH_MX_STREAM, ctx, ce);
  }
  Mx4Args a{format, dtype, (int)M, (int)N, (int)K, A, lda, As, B, ldb, Bs, C, ldc, alpha, beta,
            ep, st.sms, st.fault_injection};
  return api_done(GEMM_PATH_MX_TC, ctx, launch_mx4(a, ctx));
}

int gemm_mx(int format, int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype,
            float alpha, float beta, const void* A, int64_t lda, const void* B, int64_t ldb,
            const void* Bs, void* C, int64_t ldc, const void* bias, int act,
            gemm_stream_t stream_h) {
  api_reset();
  if (!known_format(format) || (transA != 0 && transA != 1) || (transB != 0 && transB != 1))
    return GEMM_ERR_INVALID_ARG;
  int rc = check_product(M, N, K, dtype, C, ldc, bias, act);
  if (rc != GEMM_OK || M == 0 || N == 0) return rc;
  const int64_t e = type_bytes(dtype);
  const int64_t ar = transA ? K : M, ac = transA ? M : K;
  const int64_t br = transB ? N : K, bc = transB ? K : N;
  cudaStream_t stream_ = (cudaStream_t)stream_h;
  Epilogue ep;
  ep.bias = bias;
  ep.act = act;
  if (K > 0) {
    rc = check_plain(A, ac, lda, e);
    if (rc == GEMM_OK) rc = check_stored(format, B, ldb, Bs, bc);
    if (rc != GEMM_OK) return rc;
    const Span sc = span_of(C, M, N, ldc, e);
    if (meet(sc, span_of(A, ar, ac, lda, e)) || meet(sc, span_q(format, B, ldb, br, bc)) ||
        meet(sc, span_s(format, Bs, br, bc)))
      return GEMM_ERR_ALIAS;
  }
  ApiState st;
  rc = api_state(&st);
  if (rc != GEMM_OK) return rc;
  LaunchCtx ctx{stream_, st.status, st.timeout_ns, 0};
  if (K == 0)
    return api_done(GEMM_PATH_SCALE, ctx,
                    launch_scale(dtype, (int)M, (int)N, C, ldc, beta, ctx, ep));
  // 16-bit A: kernels that read B as it is stored.  A's rows go through the
  // tensor-memory-access unit: rows off 16-byte alignment (and a single row
  // stored as a column) are copied into scratch first, once the kernel is settled.
  const bool column = transA && M == 1;  // op(A) is one row
  const bool fp4 = format != GEMM_MX_INT8;
  const int tA = column && fp4 ? 0 : transA;
  const bool stream = fp4 && transB && !tA && M <= STREAM_ROWS;
  const bool wgrad = !fp4 && tA && !transB && M <= WGRAD_ROWS;
  if (dtype != GEMM_F32 &&
      (stream || wgrad ||
       mx_mixed_takes(format, tA, transB, (int)M, (int)N, (int)K, st.sms))) {
    Scratch ws;
    const void* Ad = A;
    int64_t ldad = lda;
    cudaError_t ce = cudaSuccess;
    const int64_t rows = tA ? K : M, cols = tA ? M : K;
    const bool strided = column && !tA && lda != 1;
    if (strided || ((uintptr_t)A % 16) != 0 || (lda % 8 != 0 && rows > 1)) {
      ldad = (cols + 7) / 8 * 8;
      ce = ws.get((size_t)(rows * ldad * 2), stream_);
      if (ce == cudaSuccess)
        ce = strided ? launch_copy_rows(2, (int)K, 1, A, lda, ws.ptr, 1, ctx)
                     : launch_repack_16((int)rows, (int)cols, A, rows == 1 ? cols : lda, ws.ptr,
                                        ldad, ctx);
      Ad = ws.ptr;
      if (ce != cudaSuccess) return api_done(GEMM_PATH_NONE, ctx, ce);
    }
    if (rows == 1) ldad = (cols + 7) / 8 * 8;
    MxStreamArgs a{format, dtype, (int)M, (int)N, (int)K, Ad, ldad, nullptr, B, ldb, Bs, C, ldc,
                   alpha, beta, ep, st.sms, st.fault_injection, tA, transB};
    ce = stream  ? launch_mx_stream(a, ctx)
         : wgrad ? launch_mx_wgrad(a, ctx)
                 : launch_mx_mixed(a, ctx);
    // (not supported: more columns than the grid holds, or a pitch past a tensor
    // map's)
    if (ce != cudaErrorNotSupported)
      return api_done(stream || wgrad ? GEMM_PATH_MX_STREAM : GEMM_PATH_MX_CONVERT, ctx, ce);
  }
  // B expanded to the other operand's type in scratch, then that type's product
  const int64_t ldw = (bc + 7) / 8 * 8;
  Scratch ws;
  cudaError_t ce = ws.get((size_t)(br * ldw * e), stream_);
  if (ce != cudaSuccess) return api_done(GEMM_PATH_NONE, ctx, ce);
  MxDequantArgs d{format, dtype, (int)br, (int)bc, B, ldb, Bs, ws.ptr, ldw, st.sms};
  ce = launch_mx_dequantize(d, ctx);
  rc = api_done(GEMM_PATH_NONE, ctx, ce);
  if (rc != GEMM_OK) return rc;
  rc = api_gemm(transA, transB, M, N, K, dtype, alpha, beta, A, lda, ws.ptr, ldw, C, ldc, stream_,
                ep);
  if (rc == GEMM_OK) api_add_launches(ctx.launches);
  return rc;
}

}  // extern "C"
