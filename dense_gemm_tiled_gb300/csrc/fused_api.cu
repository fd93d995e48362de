// C entry points of the products with a full epilogue and of those grouped by expert
// (include/gemm.h, gemm_fused and gemm_grouped): argument checks, scratch, launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gemm.h"
#include "fused_plan.h"
#include "internal.h"

using namespace gb300;

namespace {

// (the kernels count tiles and strides, up to 2^17 elements past an end, in 32 bits)
constexpr int64_t SIZE_LIM = ((int64_t)1 << 31) - ((int64_t)1 << 18);
constexpr int64_t GROUP_LIM = 65535;

inline int64_t type_bytes(int d) { return d == GEMM_F32 ? 4 : 2; }
inline bool aligned16(const void* p, int64_t ld) { return ((uintptr_t)p % 16) == 0 && ld % 8 == 0; }

struct Span {
  uintptr_t lo = 0, hi = 0;
};
inline bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

struct Scratch {
  void* ptr = nullptr;
  cudaStream_t stream = nullptr;
  ~Scratch() { api_scratch_free(ptr, stream); }
  cudaError_t get(size_t bytes, cudaStream_t s) {
    stream = s;
    return bytes ? api_scratch(&ptr, bytes, s) : cudaSuccess;
  }
};
inline int64_t pad256(int64_t n) { return (n + 255) / 256 * 256; }

// A matrix (or `count` of them, `stride` elements apart) of a call: its pitch,
// pointer and alignment checked, the bytes it covers.  Extents past 2^58 elements are
// refused with the sizes.
int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t count,
                 int64_t stride, int64_t e, Span* s) {
  if (ld < (cols > 1 ? cols : 1)) return GEMM_ERR_INVALID_ARG;
  if (rows <= 0 || cols <= 0 || count <= 0) return GEMM_OK;
  if (!p || ((uintptr_t)p % (uintptr_t)e) != 0) return GEMM_ERR_INVALID_ARG;
  if (rows > 1 && ld > ((int64_t)1 << 58) / rows) return GEMM_ERR_UNSUPPORTED;
  int64_t n = (rows - 1) * ld + cols;
  if (count > 1) {
    if (stride < 0) return GEMM_ERR_INVALID_ARG;
    if (stride > ((int64_t)1 << 58) / count) return GEMM_ERR_UNSUPPORTED;
    n += (count - 1) * stride;
  }
  s->lo = (uintptr_t)p;
  s->hi = s->lo + (uintptr_t)(n * e);
  return GEMM_OK;
}

// A single row has any pitch: one that keeps it aligned.
inline void one_row(int64_t rows, int64_t cols, int64_t* ld) {
  if (rows <= 1) *ld = (cols + 15) / 16 * 16 > 0 ? (cols + 15) / 16 * 16 : 16;
}

// The sizes that a call gives, and its matrices' stored shapes.
struct Call {
  FusedArgs a;
  int64_t a_rows, a_cols, b_rows, b_cols;  // (b: of one group)
  float* dbias;
  Span sA, sB, sY;
};

int check_call(Call& c, int64_t M, int64_t N, int64_t K, int64_t groups, int dtype, int act) {
  if (dtype != GEMM_F32 && dtype != GEMM_F16_F32ACC && dtype != GEMM_BF16_F32ACC)
    return GEMM_ERR_INVALID_ARG;
  if (act < GEMM_ACT_NONE || act > GEMM_ACT_GELU) return GEMM_ERR_INVALID_ARG;
  FusedArgs& a = c.a;
  if ((a.transA != 0 && a.transA != 1) || (a.transB != 0 && a.transB != 1))
    return GEMM_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0 || groups < 0) return GEMM_ERR_INVALID_ARG;
  if (M > SIZE_LIM || N > SIZE_LIM || K > SIZE_LIM || groups > GROUP_LIM)
    return GEMM_ERR_UNSUPPORTED;
  a.M = (int)M; a.N = (int)N; a.K = (int)K;
  a.groups = (int)groups;
  a.dtype = dtype;  // (gemm_dtype_t 0, 1, 2 are the kernels' types)
  a.act = act;
  if (a.kind != FUSED_DENSE && groups > 0 && (!a.offsets || ((uintptr_t)a.offsets % 4) != 0))
    return GEMM_ERR_INVALID_ARG;
  const int64_t e = type_bytes(dtype);
  c.a_rows = a.transA ? K : M; c.a_cols = a.transA ? M : K;
  c.b_rows = a.transB ? N : K; c.b_cols = a.transB ? K : N;
  const bool inner = a.kind == FUSED_INNER;
  const int64_t nb = inner ? 1 : groups, ny = inner ? groups : 1;
  int rc = check_matrix(a.Y, M, N, a.ldy, ny, a.stride_y, e, &c.sY);
  if (rc == GEMM_OK) rc = check_matrix(a.A, c.a_rows, c.a_cols, a.lda, 1, 0, e, &c.sA);
  if (rc == GEMM_OK) rc = check_matrix(a.B, c.b_rows, c.b_cols, a.ldb, nb, a.stride_b, e, &c.sB);
  if (rc != GEMM_OK) return rc;
  // (matrices of C that would overlap one another)
  if (inner && groups > 1 && M > 0 && N > 0 && a.stride_y < (M - 1) * a.ldy + N) return GEMM_ERR_ALIAS;
  Span so;
  if (a.kind != FUSED_DENSE && groups > 0) {
    so.lo = (uintptr_t)a.offsets;
    so.hi = so.lo + (uintptr_t)(groups + 1) * 4;
  }
  if (meet(c.sY, c.sA) || meet(c.sY, c.sB) || meet(c.sY, so)) return GEMM_ERR_ALIAS;
  if (ny <= 1) one_row(M, N, &a.ldy);
  one_row(c.a_rows, c.a_cols, &a.lda);
  if (nb <= 1) one_row(c.b_rows, c.b_cols, &a.ldb);
  return GEMM_OK;
}

// The operand copied into rows of a 16-byte pitch, where it does not have one (of
// `count` matrices; one launch where they follow one another)
cudaError_t repack(const void*& p, int64_t& ld, int64_t& stride, int64_t rows, int64_t cols,
                   int64_t count, char* to, LaunchCtx& ctx) {
  const int64_t pitch = (cols + 7) / 8 * 8;
  cudaError_t e = cudaSuccess;
  if (count > 1 && stride == rows * ld && rows * count <= SIZE_LIM) {
    e = launch_repack_16((int)(rows * count), (int)cols, p, ld, to, pitch, ctx);
  } else {
    for (int64_t i = 0; i < count && e == cudaSuccess; ++i)
      e = launch_repack_16((int)rows, (int)cols, (const char*)p + i * stride * 2, ld,
                           to + i * rows * pitch * 2, pitch, ctx);
  }
  p = to;
  ld = pitch;
  if (stride != 0) stride = rows * pitch;  // (0: one matrix for all groups)
  return e;
}

int run_call(Call& c, cudaStream_t stream) {
  ApiState st;
  const int rc = api_state(&st);
  if (rc != GEMM_OK) return rc;
  LaunchCtx ctx{stream, st.status, st.timeout_ns, 0};
  FusedArgs& a = c.a;
  a.splits = 1;
  a.num_sms = st.sms;
  a.fault_injection = st.fault_injection;
  const bool inner = a.kind == FUSED_INNER, none = a.M == 0 && !inner;  // (no rows at all)
  const int64_t part_bytes = c.dbias ? pad256(fused_part_floats(a.M, a.groups, a.N) * 4) : 0;
  cudaError_t e = cudaSuccess;
  int path = GEMM_PATH_NONE;
  Scratch ws;
  if (a.dtype == GEMM_F32) {
    // The raw products go where the call writes anyway, but not over what it reads, nor
    // into rows off 16-byte alignment, which slow the products (1000 x 3001 x 777 112 us,
    // 94 into aligned rows).
    float* P = static_cast<float*>(a.U ? a.U : a.Y);
    int64_t ldp = a.U ? a.ldu : a.ldy;
    // (Bias and relu alone: the product's own kernels apply them.  Not gelu: theirs is another
    // evaluation, and a layer's values would change when U is kept.  Its pass, us: 4096^3
    // 1999 -> 2009, 1 x 5632 x 2048 73.2 -> 76.5, 1000 x 3001 x 777 116 -> 115.  The pass's form
    // in the products' own epilogues doubled their code: 4096^3 2197, and gemm() itself at
    // 1000 x 3001 x 777 110 -> 119.)
    const bool plain = a.kind == FUSED_DENSE && !a.U && a.mode == FUSED_NONE && !c.dbias &&
                       a.act != GEMM_ACT_GELU;
    // Slices of K are apart too; those of weights' gradients are finished as one matrix, so
    // only where the groups' follow one another.
    const int64_t p_rows = (int64_t)a.M * (inner ? a.groups : 1);
    if (a.kind != FUSED_DENSE && !none &&
        (!inner || (p_rows <= SIZE_LIM && (a.groups == 1 || a.stride_y == (int64_t)a.M * a.ldy))))
      a.splits = sgemm_grouped_splits(a);
    const bool apart = a.splits > 1 || (!inner && !plain &&
                                        ((a.mode != FUSED_NONE && a.in == (const void*)P) ||
                                         ((uintptr_t)P % 16) != 0 || ldp % 4 != 0));
    const int64_t pitch = (int64_t)(a.N + 3) / 4 * 4;
    const int64_t p_bytes = apart ? pad256(a.splits * p_rows * pitch * 4) : 0;
    e = ws.get((size_t)(part_bytes + p_bytes), stream);
    if (e != cudaSuccess) return api_done(GEMM_PATH_NONE, ctx, e);
    a.part = part_bytes ? static_cast<float*>(ws.ptr) : nullptr;
    if (apart) {
      P = reinterpret_cast<float*>(static_cast<char*>(ws.ptr) + part_bytes);
      ldp = pitch;
    }
    path = GEMM_PATH_FUSED_FFMA;
    if (a.kind == FUSED_DENSE && !none) {
      Epilogue ep;
      if (plain) {
        ep.bias = a.bias;
        ep.act = a.act;
      }
      const int r = api_gemm(a.transA, a.transB, a.M, a.N, a.K, GEMM_F32, plain ? a.alpha : 1.f, 0.f,
                             a.A, a.lda, a.B, a.ldb, P, ldp, stream, ep);
      if (r != GEMM_OK) return r;
      if (plain) return GEMM_OK;
      ctx.launches = 0;
      e = launch_fused_finish(a, P, ldp, ctx);
      if (e == cudaSuccess && c.dbias) e = launch_fused_dbias(a, c.dbias, ctx);
      const int before = gemm_last_launches();
      ctx.grid = gemm_last_grid();
      const int done = api_done(path, ctx, e);
      api_add_launches(before);
      return done;
    }
    if (!none) {
      e = launch_sgemm_grouped(a, P, ldp, ctx);
      if (inner) {  // (the groups' rows of C, one after another)
        a.kind = FUSED_DENSE;
        a.M = (int)p_rows;
        a.groups = 1;
      }
      if (e == cudaSuccess && (!inner || a.splits > 1)) e = launch_fused_finish(a, P, ldp, ctx);
    }
  } else {
    const bool copy_a = a.K > 0 && !aligned16(a.A, a.lda);
    const int64_t nb = inner || a.stride_b == 0 ? 1 : a.groups;
    const bool copy_b = a.K > 0 && (!aligned16(a.B, a.ldb) || (nb > 1 && a.stride_b % 8 != 0));
    const int64_t bytes_a = copy_a ? pad256(c.a_rows * ((c.a_cols + 7) / 8 * 8) * 2) : 0;
    const int64_t bytes_b = copy_b ? pad256(nb * c.b_rows * ((c.b_cols + 7) / 8 * 8) * 2) : 0;
    const bool few = !inner && !a.transA && a.transB && a.M <= FUSED_FEW_ROWS &&
                     a.mode != FUSED_SLOPE && !c.dbias;
    a.splits = 1;
    if (!few && !none) fused_plan(a);
    a.ldp = (a.N + 15) / 16 * 16;
    const int64_t bytes_p = a.splits > 1 ? pad256((int64_t)a.splits * a.M * a.ldp * 4) : 0;
    e = ws.get((size_t)(part_bytes + bytes_a + bytes_b + bytes_p), stream);
    if (e != cudaSuccess) return api_done(GEMM_PATH_NONE, ctx, e);
    char* at = static_cast<char*>(ws.ptr);
    a.part = part_bytes ? reinterpret_cast<float*>(at) : nullptr;
    path = GEMM_PATH_FUSED_TC;
    if (!none) {
      int64_t no_stride = 0;
      if (copy_a) e = repack(a.A, a.lda, no_stride, c.a_rows, c.a_cols, 1, at + part_bytes, ctx);
      if (e == cudaSuccess && copy_b)
        e = repack(a.B, a.ldb, a.stride_b, c.b_rows, c.b_cols, nb, at + part_bytes + bytes_a, ctx);
      if (e == cudaSuccess && few) {
        path = GEMM_PATH_FUSED_STREAM;
        e = launch_fused_stream(a, ctx);
      } else if (e == cudaSuccess) {
        if (a.splits > 1) a.P = reinterpret_cast<float*>(at + part_bytes + bytes_a + bytes_b);
        e = launch_fused(a, ctx);
        if (e == cudaSuccess && a.splits > 1) e = launch_fused_finish(a, a.P, a.ldp, ctx);
      }
    }
  }
  if (e == cudaSuccess && c.dbias) e = launch_fused_dbias(a, c.dbias, ctx);
  return api_done(path, ctx, e);
}

// bias, R and U of a forward call
int check_forward(Call& c, const void* bias, const void* R, int64_t ldr, void* U, int64_t ldu,
                  float beta) {
  FusedArgs& a = c.a;
  const int64_t e = type_bytes(a.dtype), N = a.N, M = a.M;
  Span sb, sr, su;
  if (bias && a.groups > 0 && N > 0) {
    if (((uintptr_t)bias % (uintptr_t)e) != 0) return GEMM_ERR_INVALID_ARG;
    sb.lo = (uintptr_t)bias;
    sb.hi = sb.lo + (uintptr_t)((int64_t)a.groups * N * e);
  }
  a.bias = bias;
  a.beta = beta;
  if (R && beta != 0.f) {  // (beta 0: R is not read)
    const int rc = check_matrix(R, M, N, ldr, 1, 0, e, &sr);
    if (rc != GEMM_OK) return rc;
    a.mode = FUSED_ADD;
    a.in = R;
    a.ld_in = ldr;
    one_row(M, N, &a.ld_in);
  }
  if (U) {
    const int rc = check_matrix(U, M, N, ldu, 1, 0, e, &su);
    if (rc != GEMM_OK) return rc;
    a.U = U;
    a.ldu = ldu;
    one_row(M, N, &a.ldu);
  }
  Span so;
  if (a.kind != FUSED_DENSE && a.groups > 0) {
    so.lo = (uintptr_t)a.offsets;
    so.hi = so.lo + (uintptr_t)(a.groups + 1) * 4;
  }
  if (meet(c.sY, sb) || meet(su, sb) || meet(su, c.sA) || meet(su, c.sB) || meet(su, c.sY) ||
      meet(su, sr) || meet(su, so))
    return GEMM_ERR_ALIAS;
  if (meet(c.sY, sr) && !(R == a.Y && a.ld_in == a.ldy)) return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

// U and dbias of a backward call
int check_backward(Call& c, const void* U, int64_t ldu, float* dbias) {
  FusedArgs& a = c.a;
  const int64_t e = type_bytes(a.dtype), N = a.N, M = a.M;
  Span su, sd;
  if (a.act != GEMM_ACT_NONE) {
    const int rc = check_matrix(U, M, N, ldu, 1, 0, e, &su);
    if (rc != GEMM_OK) return rc;
    a.mode = FUSED_SLOPE;
    a.in = U;
    a.ld_in = ldu;
    one_row(M, N, &a.ld_in);
  }
  if (dbias && a.groups > 0 && N > 0) {
    if (((uintptr_t)dbias % 4) != 0) return GEMM_ERR_INVALID_ARG;
    sd.lo = (uintptr_t)dbias;
    sd.hi = sd.lo + (uintptr_t)((int64_t)a.groups * N * 4);
  }
  c.dbias = dbias;
  if (meet(c.sY, su) && !(U == a.Y && a.ld_in == a.ldy)) return GEMM_ERR_ALIAS;
  Span so;
  if (a.kind != FUSED_DENSE && a.groups > 0) {
    so.lo = (uintptr_t)a.offsets;
    so.hi = so.lo + (uintptr_t)(a.groups + 1) * 4;
  }
  if (meet(sd, c.sY) || meet(sd, c.sA) || meet(sd, c.sB) || meet(sd, su) || meet(sd, so))
    return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

Call make_call(int kind, int transA, int transB, float alpha, const void* A, int64_t lda,
               const void* B, int64_t ldb, int64_t stride_b, void* Y, int64_t ldy) {
  Call c = {};
  c.a.kind = kind;
  c.a.transA = transA; c.a.transB = transB;
  c.a.alpha = alpha;
  c.a.A = A; c.a.lda = lda;
  c.a.B = B; c.a.ldb = ldb; c.a.stride_b = stride_b;
  c.a.Y = Y; c.a.ldy = ldy;
  return c;
}

}  // namespace

extern "C" {

int gemm_fused(int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype, float alpha,
               const void* A, int64_t lda, const void* B, int64_t ldb, const void* bias, int act,
               float beta, const void* R, int64_t ldr, void* U, int64_t ldu, void* Y, int64_t ldy,
               gemm_stream_t stream) {
  api_reset();
  Call c = make_call(FUSED_DENSE, transA, transB, alpha, A, lda, B, ldb, 0, Y, ldy);
  int rc = check_call(c, M, N, K, 1, dtype, act);
  if (rc == GEMM_OK) rc = check_forward(c, bias, R, ldr, U, ldu, beta);
  if (rc != GEMM_OK || M == 0 || N == 0) return rc;
  return run_call(c, (cudaStream_t)stream);
}

int gemm_fused_backward(int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype,
                        float alpha, const void* A, int64_t lda, const void* B, int64_t ldb, int act,
                        const void* U, int64_t ldu, void* dX, int64_t lddx, float* dbias,
                        gemm_stream_t stream) {
  api_reset();
  Call c = make_call(FUSED_DENSE, transA, transB, alpha, A, lda, B, ldb, 0, dX, lddx);
  int rc = check_call(c, M, N, K, 1, dtype, act);
  if (rc == GEMM_OK) rc = check_backward(c, U, ldu, dbias);
  if (rc != GEMM_OK || N == 0 || (M == 0 && !dbias)) return rc;
  return run_call(c, (cudaStream_t)stream);
}

int gemm_grouped(int transB, int64_t rows, int64_t N, int64_t K, int64_t groups,
                 const int32_t* offsets, int dtype, float alpha, const void* A, int64_t lda,
                 const void* B, int64_t ldb, int64_t strideB, const void* bias, int act, float beta,
                 const void* R, int64_t ldr, void* U, int64_t ldu, void* Y, int64_t ldy,
                 gemm_stream_t stream) {
  api_reset();
  Call c = make_call(FUSED_ROWS, 0, transB, alpha, A, lda, B, ldb, strideB, Y, ldy);
  c.a.offsets = offsets;
  int rc = check_call(c, rows, N, K, groups, dtype, act);
  if (rc == GEMM_OK) rc = check_forward(c, bias, R, ldr, U, ldu, beta);
  if (rc != GEMM_OK || rows == 0 || N == 0 || groups == 0) return rc;
  return run_call(c, (cudaStream_t)stream);
}

int gemm_grouped_backward(int transB, int64_t rows, int64_t N, int64_t K, int64_t groups,
                          const int32_t* offsets, int dtype, float alpha, const void* A, int64_t lda,
                          const void* B, int64_t ldb, int64_t strideB, int act, const void* U,
                          int64_t ldu, void* dX, int64_t lddx, float* dbias, gemm_stream_t stream) {
  api_reset();
  Call c = make_call(FUSED_ROWS, 0, transB, alpha, A, lda, B, ldb, strideB, dX, lddx);
  c.a.offsets = offsets;
  int rc = check_call(c, rows, N, K, groups, dtype, act);
  if (rc == GEMM_OK) rc = check_backward(c, U, ldu, dbias);
  if (rc != GEMM_OK || N == 0 || groups == 0 || (rows == 0 && !dbias)) return rc;
  return run_call(c, (cudaStream_t)stream);
}

int gemm_grouped_wgrad(int64_t rows, int64_t M, int64_t N, int64_t groups, const int32_t* offsets,
                       int dtype, float alpha, float beta, const void* A, int64_t lda, const void* B,
                       int64_t ldb, void* C, int64_t ldc, int64_t strideC, gemm_stream_t stream) {
  api_reset();
  Call c = make_call(FUSED_INNER, 1, 0, alpha, A, lda, B, ldb, 0, C, ldc);
  c.a.offsets = offsets;
  c.a.stride_y = strideC;
  c.a.beta = beta;
  int rc = check_call(c, M, N, rows, groups, dtype, GEMM_ACT_NONE);
  if (rc != GEMM_OK || M == 0 || N == 0 || groups == 0) return rc;
  if (beta != 0.f) {
    c.a.mode = FUSED_ADD;
    c.a.in = C;
    c.a.ld_in = ldc;
  }
  return run_call(c, (cudaStream_t)stream);
}

}  // extern "C"
