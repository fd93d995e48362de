/*
 * gemm.h -- C ABI of the GB300 (sm_103a) dense GEMM library, libgemm_gb300.so.
 *
 * The library computes
 *
 *     C = alpha * op(A) * op(B) + beta * C
 *
 * over row-major matrices: full SGEMM as defined in the Introduction sidenote of
 * "Optimizing GEMM on Apple's M5 from scratch, Part 1: Basics" (the pages fix
 * alpha = 1, beta = 0 for their benchmark; the library takes both), for
 *   - fp32 operands and result (the SGEMM of that page and of "Part 2"), and
 *   - fp16 operands, fp32 accumulation and an fp16 result, the regime of
 *     "Metal GEMM Kernels for LoRA Training on Apple Silicon", section 1 (table
 *     of operand/accumulator types) and section 2 (output converted from the
 *     fp32 accumulator on the way out), and the same with bfloat16,
 * in the transpose variants of that page's section 2 variant table:
 *     nn  A[M,K]   @ B[K,N]
 *     tn  A[K,M]^T @ B[K,N]
 *     nt  A[M,K]   @ B[N,K]^T
 * (tt, both transposed, is not on the pages; it falls out of the same operand
 * descriptors and is accepted.)
 *
 * Conventions (all entry points):
 *   - Row-major storage; every leading dimension (lda, ldb, ldc) is in
 *     ELEMENTS and is the distance between consecutive stored rows.
 *   - op(A) is M x K: A is stored M x K (lda >= K) when transA == 0, and
 *     K x M (lda >= M) when transA == 1.  op(B) is K x N: B is stored K x N
 *     (ldb >= N) when transB == 0, N x K (ldb >= K) when transB == 1.
 *     C is M x N, ldc >= N.  A sub-matrix is passed as a pointer at its first
 *     element plus the parent's leading dimension (the row-offset entry of the
 *     LoRA page, section 7).
 *   - alpha and beta are fp32 for both dtypes.  beta == 0 makes C write-only:
 *     it is not read, so NaN or garbage in C does not reach the result.
 *   - M == 0 or N == 0 returns GEMM_OK without touching the GPU.  K == 0 sets
 *     C = beta * C (zero when beta == 0).
 *   - Pointers passed to gemm() are DEVICE pointers (cudaMalloc, the stream-
 *     ordered allocator or a torch CUDA tensor's storage), aligned to the
 *     element size.  The caller owns every buffer; the library never frees
 *     caller memory.  C must not overlap A or B (GEMM_ERR_ALIAS).
 *   - Calls are asynchronous on `stream` (0 = the legacy default stream) and
 *     may be made from several host threads.  Scratch space the library needs
 *     (split-K partial sums; zero-padded copies of operands whose rows are not
 *     16-byte aligned; on large problems an aligned working copy of a C whose
 *     rows are not, copied into place at the end) is taken in stream order on
 *     `stream` from a memory pool the library creates once per device, and
 *     released on the same stream; the pool keeps released memory for reuse
 *     until the process exits.
 *   - The library's kernels are launched with programmatic stream
 *     serialization: each may start its set-up while the previous work on the
 *     stream is finishing, and waits for that work to complete before reading
 *     or writing any buffer.  Stream order is therefore kept exactly as for
 *     ordinary launches (environment GEMM_GB300_PDL=0 turns the overlap off).
 *   - Argument errors are returned synchronously, before anything is
 *     launched.  Launch failures return GEMM_ERR_CUDA.  A kernel whose
 *     internal wait exceeds its time limit records the fact in a per-device
 *     status word and exits early; gemm_check_device_status() reports it.
 */
#ifndef GEMM_GB300_H
#define GEMM_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without pulling in the CUDA headers. */
typedef struct CUstream_st* gemm_stream_t;

typedef enum {
    GEMM_F32 = 0,         /* A, B, C fp32; fp32 FMA accumulation */
    GEMM_F16_F32ACC = 1,  /* A, B, C fp16 (IEEE binary16); fp32 accumulation;
                             result rounded to fp16 round-to-nearest-even */
    GEMM_BF16_F32ACC = 2, /* A, B, C bfloat16; fp32 accumulation; result
                             rounded to bfloat16 round-to-nearest-even (the
                             bfloat16 row of the LoRA page's section 1 type
                             table, native on these tensor cores) */
    GEMM_F32_TF32 = 3,    /* OPT-IN reduced precision: A, B, C fp32, but the
                             products use only the TF32 part of each operand
                             (sign, 8 exponent and the top 10 fraction bits)
                             on the tensor cores; fp32 accumulation.  Error up
                             to ~2^-9 * sum|a*b|, against ~K * 2^-24 for
                             GEMM_F32.  The counterpart of the relaxed-
                             precision switch of "Optimizing GEMM on Apple's
                             M5 from scratch, Part 2"; never chosen for you.
                             Not accepted by gemm_splitk_noalloc. */
    GEMM_F32_3XTF32 = 4   /* OPT-IN: A, B, C fp32 on the tensor cores at about
                             fp32 accuracy.  Each operand is split into its
                             TF32 part hi (low 13 fraction bits cleared) and
                             the rest lo = x - hi (exact), and the products are
                             formed as hi*hi + hi*lo + lo*hi in one fp32
                             accumulation: the dropped lo*lo term and the TF32
                             reading of lo leave an error of about 2^-19 *
                             sum|a*b|, within GEMM_F32's tolerance.  Inputs
                             must be finite (an infinity in one operand meets a
                             zero lo of the other).  Takes scratch for the
                             split planes (2 x 4 bytes x (M + N) x K); not
                             accepted by gemm_splitk_noalloc. */
} gemm_dtype_t;

typedef enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = 1, /* bad dimension, leading dimension, pointer, flag or dtype */
    GEMM_ERR_UNSUPPORTED = 2, /* valid but not handled (e.g. a dimension >= 2^31) */
    GEMM_ERR_ALIAS = 3,       /* C overlaps A or B */
    GEMM_ERR_CUDA = 4,        /* a CUDA runtime/driver call or a launch failed */
    GEMM_ERR_NO_MEMORY = 5,   /* scratch allocation failed */
    GEMM_ERR_TIMEOUT = 6      /* a kernel's bounded internal wait expired */
} gemm_status_t;

/*
 * gemm -- C = alpha * op(A) * op(B) + beta * C on the GPU.
 *
 * transA, transB: 0 or 1 (see above).  M, N, K >= 0 and < 2^31.
 * dtype: a gemm_dtype_t.  A, B, C: device pointers, element-aligned.
 * lda, ldb, ldc: leading dimensions in elements (see above).
 * stream: the CUDA stream to run on.
 * Returns a gemm_status_t.  Nothing is launched unless it returns GEMM_OK.
 */
int gemm(int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype, float alpha,
         float beta, const void* A, int64_t lda, const void* B, int64_t ldb, void* C,
         int64_t ldc, gemm_stream_t stream);

/*
 * gemm_ex -- gemm() with a fused epilogue ("From a C loop to a GPU kernel",
 * section "Fusion": add the bias and apply the activation while the tile is
 * still in registers, write the result once):
 *
 *     C = act(alpha * op(A) * op(B) + beta * C + bias[j])
 *
 * bias: DEVICE pointer to N elements of the output type (fp32 for GEMM_F32,
 *   fp16 / bf16 otherwise), one per output column (the per-output offset), or
 *   NULL for none; element-aligned; must not overlap C (GEMM_ERR_ALIAS).
 * act: a gemm_act_t.  GEMM_ACT_GELU is the exact v * Phi(v) =
 *   v/2 * (1 + erf(v / sqrt 2)), evaluated in fp32 with CUDA's erff.
 * Everything else as gemm(); with bias == NULL and GEMM_ACT_NONE it is gemm().
 * The bias and activation are applied in fp32 before the output rounding, in
 * every path (split-K: by the reduction; K == 0: act(beta * C + bias)).
 */
typedef enum {
    GEMM_ACT_NONE = 0,
    GEMM_ACT_RELU = 1,  /* max(v, 0) */
    GEMM_ACT_GELU = 2   /* v * Phi(v), Phi the standard normal distribution function */
} gemm_act_t;

int gemm_ex(int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype, float alpha,
            float beta, const void* A, int64_t lda, const void* B, int64_t ldb, void* C,
            int64_t ldc, const void* bias, int act, gemm_stream_t stream);

/*
 * gemm_host -- the same product on HOST buffers: copies A, B (and C when
 * beta != 0) to device memory taken from the stream-ordered allocator, runs
 * gemm() on `stream`, copies C back and synchronises `stream` before it
 * returns.  Problems of at least 2^30 multiply-adds are cut into 2 to 4 row
 * panels of C whose copies run on two library-owned copy streams (one per
 * direction, per device), ordered by events against the GEMMs on `stream`, so
 * that copies overlap computation; the call still returns only when C is
 * complete in host memory.  A, B, C are host pointers with the same layout rules as gemm();
 * page-locked (pinned) memory gives asynchronous DMA copies, pageable memory
 * works but is staged by the driver.  The device copies are packed (ld equal
 * to the row length) and freed before return.
 */
int gemm_host(int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype, float alpha,
              float beta, const void* A, int64_t lda, const void* B, int64_t ldb, void* C,
              int64_t ldc, gemm_stream_t stream);

/*
 * gemm_splitk_noalloc -- gemm() for callers that must not allocate device
 * memory: code running under an allocator that already owns the whole GPU
 * (a framework's caching allocator), or a process that forbids runtime
 * allocation once it is serving.  It never calls cudaMalloc, cudaFree or any
 * other allocating routine.  (No page of the method describes this entry
 * point; it is a property of this library.)
 *
 * Same arguments, rules and results as gemm(), with gemm()'s kernels and
 * choice of tile and schedule.  The partial sums that gemm() keeps in scratch
 * from the stream-ordered allocator -- the fp32 kernel's K slices, and the
 * tensor-core kernel's shared (stream-K) tiles with their arrival counters --
 * live in one fixed array of 8 MiB compiled into the library, which every
 * GPU that loads the library holds until the process exits.  Differences and
 * limits:
 *   - an fp32 problem whose K slices (splits x M x N x 4 bytes) exceed 8 MiB
 *     returns GEMM_ERR_UNSUPPORTED without launching anything;
 *   - a tensor-core problem whose shared tiles would not fit the array runs
 *     with whole tiles only (no scratch needed);
 *   - gemm()'s scratch-based steps are left out: the fp32 operand packing and
 *     persistent stream-K launch on large problems (where gemm() shares the K
 *     steps of fewer tiles than SMs in one launch, this call keeps the K
 *     slices and their reduction), and the aligned working copy of an
 *     unaligned fp16 C (the kernel stores such a C row by row);
 *   - fp16/bf16 operands must have 16-byte aligned bases and row pitches (lda,
 *     ldb multiples of 8), else GEMM_ERR_UNSUPPORTED (padding them would need
 *     scratch); GEMM_F32_TF32 and GEMM_F32_3XTF32 are not accepted.
 * The first call on a device looks up the array's device address (a CUDA
 * runtime query, done once per device with that device current); make that
 * first call before any stream capture.  All calls share the array: calls
 * whose kernels can overlap on the GPU (e.g. on two unordered streams) race
 * on it, so order them on one stream or with events.  A call writes every
 * partial sum it reads, and clears the counters that must start at zero
 * (cudaMemsetAsync on `stream`, which allocates nothing) before its launch.
 */
int gemm_splitk_noalloc(int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype,
                        float alpha, float beta, const void* A, int64_t lda, const void* B,
                        int64_t ldb, void* C, int64_t ldc, gemm_stream_t stream);

/*
 * gemm_strided_batched -- `batch` independent products of one shape,
 *
 *     C_b = alpha * op(A_b) * op(B_b) + beta * C_b,   b = 0 .. batch-1,
 *
 * with A_b = A + b*strideA, B_b = B + b*strideB, C_b = C + b*strideC (pitches
 * in ELEMENTS).  This is the per-head GEMM of "Metal GEMM Kernels for LoRA
 * Training on Apple Silicon", section 8 (Attention): Q, K, V stored head-major
 * [H, N, d_h], so head h is a contiguous matrix at offset h*N*d_h and the six
 * attention products are the nn/tn/nt variants entered at a head offset.  The
 * page issues one GEMM per head; here the whole batch is one launch.
 *
 * Arguments as gemm(), plus:
 *   strideA, strideB, strideC >= 0.  A pitch of 0 shares one matrix across
 *     the batch (A or B only).  The C matrices must not overlap one another
 *     (strideC >= (M-1)*ldc + N when batch > 1), else GEMM_ERR_ALIAS.
 *   batch >= 0 and < 2^31; batch == 0 returns GEMM_OK without touching the
 *     GPU.  batch == 1 is gemm().
 * Aliasing is checked over whole extents: the span C .. C_{batch-1} must not
 * overlap the span of A's or B's matrices (GEMM_ERR_ALIAS), even where the
 * entries themselves would interleave without touching.
 * One launch covers the batch (gemm_last_path() GEMM_PATH_FFMA_BATCHED or
 * GEMM_PATH_TC_BATCHED) when the operands allow: fp32 always, in groups of
 * 65535 entries; fp16/bf16 when A and B have 16-byte aligned bases, row
 * pitches and batch pitches (lda, ldb, strideA, strideB multiples of 8).
 * Otherwise each entry runs as its own gemm() in stream order
 * (GEMM_PATH_PER_ENTRY).  No split-K within a batch.
 */
int gemm_strided_batched(int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype,
                         float alpha, float beta, const void* A, int64_t lda, int64_t strideA,
                         const void* B, int64_t ldb, int64_t strideB, void* C, int64_t ldc,
                         int64_t strideC, int64_t batch, gemm_stream_t stream);

/*
 * Microscaled operands: matrices stored in 4 or 8 bits an element with one
 * scale for each block of consecutive columns of a row.  They are what a LoRA
 * step keeps beside its 16-bit tensors: frozen weights in 4 bits, and the
 * activations that its backward pass reads again in 8.
 *
 * A stored matrix [rows, cols] is two device buffers:
 *   - codes: rows at a pitch of ldq BYTES, a multiple of 16 and at least
 *     gemm_mx_row_bytes(format, cols); the base is 16-byte aligned.  Two 4-bit
 *     codes a byte, the even column in the low half, or one signed byte a
 *     column; bytes past the last column within that row length are zero.
 *   - scales: gemm_mx_scale_bytes(format, rows, cols) bytes, 16-byte aligned,
 *     one byte a block, in tiles of 128 rows x 4 blocks (512 bytes): the byte of
 *     row r and block b lies in tile (r / 128) * ceil(blocks / 4) + b / 4, at
 *     (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4; absent rows and blocks are
 *     zero.
 * A block is cut at the row's end: it may be short there.
 *
 * The value of a code is code * scale.  Quantising takes, for each block, the
 * largest magnitude amax of mult * x (fp32 product), from it the scale, and the
 * nearest code to mult * x / scale (ties to even, saturating).  A block that
 * holds a NaN or an infinity gets a NaN scale: all of it reads as NaN.
 */
typedef enum {
    GEMM_MX_FP4 = 0,      /* e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and negatives), 32
                             columns a block, scale a power of two 2^(byte - 127)
                             (255: NaN): 2^(floor(log2 amax) - 2) */
    GEMM_MX_FP4_E4M3 = 1, /* e2m1 codes, 16 columns a block, scale an e4m3 number
                             (0x7F: NaN): amax / 6 rounded to nearest even, at most
                             448.  Values far below e4m3's 2^-9 vanish: scale them up
                             with mult and give 1 / mult to the product as alpha */
    GEMM_MX_INT8 = 2      /* whole numbers -127 .. 127, 32 columns a block, scale
                             2^(floor(log2 amax) - 6) */
} gemm_mx_format_t;

/* Sizes of the two buffers; -1 for an unknown format or size. */
int64_t gemm_mx_row_bytes(int format, int64_t cols);
int64_t gemm_mx_scale_bytes(int format, int64_t rows, int64_t cols);

/*
 * gemm_mx_quantize -- stores op(X), [rows, cols], in `format`.
 *
 * X: device matrix of dtype (GEMM_F32, GEMM_F16_F32ACC or GEMM_BF16_F32ACC),
 *   [rows, cols] or, with transX, [cols, rows]; any ldx and element alignment.
 * mult: finite; the values stored are mult * X.
 * Y: NULL, or act(X) (without mult) is written to it in the same pass, dtype,
 *   [rows, cols]: the forward pass of an activation whose input is kept in 8
 *   bits.  Not with transX (GEMM_ERR_UNSUPPORTED); act without Y is an error.
 *   Y may be X itself with the same pitch.  GEMM_ACT_GELU is x Phi(x), in fp32
 *   within a few ulp for every x, in 16 bits within 1e-7 |x| before its rounding
 *   and 1.5 % of the value down to x = -8.5.  (gemm_ex()'s fused x/2 (1 + erf(x / sqrt 2)) is
 *   evaluated as that sum, whose error is about 2^-22 |x|: in fp32 the two differ
 *   by as much, and for x below -4 mostly by gemm_ex()'s.)  GEMM_ACT_RELU is x
 *   where x > 0, else 0, as gemm_ex()'s: a NaN becomes 0.
 */
int gemm_mx_quantize(int format, int transX, int64_t rows, int64_t cols, int dtype, float mult,
                     const void* X, int64_t ldx, int act, void* Y, int64_t ldy, void* q,
                     int64_t ldq, void* scales, gemm_stream_t stream);

/* gemm_mx_dequantize -- Y = the values of a stored matrix, rounded to dtype
 * (exact but where fp16's range ends). */
int gemm_mx_dequantize(int format, int64_t rows, int64_t cols, const void* q, int64_t ldq,
                       const void* scales, int dtype, void* Y, int64_t ldy, gemm_stream_t stream);

/*
 * gemm_mx_act_backward -- the backward pass of Y = act(X) from X's checkpoint
 * in GEMM_MX_INT8:
 *     dX = dY * act'(x8),   dbias[j] = sum_i dX[i, j]
 * act'(x): GEMM_ACT_NONE 1; GEMM_ACT_RELU 1 where x > 0, else 0 (so also
 * throughout a block that reads as NaN); GEMM_ACT_GELU Phi(x) + x phi(x).  dY, dX: dtype, [rows, cols]; dX may be dY
 * itself with the same pitch.  dbias: NULL or cols fp32 sums (of the values
 * before their rounding to dtype, in an order that does not change from call to
 * call).  rows == 0 sets dbias to zero.
 */
int gemm_mx_act_backward(int64_t rows, int64_t cols, int dtype, int act, const void* dY,
                         int64_t lddy, const void* q, int64_t ldq, const void* scales, void* dX,
                         int64_t lddx, float* dbias, gemm_stream_t stream);

/*
 * gemm_mx4 -- product of two 4-bit operands,
 *     C = act(alpha * A * B^T + beta * C + bias[j]),
 * A [M, K] and B [N, K] stored in the same 4-bit format (blocks along K), C of
 * dtype; products of codes and scales exact, fp32 accumulation.  lda, ldb in
 * BYTES (see above), ldc in elements; bias and act as gemm_ex().
 * GEMM_ERR_UNSUPPORTED for GEMM_MX_INT8, and (as for gemm_mx()) where M, N or K
 * is above 2^31 - 2^18.
 */
int gemm_mx4(int format, int64_t M, int64_t N, int64_t K, int dtype, float alpha, float beta,
             const void* A, int64_t lda, const void* As, const void* B, int64_t ldb,
             const void* Bs, void* C, int64_t ldc, const void* bias, int act,
             gemm_stream_t stream);

/*
 * gemm_mx -- gemm_ex() with a stored right operand:
 *     C = act(alpha * op(A) * op(B) + beta * C + bias[j]),
 * A and C of dtype as in gemm(); B stored in `format` as [K, N] (blocks along
 * N) or, with transB, as [N, K] (blocks along K); ldb in BYTES.  The values of
 * B are rounded to dtype before the product, which is exact but where fp16's
 * range ends: a value below 2^-14 may lose bits or vanish, one above 65504 becomes
 * infinite.  (Up to 32 rows of A with transB, a power-of-two 4-bit scale beyond
 * fp16's range is kept in fp32 instead.)  Takes scratch in stream order where B is expanded for the
 * other types' kernels, and where rows of A are not 16-byte aligned.
 */
int gemm_mx(int format, int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype,
            float alpha, float beta, const void* A, int64_t lda, const void* B, int64_t ldb,
            const void* Bs, void* C, int64_t ldc, const void* bias, int act,
            gemm_stream_t stream);

/*
 * gemm_fused -- a layer's forward product with all that follows it, in one pass:
 *
 *     U = alpha * op(A) * op(B) + bias[j],    Y = act(U) + beta * R
 *
 * (gemm_ex() adds beta * C before the activation; here the residual R comes after
 * it, and U can be kept for the backward pass.)
 *
 * dtype: GEMM_F32, GEMM_F16_F32ACC or GEMM_BF16_F32ACC, of every matrix and of bias.
 * bias: N elements, or NULL.  act: a gemm_act_t, applied to the fp32 value of U
 *   before its rounding, as in gemm_mx_quantize() (relu of a NaN is 0).
 * R: M x N with ldr, or NULL; beta == 0 reads no R.  R may be Y itself with the same
 *   pitch.
 * U: M x N with ldu, stored rounded to dtype; or NULL.
 * M, N and K up to 2^31 - 2^18 (else GEMM_ERR_UNSUPPORTED).  Outputs may overlap one
 * another not at all and inputs only as said (GEMM_ERR_ALIAS; checked over whole extents,
 * so U and Y that interleave within one wider matrix are refused).  K == 0: the product
 * is zero.  16-bit operands whose rows are not 16-byte aligned are copied to scratch in
 * stream order, on each call (of grouped products all matrices of B, also those whose
 * groups have no rows).
 */
int gemm_fused(int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype, float alpha,
               const void* A, int64_t lda, const void* B, int64_t ldb, const void* bias, int act,
               float beta, const void* R, int64_t ldr, void* U, int64_t ldu, void* Y, int64_t ldy,
               gemm_stream_t stream);

/*
 * gemm_fused_backward -- the gradient that passes back through a product and the
 * activation before it:
 *
 *     dX = (alpha * op(A) * op(B)) * act'(U),    dbias[j] = sum_i dX[i, j]
 *
 * U: the stored pre-activation, M x N with ldu; not read with GEMM_ACT_NONE (may then
 *   be NULL).  act': relu 1 where U > 0, else dX is 0; gelu Phi(U) + U phi(U).
 * dX: M x N with lddx; may be U itself with the same pitch.
 * dbias: N fp32 sums of dX before its rounding (in an order that does not change from
 *   call to call), or NULL.  M == 0 sets them to zero.  With 16-bit operands dX's values
 *   are the tensor cores' sums over K, whose additions are cut rather than rounded: at K =
 *   2048 dbias is 2 10^-6 off in norm (fp32: 4 to 8 10^-7).
 */
int gemm_fused_backward(int transA, int transB, int64_t M, int64_t N, int64_t K, int dtype,
                        float alpha, const void* A, int64_t lda, const void* B, int64_t ldb, int act,
                        const void* U, int64_t ldu, void* dX, int64_t lddx, float* dbias,
                        gemm_stream_t stream);

/*
 * gemm_grouped -- gemm_fused() by groups of rows, as a router sends tokens to experts:
 * for each group g, on rows offsets[g] .. offsets[g+1] - 1 of A, R, U and Y,
 *
 *     U = alpha * A * op(B_g) + bias[g][j],    Y = act(U) + beta * R
 *
 * offsets: groups + 1 int32 in DEVICE memory, ascending within 0 .. rows; the call
 *   does not wait for them.  Groups may be empty and of any size; rows before
 *   offsets[0] and from offsets[groups] on are neither used nor written.  Offsets that
 *   do not ascend within 0 .. rows make results unspecified, but nothing outside the
 *   given matrices is read or written, and gemm_check_device_status() then returns
 *   GEMM_ERR_INVALID_ARG.
 * A: rows x K (lda).  B_g = B + g * strideB: K x N, or with transB N x K (ldb).  A
 *   stride of 0 shares one matrix.
 * bias: groups x N contiguous, or NULL.  groups up to 65535.
 */
int gemm_grouped(int transB, int64_t rows, int64_t N, int64_t K, int64_t groups,
                 const int32_t* offsets, int dtype, float alpha, const void* A, int64_t lda,
                 const void* B, int64_t ldb, int64_t strideB, const void* bias, int act, float beta,
                 const void* R, int64_t ldr, void* U, int64_t ldu, void* Y, int64_t ldy,
                 gemm_stream_t stream);

/* gemm_grouped_backward -- gemm_fused_backward() by groups of rows (see
 * gemm_grouped()); dbias: groups x N contiguous, zero for an empty group. */
int gemm_grouped_backward(int transB, int64_t rows, int64_t N, int64_t K, int64_t groups,
                          const int32_t* offsets, int dtype, float alpha, const void* A, int64_t lda,
                          const void* B, int64_t ldb, int64_t strideB, int act, const void* U,
                          int64_t ldu, void* dX, int64_t lddx, float* dbias, gemm_stream_t stream);

/*
 * gemm_grouped_wgrad -- the gradient of each group's matrix, over its rows:
 *
 *     C_g = alpha * A_g^T * B_g + beta * C_g
 *
 * A: rows x M (lda), B: rows x N (ldb), A_g and B_g their rows of group g (offsets as
 * in gemm_grouped()); C_g = C + g * strideC: M x N (ldc), strideC at least (M - 1) * ldc + N
 * (else GEMM_ERR_ALIAS).  An empty group's C_g is beta * C_g (zero with beta == 0, which reads no C).
 */
int gemm_grouped_wgrad(int64_t rows, int64_t M, int64_t N, int64_t groups, const int32_t* offsets,
                       int dtype, float alpha, float beta, const void* A, int64_t lda, const void* B,
                       int64_t ldb, void* C, int64_t ldc, int64_t strideC, gemm_stream_t stream);

/*
 * gemm_check_device_status -- synchronises `stream`, then reads and clears
 * the current device's status word.  Returns GEMM_ERR_TIMEOUT if a kernel
 * gave up on a wait since the last check, GEMM_ERR_INVALID_ARG if a grouped
 * product's offsets did not ascend within its rows, GEMM_ERR_CUDA if the stream
 * reported an error, GEMM_OK otherwise.
 */
int gemm_check_device_status(gemm_stream_t stream);

/* Human-readable name of a gemm_status_t (a static string). */
const char* gemm_status_string(int status);

/* Library version, (major << 16) | minor. */
int gemm_version(void);

/*
 * Diagnostics, per calling host thread: the kernel path the last successful
 * gemm() call on this thread launched (a gemm_path_t), and the number of
 * kernels it launched.  gemm_total_launches() counts kernels launched by the
 * library in this process since it was loaded (all threads).
 */
typedef enum {
    GEMM_PATH_NONE = 0,        /* nothing launched (empty problem or error) */
    GEMM_PATH_SCALE = 1,       /* K == 0: C = beta * C */
    GEMM_PATH_FFMA = 2,        /* fp32 FFMA tiled kernel */
    GEMM_PATH_FFMA_SPLITK = 3, /* fp32 FFMA kernel over K slices + reduction */
    GEMM_PATH_TC = 4,          /* fp16/bf16 tcgen05 kernel, fused epilogue */
    GEMM_PATH_TC_SPLITK = 5,   /* tcgen05 kernel whose persistent grid shares the K steps
                                  of some tiles (stream-K); partial sums combined inside
                                  the kernel */
    GEMM_PATH_FFMA_BATCHED = 6, /* strided batch: fp32 FFMA kernel, batch on the grid */
    GEMM_PATH_TC_BATCHED = 7,  /* strided batch: one persistent tcgen05 launch */
    GEMM_PATH_PER_ENTRY = 8,   /* strided batch run entry by entry (unaligned operands) */
    GEMM_PATH_MX = 9,          /* microscaled storage: quantise, dequantise, act backward */
    GEMM_PATH_MX_TC = 10,      /* product of 4-bit operands: block-scaled tcgen05 kernel */
    GEMM_PATH_MX_STREAM = 11,  /* few rows times a stored right operand, read once */
    GEMM_PATH_MX_CONVERT = 12, /* 16-bit rows times a stored right operand, converted inside
                                  the tcgen05 kernel */
    GEMM_PATH_FUSED_TC = 13,   /* fused or grouped product: its tcgen05 kernel */
    GEMM_PATH_FUSED_FFMA = 14, /* the same in fp32: FFMA kernels, then the epilogue */
    GEMM_PATH_FUSED_STREAM = 15 /* the same of a few rows, B read once by warp MMAs */
} gemm_path_t;

int gemm_last_path(void);
int gemm_last_launches(void);
int64_t gemm_total_launches(void);
/* Blocks in the grid of the last main GEMM kernel gemm() launched on this
 * thread (the persistent fp16 kernel sizes its grid to the resident blocks). */
int gemm_last_grid(void);

/*
 * Diagnostics: kernel timing.  With two CUDA events (cudaEvent_t, created by
 * the caller), every later gemm(), gemm_splitk_noalloc() and
 * gemm_strided_batched() call made from this host thread records `start` on
 * its stream immediately before its main GEMM kernel and `end` immediately
 * after it -- not around pre-passes (operand packing or padding) or the
 * split-K reduction -- so cudaEventElapsedTime(start, end) is that kernel's
 * device time for the latest call.  Passing NULL for either turns it off.  The
 * events stay owned by the caller and must outlive their use.
 */
void gemm_set_kernel_events(void* start, void* end);

/*
 * Diagnostics: scratch use.  Returns the largest number of bytes that were in
 * use at once, on the current device, from the stream-ordered memory pool the
 * library takes its scratch from, since the previous reset (0 if the pool has
 * not been created yet, -1 on a CUDA error); a nonzero `reset` then sets the
 * mark back to zero.  A stretch of calls that leaves the mark at zero took no
 * scratch from the pool.
 */
int64_t gemm_scratch_high_water(int reset);

/*
 * Test hook: the time limit, in nanoseconds, of every bounded wait inside the
 * kernels launched afterwards by this process (default 2e9, i.e. 2 s; values
 * <= 0 restore the default).  A wait that runs out sets the device status
 * word, releases what its block holds and returns.
 */
void gemm_set_wait_timeout_ns(int64_t ns);

/*
 * Test hook for failure detection: mode 1 makes the fp16 kernel's operand
 * producer skip its first load (no copy, no arrival), so the consumer's
 * bounded wait runs out and the kernel reports GEMM_ERR_TIMEOUT through
 * gemm_check_device_status() instead of hanging.  Mode 0 (the default) turns
 * it off.  Process-wide; not for production use.
 */
void gemm_set_fault_injection(int mode);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_GB300_H */
