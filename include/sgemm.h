/*
 * sgemm.h -- C ABI of the MI355X (gfx950) single-precision GEMM library
 * (libsgemm_mi355x.so), built from hand-written HIP kernels.
 *
 * Operation (every entry point below computes this, the 4x4 case of it, or,
 * for sgemm_f32_ex, this followed by a fused epilogue; gemm_bf16_f32 and
 * gemm_f16_f32 take A and B in 16-bit formats; the MXFP4 entry points, whose
 * operands are 4-bit elements in scaled blocks and whose B is stored by its
 * columns, and those of 8-bit integers and of the gated feed-forward block, are
 * described where they begin):
 *
 *     C[i,j] = sum_{k=0}^{K-1} A[i,k] * B[k,j]      0 <= i < M, 0 <= j < N
 *
 * with A (MxK), B (KxN) and C (MxN) single precision and row-major: element
 * (r,c) of X lives at X[r*ldx + c].  The sum is the accumulator that the
 * micro-GEMM page builds per output element ("Micro Kernel 입문하기",
 * teach-meaning.tistory.com/1544, walkthrough sections 2 and 3-1..4), and the
 * row*ld + col addressing of C is the store of "누산 개념을
 * Grid-Block-Warp-Thread 계층에 끼워넣기" (teach-meaning.tistory.com/1518),
 * section 2.  C is overwritten: the plain store of "gemm_tiled_test"
 * (teach-meaning.tistory.com/1542), section 6.  sgemm_f32_ex adds the fused
 * epilogue that page's opening paragraph says its original kernel carried
 * (alpha/beta, bias, activation); its reading is given at its declaration.
 *
 * How it is computed (results differ from the plain definition only in the
 * rounding order of the fp32 sums): one kernel launch covers all of C; each
 * workgroup owns one BM x BN block tile of C; the K axis is walked in BK-deep
 * slabs staged through LDS, double-buffered; within a workgroup each lane (or
 * each wave, on the matrix-core path) keeps a register tile of accumulators
 * updated by rank-1 outer products; the tile is stored once at the end.
 * (Page 2 section 1-2; "gemm_tiled_test" sections 1-6; "Register/Shared
 * Memory Tiling", ryotta.opik.net, sections on outer-product GEMM, tile
 * loading and double buffering.)
 *
 * Conventions shared by all entry points
 * --------------------------------------
 * - Pointers are DEVICE pointers (hipMalloc / torch CUDA tensors) owned by
 *   the caller.  The library allocates nothing and keeps no per-call state
 *   (it caches each device's compute-unit and XCD counts, read from the
 *   runtime on the first call that launches there); calls from several host
 *   threads are safe.
 * - Dimensions and leading dimensions are int; all address arithmetic inside
 *   the library is 64-bit.
 * - stream is a hipStream_t passed as void*; NULL means the null stream.
 *   Calls are stream-ordered and asynchronous: SGEMM_OK means the work was
 *   enqueued.  The caller synchronises before reading C.
 * - Every argument is validated before any HIP call; on a validation error
 *   nothing is launched and C is untouched.
 * - M == 0 or N == 0: nothing to do, returns SGEMM_OK without a launch.
 *   K == 0: A and B may be NULL; sgemm_f32 and sgemm_f32_path set
 *   C[0:M, 0:N] to 0 (the empty sum).
 * - C must not overlap A or B (the pages' kernels take all three pointers
 *   __restrict__); A and B may overlap each other.
 * - Result: within the fp32 rounding of some summation order of the exact
 *   products; integer-valued inputs whose partial sums stay below 2^24 in
 *   magnitude give the exact result on every path.
 */
#ifndef REGISTER_LDS_TILED_SGEMM_H
#define REGISTER_LDS_TILED_SGEMM_H

#ifdef __cplusplus
extern "C" {
#endif

/* Symbols of this ABI are the only ones the library exports. */
#ifndef SGEMM_API
#define SGEMM_API __attribute__((visibility("default")))
#endif

/* Return codes. */
#define SGEMM_OK             0
#define SGEMM_EINVAL_DIM    -1  /* M, N or K negative; micro-GEMM K < 0; C
                                   so large that one workgroup per 64 x 64 tile
                                   (256 threads each) would pass the 2^32 - 1
                                   threads of one launch; or a matrix whose
                                   byte extent from its pointer would pass the
                                   end of the address space                    */
#define SGEMM_EINVAL_LD     -2  /* lda < max(1,K), ldb < max(1,N) or ldc < max(1,N) */
#define SGEMM_EINVAL_PTR    -3  /* NULL pointer for a matrix with elements      */
#define SGEMM_EALIAS        -4  /* C's address range overlaps A's, B's or bias's */
#define SGEMM_EHIP          -5  /* the HIP runtime reported an error on launch  */
#define SGEMM_EINVAL_PATH   -6  /* unknown path selector                        */
#define SGEMM_EINVAL_ACT    -7  /* unknown activation selector                  */

/* Activation selectors: sgemm_f32_ex takes the first two, the gated entry
   points all of them. */
#define SGEMM_ACT_NONE        0 /* identity                                     */
#define SGEMM_ACT_RELU        1 /* x < 0 ? 0 : x  (NaN passes through)          */
#define SGEMM_ACT_SILU        2 /* x / (1 + exp(-x))                            */
#define SGEMM_ACT_GELU        3 /* x P(x), P the standard normal distribution's
                                   integral: x erfc(-x / sqrt 2) / 2            */
#define SGEMM_ACT_GELU_TANH   4 /* x (1 + tanh(y)) / 2, y = sqrt(2 / pi) (x +
                                   0.044715 x^3)                                */

/* Path selectors for sgemm_f32_path. */
#define SGEMM_PATH_AUTO       0 /* what sgemm_f32 uses: the matrix-core path;
                                   for A of at most 16 rows kernels that
                                   stream B once (9 to 16 aligned rows on the
                                   matrix cores, else on the vector ALU), and
                                   for B of at most 16 columns (A of more
                                   than 16 rows) vector-ALU kernels that
                                   stream A once */
#define SGEMM_PATH_VALU       1 /* per-lane TM x TN v_fma_f32 micro-kernel      */
#define SGEMM_PATH_MFMA       2 /* fp32 MFMA wave tiles (16x16x4 in the large
                                   wave-tile kernels, 32x32x2 in the others),
                                   for every shape                             */
#define SGEMM_PATH_VALU_PAGE  3 /* VALU path at the tiled page's own geometry:
                                   BM=BN=64, BK=16, 64 threads, 16x4 per thread,
                                   single-buffered ("gemm_tiled_test" section 7) */

/*
 * C = A.B, row-major, fp32, on the path the library picks for the shape.
 * A: M x K at A[i*lda + k]; B: K x N at B[k*ldb + j]; C: M x N at
 * C[i*ldc + j].  Returns SGEMM_OK or a negative code above.
 */
SGEMM_API int sgemm_f32(int M, int N, int K,
              const float *A, int lda,
              const float *B, int ldb,
              float *C, int ldc,
              void *stream);

/*
 * Same operation and contract as sgemm_f32 on an explicit path (one of
 * SGEMM_PATH_*), for tests and measurements that compare the paths.
 */
SGEMM_API int sgemm_f32_path(int M, int N, int K,
                   const float *A, int lda,
                   const float *B, int ldb,
                   float *C, int ldc,
                   void *stream, int path);

/*
 * Same operation and contract as sgemm_f32 on the VALU path at one of its
 * built tile configurations (tile = 0 .. sgemm_valu_tile_count() - 1): the
 * block tile BM x BN x BK, the wave tile WM x WN each wave of the block owns
 * (the warp tile of "누산 개념을 Grid-Block-Warp-Thread 계층에 끼워넣기",
 * teach-meaning.tistory.com/1518, section 2(2)), and the TM x TN register
 * tile of each lane (the thread tile, section 2(3); the MR x NR of "Micro
 * Kernel 입문하기", teach-meaning.tistory.com/1544, section 4, whose planned
 * comparison of register tiles this entry point serves).  Every
 * configuration sums each output over k in ascending order with one fused
 * multiply-add per k, so all of them return the same bits.  For tests and
 * measurements; SGEMM_PATH_VALU picks among the same configurations by
 * shape.  A tile outside the range -> SGEMM_EINVAL_PATH.
 */
SGEMM_API int sgemm_f32_valu_tile(int M, int N, int K,
                        const float *A, int lda,
                        const float *B, int ldb,
                        float *C, int ldc,
                        void *stream, int tile);

/* Number of VALU tile configurations sgemm_f32_valu_tile accepts. */
SGEMM_API int sgemm_valu_tile_count(void);

/*
 * Static text describing VALU tile configuration `tile` (block, waves, wave
 * tile, lanes, lane tile, LDS stages), or NULL outside 0 .. count - 1.
 */
SGEMM_API const char *sgemm_valu_tile_name(int tile);

/*
 * Fused form, on the default path's kernels (the same choice as sgemm_f32):
 *
 *     C[i,j] = act(alpha * sum_k A[i,k] * B[k,j] + beta * C[i,j] + bias[j])
 *
 * "gemm_tiled_test" (teach-meaning.tistory.com/1542), opening paragraph:
 * the page's test kernel is its original kernel with the epilogue, bias and
 * activation taken out, and the page leaves them undefined.  Reading taken
 * here: the BLAS alpha/beta update of C in place, one bias value per output
 * column, then act = SGEMM_ACT_NONE or SGEMM_ACT_RELU.  Each output is
 * computed once, in fp32, right after its dot product leaves the
 * accumulators, so the epilogue costs no extra pass over C.
 * - C is read only when beta != 0 (when beta == 0 it may hold anything,
 *   NaN included); it is then read and written in place, element by element.
 * - bias: NULL for none, else a device array of N floats that must not
 *   overlap C (SGEMM_EALIAS); it may overlap A or B.
 * - alpha multiplies the accumulated sum as is: alpha == 0 does not skip
 *   the product (NaN or Inf in A.B still propagates).
 * - K == 0: C = act(beta * C + bias) (the sum is the empty sum, 0).
 * - alpha == 1, beta == 0, bias == NULL, act == SGEMM_ACT_NONE runs exactly
 *   the kernel sgemm_f32 runs, the skinny-shape kernels included.
 * Other arguments, conventions and return codes as sgemm_f32; an act other
 * than SGEMM_ACT_NONE and SGEMM_ACT_RELU -> SGEMM_EINVAL_ACT.
 */
SGEMM_API int sgemm_f32_ex(int M, int N, int K,
                 const float *A, int lda,
                 const float *B, int ldb,
                 float *C, int ldc,
                 float alpha, float beta, const float *bias, int act,
                 void *stream);

/*
 * C = A.B with 16-bit floating-point inputs and fp32 accumulation and output,
 * on the matrix cores (v_mfma_f32_32x32x16_bf16 / _f16).  The pages tie the
 * register/LDS tiling to matrix instructions and half-precision inputs
 * ("Register/Shared Memory Tiling", ryotta.opik.net: advantages item 3,
 * related technologies); the reading taken is the plain one: the same sum as
 * above over the values the 16-bit inputs hold, accumulated in fp32.
 * - gemm_bf16_f32: A and B hold bfloat16 values (the upper 16 bits of an
 *   IEEE binary32); gemm_f16_f32: IEEE binary16.  Passed as raw 16-bit
 *   storage (const void *, two bytes per element); lda and ldb count
 *   elements.  C is fp32 and overwritten, as for sgemm_f32.
 * - Every product of two 16-bit values is exact in fp32, so the result is
 *   within the fp32 rounding of some summation order of the exact sum of the
 *   stored inputs; integer-valued inputs with partial sums below 2^24 give
 *   the exact result.
 * - Rows of A and B that are 16-byte aligned (base 16-byte aligned, lda and
 *   ldb multiples of 8) take the fast loader; any other layout is accepted
 *   and runs a slower one.
 * Conventions and return codes as sgemm_f32 (overlap checks use the 16-bit
 * extents of A and B).
 */
SGEMM_API int gemm_bf16_f32(int M, int N, int K,
                  const void *A, int lda,
                  const void *B, int ldb,
                  float *C, int ldc,
                  void *stream);
SGEMM_API int gemm_f16_f32(int M, int N, int K,
                 const void *A, int lda,
                 const void *B, int ldb,
                 float *C, int ldc,
                 void *stream);

/*
 * Microscaled 4-bit floating point (MXFP4): the element and block formats of
 * the OCP Microscaling Formats (MX) specification 1.0, E2M1 elements in blocks
 * of 32 with an E8M0 scale, multiplied on the matrix cores
 * (v_mfma_scale_f32_32x32x64_f8f6f4; for few rows 16x16x128).
 *
 * An MXFP4 matrix of R rows and K columns is two byte matrices:
 * - values Q: row r's ceil(K/2) bytes at Q + r*ldq.  Byte i holds element 2i
 *   in its low and 2i+1 in its high half; where K is odd, the last byte's high
 *   half belongs to no element (written as 0, never looked at).  An element is
 *   sign, two exponent bits, one mantissa bit: codes 0..7 are 0, 0.5, 1, 1.5,
 *   2, 3, 4, 6, codes 8..15 their negatives;
 * - scales S: row r's ceil(K/32) bytes at S + r*lds.  Byte j scales elements
 *   32j .. 32j+31 by 2^(byte - 127); byte 255 makes them all NaN.
 * Leading dimensions of both count bytes.  Pointers and leading dimensions may
 * have any alignment; rows of Q that are 16-byte aligned (base and ld) take
 * the fast loaders.
 *
 * Common to these entry points: device pointers, stream order, validation
 * before any HIP call and the return codes are as above (SGEMM_EINVAL_LD also
 * for a leading dimension below a row's bytes, SGEMM_EALIAS also for an output
 * that overlaps an input or another output; extents run from a matrix's first
 * byte to its last row's end, so scales may not lie between the rows of the
 * values they belong to).  What lies past a row's length is never written and
 * never matters; an input row on 16-byte boundaries may be read to the end of
 * its last 16 bytes.  Nothing is allocated, no workspace is used, and
 * every result is the same from call to call.
 */

/*
 * Quantise X (R x C, row-major, ldx in elements) to MXFP4, in one pass over X:
 * - along its rows into (Q, S): an R x C MXFP4 matrix;
 * - along its columns into (QT, ST): the C x R MXFP4 matrix of X transposed,
 *   its blocks running down X's columns.
 * Either pair may be NULL, then its leading dimensions are not looked at;
 * both NULL or half a pair -> SGEMM_EINVAL_PTR.  With both, X is read once.
 * For a block of values with the largest magnitude t the scale's exponent is
 * floor(log2 t) - 2, at least -127 (t == 0: -127); each value x becomes the
 * element nearest to x / scale, ties to the even code, magnitudes beyond 6 to
 * 6.  Signs are kept, also of zeros.  A block that holds a NaN or an infinity
 * gets scale byte 255, its codes are unspecified.  The last block of a row
 * takes its largest magnitude from the elements that exist.
 * SGEMM_EINVAL_DIM also for columns asked of an X so large that one workgroup
 * per 128 x 128 tile (256 threads each) would pass the 2^32 - 1 threads of one
 * launch.
 * _f32 takes float, _bf16 and _f16 raw 16-bit storage.
 */
SGEMM_API int gemm_mxfp4_quantize_f32(int R, int C, const void *X, int ldx,
                            void *Q, int ldq, void *S, int lds,
                            void *QT, int ldqt, void *ST, int ldst,
                            void *stream);
SGEMM_API int gemm_mxfp4_quantize_bf16(int R, int C, const void *X, int ldx,
                             void *Q, int ldq, void *S, int lds,
                             void *QT, int ldqt, void *ST, int ldst,
                             void *stream);
SGEMM_API int gemm_mxfp4_quantize_f16(int R, int C, const void *X, int ldx,
                            void *Q, int ldq, void *S, int lds,
                            void *QT, int ldqt, void *ST, int ldst,
                            void *stream);

/*
 * Y (R x C, row-major, ldy in elements) = the values of an MXFP4 matrix.
 * float and bfloat16 hold every finite one exactly, but for magnitudes of
 * 2^128 and more (scale bytes 253 and above), which become infinite; _f16
 * rounds to nearest even, to infinity beyond its range.
 */
SGEMM_API int gemm_mxfp4_dequantize_f32(int R, int C, const void *Q, int ldq,
                              const void *S, int lds, void *Y, int ldy, void *stream);
SGEMM_API int gemm_mxfp4_dequantize_bf16(int R, int C, const void *Q, int ldq,
                               const void *S, int lds, void *Y, int ldy, void *stream);
SGEMM_API int gemm_mxfp4_dequantize_f16(int R, int C, const void *Q, int ldq,
                              const void *S, int lds, void *Y, int ldy, void *stream);

/*
 * C = A.B^T with A (M x K) and B (N x K) in MXFP4, both blocked along K:
 *     C[i,j] = sum_k A[i,k] * B[j,k]
 * accumulated in fp32, C fp32 or bfloat16 (rounded once, to nearest even).  B's
 * rows are the product's columns: a layer's weights, outputs x inputs, are used
 * as they are stored.
 * Products of two elements with their scales have few significant bits: those
 * that fp32's normal range holds are exact, and where it holds them all and
 * their sums the result is within the fp32 rounding of some summation order.
 * Scales reach past that range both ways (2^-254 to 2^254): a product or
 * partial sum below 2^-126 in magnitude may lose bits, down to all of them
 * (each then adds an error of at most 2^-126); one past the largest fp32
 * number may become infinite (it does where all terms have one sign), and
 * infinities of both signs make NaN.
 * The three products of a linear layer Y = X.W^T are
 *     Y  = A.B^T of X and W, each quantised along its rows,
 *     dX = A.B^T of dY (rows) and W (columns: its QT, ST),
 *     dW = A.B^T of dY and X, both quantised along their columns.
 * K == 0 stores zeros.  M of at most 64 streams B once.
 */
SGEMM_API int gemm_mxfp4_f32(int M, int N, int K,
                   const void *A, int lda, const void *SA, int ldsa,
                   const void *B, int ldb, const void *SB, int ldsb,
                   float *C, int ldc, void *stream);
SGEMM_API int gemm_mxfp4_bf16(int M, int N, int K,
                    const void *A, int lda, const void *SA, int ldsa,
                    const void *B, int ldb, const void *SB, int ldsb,
                    void *C, int ldc, void *stream);

/*
 * C = A.B^T with 16-bit A (M x K, row-major, lda in elements) and B (N x K) in
 * MXFP4 blocked along K, fp32 accumulate and C: weights kept in four bits,
 * activations as they are.  Products that fp32's normal range holds are exact;
 * beyond it, either way, gemm_mxfp4_f32's rule holds, except that a binary16
 * A's product may lose 2^-126 twice.  An element of B of magnitude 2^128 or
 * more (possible at scale bytes 253 and above) makes the outputs it contributes
 * to infinite or NaN.  K == 0 stores zeros.  M of at most 64 streams B once.
 */
SGEMM_API int gemm_bf16_mxfp4_f32(int M, int N, int K,
                        const void *A, int lda,
                        const void *B, int ldb, const void *SB, int ldsb,
                        float *C, int ldc, void *stream);
SGEMM_API int gemm_f16_mxfp4_f32(int M, int N, int K,
                       const void *A, int lda,
                       const void *B, int ldb, const void *SB, int ldsb,
                       float *C, int ldc, void *stream);

/*
 * 8-bit integers with a scale per row, and the products of a feed-forward
 * layer.
 *
 * A quantised matrix of R rows and K columns is R x K bytes Q, signed whole
 * numbers at Q + r*ldq (ldq in bytes), and R floats S, contiguous: element (r,c)
 * stands for Q[r,c] * S[r].  Activations carry one scale per token, weights
 * (outputs x inputs, used as they are stored) one per output channel.
 *
 * Common to these entry points: device pointers, stream order, validation
 * before any HIP call and the return codes are as above (SGEMM_EALIAS also for
 * an output that overlaps an input or another output).  Pointers of 16- and
 * 32-bit data are aligned to their elements, otherwise pointers and leading
 * dimensions are free; rows that are 16-byte aligned (base and ld) take the fast
 * loaders.  What lies past a row's length is never written and never matters;
 * an input row on 16-byte boundaries may be read to the end of its last 16
 * bytes.  Nothing is allocated, no workspace is used, and every result is the
 * same from call to call.
 */

/*
 * Quantise X (R x C, row-major, ldx in elements) along its rows.  For a row
 * whose largest magnitude is t: S = max(t / 127 rounded to float, 2^-126), and
 * each value x becomes the whole number nearest to x / S, ties to the even one
 * (the quotient is not rounded before).  A row that holds a NaN or an infinity
 * gets the scale NaN and zeros.  _f32 takes float, _bf16 and _f16 raw 16-bit
 * storage.
 */
SGEMM_API int gemm_i8_quantize_f32(int R, int C, const void *X, int ldx, void *Q, int ldq,
                         float *S, void *stream);
SGEMM_API int gemm_i8_quantize_bf16(int R, int C, const void *X, int ldx, void *Q, int ldq,
                          float *S, void *stream);
SGEMM_API int gemm_i8_quantize_f16(int R, int C, const void *X, int ldx, void *Q, int ldq,
                         float *S, void *stream);

/*
 * Y (R x C, row-major, ldy in elements) = Q[r,c] * S[r], multiplied in fp32 and
 * rounded to Y's type.
 */
SGEMM_API int gemm_i8_dequantize_f32(int R, int C, const void *Q, int ldq, const float *S,
                           void *Y, int ldy, void *stream);
SGEMM_API int gemm_i8_dequantize_bf16(int R, int C, const void *Q, int ldq, const float *S,
                            void *Y, int ldy, void *stream);
SGEMM_API int gemm_i8_dequantize_f16(int R, int C, const void *Q, int ldq, const float *S,
                           void *Y, int ldy, void *stream);

/*
 * C[i,j] = (sum_k A[i,k] * B[j,k]) * SA[i] * SB[j], A (M x K) and B (N x K)
 * signed bytes, -128 included: the sum is exact in 32-bit integers, then
 * converted to fp32, multiplied by SA[i], by SB[j], and rounded to C's type (ldc
 * in elements).  K above 131071, where a sum could pass 32 bits ->
 * SGEMM_EINVAL_DIM.  K == 0 stores zeros; A, B, SA and SB may then be NULL.
 */
SGEMM_API int gemm_i8_f32(int M, int N, int K, const void *A, int lda, const float *SA,
                const void *B, int ldb, const float *SB, float *C, int ldc, void *stream);
SGEMM_API int gemm_i8_bf16(int M, int N, int K, const void *A, int lda, const float *SA,
                 const void *B, int ldb, const float *SB, void *C, int ldc, void *stream);
SGEMM_API int gemm_i8_f16(int M, int N, int K, const void *A, int lda, const float *SA,
                const void *B, int ldb, const float *SB, void *C, int ldc, void *stream);

/*
 * The gated block of a feed-forward layer on 8-bit operands, in one launch:
 *     H[i,j] = act(g) * u,  g = A.BG^T and u = A.BU^T as gemm_i8_f32 has them,
 * BG and BU (N x K) the gate's and the other projection's weights.  act is one
 * of SGEMM_ACT_*; H (M x N) is rounded once.
 */
SGEMM_API int gemm_i8_gated_bf16(int M, int N, int K, const void *A, int lda, const float *SA,
                       const void *BG, int ldbg, const float *SBG,
                       const void *BU, int ldbu, const float *SBU,
                       void *H, int ldh, int act, void *stream);
SGEMM_API int gemm_i8_gated_f16(int M, int N, int K, const void *A, int lda, const float *SA,
                      const void *BG, int ldbg, const float *SBG,
                      const void *BU, int ldbu, const float *SBU,
                      void *H, int ldh, int act, void *stream);

/*
 * The gated block in 16 bits, in one launch:
 *     H[i,j] = act(g) * u,  g = sum_k X[i,k] * WG[j,k],  u = sum_k X[i,k] * WU[j,k]
 * with X (M x K: tokens), WG and WU (N x K: outputs x inputs, as they are
 * stored), all matrices of one 16-bit type, leading dimensions in elements.
 * Sums, act and the product are fp32; H is rounded once.  G and U, both or
 * neither NULL, receive g and u rounded to 16 bits, for the backward pass.
 * For g = -infinity act is what its formula gives in fp32: NaN of SILU and both
 * forms of GELU, as of -infinity times 0.
 * K == 0 stores zeros.
 */
SGEMM_API int gemm_gated_bf16(int M, int N, int K, const void *X, int ldx,
                    const void *WG, int ldwg, const void *WU, int ldwu,
                    void *G, int ldg, void *U, int ldu, void *H, int ldh, int act, void *stream);
SGEMM_API int gemm_gated_f16(int M, int N, int K, const void *X, int ldx,
                   const void *WG, int ldwg, const void *WU, int ldwu,
                   void *G, int ldg, void *U, int ldu, void *H, int ldh, int act, void *stream);

/*
 * Its backward pass, from DH (M x N) and what the forward pass kept in G and U:
 *     DG = DH * U * act'(G)      DU = DH * act(G)                (M x N)
 *     DX = DG.WG + DU.WU                                         (M x K)
 *     DWG = DG^T.X               DWU = DU^T.X                    (N x K)
 * all of one 16-bit type, sums and act in fp32.  Each result is rounded once;
 * DX, DWG and DWU are products of DG and DU as rounded.  ReLU's slope at 0 is 0.
 * G and U hold infinities for sums beyond their type's range, of which the forward
 * pass took the finite values: at G = -infinity act and act' are their limits, 0 of
 * SILU and both forms of GELU, and where act' is 0 so is DG, also for an infinite
 * U.  Otherwise infinities and NaN are multiplied as they are.
 * - DX may be NULL, then it is not computed, and WG, WU and the three leading
 *   dimensions are not looked at; DWG and DWU may both be NULL, then they are
 *   not computed and neither they nor X are looked at (one of the two ->
 *   SGEMM_EINVAL_PTR).  Results overwrite.
 * - M == 0 sets DWG and DWU to zero, N == 0 sets DX to zero.
 * - Of SGEMM_EINVAL_DIM's threads of one launch, DWG and DWU together count.
 * Up to three launches, in stream order.
 */
SGEMM_API int gemm_gated_backward_bf16(int M, int N, int K, const void *X, int ldx,
                             const void *WG, int ldwg, const void *WU, int ldwu,
                             const void *G, int ldg, const void *U, int ldu,
                             const void *DH, int lddh, void *DG, int lddg, void *DU, int lddu,
                             void *DX, int lddx, void *DWG, int lddwg, void *DWU, int lddwu,
                             int act, void *stream);
SGEMM_API int gemm_gated_backward_f16(int M, int N, int K, const void *X, int ldx,
                            const void *WG, int ldwg, const void *WU, int ldwu,
                            const void *G, int ldg, const void *U, int ldu,
                            const void *DH, int lddh, void *DG, int lddg, void *DU, int lddu,
                            void *DX, int lddx, void *DWG, int lddwg, void *DWU, int lddwu,
                            int act, void *stream);

/*
 * The micro-GEMM of "Micro Kernel 입문하기" (teach-meaning.tistory.com/1544),
 * section 2: one GPU thread holds the whole 4x4 tile of C in 16 registers and
 * walks k = 0..K-1 in order, loading column k of A (4 values) and row k of B
 * (4 values) and doing 16 fused multiply-adds (the fmaf form of the tiled
 * page's section 5).  The launch is one wave: its 64 lanes first stage
 * chunks of A's columns and B's rows in LDS with coalesced loads, and the
 * thread reads its operands from there.  Layouts are the page's: A is 4 x K with leading
 * dimension K (A[r*K + k]), B is K x 4 with leading dimension 4 (B[k*4 + j]),
 * C is 4 x 4 row-major (C[r*4 + j]).  Each output is the sequential fp32
 * fused sum in ascending k, so results are reproducible bit for bit.
 * K == 0 stores zeros.  K < 0 -> SGEMM_EINVAL_DIM; NULL A/B (K > 0) or NULL C
 * -> SGEMM_EINVAL_PTR; C overlapping A or B -> SGEMM_EALIAS.
 */
SGEMM_API int sgemm_micro4x4_f32(int K, const float *A, const float *B, float *C, void *stream);

/* Static description of a return code (never NULL). */
SGEMM_API const char *sgemm_status_string(int status);

/*
 * Detail of the last SGEMM_EHIP on the calling host thread (the HIP error
 * name and message), or "" if there was none.  Thread-local; valid until the
 * thread's next failing call.
 */
SGEMM_API const char *sgemm_last_error(void);

/* Version of this ABI; bumped when a signature or contract changes. */
SGEMM_API int sgemm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* REGISTER_LDS_TILED_SGEMM_H */
