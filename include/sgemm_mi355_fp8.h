/*
 * sgemm_mi355: matrix products in 8-bit floating point with a scale for each
 * block of 128 values of the summed axis, for AMD Instinct MI355X (gfx950),
 * and the quantisers that make their operands.
 *
 * Values are OCP e4m3 (one byte, largest 448, no infinities). A quantised
 * matrix is a byte matrix Q, row-major, and a matrix S of FP32 scales. Block b
 * of a row is its columns 128*b .. 128*b+127 (the last one may be shorter). The
 * value that Q's element (i, k) stands for is
 *   Q(i,k) * S(i, k/128)        one scale for each block of a row, or
 *   Q(i,k) * S(i/128, k/128)    one for each 128 x 128 tile.
 * Element (r, b) of S lies at S[r*s_row + b*s_block]; strides count floats, may
 * be 0 and are not negative. The quantisers of the Python package store the
 * rows' scales block by block (s_row = 1), which the products read fastest.
 *
 * The product multiplies by rows of both operands (B is stored as N x K, like
 * the weights of a linear layer):
 *   C[m][n] = sum_b sA[m][b] * sB[n][b] * sum_{k in b} A[m][k]*B[n][k].
 * A block's sum enters an FP32 accumulator with one fused multiply-add by the
 * FP32 product of the two scales, and the result is rounded once to the type
 * of C. Products are exact and a block's sum is FP32, with one exception: into
 * a 16-bit C, the kernels that sgemm_mi355_fp8_kernel_name calls tile_*_fp8
 * (aligned operands and more than a few rows) take the FP8 matrix unit's sum. It
 * adds products by eight in fixed point, where each loses less than 2^-13 of
 * the largest of its eight, and the eights' sums in FP32 (on quantised normal
 * data 2e-5 of the result, against 2e-3 and 2e-4 of the rounding to bf16 and
 * fp16; up to 7 * 2^-13 of the products' magnitudes where they cancel). A
 * product whose `type` includes SGEMM_MI355_FP32_SUMS has FP32 sums in every
 * kernel, at up to twice the time.
 *
 * Ownership, streams and errors are those of sgemm_mi355.h: device pointers
 * owned by the caller, arguments checked on the host before any HIP call, one
 * kernel enqueued on `stream`, no synchronisation, no allocation. Additional
 * codes: SGEMM_MI355_ERR_TYPE for an element type that is none of the three
 * below, SGEMM_MI355_ERR_STRIDE for a negative stride of scales or experts.
 * Integers the device reads (index, offsets) cannot be checked on the host;
 * the kernels bound them: an index outside the matrix reads as a row of
 * zeros, offsets are limited to 0 .. rows, an expert whose end is before its
 * beginning has no rows, and offsets[0] counts as 0. `experts` is at least 1
 * where it counts (else SGEMM_MI355_ERR_DIM).
 */
#ifndef SGEMM_MI355_FP8_H
#define SGEMM_MI355_FP8_H

#include "sgemm_mi355.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the wide matrices. */
#define SGEMM_MI355_F32 0
#define SGEMM_MI355_BF16 1
#define SGEMM_MI355_F16 2

/* Added to a product's `type`: block sums are FP32 whatever the type of C. */
#define SGEMM_MI355_FP32_SUMS 0x100

/*
 * Rows to e4m3. For each block of a row, most = max |x| over the block (2^-64
 * at least), s = most / 448 and Q = e4m3(x / s): both quotients rounded to
 * FP32, then to the nearest e4m3 number (half to even). A block that holds a
 * NaN or an infinity gets scale NaN and NaN throughout.
 *
 * X is rows x cols of `type`, row stride ldx elements. With `index` null, Q is
 * rows x cols and n is ignored; with `index` (n device ints), row i of Q is
 * row index[i] of X, so that tokens can be sent to several experts without a
 * copy. Q's row stride is ldq bytes; a multiple of 16 (and a 16-byte aligned
 * Q) lets the products load it directly.
 */
int sgemm_mi355_fp8_quantize_rows(int type, int rows, int cols, const void *X, int ldx,
                                  const int *index, int n, unsigned char *Q, int ldq,
                                  float *S, long long s_row, long long s_block, hipStream_t stream);

/*
 * Columns to e4m3, stored transposed: for products that sum over X's rows
 * (weight gradients). Row c of Q is column c of X, its blocks are of 128
 * consecutive rows of X. With `index`, row i of the matrix that is transposed
 * is row index[i] of X (n rows). With `offsets` (experts + 1 device ints,
 * ascending) the rows are sorted by expert and every expert's rows begin a
 * block: expert e's first block is offsets[e]/128 + e, Q has
 * 128*(n/128 + experts) columns, and what no row fills is zero (scale 2^-64/448).
 * Without `offsets`, Q has n columns and `experts` is ignored.
 */
int sgemm_mi355_fp8_quantize_cols(int type, int rows, int cols, const void *X, int ldx,
                                  const int *index, int n, const int *offsets, int experts,
                                  unsigned char *Q, int ldq,
                                  float *S, long long s_row, long long s_block, hipStream_t stream);

/* 128 x 128 tiles to e4m3, one scale each (weights): S is rows/128 x cols/128, rounded up. */
int sgemm_mi355_fp8_quantize_tiles(int type, int rows, int cols, const void *X, int ldx,
                                   unsigned char *Q, int ldq,
                                   float *S, long long s_row, long long s_block, hipStream_t stream);

/*
 * C = A.B^T + beta*C as above: A M x K with a scale for each block of a row, B
 * N x K with one for each block of `sb_rows` rows, 1 or 128 (else
 * SGEMM_MI355_ERR_OP). C is M x N of `type`, row stride ldc elements. When
 * beta == 0, C is not read; otherwise beta * C is added in FP32 before the
 * rounding to C's type. K == 0 gives C = beta * C. lda and ldb are in bytes,
 * at least K. Operands of any alignment are accepted; 16-byte aligned ones
 * whose row strides are multiples of 16 are loaded directly to LDS.
 */
int sgemm_mi355_fp8_gemm(int type, int M, int N, int K,
                         const unsigned char *A, int lda, const float *SA, long long sa_row, long long sa_block,
                         const unsigned char *B, int ldb, const float *SB, long long sb_row, long long sb_block,
                         int sb_rows, float beta, void *C, int ldc, hipStream_t stream);

/*
 * Experts: rows offsets[e] .. offsets[e+1]-1 of A (rows x K, sorted by
 * expert) meet B_e = B + e*strideB (N x K), with SB_e = SB + e*stride_sb:
 *   C[r] = A[r] . B_e^T.
 * `offsets` are experts + 1 device ints, ascending. Rows of C that no expert
 * has (from offsets[experts] on) are set to zero.
 */
int sgemm_mi355_fp8_gemm_experts(int type, int rows, int N, int K, int experts,
                                 const unsigned char *A, int lda, const float *SA, long long sa_row, long long sa_block,
                                 const unsigned char *B, int ldb, long long strideB,
                                 const float *SB, long long sb_row, long long sb_block, long long stride_sb,
                                 int sb_rows, const int *offsets, void *C, int ldc, hipStream_t stream);

/*
 * The experts' weight gradients: A (M x P) and B (N x P) as
 * sgemm_mi355_fp8_quantize_cols makes them for the same offsets, with
 * P = 128*(rows/128 + experts);
 *   C_e = sum over expert e's rows r of A[:, r] . B[:, r]^T + beta*C_e,
 * C_e = C + e*strideC (M x N). An expert without rows gets C_e = beta*C_e.
 * strideC must keep the C_e apart, as for sgemm_mi355_strided_batched.
 */
int sgemm_mi355_fp8_gemm_experts_wgrad(int type, int rows, int M, int N, int experts,
                                       const unsigned char *A, int lda, const float *SA, long long sa_row, long long sa_block,
                                       const unsigned char *B, int ldb, const float *SB, long long sb_row, long long sb_block,
                                       const int *offsets, float beta, void *C, int ldc, long long strideC, hipStream_t stream);

/*
 * Name of the kernel that a product with these arguments runs (host only; the
 * pointers are inspected, never read): staged_*, rows_* or tile_*, then its
 * tile of C (rows_*: the rows of A in it), then the matrix instructions that
 * form a block's sum, fp8 or bf16. form: one of the three below; the sizes are
 * those of the call (weight gradients: K is `rows`), experts and strideB count
 * where the form has them. Null where nothing would be launched.
 */
#define SGEMM_MI355_FP8_DENSE 0   /* sgemm_mi355_fp8_gemm */
#define SGEMM_MI355_FP8_EXPERTS 1 /* sgemm_mi355_fp8_gemm_experts */
#define SGEMM_MI355_FP8_WGRAD 2   /* sgemm_mi355_fp8_gemm_experts_wgrad */
const char *sgemm_mi355_fp8_kernel_name(int form, int type, int M, int N, int K, int experts,
                                        const unsigned char *A, int lda,
                                        const unsigned char *B, int ldb, long long strideB);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_MI355_FP8_H */
