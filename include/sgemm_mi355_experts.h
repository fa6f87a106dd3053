/*
 * sgemm_mi355: products by expert of 16-bit operands, for AMD Instinct MI355X
 * (gfx950): the rows of a layer of experts times each expert's weights, and
 * the gradients of the rows and of the weights.
 *
 * `offsets` are experts + 1 device ints, ascending, as sgemm_mi355_route_plan
 * makes them: rows offsets[e] .. offsets[e+1]-1 of the rows' matrices belong
 * to expert e. They are bounded as in sgemm_mi355_fp8.h: limited to 0 .. rows,
 * offsets[0] counts as 0, and one below an earlier one as that one, so that every
 * row of C is written once; in the weights' gradient, where an expert's end before
 * its beginning leaves it no rows, each expert's offsets count by themselves. An expert's weights W_e = W + e*strideW are N x K, row-major,
 * as in a linear layer.
 *
 * Operands are bf16 or fp16 (`type`, else SGEMM_MI355_ERR_TYPE). Their products
 * are exact, the sums are FP32 and are rounded once to `c_type`: FP32 or
 * `type`. Row strides count elements. Ownership, streams and errors are those
 * of sgemm_mi355.h: one kernel on `stream`, no allocation. Operands of any
 * alignment are accepted; 16-byte aligned ones whose strides are multiples of
 * 8 elements are loaded directly to LDS. The stride of a single row is looked at
 * like any other: as no row follows, a multiple of 8 may be given for it. That of a
 * single expert's weights is not.
 */
#ifndef SGEMM_MI355_EXPERTS_H
#define SGEMM_MI355_EXPERTS_H

#include "sgemm_mi355_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* C[r] = A[r] . W_e^T for expert e's rows r: A is rows x K, C rows x N. Rows that no expert has
   (from offsets[experts] on) are set to zero. */
int sgemm_mi355_experts_gemm(int type, int c_type, int rows, int N, int K, int experts, const void *A, int lda,
                             const void *W, int ldw, long long strideW, const int *offsets, void *C, int ldc,
                             hipStream_t stream);

/* The gradient of the rows, C[r] = A[r] . W_e: A is rows x N, C rows x K. Rows that no expert has are set to zero. */
int sgemm_mi355_experts_gemm_dgrad(int type, int c_type, int rows, int N, int K, int experts, const void *A, int lda,
                                   const void *W, int ldw, long long strideW, const int *offsets, void *C, int ldc,
                                   hipStream_t stream);

/*
 * The gradient of the weights, C_e = sum over expert e's rows r of A[r]^T . B[r] + beta*C_e:
 * A is rows x N, B rows x K, C_e = C + e*strideC N x K. When beta == 0, C is not
 * read; otherwise beta * C is added in FP32 before the rounding. An expert without rows
 * gets C_e = beta*C_e. strideC must keep the C_e apart (else SGEMM_MI355_ERR_STRIDE).
 */
int sgemm_mi355_experts_gemm_wgrad(int type, int c_type, int rows, int N, int K, int experts, const void *A, int lda,
                                   const void *B, int ldb, const int *offsets, float beta, void *C, int ldc,
                                   long long strideC, hipStream_t stream);

/*
 * Name of the kernel that a call with these arguments runs (host only; the
 * pointers are inspected, never read): staged_*, rows_* or tile_*, then its
 * tile of C (rows_*: the rows of A in it; tile_256x256 takes tiles of 192 rows,
 * or the last ones in pieces, where the experts' rows, which only the device
 * knows, fill the chip better so). form: one of the three below; W is B, and
 * strideW unused, in the weights' form. Null where a call has no results to
 * write (those of a sum over nothing are zeros), and for a stride under 1.
 */
#define SGEMM_MI355_EXPERTS_FORWARD 0
#define SGEMM_MI355_EXPERTS_DGRAD 1
#define SGEMM_MI355_EXPERTS_WGRAD 2
const char *sgemm_mi355_experts_kernel_name(int form, int rows, int N, int K, int experts, const void *A, int lda,
                                            const void *W, int ldw, long long strideW);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_MI355_EXPERTS_H */
