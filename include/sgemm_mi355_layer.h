/*
 * sgemm_mi355: what stands around the products of a layer in 8 bits, forward
 * and backward: the root-mean-square norm with the residual's addition, gated
 * activations, and the epilogue's backward pass. (The product with an epilogue
 * is sgemm_mi355_fp8_gemm_epilogue.)
 *
 * Ownership, streams and errors are those of sgemm_mi355.h; element types and
 * the form of quantised rows (Q, S) are those of sgemm_mi355_fp8.h: blocks of
 * 128 values of a row, each value rounded to e4m3 from its FP32 value, without
 * a rounding to a wide type between. Matrices have contiguous rows and a row
 * stride in elements (bytes for Q). Outputs marked "or null" are not written
 * when null; a call without any output is refused (SGEMM_MI355_ERR_NULL). No output may overlap another matrix of the call, with the
 * exceptions named below. Results repeat bit for bit.
 */
#ifndef SGEMM_MI355_LAYER_H
#define SGEMM_MI355_LAYER_H

#include "sgemm_mi355_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_MI355_MAX_NORM_COLS 16384

/*
 * The norm. X and R (the residual, or null) are rows x cols of `type`, W
 * (cols) is of `w_type`: FP32 or `type` (else SGEMM_MI355_ERR_TYPE). For each row
 *   h = x + r, added in FP32 and rounded to `type` (h = x without R);
 *   a = 1 / sqrt(mean(h^2) + eps);
 *   y = h * a * w, in FP32.
 * Outputs: H (or null; it may be R or X itself, at the same address and row
 * stride), rstd = a (rows floats, or null), Y (or null) y rounded to `type`, Q
 * and S (both or neither, else SGEMM_MI355_ERR_NULL) y in e4m3 as
 * sgemm_mi355_fp8_quantize_rows makes them. Sums are FP32, and FP64 in rows
 * whose squares leave FP32's range. eps is finite and not negative (else
 * SGEMM_MI355_ERR_OP); cols is 1 .. SGEMM_MI355_MAX_NORM_COLS (else
 * SGEMM_MI355_ERR_DIM, SGEMM_MI355_ERR_EXTENT).
 */
int sgemm_mi355_rms_norm(int type, int rows, int cols, const void *X, int ldx, const void *R, int ldr,
                         const void *W, int w_type, float eps, void *H, int ldh, float *rstd, void *Y, int ldy,
                         unsigned char *Q, int ldq, float *S, long long s_row, long long s_block,
                         hipStream_t stream);

/*
 * Its backward pass, for the gradients dY of y and dH of h (or null: none),
 * both of `type`. With n = h * rstd and g = w * dy,
 *   dx = rstd * (g - n * mean(g * n)) + dh   (the gradient of x and of r);
 *   dw = sum over the rows of dy * n          (cols floats, or null), FP32.
 * dX may be dY or dH itself, at the same address and row stride. One kernel, a
 * second where dW is asked for and there are many rows. `workspace`: device
 * memory of sgemm_mi355_rms_norm_backward_workspace_size(rows, cols) bytes,
 * 4-byte aligned (null where that is 0, or without dW), free again once the
 * work is done. Without rows, dW is not written.
 */
int sgemm_mi355_rms_norm_backward(int type, int rows, int cols, const void *dY, int lddy, const void *H, int ldh,
                                  const float *rstd, const void *W, int w_type, const void *dH, int lddh,
                                  void *dX, int lddx, float *dW, void *workspace, size_t workspace_bytes,
                                  hipStream_t stream);
size_t sgemm_mi355_rms_norm_backward_workspace_size(int rows, int cols);

/*
 * Gated activation: H is rows x 2*cols of `type`, g its first cols columns and
 * u the others; z = act(g) * u in FP32. Outputs: Z (or null) z rounded to
 * `type`, Q and S (both or neither) z in e4m3. act: one of the activations of
 * sgemm_mi355_fp8.h (else SGEMM_MI355_ERR_OP).
 */
int sgemm_mi355_gated(int type, int act, int rows, int cols, const void *H, int ldh, void *Z, int ldz,
                      unsigned char *Q, int ldq, float *S, long long s_row, long long s_block, hipStream_t stream);

/* Its backward pass: dH = [act'(g) * u * dz | act(g) * dz], rows x 2*cols. */
int sgemm_mi355_gated_backward(int type, int act, int rows, int cols, const void *dZ, int lddz,
                               const void *H, int ldh, void *dH, int lddh, hipStream_t stream);

/*
 * The backward pass of sgemm_mi355_fp8_gemm_epilogue from the gradient dC of
 * its result to its product: dP = act'(P) * dC for the kept P (all rows x cols
 * of `type`), and dbias (cols floats, or null), the sum of dP over the rows,
 * from the FP32 values of dP. (The residual's gradient is dC.) One kernel, a
 * second where dbias is asked for and there are many rows; workspace as
 * above, of sgemm_mi355_epilogue_backward_workspace_size(rows, cols) bytes.
 * Without rows, dbias is not written.
 */
int sgemm_mi355_epilogue_backward(int type, int act, int rows, int cols, const void *dC, int lddc,
                                  const void *P, int ldp, void *dP, int lddp, float *dbias,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t sgemm_mi355_epilogue_backward_workspace_size(int rows, int cols);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_MI355_LAYER_H */
