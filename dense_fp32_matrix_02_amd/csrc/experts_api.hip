// Host side of include/sgemm_mi355_experts.h: argument checks, then one launch.

#include "sgemm_mi355_experts.h"

#include "api_checks.h"
#include "experts_internal.h"

namespace sgemm_impl {
namespace {

// A has rows_a x cols_a elements, B groups_b matrices of rows_b x cols_b, C groups_c of M x N.
int check(ExpertsForm form, const ExpertsArgs& g, int rows) {
  if ((g.type != SGEMM_MI355_BF16 && g.type != SGEMM_MI355_F16) || (g.c_type != g.type && g.c_type != SGEMM_MI355_F32))
    return SGEMM_MI355_ERR_TYPE;
  if (g.M < 0 || g.N < 0 || g.K < 0 || g.experts < 1) return SGEMM_MI355_ERR_DIM;
  // Twice a row's length, in bytes, is an int too.
  if (g.M > kMostRows || g.N > kMostRows / 2 || g.K > kMostRows) return SGEMM_MI355_ERR_EXTENT;
  if (form == EXPERTS_WGRAD ? g.M > kMostRows / 2 : g.K > kMostRows / 2) return SGEMM_MI355_ERR_EXTENT;
  const bool wgrad = form == EXPERTS_WGRAD;
  const int64_t rows_a = rows, cols_a = wgrad ? g.M : g.K, rows_b = form == EXPERTS_FORWARD ? g.N : g.K;
  const int64_t cols_b = form == EXPERTS_FORWARD ? g.K : g.N, groups_b = wgrad ? 1 : g.experts, groups_c = wgrad ? g.experts : 1;
  if (g.lda < at_least_1((int)cols_a) || g.ldb < at_least_1((int)cols_b) || g.ldc < at_least_1(g.N)) return SGEMM_MI355_ERR_LD;
  if (g.strideB < 0 || g.strideC < 0) return SGEMM_MI355_ERR_STRIDE;
  if (groups_c > 1 && g.M > 0 && g.N > 0 && (Bytes)g.strideC < (Bytes)(g.M - 1) * (Bytes)g.ldc + (Bytes)g.N)
    return SGEMM_MI355_ERR_STRIDE;
  if (g.M == 0 || g.N == 0) return SGEMM_MI355_OK;
  Matrices m;
  m.dense(g.A, rows_a, cols_a, g.lda, 2, false);
  m.strided(g.B, groups_b, g.strideB, rows_b, g.ldb, cols_b, 1, 2, false);
  m.dense(g.offsets, 1, (int64_t)g.experts + 1, g.experts + 1, 4, false);
  m.strided(g.C, groups_c, g.strideC, g.M, g.ldc, g.N, 1, element_size(g.c_type), true);
  return m.check();
}

// What a call's kernel is chosen by: one expert has no stride between experts.
void settle(ExpertsArgs& g) {
  if (g.experts == 1) g.strideB = 0;
}

int run(ExpertsForm form, ExpertsArgs g, int rows, hipStream_t stream) {
  const int v = check(form, g, rows);
  if (v != SGEMM_MI355_OK || g.M == 0 || g.N == 0) return v;
  settle(g);
  if (!experts_launchable(form, g)) return SGEMM_MI355_ERR_EXTENT;
  // Past the caches go results that they do not hold for whoever comes next, as
  // long as rows share no lines (weights' gradients of 8 experts of 512 rows,
  // 4096 x 4096 FP32: 181 us against 213 through them).
  const int size = element_size(g.c_type);
  g.past = (int64_t)(form == EXPERTS_WGRAD ? g.experts : 1) * g.M * g.N * size >= (int64_t)64 << 20 &&
           (((uintptr_t)g.C | (uint64_t)(g.ldc * size) | (uint64_t)(g.strideC * size)) & 15) == 0;
  return done(launch_experts(form, g, stream));
}

}  // namespace
}  // namespace sgemm_impl

using namespace sgemm_impl;

extern "C" {

int sgemm_mi355_experts_gemm(int type, int c_type, int rows, int N, int K, int experts, const void* A, int lda,
                             const void* W, int ldw, long long strideW, const int* offsets, void* C, int ldc,
                             hipStream_t stream) {
  return run(EXPERTS_FORWARD, {type, c_type, rows, N, K, experts, A, lda, W, ldw, strideW, offsets, 0.0f, C, ldc, 0}, rows, stream);
}

int sgemm_mi355_experts_gemm_dgrad(int type, int c_type, int rows, int N, int K, int experts, const void* A, int lda,
                                   const void* W, int ldw, long long strideW, const int* offsets, void* C, int ldc,
                                   hipStream_t stream) {
  return run(EXPERTS_DGRAD, {type, c_type, rows, K, N, experts, A, lda, W, ldw, strideW, offsets, 0.0f, C, ldc, 0}, rows, stream);
}

int sgemm_mi355_experts_gemm_wgrad(int type, int c_type, int rows, int N, int K, int experts, const void* A, int lda,
                                   const void* B, int ldb, const int* offsets, float beta, void* C, int ldc,
                                   long long strideC, hipStream_t stream) {
  return run(EXPERTS_WGRAD, {type, c_type, N, K, rows, experts, A, lda, B, ldb, 0, offsets, beta, C, ldc, strideC}, rows, stream);
}

const char* sgemm_mi355_experts_kernel_name(int form, int rows, int N, int K, int experts, const void* A, int lda,
                                            const void* W, int ldw, long long strideW) {
  if (form < EXPERTS_FORWARD || form > EXPERTS_WGRAD || rows < 0 || N < 0 || K < 0 || experts < 1 || lda < 1 || ldw < 1 || strideW < 0)
    return nullptr;
  // No results; a sum over nothing has some, zeros.
  if (form == EXPERTS_FORWARD ? rows == 0 || N == 0 : form == EXPERTS_DGRAD ? rows == 0 || K == 0 : N == 0 || K == 0) return nullptr;
  ExpertsArgs g{};
  g.experts = experts, g.A = A, g.lda = lda, g.B = W, g.ldb = ldw;
  g.M = form == EXPERTS_WGRAD ? N : rows, g.N = form == EXPERTS_FORWARD ? N : K;
  g.K = form == EXPERTS_FORWARD ? K : form == EXPERTS_DGRAD ? N : rows;
  if (form != EXPERTS_WGRAD) g.strideB = strideW;
  settle(g);
  return experts_kernel_name((ExpertsForm)form, g);
}

}  // extern "C"
