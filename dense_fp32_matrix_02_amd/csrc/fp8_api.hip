// Host side of include/sgemm_mi355_fp8.h: argument checks, then one launch.

#include "sgemm_mi355_fp8.h"

#include "api_checks.h"
#include "fp8_internal.h"

namespace sgemm_impl {
namespace {

// One quantiser call. n: rows of the quantised matrix before any transposition.
struct Quantize {
  int type, rows, cols;
  const void* X;
  int ldx;
  const int* index;
  int n;
  unsigned char* Q;
  int64_t q_rows, q_cols;
  int ldq;
  float* S;
  int64_t s_rows, s_blocks;
  long long s_row, s_block;
};

int check(const Quantize& q, const int* offsets, int experts) {
  if (!known_type(q.type)) return SGEMM_MI355_ERR_TYPE;
  if (q.rows < 0 || q.cols < 0 || q.n < 0) return SGEMM_MI355_ERR_DIM;
  if (offsets != nullptr && experts < 1) return SGEMM_MI355_ERR_DIM;
  if (q.rows > kMostRows || q.cols > kMostRows || q.n > kMostRows || q.q_cols > kMostRows) return SGEMM_MI355_ERR_EXTENT;
  if (q.ldx < at_least_1(q.cols) || q.ldq < at_least_1((int)q.q_cols)) return SGEMM_MI355_ERR_LD;
  if (q.s_row < 0 || q.s_block < 0 || !apart(q.s_rows, q.s_row, q.s_blocks, q.s_block)) return SGEMM_MI355_ERR_STRIDE;
  Matrices m;
  if (q.q_rows > 0 && q.q_cols > 0) {
    m.dense(q.X, q.rows, q.cols, q.ldx, element_size(q.type), false);
    if (q.index != nullptr) m.dense(q.index, 1, q.n, q.n, 4, false);
    if (offsets != nullptr) m.dense(offsets, 1, (int64_t)experts + 1, experts, 4, false);
    m.dense(q.Q, q.q_rows, q.q_cols, q.ldq, 1, true);
    m.strided(q.S, 1, 0, q.s_rows, q.s_row, q.s_blocks, q.s_block, 4, true);
  }
  return m.check();
}

QuantArgs args_of(const Quantize& q, const int* offsets, int experts) {
  return QuantArgs{q.X, q.ldx, q.rows, q.cols, q.index, q.n, offsets, experts, q.Q, q.ldq, q.S, q.s_row, q.s_block};
}

// The type of C, and whether block sums have to be FP32, of a product's `type` argument.
int type_of_c(int type) { return type & ~SGEMM_MI355_FP32_SUMS; }
bool fp32_sums(int type) { return type_of_c(type) == SGEMM_MI355_F32 || (type & SGEMM_MI355_FP32_SUMS) != 0; }

int check_product(const Fp8Args& g, Fp8Form form, int64_t p, int64_t groups) {
  if (!known_type(g.type)) return SGEMM_MI355_ERR_TYPE;
  if (g.sb_rows != 1 && g.sb_rows != 128) return SGEMM_MI355_ERR_OP;
  if (g.M < 0 || g.N < 0 || g.K < 0 || (form != FP8_DENSE && g.experts < 1)) return SGEMM_MI355_ERR_DIM;
  if (g.M > kMostRows || g.N > kMostRows || g.K > kMostRows || p > kMostRows) return SGEMM_MI355_ERR_EXTENT;
  const int least = at_least_1((int)p);
  if (g.lda < least || g.ldb < least || g.ldc < at_least_1(g.N)) return SGEMM_MI355_ERR_LD;
  if (g.sa_row < 0 || g.sa_block < 0 || g.sb_row < 0 || g.sb_block < 0 || g.strideB < 0 || g.stride_sb < 0)
    return SGEMM_MI355_ERR_STRIDE;
  if (g.strideC < 0 || (form == FP8_WGRAD && groups > 1 && g.M > 0 && g.N > 0 &&
                        (Bytes)g.strideC < (Bytes)(g.M - 1) * (Bytes)g.ldc + (Bytes)g.N))
    return SGEMM_MI355_ERR_STRIDE;
  if (g.M == 0 || g.N == 0) return SGEMM_MI355_OK;
  Matrices m;
  const int blocks = blocks_of((int)p);
  const int64_t sb_rows = g.sb_rows == 1 ? g.N : blocks_of(g.N);
  const int64_t experts = form == FP8_EXPERTS ? groups : 1;
  m.dense(g.A, g.M, p, g.lda, 1, false);
  m.strided(g.SA, 1, 0, g.M, g.sa_row, blocks, g.sa_block, 4, false);
  m.strided(g.B, p > 0 ? experts : 0, g.strideB, g.N, g.ldb, p, 1, 1, false);
  m.strided(g.SB, experts, g.stride_sb, sb_rows, g.sb_row, blocks, g.sb_block, 4, false);
  if (form != FP8_DENSE) m.dense(g.offsets, 1, (int64_t)g.experts + 1, g.experts, 4, false);
  const int64_t results = form == FP8_WGRAD ? groups : 1;
  m.strided(g.C, results, g.strideC, g.M, g.ldc, g.N, 1, element_size(g.type), true);
  return m.check();
}

}  // namespace
}  // namespace sgemm_impl

using namespace sgemm_impl;

extern "C" {

int sgemm_mi355_fp8_quantize_rows(int type, int rows, int cols, const void* X, int ldx, const int* index, int n,
                                  unsigned char* Q, int ldq, float* S, long long s_row, long long s_block,
                                  hipStream_t stream) {
  if (index == nullptr) n = rows;
  const Quantize q{type, rows, cols, X, ldx, index, n, Q, n, cols, ldq, S, n, blocks_of(cols), s_row, s_block};
  const int v = check(q, nullptr, 0);
  if (v != SGEMM_MI355_OK || n == 0 || cols == 0) return v;
  if (!launchable(((int64_t)blocks_of(cols) * n + 15) / 16, 256)) return SGEMM_MI355_ERR_EXTENT;
  return done(launch_quantize_rows(type, args_of(q, nullptr, 0), stream));
}

int sgemm_mi355_fp8_quantize_cols(int type, int rows, int cols, const void* X, int ldx, const int* index, int n,
                                  const int* offsets, int experts, unsigned char* Q, int ldq, float* S,
                                  long long s_row, long long s_block, hipStream_t stream) {
  if (index == nullptr) n = rows;
  const int64_t slots = offsets != nullptr ? (int64_t)n / 128 + experts : blocks_of(n);
  const Quantize q{type, rows, cols, X, ldx, index, n, Q, cols, offsets != nullptr ? slots * 128 : n, ldq,
                   S, cols, slots, s_row, s_block};
  const int v = check(q, offsets, experts);
  if (v != SGEMM_MI355_OK || slots == 0 || cols == 0) return v;
  if (!launchable(slots * blocks_of(cols), 256)) return SGEMM_MI355_ERR_EXTENT;
  return done(launch_quantize_cols(type, args_of(q, offsets, experts), stream));
}

int sgemm_mi355_fp8_quantize_tiles(int type, int rows, int cols, const void* X, int ldx, unsigned char* Q, int ldq,
                                   float* S, long long s_row, long long s_block, hipStream_t stream) {
  const Quantize q{type, rows, cols, X, ldx, nullptr, rows, Q, rows, cols, ldq,
                   S, blocks_of(rows), blocks_of(cols), s_row, s_block};
  const int v = check(q, nullptr, 0);
  if (v != SGEMM_MI355_OK || rows == 0 || cols == 0) return v;
  if (!launchable((int64_t)blocks_of(rows) * blocks_of(cols), 256)) return SGEMM_MI355_ERR_EXTENT;
  return done(launch_quantize_tiles(type, args_of(q, nullptr, 0), stream));
}

int sgemm_mi355_fp8_gemm(int type, int M, int N, int K, const unsigned char* A, int lda, const float* SA,
                         long long sa_row, long long sa_block, const unsigned char* B, int ldb, const float* SB,
                         long long sb_row, long long sb_block, int sb_rows, float beta, void* C, int ldc,
                         hipStream_t stream) {
  const Fp8Args g{type_of_c(type), M, N, K, A, lda, SA, sa_row, sa_block, B, ldb, 0, SB, sb_row, sb_block, 0, sb_rows,
                  nullptr, 0, beta, C, ldc, 0, fp32_sums(type)};
  const int v = check_product(g, FP8_DENSE, K, 1);
  if (v != SGEMM_MI355_OK || M == 0 || N == 0) return v;
  if (!fp8_launchable(FP8_DENSE, g)) return SGEMM_MI355_ERR_EXTENT;
  return done(launch_fp8_gemm(FP8_DENSE, g, stream));
}

int sgemm_mi355_fp8_gemm_experts(int type, int rows, int N, int K, int experts, const unsigned char* A, int lda,
                                 const float* SA, long long sa_row, long long sa_block, const unsigned char* B,
                                 int ldb, long long strideB, const float* SB, long long sb_row, long long sb_block,
                                 long long stride_sb, int sb_rows, const int* offsets, void* C, int ldc,
                                 hipStream_t stream) {
  const Fp8Args g{type_of_c(type), rows, N, K, A, lda, SA, sa_row, sa_block, B, ldb, strideB, SB, sb_row, sb_block,
                  stride_sb, sb_rows, offsets, experts, 0.0f, C, ldc, 0, fp32_sums(type)};
  const int v = check_product(g, FP8_EXPERTS, K, experts);
  if (v != SGEMM_MI355_OK || rows == 0 || N == 0) return v;
  if (!fp8_launchable(FP8_EXPERTS, g)) return SGEMM_MI355_ERR_EXTENT;
  return done(launch_fp8_gemm(FP8_EXPERTS, g, stream));
}

int sgemm_mi355_fp8_gemm_experts_wgrad(int type, int rows, int M, int N, int experts, const unsigned char* A,
                                       int lda, const float* SA, long long sa_row, long long sa_block,
                                       const unsigned char* B, int ldb, const float* SB, long long sb_row,
                                       long long sb_block, const int* offsets, float beta, void* C, int ldc,
                                       long long strideC, hipStream_t stream) {
  const Fp8Args g{type_of_c(type), M, N, rows, A, lda, SA, sa_row, sa_block, B, ldb, 0, SB, sb_row, sb_block, 0, 1,
                  offsets, experts, beta, C, ldc, strideC, fp32_sums(type)};
  const int64_t p = rows < 0 || experts < 0 ? 0 : 128 * ((int64_t)rows / 128 + experts);
  const int v = check_product(g, FP8_WGRAD, p, experts);
  if (v != SGEMM_MI355_OK || M == 0 || N == 0) return v;
  if (!fp8_launchable(FP8_WGRAD, g)) return SGEMM_MI355_ERR_EXTENT;
  return done(launch_fp8_gemm(FP8_WGRAD, g, stream));
}

const char* sgemm_mi355_fp8_kernel_name(int form, int type, int M, int N, int K, int experts, const unsigned char* A,
                                        int lda, const unsigned char* B, int ldb, long long strideB) {
  if (form < FP8_DENSE || form > FP8_WGRAD || !known_type(type_of_c(type)) || M < 1 || N < 1 || K < 0) return nullptr;
  if ((form != FP8_DENSE && experts < 1) || lda < 1 || ldb < 1 || strideB < 0) return nullptr;
  Fp8Args g{};
  g.type = type_of_c(type), g.wide = fp32_sums(type), g.M = M, g.N = N, g.K = K, g.experts = experts;
  g.A = A, g.lda = lda, g.B = B, g.ldb = ldb;
  if (form == FP8_EXPERTS) g.strideB = strideB;
  return fp8_kernel_name((Fp8Form)form, g);
}

}  // extern "C"
