// Host side of include/sgemm_mi355_layer.h: argument checks, then the launches.

#include "sgemm_mi355_layer.h"

#include <cmath>

#include "api_checks.h"
#include "layer_internal.h"

namespace sgemm_impl {
namespace {

bool known_act(int act) { return act >= SGEMM_MI355_NONE && act <= SGEMM_MI355_GELU_TANH; }

int check_norm(int type, int w_type, int rows, int cols) {
  if (!known_type(type) || (w_type != type && w_type != SGEMM_MI355_F32)) return SGEMM_MI355_ERR_TYPE;
  if (rows < 0 || cols < 1) return SGEMM_MI355_ERR_DIM;
  if (rows > kMostRows || cols > SGEMM_MI355_MAX_NORM_COLS) return SGEMM_MI355_ERR_EXTENT;
  return SGEMM_MI355_OK;
}

// Q and S of rows x cols: strides, then their places among the matrices.
int check_quantised(int rows, int cols, const void* Q, int ldq, const void* S, long long s_row, long long s_block) {
  if ((Q == nullptr) != (S == nullptr)) return SGEMM_MI355_ERR_NULL;
  if (Q == nullptr) return SGEMM_MI355_OK;
  if (ldq < at_least_1(cols)) return SGEMM_MI355_ERR_LD;
  if (s_row < 0 || s_block < 0 || !apart(rows, s_row, blocks_of(cols), s_block)) return SGEMM_MI355_ERR_STRIDE;
  return SGEMM_MI355_OK;
}
void add_quantised(Matrices& m, int rows, int cols, const void* Q, int ldq, const void* S, long long s_row, long long s_block) {
  if (Q == nullptr) return;
  m.dense(Q, rows, cols, ldq, 1, true);
  m.strided(S, 1, 0, rows, s_row, blocks_of(cols), s_block, 4, true);
}

int check_activation(int type, int act, int rows, int cols) {
  if (!known_type(type)) return SGEMM_MI355_ERR_TYPE;
  if (!known_act(act)) return SGEMM_MI355_ERR_OP;
  if (rows < 0 || cols < 0) return SGEMM_MI355_ERR_DIM;
  if (rows > kMostRows || cols > kMostRows) return SGEMM_MI355_ERR_EXTENT;
  return SGEMM_MI355_OK;
}

// The form of the rows of matrices of rows x cols elements; `aligned`: each of
// them 16-byte aligned. Past the caches (8192 x 8192 bf16 in the epilogue's
// backward pass 75.5 us against 96.2 through them, 16384 x 2048 in the gated
// one 57.4 and 70.1) go those that the caches do not hold for whoever comes
// next; of smaller ones, or with rows that share lines with their neighbours
// (3001 x 2047 in the norm: 23.7 against 17.7), it costs time.
int runs_of(int rows, int cols, int size, bool aligned) {
  if (cols % 8 != 0) return RUNS_ANY;
  return aligned && (int64_t)rows * cols * size >= (int64_t)64 << 20 ? RUNS_ONCE : RUNS_WHOLE;
}
bool aligned16(const void* p, int64_t ld, int size) { return (((uintptr_t)p | (uint64_t)(ld * size)) & 15) == 0; }

size_t sums_bytes(int groups, int cols) { return groups > 1 ? (size_t)groups * (size_t)cols * 4 : 0; }

}  // namespace
}  // namespace sgemm_impl

using namespace sgemm_impl;

extern "C" {

int sgemm_mi355_rms_norm(int type, int rows, int cols, const void* X, int ldx, const void* R, int ldr, const void* W,
                         int w_type, float eps, void* H, int ldh, float* rstd, void* Y, int ldy, unsigned char* Q,
                         int ldq, float* S, long long s_row, long long s_block, hipStream_t stream) {
  int v = check_norm(type, w_type, rows, cols);
  if (v != SGEMM_MI355_OK) return v;
  if (!(eps >= 0.0f) || std::isinf(eps)) return SGEMM_MI355_ERR_OP;
  if (ldx < cols || (R != nullptr && ldr < cols) || (H != nullptr && ldh < cols) || (Y != nullptr && ldy < cols))
    return SGEMM_MI355_ERR_LD;
  v = check_quantised(rows, cols, Q, ldq, S, s_row, s_block);
  if (v != SGEMM_MI355_OK || rows == 0) return v;
  if (H == nullptr && rstd == nullptr && Y == nullptr && Q == nullptr) return SGEMM_MI355_ERR_NULL;
  const int size = element_size(type);
  Matrices m;
  // H in the place of X or of R is one matrix, an output.
  if (X == nullptr || H != X || ldh != ldx) m.dense(X, rows, cols, ldx, size, false);
  if (R != nullptr && (H != R || ldh != ldr)) m.dense(R, rows, cols, ldr, size, false);
  m.dense(W, 1, cols, cols, element_size(w_type), false);
  if (H != nullptr) m.dense(H, rows, cols, ldh, size, true);
  if (rstd != nullptr) m.dense(rstd, 1, rows, rows, 4, true);
  if (Y != nullptr) m.dense(Y, rows, cols, ldy, size, true);
  add_quantised(m, rows, cols, Q, ldq, S, s_row, s_block);
  v = m.check();
  if (v != SGEMM_MI355_OK) return v;
  const NormArgs a{rows, cols, X, ldx, R, ldr, W, w_type == SGEMM_MI355_F32, eps, H, ldh, rstd, Y, ldy, Q, ldq, S, s_row, s_block,
                   runs_of(rows, cols, size, aligned16(X, ldx, size) && aligned16(R, R ? ldr : 0, size) && aligned16(H, H ? ldh : 0, size))};
  return done(launch_norm(type, a, stream));
}

size_t sgemm_mi355_rms_norm_backward_workspace_size(int rows, int cols) {
  if (rows < 1 || cols < 1 || cols > SGEMM_MI355_MAX_NORM_COLS) return 0;
  return sums_bytes(norm_groups(rows, cols), cols);
}

int sgemm_mi355_rms_norm_backward(int type, int rows, int cols, const void* dY, int lddy, const void* H, int ldh,
                                  const float* rstd, const void* W, int w_type, const void* dH, int lddh, void* dX,
                                  int lddx, float* dW, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int v = check_norm(type, w_type, rows, cols);
  if (v != SGEMM_MI355_OK) return v;
  if (lddy < cols || ldh < cols || (dH != nullptr && lddh < cols) || lddx < cols) return SGEMM_MI355_ERR_LD;
  if (rows == 0) return SGEMM_MI355_OK;
  const size_t need = dW != nullptr ? sgemm_mi355_rms_norm_backward_workspace_size(rows, cols) : 0;
  const int size = element_size(type);
  Matrices m;
  if (dY == nullptr || dX != dY || lddx != lddy) m.dense(dY, rows, cols, lddy, size, false);
  m.dense(H, rows, cols, ldh, size, false);
  m.dense(rstd, 1, rows, rows, 4, false);
  m.dense(W, 1, cols, cols, element_size(w_type), false);
  if (dH != nullptr && (dX != dH || lddx != lddh)) m.dense(dH, rows, cols, lddh, size, false);
  m.dense(dX, rows, cols, lddx, size, true);
  if (dW != nullptr) m.dense(dW, 1, cols, cols, 4, true);
  if (need > 0 && workspace_bytes >= need) m.dense(workspace, 1, (int64_t)(need / 4), (int64_t)(need / 4), 4, true);
  v = m.check();
  if (v != SGEMM_MI355_OK) return v;
  if (workspace_bytes < need) return SGEMM_MI355_ERR_WORKSPACE;
  const int groups = norm_groups(rows, cols);
  const NormBackArgs a{rows, cols, dY, lddy, H, ldh, rstd, W, w_type == SGEMM_MI355_F32, dH, lddh, dX, lddx,
                       dW == nullptr ? nullptr : groups > 1 ? (float*)workspace : dW, groups,
                       runs_of(rows, cols, size, aligned16(dX, lddx, size))};
  return done(launch_norm_backward(type, a, dW, stream));
}

int sgemm_mi355_gated(int type, int act, int rows, int cols, const void* H, int ldh, void* Z, int ldz,
                      unsigned char* Q, int ldq, float* S, long long s_row, long long s_block, hipStream_t stream) {
  int v = check_activation(type, act, rows, cols);
  if (v != SGEMM_MI355_OK) return v;
  if (2 * (int64_t)cols > kMostRows) return SGEMM_MI355_ERR_EXTENT;
  if (ldh < at_least_1(2 * cols) || (Z != nullptr && ldz < at_least_1(cols))) return SGEMM_MI355_ERR_LD;
  v = check_quantised(rows, cols, Q, ldq, S, s_row, s_block);
  if (v != SGEMM_MI355_OK || rows == 0 || cols == 0) return v;
  if (Z == nullptr && Q == nullptr) return SGEMM_MI355_ERR_NULL;
  if (!launchable(((int64_t)blocks_of(cols) * rows + 15) / 16, 256)) return SGEMM_MI355_ERR_EXTENT;
  Matrices m;
  m.dense(H, rows, 2 * (int64_t)cols, ldh, element_size(type), false);
  if (Z != nullptr) m.dense(Z, rows, cols, ldz, element_size(type), true);
  add_quantised(m, rows, cols, Q, ldq, S, s_row, s_block);
  v = m.check();
  if (v != SGEMM_MI355_OK) return v;
  GatedArgs a{};
  a.rows = rows, a.cols = cols, a.H = H, a.ldh = ldh, a.Z = Z, a.ldz = ldz, a.Q = Q, a.ldq = ldq;
  a.S = S, a.s_row = s_row, a.s_block = s_block, a.runs = cols % 8 == 0 ? RUNS_WHOLE : RUNS_ANY;
  return done(launch_gated(type, act, a, stream));
}

int sgemm_mi355_gated_backward(int type, int act, int rows, int cols, const void* dZ, int lddz, const void* H, int ldh,
                               void* dH, int lddh, hipStream_t stream) {
  int v = check_activation(type, act, rows, cols);
  if (v != SGEMM_MI355_OK) return v;
  if (2 * (int64_t)cols > kMostRows) return SGEMM_MI355_ERR_EXTENT;
  if (lddz < at_least_1(cols) || ldh < at_least_1(2 * cols) || lddh < at_least_1(2 * cols)) return SGEMM_MI355_ERR_LD;
  if (rows == 0 || cols == 0) return SGEMM_MI355_OK;
  if (!launchable(((int64_t)((cols + 7) / 8) * rows + 255) / 256, 256)) return SGEMM_MI355_ERR_EXTENT;
  Matrices m;
  m.dense(dZ, rows, cols, lddz, element_size(type), false);
  m.dense(H, rows, 2 * (int64_t)cols, ldh, element_size(type), false);
  m.dense(dH, rows, 2 * (int64_t)cols, lddh, element_size(type), true);
  v = m.check();
  if (v != SGEMM_MI355_OK) return v;
  GatedArgs a{};
  a.rows = rows, a.cols = cols, a.H = H, a.ldh = ldh, a.dZ = dZ, a.lddz = lddz, a.dH = dH, a.lddh = lddh;
  const int size = element_size(type);
  a.runs = runs_of(rows, cols, size, aligned16(dZ, lddz, size) && aligned16(H, ldh, size) && aligned16(dH, lddh, size));
  return done(launch_gated_backward(type, act, a, stream));
}

size_t sgemm_mi355_epilogue_backward_workspace_size(int rows, int cols) {
  if (rows < 1 || cols < 1 || rows > kMostRows || cols > kMostRows) return 0;
  EpilogueBackArgs a{};
  epilogue_groups(rows, cols, a);
  return sums_bytes(a.groups, cols);
}

int sgemm_mi355_epilogue_backward(int type, int act, int rows, int cols, const void* dC, int lddc, const void* P,
                                  int ldp, void* dP, int lddp, float* dbias, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
  int v = check_activation(type, act, rows, cols);
  if (v != SGEMM_MI355_OK) return v;
  if (lddc < at_least_1(cols) || ldp < at_least_1(cols) || lddp < at_least_1(cols)) return SGEMM_MI355_ERR_LD;
  if (rows == 0 || cols == 0) return SGEMM_MI355_OK;
  if (!launchable(((int64_t)cols + 63) / 64, 1024)) return SGEMM_MI355_ERR_EXTENT;
  const size_t need = dbias != nullptr ? sgemm_mi355_epilogue_backward_workspace_size(rows, cols) : 0;
  Matrices m;
  m.dense(dC, rows, cols, lddc, element_size(type), false);
  m.dense(P, rows, cols, ldp, element_size(type), false);
  m.dense(dP, rows, cols, lddp, element_size(type), true);
  if (dbias != nullptr) m.dense(dbias, 1, cols, cols, 4, true);
  if (need > 0 && workspace_bytes >= need) m.dense(workspace, 1, (int64_t)(need / 4), (int64_t)(need / 4), 4, true);
  v = m.check();
  if (v != SGEMM_MI355_OK) return v;
  if (workspace_bytes < need) return SGEMM_MI355_ERR_WORKSPACE;
  EpilogueBackArgs a{};
  a.rows = rows, a.cols = cols, a.dC = dC, a.lddc = lddc, a.P = P, a.ldp = ldp, a.dP = dP, a.lddp = lddp;
  epilogue_groups(rows, cols, a);
  const int size = element_size(type);
  a.runs = runs_of(rows, cols, size, aligned16(dC, lddc, size) && aligned16(P, ldp, size) && aligned16(dP, lddp, size));
  a.sums = dbias == nullptr ? nullptr : a.groups > 1 ? (float*)workspace : dbias;
  return done(launch_epilogue_backward(type, act, a, dbias, stream));
}

}  // extern "C"
