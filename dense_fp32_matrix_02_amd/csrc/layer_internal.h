// Declarations shared by the norm, activation and column-sum kernels and their host sides.
#pragma once

#include "fp8_internal.h"
#include "sgemm_mi355_layer.h"

namespace sgemm_impl {

struct NormArgs {
  int rows, cols;
  const void* X;
  int64_t ldx;
  const void* R;  // null: no residual
  int64_t ldr;
  const void* W;
  bool w_f32;  // W is FP32, else of X's type
  float eps;
  void* H;  // the outputs: each null where it is not asked for
  int64_t ldh;
  float* rstd;
  void* Y;
  int64_t ldy;
  uint8_t* Q;
  int64_t ldq;
  float* S;
  int64_t s_row, s_block;
};
hipError_t launch_norm(int type, const NormArgs& a, hipStream_t s);

struct NormBackArgs {
  int rows, cols;
  const void* dY;
  int64_t lddy;
  const void* H;
  int64_t ldh;
  const float* rstd;
  const void* W;
  bool w_f32;
  const void* dH;  // null: none
  int64_t lddh;
  void* dX;
  int64_t lddx;
  float* sums;  // a row of partial column sums for each group of rows; null: no dW
  int groups;
};
hipError_t launch_norm_backward(int type, const NormBackArgs& a, float* dW, hipStream_t s);
// Groups of rows that the norm's backward pass sums dW over.
int norm_groups(int rows, int cols);

struct GatedArgs {
  int rows, cols;  // of Z
  const void* H;
  int64_t ldh;
  void* Z;  // null: not asked for
  int64_t ldz;
  uint8_t* Q;  // null: not asked for
  int64_t ldq;
  float* S;
  int64_t s_row, s_block;
  const void* dZ;  // backward
  int64_t lddz;
  void* dH;
  int64_t lddh;
};
hipError_t launch_gated(int type, int act, const GatedArgs& a, hipStream_t s);
hipError_t launch_gated_backward(int type, int act, const GatedArgs& a, hipStream_t s);

struct EpilogueBackArgs {
  int rows, cols;
  const void* dC;
  int64_t lddc;
  const void* P;
  int64_t ldp;
  void* dP;
  int64_t lddp;
  float* sums;  // as in NormBackArgs
  int groups;
  int per;  // rows of a group
};
hipError_t launch_epilogue_backward(int type, int act, const EpilogueBackArgs& a, float* dbias, hipStream_t s);
// out[c] = sum over groups of sums[group*cols + c].
hipError_t launch_column_sums(const float* sums, int groups, int cols, float* out, hipStream_t s);
// Sets the groups of rows that the bias' gradient is summed over.
void epilogue_groups(int rows, int cols, EpilogueBackArgs& a);

}  // namespace sgemm_impl
