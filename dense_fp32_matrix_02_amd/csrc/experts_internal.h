// Declarations shared by the 16-bit experts' products and their host side.
#pragma once

#include "fp8_internal.h"
#include "sgemm_mi355_experts.h"

namespace sgemm_impl {

// C = A.B^T, C = A.B, or C_e = A^T.B, with M x N results summed over K.
// FORWARD: rows of A (M x K) meet B_e (N x K). DGRAD: rows of A (M x K) meet
// B_e (K x N). WGRAD: expert e's rows, of K, of A (K x M) and B (K x N).
enum ExpertsForm { EXPERTS_FORWARD = 0, EXPERTS_DGRAD = 1, EXPERTS_WGRAD = 2 };

struct ExpertsArgs {
  int type, c_type, M, N, K, experts;
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb, strideB;
  const int* offsets;
  float beta;
  void* C;
  int64_t ldc, strideC;
  bool past;  // C goes past the caches
};

hipError_t launch_experts(ExpertsForm form, const ExpertsArgs& g, hipStream_t s);
bool experts_launchable(ExpertsForm form, const ExpertsArgs& g);
const char* experts_kernel_name(ExpertsForm form, const ExpertsArgs& g);
// Kernels for aligned operands (kernels_experts_tile.hip, kernels_experts.hip).
const void* experts_tile_kernel_for(ExpertsForm form, int type, int bm);

}  // namespace sgemm_impl
