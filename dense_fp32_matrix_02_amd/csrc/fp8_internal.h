// Declarations shared by the FP8 and routing kernels and their host sides.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sgemm_mi355_route.h"

namespace sgemm_impl {

constexpr int kBlock = 128;  // values of the summed axis that share a scale

struct QuantArgs {
  const void* X;
  int64_t ldx;
  int rows, cols;      // of X
  const int* index;    // row i of the quantised matrix is row index[i] of X; null: row i
  int n;               // rows that are quantised
  const int* offsets;  // expert boundaries of the columns form; null: one run of n rows
  int experts;
  uint8_t* Q;
  int64_t ldq;
  float* S;
  int64_t s_row, s_block;
};

hipError_t launch_quantize_rows(int type, const QuantArgs& q, hipStream_t s);
hipError_t launch_quantize_cols(int type, const QuantArgs& q, hipStream_t s);
hipError_t launch_quantize_tiles(int type, const QuantArgs& q, hipStream_t s);

// One FP8 product, or one for each expert. DENSE: C = A.B^T + beta*C. EXPERTS:
// rows of A and C belong to experts by `offsets`, B_e = B + e*strideB.
// WGRAD: the summed axis belongs to experts, C_e = C + e*strideC.
enum Fp8Form { FP8_DENSE = 0, FP8_EXPERTS = 1, FP8_WGRAD = 2 };

struct Fp8Args {
  int type, M, N, K;  // WGRAD: K = the rows that offsets count
  const uint8_t* A;
  int64_t lda;
  const float* SA;
  int64_t sa_row, sa_block;
  const uint8_t* B;
  int64_t ldb, strideB;
  const float* SB;
  int64_t sb_row, sb_block, stride_sb;
  int sb_rows;  // rows of B that share a scale: 1 or 128
  const int* offsets;
  int experts;
  float beta;
  void* C;
  int64_t ldc, strideC;
  bool wide;  // block sums have to be FP32 sums: C is FP32, or the caller asks for it
};

hipError_t launch_fp8_gemm(Fp8Form form, const Fp8Args& g, hipStream_t s);
// Kernels for aligned operands (kernels_fp8_tile.hip, kernels_fp8_skinny.hip). wide: the values are widened to bf16.
// tall: B has a scale for each 128 rows; bm: rows of A in a workgroup's tile.
const void* fp8_tile_kernel_for(Fp8Form form, bool wide, bool tall, int bm);
const void* fp8_skinny_kernel_for(Fp8Form form, bool tall, int bm);
// Whether the grids launch_fp8_gemm would use for g fit a launch.
bool fp8_launchable(Fp8Form form, const Fp8Args& g);
// The name of the kernel that launch_fp8_gemm would run for g.
const char* fp8_kernel_name(Fp8Form form, const Fp8Args& g);

// Beginning and end of expert e's rows: offsets limited to 0 .. rows, an end
// before the beginning gives no rows, and the first expert begins at 0.
__device__ __forceinline__ void expert_rows(const int* offsets, int e, int rows, int& begin, int& end) {
  const int b = e == 0 ? 0 : offsets[e], t = offsets[e + 1];
  begin = b < 0 ? 0 : (b > rows ? rows : b);
  end = t < begin ? begin : (t > rows ? rows : t);
}

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int tokens, experts, groups, top_groups, choices, renorm;
  float scale;
  float* weights;
  int* ids;
  // backward
  const int* ids_in;
  const float* dweights;
  float* dlogits;
  int64_t ldd;
};

hipError_t launch_route(int type, int score, const RouteArgs& r, hipStream_t s);
hipError_t launch_route_backward(int type, int score, const RouteArgs& r, hipStream_t s);

struct PlanArgs {
  int entries, choices, experts;
  const int* ids;
  int *offsets, *row_token, *place;
  int* counts;  // workspace: entries of each expert in each run, then (with groups) in each group of runs
  int runs;     // runs of kPlanRun entries; 1 for no entries: the offsets are written all the same
  int per;      // runs in a group; 0 where they are not grouped
  int groups;   // groups of runs, the last one shorter
};
constexpr int kPlanRun = 2048;
constexpr int kPlanGroups = 512;  // groups at most
// The division of up to 2^31 - 1 entries, whose number rounded up to whole runs needs 64 bits.
// Runs are grouped where every run reading the counts of all costs more than the
// groups' kernel (us, without and with groups, 8 choices of
//   8 experts, 512 / 1024 / 4096 runs      15.9, 20.6 / 28.8, 31.4 / 130, 87
//   64 experts, 256 / 512 / 1024 runs      11.4, 15.1 / 20.9, 22.6 / 47.8, 35.5
//   256 experts, 128 / 256 / 4096 runs     12.3, 14.1 / 17.2, 16.7 / 1363, 107
//   1024 experts, 32 / 64 / 128 runs       13.3, 15.2 / 16.4, 15.8 / 22.5, 17.3).
inline void plan_division(int64_t entries, int experts, PlanArgs& p) {
  p.runs = entries > kPlanRun ? (int)((entries + kPlanRun - 1) / kPlanRun) : 1;
  const int64_t numbers = (int64_t)p.runs * (experts + 1);  // that each run reads
  const bool grouped = numbers > 1 << 16 || numbers * p.runs > 1 << 25;
  p.per = grouped ? (p.runs + kPlanGroups - 1) / kPlanGroups : 0;
  p.groups = grouped ? (p.runs + p.per - 1) / p.per : 0;
}
hipError_t launch_route_plan(const PlanArgs& p, hipStream_t s);

struct CombineArgs {
  int tokens, choices, rows, cols;
  const void* Z;
  int64_t ldz;
  const int* place;
  const float* weights;
  void* Y;
  int64_t ldy;
  // backward
  const void* dY;
  int64_t lddy;
  void* dZ;
  int64_t lddz;
  float* dweights;
};
hipError_t launch_combine(int type, const CombineArgs& c, hipStream_t s);
hipError_t launch_combine_backward(int type, const CombineArgs& c, hipStream_t s);

// Kernel arguments by value through hipLaunchKernel.
template <class Args>
inline hipError_t launch_with(const void* kernel, dim3 grid, dim3 block, const Args& a, hipStream_t s) {
  Args copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(kernel, grid, block, args, 0, s);
}

// f(T{}) for the element type that `type` names.
template <class F>
inline hipError_t by_type(int type, F&& f) {
  switch (type) {
    case SGEMM_MI355_F32: return f(float{});
    case SGEMM_MI355_BF16: return f(__hip_bfloat16{});
    default: return f(__half{});
  }
}

#if defined(__HIP_DEVICE_COMPILE__) || defined(__HIPCC__)
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__hip_bfloat16 x) {
  uint16_t u;
  __builtin_memcpy(&u, &x, 2);
  return __uint_as_float((uint32_t)u << 16);
}
// Rounded to the nearest, half to even; NaN stays NaN.
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __hip_bfloat16 from_f32<__hip_bfloat16>(float x) {
  const __bf16 r = (__bf16)x;
  __hip_bfloat16 y;
  __builtin_memcpy(&y, &r, 2);
  return y;
}

// `valid` (any number) of eight consecutive elements at p as FP32, the rest
// zero. p needs only its element's alignment: a whole vector load needs none
// on this hardware beyond that.
template <class T>
__device__ __forceinline__ void load8(const T* p, int valid, float (&v)[8]) {
  if (valid >= 8) {
    T e[8];
    __builtin_memcpy(e, p, sizeof(e));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < valid ? to_f32(p[i]) : 0.0f;
  }
}
template <class T>
__device__ __forceinline__ void store8(T* p, int valid, const float (&v)[8]) {
  if (valid >= 8) {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
    __builtin_memcpy(p, e, sizeof(e));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = from_f32<T>(v[i]);
  }
}

// load8 and store8, for what is used once.
template <class T>
__device__ __forceinline__ void load8_once(const T* p, int valid, float (&v)[8]) {
  typedef int words __attribute__((ext_vector_type(4), aligned(2)));
  if (valid >= 8) {
    T e[8];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const words w = __builtin_nontemporal_load((const words*)p + i);
      __builtin_memcpy((char*)e + 16 * i, &w, 16);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  } else {
    load8(p, valid, v);
  }
}
template <class T>
__device__ __forceinline__ void store8_once(T* p, int valid, const float (&v)[8]) {
  typedef int words __attribute__((ext_vector_type(4), aligned(2)));
  if (valid >= 8) {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      words w;
      __builtin_memcpy(&w, (const char*)e + 16 * i, 16);
      __builtin_nontemporal_store(w, (words*)p + i);
    }
  } else {
    store8(p, valid, v);
  }
}
#endif

}  // namespace sgemm_impl
