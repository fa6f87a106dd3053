// Declarations shared by the norm, activation and column-sum kernels and their host sides.
#pragma once

#include "fp8_internal.h"
#include "sgemm_mi355_layer.h"

namespace sgemm_impl {

// How a kernel reads and writes the rows of its wide matrices, eight columns at a time.
enum Runs {
  RUNS_WHOLE = 0,  // rows are a multiple of eight
  RUNS_ONCE = 1,   // and go past the caches: the matrices are larger than they hold for whoever comes next
  RUNS_ANY = 2     // of any length
};

#if defined(__HIP_DEVICE_COMPILE__) || defined(__HIPCC__)
// Columns col .. col+7 of a row of `cols` as FP32, zeros past its end. At the
// end of a row of any length its last eight are loaded and moved to their
// places (a load for each value, which all of a wave waits for, took a quarter
// of the norm's time for 3001 rows of 2047).
template <int RUNS, class T>
__device__ __forceinline__ void load_run(const T* row, int col, int cols, float (&v)[8]) {
  if constexpr (RUNS == RUNS_ANY) {
    if (cols < 8) {
      load8(row + col, cols - col, v);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (col >= cols) return;
  if constexpr (RUNS == RUNS_WHOLE) {
    load8(row + col, 8, v);
  } else if constexpr (RUNS == RUNS_ONCE) {
    load8_once(row + col, 8, v);
  } else {
    const int at = col + 8 <= cols ? col : cols - 8, by = col - at;
    load8(row + at, 8, v);
    if (by != 0) {
#pragma unroll
      for (int d = 4; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = by & d ? (i + d < 8 ? v[i + d < 8 ? i + d : 0] : 0.0f) : v[i];
    }
  }
}

// The first `valid` (1 .. 7) of eight values, given as two or eight words, in runs of four, two and one.
__device__ __forceinline__ void store_part(uint16_t* p, int valid, uint64_t lo, uint64_t hi) {
  if (valid & 4) __builtin_memcpy(p, &lo, 8), p += 4, lo = hi;
  if (valid & 2) __builtin_memcpy(p, &lo, 4), p += 2, lo >>= 32;
  if (valid & 1) *p = (uint16_t)lo;
}
__device__ __forceinline__ void store_part(float* p, int valid, const float (&v)[8]) {
  float a = v[0], b = v[1], c = v[2];
  if (valid & 4) {
    const float four[4] = {v[0], v[1], v[2], v[3]};
    __builtin_memcpy(p, four, 16);
    p += 4, a = v[4], b = v[5], c = v[6];
  }
  if (valid & 2) {
    p[0] = a, p[1] = b;
    p += 2, a = c;
  }
  if (valid & 1) *p = a;
}

// load_run's values back.
template <int RUNS, class T>
__device__ __forceinline__ void store_run(T* row, int col, int cols, const float (&v)[8]) {
  const int valid = cols - col;
  if (valid >= 8) {
    if constexpr (RUNS == RUNS_ONCE) store8_once(row + col, 8, v);
    else store8(row + col, 8, v);
  } else if constexpr (RUNS == RUNS_ANY) {
    if (valid > 0) {
      if constexpr (sizeof(T) == 4) {
        store_part(row + col, valid, v);
      } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
        uint64_t w[2];
        __builtin_memcpy(w, e, 16);
        store_part((uint16_t*)(row + col), valid, w[0], w[1]);
      }
    }
  }
}

// Eight e4m3 bytes, likewise.
template <int RUNS>
__device__ __forceinline__ void store_run(uint8_t* row, int col, int cols, uint2 b) {
  typedef uint32_t words __attribute__((ext_vector_type(2), aligned(1)));
  const int valid = cols - col;
  uint8_t* p = row + col;
  if (valid >= 8) {
    *(words*)p = words{b.x, b.y};
  } else if constexpr (RUNS == RUNS_ANY) {
    if (valid > 0) {
      uint32_t w = b.x;
      if (valid & 4) __builtin_memcpy(p, &w, 4), p += 4, w = b.y;
      if (valid & 2) __builtin_memcpy(p, &w, 2), p += 2, w >>= 16;
      if (valid & 1) *p = (uint8_t)w;
    }
  }
}
#endif

// f(Act<RUNS>) for the form that a kernel's rows take.
template <class F>
inline hipError_t by_runs(int runs, F&& f) {
  return runs == RUNS_WHOLE ? f(Act<RUNS_WHOLE>{}) : runs == RUNS_ONCE ? f(Act<RUNS_ONCE>{}) : f(Act<RUNS_ANY>{});
}

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
  int runs;  // a Runs
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
  int runs;
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
  int runs;
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
  int runs;
};
hipError_t launch_epilogue_backward(int type, int act, const EpilogueBackArgs& a, float* dbias, hipStream_t s);
// out[c] = sum over groups of sums[group*cols + c].
hipError_t launch_column_sums(const float* sums, int groups, int cols, float* out, hipStream_t s);
// Sets the groups of rows that the bias' gradient is summed over.
void epilogue_groups(int rows, int cols, EpilogueBackArgs& a);

}  // namespace sgemm_impl
