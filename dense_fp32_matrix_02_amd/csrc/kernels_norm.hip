// Root-mean-square norm with the residual's addition, into e4m3 with a scale
// for each block of 128 values and into wide rows, and its backward pass.
//
//   h = x + r, rounded to x's type;  a = 1 / sqrt(mean(h^2) + eps);  y = h a w
//   g = w dy, n = h a:  dx = a (g - n mean(g n)) + dh,  dw = sum over rows of dy n
//
// One pass over the data: a team of threads holds a row in registers, eight
// neighbours of it per thread and step, so that sixteen lanes hold a block of
// 128 and find its scale among themselves. Bound by the bytes read and written:
// 8192 x 4096 bf16 with a residual, into h and e4m3, 47.5 us (5.0 TB/s), its
// backward pass with dh 53.6 us (5.0 TB/s) and the column sums of dw 6; 8 rows
// 5 us, latency.

#include "fp8_quantize.h"
#include "layer_internal.h"

namespace sgemm_impl {
namespace {

template <class V>
__device__ __forceinline__ V wave_sum(V x) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d, 64);
  return x;
}

// Sums over a team of NT threads, the same in all of them. A team larger than
// a wave is the whole workgroup; calls in a row alternate between two places,
// so that one barrier each is enough.
template <int NT, class V>
struct TeamSum {
  V (*room)[NT / 64];
  int turn = 0;
  __device__ __forceinline__ V operator()(V x) {
    x = wave_sum(x);
    if constexpr (NT > 64) {
      if (threadIdx.x % 64 == 0) room[turn][threadIdx.x / 64] = x;
      __syncthreads();
      x = 0;
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) x += room[turn][w];
      turn ^= 1;
    }
    return x;
  }
};

template <int RUNS, class T>
__device__ __forceinline__ void load_weights(const void* W, bool f32, int col, int cols, float (&w)[8]) {
  if (f32) load_run<RUNS == RUNS_ONCE ? RUNS_WHOLE : RUNS>((const float*)W, col, cols, w);
  else load_run<RUNS == RUNS_ONCE ? RUNS_WHOLE : RUNS>((const T*)W, col, cols, w);
}

// Eight neighbours of h at column col (zeros past the row), written to H where that is asked for.
template <int RUNS, class T>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t row, int col, float (&v)[8]) {
  load_run<RUNS>((const T*)a.X + row * a.ldx, col, a.cols, v);
  if (a.R != nullptr) {
    float r[8];
    load_run<RUNS>((const T*)a.R + row * a.ldr, col, a.cols, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(from_f32<T>(v[i] + r[i]));
  }
  if (a.H != nullptr) store_run<RUNS>((T*)a.H + row * a.ldh, col, a.cols, v);
}

// Eight neighbours of y = h a w to Y and, sixteen lanes together, to Q and S.
template <int RUNS, class T>
__device__ __forceinline__ void finish(const NormArgs& a, int64_t row, int col, const float (&h)[8], float norm,
                                       const float (&w)[8]) {
  const int valid = a.cols - col;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = h[i] * norm * w[i];
  if (a.Y != nullptr) store_run<RUNS == RUNS_ONCE ? RUNS_WHOLE : RUNS>((T*)a.Y + row * a.ldy, col, a.cols, y);
  if (a.Q == nullptr) return;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, i < valid ? mag(y[i]) : 0u);
#pragma unroll
  for (int d = 1; d < 16; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  const float s = scale_of(m);
  store_run<RUNS>(a.Q + row * a.ldq, col, a.cols, quantize8(y, s));
  if (threadIdx.x % 16 == 0 && valid > 0) a.S[row * a.s_row + (int64_t)(col / kBlock) * a.s_block] = s;
}

// 1 / sqrt(mean(h^2) + eps). Squares are added in FP32, unless their sum shows
// that some left its range or its whole precision: then in FP64.
template <int NT, int NC>
__device__ __forceinline__ float norm_of(const float (&h)[NC][8], int cols, float eps, TeamSum<NT, float>& team_sum,
                                         TeamSum<NT, double>& wide_sum) {
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(h[c][i], h[c][i], sum);
  sum = team_sum(sum);
  if (sum < 0x1p127f && sum > 0x1p-90f) return 1.0f / sqrtf(sum / (float)cols + eps);
  double wide = 0.0;  // the whole team is here
#pragma unroll 1
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) wide += (double)h[c][i] * h[c][i];
  return (float)(1.0 / sqrt(wide_sum(wide) / cols + (double)eps));
}

// NC steps of a team of NT threads hold a row of up to 8*NT*NC columns.
template <class T, int NT, int NC, int RUNS>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) norm_kernel(NormArgs a) {
  constexpr int TEAMS = NT < 256 ? 256 / NT : 1;
  __shared__ float room[2][NT / 64];
  __shared__ double wide_room[2][NT / 64];
  TeamSum<NT, float> team_sum{room};
  TeamSum<NT, double> wide_sum{wide_room};
  const int t = threadIdx.x % NT;
  float w[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) load_weights<RUNS, T>(a.W, a.w_f32, 8 * (t + NT * c), a.cols, w[c]);
  for (int64_t row = (int64_t)blockIdx.x * TEAMS + threadIdx.x / NT; row < a.rows; row += (int64_t)gridDim.x * TEAMS) {
    float h[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) load_h<RUNS, T>(a, row, 8 * (t + NT * c), h[c]);
    const float norm = norm_of<NT, NC>(h, a.cols, a.eps, team_sum, wide_sum);
#pragma unroll
    for (int c = 0; c < NC; ++c) finish<RUNS, T>(a, row, 8 * (t + NT * c), h[c], norm, w[c]);
    if (t == 0 && a.rstd != nullptr) a.rstd[row] = norm;
  }
}

// The backward pass: the workgroups' teams take turns at the rows and keep
// their shares of dw in registers; a workgroup's are added in the teams' order,
// the groups' by column_sums.
template <class T, int NT, int NC, int RUNS>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) norm_backward_kernel(NormBackArgs a) {
  constexpr int TEAMS = NT < 256 ? 256 / NT : 1;
  constexpr int LOADS = RUNS == RUNS_ONCE ? RUNS_WHOLE : RUNS;  // 8192 x 4096 bf16: stores alone past the caches 61.7 us, loads too 62.7
  __shared__ float room[2][NT / 64];
  TeamSum<NT, float> team_sum{room};
  const int t = threadIdx.x % NT;
  const int group = blockIdx.x, team = threadIdx.x / NT;
  float w[NC][8], dw[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    load_weights<RUNS, T>(a.W, a.w_f32, 8 * (t + NT * c), a.cols, w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  }
  for (int64_t row = (int64_t)group * TEAMS + team; row < a.rows; row += (int64_t)a.groups * TEAMS) {
    const float norm = a.rstd[row];
    float n[NC][8], g[NC][8], dot = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = 8 * (t + NT * c);
      load_run<LOADS>((const T*)a.H + row * a.ldh, col, a.cols, n[c]);
      load_run<LOADS>((const T*)a.dY + row * a.lddy, col, a.cols, g[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[c][i] *= norm;
        dw[c][i] = __builtin_fmaf(g[c][i], n[c][i], dw[c][i]);
        g[c][i] *= w[c][i];
        dot = __builtin_fmaf(g[c][i], n[c][i], dot);
      }
    const float mean = team_sum(dot) / (float)a.cols;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = 8 * (t + NT * c);
      float d[8] = {};
      if (a.dH != nullptr) load_run<LOADS>((const T*)a.dH + row * a.lddh, col, a.cols, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] += norm * (g[c][i] - n[c][i] * mean);
      store_run<RUNS>((T*)a.dX + row * a.lddx, col, a.cols, d);
    }
  }
  if (a.sums == nullptr) return;
  if constexpr (TEAMS > 1) {
    __shared__ __align__(16) float shares[TEAMS - 1][NC * NT * 8];
    if (team > 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) shares[team - 1][(c * 8 + i) * NT + t] = dw[c][i];
    }
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int x = 0; x < TEAMS - 1; ++x) dw[c][i] += shares[x][(c * 8 + i) * NT + t];
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = 8 * (t + NT * c);
    store8(a.sums + (int64_t)group * a.cols + col, a.cols - col, dw[c]);
  }
}

// f with the team size and steps for rows of `cols`.
template <class F>
hipError_t by_columns(int cols, F&& f) {
  if (cols <= 512) return f(Act<64>{}, Act<1>{});
  if (cols <= 1024) return f(Act<64>{}, Act<2>{});
  if (cols <= 2048) return f(Act<256>{}, Act<1>{});
  if (cols <= 4096) return f(Act<256>{}, Act<2>{});
  if (cols <= 8192) return f(Act<512>{}, Act<2>{});
  return f(Act<1024>{}, Act<2>{});
}

}  // namespace

hipError_t launch_norm(int type, const NormArgs& a, hipStream_t s) {
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto nt, auto nc) {
      constexpr int NT = decltype(nt)::value, NC = decltype(nc)::value, TEAMS = NT < 256 ? 256 / NT : 1;
      const int64_t grid = ((int64_t)a.rows + TEAMS - 1) / TEAMS;
      return by_runs(a.runs, [&](auto runs) {
        return launch_with((const void*)&norm_kernel<T, NT, NC, decltype(runs)::value>, dim3((unsigned)(grid < 1 << 20 ? grid : 1 << 20)),
                         dim3(NT < 256 ? 256 : NT), a, s);
      });
    };
    return by_columns(a.cols, go);
  });
}

int norm_groups(int rows, int cols) {
  const int teams = cols <= 1024 ? 4 : 1, most = cols <= 1024 || cols > 4096 ? 512 : 1024;
  const int all = rows / teams + (rows % teams != 0);
  return all < most ? all : most;
}

hipError_t launch_norm_backward(int type, const NormBackArgs& a, float* dW, hipStream_t s) {
  const hipError_t e = by_type(type, [&](auto t) {
    using T = decltype(t);
    return by_columns(a.cols, [&](auto nt, auto nc) {
      constexpr int NT = decltype(nt)::value, NC = decltype(nc)::value;
      return by_runs(a.runs, [&](auto runs) {
        return launch_with((const void*)&norm_backward_kernel<T, NT, NC, decltype(runs)::value>, dim3((unsigned)a.groups),
                         dim3(NT < 256 ? 256 : NT), a, s);
      });
    });
  });
  if (e != hipSuccess || a.sums == nullptr || a.groups == 1) return e;
  return launch_column_sums(a.sums, a.groups, a.cols, dW, s);
}

}  // namespace sgemm_impl
