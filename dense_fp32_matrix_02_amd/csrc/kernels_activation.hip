// Gated activations into e4m3, their backward pass, the backward pass of a
// product's epilogue, and sums of columns. Bound by the bytes read and written:
// bf16, 16384 x 2048 of z, SiLU, into e4m3 41 us (4.1 TB/s) and back 59 us (5.7
// TB/s, some of it from the caches); 8192 x 8192 of the epilogue, the tanh form of
// GELU, back 74 us (5.4 TB/s).

#include "activation.h"
#include "fp8_quantize.h"
#include "layer_internal.h"

namespace sgemm_impl {
namespace {

// z = act(g) u of H = [g | u]. Sixteen lanes hold one block of 128 of a row of
// z, eight values each.
template <class T, int ACT, int RUNS>
__global__ void __launch_bounds__(256) gated_kernel(GatedArgs a) {
  const uint32_t blocks = (uint32_t)(a.cols + kBlock - 1) / kBlock;
  const uint64_t group = (uint64_t)blockIdx.x * 16 + threadIdx.x / 16;
  if (group >= (uint64_t)blocks * (uint32_t)a.rows) return;  // the same for all 16 lanes of a block
  const uint32_t row = (uint32_t)group / blocks, b = (uint32_t)group - row * blocks;
  const int col = (int)(b * kBlock) + 8 * (threadIdx.x % 16), valid = a.cols - col;
  const T* h = (const T*)a.H + row * a.ldh;
  float g[8], z[8];
  load_run<RUNS>(h, col, a.cols, g);
  load_run<RUNS>(h + a.cols, col, a.cols, z);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float value, slope;
    activation<ACT>(g[i], value, slope);
    z[i] *= value;
    m = max(m, i < valid ? mag(z[i]) : 0u);
  }
  if (a.Z != nullptr) store_run<RUNS>((T*)a.Z + row * a.ldz, col, a.cols, z);
  if (a.Q == nullptr) return;
#pragma unroll
  for (int d = 1; d < 16; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  const float s = scale_of(m);
  store_run<RUNS>(a.Q + row * a.ldq, col, a.cols, quantize8(z, s));
  if (threadIdx.x % 16 == 0) a.S[row * a.s_row + b * a.s_block] = s;
}

// dg = act'(g) u dz and du = act(g) dz: eight neighbours of a row of z per
// thread.
template <class T, int ACT, int RUNS>
__global__ void __launch_bounds__(256) gated_backward_kernel(GatedArgs a) {
  const uint32_t chunks = (uint32_t)(a.cols + 7) / 8;
  const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (uint64_t)chunks * (uint32_t)a.rows) return;
  const uint32_t row = (uint32_t)id / chunks;
  const int col = (int)(8 * ((uint32_t)id - row * chunks));
  const T* h = (const T*)a.H + row * a.ldh;
  float g[8], u[8], dz[8];
  load_run<RUNS>(h, col, a.cols, g);
  load_run<RUNS>(h + a.cols, col, a.cols, u);
  load_run<RUNS>((const T*)a.dZ + row * a.lddz, col, a.cols, dz);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float value, slope;
    activation<ACT>(g[i], value, slope);
    g[i] = slope * u[i] * dz[i];
    u[i] = value * dz[i];
  }
  T* d = (T*)a.dH + row * a.lddh;
  store_run<RUNS>(d, col, a.cols, g);
  store_run<RUNS>(d + a.cols, col, a.cols, u);
}

// dp = act'(p) dc, and its sum over a group's rows. A workgroup has 8*LANES
// columns of one group: LANES threads side by side, 256/LANES rows at a time,
// every groups-th such run of rows; these threads' sums are added in their order.
template <class T, int ACT, int LANES, int RUNS>
__global__ void __launch_bounds__(256) epilogue_backward_kernel(EpilogueBackArgs a) {
  constexpr int ROWS = 256 / LANES;
  __shared__ __align__(16) float part[ROWS][8 * LANES];
  const int lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
  const int strips = (a.cols + 8 * LANES - 1) / (8 * LANES);
  const int group = blockIdx.x / strips;
  const int col = 8 * ((blockIdx.x - group * strips) * LANES + lane);
  float sum[8] = {};
  if (col < a.cols) {
#pragma unroll 4
    for (int64_t row = (int64_t)group * ROWS + team; row < a.rows; row += (int64_t)a.groups * ROWS) {
      float p[8], d[8];
      load_run<RUNS>((const T*)a.P + row * a.ldp, col, a.cols, p);
      load_run<RUNS>((const T*)a.dC + row * a.lddc, col, a.cols, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float value, slope;
        if constexpr (sizeof(T) == 2) slope = slope16<ACT>(p[i]);
        else activation<ACT>(p[i], value, slope);
        d[i] *= slope;
        sum[i] += d[i];
      }
      store_run<RUNS>((T*)a.dP + row * a.lddp, col, a.cols, d);
    }
  }
  if (a.sums == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) part[team][8 * lane + i] = sum[i];
  __syncthreads();
  for (int c = threadIdx.x; c < 8 * LANES; c += 256) {
    const int at = 8 * LANES * (blockIdx.x - group * strips) + c;
    float total = 0.0f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) total += part[r][c];
    if (at < a.cols) a.sums[(int64_t)group * a.cols + at] = total;
  }
}

// out[c] = sum over the groups of P[group][c], in an order that depends on the
// number of groups alone. A workgroup has 64 columns: 16 threads side by side,
// 64 groups at a time, so that few columns have many loads on the way too.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* P, int groups, int cols, float* out) {
  __shared__ __align__(16) float part[64][64];
  const int lane = threadIdx.x % 16, team = threadIdx.x / 16;
  const int col = blockIdx.x * 64 + 4 * lane;
  float sum[4] = {};
  if (col + 4 <= cols) {
#pragma unroll 4
    for (int g = team; g < groups; g += 64) {
      float v[4];
      __builtin_memcpy(v, P + (int64_t)g * cols + col, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += v[i];
    }
  } else {
    for (int g = team; g < groups; g += 64)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < cols) sum[i] += P[(int64_t)g * cols + col + i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[team][4 * lane + i] = sum[i];
  __syncthreads();
  // 16 threads to a column, four groups' teams each, and then these in a wave's order.
  const int c = threadIdx.x / 16, x = threadIdx.x % 16;
  float total = part[4 * x][c];
#pragma unroll
  for (int i = 1; i < 4; ++i) total += part[4 * x + i][c];
#pragma unroll
  for (int d = 1; d < 16; d *= 2) total += __shfl_xor(total, d, 64);
  if (x == 0 && blockIdx.x * 64 + c < cols) out[blockIdx.x * 64 + c] = total;
}

}  // namespace

hipError_t launch_column_sums(const float* sums, int groups, int cols, float* out, hipStream_t s) {
  void* args[] = {&sums, &groups, &cols, &out};
  return hipLaunchKernel((const void*)&column_sums_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024), args, 0, s);
}

hipError_t launch_gated(int type, int act, const GatedArgs& a, hipStream_t s) {
  const int64_t groups = (int64_t)((a.cols + kBlock - 1) / kBlock) * a.rows;
  return by_type(type, [&](auto t) {
    return by_act(act, [&](auto f) {
      constexpr int ACT = decltype(f)::value;
      return launch_with(a.runs == RUNS_WHOLE ? (const void*)&gated_kernel<decltype(t), ACT, RUNS_WHOLE>
                                              : (const void*)&gated_kernel<decltype(t), ACT, RUNS_ANY>,
                         dim3((unsigned)((groups + 15) / 16)), dim3(256), a, s);
    });
  });
}

hipError_t launch_gated_backward(int type, int act, const GatedArgs& a, hipStream_t s) {
  const int64_t chunks = (int64_t)((a.cols + 7) / 8) * a.rows;
  return by_type(type, [&](auto t) {
    return by_act(act, [&](auto f) {
      constexpr int ACT = decltype(f)::value;
      return by_runs(a.runs, [&](auto runs) {
        return launch_with((const void*)&gated_backward_kernel<decltype(t), ACT, decltype(runs)::value>,
                           dim3((unsigned)((chunks + 255) / 256)), dim3(256), a, s);
      });
    });
  });
}

namespace {
constexpr int kNarrow = 128;  // columns up to which sixteen threads share a row
int strips_of(int cols) { return cols <= kNarrow ? 1 : (cols + 511) / 512; }
}  // namespace

void epilogue_groups(int rows, int cols, EpilogueBackArgs& a) {
  const int64_t wanted = 2048 / strips_of(cols) > 1 ? 2048 / strips_of(cols) : 1;
  const int least = cols <= kNarrow ? 64 : 32;  // rows of a group: some for each thread
  const int64_t groups = ((int64_t)rows + least - 1) / least;
  a.groups = (int)(groups < wanted ? groups : wanted);
}

hipError_t launch_epilogue_backward(int type, int act, const EpilogueBackArgs& a, float* dbias, hipStream_t s) {
  const hipError_t e = by_type(type, [&](auto t) {
    return by_act(act, [&](auto f) {
      using T = decltype(t);
      constexpr int ACT = decltype(f)::value;
      const dim3 grid((unsigned)(a.groups * strips_of(a.cols)));
      if (a.cols <= kNarrow) return launch_with((const void*)&epilogue_backward_kernel<T, ACT, 16, RUNS_ANY>, grid, dim3(256), a, s);
      return by_runs(a.runs, [&](auto runs) {
        return launch_with((const void*)&epilogue_backward_kernel<T, ACT, 64, decltype(runs)::value>, grid, dim3(256), a, s);
      });
    });
  });
  if (e != hipSuccess || a.sums == nullptr || a.groups == 1) return e;
  return launch_column_sums(a.sums, a.groups, a.cols, dbias, s);
}

}  // namespace sgemm_impl
