// Quantisers to e4m3 with a scale for each block of 128 values: along rows,
// down columns (stored transposed), and for 128 x 128 tiles.
//
// For a block with largest magnitude m: s = max(m, 2^-64) / 448 and
// q = e4m3(x / s), the quotient rounded to FP32 first. All three are one pass
// over X, bound by its bytes (4 or 2 read and 1 written per value): a block's
// values stay in registers between the search for the largest and the
// rounding.

#include "fp8_internal.h"

namespace sgemm_impl {
namespace {

constexpr float kTop = 448.0f;
constexpr float kLeast = 0x1p-64f;

// The magnitude's bits order like the magnitudes, with infinities and then
// NaNs above all numbers, so their integer maximum keeps a NaN.
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The scale of a block whose largest magnitude has these bits; NaN where the
// block holds a NaN or an infinity.
__device__ __forceinline__ float scale_of(uint32_t most) {
  if (most >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  return fmaxf(__uint_as_float(most), kLeast) / kTop;
}

// x / s rounded to FP32, for r = 1 / s rounded: two residual corrections of
// the product x*r. The first brings it within one unit in the last place; the
// second, with r correctly rounded, rounds it correctly (Markstein). With
// s >= 2^-64/448 and |x| <= 448 s no residual that could matter to a quotient
// of 2^-10 or more (the rest round to zero) leaves FP32's range.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  float q = x * r;
  q = __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
  return __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
}

// Eight values as e4m3, value i in byte i.
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float s) {
  const float r = 1.0f / s;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], s, r);
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return uint2{(uint32_t)lo, (uint32_t)hi};
}

template <bool ONCE = false>
__device__ __forceinline__ void store_bytes(uint8_t* p, uint2 b, int valid) {
  typedef uint32_t words __attribute__((ext_vector_type(2), aligned(1)));
  if (valid >= 8) {
    const words w = {b.x, b.y};
    if constexpr (ONCE) __builtin_nontemporal_store(w, (words*)p);
    else *(words*)p = w;
  } else {
    const uint64_t w = ((uint64_t)b.y << 32) | b.x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = (uint8_t)(w >> (8 * i));
  }
}

// The row of X that row i of the quantised matrix is; -1 (zeros) for an index
// outside X.
__device__ __forceinline__ int source_row(const QuantArgs& a, int i) {
  const int r = a.index ? a.index[i] : i;
  return (unsigned)r < (unsigned)a.rows ? r : -1;
}

// Rows. Sixteen lanes hold one block of a row, eight values each; a wave has
// four consecutive blocks of its row, so it reads 1 or 2 KiB at a stretch.
template <class T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantArgs a) {
  const int blocks = (a.cols + kBlock - 1) / kBlock;
  const int64_t group = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
  const int lane = threadIdx.x % 16;
  if (group >= (int64_t)blocks * a.n) return;  // the same for all 16 lanes of a block
  const int row = (int)(group / blocks), b = (int)(group - (int64_t)row * blocks);
  const int src = source_row(a, row);
  const int col = b * kBlock + 8 * lane;
  const int valid = a.cols - col;
  float v[8];
  load8((const T*)a.X + (int64_t)(src < 0 ? 0 : src) * a.ldx + col, src < 0 ? 0 : valid, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag(v[i]));
#pragma unroll
  for (int d = 1; d < 16; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  const float s = scale_of(m);
  store_bytes(a.Q + (int64_t)row * a.ldq + col, quantize8(v, s), valid);
  if (lane == 0) a.S[(int64_t)row * a.s_row + (int64_t)b * a.s_block] = s;
}

// Tiles. 256 threads hold a 128 x 128 tile, eight columns of eight rows each
// (thread t: columns 8*(t%16) on, rows t/16 + 16*i).
template <class T>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(QuantArgs a) {
  __shared__ uint32_t most[4];
  const int blocks = (a.cols + kBlock - 1) / kBlock;
  const int tr = blockIdx.x / blocks, tc = blockIdx.x - tr * blocks;
  const int t = threadIdx.x;
  const int col = tc * kBlock + 8 * (t % 16);
  const int valid = a.cols - col;
  const int row0 = tr * kBlock + t / 16;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    load8((const T*)a.X + (int64_t)(row < a.rows ? row : 0) * a.ldx + col, row < a.rows ? valid : 0, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, mag(v[i][j]));
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  if (t % 64 == 0) most[t / 64] = m;
  __syncthreads();
  m = max(max(most[0], most[1]), max(most[2], most[3]));
  const float s = scale_of(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    if (row < a.rows) store_bytes(a.Q + (int64_t)row * a.ldq + col, quantize8(v[i], s), valid);
  }
  if (t == 0) a.S[(int64_t)tr * a.s_row + (int64_t)tc * a.s_block] = s;
}

// The rows that fill block slot b of the columns form, [begin, end).
__device__ __forceinline__ void slot_rows(const QuantArgs& a, int slot, int& begin, int& end) {
  if (a.offsets == nullptr) {
    begin = slot * kBlock;
    end = min(begin + kBlock, a.n);
    return;
  }
  // The last expert whose first slot, begin/128 + e, is not after this one.
  int lo = 0, hi = a.experts - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    int b, e;
    expert_rows(a.offsets, mid, a.n, b, e);
    if (b / kBlock + mid <= slot) lo = mid;
    else hi = mid - 1;
  }
  int b, e;
  expert_rows(a.offsets, lo, a.n, b, e);
  const int64_t first = b + (int64_t)(slot - (b / kBlock + lo)) * kBlock;
  begin = first < e ? (int)first : e;
  end = min(begin + kBlock, e);
}

// Columns. 256 threads hold 128 rows by 128 columns, eight columns of eight
// consecutive rows each (thread t: columns 8*(t%16) on, rows 8*(t/16) on), so
// each of a thread's columns is eight bytes of a row of Q. The transposed
// tile goes through LDS, from where a wave writes whole rows' 128 bytes. X and Q
// go past the caches: 8192 x 4096 FP32 takes 39 us (4.3 TB/s), 46 with ordinary
// loads and stores.
template <class T>
__global__ void __launch_bounds__(256) quantize_cols_kernel(QuantArgs a, int slots) {
  constexpr int kPitch = kBlock + 16;
  __shared__ uint32_t most[4][kBlock];
  __shared__ __align__(16) uint8_t tile[kBlock * kPitch];
  const int slot = blockIdx.x % slots, c0 = (blockIdx.x / slots) * kBlock;
  const int t = threadIdx.x;
  int begin, end;
  slot_rows(a, slot, begin, end);
  const int col = c0 + 8 * (t % 16);
  const int valid = a.cols - col;
  const int row0 = begin + 8 * (t / 16);
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int src = row0 + i < end ? source_row(a, row0 + i) : -1;
    load8_once((const T*)a.X + (int64_t)(src < 0 ? 0 : src) * a.ldx + col, src < 0 ? 0 : valid, v[i]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, mag(v[i][j]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    if (t % 64 < 16) most[t / 64][8 * (t % 16) + j] = m;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = 8 * (t % 16) + j;
    const float s = scale_of(max(max(most[0][c], most[1][c]), max(most[2][c], most[3][c])));
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i][j];
    *(uint2*)(tile + c * kPitch + 8 * (t / 16)) = quantize8(w, s);
    if (t < 16 && c0 + c < a.cols) a.S[(int64_t)(c0 + c) * a.s_row + (int64_t)slot * a.s_block] = s;
  }
  __syncthreads();
  const int64_t width = a.offsets ? (int64_t)slots * kBlock : a.n;  // columns of Q
  const int64_t at = (int64_t)slot * kBlock + 8 * (t % 16);
  const int room = (int)(width - at < 8 ? width - at : 8);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = t / 16 + 16 * i;
    if (c0 + c < a.cols)
      store_bytes<true>(a.Q + (int64_t)(c0 + c) * a.ldq + at, *(const uint2*)(tile + c * kPitch + 8 * (t % 16)), room);
  }
}

}  // namespace

hipError_t launch_quantize_rows(int type, const QuantArgs& q, hipStream_t s) {
  const int64_t groups = (int64_t)((q.cols + kBlock - 1) / kBlock) * q.n;
  return by_type(type, [&](auto t) {
    return launch_with((const void*)&quantize_rows_kernel<decltype(t)>, dim3((unsigned)((groups + 15) / 16)),
                       dim3(256), q, s);
  });
}

hipError_t launch_quantize_tiles(int type, const QuantArgs& q, hipStream_t s) {
  const int64_t tiles = (int64_t)((q.rows + kBlock - 1) / kBlock) * ((q.cols + kBlock - 1) / kBlock);
  return by_type(type, [&](auto t) {
    return launch_with((const void*)&quantize_tiles_kernel<decltype(t)>, dim3((unsigned)tiles), dim3(256), q, s);
  });
}

hipError_t launch_quantize_cols(int type, const QuantArgs& q, hipStream_t s) {
  int slots = q.offsets ? q.n / kBlock + q.experts : (q.n + kBlock - 1) / kBlock;
  const int64_t grid = (int64_t)slots * ((q.cols + kBlock - 1) / kBlock);
  return by_type(type, [&](auto t) {
    QuantArgs copy = q;
    void* args[] = {&copy, &slots};
    return hipLaunchKernel((const void*)&quantize_cols_kernel<decltype(t)>, dim3((unsigned)grid), dim3(256), args, 0, s);
  });
}

}  // namespace sgemm_impl
