// FP8 products of few rows of A (a decoding step), of operands that are
// 16-byte aligned in rows of a multiple of 16 bytes; K is 16 or more.

#include <type_traits>

#include "sgemm_internal.h"
#include "fp8_device.h"

namespace sgemm_impl {
namespace {

constexpr int kSkinnyWaves = 8;

// A workgroup has 16 rows of B and 16*MF of A over the whole of K: its waves
// take every eighth block, straight from memory to registers, and their sums
// are added in wave order through LDS. Bound by B's bytes as long as enough
// workgroups share a CU: the loads of one then fill the pauses of another (its
// start, its sums' way through LDS). 16 tokens of 4 of 32 experts, N 2048, K
// 4096: 45 us (5.2 TB/s) with six waves a SIMD and two blocks of each in
// flight, 51 with four and four. Values are widened whatever C's type: the
// matrix unit waits for memory here, and FP32 block sums cost 45.3 us against
// 44.0 with the FP8 unit's (8 x 4096 x 4096: 5.4 and 5.2; 64 rows: 12.7 and 11.9).
template <int FORM, bool TALL, int MF>
__global__ void __launch_bounds__(64 * kSkinnyWaves, MF == 4 ? 2 : MF == 1 ? 6 : 4) fp8_skinny_kernel(Fp8Args g) {
  constexpr int BM = 16 * MF, BN = 16, NW = kSkinnyWaves;
  constexpr int AHEAD = 2;  // blocks that a wave has in flight
  __shared__ __align__(16) f32x4 part[NW][MF][64];
  Tile t;
  if (!find_tile<FORM, BM, BN>(g, t)) return;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int r16 = lane % 16, quad = lane / 16;
  const uint8_t* b = t.B + (int64_t)min(t.n0 + r16, t.rows_b - 1) * g.ldb;
  const uint8_t* a[MF];
  const float* sa[MF];
  bool there[MF];  // rows that do not exist cost no loads
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    there[i] = t.m0 + 16 * i + r16 < t.rows_a;
    const int64_t row = there[i] ? t.m0 + 16 * i + r16 : t.m0;
    a[i] = t.A + row * g.lda;
    sa[i] = t.SA + row * g.sa_row;
  }
  // TALL: one scale for all 16 rows of B; else a lane loads that of row r16.
  const float* sb = t.SB + (int64_t)(TALL ? t.n0 / kBlock : min(t.n0 + r16, t.rows_b - 1)) * g.sb_row;
  f32x4 acc[MF] = {};
  // What a lane holds of block blk; `whole`: no byte of it lies past K.
  struct Held {
    i32x4 b[2], a[MF][2];
    float sb, sa[MF];
  };
  auto fetch = [&](Held& h, int blk, auto whole) __attribute__((always_inline)) {
    const int k = blk * kBlock + 16 * quad;
    auto chunk = [&](const uint8_t* row, int at) __attribute__((always_inline)) {
      if constexpr (decltype(whole)::value) return *(const i32x4*)(row + at);
      else return load16_end(row, at, t.K);
    };
    h.b[0] = chunk(b, k), h.b[1] = chunk(b, k + 64);
    h.sb = sb[(int64_t)blk * g.sb_block];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      h.a[i][0] = h.a[i][1] = i32x4{0, 0, 0, 0};
      h.sa[i] = 0.0f;
      if (there[i]) {
        h.a[i][0] = chunk(a[i], k), h.a[i][1] = chunk(a[i], k + 64);
        h.sa[i] = sa[i][(int64_t)blk * g.sa_block];
      }
    }
  };
  auto multiply = [&](const Held& h) __attribute__((always_inline)) {
    Frag<true> fb, fa;
    fb.set(h.b[0], h.b[1]);
    f32x4 rows_sb;  // of the four rows of B that a lane has results of
#pragma unroll
    for (int x = 0; x < 4; ++x) rows_sb[x] = TALL ? h.sb : __shfl(h.sb, 4 * quad + x, 64);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      fa.set(h.a[i][0], h.a[i][1]);
      const f32x4 p = block_product(fb, fa);
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[i][x] = __builtin_fmaf(p[x], h.sa[i] * rows_sb[x], acc[i][x]);
    }
  };
  const int full = t.K / kBlock;
  int blk = wave;
  for (; blk + (AHEAD - 1) * NW < full; blk += NW * AHEAD) {
    Held h[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) fetch(h[u], blk + u * NW, std::true_type{});
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) multiply(h[u]);
  }
#pragma unroll 1
  for (; blk < full; blk += NW) {
    Held h;
    fetch(h, blk, std::true_type{});
    multiply(h);
  }
  if (blk == full && t.K % kBlock != 0) {  // the wave whose turn the partial block is
    Held h;
    fetch(h, blk, std::false_type{});
    multiply(h);
  }
#pragma unroll
  for (int i = 0; i < MF; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave < MF) {
    f32x4 sum = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += part[w][wave][lane];
    const int m = t.m0 + 16 * wave + r16, n = t.n0 + 4 * quad;
    float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    if (m >= t.rows_a) return;
    if constexpr (FORM == FP8_EPILOGUE) finish_c(g, m, n, v);
    else store_c(g, t.C, (int64_t)m * g.ldc + n, g.N - n, v);
  }
}

template <int MF>
const void* of_width(Fp8Form form, bool tall) {
  if (form == FP8_EXPERTS)
    return tall ? (const void*)&fp8_skinny_kernel<FP8_EXPERTS, true, MF> : (const void*)&fp8_skinny_kernel<FP8_EXPERTS, false, MF>;
  if (form == FP8_EPILOGUE)
    return tall ? (const void*)&fp8_skinny_kernel<FP8_EPILOGUE, true, MF> : (const void*)&fp8_skinny_kernel<FP8_EPILOGUE, false, MF>;
  return tall ? (const void*)&fp8_skinny_kernel<FP8_DENSE, true, MF> : (const void*)&fp8_skinny_kernel<FP8_DENSE, false, MF>;
}

}  // namespace

const void* fp8_skinny_kernel_for(Fp8Form form, bool tall, int bm) {
  return bm == 16 ? of_width<1>(form, tall) : bm == 32 ? of_width<2>(form, tall) : of_width<4>(form, tall);
}

}  // namespace sgemm_impl
