// FP8 (e4m3) products with a scale for each block of 128 values of the summed
// axis:
//   C[m][n] = sum_b sA[m][b] * sB[n][b] * P_b[m][n],  P_b = sum_{k in b} A[m][k]*B[n][k].
//
// Two ways to a block's sum:
// * The FP8 matrix unit (v_mfma_f32_16x16x128_f8f6f4) has twice the rate of
//   bf16, but adds products in groups of eight in fixed point, dropping of
//   each what lies more than 13 bits below the group's largest (measured:
//   2^15 + 2^2 in one group is exact, 2^15 + 2^1 gives 2^15; group sums and
//   the accumulator add up as FP32). On quantised normal data that is 2e-5 of
//   the result, a hundredth of the rounding to bf16 and a tenth of fp16's. It
//   is used where the matrix unit's rate is what a product waits for, C has 16
//   bits and the caller has not asked for FP32 sums: in the tiles (8192^3: 421
//   us, 867 with FP32 sums; 4096 tokens of 4 of 32 experts, N 2048, K 4096: 173
//   and 286).
// * Otherwise values are widened to bf16, which holds every e4m3 number, and
//   multiplied with bf16 matrix instructions, whose sums measure as FP32 sums.
// Either starts a block from zero, and one fused multiply-add per element by
// the block's scale adds P_b to the result in FP32.
// B's rows are the instruction's rows and A's rows its columns, so that a
// lane's 16 results are one row of C (one m): sA is then one value per lane,
// and a lane's results are four runs of four neighbours in C.

#include <cmath>

#include "sgemm_internal.h"
#include "fp8_device.h"

namespace sgemm_impl {
namespace {

// A 128 x 128 tile by four waves of 64 x 64, slabs of one block staged through
// registers: operands of any alignment.
template <int FORM>
__global__ void __launch_bounds__(256) fp8_gemm_kernel(Fp8Args g) {
  constexpr int BM = 128, BN = 128, FM = 2, FN = 2;
  __shared__ __align__(16) uint8_t lds[2][128 * kBlock];
  __shared__ __align__(16) float scale[2][128];
  Tile t;
  if (!find_tile<FORM, BM, BN>(g, t)) return;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int l32 = lane % 32, h = lane / 32;
  const int wm = (wave % 2) * 64, wn = (wave / 2) * 64;
  f32x16 acc[FN][FM] = {};
  const int blocks = (t.K + kBlock - 1) / kBlock;
  for (int b = 0; b < blocks; ++b) {
    i32x4 ra[4], rb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int chunk = i * 256 + tid, r = chunk / 8, k = b * kBlock + 16 * (chunk % 8);
      ra[i] = load16(t.A + (int64_t)(t.m0 + r) * g.lda, k, t.m0 + r < t.rows_a ? t.K : 0);
      rb[i] = load16(t.B + (int64_t)(t.n0 + r) * g.ldb, k, t.n0 + r < t.rows_b ? t.K : 0);
    }
    float s = 0.0f;
    if (tid < 128) {
      const int r = t.m0 + tid;
      if (r < t.rows_a) s = t.SA[(int64_t)r * g.sa_row + (int64_t)b * g.sa_block];
    } else {
      const int r = t.n0 + tid - 128;
      if (r < t.rows_b) s = t.SB[(int64_t)(g.sb_rows == 1 ? r : r / 128) * g.sb_row + (int64_t)b * g.sb_block];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int chunk = i * 256 + tid, r = chunk / 8;
      const int at = r * kBlock + 16 * swz(r, chunk % 8);
      *(i32x4*)(lds[0] + at) = ra[i];
      *(i32x4*)(lds[1] + at) = rb[i];
    }
    scale[tid / 128][tid % 128] = s;
    __syncthreads();
    f32x16 p[FN][FM] = {};
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      bf16x8 fa[FM][2], fb[FN][2];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = wm + 32 * i + l32;
        const i32x4 v = *(const i32x4*)(lds[0] + r * kBlock + 16 * swz(r, 2 * kk + h));
        fa[i][0] = widen(v[0], v[1]), fa[i][1] = widen(v[2], v[3]);
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int r = wn + 32 * j + l32;
        const i32x4 v = *(const i32x4*)(lds[1] + r * kBlock + 16 * swz(r, 2 * kk + h));
        fb[j][0] = widen(v[0], v[1]), fb[j][1] = widen(v[2], v[3]);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int i = 0; i < FM; ++i) p[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j][x], fa[i][x], p[j][i], 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const float sa = scale[0][wm + 32 * i + l32];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 sb = *(const f32x4*)&scale[1][wn + 32 * j + 8 * q + 4 * h];
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[j][i][4 * q + x] = __builtin_fmaf(p[j][i][4 * q + x], sa * sb[x], acc[j][i][4 * q + x]);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = t.m0 + wm + 32 * i + l32;
    if (m >= t.rows_a) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = t.n0 + wn + 32 * j + 8 * q + 4 * h;
        const float v[4] = {acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
        store_c(g, t.C, (int64_t)m * g.ldc + n, g.N - n, v);
      }
  }
}

}  // namespace

namespace {

// The kernel for a call and its tile.
struct Choice {
  enum Kernel { STAGED, TILE, SKINNY } kernel;
  bool wide;  // values are widened to bf16
  int bm, bn, threads;
};

Choice choose(Fp8Form form, const Fp8Args& g) {
  const bool direct = (((uintptr_t)g.A | (uintptr_t)g.B | (uint64_t)g.lda | (uint64_t)g.ldb | (uint64_t)g.strideB) & 15) == 0 &&
                      g.lda < 1 << 23 && g.ldb < 1 << 23 &&  // offsets within a tile fit 31 bits
                      (form == FP8_WGRAD || g.K >= 16);
  if (!direct) return {Choice::STAGED, true, 128, 128, 256};
  const bool wide = g.wide;
  // The least of the estimated times (us; r: rounds of 256 workgroups, one for
  // each CU; k: K/1024), fitted to times of M 8 .. 2048, N 256 .. 4096, K 256 ..
  // 8192 and 8192^3, as K 2048, N 4096, bf16, M 128 / 512 / 2048:
  //   few-rows kernel, 16, 32, 64 rows   20.5, 15.7, 15.4 / 66, 50, 56 / 237, 182, 211
  //   128 x 128 tiles, 256 x 256 tiles   11.8, 17.4 / 12.7, 25.3 / 23.1, 29.0
  // Widened values need more registers than the strip of a wave of a 256 x 256
  // tile leaves, so that form has smaller tiles only (24.4 us at M 512, fp32).
  const double k = g.K / 1024.0 / (form == FP8_WGRAD ? g.experts : 1);
  auto groups = [&](int bm, int bn) {
    // An expert with rows has one tile of rows, and half a tile more on average
    // where it has many.
    const int64_t used = g.experts < g.M ? g.experts : g.M, whole = (g.M + bm - 1) / bm;
    const int64_t tiles_m = form == FP8_EXPERTS ? (whole + used / 2 > used ? whole + used / 2 : used) : whole;
    return (double)((form == FP8_WGRAD ? g.experts : 1) * tiles_m * ((g.N + bn - 1) / bn)) / 256.0;
  };
  const double tail = g.K % kBlock != 0 ? 2.0 : 0.0;  // of the tiles: the partial block is not overlapped
  Choice best{};
  double least = 0.0;
  auto offer = [&](Choice c, double time) {
    if (best.threads == 0 || time < least) best = c, least = time;
  };
  // Experts' tiles with few rows wait for the weights: at 5 TB/s, and the tiled
  // kernels 1.25 times that. The few-rows kernel loads no rows that do not
  // exist (16 tokens of 4 of 32 experts, N 2048, K 4096, weights not in a
  // cache: 43.5 us in 16-row tiles, 54 in 128 x 128, 57 in 256 x 256; 128
  // tokens 89, 68, 69).
  const bool experts = form == FP8_EXPERTS;
  const double weights = experts ? 1.25 * (g.experts < g.M ? g.experts : g.M) * g.N * (double)g.K / 5.0e6 : 0.0;
  const double r = std::ceil(groups(128, 128));
  offer({Choice::TILE, wide, 128, 128, 256},
        std::fmax(weights, (wide ? 2.5 + r * (4.0 + 8.4 * k) : 1.0 + r * (3.3 + 4.2 * k)) + tail));
  // Widened values take 192 x 128 tiles where these fit one round and 128 x 128
  // tiles do not, so that some CUs would work on two (N 4096, K 2048, fp32: M
  // 1536 33.3 us against 37.6; else they are slower: M 768 30.2 against 26.4,
  // M 2304 56.8 against 55.3).
  if (wide && form == FP8_DENSE && groups(192, 128) <= 1.0) offer({Choice::TILE, wide, 192, 128, 512}, 8.0 + 12.6 * k + tail);
  if (!wide) {
    const double r = groups(256, 256);
    offer({Choice::TILE, wide, 256, 256, 512},
          std::fmax(weights, 2.5 + std::ceil(r) * (4.0 + (8.75 + 4.5 * (r < 1.0 ? r : 1.0)) * k) + tail));
  }
  if (form != FP8_WGRAD) {
    auto rounds = [&](int bm) { return groups(bm, 16) > 1.0 ? groups(bm, 16) : 1.0; };
    // A CU holds one workgroup of 64 rows at a time (N 2048, K 4096, M 192: 25.1 us
    // in its two rounds, 19.2 in 128 x 128 tiles).
    offer({Choice::SKINNY, true, 64, 16, 512},
          2.4 + (experts ? rounds(64) * (1.3 + 1.2 * k) : std::ceil(rounds(64)) * (1.3 + 2.5 * k)));
    offer({Choice::SKINNY, true, 32, 16, 512}, 2.6 + rounds(32) * (0.8 + (experts ? 0.9 : 1.41) * k));
    offer({Choice::SKINNY, true, 16, 16, 512}, 2.6 + rounds(16) * (experts ? 0.6 + 0.74 * k : 0.8 + 0.98 * k));
  }
  return best;
}

}  // namespace

bool fp8_launchable(Fp8Form form, const Fp8Args& g) {
  const Choice c = choose(form, g);
  return grid_tiles(form, g, c.bm, c.bn) * c.threads <= (int64_t)UINT32_MAX && (form != FP8_WGRAD || g.experts <= kMaxGridY);
}

const char* fp8_kernel_name(Fp8Form form, const Fp8Args& g) {
  const Choice c = choose(form, g);
  if (c.kernel == Choice::STAGED) return "staged_128x128_bf16";
  if (c.kernel == Choice::TILE)
    return c.bm == 256 ? "tile_256x256_fp8" : c.bm == 192 ? "tile_192x128_bf16" : c.wide ? "tile_128x128_bf16" : "tile_128x128_fp8";
  return c.bm == 64 ? "rows_64_bf16" : c.bm == 32 ? "rows_32_bf16" : "rows_16_bf16";
}

hipError_t launch_fp8_gemm(Fp8Form form, const Fp8Args& g, hipStream_t s) {
  const Choice c = choose(form, g);
  const dim3 grid((unsigned)grid_tiles(form, g, c.bm, c.bn), form == FP8_WGRAD ? (unsigned)g.experts : 1u);
  const void* kernel = c.kernel == Choice::TILE     ? fp8_tile_kernel_for(form, c.wide, g.sb_rows == kBlock, c.bm)
                       : c.kernel == Choice::SKINNY ? fp8_skinny_kernel_for(form, g.sb_rows == kBlock, c.bm)
                       : form == FP8_EXPERTS        ? (const void*)&fp8_gemm_kernel<FP8_EXPERTS>
                       : form == FP8_WGRAD          ? (const void*)&fp8_gemm_kernel<FP8_WGRAD>
                                                    : (const void*)&fp8_gemm_kernel<FP8_DENSE>;
  return launch_with(kernel, grid, dim3((unsigned)c.threads), g, s);
}

}  // namespace sgemm_impl
