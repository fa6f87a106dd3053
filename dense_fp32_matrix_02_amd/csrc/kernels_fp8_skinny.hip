// FP8 products of few rows of A (a decoding step), of operands that are
// 16-byte aligned in rows of a multiple of 16 bytes.

#include "sgemm_internal.h"
#include "fp8_device.h"

namespace sgemm_impl {
namespace {

constexpr int kSkinnyWaves = 8;

// A workgroup has 16 rows of B and 16*MF of A over the whole of K: its waves
// take every eighth block, straight from memory to registers, and their sums
// are added in wave order through LDS.
template <int FORM, bool WIDE, int MF>
__global__ void __launch_bounds__(64 * kSkinnyWaves) fp8_skinny_kernel(Fp8Args g) {
  constexpr int BM = 16 * MF, BN = 16, NW = kSkinnyWaves;
  constexpr int AHEAD = MF == 1 ? 4 : 2;  // blocks that a wave has in flight
  __shared__ __align__(16) f32x4 part[NW][MF][64];
  Tile t;
  if (!find_tile<FORM, BM, BN>(g, t)) return;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int r16 = lane % 16, quad = lane / 16;
  const int blocks = (t.K + kBlock - 1) / kBlock;
  const uint8_t* b = t.B + (int64_t)min(t.n0 + r16, t.rows_b - 1) * g.ldb;
  const uint8_t* a[MF];
  const float* sa[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int64_t row = min(t.m0 + 16 * i + r16, t.rows_a - 1);
    a[i] = t.A + row * g.lda;
    sa[i] = t.SA + row * g.sa_row;
  }
  const float* sb[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int n = min(t.n0 + 4 * quad + x, t.rows_b - 1);
    sb[x] = t.SB + (int64_t)(g.sb_rows == 1 ? n : n / kBlock) * g.sb_row;
  }
  f32x4 acc[MF] = {};
  const int k0 = 16 * quad;
  auto load = [&](const uint8_t* row, int k) __attribute__((always_inline)) {
    if (k + 16 <= t.K) return *(const i32x4*)(row + k);
    return load16(row, k, t.K);
  };
  for (int first = wave; first < blocks; first += NW * AHEAD) {
    i32x4 rb[AHEAD][2], ra[AHEAD][MF][2];
    float vb[AHEAD][4], va[AHEAD][MF];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int blk = first + u * NW;
      if (blk < blocks) {  // the same for the whole wave
        const int k = blk * kBlock + k0;
        rb[u][0] = load(b, k), rb[u][1] = load(b, k + 64);
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          ra[u][i][0] = load(a[i], k), ra[u][i][1] = load(a[i], k + 64);
          va[u][i] = sa[i][(int64_t)blk * g.sa_block];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) vb[u][x] = sb[x][(int64_t)blk * g.sb_block];
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (first + u * NW >= blocks) break;
      Frag<WIDE> fb, fa;
      fb.set(rb[u][0], rb[u][1]);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        fa.set(ra[u][i][0], ra[u][i][1]);
        const f32x4 p = block_product(fb, fa);
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[i][x] = __builtin_fmaf(p[x], va[u][i] * vb[u][x], acc[i][x]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MF; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave < MF) {
    f32x4 sum = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += part[w][wave][lane];
    const int m = t.m0 + 16 * wave + r16, n = t.n0 + 4 * quad;
    const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    if (m < t.rows_a) store_c(g, t.C, (int64_t)m * g.ldc + n, g.N - n, v);
  }
}

template <int MF>
const void* of_width(Fp8Form form, bool wide) {
  if (form == FP8_EXPERTS)
    return wide ? (const void*)&fp8_skinny_kernel<FP8_EXPERTS, true, MF> : (const void*)&fp8_skinny_kernel<FP8_EXPERTS, false, MF>;
  return wide ? (const void*)&fp8_skinny_kernel<FP8_DENSE, true, MF> : (const void*)&fp8_skinny_kernel<FP8_DENSE, false, MF>;
}

}  // namespace

const void* fp8_skinny_kernel_for(Fp8Form form, bool wide, int bm) {
  return bm == 16 ? of_width<1>(form, wide) : bm == 32 ? of_width<2>(form, wide) : of_width<4>(form, wide);
}

}  // namespace sgemm_impl
