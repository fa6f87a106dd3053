// FP8 (e4m3) products with a scale for each block of 128 values of the summed
// axis:
//   C[m][n] = sum_b sA[m][b] * sB[n][b] * P_b[m][n],  P_b = sum_{k in b} A[m][k]*B[n][k].
//
// Sums are held in FP32. The FP8 matrix unit does not do that: it adds products
// in groups of eight, keeping of each only what lies within 13 bits of the
// group's largest (measured: 16*16 + 2^-6 in one group gives 256; in different
// groups nothing is lost). So the values are widened to bf16, which holds
// every e4m3 number, and multiplied with v_mfma_f32_32x32x16_bf16, whose sums
// measure as FP32 sums. A block's eight such steps start from zero, and one
// fused multiply-add per element by the block's scale adds P_b to the result.
// B's rows are the instruction's rows and A's rows its columns, so that a
// lane's 16 results are one row of C (one m): sA is then one value per lane,
// and a lane's results are four runs of four neighbours in C.

#include "fp8_internal.h"
#include "sgemm_internal.h"

namespace sgemm_impl {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// What one workgroup computes: a tile of one product.
struct Tile {
  const uint8_t *A, *B;  // row 0 of the operands
  const float *SA, *SB;
  int rows_a, rows_b;  // rows that exist
  int m0, n0;          // first row and column of the tile
  int K;
  void* C;  // row 0 of the product's C
};

// Bytes [k, k + 16) of a row of K, zero from K on; any alignment.
__device__ __forceinline__ i32x4 load16(const uint8_t* row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k + i < K) v[i / 4] |= (int)((uint32_t)row[k + i] << (8 * (i % 4)));
  }
  return v;
}

// Position of 16-byte chunk c of row r of a 128-byte-row slab: gfx950 serves
// a 128-bit LDS read 16 lanes at a time from 64 banks, so 16 consecutive rows
// (each starting at bank 0 or 32) have to hold one chunk in different places.
__device__ __forceinline__ int swz(int r, int c) { return c ^ ((r >> 1) & 7); }

// Eight e4m3 bytes as bf16, exactly.
__device__ __forceinline__ bf16x8 widen(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <class T>
__device__ __forceinline__ void store4(T* c, int valid, f32x4 v, float beta) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < valid) c[i] = from_f32<T>(beta != 0.0f ? __builtin_fmaf(beta, to_f32(c[i]), v[i]) : v[i]);
}

// Which tile of which product this workgroup has. False: none.
template <int FORM, int BM, int BN>
__device__ __forceinline__ bool find_tile(const Fp8Args& g, Tile& t) {
  const int tiles_n = (g.N + BN - 1) / BN;
  t.A = g.A, t.B = g.B, t.SA = g.SA, t.SB = g.SB, t.C = g.C;
  t.rows_a = g.M, t.rows_b = g.N, t.K = g.K;
  if constexpr (FORM == FP8_EXPERTS) {
    // Tiles are numbered expert by expert; the wave counts 64 experts at a time.
    const int lane = threadIdx.x % 64;
    const int tm = blockIdx.x / tiles_n;
    t.n0 = (blockIdx.x - tm * tiles_n) * BN;
    int before = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 64) {
      int begin = 0, end = 0;
      if (e0 + lane < g.experts) expert_rows(g.offsets, e0 + lane, g.M, begin, end);
      const int own = (end - begin + BM - 1) / BM;
      int upto = own;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int x = __shfl_up(upto, d, 64);
        if (lane >= d) upto += x;
      }
      const uint64_t past = __ballot(tm < before + upto);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        const int e = e0 + l;
        t.m0 = __shfl(begin, l, 64) + (tm - before - __shfl(upto - own, l, 64)) * BM;
        t.rows_a = __shfl(end, l, 64);
        t.B = g.B + (int64_t)e * g.strideB;
        t.SB = g.SB + (int64_t)e * g.stride_sb;
        return true;
      }
      before += __shfl(upto, 63, 64);
    }
    // Rows no expert has: a product over nothing.
    int begin, end;
    expert_rows(g.offsets, g.experts - 1, g.M, begin, end);
    t.m0 = end + (tm - before) * BM;
    t.K = 0;
    return t.m0 < g.M;
  } else {
    const int tiles_m = (g.M + BM - 1) / BM;
    const int tm = blockIdx.x % tiles_m;
    t.m0 = tm * BM;
    t.n0 = (blockIdx.x / tiles_m) * BN;
    if constexpr (FORM == FP8_WGRAD) {
      const int e = blockIdx.y;
      int begin, end;
      expert_rows(g.offsets, e, g.K, begin, end);
      const int64_t slot = begin / kBlock + e;
      t.K = end - begin;
      t.A += slot * kBlock, t.B += slot * kBlock;
      t.SA += slot * g.sa_block, t.SB += slot * g.sb_block;
      const int64_t size = g.type == SGEMM_MI355_F32 ? 4 : 2;
      t.C = (char*)g.C + (int64_t)e * g.strideC * size;
    }
    return true;
  }
}

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
        const f32x4 v = {acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
        const int64_t at = (int64_t)m * g.ldc + n;
        if (g.type == SGEMM_MI355_F32) store4((float*)t.C + at, g.N - n, v, g.beta);
        else if (g.type == SGEMM_MI355_BF16) store4((__hip_bfloat16*)t.C + at, g.N - n, v, g.beta);
        else store4((__half*)t.C + at, g.N - n, v, g.beta);
      }
  }
}

}  // namespace

namespace {
// The grid of BM x BN tiles: in the experts' form each expert's last tile of
// rows may be short, and the rest's.
int64_t grid_tiles(Fp8Form form, const Fp8Args& g, int bm, int bn) {
  const int64_t tiles_n = (g.N + bn - 1) / bn;
  return tiles_n * (form == FP8_EXPERTS ? (int64_t)g.M / bm + g.experts + 1 : (int64_t)((g.M + bm - 1) / bm));
}
}  // namespace

bool fp8_launchable(Fp8Form form, const Fp8Args& g) {
  return grid_tiles(form, g, 128, 128) * 256 <= (int64_t)UINT32_MAX && (form != FP8_WGRAD || g.experts <= kMaxGridY);
}

hipError_t launch_fp8_gemm(Fp8Form form, const Fp8Args& g, hipStream_t s) {
  const void* kernel = form == FP8_EXPERTS ? (const void*)&fp8_gemm_kernel<FP8_EXPERTS>
                       : form == FP8_WGRAD ? (const void*)&fp8_gemm_kernel<FP8_WGRAD>
                                           : (const void*)&fp8_gemm_kernel<FP8_DENSE>;
  return launch_with(kernel, dim3((unsigned)grid_tiles(form, g, 128, 128), form == FP8_WGRAD ? (unsigned)g.experts : 1u),
                     dim3(256), g, s);
}

}  // namespace sgemm_impl
