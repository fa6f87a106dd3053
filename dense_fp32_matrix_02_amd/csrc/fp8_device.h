// Device code shared by the FP8 product kernels.
#pragma once

#include "fp8_internal.h"

namespace sgemm_impl {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(1))) void global_void;
typedef __attribute__((address_space(3))) void lds_void;

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

// The same for K >= 16, in one load: of the 16 bytes at k or, where they would
// pass K, of the row's last 16, shifted to their places.
__device__ __forceinline__ i32x4 load16_end(const uint8_t* row, int k, int K) {
  const int at = min(k, K - 16), skip = k - at;
  uint64_t v[2];
  __builtin_memcpy(v, row + at, 16);
  if (skip >= 8) v[0] = v[1], v[1] = 0;
  const int bits = 8 * (skip % 8);
  if (bits > 0) v[0] = v[0] >> bits | v[1] << (64 - bits), v[1] >>= bits;
  if (skip >= 16) v[0] = 0;
  i32x4 r;
  __builtin_memcpy(&r, v, 16);
  return r;
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

// A row's 128 values of one block as a lane of a 16-row fragment holds them:
// 32 of them (those of chunks g and g + 4, g = lane / 16; any split will do
// where both operands use the same), as e4m3 or widened to bf16.
template <bool WIDE>
struct Frag;
template <>
struct Frag<false> {
  i32x8 v;
  __device__ __forceinline__ void set(i32x4 a, i32x4 b) { v = i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }
};
template <>
struct Frag<true> {
  bf16x8 v[4];
  __device__ __forceinline__ void set(i32x4 a, i32x4 b) {
    v[0] = widen(a[0], a[1]), v[1] = widen(a[2], a[3]), v[2] = widen(b[0], b[1]), v[3] = widen(b[2], b[3]);
  }
};

// Step x of STEPS of the 16 x 16 products of two fragments over a block: rows
// of the result are b's rows, columns a's; lane l holds rows 4*(l/16) .. +3 of
// column l%16. Step 0 begins from zero.
template <bool WIDE>
constexpr int kSteps = WIDE ? 4 : 1;
__device__ __forceinline__ f32x4 block_step(const Frag<false>& b, const Frag<false>& a, int, f32x4) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_step(const Frag<true>& b, const Frag<true>& a, int x, f32x4 p) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[x], a.v[x], x == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : p, 0, 0, 0);
}
template <bool WIDE>
__device__ __forceinline__ f32x4 block_product(const Frag<WIDE>& b, const Frag<WIDE>& a) {
  f32x4 p = {};
#pragma unroll
  for (int x = 0; x < kSteps<WIDE>; ++x) p = block_step(b, a, x, p);
  return p;
}

// `valid` of W neighbours of C at element `at`.
template <class T, int W>
__device__ __forceinline__ void store_as(T* c, int valid, const float (&v)[W], float beta) {
  if (valid >= W && beta == 0.0f) {
    T e[W];
#pragma unroll
    for (int i = 0; i < W; ++i) e[i] = from_f32<T>(v[i]);
    __builtin_memcpy(c, e, sizeof(e));
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i < valid) c[i] = from_f32<T>(beta != 0.0f ? __builtin_fmaf(beta, to_f32(c[i]), v[i]) : v[i]);
}
template <int W>
__device__ __forceinline__ void store_c(const Fp8Args& g, void* C, int64_t at, int valid, const float (&v)[W]) {
  if (g.type == SGEMM_MI355_F32) store_as((float*)C + at, valid, v, g.beta);
  else if (g.type == SGEMM_MI355_BF16) store_as((__hip_bfloat16*)C + at, valid, v, g.beta);
  else store_as((__half*)C + at, valid, v, g.beta);
}

// The experts' tiles of BM rows, numbered expert by expert and then those of
// the rows that no expert has. The wave counts 64 experts at a time.
template <int BM>
__device__ __forceinline__ int expert_tiles(const Fp8Args& g, int e0, int lane, int& begin, int& end, int& upto) {
  begin = 0, end = 0;
  if (e0 + lane < g.experts) expert_rows(g.offsets, e0 + lane, g.M, begin, end);
  const int own = (end - begin + BM - 1) / BM;
  upto = own;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int x = __shfl_up(upto, d, 64);
    if (lane >= d) upto += x;
  }
  return own;
}

// Which tile of which product this workgroup has. False: none.
// Workgroups go round the eight XCDs; each XCD gets a run of neighbouring
// tiles, so that its L2 serves the rows they share.
template <int FORM, int BM, int BN>
__device__ __forceinline__ bool find_tile(const Fp8Args& g, Tile& t) {
  const int tiles_n = (g.N + BN - 1) / BN;
  t.A = g.A, t.B = g.B, t.SA = g.SA, t.SB = g.SB, t.C = g.C;
  t.rows_a = g.M, t.rows_b = g.N, t.K = g.K;
  if constexpr (FORM == FP8_EXPERTS) {
    const int lane = threadIdx.x % 64;
    int begin, end, upto;
    int total = 0, last_end = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 64) {
      expert_tiles<BM>(g, e0, lane, begin, end, upto);
      total += __builtin_amdgcn_readlane(upto, 63);
      last_end = __builtin_amdgcn_readlane(end, min(63, g.experts - 1 - e0));
    }
    total += (g.M - last_end + BM - 1) / BM;
    const int64_t tiles = (int64_t)total * tiles_n;
    if (blockIdx.x >= tiles) return false;
    const int64_t each = tiles / 8, more = tiles % 8, xcd = blockIdx.x % 8;
    const int64_t id = xcd * each + (xcd < more ? xcd : more) + blockIdx.x / 8;
    const int tm = (int)(id / tiles_n);
    t.n0 = (int)(id - (int64_t)tm * tiles_n) * BN;
    int before = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 64) {
      const int own = expert_tiles<BM>(g, e0, lane, begin, end, upto);
      const uint64_t past = __ballot(tm < before + upto);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        const int e = e0 + l;
        // The same in every lane: kept in scalar registers.
        t.m0 = __builtin_amdgcn_readlane(begin, l) + (tm - before - __builtin_amdgcn_readlane(upto - own, l)) * BM;
        t.rows_a = __builtin_amdgcn_readlane(end, l);
        t.B = g.B + (int64_t)e * g.strideB;
        t.SB = g.SB + (int64_t)e * g.stride_sb;
        return true;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
    }
    // Rows no expert has: a product over nothing.
    t.m0 = last_end + (tm - before) * BM;
    t.K = 0;
    return t.m0 < g.M;
  } else {
    int tm, tn;
    tile_coords(blockIdx.x, (g.M + BM - 1) / BM, tiles_n, BM >= 128 ? 8 : 1, tm, tn);
    t.m0 = tm * BM;
    t.n0 = tn * BN;
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

// The grid of BM x BN tiles: in the experts' form each expert's last tile of
// rows may be short, and the rest's.
inline int64_t grid_tiles(Fp8Form form, const Fp8Args& g, int bm, int bn) {
  const int64_t tiles_n = (g.N + bn - 1) / bn;
  return tiles_n * (form == FP8_EXPERTS ? (int64_t)g.M / bm + g.experts + 1 : (int64_t)((g.M + bm - 1) / bm));
}

}  // namespace
}  // namespace sgemm_impl
