// Products by expert of 16-bit operands that load directly to LDS (16-byte
// aligned, strides multiples of eight elements): tiles of C from slabs of 64
// values of the summed axis.
//
// An operand whose rows run along the summed axis lies in LDS as 128-byte rows,
// one for each row of the tile. One whose rows run across it (B of the rows'
// gradient, both of the weights') lies as it is in memory, 64 rows of the
// tile's columns, and its fragments are read transposed (ds_read_b64_tr_b16:
// sixteen lanes read four rows by sixteen columns, and each gets the four
// values of its column). No operand is copied or transposed beforehand.
//
// 256 x 256 tiles by eight waves of 64 x 128, one workgroup to a CU: a wave's
// slab is 64 matrix instructions for 24 reads of 16 bytes, and LDS holds two
// slabs of 64 KiB; or 192 x 256, and pieces of either, where rounds of the chip
// are better filled so. Where these are too few for the chip, 128 x 128 by four
// waves, two to a CU. Bound by the matrix unit and the power it may draw: one
// expert of 8192 rows, N 8192, K 4096 bf16 440 us (1.25 PFLOP/s, half of its
// cycles busy); 32 ragged ones of 512 rows on average, N 2048, K 4096 304 us
// (0.9), a fifth of whose tiles' rows are empty.

#include "experts_device.h"

namespace sgemm_impl {
namespace {

// The tile t of BM x BN by WM x WN waves; a slab each at slab0 and slab1, two
// arrays, so that the compiler sees that reads of one do not wait for loads
// into the other.
template <int FORM, class E, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void multiply_tile(const ExpertsArgs& g, const ExpertsTile& t, uint8_t* slab0, uint8_t* slab1) {
  constexpr bool ACROSS_A = FORM == EXPERTS_WGRAD, ACROSS_B = FORM != EXPERTS_FORWARD;
  constexpr int NW = WM * WN, NT = 64 * NW, MF = BM / WM / 16, NF = BN / WN / 16;
  using PA = Part<ACROSS_A, BM, NW>;
  using PB = Part<ACROSS_B, BN, NW>;
  constexpr int REGIONS = PA::REGIONS + PB::REGIONS, BYTES_A = PA::BYTES, BYTES = BYTES_A + PB::BYTES;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
  const int rows_c = FORM == EXPERTS_WGRAD ? g.M : t.rows_a;  // C's end below the tile
  // Whole slabs, and what is left. Where both operands run across the summed
  // axis, rows past its end load as zeros and nothing is left.
  const int full = FORM == EXPERTS_WGRAD ? (t.K + kSlab - 1) / kSlab : t.K / kSlab, tail = FORM == EXPERTS_WGRAD ? 0 : t.K % kSlab;

  int row_a, in_a, row_b, in_b;
  PA::source(wave, lane, row_a, in_a);
  PB::source(wave, lane, row_b, in_b);
  const uint32_t lda = 2 * (uint32_t)g.lda, ldb = 2 * (uint32_t)g.ldb;  // bytes
  const uint32_t a_src = row_a * lda + in_a, b_src = row_b * ldb + in_b;
  const uint8_t* a0 = t.A + (ACROSS_A ? 2 * (int64_t)t.m0 : t.m0 * (int64_t)lda);
  const uint8_t* b0 = t.B + (ACROSS_B ? 2 * (int64_t)t.n0 : t.n0 * (int64_t)ldb);
  const int64_t a_step = ACROSS_A ? kSlab * (int64_t)lda : 2 * kSlab, b_step = ACROSS_B ? kSlab * (int64_t)ldb : 2 * kSlab;
  // Bytes from the part's beginning in slab b to the operand's end.
  auto left_of = [&](bool across, int cols, int rows, int ld, int b) __attribute__((always_inline)) {
    return across ? (min(t.K - b * kSlab, kSlab) - 1) * ld + 2 * cols : (rows - 1) * ld + 2 * (t.K - b * kSlab);
  };
  const int rows_in_a = ACROSS_A ? 0 : min(t.rows_a - t.m0, BM), rows_in_b = ACROSS_B ? 0 : min(g.N - t.n0, BN);
  // Regions [from, to) of slab b, or nothing (and no memory traffic) when there is none.
  auto load = [&](int b, bool there, uint8_t* slab, int from, int to) __attribute__((always_inline)) {
#pragma unroll
    for (int q = from; q < to; ++q) {
      if (q < PA::REGIONS)
        copy16_to_lds(a0 + b * a_step, there ? left_of(ACROSS_A, g.M - t.m0, rows_in_a, lda, b) : 0, a_src + q * PA::STEP * lda,
                      slab + (q * NW + wave) * 1024);
      else
        copy16_to_lds(b0 + b * b_step, there ? left_of(ACROSS_B, g.N - t.n0, rows_in_b, ldb, b) : 0,
                      b_src + (q - PA::REGIONS) * PB::STEP * ldb, slab + (q * NW + wave) * 1024);
    }
  };
  // The partial slab goes before the others, in slab 1: once it has landed, the
  // chunks of its 128-byte rows that are not whole are replaced.
  auto mend_rows = [&](uint8_t* part, const uint8_t* base, int64_t ld, int first, int end, int rows) __attribute__((always_inline)) {
    for (int r = tid; r < rows; r += NT) {
      const i32x4 chunk = load16_end(base + min(first + r, end - 1) * ld, 2 * (t.K - tail % 8), 2 * t.K);
      *(i32x4*)(part + r * 2 * kSlab + 16 * swz(r, tail / 8)) = chunk;
      for (int c = tail / 8 + 1; c < 8; ++c) *(i32x4*)(part + r * 2 * kSlab + 16 * swz(r, c)) = i32x4{0, 0, 0, 0};
    }
  };
  auto stage_tail = [&]() __attribute__((always_inline)) {
    load(full, true, slab1, 0, REGIONS);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
    if constexpr (!ACROSS_A) mend_rows(slab1, t.A, lda, t.m0, t.rows_a, BM);
    if constexpr (!ACROSS_B) mend_rows(slab1 + BYTES_A, t.B, ldb, t.n0, g.N, BN);
    __syncthreads();
  };
  // A slab's direct loads are issued over the first half of the slab before it.
  constexpr int PER = (REGIONS + NF / 2 - 1) / (NF / 2);
  if (full > 0) load(0, true, slab0, 0, REGIONS);
  auto first_slabs = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
    load(1, full > 1, slab1, 0, PER);
  };
  if (t.m0 + wm >= rows_c || t.n0 + wn >= g.N) {
    // Nothing of C is this wave's: it makes its loads and keeps the barriers.
    if (tail > 0) stage_tail();
    if (full > 0) first_slabs();
    for (int b = 0; b < full; ++b) {
      load(b + 1, b + 1 < full, b % 2 ? slab0 : slab1, PER, REGIONS);
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      __syncthreads();
      load(b + 2, b + 2 < full, b % 2 ? slab1 : slab0, 0, PER);
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();  // with the others, before they use the slabs for C
    return;
  }

  // A slab is multiplied in NF groups, one fragment of B with the wave's MF of
  // A, while the next fragment is read. Before the last group, all reads of
  // slab b have been made and slab b + 1 has landed: there is the slab's one
  // barrier, after which slab b + 2 is asked for in slab b's place, and the
  // last group's fragments of A are replaced by the next slab's as soon as
  // they are used, so that the next slab begins without a pause.
  f32x4 acc[NF][MF] = {};
  i32x4 fa[MF][2], fb[2][2];
  const int at_a = PA::place(wm, lane), at_b = PB::place(wn, lane);
  auto read_a = [&](int i, int x, const uint8_t* slab) __attribute__((always_inline)) { fa[i][x] = PA::read(slab, at_a, i, x); };
  auto read_b = [&](int j, const uint8_t* slab) __attribute__((always_inline)) {
    fb[j & 1][0] = PB::read(slab + BYTES_A, at_b, j, 0), fb[j & 1][1] = PB::read(slab + BYTES_A, at_b, j, 1);
  };
  auto step = [&](int b, uint8_t* cur, uint8_t* next) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      if (j + 1 == NF) {
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        __syncthreads();
        load(b + 2, b + 2 < full, cur, 0, PER);
      } else {
        load(b + 1, b + 1 < full, next, min((j + 1) * PER, REGIONS), min((j + 2) * PER, REGIONS));
      }
      __builtin_amdgcn_sched_barrier(0);
      // All fragments of one half before the other half of any: a fragment's products depend on each other.
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          acc[j][i] = mfma16<E>(fb[j & 1][x], fa[i][x], acc[j][i]);
          // After the group's first product: the compiler waits for every outstanding LDS read before it.
          if (x == 0 && i == 0) read_b(j + 1 < NF ? j + 1 : 0, j + 1 < NF ? cur : next);
          if (j + 1 == NF) read_a(i, x, next);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  };
  if (tail > 0) {
    stage_tail();
#pragma unroll
    for (int i = 0; i < MF; ++i) read_a(i, 0, slab1), read_a(i, 1, slab1);
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      read_b(j, slab1);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < MF; ++i) acc[j][i] = mfma16<E>(fb[j & 1][x], fa[i][x], acc[j][i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (full > 0) {
    first_slabs();
#pragma unroll
    for (int i = 0; i < MF; ++i) read_a(i, 0, slab0), read_a(i, 1, slab0);
    read_b(0, slab0);
    int b = 0;
    for (; b + 2 <= full; b += 2) {
      step(b, slab0, slab1);
      step(b + 1, slab1, slab0);
    }
    if (b < full) step(b, slab0, slab1);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // no load into LDS outlives the workgroup
  }
  float* out = (float*)(wave < NW / 2 ? slab0 : slab1) + wave % (NW / 2) * (BYTES * 2 / NW / 4);
  __syncthreads();  // all reads of the slabs have been made
  strips_to_c<E, MF, NF, BYTES * 2 / NW>(g, t, acc, out, wm, wn, rows_c, lane);
}

// Tiles of 256 x 256 that begin a last round of the chip with few workgroups are
// multiplied in pieces (find_experts_tile).
template <int FORM, class E, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, 2) experts_tile_kernel(ExpertsArgs g) {
  constexpr bool SPLIT = splits_last_round(FORM, BM);
  constexpr int BYTES = 2 * kSlab * (BM + BN);
  __shared__ __align__(1024) uint8_t slab0[BYTES], slab1[BYTES];
  ExpertsTile t;
  if (!find_experts_tile<FORM, BM, BN, SPLIT>(g, t)) return;
  if constexpr (SPLIT) {
    if (t.rows == kLowerRows) {
      if (t.pieces == 1) multiply_tile<FORM, E, kLowerRows, BN, WM, WN>(g, t, slab0, slab1);
      else multiply_tile<FORM, E, kLowerRows, BN / 2, WM, WN>(g, t, slab0, slab1);
      return;
    }
    if (t.pieces > 1) {
      if (t.pieces == 4) multiply_tile<FORM, E, BM / 2, BN / 2, WM, WN>(g, t, slab0, slab1);
      else multiply_tile<FORM, E, BM, BN / 2, WM, WN>(g, t, slab0, slab1);
      return;
    }
  }
  multiply_tile<FORM, E, BM, BN, WM, WN>(g, t, slab0, slab1);
}

template <class E, int BM, int BN, int WM, int WN>
const void* of_shape(ExpertsForm form) {
  return form == EXPERTS_FORWARD ? (const void*)&experts_tile_kernel<EXPERTS_FORWARD, E, BM, BN, WM, WN>
         : form == EXPERTS_DGRAD ? (const void*)&experts_tile_kernel<EXPERTS_DGRAD, E, BM, BN, WM, WN>
                                 : (const void*)&experts_tile_kernel<EXPERTS_WGRAD, E, BM, BN, WM, WN>;
}

}  // namespace

const void* experts_tile_kernel_for(ExpertsForm form, int type, int bm) {
  if (type == SGEMM_MI355_BF16)
    return bm == 256 ? of_shape<__hip_bfloat16, 256, 256, 4, 2>(form) : of_shape<__hip_bfloat16, 128, 128, 2, 2>(form);
  return bm == 256 ? of_shape<__half, 256, 256, 4, 2>(form) : of_shape<__half, 128, 128, 2, 2>(form);
}

}  // namespace sgemm_impl
