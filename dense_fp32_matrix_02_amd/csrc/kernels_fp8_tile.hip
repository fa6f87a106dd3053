// FP8 products of operands that load directly to LDS (16-byte aligned, row
// strides multiples of 16, K 16 or more): tiles of C from whole slabs of one
// block of 128.

#include <type_traits>

#include "sgemm_internal.h"
#include "fp8_device.h"

namespace sgemm_impl {
namespace {

constexpr int vmcnt_imm(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }

// 16 bytes at base + offset (none beyond base + bytes) to LDS at lds + 16*lane.
__device__ __forceinline__ void copy16_to_lds(const uint8_t* base, int bytes, uint32_t offset, uint8_t* lds) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass has no type for the buffer
  const auto buffer = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, 0x00027000);  // plain bytes, range-checked
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer, (lds_void*)lds, 16, offset, 0, 0, 0);
#endif
}

template <int BM, int BN, int WM, int WN>
struct TileShape {
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int ROWS = BM + BN;           // of a slab: A's, then B's
  static constexpr int REGIONS = ROWS / 8 / NW;  // 1 KiB direct loads per wave and slab
  static constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
  static_assert(NW % 2 == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole regions of either operand per wave");
};

template <int FORM, bool WIDE, bool TALL, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, 2) fp8_tile_kernel(Fp8Args g) {
  using S = TileShape<BM, BN, WM, WN>;
  constexpr int MF = S::MF, NF = S::NF, NT = S::NT, ROWS = S::ROWS;
  // One array per stage, so that the compiler sees that reads of one do not
  // wait for loads into the other.
  __shared__ __align__(1024) uint8_t slab0[ROWS * kBlock], slab1[ROWS * kBlock];
  constexpr int NS = (ROWS + NT - 1) / NT;  // scales per thread: every thread has a place for them, so that no step has a branch
  __shared__ __align__(16) float scale0[NS * NT], scale1[NS * NT];
  Tile t;
  if (!find_tile<FORM, BM, BN>(g, t)) return;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int r16 = lane % 16, quad = lane / 16;
  // Waves w and w + 4 share a SIMD: their strips of rows lie apart, so that a
  // tile with half its rows still keeps every SIMD at work.
  const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
  const int full = t.K / kBlock, tail = t.K % kBlock;  // whole blocks, and what is left

  // Direct loads: region q of this wave is rows 8*(q*NW + wave) .. +7; a lane
  // brings one chunk, the same for all its regions. Rows that do not exist lie
  // past the buffers' ends and load as zeros.
  const uint32_t chunk = 16 * swz(8 * wave + lane / 8, lane % 8), row = 8 * wave + lane / 8;
  const uint32_t a_src = row * (uint32_t)g.lda + chunk, b_src = row * (uint32_t)g.ldb + chunk;
  const uint32_t a_region = 8 * S::NW * (uint32_t)g.lda, b_region = 8 * S::NW * (uint32_t)g.ldb;
  const uint8_t* a0 = t.A + (int64_t)t.m0 * g.lda;
  const uint8_t* b0 = t.B + (int64_t)t.n0 * g.ldb;
  const int a_bytes = (min(t.rows_a - t.m0, BM) - 1) * (int)g.lda + t.K;
  const int b_bytes = (min(t.rows_b - t.n0, BN) - 1) * (int)g.ldb + t.K;
  // Regions [from, to) of slab b, or nothing (and no memory traffic) when there is none.
  auto load = [&](int b, bool there, uint8_t* slab, int from, int to) __attribute__((always_inline)) {
#pragma unroll
    for (int q = from; q < to; ++q) {
      const bool a = q * S::NW * 8 < BM;
      const int left = there ? (a ? a_bytes : b_bytes) - b * kBlock : 0;
      // An addition here costs less than the registers of an offset for each region.
      const uint32_t at = a ? a_src + q * a_region : b_src + (q - BM / (8 * S::NW)) * b_region;
      copy16_to_lds((a ? a0 : b0) + b * kBlock, left, at, slab + (q * S::NW + wave) * 1024);
    }
  };
  // This thread's scales: rows tid (+ NT ..) of the slab, of the same operand for the whole wave.
  static_assert(ROWS % 64 == 0 && BM % 64 == 0, "a wave's scales are of one operand");
  const float* scales[NS];
  int64_t scale_step[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int r = tid + i * NT;
    const bool a = 64 * wave + i * NT < BM;
    const int n = min(t.n0 + r - BM, t.rows_b - 1);
    scales[i] = a ? t.SA + (int64_t)min(t.m0 + r, t.rows_a - 1) * g.sa_row : t.SB + (int64_t)(TALL ? n / kBlock : n) * g.sb_row;
    scale_step[i] = a ? g.sa_block : g.sb_block;
  }
  auto load_scale = [&](int b, float (&s)[NS]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] = scales[i][b * scale_step[i]];
  };
  auto keep_scale = [&](const float (&s)[NS], float* scale) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      scale[tid + i * NT] = s[i];
  };

  // A slab's direct loads are issued over the first half of a block: all at
  // once they hold up the waves that issue them (8192^3: 466 us, against 440
  // with two a group and 467 with one, whose last loads land too late).
  constexpr int PER = (S::REGIONS + NF / 2 - 1) / (NF / 2);
  float s[NS] = {};
  if (full > 0) load(0, true, slab0, 0, S::REGIONS);
  // The partial block goes before the others, in slab 1: once it has landed, a
  // thread replaces its row's chunks that are not whole.
  auto stage_tail = [&]() __attribute__((always_inline)) {
    float part[NS];
    i32x4 chunks[NS];
    load(full, true, slab1, 0, S::REGIONS);
    load_scale(full, part);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int r = tid + i * NT;
      const bool isa = r < BM;
      const int row = isa ? min(t.m0 + r, t.rows_a - 1) : min(t.n0 + r - BM, t.rows_b - 1);
      const uint8_t* line = isa ? t.A + (int64_t)row * g.lda : t.B + (int64_t)row * g.ldb;
      const int k = t.K - tail % 16;
      if (FORM != FP8_WGRAD || t.K >= 16) chunks[i] = load16_end(line, k, t.K);
      else chunks[i] = load16(line, k, t.K);
    }
    keep_scale(part, scale1);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int r = tid + i * NT;
      if (ROWS % NT != 0 && 64 * wave + i * NT >= ROWS) break;
      *(i32x4*)(slab1 + r * kBlock + 16 * swz(r, tail / 16)) = chunks[i];
      for (int c = tail / 16 + 1; c < 8; ++c) *(i32x4*)(slab1 + r * kBlock + 16 * swz(r, c)) = i32x4{0, 0, 0, 0};
    }
    __syncthreads();
  };
  // Block 0 has landed, block 1 is asked for, their scales are in LDS and those of block 2 in registers.
  auto first_blocks = [&]() __attribute__((always_inline)) {
    float second[NS];
    load_scale(0, s);
    load_scale(min(1, full - 1), second);
    keep_scale(s, scale0);
    load_scale(min(2, full - 1), s);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
    load(1, full > 1, slab1, 0, PER);
    keep_scale(second, scale1);
  };
  if (t.m0 + wm >= t.rows_a || t.n0 + wn >= t.rows_b) {
    // Nothing of C is this wave's: it makes its loads and keeps the barriers.
    if (tail > 0) stage_tail();
    if (full > 0) first_blocks();
    for (int b = 0; b < full; ++b) {
      load(b + 1, b + 1 < full, b % 2 ? slab0 : slab1, PER, S::REGIONS);
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      __syncthreads();
      load(b + 2, b + 2 < full, b % 2 ? slab1 : slab0, 0, PER);
      keep_scale(s, b % 2 ? scale1 : scale0);
      load_scale(min(b + 3, full - 1), s);
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    return;
  }

  // Block b is multiplied in NF groups, one fragment of B with the wave's MF
  // of A. While the matrix unit works on a group, the group before it enters
  // the accumulators and the next fragment is read. Before the last group, all
  // reads of slab b have been made and slab b + 1 has landed: there is the
  // block's one barrier, after which slab b + 2 is asked for in slab b's place,
  // and the last group's fragments of A are replaced by the next block's as
  // soon as they are used, so that the next block begins without a pause.
  // (Everything in one block, from its barrier to its last product, measured
  // 496 us at 8192^3.) Scales go one block further ahead, through registers.
  // There is no branch in a step: the compiler would move additions behind it.
  f32x4 acc[NF][MF] = {}, p[MF] = {};
  Frag<WIDE> fa[MF];
  i32x4 raw[2][2], raw_a[MF][2];
  float sa[MF] = {}, sa_before[MF] = {};
  f32x4 sv_before, sv = {}, sv_next = {};  // without TALL: B's scales of the groups before, at and after this one
  const int at0 = r16 * kBlock + 16 * swz(r16, quad), at1 = at0 ^ 64;
  auto read_a = [&](int i, const uint8_t* slab) __attribute__((always_inline)) {
    const uint8_t* a = slab + (wm + 16 * i) * kBlock;
    raw_a[i][0] = *(const i32x4*)(a + at0), raw_a[i][1] = *(const i32x4*)(a + at1);
  };
  // Apart from the reads, which widening has to wait for.
  auto set_a = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MF; ++i) fa[i].set(raw_a[i][0], raw_a[i][1]);
  };
  auto read_b = [&](int j, const uint8_t* slab, const float* scale) __attribute__((always_inline)) {
    const uint8_t* b = slab + (BM + wn + 16 * j) * kBlock;
    raw[j & 1][0] = *(const i32x4*)(b + at0), raw[j & 1][1] = *(const i32x4*)(b + at1);
    if constexpr (!TALL) sv_next = *(const f32x4*)&scale[BM + wn + 16 * j + 4 * quad];
  };
  auto read_scales = [&](const float* scale) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MF; ++i) sa[i] = scale[wm + 16 * i + r16];
    if constexpr (TALL) {
      const float sb = scale[BM + wn];
#pragma unroll
      for (int i = 0; i < MF; ++i) sa[i] *= sb;
    }
  };
  auto add = [&](f32x4& c, int i, const float (&w)[MF], f32x4 v) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < 4; ++x) c[x] = __builtin_fmaf(p[i][x], TALL ? w[i] : w[i] * v[x], c[x]);
  };
  auto step = [&](int b, uint8_t* cur, float* scur, uint8_t* next, float* snext) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      sv_before = sv, sv = sv_next;
      if (j + 1 == NF) {
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        __syncthreads();
        load(b + 2, b + 2 < full, cur, 0, PER);
        keep_scale(s, scur);
        load_scale(min(b + 3, full - 1), s);
      }
      if (j + 1 < NF) load(b + 1, b + 1 < full, next, min((j + 1) * PER, S::REGIONS), min((j + 2) * PER, S::REGIONS));
      __builtin_amdgcn_sched_barrier(0);
      if (j == 0) set_a();
      Frag<WIDE> fb;
      fb.set(raw[j & 1][0], raw[j & 1][1]);
      // A step of all fragments before the next step of any: a fragment's steps
      // depend on each other.
#pragma unroll
      for (int x = 0; x < kSteps<WIDE>; ++x) {
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          if (x == 0) {
            if (j > 0) add(acc[j - 1][i], i, sa, sv_before);
            else add(acc[NF - 1][i], i, sa_before, sv_before);
          }
          p[i] = block_step(fb, fa[i], x, p[i]);
          // After the group's first product: the compiler waits for every
          // outstanding LDS read before it.
          if (x == 0 && i == 0 && j + 1 < NF) read_b(j + 1, cur, scur);
          if (x == 0 && i == 0 && j + 1 == NF) read_b(0, next, snext);
          if (x == kSteps<WIDE> - 1 && j + 1 == NF) read_a(i, next);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) sa_before[i] = sa[i];
    read_scales(snext);
  };
  if (tail > 0) {
    stage_tail();
    read_scales(scale1);
#pragma unroll
    for (int i = 0; i < MF; ++i) read_a(i, slab1);
    set_a();
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      Frag<WIDE> fb;
      read_b(j, slab1, scale1);
      fb.set(raw[j & 1][0], raw[j & 1][1]);
#pragma unroll
      for (int i = 0; i < MF; ++i) p[i] = block_product(fb, fa[i]);
#pragma unroll
      for (int i = 0; i < MF; ++i) add(acc[j][i], i, sa, sv_next), p[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (full > 0) {
    first_blocks();
#pragma unroll
    for (int i = 0; i < MF; ++i) read_a(i, slab0);
    read_b(0, slab0, scale0);
    read_scales(scale0);
    int b = 0;
    for (; b + 2 <= full; b += 2) {
      step(b, slab0, scale0, slab1, scale1);
      step(b + 1, slab1, scale1, slab0, scale0);
    }
    if (b < full) step(b, slab0, scale0, slab1, scale1);
#pragma unroll
    for (int i = 0; i < MF; ++i) add(acc[NF - 1][i], i, sa_before, sv);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // no load into LDS outlives the workgroup
  }
  // To C by way of LDS, ROUND fragments of A's rows at a time, so that a lane
  // stores eight neighbours and a row's strip is stored at a stretch. The rows
  // go round a loop that is not unrolled: this code runs once per tile, and
  // fetching it costs more than running it (with a copy of the stores for each
  // fragment this took 3.5 us of a tile, unrolled wholly 8 us of a 256 x 256 one).
  constexpr int WIDTH = 16 * NF, LANES = WIDTH / 8;  // floats of a row of the strip, and lanes that store one
  constexpr int ROOM = kBlock * ROWS * 2 / S::NW / (16 * WIDTH * 4);  // fragments that a wave's share of the slabs holds
  constexpr int ROUND = ROOM >= MF ? MF : ROOM >= 2 && MF % 2 == 0 ? 2 : 1;
  static_assert(ROUND >= 1 && MF % ROUND == 0, "whole rounds");
  float* out = (float*)(wave < S::NW / 2 ? slab0 : slab1) + wave % (S::NW / 2) * (ROUND * 16 * WIDTH);
  __syncthreads();  // all reads of the slabs have been made
#pragma unroll
  for (int i0 = 0; i0 < MF; i0 += ROUND) {
    // Chunk c of four floats of row r lies at place c ^ (r % 16): 16 rows' writes of one chunk meet all banks.
#pragma unroll
    for (int i = 0; i < ROUND; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
        *(f32x4*)(out + (16 * i + r16) * WIDTH + 4 * ((4 * j + quad) ^ r16)) = acc[j][i0 + i];
    __builtin_amdgcn_wave_barrier();  // LDS serves a wave in order
    const int c = 2 * (lane % LANES), n = t.n0 + wn + 4 * c;
    const int rows = min(16 * ROUND, t.rows_a - t.m0 - wm - 16 * i0);
    auto strip = [&](int r, float (&v)[8]) __attribute__((always_inline)) {
      *(f32x4*)v = *(const f32x4*)(out + r * WIDTH + 4 * (c ^ (r % 16)));
      *(f32x4*)(v + 4) = *(const f32x4*)(out + r * WIDTH + 4 * ((c + 1) ^ (r % 16)));
    };
    const int64_t at = (int64_t)(t.m0 + wm + 16 * i0) * g.ldc + n;
    auto rows_to_c = [&](auto* C) __attribute__((always_inline)) {
      using T = std::remove_pointer_t<decltype(C)>;
      if (g.beta == 0.0f && n + 8 <= g.N) {
#pragma unroll 4
        for (int r = lane / LANES; r < rows; r += 64 / LANES) {
          float v[8];
          strip(r, v);
          store8(C + at + r * g.ldc, 8, v);
        }
      } else {
#pragma unroll 1
        for (int r = lane / LANES; r < rows; r += 64 / LANES) {
          float v[8];
          strip(r, v);
          store_as<T, 8>(C + at + r * g.ldc, g.N - n, v, g.beta);
        }
      }
    };
    if (g.type == SGEMM_MI355_F32) rows_to_c((float*)t.C);
    else if (g.type == SGEMM_MI355_BF16) rows_to_c((__hip_bfloat16*)t.C);
    else rows_to_c((__half*)t.C);
    __builtin_amdgcn_wave_barrier();
  }
}

template <bool WIDE, int BM, int BN, int WM, int WN>
const void* of_shape(Fp8Form form, bool tall) {
  if (form == FP8_WGRAD) return (const void*)&fp8_tile_kernel<FP8_WGRAD, WIDE, false, BM, BN, WM, WN>;
  if (form == FP8_EXPERTS)
    return tall ? (const void*)&fp8_tile_kernel<FP8_EXPERTS, WIDE, true, BM, BN, WM, WN>
                : (const void*)&fp8_tile_kernel<FP8_EXPERTS, WIDE, false, BM, BN, WM, WN>;
  return tall ? (const void*)&fp8_tile_kernel<FP8_DENSE, WIDE, true, BM, BN, WM, WN>
              : (const void*)&fp8_tile_kernel<FP8_DENSE, WIDE, false, BM, BN, WM, WN>;
}

}  // namespace

const void* fp8_tile_kernel_for(Fp8Form form, bool wide, bool tall, int bm) {
  if (bm == 256) return of_shape<false, 256, 256, 4, 2>(form, tall);
  if (bm == 192)  // dense products into FP32 only
    return tall ? (const void*)&fp8_tile_kernel<FP8_DENSE, true, true, 192, 128, 4, 2>
                : (const void*)&fp8_tile_kernel<FP8_DENSE, true, false, 192, 128, 4, 2>;
  return wide ? of_shape<true, 128, 128, 2, 2>(form, tall) : of_shape<false, 128, 128, 2, 2>(form, tall);
}

}  // namespace sgemm_impl
