// FP8 products of operands that load directly to LDS (16-byte aligned, row
// strides multiples of 16): tiles of C from whole slabs of one block of 128.

#include "sgemm_internal.h"
#include "fp8_device.h"

namespace sgemm_impl {
namespace {

constexpr int vmcnt_imm(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }

template <int BM, int BN, int WM, int WN>
struct TileShape {
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int ROWS = BM + BN;           // of a slab: A's, then B's
  static constexpr int REGIONS = ROWS / 8 / NW;  // 1 KiB direct loads per wave and slab
  static constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
  static_assert(NW % 2 == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole regions of either operand per wave");
  static_assert(ROWS % NT == 0 || NT % ROWS == 0, "scales per thread");
};

template <int FORM, bool WIDE, bool TALL, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN) fp8_tile_kernel(Fp8Args g) {
  using S = TileShape<BM, BN, WM, WN>;
  constexpr int MF = S::MF, NF = S::NF, NT = S::NT, ROWS = S::ROWS;
  // One array per stage, so that the compiler sees that reads of one do not
  // wait for loads into the other.
  __shared__ __align__(1024) uint8_t slab0[ROWS * kBlock], slab1[ROWS * kBlock];
  __shared__ __align__(16) float scale0[ROWS], scale1[ROWS];
  Tile t;
  if (!find_tile<FORM, BM, BN>(g, t)) return;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int r16 = lane % 16, quad = lane / 16;
  const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);
  const int blocks = (t.K + kBlock - 1) / kBlock;

  // Direct loads: region q of this wave is rows 8*(q*NW + wave) .. +7; a lane
  // brings one chunk, the same for all its regions.
  const int chunk = swz(8 * wave + lane / 8, lane % 8);
  uint32_t src[S::REGIONS];  // its row's offset from the tile's first row
#pragma unroll
  for (int q = 0; q < S::REGIONS; ++q) {
    const int r = 8 * (q * S::NW + wave) + lane / 8;
    src[q] = q * S::NW * 8 < BM ? (uint32_t)(min(t.m0 + r, t.rows_a - 1) - t.m0) * (uint32_t)g.lda
                                : (uint32_t)(min(t.n0 + r - BM, t.rows_b - 1) - t.n0) * (uint32_t)g.ldb;
  }
  const uint8_t* a0 = t.A + (int64_t)t.m0 * g.lda;
  const uint8_t* b0 = t.B + (int64_t)t.n0 * g.ldb;
  auto load = [&](int b, uint8_t* slab) __attribute__((always_inline)) {
    // A chunk that is not whole is replaced once it has landed; its load
    // brings the row's first 16 bytes.
    const int k = b * kBlock + 16 * chunk;
    const uint32_t at = k + 16 <= t.K ? k : 0;
#pragma unroll
    for (int q = 0; q < S::REGIONS; ++q)
      __builtin_amdgcn_global_load_lds((global_void*)((q * S::NW * 8 < BM ? a0 : b0) + (src[q] + at)),
                                       (lds_void*)(slab + (q * S::NW + wave) * 1024), 16, 0, 0);
  };
  // This thread's scales of block b: row tid (+ NT ...) of the slab.
  constexpr int NS = (ROWS + NT - 1) / NT;
  auto load_scale = [&](int b, float (&s)[NS]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int r = tid + i * NT;
      if (r < BM) {
        s[i] = t.SA[(int64_t)min(t.m0 + r, t.rows_a - 1) * g.sa_row + (int64_t)b * g.sa_block];
      } else if (r < ROWS) {
        const int n = min(t.n0 + r - BM, t.rows_b - 1);
        s[i] = t.SB[(int64_t)(TALL ? n / kBlock : n) * g.sb_row + (int64_t)b * g.sb_block];
      }
    }
  };
  auto keep_scale = [&](const float (&s)[NS], float* scale) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (ROWS % NT == 0 || tid + i * NT < ROWS) scale[tid + i * NT] = s[i];
  };

  f32x4 acc[NF][MF] = {};
  const int at0 = r16 * kBlock + 16 * swz(r16, quad), at1 = at0 ^ 64;
  auto compute = [&](const uint8_t* slab, const float* scale) __attribute__((always_inline)) {
    Frag<WIDE> fa[MF];
    float sa[MF];
    i32x4 raw[2][2];
    const uint8_t* a = slab + wm * kBlock;
    const uint8_t* b = slab + (BM + wn) * kBlock;
    auto read_b = [&](int j) __attribute__((always_inline)) {
      raw[j & 1][0] = *(const i32x4*)(b + j * 16 * kBlock + at0);
      raw[j & 1][1] = *(const i32x4*)(b + j * 16 * kBlock + at1);
    };
    read_b(0);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      fa[i].set(*(const i32x4*)(a + i * 16 * kBlock + at0), *(const i32x4*)(a + i * 16 * kBlock + at1));
      sa[i] = scale[wm + 16 * i + r16];
    }
    if constexpr (TALL) {
      const float sb = scale[BM + wn];
#pragma unroll
      for (int i = 0; i < MF; ++i) sa[i] *= sb;
    }
    // Products of fragment j of B with A's, while those of fragment j - 1
    // enter the accumulators and fragment j + 1 is read.
    f32x4 p[MF], sv = {};
#pragma unroll
    for (int j = 0; j <= NF; ++j) {
      Frag<WIDE> fb;
      if (j + 1 < NF) read_b(j + 1);
      __builtin_amdgcn_sched_barrier(0);
      if (j < NF) fb.set(raw[j & 1][0], raw[j & 1][1]);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        if (j > 0)
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[j - 1][i][x] = __builtin_fmaf(p[i][x], TALL ? sa[i] : sa[i] * sv[x], acc[j - 1][i][x]);
        if (j < NF) p[i] = block_product(fb, fa[i]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!TALL)
        if (j < NF) sv = *(const f32x4*)&scale[BM + wn + 16 * j + 4 * quad];
    }
  };

  // Step b: slab b has been asked for one step ago; slab b + 1 is asked for
  // while it is multiplied. Scales go one step further ahead, through
  // registers. `cur`/`next`: the stages.
  float s[NS] = {};
  auto step = [&](int b, uint8_t* cur, float* scur, uint8_t* next, float* snext) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
    const int left = t.K - b * kBlock;
    if (left < kBlock) {  // the last, partial block: bytes from K on are zero
      for (int r = tid; r < ROWS; r += NT) {
        const bool isa = r < BM;
        const int row = isa ? min(t.m0 + r, t.rows_a - 1) : min(t.n0 + r - BM, t.rows_b - 1);
        const uint8_t* p = isa ? t.A + (int64_t)row * g.lda : t.B + (int64_t)row * g.ldb;
        for (int c = left / 16; c < 8; ++c)
          *(i32x4*)(cur + r * kBlock + 16 * swz(r, c)) = load16(p, b * kBlock + 16 * c, t.K);
      }
      __syncthreads();
    }
    if (b + 1 < blocks) {
      load(b + 1, next);
      keep_scale(s, snext);
      if (b + 2 < blocks) load_scale(b + 2, s);
    }
    __builtin_amdgcn_sched_barrier(0);
    compute(cur, scur);
  };
  if (blocks > 0) {
    load(0, slab0);
    float first[NS];
    load_scale(0, first);
    if (blocks > 1) load_scale(1, s);
    keep_scale(first, scale0);
    int b = 0;
    do {
      step(b, slab0, scale0, slab1, scale1);
      if (++b == blocks) break;
      step(b, slab1, scale1, slab0, scale0);
    } while (++b < blocks);
  }
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = t.m0 + wm + 16 * i + r16;
    if (m >= t.rows_a) continue;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int n = t.n0 + wn + 16 * j + 4 * quad;
      store_c(g, t.C, (int64_t)m * g.ldc + n, g.N - n, acc[j][i]);
    }
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
  return wide ? of_shape<true, 128, 128, 2, 2>(form, tall) : of_shape<false, 128, 128, 2, 2>(form, tall);
}

}  // namespace sgemm_impl
