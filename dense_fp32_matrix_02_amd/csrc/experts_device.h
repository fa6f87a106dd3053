// Device code shared by the kernels of the 16-bit experts' products.
#pragma once

#include <type_traits>

#include "sgemm_internal.h"
#include "experts_internal.h"
#include "fp8_device.h"

namespace sgemm_impl {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kSlab = 64;  // values of the summed axis in a slab: 128 bytes of a row

// 16 x 16 products over 32 values of the summed axis, added to c: a lane has
// eight of them, of row l%16 of either operand; rows of the result are b's,
// columns a's; lane l holds rows 4*(l/16) .. +3 of column l%16.
template <class E>
__device__ __forceinline__ f32x4 mfma16(i32x4 b, i32x4 a, f32x4 c) {
  if constexpr (sizeof(E) == sizeof(__half) && __is_same(E, __half))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
}

constexpr int vmcnt_imm(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }

// 16 bytes at base + offset (none beyond base + bytes) to LDS at lds + 16*lane.
__device__ __forceinline__ void copy16_to_lds(const uint8_t* base, int bytes, uint32_t offset, uint8_t* lds) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass has no type for the buffer
  const auto buffer = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, 0x00027000);  // plain bytes, range-checked
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer, (lds_void*)lds, 16, offset, 0, 0, 0);
#endif
}

__device__ __forceinline__ s16x4 read_transposed(const uint8_t* p) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
#else
  return s16x4{};
#endif
}

// Sixteen bytes whose address is a multiple of two only, as a load of them from
// the next multiple of four and a load of the first value: one load of that
// alignment takes four times as long (the few-rows kernel, 64 rows of 16
// experts, N 2048, K 4095: 148 us, 65 so). Two bytes more than the sixteen are
// read.
struct OddChunk {
  i32x4 v;
  uint32_t first, odd;
};
__device__ __forceinline__ OddChunk load_odd(const uint8_t* p) {
  OddChunk c;
  c.odd = (uint32_t)(uintptr_t)p & 2;
  __builtin_memcpy(&c.v, __builtin_assume_aligned(p + c.odd, 4), 16);
  c.first = *(const uint16_t*)p;
  return c;
}
__device__ __forceinline__ i32x4 in_place(const OddChunk& c) {
  if (c.odd == 0) return c.v;
  return i32x4{(int)(c.first | (uint32_t)c.v[0] << 16), (int)__builtin_amdgcn_alignbit(c.v[1], c.v[0], 16),
               (int)__builtin_amdgcn_alignbit(c.v[2], c.v[1], 16), (int)__builtin_amdgcn_alignbit(c.v[3], c.v[2], 16)};
}
__device__ __forceinline__ i32x4 in_place(const i32x4& v) { return v; }

// An operand's part of a slab: BX rows (or, ACROSS, columns) of the tile.
template <bool ACROSS_, int BX, int NW>
struct Part {
  static constexpr bool ACROSS = ACROSS_;
  static constexpr int PITCH = ACROSS ? 2 * BX : 2 * kSlab;  // bytes of a row in LDS
  static constexpr int BYTES = 2 * BX * kSlab;
  static constexpr int REGIONS = BYTES / 1024 / NW;          // 1 KiB direct loads per wave
  static constexpr int LANES = PITCH / 16;                   // lanes that load a row
  static constexpr int STEP = NW * 64 / LANES;               // rows from one of a wave's regions to its next
  static_assert(BYTES % (1024 * NW) == 0 && STEP % 16 == 0, "a lane's place in its row is the same in all its regions");

  // Which of the groups of 32 bytes of row k of an ACROSS part lies where:
  // group c at c ^ f(k). A transposed read takes 32 bytes of each of rows k ..
  // k+3 and k+8 .. k+11 at once, which have to meet different banks.
  static __device__ __forceinline__ int f(int k) { return (k & 3) | ((k >> 1) & 4); }

  // The row of its first region that a lane loads, and the bytes in it.
  static __device__ __forceinline__ void source(int wave, int lane, int& row, int& bytes) {
    row = wave * (64 / LANES) + lane / LANES;
    const int c = lane % LANES;
    bytes = 16 * (ACROSS ? c ^ (f(row) << 1) : swz(row, c));
  }
  // Where a lane reads its share of fragment 0 of the strip that begins at row
  // (column) w0; fragment j is at this ^ (j << 5) (ACROSS) or + j * 16 * PITCH.
  static __device__ __forceinline__ int place(int w0, int lane) {
    const int r16 = lane % 16, quad = lane / 16;
    if (!ACROSS) return (w0 + r16) * PITCH + 16 * swz(r16, quad);
    return (8 * quad + r16 / 4) * PITCH + (((w0 / 16) ^ f(8 * quad + r16 / 4)) << 5) + 8 * (r16 % 4);
  }
  // Values 8*quad .. +7 of half x of the slab, of row l%16 of fragment j.
  static __device__ __forceinline__ i32x4 read(const uint8_t* part, int place, int j, int x) {
    if constexpr (!ACROSS) {
      return *(const i32x4*)(part + ((place + j * 16 * PITCH) ^ (x * 64)));
    } else {
      const uint8_t* p = part + (place ^ (j << 5)) + 32 * x * PITCH;
      const s16x4 lo = read_transposed(p), hi = read_transposed(p + 4 * PITCH);
      i32x4 v;
      __builtin_memcpy(&v, &lo, 8);
      __builtin_memcpy((char*)&v + 8, &hi, 8);
      return v;
    }
  }
};

// What one workgroup computes: a tile of one product. A and B begin with the
// first row of their product; rows_a is an end in rows of A (FORWARD, DGRAD).
struct ExpertsTile {
  const uint8_t *A, *B;
  int rows_a;
  int m0, n0;
  int K;
  void* C;
  int rows, pieces;  // this is one of so many pieces of a tile of so many rows
};

// The kernel with 256 x 256 tiles, one to a CU, multiplies the tiles left for the
// chip's last round in pieces where these fit the round: up to 64 tiles in four
// (128 x 128), up to 128 in two (256 x 128). Us without and with pieces: 8 experts
// of 1024 rows, N 2048, K 1024, 32 tiles left 49.3 and 40.7; rows' gradients of 8
// of 512 rows, N and K 4096, 32 left 188 and 159; 32 of 512 rows, N 2048, K 4096,
// 120 left 316 and 304. (That in four pieces, two rounds then: 324. 144 left in
// halves, two rounds: 58.5 against 44.6 whole.)
constexpr int kCUs = 256, kMostPieces = 256, kLowerRows = 192;
constexpr bool splits_last_round(int form, int bm) { return form != EXPERTS_WGRAD && bm == 256; }

// Tiles of BM rows in all, of experts and then of the rows that no expert has,
// which begin at last_end.
template <int BM>
__device__ __forceinline__ int count_experts_tiles(const ExpertsArgs& g, int& last_end) {
  const int lane = threadIdx.x % 64;
  int begin, end, upto, total = 0;
  last_end = 0;
  for (int e0 = 0; e0 < g.experts; e0 += 64) {
    expert_tiles<BM>(g, e0, lane, begin, end, upto, last_end);
    total += __builtin_amdgcn_readlane(upto, 63);
  }
  return total + (g.M - last_end + BM - 1) / BM;
}

// Workgroup `block` of `total` rows of BM x BN tiles, those of the last round in
// pieces where SPLIT.
template <int BM, int BN, bool SPLIT>
__device__ __forceinline__ bool place_experts_tile(const ExpertsArgs& g, int total, int last_end, ExpertsTile& t) {
  const int lane = threadIdx.x % 64, tiles_n = (g.N + BN - 1) / BN;
  const int64_t tiles = (int64_t)total * tiles_n;
  int64_t block = blockIdx.x, whole = tiles, parts = tiles;
  int pieces = 1;
  if (SPLIT && tiles % kCUs <= kMostPieces / 2) {
    whole -= tiles % kCUs, parts = whole;
    if (block >= whole) {
      pieces = BM == 256 && tiles - whole <= kMostPieces / 4 ? 4 : 2;
      block -= whole, parts = (tiles - whole) * pieces;
    }
  }
  if (block >= parts) return false;
  // Each XCD gets a run of neighbouring tiles, so that its L2 serves the rows
  // they share. (Whole tiles first and partial ones last, for a shorter last
  // round, measured 352 us against 318 for 16384 rows of 32 experts, N 2048, K
  // 4096: the weights are then read twice.)
  const int64_t each = parts / 8, more = parts % 8, xcd = block % 8;
  int64_t id = xcd * each + (xcd < more ? xcd : more) + block / 8;
  int down = 0, right = 0;  // a piece's place in its tile
  if (pieces > 1) {
    const int piece = (int)(id & (pieces - 1));
    id = whole + (pieces == 4 ? id >> 2 : id >> 1);
    down = piece >> 1, right = piece & 1;
  }
  t.pieces = pieces;
  const int tm = (int)(id / tiles_n);
  t.n0 = (int)(id - (int64_t)tm * tiles_n) * BN + right * (BN / 2);
  int begin, end, upto, before = 0, last = 0;
  for (int e0 = 0; e0 < g.experts; e0 += 64) {
    const int own = expert_tiles<BM>(g, e0, lane, begin, end, upto, last);
    const uint64_t past = __ballot(tm < before + upto);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      // The same in every lane: kept in scalar registers.
      t.m0 = __builtin_amdgcn_readlane(begin, l) + (tm - before - __builtin_amdgcn_readlane(upto - own, l)) * BM + down * (BM / 2);
      t.rows_a = __builtin_amdgcn_readlane(end, l);
      t.B += 2 * (e0 + l) * g.strideB;
      return !SPLIT || (t.m0 < t.rows_a && t.n0 < g.N);
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  // Rows no expert has: a product over nothing.
  t.m0 = last_end + (tm - before) * BM + down * (BM / 2);
  t.K = 0;
  return t.m0 < g.M && t.n0 < g.N;
}

// Hundredths of the time of a full round of 256 x 256 tiles that so many tiles
// take, each round of them `round`, a last one in pieces `halves` or `quarters`.
__device__ __forceinline__ int64_t rounds_of(int64_t tiles, int round, int halves, int quarters) {
  const int64_t left = tiles % kCUs;
  return tiles / kCUs * round + (left == 0 ? 0 : left <= kMostPieces / 4 ? quarters : left <= kMostPieces / 2 ? halves : round);
}

// The tile of this workgroup. SPLIT: of 256 x 256 or 192 x 256 (t.rows), as the
// experts' rows decide, which the host does not know.
template <int FORM, int BM, int BN, bool SPLIT = false>
__device__ __forceinline__ bool find_experts_tile(const ExpertsArgs& g, ExpertsTile& t) {
  t.A = (const uint8_t*)g.A, t.B = (const uint8_t*)g.B, t.C = g.C;
  t.rows_a = g.M, t.K = g.K, t.rows = BM, t.pieces = 1;
  if constexpr (FORM == EXPERTS_WGRAD) {
    int tm, tn, begin, end;
    tile_coords(blockIdx.x, (g.M + BM - 1) / BM, (g.N + BN - 1) / BN, 8, tm, tn);
    t.m0 = tm * BM, t.n0 = tn * BN;
    const int e = blockIdx.y;
    expert_rows(g.offsets, e, g.K, begin, end);
    t.K = end - begin;
    t.A += 2 * (begin * g.lda), t.B += 2 * (begin * g.ldb);
    t.C = (char*)g.C + e * g.strideC * (g.c_type == SGEMM_MI355_F32 ? 4 : 2);
    return true;
  } else {
    int last_end = 0;
    const int total = count_experts_tiles<BM>(g, last_end);
    // Tiles of 192 rows where they fill the chip's rounds better: as many in one
    // round do less, in less time (us, 256 and 192 rows: rows' gradients of 8
    // experts of 1024 rows, N 2048, K 1024, 144 and 192 tiles 45.6 and 38.3; of
    // 32 of 256 rows, N 4096, K 1024, 192 and 256 tiles 107.7 and 96.3; 8192
    // rows, N 8192, K 4096, 1024 and 1376 tiles 437 and 554). A short axis is all
    // start and end (6144 rows, N 2048, 192 and 256 tiles: K 8192 186 and 174, K
    // 2048 45.9 and 46.3, K 256 14.8 and 16.9).
    if constexpr (SPLIT) {
      const int lower = count_experts_tiles<kLowerRows>(g, last_end), tiles_n = (g.N + BN - 1) / BN;
      if (g.K >= 512 && rounds_of((int64_t)lower * tiles_n, 88, 54, 54) < rounds_of((int64_t)total * tiles_n, 100, 60, 40)) {
        t.rows = kLowerRows;
        return place_experts_tile<kLowerRows, BN, true>(g, lower, last_end, t);
      }
    }
    return place_experts_tile<BM, BN, SPLIT>(g, total, last_end, t);
  }
}

// `valid` of W neighbours of C at element `at`, added to beta * C.
template <int W>
__device__ __forceinline__ void store_experts(const ExpertsArgs& g, void* C, int64_t at, int valid, const float (&v)[W]) {
  if (g.c_type == SGEMM_MI355_F32) store_as((float*)C + at, valid, v, g.beta);
  else if (g.c_type == SGEMM_MI355_BF16) store_as((__hip_bfloat16*)C + at, valid, v, g.beta);
  else store_as((__half*)C + at, valid, v, g.beta);
}

// A wave's accumulators to C by way of its own ROOM bytes of LDS at `out`, some
// fragments of A's rows at a time, so that a lane stores 16 bytes next to its
// neighbour's and a row's strip is stored at a stretch, in a loop of rows that
// is not unrolled: its code runs once per tile. (FP32 in two runs of 16 bytes a
// lane, which leaves every other 16 to the next instruction: 8 experts of 512 rows, weight gradients of 4096 x 4096 233 us, 213 so.) The
// strip begins at (wm, wn) of the tile; C has rows up to rows_c.
template <class E, int MF, int NF, int ROOM>
__device__ __forceinline__ void strips_to_c(const ExpertsArgs& g, const ExpertsTile& t, const f32x4 (&acc)[NF][MF], float* out,
                                            int wm, int wn, int rows_c, int lane) {
  constexpr int WIDTH = 16 * NF;                // floats of a row of the strip
  constexpr int FIT = ROOM / (16 * WIDTH * 4);  // fragments that the room holds
  constexpr int ROUND = FIT >= MF ? MF : FIT >= 2 && MF % 2 == 0 ? 2 : 1;
  static_assert(FIT >= 1 && MF % ROUND == 0, "whole rounds");
  const int r16 = lane % 16, quad = lane / 16;
#pragma unroll
  for (int i0 = 0; i0 < MF; i0 += ROUND) {
    // Chunk c of four floats of row r lies at place c ^ (r % 16): 16 rows' writes of one chunk meet all banks.
#pragma unroll
    for (int i = 0; i < ROUND; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) *(f32x4*)(out + (16 * i + r16) * WIDTH + 4 * ((4 * j + quad) ^ r16)) = acc[j][i0 + i];
    __builtin_amdgcn_wave_barrier();  // LDS serves a wave in order
    const int rows = min(16 * ROUND, rows_c - t.m0 - wm - 16 * i0);
    auto rows_to_c = [&](auto* C) __attribute__((always_inline)) {
      using T = std::remove_pointer_t<decltype(C)>;
      constexpr int W = 16 / sizeof(T), LANES = WIDTH / W;  // values that a lane stores, and lanes that store a row
      const int c = W / 4 * (lane % LANES), n = t.n0 + wn + 4 * c;
      const int64_t at = (int64_t)(t.m0 + wm + 16 * i0) * g.ldc + n;
      auto strip = [&](int r, float (&v)[W]) __attribute__((always_inline)) {
#pragma unroll
        for (int x = 0; x < W / 4; ++x) *(f32x4*)(v + 4 * x) = *(const f32x4*)(out + r * WIDTH + 4 * ((c + x) ^ (r % 16)));
      };
      if (g.beta == 0.0f && n + W <= g.N) {
#pragma unroll 4
        for (int r = lane / LANES; r < rows; r += 64 / LANES) {
          float v[W];
          strip(r, v);
          if (g.past) {
            store16_once(C + at + r * g.ldc, v);
          } else {
            store_as<T, W>(C + at + r * g.ldc, W, v, 0.0f);
          }
        }
      } else {
#pragma unroll 1
        for (int r = lane / LANES; r < rows; r += 64 / LANES) {
          float v[W];
          strip(r, v);
          store_as<T, W>(C + at + r * g.ldc, g.N - n, v, g.beta);
        }
      }
    };
    if (g.c_type == SGEMM_MI355_F32) rows_to_c((float*)t.C);
    else rows_to_c((E*)t.C);
    __builtin_amdgcn_wave_barrier();
  }
}

inline int64_t experts_grid(ExpertsForm form, const ExpertsArgs& g, int bm, int bn) {
  const int64_t tiles_n = ((int64_t)g.N + bn - 1) / bn;
  return tiles_n * (form == EXPERTS_WGRAD ? ((int64_t)g.M + bm - 1) / bm
                                         : (int64_t)g.M / (splits_last_round(form, bm) ? kLowerRows : bm) + g.experts + 1) +
         (splits_last_round(form, bm) ? kMostPieces : 0);
}

}  // namespace
}  // namespace sgemm_impl
