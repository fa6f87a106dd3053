// Products by expert of 16-bit operands: the kernel for operands of any
// alignment, the kernel for few rows, and the choice.

#include <cmath>
#include <type_traits>

#include "experts_device.h"

namespace sgemm_impl {
namespace {

// A 128 x 128 tile by four waves of 64 x 64: operands of any alignment. Slabs
// come through registers, the next two on the way while one is multiplied, and
// lie in LDS as in the kernel for aligned operands; so do its results on their
// way to C (16 experts of 844 rows, rows' gradients, N 176, K 1862: 33.3 us,
// 49.2 with stores of four neighbours from the accumulators; 8 of 512 rows, N
// 1538, K 2046 48, 71 and 62 in the three forms).
// WIDE: rows of either operand have sixteen bytes.
template <int FORM, class E, bool WIDE>
__global__ void __launch_bounds__(256, 2) experts_staged_kernel(ExpertsArgs g) {
  constexpr bool ACROSS_A = FORM == EXPERTS_WGRAD, ACROSS_B = FORM != EXPERTS_FORWARD;
  constexpr int BM = 128, BN = 128, MF = 4, NF = 4, NW = 4;
  using PA = Part<ACROSS_A, BM, NW>;
  using PB = Part<ACROSS_B, BN, NW>;
  constexpr int BYTES_A = 2 * kSlab * BM, BYTES = BYTES_A + 2 * kSlab * BN;
  __shared__ __align__(1024) uint8_t slabs[2][BYTES];
  ExpertsTile t;
  if (!find_experts_tile<FORM, BM, BN>(g, t)) return;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int wm = (wave / 2) * 64, wn = (wave % 2) * 64;
  const int rows_c = FORM == EXPERTS_WGRAD ? g.M : t.rows_a;
  const int count = (t.K + kSlab - 1) / kSlab;
  // What this lane brings of region q of a part in slab b: bytes [k, k + 16) of
  // a row of `length`. Rows past the summed axis' end have none; rows past the
  // tile's last are that one, for results that nobody stores.
  struct Place {
    const uint8_t* row;
    int k, length;
  };
  auto place_of = [&](auto part, const uint8_t* base, int64_t ld, int first, int end, int q, int b) __attribute__((always_inline)) {
    using P = decltype(part);
    int row, in;
    P::source(wave, lane, row, in);
    row += q * P::STEP;
    if constexpr (P::ACROSS) {
      const int k = b * kSlab + row;
      return Place{base + 2 * (min(k, t.K - 1) * ld), 2 * first + in, k < t.K ? 2 * end : 0};
    } else {
      return Place{base + 2 * (min(first + row, end - 1) * ld), 2 * (b * kSlab) + in, 2 * t.K};
    }
  };
  // Sixteen bytes at once, where a row's end is near its last sixteen, which are
  // moved to their places only when they go to LDS, after the products that
  // hide the load. (Byte by byte at the ends of rows, 16 experts of 512 rows, N
  // 1538, K 2046, rows' gradients take 259 us; moved at once 259; so 96.)
  auto fetch = [&](const Place& p) __attribute__((always_inline)) {
    if constexpr (WIDE) {
      i32x4 v;
      __builtin_memcpy(&v, p.row + min(p.k, max(p.length, 16) - 16), 16);
      return v;
    } else {
      return load16(p.row, p.k, p.length);
    }
  };
  auto mended = [&](const Place& p, i32x4 v) __attribute__((always_inline)) {
    const int skip = p.k - (p.length - 16);  // bytes that the load began too early
    if (skip <= 0) return v;
    uint64_t w[2];
    __builtin_memcpy(w, &v, 16);
    if (skip >= 8) w[0] = w[1], w[1] = 0;
    const int bits = 8 * (skip % 8);
    if (bits > 0) w[0] = w[0] >> bits | w[1] << (64 - bits), w[1] >>= bits;
    if (skip >= 16) w[0] = 0;
    __builtin_memcpy(&v, w, 16);
    return v;
  };
  const int end_a = ACROSS_A ? g.M : t.rows_a, end_b = g.N;
  typedef i32x4 Held[PA::REGIONS + PB::REGIONS];
  auto fetch_all = [&](Held& held, int b) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < PA::REGIONS; ++q) held[q] = fetch(place_of(PA{}, t.A, g.lda, t.m0, end_a, q, b));
#pragma unroll
    for (int q = 0; q < PB::REGIONS; ++q) held[PA::REGIONS + q] = fetch(place_of(PB{}, t.B, g.ldb, t.n0, end_b, q, b));
  };
  // Whether a part's chunks of slab b may pass their rows' ends: the same for the whole tile.
  auto mend_all = [&](Held& held, int b) __attribute__((always_inline)) {
    if constexpr (!WIDE) return;
    const bool last = (b + 1) * kSlab > t.K;
    if (last || (ACROSS_A && t.m0 + BM > end_a)) {
#pragma unroll
      for (int q = 0; q < PA::REGIONS; ++q) held[q] = mended(place_of(PA{}, t.A, g.lda, t.m0, end_a, q, b), held[q]);
    }
    if (last || (ACROSS_B && t.n0 + BN > end_b)) {
#pragma unroll
      for (int q = 0; q < PB::REGIONS; ++q)
        held[PA::REGIONS + q] = mended(place_of(PB{}, t.B, g.ldb, t.n0, end_b, q, b), held[PA::REGIONS + q]);
    }
  };
  f32x4 acc[NF][MF] = {};
  const int at_a = PA::place(wm, lane), at_b = PB::place(wn, lane);
  // Slab b, from registers to LDS and through the products, while slabs b + 1
  // and b + 2 are on the way.
  auto step = [&](Held& held, uint8_t* slab, int b) __attribute__((always_inline)) {
    mend_all(held, b);
#pragma unroll
    for (int q = 0; q < PA::REGIONS + PB::REGIONS; ++q) *(i32x4*)(slab + (q * NW + wave) * 1024 + 16 * lane) = held[q];
    // One barrier: the other buffer's readers passed it a slab ago.
    __syncthreads();
    if (b + 2 < count) fetch_all(held, b + 2);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      i32x4 fa[MF];
#pragma unroll
      for (int i = 0; i < MF; ++i) fa[i] = PA::read(slab, at_a, i, x);
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const i32x4 fb = PB::read(slab + BYTES_A, at_b, j, x);
#pragma unroll
        for (int i = 0; i < MF; ++i) acc[j][i] = mfma16<E>(fb, fa[i], acc[j][i]);
      }
    }
  };
  Held even, odd;
  if (count > 0) fetch_all(even, 0);
  if (count > 1) fetch_all(odd, 1);
#pragma unroll 1
  for (int b = 0; b < count; b += 2) {
    step(even, slabs[0], b);
    if (b + 1 < count) step(odd, slabs[1], b + 1);
  }
  __syncthreads();  // all reads of the slabs have been made
  if (t.m0 + wm >= rows_c || t.n0 + wn >= g.N) return;
  strips_to_c<E, MF, NF, 2 * BYTES / NW>(g, t, acc, (float*)(&slabs[0][0] + wave * (2 * BYTES / NW)), wm, wn, rows_c, lane);
}

constexpr int kRowsWaves = 8;

// FORWARD with few rows (a decoding step): a workgroup has 16 rows of an
// expert's weights and 16*MF of A over the whole of K. Its waves take every
// eighth slab, straight from memory to registers, and their sums are added in
// wave order through LDS. Bound by the weights' bytes. ODD: rows need not begin
// at a multiple of four bytes.
template <class E, int MF, bool ODD>
__global__ void __launch_bounds__(64 * kRowsWaves, MF == 4 ? 2 : MF == 1 ? 6 : 4) experts_rows_kernel(ExpertsArgs g) {
  constexpr int BM = 16 * MF, BN = 16, NW = kRowsWaves;
  constexpr int AHEAD = 2;  // slabs that a wave has in flight
  __shared__ __align__(16) f32x4 part[NW][MF][64];
  ExpertsTile t;
  if (!find_experts_tile<EXPERTS_FORWARD, BM, BN>(g, t)) return;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int r16 = lane % 16, quad = lane / 16;
  const uint8_t* b = t.B + 2 * (min(t.n0 + r16, g.N - 1) * g.ldb);
  const uint8_t* a[MF];
  bool there[MF];  // rows that do not exist cost no loads
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    there[i] = t.m0 + 16 * i + r16 < t.rows_a;
    a[i] = t.A + 2 * ((there[i] ? t.m0 + 16 * i + r16 : t.m0) * g.lda);
  }
  f32x4 acc[MF] = {};
  using Chunk = std::conditional_t<ODD, OddChunk, i32x4>;
  struct Held {
    Chunk b[2], a[MF][2];
  };
  struct HeldEnd {
    i32x4 b[2], a[MF][2];
  };
  auto chunk = [&](const uint8_t* p) __attribute__((always_inline)) {
    if constexpr (ODD) {
      return load_odd(p);
    } else {
      i32x4 v;
      __builtin_memcpy(&v, __builtin_assume_aligned(p, 4), 16);
      return v;
    }
  };
  auto fetch_with = [&](auto& h, int slab, auto&& load) __attribute__((always_inline)) {
    const int k = 2 * slab * kSlab + 16 * quad;
    h.b[0] = load(b, k), h.b[1] = load(b, k + 64);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      h.a[i][0] = h.a[i][1] = {};
      if (there[i]) h.a[i][0] = load(a[i], k), h.a[i][1] = load(a[i], k + 64);
    }
  };
  auto fetch = [&](Held& h, int slab) __attribute__((always_inline)) {
    fetch_with(h, slab, [&](const uint8_t* row, int at) __attribute__((always_inline)) { return chunk(row + at); });
  };
  auto multiply = [&](const auto& h) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const i32x4 fb = in_place(h.b[x]);
#pragma unroll
      for (int i = 0; i < MF; ++i) acc[i] = mfma16<E>(fb, in_place(h.a[i][x]), acc[i]);
    }
  };
  // Slabs that can be loaded whole, with ODD's two bytes behind them, and one that cannot.
  const int full = (t.K - (ODD ? 1 : 0)) / kSlab;
  int slab = wave;
  for (; slab + (AHEAD - 1) * NW < full; slab += NW * AHEAD) {
    Held h[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) fetch(h[u], slab + u * NW);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) multiply(h[u]);
  }
#pragma unroll 1
  for (; slab < full; slab += NW) {
    Held h;
    fetch(h, slab);
    multiply(h);
  }
  if (slab == full && t.K > full * kSlab) {  // the wave whose turn the last slab is
    HeldEnd h;
    fetch_with(h, slab, [&](const uint8_t* row, int at) __attribute__((always_inline)) { return load16_end(row, at, 2 * t.K); });
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
    const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    if (m < t.rows_a) store_experts(g, t.C, (int64_t)m * g.ldc + n, g.N - n, v);
  }
}

template <class E, bool ODD>
const void* rows_kernel_of(int bm) {
  return bm == 16   ? (const void*)&experts_rows_kernel<E, 1, ODD>
         : bm == 32 ? (const void*)&experts_rows_kernel<E, 2, ODD>
                    : (const void*)&experts_rows_kernel<E, 4, ODD>;
}
// Whether some row or expert begins at no multiple of four bytes.
bool odd_rows(const ExpertsArgs& g) { return (((uintptr_t)g.A | (uintptr_t)g.B) & 2) != 0 || ((g.lda | g.ldb | g.strideB) & 1) != 0; }
template <class E>
const void* rows_kernel(const ExpertsArgs& g, int bm) {
  return odd_rows(g) ? rows_kernel_of<E, true>(bm) : rows_kernel_of<E, false>(bm);
}
template <class E, bool WIDE>
const void* staged_kernel_of(ExpertsForm form) {
  return form == EXPERTS_FORWARD ? (const void*)&experts_staged_kernel<EXPERTS_FORWARD, E, WIDE>
         : form == EXPERTS_DGRAD ? (const void*)&experts_staged_kernel<EXPERTS_DGRAD, E, WIDE>
                                 : (const void*)&experts_staged_kernel<EXPERTS_WGRAD, E, WIDE>;
}
template <class E>
const void* staged_kernel(ExpertsForm form, const ExpertsArgs& g) {
  const bool wide = (form == EXPERTS_WGRAD ? g.M : g.K) >= 8 && (form == EXPERTS_FORWARD || g.N >= 8);
  return wide ? staged_kernel_of<E, true>(form) : staged_kernel_of<E, false>(form);
}

// The kernel for a call and its tile.
struct Choice {
  enum Kernel { STAGED, TILE, ROWS } kernel;
  int bm, bn, threads;
};

Choice choose(ExpertsForm form, const ExpertsArgs& g) {
  // Direct loads: chunks of 16 bytes that lie in one row, offsets within a tile below 2^31.
  const bool direct = (((uintptr_t)g.A | (uintptr_t)g.B) & 15) == 0 && ((g.lda | g.ldb | g.strideB) & 7) == 0 &&
                      g.lda < 1 << 22 && g.ldb < 1 << 22 && (form == EXPERTS_WGRAD ? g.M % 8 == 0 : g.K >= 8) &&
                      (form == EXPERTS_FORWARD || g.N % 8 == 0);
  const Choice small = direct ? Choice{Choice::TILE, 128, 128, 256} : Choice{Choice::STAGED, 128, 128, 256};
  // The number of BM x BN tiles: an expert with rows has one tile of rows, and
  // half a tile more on average where it has many.
  const int used = g.experts < g.M ? g.experts : g.M < 1 ? 1 : g.M;
  auto tiles = [&](int bm, int bn) {
    const int64_t whole = ((int64_t)g.M + bm - 1) / bm;
    const int64_t tiles_m = form == EXPERTS_WGRAD ? whole * g.experts
                            : g.experts == 1      ? whole
                            : whole + used / 2 > used ? whole + used / 2 : (int64_t)used;
    return (double)tiles_m * (double)(((int64_t)g.N + bn - 1) / bn);
  };
  // 256 x 256 tiles, one to a CU, where tiles of 128 x 128, two to a CU, would
  // need more than one round of the chip, and where they have rows to fill (us,
  // 256 x 256 and 128 x 128 tiles: 8 experts of 512 rows, N 2048, K 4096, 576
  // small tiles 99.7 and 115.8, of 256 rows, 320 of them 80.8 and 64.1; 4200 rows,
  // N and K 2048, 528 of them 41.6 and 49.2; 16 experts of 128 rows, N 2304, K
  // 2048, 432 of them 57.2 and 44.1; weights' gradients of 1024 rows, 2048 x 4096,
  // 512 of them 33.1 and 24.8, of 2048 rows, 2176 x 4096, 544 of them 47.4 and
  // 54.2; 32 experts, N 2048, K 1024, of 128 rows 33.6 and 43.5, of 64 rows 28.7
  // and 25.4).
  if (direct && tiles(128, 128) > 2 * kCUs && (form == EXPERTS_WGRAD || g.M / used >= 96)) return {Choice::TILE, 256, 256, 512};
  if (form != EXPERTS_FORWARD || g.K < 8) return small;
  // The least of the estimated times: for each round of the chip a start and
  // the slabs, or the weights at the rate that the kernel reaches, fitted to 1
  // to 32 experts of 1 to 128 rows, N and K 256 to 4096 (the choice is 1.018
  // of the fastest there on average). Few rows a workgroup load less and begin
  // sooner, but read the weights again for each 16 to 64 rows (8 experts, N
  // 2048, K 4096, rows 16 / 32 / 64 and tiles: of 4 rows 32, 32, 31 and 60, of
  // 32 rows 73, 66, 58 and 60).
  const double k = g.K / 1024.0, weights = (double)used * g.N * (double)g.K * 2.0 / 1.0e6;
  const double rounds = std::ceil(tiles(128, 128) / 512.0);
  Choice best = small;
  // Rows that begin at odd multiples of two bytes cost the few-rows kernel loads
  // and shifts by the rows that there are, and the staged kernel less (16 experts,
  // us, few rows at best and staged: 1224 rows, N 604, K 1817 53 and 36, K 1818 28
  // and 29; 64 rows, N 2048, K 4095 65 and 91).
  const bool odd = odd_rows(g);
  double least = std::fmax(2.3 + rounds * (0.6 + (direct ? 11.0 : odd ? 20.0 : 14.0) * k), 2.0 + weights / 4.8);
  auto offer = [&](int bm, double start, double slabs, double rate) {
    const double r = std::fmax(tiles(bm, 16) / 256.0, 1.0), time = std::fmax(3.2 + r * (start + slabs * k), 2.0 + weights / rate);
    if (time < least) best = {Choice::ROWS, bm, 16, 64 * kRowsWaves}, least = time;
  };
  const double each = (double)g.M / used;  // rows of an expert
  offer(64, 1.08, odd ? 1.9 + 3.9 * std::fmin(each / 64.0, 1.0) : 1.65, odd ? 4.0 : 5.0);
  offer(32, 0.76, odd ? 1.55 + 1.7 * std::fmin(each / 32.0, 1.0) : 1.58, 5.0);
  offer(16, 0.58, odd ? 1.4 + 0.75 * std::fmin(each / 16.0, 1.0) : 1.43, odd ? 5.0 : 5.7);
  return best;
}

}  // namespace

bool experts_launchable(ExpertsForm form, const ExpertsArgs& g) {
  const Choice c = choose(form, g);
  return experts_grid(form, g, c.bm, c.bn) * c.threads <= (int64_t)UINT32_MAX && (form != EXPERTS_WGRAD || g.experts <= kMaxGridY);
}

const char* experts_kernel_name(ExpertsForm form, const ExpertsArgs& g) {
  const Choice c = choose(form, g);
  if (c.kernel == Choice::STAGED) return "staged_128x128";
  if (c.kernel == Choice::TILE) return c.bm == 256 ? "tile_256x256" : "tile_128x128";
  return c.bm == 64 ? "rows_64" : c.bm == 32 ? "rows_32" : "rows_16";
}

hipError_t launch_experts(ExpertsForm form, const ExpertsArgs& g, hipStream_t s) {
  const Choice c = choose(form, g);
  const bool bf16 = g.type == SGEMM_MI355_BF16;
  const dim3 grid((unsigned)experts_grid(form, g, c.bm, c.bn), form == EXPERTS_WGRAD ? (unsigned)g.experts : 1u);
  const void* kernel = c.kernel == Choice::TILE   ? experts_tile_kernel_for(form, g.type, c.bm)
                       : c.kernel == Choice::ROWS ? (bf16 ? rows_kernel<__hip_bfloat16>(g, c.bm) : rows_kernel<__half>(g, c.bm))
                                                  : (bf16 ? staged_kernel<__hip_bfloat16>(form, g) : staged_kernel<__half>(form, g));
  return launch_with(kernel, grid, dim3((unsigned)c.threads), g, s);
}

}  // namespace sgemm_impl
