// Routing of tokens to experts, the order of the experts' rows, and the
// weighted return of those rows (forward and backward).

#include "fp8_internal.h"

namespace sgemm_impl {
namespace {

constexpr int kNone = 0x7FFFFFFF;

// ---- routing ------------------------------------------------------------------
//
// A wave has one token; lane l holds experts l*V .. l*V + V-1. Scores and choice
// values are FP64: two experts whose values differ by less than FP32 tells apart
// are still ordered as the formula orders them, and FP64 vector instructions run
// at the rate of FP32 ones here. Bound by the vector unit: a score is about 70
// instructions, a choice is a reduction over the lanes. 8192 tokens, 8 of 256
// experts from 4 of 8 groups: 13.5 us; 18.6 with groups by way of LDS and a
// search of the lane's experts for each choice instead of a sort before the
// first (1 choice without groups 7.3 us, with the sort 8.7). That form took 52
// with reductions as shuffles through LDS instead of in the vector unit (DPP),
// 24 with loads of single logits and biases under conditions, and 19 with 16
// lanes to a token, so that a reduction serves four tokens (15 where it took 8,
// at 2048 tokens).
//
// A choice value is compared as a 64-bit key whose halves are reduced one after
// the other: the largest first half, then, if several lanes have it, the largest
// second half among them, then the first lane that has both.

template <class T>
__device__ __forceinline__ double to_f64(T x) { return (double)to_f32(x); }

// x of another lane by a DPP control, `none` where there is no such lane.
template <int CONTROL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t x, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, CONTROL, ROWS, 0xF, false);
}
template <int CONTROL, int ROWS>
__device__ __forceinline__ double dpp(double x, double none) {
  const uint64_t b = __double_as_longlong(x), n = __double_as_longlong(none);
  const uint32_t lo = dpp<CONTROL, ROWS>((uint32_t)b, (uint32_t)n), hi = dpp<CONTROL, ROWS>((uint32_t)(b >> 32), (uint32_t)(n >> 32));
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ uint32_t lane_value(uint32_t x, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)x, lane); }
__device__ __forceinline__ double lane_value(double x, int lane) {
  const uint64_t b = __double_as_longlong(x);
  const uint32_t lo = lane_value((uint32_t)b, lane), hi = lane_value((uint32_t)(b >> 32), lane);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// f over all lanes, in every lane: shifts by 1, 2, 4, 8 within rows of 16 lanes,
// then rows 0 to 1 and 2 to 3, then 1 to 3; the last lane has it all.
template <class X, class F>
__device__ __forceinline__ X reduce(X x, X none, F&& f) {
  x = f(x, dpp<0x111, 0xF>(x, none));
  x = f(x, dpp<0x112, 0xF>(x, none));
  x = f(x, dpp<0x114, 0xF>(x, none));
  x = f(x, dpp<0x118, 0xF>(x, none));
  x = f(x, dpp<0x142, 0xA>(x, none));
  x = f(x, dpp<0x143, 0xC>(x, none));
  return lane_value(x, 63);
}
__device__ __forceinline__ uint32_t most_of(uint32_t x) {
  return reduce(x, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ double sum_of(double x) {
  return reduce(x, 0.0, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ double max_of(double x) {
  return reduce(x, (double)-INFINITY, [](double a, double b) { return fmax(a, b); });
}

// Orders like the number, NaN as minus infinity; never 0, which stands for none.
__device__ __forceinline__ uint64_t key_of(double x) {
  if (!(x == x)) x = -INFINITY;
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);  // -0 is 0
  return b >> 63 ? ~b : b | 1ull << 63;
}
// The lanes that hold the largest key.
__device__ __forceinline__ uint64_t lanes_of_most(uint64_t key) {
  const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
  const uint32_t most_hi = most_of(hi);
  const uint64_t lanes = __ballot(hi == most_hi);
  if (__popcll(lanes) == 1) return lanes;
  const uint32_t most_lo = most_of(hi == most_hi ? lo : 0);
  return __ballot(hi == most_hi && lo == most_lo);
}

// A wave's accesses to its own LDS stay in order.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Scores of the token; experts past the last get 0. A NaN logit of a softmax
// makes the whole row NaN.
template <class T, int SCORE, int V>
__device__ __forceinline__ void scores(const T* row, int experts, int l, double (&s)[V]) {
  if (l * V + V <= experts) {
    T x[V];
    __builtin_memcpy(x, row + l * V, sizeof(x));
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = to_f64(x[v]);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = l * V + v < experts ? to_f64(row[l * V + v]) : -INFINITY;
  }
  if constexpr (SCORE == SGEMM_MI355_SOFTMAX) {
    double most = s[0], sum = 0.0;
#pragma unroll
    for (int v = 1; v < V; ++v) most = fmax(most, s[v]);
    most = max_of(most);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = l * V + v < experts ? exp(s[v] - most) : 0.0;
      sum += s[v];
    }
    const double inverse = 1.0 / sum_of(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = l * V + v < experts ? s[v] * inverse : 0.0;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = 1.0 / (1.0 + exp(-s[v]));
    }
  }
}

// Bit v: the lane's expert v is in one of the top_groups strongest groups.
// `row`: room for the token's choice values, `keys` for a key of each group.
template <int V>
__device__ __forceinline__ uint32_t kept_experts(const RouteArgs& a, const double (&c)[V], int l, double* row, uint64_t* keys) {
  const int size = a.experts / a.groups;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (l * V + v < a.experts) row[l * V + v] = c[v];
  wave_sync();
  // L neighbouring lanes find a group's strength, each from every L-th of its
  // experts, beginning at places of their own, so that lanes of different
  // groups read different banks.
  int L = 1;
  while (2 * L * a.groups <= 64) L *= 2;
#pragma unroll 1
  for (int g0 = 0; g0 < a.groups; g0 += 64 / L) {
    const int g = g0 + l / L;
    const int n = g < a.groups ? (size - l % L + L - 1) / L : 0;  // this lane's experts of the group
    double one = -INFINITY, two = -INFINITY;
    int at = n > 0 ? g % n : 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const double x = row[g * size + l % L + at * L];
      two = fmax(two, fmin(one, x));
      one = fmax(one, x);
      at = at + 1 == n ? 0 : at + 1;
    }
#pragma unroll 1
    for (int d = 1; d < L; d *= 2) {
      const double x = __shfl_xor(one, d, 64), y = __shfl_xor(two, d, 64);
      two = fmax(fmin(one, x), fmax(two, y));
      one = fmax(one, x);
    }
    if (g < a.groups && l % L == 0) keys[g] = key_of(size > 1 ? one + two : one);
  }
  wave_sync();
  int* kept = (int*)row;  // of each group, in the values' place
  for (int g = l; g < a.groups; g += 64) kept[g] = 0;
  for (int r = 0; r < a.top_groups; ++r) {
    uint64_t best = 0;
    int mine = 0;
    for (int g = l; g < a.groups; g += 64) {
      const uint64_t k = keys[g];
      if (k > best) best = k, mine = g;
    }
    const uint64_t lanes = lanes_of_most(best);
    int g = (int)lane_value((uint32_t)mine, __builtin_ctzll(lanes));
    // More groups than lanes: of equal ones the lowest need not be the first lane's.
    if (a.groups > 64) g = kNone - (int)most_of(lanes >> l & 1 ? (uint32_t)(kNone - mine) : 0u);
    if (g % 64 == l) keys[g] = 0, kept[g] = 1;
  }
  wave_sync();
  // e / size for e < 1024 as a product: the quotient's excess is under 2^-10.
  const uint32_t inverse = ((1u << 20) + size - 1) / size;
  uint32_t open = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (l * V + v < a.experts && kept[(l * V + v) * inverse >> 20] != 0) open |= 1u << v;
  return open;
}

// With the two largest values of the lane that CONTROL names.
template <int CONTROL>
__device__ __forceinline__ void with_two_of(double& one, double& two) {
  const double x = dpp<CONTROL, 0xF>(one, one), y = dpp<CONTROL, 0xF>(two, two);
  two = fmax(fmin(one, x), fmax(two, y));
  one = fmax(one, x);
}

// The same where a group's experts fill L neighbouring lanes, L a power of 2 of
// at most 16, so that a group lies in one row of 16 lanes: nothing goes through LDS.
template <int V>
__device__ __forceinline__ uint32_t kept_neighbours(const RouteArgs& a, const double (&c)[V], int l, int L) {
  double one = c[0], two = -INFINITY;
#pragma unroll
  for (int v = 1; v < V; ++v) {
    two = fmax(two, fmin(one, c[v]));
    one = fmax(one, c[v]);
  }
  if (L > 1) with_two_of<0xB1>(one, two);   // lane ^ 1
  if (L > 2) with_two_of<0x4E>(one, two);   // lane ^ 2
  if (L > 4) with_two_of<0x141>(one, two);  // 7 - lane of 8
  if (L > 8) with_two_of<0x140>(one, two);  // 15 - lane of 16
  const int first = l & -L;
  uint64_t key = l == first && l < a.groups * L ? key_of(V * L > 1 ? one + two : one) : 0;
  uint64_t kept = 0;  // the kept groups' first lanes
  for (int r = 0; r < a.top_groups; ++r) {
    const int lane = __builtin_ctzll(lanes_of_most(key));
    kept |= 1ull << lane;
    if (l == lane) key = 0;
  }
  return kept >> first & 1 ? 0xFFFFFFFF : 0;
}

template <class T, int SCORE, int V>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
  __shared__ double rows[4][64 * V];  // choice values, then which groups are kept, then scores
  __shared__ uint64_t strengths[4][64 * V];
  const int l = threadIdx.x % 64;
  const int token = blockIdx.x * 4 + threadIdx.x / 64;
  if (token >= a.tokens) return;  // whole waves
  double s[V], c[V];
  scores<T, SCORE, V>((const T*)a.logits + (int64_t)token * a.ld, a.experts, l, s);
  float bias[V] = {};
  if (a.bias != nullptr) {
    if (l * V + V <= a.experts) {
      __builtin_memcpy(bias, a.bias + l * V, sizeof(bias));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) bias[v] = l * V + v < a.experts ? a.bias[l * V + v] : 0.0f;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    c[v] = s[v] + (double)bias[v];
    if (!(c[v] == c[v])) c[v] = -INFINITY;  // NaN ranks as minus infinity
  }
  uint32_t open = 0xFFFFFFFF;
  double* row = rows[threadIdx.x / 64];
  if (a.groups > 1) {
    const int size = a.experts / a.groups, L = size / V;
    open = L * V == size && (L & (L - 1)) == 0 && L <= 16 ? kept_neighbours<V>(a, c, l, L)
                                                          : kept_experts<V>(a, c, l, row, strengths[threadIdx.x / 64]);
  }
  uint64_t key[V];
  int at[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = l * V + v < a.experts && (open >> v & 1) ? key_of(c[v]) : 0, at[v] = v;
  wave_sync();
#pragma unroll
  for (int v = 0; v < V; ++v) row[l * V + v] = s[v];
  // A lane's experts in their order, equal ones by index, so that a choice takes
  // the first of them and moves up the rest. More than 4 are searched anew for
  // each choice instead, since the sort grows with their square.
  constexpr bool SORTED = V <= 4;
  if constexpr (SORTED) {
#pragma unroll
    for (int round = 0; round < V; ++round)
#pragma unroll
      for (int v = round % 2; v + 1 < V; v += 2) {
        const bool swap = key[v + 1] > key[v];
        const uint64_t high = swap ? key[v + 1] : key[v], low = swap ? key[v] : key[v + 1];
        const int first = swap ? at[v + 1] : at[v], second = swap ? at[v] : at[v + 1];
        key[v] = high, key[v + 1] = low, at[v] = first, at[v + 1] = second;
      }
  }
  uint32_t order = 0;  // the experts' numbers in the lane, a byte each
  if constexpr (SORTED) {
#pragma unroll
    for (int v = 0; v < V; ++v) order |= (uint32_t)at[v] << (8 * v);
  }
  int id = 0;  // of choice l
  for (int k = 0; k < a.choices; ++k) {
    uint64_t best = key[0];
    if constexpr (!SORTED) {
      order = 0;
#pragma unroll
      for (int v = 1; v < V; ++v)
        if (key[v] > best) best = key[v], order = v;
    }
    const int owner = __builtin_ctzll(lanes_of_most(best));
    const int chosen = owner * V + (int)(lane_value(order, owner) & 0xFF);
    if (l == k) id = chosen;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (SORTED) {
        key[v] = l != owner ? key[v] : v + 1 < V ? key[v + 1] : 0;
      } else if (l == owner && v == (int)order) {
        key[v] = 0;
      }
    }
    if constexpr (SORTED) order = l != owner ? order : order >> 8;
  }
  wave_sync();
  double w = l < a.choices ? row[id] : 0.0;
  if (a.renorm) {
    const double total = sum_of(w);
    w = total == 0.0 ? 0.0 : w / total;
  }
  if (l < a.choices) {
    a.weights[(int64_t)token * a.choices + l] = (float)((double)a.scale * w);
    a.ids[(int64_t)token * a.choices + l] = id;
  }
}

// A wave has one token, lane k its choice k. A sigmoid's gradient needs the
// chosen experts' scores alone; a softmax's needs the whole row.
// Nothing is computed as a difference of nearly equal numbers that is small by
// the formula: 1 - s of a sigmoid comes from the exponential, and a weighted
// mean is taken of the differences from the value of the largest score, which
// may be nearly the whole weight (dw_j - sum_m dw_m s_m / S with S nearly one
// s_m, and ds_i - sum_m ds_m s_m with one s_m nearly 1).
template <class T, int SCORE, int V>
__global__ void __launch_bounds__(256) route_backward_kernel(RouteArgs a) {
  __shared__ double rows[4][64 * V];  // scores, then the lanes of the chosen experts' choices, then their gradients
  const int lane = threadIdx.x % 64;
  const int token = blockIdx.x * 4 + threadIdx.x / 64;
  if (token >= a.tokens) return;
  const T* logits = (const T*)a.logits + (int64_t)token * a.ld;
  int id = -1;
  double dw = 0.0, w = 0.0, rest = 0.0;  // rest: 1 - w of a sigmoid
  if (lane < a.choices) {
    id = a.ids_in[(int64_t)token * a.choices + lane];
    if ((unsigned)id >= (unsigned)a.experts) id = -1;
    else dw = (double)a.dweights[(int64_t)token * a.choices + lane];
  }
  double s[V];
  double* row = rows[threadIdx.x / 64];
  if constexpr (SCORE == SGEMM_MI355_SOFTMAX) {
    scores<T, SCORE, V>(logits, a.experts, lane, s);
#pragma unroll
    for (int v = 0; v < V; ++v) row[lane * V + v] = s[v];
    wave_sync();
    if (id >= 0) w = row[id];
  } else if (id >= 0) {
    const double x = to_f64(logits[id]), t = exp(-fabs(x)), one = 1.0 / (1.0 + t);
    w = x < 0.0 ? t * one : one;
    rest = x < 0.0 ? one : t * one;
  }
  double most = 0.0;  // the largest of the chosen scores, and a choice that has it
  int first = 0;
  if (SCORE == SGEMM_MI355_SOFTMAX || a.renorm) {
    most = max_of(w);
    const uint64_t lanes = __ballot(w == most);
    if (lanes != 0) first = __builtin_ctzll(lanes);  // none: NaN
  }
  // total = S, dot = sum of dw_m s_m over the chosen
  double total = 1.0, dot = 0.0;
  if (a.renorm) {
    dw -= lane_value(dw, first);
    total = sum_of(w), dot = sum_of(w * dw);
  }
  double d = id < 0 || total == 0.0 ? 0.0 : (double)a.scale * (dw - dot / total) / total;
  if constexpr (SCORE == SGEMM_MI355_SIGMOID) d = d * w * rest;
  // Through LDS to the lanes that hold the experts (8192 tokens, 8 of 256: 6.4 us;
  // 8.5 with every choice compared with all experts). Experts that are chosen
  // more than once are found first, and added up in the choices' order.
  double ds[V] = {};
  wave_sync();
  if (id >= 0) *(int*)&row[id] = lane;
  wave_sync();
  const bool twice = __ballot(id >= 0 && *(int*)&row[id >= 0 ? id : 0] != lane) != 0;
  wave_sync();
  if (!twice) {
#pragma unroll
    for (int v = 0; v < V; ++v) row[lane * V + v] = 0.0;
    wave_sync();
    if (id >= 0) row[id] = d;
    wave_sync();
#pragma unroll
    for (int v = 0; v < V; ++v) ds[v] = row[lane * V + v];
  } else {
    for (int k = 0; k < a.choices; ++k) {
      const int e = (int)lane_value((uint32_t)id, k);
      const double x = lane_value(d, k);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e == lane * V + v) ds[v] += x;
    }
  }
  if constexpr (SCORE == SGEMM_MI355_SOFTMAX) {
    if (most > 0.5) {  // else no score is nearly 1, or one that was not chosen, whose ds is 0
      const int e = (int)lane_value((uint32_t)id, first);
      double base = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e % V == v) base = lane_value(ds[v], e / V);
#pragma unroll
      for (int v = 0; v < V; ++v) ds[v] -= base;
    }
    double inner = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) inner += ds[v] * s[v];
    inner = sum_of(inner);
#pragma unroll
    for (int v = 0; v < V; ++v) ds[v] = s[v] * (ds[v] - inner);
  }
  float out[V];
#pragma unroll
  for (int v = 0; v < V; ++v) out[v] = (float)ds[v];
  float* to = a.dlogits + (int64_t)token * a.ldd + lane * V;
  if (lane * V + V <= a.experts) {
    __builtin_memcpy(to, out, sizeof(out));
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane * V + v < a.experts) to[v] = out[v];
  }
}

// ---- the order of the experts' rows ---------------------------------------------
//
// A counting sort that keeps the order of equal ids. The entries are cut into
// runs of kPlanRun, one to a workgroup of 16 waves with 1/16 of the run each.
// With several runs the first kernel counts each run's entries of each expert.
// In the second a run adds up the counts before it, and each of its waves,
// having counted its own entries, knows where its first of each expert goes;
// then the waves place theirs without waiting for each other. Ids outside the
// experts count as expert number `experts`, the last.
//
// Every run reading the counts of all runs is work of their square. Where there
// are many, the first kernel takes a group of neighbouring runs to a workgroup,
// one after the other, and writes for each run what its group has before it; a
// kernel between the two adds up the groups; and a run reads three numbers of
// each expert (1048576 tokens of 8 of 256 experts: 107 us, 1363 without groups).

__device__ __forceinline__ int expert_of(const PlanArgs& p, int entry) {
  const int id = p.ids[entry];
  return (unsigned)id < (unsigned)p.experts ? id : p.experts;
}

__global__ void __launch_bounds__(1024) plan_count_kernel(PlanArgs p) {
  __shared__ int count[SGEMM_MI355_MAX_EXPERTS + 1];
  for (int e = threadIdx.x; e <= p.experts; e += 1024) count[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * kPlanRun;
#pragma unroll
  for (int i = 0; i < kPlanRun / 1024; ++i) {
    const int entry = first + i * 1024 + threadIdx.x;
    if (entry < p.entries) atomicAdd(&count[expert_of(p, entry)], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= p.experts; e += 1024) p.counts[(int64_t)blockIdx.x * (p.experts + 1) + e] = count[e];
}

// Rows of counts after those of the runs: the entries before each group, and all.
__device__ __forceinline__ int* group_counts(const PlanArgs& p, int group) {
  return p.counts + ((int64_t)p.runs + group) * (p.experts + 1);
}

__global__ void __launch_bounds__(1024) plan_group_kernel(PlanArgs p) {
  constexpr int PER = kPlanRun / 1024;
  __shared__ int count[SGEMM_MI355_MAX_EXPERTS + 1];
  const int t = threadIdx.x, width = p.experts + 1;
  const int from = blockIdx.x * p.per, to = min(from + p.per, p.runs);
  for (int e = t; e < width; e += 1024) count[e] = 0;
  int expert[PER];
  auto load = [&](int run) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int entry = run * kPlanRun + i * 1024 + t;
      expert[i] = entry < p.entries ? expert_of(p, entry) : -1;
    }
  };
  load(from);
  __syncthreads();
  for (int run = from; run < to; ++run) {
    for (int e = t; e < width; e += 1024) p.counts[(int64_t)run * width + e] = count[e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (expert[i] >= 0) atomicAdd(&count[expert[i]], 1);
    if (run + 1 < to) load(run + 1);
    // The additions are done before the barrier: with the barrier at the loop's
    // head, the compiler has left out its wait for them.
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __syncthreads();
  }
  for (int e = t; e < width; e += 1024) group_counts(p, blockIdx.x)[e] = count[e];
}

// A lane has an expert and a wave 1/16 of the groups: their entries become those
// before them.
__global__ void __launch_bounds__(1024) plan_sum_kernel(PlanArgs p) {
  constexpr int WAVES = 16, MOST = kPlanGroups / WAVES;
  __shared__ int part[WAVES][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, e = blockIdx.x * 64 + lane;
  const bool there = e <= p.experts;
  const int each = (p.groups + WAVES - 1) / WAVES, from = wave * each;
  int c[MOST], own = 0;
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    c[i] = there && i < each && from + i < p.groups ? group_counts(p, from + i)[e] : 0;
    own += c[i];
  }
  part[wave][lane] = own;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += part[w][lane];
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    if (there && i < each && from + i < p.groups) group_counts(p, from + i)[e] = before;
    before += c[i];
  }
  if (there && wave == WAVES - 1) group_counts(p, p.groups)[e] = before;
}

// Lanes of the wave that have the same key (of `bits` bits).
__device__ __forceinline__ uint64_t same_key(int key, bool active, int bits) {
  uint64_t same = __ballot(active);
  for (int b = 0; b < bits; ++b) {
    const uint64_t ones = __ballot(active && (key >> b & 1));
    same &= (key >> b & 1) ? ones : ~ones;
  }
  return same;
}

__global__ void __launch_bounds__(1024) plan_place_kernel(PlanArgs p) {
  constexpr int WAVES = 16, PER = kPlanRun / WAVES / 64;  // entries per lane
  // next[w][e]: first the wave's entries of expert e, then the row of its next one.
  __shared__ int next[WAVES * (SGEMM_MI355_MAX_EXPERTS + 1)];
  __shared__ int in_all[SGEMM_MI355_MAX_EXPERTS + 1], in_earlier[SGEMM_MI355_MAX_EXPERTS + 1];
  __shared__ int wave_total[WAVES];
  const int t = threadIdx.x, lane = t % 64, wave = t / 64, width = p.experts + 1;
  for (int i = t; i < WAVES * width; i += 1024) next[i] = 0;
  __syncthreads();
  const int first = blockIdx.x * kPlanRun + wave * (kPlanRun / WAVES);
  int expert[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int entry = first + i * 64 + lane;
    expert[i] = entry < p.entries ? expert_of(p, entry) : -1;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (expert[i] >= 0) atomicAdd(&next[wave * width + expert[i]], 1);
  __syncthreads();
  if (p.per > 0) {
    const int* group = group_counts(p, blockIdx.x / p.per);
    const int* all = group_counts(p, p.groups);
    for (int e = t; e < width; e += 1024) {
      in_all[e] = all[e];
      in_earlier[e] = group[e] + p.counts[(int64_t)blockIdx.x * width + e];
    }
    __syncthreads();
  } else if (p.runs > 1) {
    // Of each expert, the entries in all runs and those in the runs before this
    // one: the threads share the runs, and add up their parts in LDS (65536
    // tokens of 8 choices: 18 us, 42 with a thread for each expert).
    for (int e = t; e < width; e += 1024) in_all[e] = in_earlier[e] = 0;
    __syncthreads();
    const int parts = width < 1024 ? 1024 / width : 1;
    for (int i = t; i < parts * width; i += 1024) {
      const int part = i / width, e = i - part * width;
      int here = 0, all = 0;
#pragma unroll 8
      for (int r = part; r < p.runs; r += parts) {
        const int c = p.counts[(int64_t)r * width + e];
        all += c;
        if (r < (int)blockIdx.x) here += c;
      }
      if (all > 0) atomicAdd(&in_all[e], all);
      if (here > 0) atomicAdd(&in_earlier[e], here);
    }
    __syncthreads();
  }
  int carry = 0;  // entries of all experts before this turn's
  for (int e0 = 0; e0 < width; e0 += 1024) {
    const int e = e0 + t;
    int here = 0, all = 0;
    if (e < width) {
      if (p.runs == 1) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) all += next[w * width + e];
      } else {
        here = in_earlier[e], all = in_all[e];
      }
    }
    int upto = all;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int x = __shfl_up(upto, d, 64);
      if (lane >= d) upto += x;
    }
    if (lane == 63) wave_total[wave] = upto;
    __syncthreads();
    int base = carry;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      base += w < wave ? wave_total[w] : 0;
      carry += wave_total[w];
    }
    if (e < width) {
      if (blockIdx.x == 0) p.offsets[e] = base + upto - all;
      int row = base + upto - all + here;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int c = next[w * width + e];
        next[w * width + e] = row;
        row += c;
      }
    }
    __syncthreads();
  }
  const int bits = 32 - __builtin_clz(width);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = expert[i], entry = first + i * 64 + lane;
    const uint64_t same = same_key(e, e >= 0, bits);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = 0;
    if (e >= 0) row = next[wave * width + e] + rank;
    __builtin_amdgcn_wave_barrier();  // the wave's reads before its writes
    if (e >= 0 && rank == 0) next[wave * width + e] = row + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (e >= 0) {
      p.place[entry] = row;
      p.row_token[row] = entry / p.choices;
    }
  }
}

// ---- the rows' return --------------------------------------------------------------
//
// Bound by the bytes of Z and dZ. A place and a weight are the same for a whole
// wave, so they are scalars; forward, 4 rows of Z are asked for at once. Z is
// read and Y and dZ are written past the caches (each once). 4096 tokens of 8
// choices of 4096 bf16 columns: 51 us forward (5.7 TB/s) and 115 back (4.9
// TB/s; 111 without the search for rows that have no name). Back with a token to a workgroup, 2 of its rows at a time,
// 121 (512 columns, 16384 tokens: 127, here 59); with 2, 4, 8 pieces of a row at
// once 117, 118, 151: their registers leave fewer waves. Few tokens of long
// rows are slower this way (8 of 2 choices, 16384 columns: 16.5 us, 13.6).

constexpr int kRows = 4;

// A wave has 512 columns of one token and adds the choices in order.
template <class T>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a, int slabs) {
  const int64_t item = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t token = item / slabs;
  if (token >= a.tokens) return;
  const int col = (int)(item - token * slabs) * 512 + 8 * (threadIdx.x % 64);
  const int valid = a.cols - col;
  const int* place = a.place + token * a.choices;
  const float* weights = a.weights + token * a.choices;
  float y[8] = {};
  for (int j0 = 0; j0 < a.choices; j0 += kRows) {
    float z[kRows][8], w[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int row = j0 + j < a.choices ? place[j0 + j] : -1;
      const bool there = (unsigned)row < (unsigned)a.rows;
      w[j] = there ? weights[j0 + j] : 0.0f;
      load8_once((const T*)a.Z + (int64_t)(there ? row : 0) * a.ldz + col, there ? valid : 0, z[j]);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(w[j], z[j][i], y[i]);
  }
  store8_once((T*)a.Y + token * a.ldy + col, valid, y);
}

// Zeros in the rows of dZ that no place names, of the `each` rows of this
// workgroup: a bit for each in LDS, and all places are read. Workgroups of the
// gradient's own launch do it, while the others wait for memory: 4096 tokens of
// 8 rows of 4096 126 us, 123 without; 16384 of 512 columns 60.4, 59.2; 1048576
// of 64 columns 2.47 ms, 2.39 (as a launch of its own 128, 75, 3.3 ms). With 32 or
// 256 such workgroups 16384 of 512 columns take 59.6 or 62.6, and with as many
// unnamed rows more 298 or 87, 110 with these.
constexpr int kZeroGroups = 128;
constexpr int kMostNamed = 1 << 17;  // rows of one of them

template <class T>
__device__ __forceinline__ void zero_unnamed_rows(const CombineArgs& a, int each, uint32_t* named) {
  typedef int ints __attribute__((ext_vector_type(4), aligned(4)));
  const int first = (int)blockIdx.x * each, rows = min(each, a.rows - first), words = (rows + 31) / 32;
  for (int w = threadIdx.x; w < words; w += 256) named[w] = 0;
  __syncthreads();
  auto name = [&](int place) {
    const uint32_t r = (uint32_t)place - (uint32_t)first;
    if (r < (uint32_t)rows) atomicOr(&named[r / 32], 1u << (r % 32));
  };
  constexpr int DEEP = 8;  // loads in flight
  const int entries = a.tokens * a.choices, whole = entries / (1024 * DEEP) * (1024 * DEEP);
  for (int i = 4 * threadIdx.x; i < whole; i += 1024 * DEEP) {
    ints p[DEEP];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) p[d] = *(const ints*)(a.place + i + 1024 * d);
#pragma unroll
    for (int d = 0; d < DEEP; ++d) name(p[d][0]), name(p[d][1]), name(p[d][2]), name(p[d][3]);
  }
#pragma unroll 8
  for (int i = whole + threadIdx.x; i < entries; i += 256) name(a.place[i]);
  __syncthreads();
  for (int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64); w < words; w += 4) {
    const uint32_t there = 32 * w + 32 <= rows ? ~0u : (1u << (rows % 32)) - 1;
    uint32_t left = __builtin_amdgcn_readfirstlane(~named[w] & there);
    for (; left != 0; left &= left - 1) {
      T* to = (T*)a.dZ + (int64_t)(first + 32 * w + __builtin_ctz(left)) * a.lddz;
      const float zeros[8] = {};
      for (uint32_t col = 8 * (threadIdx.x % 64); col < (uint32_t)a.cols; col += 512)
        store8_once(to + col, (int)((uint32_t)a.cols - col), zeros);
    }
  }
}

// A wave has one choice of a token, and so a row of Z and dZ: nothing is shared
// between waves, and nothing waits for another row's sum. The first `zeros`
// workgroups look for the rows without a name meanwhile.
template <class T>
__global__ void __launch_bounds__(256) combine_backward_kernel(CombineArgs a, int zeros, int each) {
  __shared__ uint32_t named[kMostNamed / 32];
  if ((int)blockIdx.x < zeros) return zero_unnamed_rows<T>(a, each, named);
  const int64_t item = (int64_t)(blockIdx.x - zeros) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t token = item / a.choices;
  if (token >= a.tokens) return;
  const int lane = threadIdx.x % 64, row = a.place[item];
  float dot = 0.0f;
  if ((unsigned)row < (unsigned)a.rows) {
    const float w = a.weights[item];
    const T* dy = (const T*)a.dY + token * a.lddy;
    const T* from = (const T*)a.Z + (int64_t)row * a.ldz;
    T* to = (T*)a.dZ + (int64_t)row * a.lddz;
    for (uint32_t col = 8 * lane; col < (uint32_t)a.cols; col += 512) {
      const int valid = (int)((uint32_t)a.cols - col);
      float g[8], z[8], d[8];
      load8(dy + col, valid, g);
      load8_once(from + col, valid, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(g[i], z[i], dot), d[i] = g[i] * w;
      store8_once(to + col, valid, d);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) dot += __shfl_xor(dot, d, 64);
  if (lane == 0) a.dweights[item] = dot;
}

// Zeros in all of dZ, before the gradient, where there are more rows than those
// workgroups have bits for.
template <class T>
__global__ void __launch_bounds__(256) zero_rows_kernel(CombineArgs a) {
  const float zeros[8] = {};
  for (int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; r < a.rows; r += (int64_t)gridDim.x * 4)
    for (uint32_t col = 8 * (threadIdx.x % 64); col < (uint32_t)a.cols; col += 512)
      store8_once((T*)a.dZ + r * a.lddz + col, (int)((uint32_t)a.cols - col), zeros);
}

// f(V) for the least V of 1, 2, 4, 8, 16 with 64 V >= experts.
template <class F>
hipError_t by_width(int experts, F&& f) {
  if (experts <= 64) return f(std::integral_constant<int, 1>{});
  if (experts <= 128) return f(std::integral_constant<int, 2>{});
  if (experts <= 256) return f(std::integral_constant<int, 4>{});
  if (experts <= 512) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_route(int type, int score, const RouteArgs& r, hipStream_t s) {
  const dim3 grid((unsigned)((r.tokens + 3) / 4));
  return by_type(type, [&](auto t) {
    return by_width(r.experts, [&](auto v) {
      return launch_with(score == SGEMM_MI355_SOFTMAX
                             ? (const void*)&route_kernel<decltype(t), SGEMM_MI355_SOFTMAX, decltype(v)::value>
                             : (const void*)&route_kernel<decltype(t), SGEMM_MI355_SIGMOID, decltype(v)::value>,
                         grid, dim3(256), r, s);
    });
  });
}

hipError_t launch_route_backward(int type, int score, const RouteArgs& r, hipStream_t s) {
  const dim3 grid((unsigned)((r.tokens + 3) / 4));
  return by_type(type, [&](auto t) {
    return by_width(r.experts, [&](auto v) {
      return launch_with(score == SGEMM_MI355_SOFTMAX
                             ? (const void*)&route_backward_kernel<decltype(t), SGEMM_MI355_SOFTMAX, decltype(v)::value>
                             : (const void*)&route_backward_kernel<decltype(t), SGEMM_MI355_SIGMOID, decltype(v)::value>,
                         grid, dim3(256), r, s);
    });
  });
}

hipError_t launch_route_plan(const PlanArgs& p, hipStream_t s) {
  hipError_t err = hipSuccess;
  if (p.per > 0) {
    err = launch_with((const void*)&plan_group_kernel, dim3((unsigned)p.groups), dim3(1024), p, s);
    if (err == hipSuccess)
      err = launch_with((const void*)&plan_sum_kernel, dim3((unsigned)(p.experts / 64 + 1)), dim3(1024), p, s);
  } else if (p.runs > 1) {
    err = launch_with((const void*)&plan_count_kernel, dim3((unsigned)p.runs), dim3(1024), p, s);
  }
  if (err != hipSuccess) return err;
  return launch_with((const void*)&plan_place_kernel, dim3((unsigned)p.runs), dim3(1024), p, s);
}

hipError_t launch_combine(int type, const CombineArgs& c, hipStream_t s) {
  int slabs = (c.cols + 511) / 512;
  const int64_t items = (int64_t)slabs * c.tokens;
  return by_type(type, [&](auto t) {
    CombineArgs copy = c;
    void* args[] = {&copy, &slabs};
    return hipLaunchKernel((const void*)&combine_kernel<decltype(t)>, dim3((unsigned)((items + 3) / 4)), dim3(256), args, 0, s);
  });
}

hipError_t launch_combine_backward(int type, const CombineArgs& c, hipStream_t s) {
  const int64_t blocks = ((int64_t)c.tokens * c.choices + 3) / 4;
  int each = (int)(((int64_t)c.rows + kZeroGroups - 1) / kZeroGroups);
  int zeros = c.rows > 0 && c.cols > 0 ? (c.rows + each - 1) / each : 0;
  // A launch counts its threads in 32 bits.
  const bool apart = each > kMostNamed || (blocks + zeros) * 256 > (int64_t)UINT32_MAX;
  if (apart) zeros = 0;
  return by_type(type, [&](auto t) {
    if (apart) {
      const hipError_t err = launch_with((const void*)&zero_rows_kernel<decltype(t)>, dim3(8192), dim3(256), c, s);
      if (err != hipSuccess) return err;
    }
    CombineArgs copy = c;
    void* args[] = {&copy, &zeros, &each};
    return hipLaunchKernel((const void*)&combine_backward_kernel<decltype(t)>, dim3((unsigned)(zeros + blocks)), dim3(256), args, 0, s);
  });
}

}  // namespace sgemm_impl
