// Routing of tokens to experts, the order of the experts' rows, and the
// weighted return of those rows (forward and backward).

#include "fp8_internal.h"

namespace sgemm_impl {
namespace {

// ---- routing ------------------------------------------------------------------
//
// One wave has one token; lane l holds experts l, l + 64, ... (V of them).
// Scores and choice values are FP64: two experts whose values differ by less
// than FP32 tells apart are still ordered as the formula orders them, and
// FP64 vector instructions run at the rate of FP32 ones here.

template <class T>
__device__ __forceinline__ double to_f64(T x) { return (double)to_f32(x); }

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d, 64);
  return x;
}
__device__ __forceinline__ double wave_max(double x) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x = fmax(x, __shfl_xor(x, d, 64));
  return x;
}

// Scores of the wave's token; experts past the last get 0. A NaN logit of a
// softmax makes the whole row NaN.
template <class T, int SCORE, int V>
__device__ __forceinline__ void scores(const T* row, int experts, int lane, double (&s)[V]) {
  if constexpr (SCORE == SGEMM_MI355_SOFTMAX) {
    double most = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 64 * v;
      s[v] = e < experts ? to_f64(row[e]) : -INFINITY;
      most = fmax(most, s[v]);
    }
    most = wave_max(most);
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = lane + 64 * v < experts ? exp(s[v] - most) : 0.0;
      sum += s[v];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = lane + 64 * v < experts ? s[v] / sum : 0.0;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 64 * v;
      s[v] = e < experts ? 1.0 / (1.0 + exp(-to_f64(row[e]))) : 0.0;
    }
  }
}

// (value, index) pairs: the larger value first, of equal values the lower
// index. Values are never NaN here.
__device__ __forceinline__ bool before(double a, int ia, double b, int ib) {
  return a > b || (a == b && ia < ib);
}
__device__ __forceinline__ void wave_first(double& x, int& i) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double y = __shfl_xor(x, d, 64);
    const int j = __shfl_xor(i, d, 64);
    if (before(y, j, x, i)) x = y, i = j;
  }
}

// The index that goes with no expert: behind every expert of equal value.
constexpr int kNone = 0x7FFFFFFF;

template <class T, int SCORE, int V>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
  const int lane = threadIdx.x % 64;
  const int token = blockIdx.x * 4 + threadIdx.x / 64;
  if (token >= a.tokens) return;  // whole waves
  double s[V], c[V];
  scores<T, SCORE, V>((const T*)a.logits + (int64_t)token * a.ld, a.experts, lane, s);
  uint32_t open = 0;  // bit v: the lane's expert v can be chosen
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    if (e < a.experts) open |= 1u << v;
    c[v] = s[v];
    if (a.bias != nullptr && e < a.experts) c[v] += (double)a.bias[e];
    if (!(c[v] == c[v])) c[v] = -INFINITY;  // NaN ranks as minus infinity
  }
  if (a.groups > 1) {
    const int size = a.experts / a.groups;
    // A group's strength, on the lane that has its number (modulo 64).
    double strength[V];
#pragma unroll
    for (int v = 0; v < V; ++v) strength[v] = -INFINITY;
    for (int g = 0; g < a.groups; ++g) {
      double one = -INFINITY, two = -INFINITY;
      int at = kNone;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = lane + 64 * v;
        if (e / size == g && e < a.experts && before(c[v], e, one, at)) one = c[v], at = e;
      }
      wave_first(one, at);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = lane + 64 * v;
        if (e / size == g && e < a.experts && e != at) two = fmax(two, c[v]);
      }
      two = wave_max(two);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (lane + 64 * v == g) {
          const double x = size > 1 ? one + two : one;
          strength[v] = x == x ? x : -INFINITY;  // infinities of both signs
        }
    }
    uint32_t kept = 0;
    uint32_t left = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + 64 * v < a.groups) left |= 1u << v;
    for (int r = 0; r < a.top_groups; ++r) {
      double x = -INFINITY;
      int i = kNone;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if ((left >> v & 1) && before(strength[v], lane + 64 * v, x, i)) x = strength[v], i = lane + 64 * v;
      wave_first(x, i);
      if (i % 64 == lane) left &= ~(1u << (i / 64));
#pragma unroll
      for (int v = 0; v < V; ++v)
        if ((lane + 64 * v) / size == i) kept |= 1u << v;
    }
    open &= kept;
  }
  double total = 0.0, mine = 0.0;
  int my_id = 0;
  for (int k = 0; k < a.choices; ++k) {
    double x = -INFINITY, w = 0.0;
    int i = kNone;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if ((open >> v & 1) && before(c[v], lane + 64 * v, x, i)) x = c[v], i = lane + 64 * v, w = s[v];
    const int local = i;
    wave_first(x, i);
    const uint64_t owner = __ballot(local == i);
    w = __shfl(w, __builtin_ctzll(owner), 64);
    if (local == i) open &= ~(1u << (i / 64));
    total += w;
    if (lane == k) mine = w, my_id = i;
  }
  if (lane < a.choices) {
    double w = mine;
    if (a.renorm) w = total == 0.0 ? 0.0 : w / total;
    a.weights[(int64_t)token * a.choices + lane] = (float)((double)a.scale * w);
    a.ids[(int64_t)token * a.choices + lane] = my_id;
  }
}

template <class T, int SCORE, int V>
__global__ void __launch_bounds__(256) route_backward_kernel(RouteArgs a) {
  const int lane = threadIdx.x % 64;
  const int token = blockIdx.x * 4 + threadIdx.x / 64;
  if (token >= a.tokens) return;
  double s[V], ds[V];
  scores<T, SCORE, V>((const T*)a.logits + (int64_t)token * a.ld, a.experts, lane, s);
#pragma unroll
  for (int v = 0; v < V; ++v) ds[v] = 0.0;
  // total = S, dot = sum of dw_m s_m over the chosen
  double total = 0.0, dot = 0.0;
  for (int k = 0; k < a.choices; ++k) {
    const int id = a.ids_in[(int64_t)token * a.choices + k];
    if ((unsigned)id >= (unsigned)a.experts) continue;
    double w = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (id / 64 == v) w = s[v];
    w = __shfl(w, id % 64, 64);
    total += w;
    dot += w * (double)a.dweights[(int64_t)token * a.choices + k];
  }
  if (!a.renorm) total = 1.0, dot = 0.0;
  for (int k = 0; k < a.choices; ++k) {
    const int id = a.ids_in[(int64_t)token * a.choices + k];
    if ((unsigned)id >= (unsigned)a.experts) continue;
    const double d = total == 0.0 ? 0.0
        : (double)a.scale * ((double)a.dweights[(int64_t)token * a.choices + k] - dot / total) / total;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (id == lane + 64 * v) ds[v] += d;
  }
  if constexpr (SCORE == SGEMM_MI355_SOFTMAX) {
    double inner = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) inner += ds[v] * s[v];
    inner = wave_sum(inner);
#pragma unroll
    for (int v = 0; v < V; ++v) ds[v] = s[v] * (ds[v] - inner);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) ds[v] = ds[v] * s[v] * (1.0 - s[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane + 64 * v < a.experts) a.dlogits[(int64_t)token * a.ldd + lane + 64 * v] = (float)ds[v];
}

// ---- the order of the experts' rows ---------------------------------------------
//
// A counting sort that keeps the order of equal ids. The entries are cut into
// runs of kPlanRun. The first kernel counts each run's entries of each expert;
// in the second every run adds up the counts before it and places its own.
// Ids outside the experts count as expert number `experts`, the last.

__device__ __forceinline__ int expert_of(const PlanArgs& p, int entry) {
  const int id = p.ids[entry];
  return (unsigned)id < (unsigned)p.experts ? id : p.experts;
}

__global__ void __launch_bounds__(256) plan_count_kernel(PlanArgs p) {
  __shared__ int count[SGEMM_MI355_MAX_EXPERTS + 1];
  for (int e = threadIdx.x; e <= p.experts; e += 256) count[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * kPlanRun;
  for (int i = first + threadIdx.x; i < min(first + kPlanRun, p.entries); i += 256) atomicAdd(&count[expert_of(p, i)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.experts; e += 256) p.counts[(int64_t)blockIdx.x * (p.experts + 1) + e] = count[e];
}

// Lanes of the wave that have the same key (of keys under 2048).
__device__ __forceinline__ uint64_t same_key(int key, bool active) {
  uint64_t same = __ballot(active);
#pragma unroll
  for (int b = 0; b < 11; ++b) {
    const uint64_t ones = __ballot(active && (key >> b & 1));
    same &= (key >> b & 1) ? ones : ~ones;
  }
  return same;
}

__global__ void __launch_bounds__(256) plan_place_kernel(PlanArgs p, int runs) {
  __shared__ int next[SGEMM_MI355_MAX_EXPERTS + 1];  // the row of the run's next entry of each expert
  __shared__ int wave_total[4];
  const int t = threadIdx.x, lane = t % 64, wave = t / 64;
  int carry = 0;  // entries of all experts before this turn's
  for (int e0 = 0; e0 <= p.experts; e0 += 256) {
    const int e = e0 + t;
    int here = 0, all = 0;
    if (e <= p.experts) {
      for (int r = 0; r < runs; ++r) {
        const int c = p.counts[(int64_t)r * (p.experts + 1) + e];
        all += c;
        if (r < (int)blockIdx.x) here += c;
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
    for (int w = 0; w < wave; ++w) base += wave_total[w];
    if (e <= p.experts) {
      next[e] = base + upto - all + here;
      if (blockIdx.x == 0) p.offsets[e] = base + upto - all;
    }
    carry += wave_total[0] + wave_total[1] + wave_total[2] + wave_total[3];
    __syncthreads();
  }
  const int first = blockIdx.x * kPlanRun;
  const int last = min(first + kPlanRun, p.entries);
  for (int i0 = first; i0 < last; i0 += 256) {
    const int i = i0 + t;
    const bool active = i < last;
    const int e = active ? expert_of(p, i) : 0;
    const uint64_t same = same_key(e, active);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = 0;
    for (int w = 0; w < 4; ++w) {  // the waves in order
      if (wave == w && active) {
        row = next[e] + rank;
      }
      __syncthreads();
      if (wave == w && active && rank == 0) next[e] += __popcll(same);
      __syncthreads();
    }
    if (active) {
      p.place[i] = row;
      p.row_token[row] = i / p.choices;
    }
  }
}

// ---- the rows' return --------------------------------------------------------------

// A thread has eight columns of one token and adds the choices in order.
template <class T>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a, int chunks) {
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t token = item / chunks;
  if (token >= a.tokens) return;
  const int col = (int)(item - token * chunks) * 8;
  const int valid = a.cols - col;
  float y[8] = {};
  for (int j = 0; j < a.choices; ++j) {
    const int row = a.place[token * a.choices + j];
    if ((unsigned)row >= (unsigned)a.rows) continue;
    const float w = a.weights[token * a.choices + j];
    float z[8];
    load8((const T*)a.Z + (int64_t)row * a.ldz + col, valid, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(w, z[i], y[i]);
  }
  store8((T*)a.Y + token * a.ldy + col, valid, y);
}

// A wave has one entry (token, choice).
template <class T>
__global__ void __launch_bounds__(256) combine_backward_kernel(CombineArgs a) {
  const int lane = threadIdx.x % 64;
  const int64_t entry = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  if (entry >= (int64_t)a.tokens * a.choices) return;
  const int row = a.place[entry];
  float dot = 0.0f;
  if ((unsigned)row < (unsigned)a.rows) {
    const float w = a.weights[entry];
    const T* dy = (const T*)a.dY + entry / a.choices * a.lddy;
    const T* z = (const T*)a.Z + (int64_t)row * a.ldz;
    T* dz = (T*)a.dZ + (int64_t)row * a.lddz;
    for (int col = 8 * lane; col < a.cols; col += 512) {
      float g[8], x[8];
      load8(dy + col, a.cols - col, g);
      load8(z + col, a.cols - col, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(g[i], x[i], dot), g[i] *= w;
      store8(dz + col, a.cols - col, g);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) dot += __shfl_xor(dot, d, 64);
  if (lane == 0) a.dweights[entry] = dot;
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
  int runs = (p.entries + kPlanRun - 1) / kPlanRun;
  if (runs < 1) runs = 1;  // offsets are written all the same
  const hipError_t err = launch_with((const void*)&plan_count_kernel, dim3((unsigned)runs), dim3(256), p, s);
  if (err != hipSuccess) return err;
  PlanArgs copy = p;
  void* args[] = {&copy, &runs};
  return hipLaunchKernel((const void*)&plan_place_kernel, dim3((unsigned)runs), dim3(256), args, 0, s);
}

hipError_t launch_combine(int type, const CombineArgs& c, hipStream_t s) {
  int chunks = (c.cols + 7) / 8;
  const int64_t items = (int64_t)chunks * c.tokens;
  return by_type(type, [&](auto t) {
    CombineArgs copy = c;
    void* args[] = {&copy, &chunks};
    return hipLaunchKernel((const void*)&combine_kernel<decltype(t)>, dim3((unsigned)((items + 255) / 256)), dim3(256),
                           args, 0, s);
  });
}

hipError_t launch_combine_backward(int type, const CombineArgs& c, hipStream_t s) {
  const int64_t entries = (int64_t)c.tokens * c.choices;
  return by_type(type, [&](auto t) {
    return launch_with((const void*)&combine_backward_kernel<decltype(t)>, dim3((unsigned)((entries + 3) / 4)), dim3(256),
                       c, s);
  });
}

}  // namespace sgemm_impl
