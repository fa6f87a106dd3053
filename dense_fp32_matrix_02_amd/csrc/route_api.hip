// Host side of include/sgemm_mi355_route.h: argument checks, then the launches.

#include "sgemm_mi355_route.h"

#include "api_checks.h"
#include "fp8_internal.h"

namespace sgemm_impl {
namespace {

int check_route(int type, int tokens, int experts, int ld, int score, int choices) {
  if (!known_type(type)) return SGEMM_MI355_ERR_TYPE;
  if (score != SGEMM_MI355_SOFTMAX && score != SGEMM_MI355_SIGMOID) return SGEMM_MI355_ERR_OP;
  if (tokens < 0 || experts < 1 || choices < 0) return SGEMM_MI355_ERR_DIM;
  if (experts > SGEMM_MI355_MAX_EXPERTS || choices > SGEMM_MI355_MAX_CHOICES) return SGEMM_MI355_ERR_ROUTE;
  if (ld < experts) return SGEMM_MI355_ERR_LD;
  if (tokens > kMostRows || !launchable(((int64_t)tokens + 3) / 4, 256)) return SGEMM_MI355_ERR_EXTENT;
  return SGEMM_MI355_OK;
}

int check_combine(int type, int tokens, int choices, int rows, int cols) {
  if (!known_type(type)) return SGEMM_MI355_ERR_TYPE;
  if (tokens < 0 || choices < 0 || rows < 0 || cols < 0) return SGEMM_MI355_ERR_DIM;
  if (tokens > kMostRows || cols > kMostRows || rows > kMostRows || (int64_t)tokens * choices > kMostRows)
    return SGEMM_MI355_ERR_EXTENT;
  return SGEMM_MI355_OK;
}

}  // namespace
}  // namespace sgemm_impl

using namespace sgemm_impl;

extern "C" {

int sgemm_mi355_route(int type, int tokens, int experts, const void* logits, int ld, const float* bias, int score,
                      int groups, int top_groups, int choices, int renorm, float scale, float* weights, int* ids,
                      hipStream_t stream) {
  const int v = check_route(type, tokens, experts, ld, score, choices);
  if (v != SGEMM_MI355_OK) return v;
  if (groups < 1 || groups > experts || experts % groups != 0 || top_groups < 1 || top_groups > groups ||
      choices > top_groups * (experts / groups))
    return SGEMM_MI355_ERR_ROUTE;
  if (tokens == 0 || choices == 0) return SGEMM_MI355_OK;
  Matrices m;
  m.dense(logits, tokens, experts, ld, element_size(type), false);
  if (bias != nullptr) m.dense(bias, 1, experts, experts, 4, false);
  m.dense(weights, tokens, choices, choices, 4, true);
  m.dense(ids, tokens, choices, choices, 4, true);
  const int c = m.check();
  if (c != SGEMM_MI355_OK) return c;
  RouteArgs r{};
  r.logits = logits, r.ld = ld, r.bias = bias, r.tokens = tokens, r.experts = experts, r.groups = groups;
  r.top_groups = top_groups, r.choices = choices, r.renorm = renorm, r.scale = scale, r.weights = weights, r.ids = ids;
  return done(launch_route(type, score, r, stream));
}

int sgemm_mi355_route_backward(int type, int tokens, int experts, const void* logits, int ld, const int* ids,
                               const float* dweights, int score, int choices, int renorm, float scale,
                               float* dlogits, int ldd, hipStream_t stream) {
  const int v = check_route(type, tokens, experts, ld, score, choices);
  if (v != SGEMM_MI355_OK) return v;
  if (ldd < experts) return SGEMM_MI355_ERR_LD;
  if (tokens == 0) return SGEMM_MI355_OK;
  Matrices m;
  m.dense(logits, tokens, experts, ld, element_size(type), false);
  m.dense(ids, tokens, choices, choices, 4, false);
  m.dense(dweights, tokens, choices, choices, 4, false);
  m.dense(dlogits, tokens, experts, ldd, 4, true);
  const int c = m.check();
  if (c != SGEMM_MI355_OK) return c;
  RouteArgs r{};
  r.logits = logits, r.ld = ld, r.tokens = tokens, r.experts = experts, r.choices = choices, r.renorm = renorm;
  r.scale = scale, r.ids_in = ids, r.dweights = dweights, r.dlogits = dlogits, r.ldd = ldd;
  return done(launch_route_backward(type, score, r, stream));
}

size_t sgemm_mi355_route_plan_workspace_size(int tokens, int choices, int experts) {
  if (tokens < 0 || choices < 0 || experts < 1 || experts > SGEMM_MI355_MAX_EXPERTS) return 0;
  const int64_t entries = (int64_t)tokens * choices;
  if (entries > kMostRows) return 0;
  PlanArgs p{};
  plan_division(entries, experts, p);
  const size_t rows = p.runs == 1 ? 0 : (size_t)p.runs + (p.per > 0 ? p.groups + 1 : 0);
  return rows * ((size_t)experts + 1) * 4;
}

int sgemm_mi355_route_plan(int tokens, int choices, int experts, const int* ids, int* offsets, int* row_token,
                           int* place, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (tokens < 0 || choices < 0 || experts < 1) return SGEMM_MI355_ERR_DIM;
  if (experts > SGEMM_MI355_MAX_EXPERTS) return SGEMM_MI355_ERR_ROUTE;
  const int64_t entries = (int64_t)tokens * choices;
  if (entries > kMostRows) return SGEMM_MI355_ERR_EXTENT;
  const size_t need = sgemm_mi355_route_plan_workspace_size(tokens, choices, experts);
  Matrices m;
  m.dense(ids, tokens, choices, choices, 4, false);
  m.dense(offsets, 1, experts + 1, experts + 1, 4, true);
  m.dense(row_token, 1, entries, entries, 4, true);
  m.dense(place, tokens, choices, choices, 4, true);
  if (need > 0 && workspace_bytes >= need) m.dense(workspace, 1, (int64_t)(need / 4), (int64_t)(need / 4), 4, true);
  const int c = m.check();
  if (c != SGEMM_MI355_OK) return c;
  if (workspace_bytes < need) return SGEMM_MI355_ERR_WORKSPACE;
  PlanArgs p{(int)entries, choices, experts, ids, offsets, row_token, place, (int*)workspace, 0, 0, 0};
  plan_division(entries, experts, p);
  return done(launch_route_plan(p, stream));
}

int sgemm_mi355_route_combine(int type, int tokens, int choices, int rows, int cols, const void* Z, int ldz,
                              const int* place, const float* weights, void* Y, int ldy, hipStream_t stream) {
  const int v = check_combine(type, tokens, choices, rows, cols);
  if (v != SGEMM_MI355_OK) return v;
  if (ldz < at_least_1(cols) || ldy < at_least_1(cols)) return SGEMM_MI355_ERR_LD;
  if (tokens == 0 || cols == 0) return SGEMM_MI355_OK;
  if (!launchable(((int64_t)tokens * ((cols + 511) / 512) + 3) / 4, 256)) return SGEMM_MI355_ERR_EXTENT;
  Matrices m;
  m.dense(Z, rows, cols, ldz, element_size(type), false);
  m.dense(place, tokens, choices, choices, 4, false);
  m.dense(weights, tokens, choices, choices, 4, false);
  m.dense(Y, tokens, cols, ldy, element_size(type), true);
  const int c = m.check();
  if (c != SGEMM_MI355_OK) return c;
  CombineArgs a{};
  a.tokens = tokens, a.choices = choices, a.rows = rows, a.cols = cols, a.Z = Z, a.ldz = ldz, a.place = place;
  a.weights = weights, a.Y = Y, a.ldy = ldy;
  return done(launch_combine(type, a, stream));
}

int sgemm_mi355_route_combine_backward(int type, int tokens, int choices, int rows, int cols, const void* dY,
                                       int lddy, const void* Z, int ldz, const int* place, const float* weights,
                                       void* dZ, int lddz, float* dweights, hipStream_t stream) {
  const int v = check_combine(type, tokens, choices, rows, cols);
  if (v != SGEMM_MI355_OK) return v;
  if (lddy < at_least_1(cols) || ldz < at_least_1(cols) || lddz < at_least_1(cols)) return SGEMM_MI355_ERR_LD;
  if (tokens == 0 || choices == 0) return SGEMM_MI355_OK;
  if (!launchable(((int64_t)tokens * choices + 3) / 4, 256)) return SGEMM_MI355_ERR_EXTENT;
  Matrices m;
  m.dense(dY, tokens, cols, lddy, element_size(type), false);
  m.dense(Z, rows, cols, ldz, element_size(type), false);
  m.dense(place, tokens, choices, choices, 4, false);
  m.dense(weights, tokens, choices, choices, 4, false);
  m.dense(dZ, rows, cols, lddz, element_size(type), true);
  m.dense(dweights, tokens, choices, choices, 4, true);
  const int c = m.check();
  if (c != SGEMM_MI355_OK) return c;
  CombineArgs a{};
  a.tokens = tokens, a.choices = choices, a.rows = rows, a.cols = cols, a.Z = Z, a.ldz = ldz, a.place = place;
  a.weights = weights, a.dY = dY, a.lddy = lddy, a.dZ = dZ, a.lddz = lddz, a.dweights = dweights;
  return done(launch_combine_backward(type, a, stream));
}

}  // extern "C"
