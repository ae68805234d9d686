// route_api.cu -- the C ABI of the router and of the rows' way to the experts
// and back (declared in include/route_f32.h): argument validation and launches.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/route_f32.h"
#include "args.h"
#include "route.h"

namespace {

using gemm::array_ok;
using gemm::dim_ok;
using gemm::overlap;
using gemm::Range;
using gemm::SegMatrix;
using gemm::stack_ok;

bool type_ok(int type) { return type == GEMM_F32_TYPE_F32 || type == GEMM_F32_TYPE_BF16; }

// T tokens of k slots: both and their product.
bool slots_ok(int64_t T, int64_t k) {
  return dim_ok(T) && k >= 1 && k <= GEMM_F32_MAX_ROUTE_SLOTS && dim_ok(T * k);
}

bool disjoint(const Range *in, int ins, const Range *out, int outs) {
  for (int i = 0; i < outs; ++i) {
    for (int j = 0; j < ins; ++j)
      if (overlap(in[j], out[i])) return false;
    for (int j = 0; j < i; ++j)
      if (overlap(out[j], out[i])) return false;
  }
  return true;
}

bool matrix_ok(const void *p, int64_t rows, int64_t cols, int64_t ld, int elem, Range *r) {
  return stack_ok(SegMatrix{p, ld, 0, rows, cols, 1}, elem, false, r);
}

int elem_of(int type) { return type == GEMM_F32_TYPE_BF16 ? 2 : 4; }

// Arguments of dispatch, combine and its gradients.
bool rows_ok(int type, int64_t T, int64_t D, int64_t k, int64_t rows) {
  return type_ok(type) && slots_ok(T, k) && dim_ok(D) && dim_ok(rows);
}

}  // namespace

extern "C" {

int gemm_f32_route(int type, int score, int64_t T, int64_t E, int64_t k, const void *logits,
                   int64_t ldx, const float *bias, const uint8_t *mask, int64_t groups,
                   int64_t top_groups, int64_t group_best, int renormalise, float scale,
                   int32_t *experts, float *weights, int64_t *offsets, int32_t *order,
                   int32_t *places, void *stream) {
  if (!type_ok(type) || (score != GEMM_F32_SCORE_SOFTMAX && score != GEMM_F32_SCORE_SIGMOID) ||
      E < 1 || E > GEMM_F32_MAX_SEGMENTS || !slots_ok(T, k) || k > E || groups < 1 || groups > 32 ||
      E % groups != 0 || top_groups < 1 || top_groups > groups || group_best < 1 ||
      group_best > 2 || (renormalise != 0 && renormalise != 1) || std::isnan(scale))
    return GEMM_ERR_INVALID_ARG;
  const bool plan = offsets != nullptr || order != nullptr || places != nullptr;
  Range rx, rb, rm, re, rw, ro, rr, rp;
  if (!matrix_ok(logits, T, E, ldx, elem_of(type), &rx) || !array_ok(bias, E, 4, true, &rb) ||
      !array_ok(mask, T, 1, true, &rm) || !array_ok(experts, T * k, 4, false, &re) ||
      !array_ok(weights, T * k, 4, false, &rw))
    return GEMM_ERR_INVALID_ARG;
  if (plan && (!array_ok(offsets, E + 1, 8, false, &ro) || !array_ok(order, T * k, 4, false, &rr) ||
               !array_ok(places, T * k, 4, false, &rp)))
    return GEMM_ERR_INVALID_ARG;
  const Range in[] = {rx, rb, rm}, out[] = {re, rw, ro, rr, rp};
  if (!disjoint(in, 3, out, 5)) return GEMM_ERR_ALIAS;
  if (T == 0 && !plan) return GEMM_OK;
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)  // no rows
    return cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * 8, s) == cudaSuccess
               ? GEMM_OK : GEMM_ERR_LAUNCH;
  gemm::RouteArgs a;
  a.bf16 = type == GEMM_F32_TYPE_BF16;
  a.sigmoid = score == GEMM_F32_SCORE_SIGMOID;
  a.renormalise = renormalise != 0;
  a.T = T;
  a.E = E;
  a.k = k;
  a.logits = logits;
  a.ldx = ldx;
  a.bias = bias;
  a.mask = mask;
  a.groups = static_cast<int>(groups);
  a.top_groups = static_cast<int>(top_groups);
  a.group_best = static_cast<int>(group_best);
  a.scale = scale;
  a.experts = experts;
  a.weights = weights;
  a.offsets = offsets;
  a.order = order;
  a.places = places;
  return gemm::route_launch(a, sms, s);
}

int gemm_f32_route_backward(int type, int score, int64_t T, int64_t E, int64_t k,
                            const float *dweights, const void *logits, int64_t ldx,
                            const int32_t *experts, const float *weights, int renormalise,
                            float scale, void *dlogits, int64_t lddx, void *stream) {
  if (!type_ok(type) || (score != GEMM_F32_SCORE_SOFTMAX && score != GEMM_F32_SCORE_SIGMOID) ||
      E < 1 || E > GEMM_F32_MAX_SEGMENTS || !slots_ok(T, k) ||
      (renormalise != 0 && renormalise != 1) || std::isnan(scale) ||
      (renormalise != 0 && scale == 0.0f))
    return GEMM_ERR_INVALID_ARG;
  const int elem = elem_of(type);
  Range rg, rx, re, rw, rd;
  if (!array_ok(dweights, T * k, 4, false, &rg) || !matrix_ok(logits, T, E, ldx, elem, &rx) ||
      !array_ok(experts, T * k, 4, false, &re) || !array_ok(weights, T * k, 4, false, &rw) ||
      !matrix_ok(dlogits, T, E, lddx, elem, &rd))
    return GEMM_ERR_INVALID_ARG;
  const Range in[] = {rg, rx, re, rw};
  if (!disjoint(in, 4, &rd, 1)) return GEMM_ERR_ALIAS;
  if (T == 0) return GEMM_OK;
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  gemm::RouteBackwardArgs a;
  a.bf16 = type == GEMM_F32_TYPE_BF16;
  a.sigmoid = score == GEMM_F32_SCORE_SIGMOID;
  a.renormalise = renormalise != 0;
  a.T = T;
  a.E = E;
  a.k = k;
  a.dweights = dweights;
  a.logits = logits;
  a.ldx = ldx;
  a.experts = experts;
  a.weights = weights;
  a.scale = scale;
  a.dlogits = dlogits;
  a.lddx = lddx;
  return gemm::route_backward_launch(a, sms, static_cast<cudaStream_t>(stream));
}

int gemm_f32_route_plan(int64_t slots, int64_t E, const int32_t *experts, int64_t *offsets,
                        int32_t *order, int32_t *places, void *stream) {
  if (!dim_ok(slots) || E < 1 || E > GEMM_F32_MAX_SEGMENTS) return GEMM_ERR_INVALID_ARG;
  Range re, out[3];
  if (!array_ok(experts, slots, 4, false, &re) || !array_ok(offsets, E + 1, 8, false, &out[0]) ||
      !array_ok(order, slots, 4, false, &out[1]) || !array_ok(places, slots, 4, false, &out[2]))
    return GEMM_ERR_INVALID_ARG;
  if (!disjoint(&re, 1, out, 3)) return GEMM_ERR_ALIAS;
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (slots == 0)
    return cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * 8, s) == cudaSuccess
               ? GEMM_OK : GEMM_ERR_LAUNCH;
  return gemm::route_plan_launch(slots, E, experts, offsets, order, places, sms, s);
}

int gemm_f32_dispatch(int type, int64_t T, int64_t D, int64_t k, int64_t rows, const void *X,
                      int64_t ldx, const int32_t *places, void *Y, int64_t ldy, void *stream) {
  if (!rows_ok(type, T, D, k, rows)) return GEMM_ERR_INVALID_ARG;
  const int elem = elem_of(type);
  Range in[2], out;
  if (!matrix_ok(X, T, D, ldx, elem, &in[0]) || !array_ok(places, T * k, 4, false, &in[1]) ||
      !matrix_ok(Y, rows, D, ldy, elem, &out))
    return GEMM_ERR_INVALID_ARG;
  if (!disjoint(in, 2, &out, 1)) return GEMM_ERR_ALIAS;
  if (T == 0 || D == 0 || rows == 0) return GEMM_OK;
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  gemm::RowsArgs a;
  a.bf16 = type == GEMM_F32_TYPE_BF16;
  a.T = T;
  a.D = D;
  a.k = k;
  a.rows = rows;
  a.token = X;
  a.ld_token = ldx;
  a.places = places;
  a.out = Y;
  a.ld_out = ldy;
  return gemm::rows_dispatch_launch(a, sms, static_cast<cudaStream_t>(stream));
}

int gemm_f32_combine(int type, int64_t T, int64_t D, int64_t k, int64_t rows, const void *Y,
                     int64_t ldy, const int32_t *places, const float *weights, void *O,
                     int64_t ldo, void *stream) {
  if (!rows_ok(type, T, D, k, rows)) return GEMM_ERR_INVALID_ARG;
  const int elem = elem_of(type);
  Range in[3], out;
  if (!matrix_ok(Y, rows, D, ldy, elem, &in[0]) || !array_ok(places, T * k, 4, false, &in[1]) ||
      !array_ok(weights, T * k, 4, true, &in[2]) || !matrix_ok(O, T, D, ldo, elem, &out))
    return GEMM_ERR_INVALID_ARG;
  if (!disjoint(in, 3, &out, 1)) return GEMM_ERR_ALIAS;
  if (T == 0 || D == 0) return GEMM_OK;
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  gemm::RowsArgs a;
  a.bf16 = type == GEMM_F32_TYPE_BF16;
  a.T = T;
  a.D = D;
  a.k = k;
  a.rows = rows;
  a.expert = Y;
  a.ld_expert = ldy;
  a.places = places;
  a.weights = weights;
  a.out = O;
  a.ld_out = ldo;
  return gemm::rows_combine_launch(a, sms, static_cast<cudaStream_t>(stream));
}

int gemm_f32_combine_backward(int type, int64_t T, int64_t D, int64_t k, int64_t rows,
                              const void *dO, int64_t lddo, const void *Y, int64_t ldy,
                              const int32_t *places, const float *weights, void *dY, int64_t lddy,
                              float *dweights, void *stream) {
  if (!rows_ok(type, T, D, k, rows) || (dY == nullptr && dweights == nullptr && T > 0 && D > 0 && rows > 0))
    return GEMM_ERR_INVALID_ARG;
  const int elem = elem_of(type);
  Range in[4], out[2];
  if (!matrix_ok(dO, T, D, lddo, elem, &in[0]) ||
      (dweights != nullptr && !matrix_ok(Y, rows, D, ldy, elem, &in[1])) ||
      !array_ok(places, T * k, 4, false, &in[2]) || !array_ok(weights, T * k, 4, true, &in[3]) ||
      (dY != nullptr && !matrix_ok(dY, rows, D, lddy, elem, &out[0])) ||
      !array_ok(dweights, T * k, 4, true, &out[1]))
    return GEMM_ERR_INVALID_ARG;
  if (!disjoint(in, 4, out, 2)) return GEMM_ERR_ALIAS;
  if (T == 0 || (dweights == nullptr && (D == 0 || rows == 0))) return GEMM_OK;
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  gemm::RowsArgs a;
  a.bf16 = type == GEMM_F32_TYPE_BF16;
  a.T = T;
  a.D = D;
  a.k = k;
  a.rows = rows;
  a.token = dO;
  a.ld_token = lddo;
  a.expert = dweights != nullptr ? Y : nullptr;
  a.ld_expert = ldy;
  a.places = places;
  a.weights = weights;
  a.out = dY;
  a.ld_out = lddy;
  a.dweights = dweights;
  return gemm::rows_backward_launch(a, sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
