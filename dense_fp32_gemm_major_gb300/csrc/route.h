// route.h -- host-side interface between the C ABI of the router, of the rows'
// way to the experts and back (route_api.cu) and their kernels (route.cu,
// route_rows.cu). Internal to libgemm_f32.so.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace gemm {

struct RouteArgs {
  bool bf16 = false, sigmoid = false, renormalise = false;
  int64_t T = 0, E = 0, k = 0;
  const void *logits = nullptr;
  int64_t ldx = 0;
  const float *bias = nullptr;
  const uint8_t *mask = nullptr;
  int groups = 1, top_groups = 1, group_best = 1;
  float scale = 1.0f;
  int32_t *experts = nullptr;
  float *weights = nullptr;
  // The plan, or null.
  int64_t *offsets = nullptr;
  int32_t *order = nullptr, *places = nullptr;
};

struct RouteBackwardArgs {
  bool bf16 = false, sigmoid = false, renormalise = false;
  int64_t T = 0, E = 0, k = 0;
  const float *dweights = nullptr, *weights = nullptr;
  const void *logits = nullptr;
  int64_t ldx = 0;
  const int32_t *experts = nullptr;
  float scale = 1.0f;
  void *dlogits = nullptr;
  int64_t lddx = 0;
};

// T, E, k >= 1. Both take a workspace from the library's pool where the plan is
// made by several CTAs.
int route_launch(const RouteArgs &a, int sm_count, cudaStream_t stream);
int route_plan_launch(int64_t slots, int64_t E, const int32_t *experts, int64_t *offsets,
                      int32_t *order, int32_t *places, int sm_count, cudaStream_t stream);
int route_backward_launch(const RouteBackwardArgs &a, int sm_count, cudaStream_t stream);

// X or dO (T x D), Y or dY (rows x D).
struct RowsArgs {
  bool bf16 = false;
  int64_t T = 0, D = 0, k = 0, rows = 0;
  const void *token = nullptr;  // X, dO
  int64_t ld_token = 0;
  const void *expert = nullptr;  // Y
  int64_t ld_expert = 0;
  const int32_t *places = nullptr;
  const float *weights = nullptr;
  void *out = nullptr;  // of dispatch, combine: the result; of backward: dY
  int64_t ld_out = 0;
  float *dweights = nullptr;
};

// T, k >= 1; D >= 1 (backward: 0 too).
int rows_dispatch_launch(const RowsArgs &a, int sm_count, cudaStream_t stream);
int rows_combine_launch(const RowsArgs &a, int sm_count, cudaStream_t stream);
int rows_backward_launch(const RowsArgs &a, int sm_count, cudaStream_t stream);

int route_index_fault_take(IndexFault *out, bool clear);
int rows_index_fault_take(IndexFault *out, bool clear);

// Capability check and SM count of the current device (api.cu).
int current_device_info(int *dev_out, int *sm_count);

}  // namespace gemm
