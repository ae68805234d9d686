// clip.h -- host-side interface between the C ABI of the norm of many tensors
// and their clipping (reduce_api.cu) and its kernels (clip.cu). Internal to
// libgemm_f32.so.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <cuda_runtime.h>

#include "kernels.h"

namespace gemm {

struct ClipArgs {
  int64_t count = 0;
  const void *const *x = nullptr;
  void *const *y = nullptr;  // null: in place
  const int64_t *n = nullptr;
  const int *type = nullptr;  // gemm_f32_type, one a tensor
  float limit = 0.0f;
  float *norm = nullptr;
  bool scale = false;  // false: the norm alone
  bool bf16(int64_t i) const { return type[i] == 1; }
};

int clip_launch(const ClipArgs &a, int sm_count, cudaStream_t stream);
int clip_index_fault_take(IndexFault *out, bool clear);

int current_device_info(int *dev_out, int *sm_count);

}  // namespace gemm
