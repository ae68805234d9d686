// w4.h -- host-side interface between the C ABI of products with 4-bit weights
// (w4_api.cu) and their kernels (w4.cu). Internal to libgemm_f32.so.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace gemm {

// C[t, n] = sum_k A[t, k] s (q - z), the rows t of segment g with matrix g (no
// offsets: all rows with matrix 0).
struct W4Args {
  bool bf16 = false;
  int64_t groups = 1, M = 0, N = 0, K = 0, group = 0;
  const void *A = nullptr;
  int64_t lda = 0;
  const uint8_t *Q = nullptr;  // N x ceil(K / 2) bytes each
  int64_t ldq = 0, strideq = 0;
  const void *scales = nullptr;  // N x ceil(K / group) each
  int64_t lds = 0, strides = 0;
  const uint8_t *zeros = nullptr;
  int64_t ldz = 0, stridez = 0;
  void *C = nullptr;
  int64_t ldc = 0;
  const int64_t *offsets = nullptr;
};

// Few rows: the kernel that reads the weights as they are (rows that do not start on
// 16 bytes, for TMA, are copied first). M, N, K >= 1.
int w4_launch(const W4Args &a, int sm_count, cudaStream_t stream);

// Rows [n0, n0 + rows) of each W in fp32, or as the sum of two bf16 terms; pitch
// ldd, stride rows * ldd.
int w4_expand_launch(const W4Args &a, int64_t n0, int64_t rows, void *hi, void *lo, int64_t ldd,
                     int sm_count, cudaStream_t stream);

int w4_poll_status(cudaStream_t stream);
int w4_index_fault_take(IndexFault *out, bool clear);

int current_device_info(int *dev_out, int *sm_count);

}  // namespace gemm
