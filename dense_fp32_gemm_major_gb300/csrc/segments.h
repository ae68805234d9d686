// segments.h -- host-side interface between the segmented products' C ABI
// (seg_api.cu) and their kernels. Internal to libgemm_f32.so.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace gemm {

constexpr int kMaxSegments = 2048;

// A stack of equal row-major matrices: element (z, i, j) at p[z * stride +
// i * ld + j].
struct SegMatrix {
  const void *p = nullptr;
  int64_t ld = 0, stride = 0;
  int64_t rows = 0, cols = 0, count = 1;  // as stored
};

// One segmented product. The result's rows are tokens (wgrad = false) or a
// matrix for each segment (wgrad = true):
//
//   rows:     C[t, :] = scale_z A[t, :] op(B_z)  for the rows t of segment g,
//             z = index[g] (or g)
//   dense:    all M rows with B_0, plus `add` in the segments' rows
//   adapted:  (R > 0) all M rows with B_0, plus U[t, :] op(L_a) for the rows t
//             of segment g, a = index[g] (or g)
//   wgrad:    C_g = A_g^T B_g, the sum over the rows of segment g
struct SegArgs {
  bool bf16 = false, wgrad = false, dense = false;
  int64_t groups = 0, M = 0, N = 0, K = 0;
  SegMatrix A, B, C;
  int transb = 0;  // of B, and of L
  const int64_t *offsets = nullptr;
  const int32_t *index = nullptr;
  const float *scales = nullptr;
  int64_t bank = 0;  // matrices the index may name; others: no product
  // Second terms of A and B (the sum A + A_lo, or B + B_lo, is meant; at most
  // one of them), and of the result: C + C_lo, C rounded.
  SegMatrix A_lo, B_lo, C_lo;
  bool c_f32 = false;  // a float32 result of bf16 operands
  SegMatrix add;       // dense: float32 addend of the result
  int64_t R = 0;       // adapted: width of U
  SegMatrix U, U_lo, L;
  // The launch before, of the same call, writes nothing that this product reads
  // but `add` and U: it may start while that one ends. (What earlier launches
  // wrote is complete: see seg_tc_kernel.)
  bool ahead = false;
  // Scratch for tiles split along k: seg_tc_slots() floats, and 2 counters a
  // pair, zero before the launch. null: no splits.
  float *slots = nullptr;
  unsigned *arrived = nullptr;
  // rows: > 0: two launches share the product, seg_rows the segments of up to
  // this many rows, seg_tc the others.
  int few = 0;
};

// Whether a product's contraction is long enough to be worth splitting (terms:
// of its operands, before the second one's place is known), and the floats that
// its slots take.
bool seg_tc_splits(const SegArgs &a, int terms = 1);
int64_t seg_tc_slots(int sm_count);

// Whether the kernels can read a matrix as it lies (by TMA: 16-byte aligned
// rows). Others are copied first (seg_pack_launch).
bool seg_tc_readable(const SegMatrix &m, bool bf16);

// Operands readable; M, N >= 1 (rows) or groups, N, K >= 1 (wgrad).
int seg_tc_launch(const SegArgs &a, int sm_count, cudaStream_t stream);

// Products of very few rows (rows and dense forms): whether these arguments are
// such a product, its launch (operands readable), and the rows a segment may
// have in it (SegArgs::few): 0 where the launch is fast enough whichever
// segments hold the rows.
bool seg_rows_fits(const SegArgs &a);
int seg_rows_few(const SegArgs &a);
int seg_rows_launch(const SegArgs &a, int sm_count, cudaStream_t stream);

int seg_rows_index_fault_take(IndexFault *out, bool clear);

// Copies a stack of matrices, of equal shape, to another pitch and stride.
// offsets: only rows that the segments hold (by_matrix: only the matrices of
// segments that have rows).
struct SegCopy {
  SegMatrix src, dst;
  const int64_t *offsets = nullptr;
  int64_t groups = 0, M = 0;
  bool by_matrix = false;
};
int seg_pack_launch(const SegCopy &c, bool bf16, int sm_count, cudaStream_t stream);

int seg_pack_index_fault_take(IndexFault *out, bool clear);
int seg_tc_index_fault_take(IndexFault *out, bool clear);

// Synchronise `stream`, then read and clear the kernels' status word.
int seg_tc_poll_status(cudaStream_t stream);

// Capability check and SM count of the current device (api.cu).
int current_device_info(int *dev_out, int *sm_count);

}  // namespace gemm
