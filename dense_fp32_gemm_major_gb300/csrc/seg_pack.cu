// seg_pack.cu -- copies of stacks of row-major matrices to another pitch.
//
// The segmented products read their operands by TMA, which wants rows that
// start on 16 bytes. Others (an odd pitch, a shifted base) are copied here
// first, to rows padded to 16 bytes: one read and one write at the rate of
// memory, and only of what the segments use, in place of a second way into the
// tensor-core kernels with plain loads (which ran at a fifth of their rate:
// 1000 x 777 x 1531 in five segments 70 us). The same copy hands a result that
// was made in a padded workspace back to the caller's pitch.
//
// A warp takes a row's piece of 1024 elements, neighbouring lanes neighbouring
// elements, eight loads in flight a lane.

#include <cuda_runtime.h>

#include <cstdint>

#include "segments.h"

namespace gemm {
namespace {

constexpr int kThreads = 256, kPiece = 1024, kFlight = 8;

struct P {
  const void *src;
  void *dst;
  long long src_ld, src_stride, dst_ld, dst_stride, src_extent, dst_extent;
  long long rows, count;
  int cols, pieces;
  const int64_t *offsets;
  int groups, by_matrix;
  long long M;
};

__device__ __forceinline__ long long held(long long a, long long m) {
  return a < 0 ? 0 : (a > m ? m : a);
}

template <class T>
__global__ void __launch_bounds__(kThreads) seg_pack_kernel(const P p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
  long long first = 0, last = p.rows;
  if (p.offsets != nullptr && !p.by_matrix) {
    first = held(p.offsets[0], p.M);
    last = held(p.offsets[p.groups], p.M);
  }
  const long long total = p.count * p.rows * p.pieces;
  const T *src = static_cast<const T *>(p.src);
  T *dst = static_cast<T *>(p.dst);
  for (long long i = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
       i < total; i += warps) {
    const long long line = i / p.pieces, z = line / p.rows, row = line - z * p.rows;
    const int c0 = static_cast<int>(i - line * p.pieces) * kPiece;
    if (row < first || row >= last) continue;
    if (p.by_matrix && held(p.offsets[z], p.M) >= held(p.offsets[z + 1], p.M)) continue;
    const long long from = z * p.src_stride + row * p.src_ld, to = z * p.dst_stride + row * p.dst_ld;
    const int end = c0 + kPiece < p.cols ? c0 + kPiece : p.cols;
    for (int c = c0 + lane; c < end; c += 32 * kFlight) {
      T v[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int x = c + 32 * k;
        v[k] = x < end && index_ok(kSiteCopySrc, from + x, 1, p.src_extent) ? src[from + x] : T(0);
      }
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int x = c + 32 * k;
        if (x < end && index_ok(kSiteCopyDst, to + x, 1, p.dst_extent)) dst[to + x] = v[k];
      }
    }
  }
}

long long extent_of(const SegMatrix &m) {
  return (m.count - 1) * m.stride + matrix_extent(m.rows, m.cols, m.ld);
}

}  // namespace

GEMM_INDEX_FAULT_TAKE(seg_pack_index_fault_take)

int seg_pack_launch(const SegCopy &c, bool bf16, int sm_count, cudaStream_t stream) {
  if (c.src.rows <= 0 || c.src.cols <= 0 || c.src.count <= 0) return kOk;
  P p = {};
  p.src = c.src.p;
  p.dst = const_cast<void *>(c.dst.p);
  p.src_ld = c.src.ld;
  p.src_stride = c.src.stride;
  p.dst_ld = c.dst.ld;
  p.dst_stride = c.dst.stride;
  p.src_extent = extent_of(c.src);
  p.dst_extent = extent_of(c.dst);
  p.rows = c.src.rows;
  p.count = c.src.count;
  p.cols = static_cast<int>(c.src.cols);
  p.pieces = static_cast<int>((c.src.cols + kPiece - 1) / kPiece);
  p.offsets = c.offsets;
  p.groups = static_cast<int>(c.groups);
  p.M = c.M;
  p.by_matrix = c.by_matrix;
  const long long blocks = (p.count * p.rows * p.pieces + kThreads / 32 - 1) / (kThreads / 32);
  const long long cap = 8LL * (sm_count > 0 ? sm_count : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < cap ? blocks : cap), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, seg_pack_kernel<uint16_t>, p)
                             : cudaLaunchKernelEx(&cfg, seg_pack_kernel<float>, p);
  return e == cudaSuccess ? kOk : kErrLaunch;
}

}  // namespace gemm
