// seg_simt.cu -- segmented matrix products on the FP32 pipe: any type, layout,
// pitch and alignment.
//
// With z the segment's matrix, a tile of the result is
//
//   rows:   C[t, n] = s_z sum_k A[t, k] B_z[k, n]        t in the segment
//   dense:  C[t, n] = sum_k A[t, k] B[k, n] + sum_r U[t, r] L_z(t)[r, n]
//   wgrad:  C_g[i, n] = sum_t A[t, i] B[t, n]            t in segment g
//
// A CTA of 256 threads computes 64 x 64 results, 4 x 4 a thread, from 64 x 16
// slices of both operands in shared memory (fp32, whatever the type), walking
// the tiles of all segments in steps of the grid. Each slice is masked as it
// is loaded; a tile of the dense form adds each adapter's product to the rows
// of its segments. Bound by the FP32 pipe and by shared memory; no tensor cores.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "segments.h"

namespace gemm {
namespace {

constexpr int kT = 64, kBK = 16, kThreads = 256;

struct Op {  // element (z, i, j) at p[z * zs + i * is + j * js]
  const void *p;
  long long zs, is, js, extent;
};

struct P {
  int groups, M, N, K, R, bank, wgrad, dense;
  Op A, B, U, L;
  void *C;
  long long c_ld, c_stride, c_extent;
  const int64_t *offsets;
  const int32_t *index;
  const float *scales;
};

template <typename T>
__device__ __forceinline__ float load1(const Op &o, int site, long long off) {
  if (!index_ok(site, off, 1, o.extent)) return 0.0f;
  return static_cast<float>(static_cast<const T *>(o.p)[off]);
}

__device__ __forceinline__ void span_of(const P &p, int g, int *r0, int *r1) {
  const long long a = p.offsets[g], b = p.offsets[g + 1];
  const long long s = a < 0 ? 0 : (a > p.M ? p.M : a);
  *r0 = static_cast<int>(s);
  *r1 = static_cast<int>(b < s ? s : (b > p.M ? p.M : b));
}

__device__ __forceinline__ int matrix_of(const P &p, int g) {
  const int z = p.index != nullptr ? p.index[g] : g;
  return z >= 0 && z < p.bank ? z : -1;
}

// acc += X Y for one slice range: X rows r0 .. r0 + 63 (those in [lo, hi)),
// Y columns c0 .. , k in [k0, k1).
template <typename T>
__device__ void accumulate(float (&acc)[4][4], float (&xs)[kBK][kT + 1], float (&ys)[kBK][kT + 1],
                           const Op &X, int zx, const Op &Y, int zy, int r0, int lo, int hi, int c0,
                           int cols, int k0, int k1) {
  const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
  for (int kb = k0; kb < k1; kb += kBK) {
    for (int e = tid; e < kT * kBK; e += kThreads) {
      // neighbouring threads along the operand's contiguous direction
      const int i = X.js == 1 ? e / kBK : e % kT, k = X.js == 1 ? e % kBK : e / kT;
      const int r = r0 + i, kk = kb + k;
      xs[k][i] = r >= lo && r < hi && kk < k1
                     ? load1<T>(X, kSiteLoadA, zx * X.zs + r * X.is + kk * X.js)
                     : 0.0f;
      const int j = Y.js == 1 ? e % kT : e / kBK, l = Y.js == 1 ? e / kT : e % kBK;
      const int c = c0 + j, ll = kb + l;
      ys[l][j] = c < cols && ll < k1 ? load1<T>(Y, kSiteLoadB, zy * Y.zs + ll * Y.is + c * Y.js)
                                     : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kBK; ++k) {
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = xs[k][tr * 4 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = ys[k][tc + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) seg_simt_kernel(const P p) {
  __shared__ float xs[kBK][kT + 1], ys[kBK][kT + 1];
  const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
  const int tiles_n = (p.N + kT - 1) / kT;
  long long base = 0;  // tiles of the segments before g
  const int groups = p.dense ? 1 : p.groups;
  for (int g = 0; g < groups; ++g) {
    int s0 = 0, s1 = p.M;
    if (!p.dense) span_of(p, g, &s0, &s1);
    const int height = p.wgrad ? p.K : s1 - s0;
    const long long count = static_cast<long long>((height + kT - 1) / kT) * tiles_n;
    const int z = p.dense ? 0 : (p.wgrad ? 0 : matrix_of(p, g));
    // first tile of this segment that is this CTA's
    long long t = (blockIdx.x + gridDim.x - base % gridDim.x) % gridDim.x;
    for (; t < count; t += gridDim.x) {
      const int r0 = static_cast<int>(t / tiles_n) * kT, c0 = static_cast<int>(t % tiles_n) * kT;
      float acc[4][4] = {};
      if (p.wgrad) {
        accumulate<T>(acc, xs, ys, p.A, 0, p.B, 0, r0, 0, p.K, c0, p.N, s0, s1);
      } else {
        const int lo = s0 + r0;
        if (z >= 0)
          accumulate<T>(acc, xs, ys, p.A, 0, p.B, z, lo, lo, s1, c0, p.N, 0, p.K);
        if (p.dense && p.R > 0)
          for (int h = 0; h < p.groups; ++h) {
            int h0, h1;
            span_of(p, h, &h0, &h1);
            const int a = matrix_of(p, h);
            if (h1 <= lo || h0 >= lo + kT || h0 == h1 || a < 0) continue;
            // A sum of its own, added to the segment's rows alone: what is not
            // finite in one adapter reaches no other's rows (0 * inf is NaN).
            float part[4][4] = {};
            accumulate<T>(part, xs, ys, p.U, 0, p.L, a, lo, h0, h1, c0, p.N, 0, p.R);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = lo + tr * 4 + i;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (r >= h0 && r < h1) acc[i][j] += part[i][j];
            }
          }
      }
      const float scale = !p.wgrad && !p.dense && z >= 0 && p.scales != nullptr ? p.scales[z] : 1.0f;
      T *C = static_cast<T *>(p.C);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = r0 + tr * 4 + i, c = c0 + tc + 16 * j;
          const long long off = p.wgrad ? g * p.c_stride + r * p.c_ld + c
                                        : (s0 + r) * p.c_ld + c;
          if (r < height && c < p.N && index_ok(kSiteCStore, off, 1, p.c_extent))
            C[off] = static_cast<T>(scale * acc[i][j]);
        }
    }
    base += count;
  }
}

Op op_of(const SegMatrix &m, bool trans) {
  return Op{m.p, m.stride, trans ? 1 : m.ld, trans ? m.ld : 1,
            (m.count - 1) * m.stride + matrix_extent(m.rows, m.cols, m.ld)};
}

}  // namespace

GEMM_INDEX_FAULT_TAKE(seg_simt_index_fault_take)

int seg_simt_launch(const SegArgs &a, int sm_count, cudaStream_t stream) {
  P p = {};
  p.groups = static_cast<int>(a.groups);
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.R = static_cast<int>(a.R);
  p.bank = static_cast<int>(a.bank);
  p.wgrad = a.wgrad;
  p.dense = a.dense;
  p.A = op_of(a.A, a.wgrad);
  p.B = op_of(a.B, a.transb);
  p.U = op_of(a.U, false);
  p.L = op_of(a.L, a.transl);
  p.C = const_cast<void *>(a.C.p);
  p.c_ld = a.C.ld;
  p.c_stride = a.C.stride;
  p.c_extent = (a.C.count - 1) * a.C.stride + matrix_extent(a.C.rows, a.C.cols, a.C.ld);
  p.offsets = a.offsets;
  p.index = a.index;
  p.scales = a.scales;
  const unsigned grid = static_cast<unsigned>(8 * (sm_count > 0 ? sm_count : 1));
  if (a.bf16)
    seg_simt_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
  else
    seg_simt_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? kOk : kErrLaunch;
}

}  // namespace gemm
