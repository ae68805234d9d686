// seg_rows.cu -- segmented products of very few rows: single tokens.
//
//   rows, dense:  C[t, n] = s_z sum_k A[t, k] op(B_z)[k, n] (+ add[t, n])
//
// With one or two rows a segment the product is a reading of B: its bytes at
// the rate of memory, or, where they are few, the latency of one way to memory
// and back. The tensor-core kernels' set-up, TMEM and hand-overs take longer
// than that, so up to four rows of a segment go to one CTA of plain FMAs that
// has nothing to set up:
//
//   B stored K x N: a thread holds 16 bytes of n; TX threads span the CTA's
//     columns, the others share k, DEEP rows of B each at a time (as many loads
//     in flight), and their sums meet in shared memory in a fixed order.
//   B stored N x K: a warp holds four n, its lanes share k (four loads in
//     flight) and add by shuffles.
//
// Few columns a CTA (16 to 1024 of bf16) make many CTAs of short loops: 1 x 512
// x 512 float32 is sixteen CTAs of two rounds of loads. A long contraction goes
// to the four CTAs of a cluster, whose first adds the others' sums from their
// shared memory (32 rows of their own adapters, 4096 x 16: one SM reads its 128
// KB in 8 us).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "seg_terms.cuh"
#include "segments.h"

namespace gemm {
namespace {

constexpr int kThreads = 256, kRows = 4, kWarpN = 4;
constexpr int kSlices = 4, kSliceK = 1024;  // CTAs of a contraction, from this k on
// bf16 operands longer than kShortK: most of N (M + 2 CTAs' rows), seg_rows_fits.
constexpr int64_t kShortK = 128, kMostBf16 = 36 * 1024;
// FMAs of a product whose rows may all lie in one segment: 2 million of them take
// a microsecond, since every four rows read the matrix again (seg_rows_few).
constexpr double kMostSkewed = 128e6;
constexpr int kStaged = 8192;  // values of A that stand in shared memory at a time

struct P {
  const void *A, *A_lo, *B;
  void *C, *C_lo;
  const float *add, *scales;
  const int64_t *offsets;
  const int32_t *index;
  long long a_ld, a_lo_ld, b_ld, b_stride, c_ld, c_lo_ld, add_ld;
  long long a_extent, b_extent, c_extent, c_lo_extent, add_extent, a_lo_extent;
  int M, N, K, groups, bank, dense, c_f32, slices;
  int alone;  // one row a CTA
  int few;    // rows of a segment, at most (0: any number)
  int span;   // rows that a CTA looks at, one after another
};

template <class T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
};

// 16 bytes from p + off, the values at or past `left` zero.
template <class T>
__device__ __forceinline__ uint4 load16(const T *p, long long off, int left, int site,
                                        long long extent) {
  constexpr int n = Vec<T>::n;
  if (left >= n && index_ok(site, off, n, extent))
    return __ldg(reinterpret_cast<const uint4 *>(p + off));
  uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < n; ++i)
    if (i < left && index_ok(site, off + i, 1, extent)) {
      if constexpr (n == 4)
        u[i] = __float_as_uint(p[off + i]);
      else
        u[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[off + i])) << (i % 2 * 16);
    }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// A load16 as floats.
template <class T>
__device__ __forceinline__ void unpack(const uint4 &w, float (&v)[Vec<T>::n]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (Vec<T>::n == 4) {
      v[i] = __uint_as_float(u[i]);
    } else {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

// One value of A: the sum of its terms.
template <class T>
__device__ __forceinline__ float load_a(const P &p, long long row, int k) {
  float v = 0.0f;
  const long long at = row * p.a_ld + k;
  if (index_ok(kSiteLoadA, at, 1, p.a_extent)) v = static_cast<float>(static_cast<const T *>(p.A)[at]);
  if (p.A_lo != nullptr) {
    const long long lo = row * p.a_lo_ld + k;
    if (index_ok(kSiteLoadA, lo, 1, p.a_lo_extent))
      v += static_cast<float>(static_cast<const T *>(p.A_lo)[lo]);
  }
  return v;
}

// k of A that stand in shared memory at a time, for `count` rows.
__device__ __forceinline__ int chunk_of(int count) {
  return count == 1 ? kStaged : (count == 2 ? kStaged / 2 : kStaged / 4);
}

// Rows [t, t + count) of A, k [k0, k0 + chunk), as floats.
template <class T>
__device__ __forceinline__ void stage_a(const P &p, float *as, int t, int count, int k0, int k_end,
                                        int chunk) {
  const int n = min(chunk, k_end - k0), end = (n + 15) / 16 * 16;
  for (int r = 0; r < count; ++r)
    for (int k = threadIdx.x; k < end; k += kThreads)
      as[r * chunk + k] = k < n ? load_a<T>(p, t + r, k0 + k) : 0.0f;
}

// Rows [t, t + count) that this CTA computes, their matrix (-1: none), its
// scale, and the rows that have an addend: t is a row; unless each is alone,
// every fourth of a segment takes those behind it.
struct Rows {
  int count, z, add0, add1;
  int next;  // where a CTA of several rows goes on
  float scale;
};

__device__ __forceinline__ bool rows_of(const P &p, int t, Rows *o) {
  int first = 0, last = p.M;
  o->next = t + 1;
  o->z = 0;
  o->scale = 1.0f;
  o->add0 = o->add1 = 0;
  if (p.dense) {
    if (p.add != nullptr) {
      const long long a = p.offsets[0], b = p.offsets[p.groups];
      o->add0 = static_cast<int>(a < 0 ? 0 : (a > p.M ? p.M : a));
      o->add1 = static_cast<int>(b < 0 ? 0 : (b > p.M ? p.M : b));
    }
  } else {
    // Each thread looks at its segments; all loads are on their way at once.
    __shared__ int found[3];
    if (threadIdx.x == 0) found[0] = -1;
    __syncthreads();
    for (int g = threadIdx.x; g < p.groups; g += kThreads) {
      const long long a = p.offsets[g], b = p.offsets[g + 1];
      const int z = p.index != nullptr ? p.index[g] : g;
      if (a <= t && t < b) {
        found[1] = static_cast<int>(a < 0 ? 0 : a);
        found[2] = static_cast<int>(b > p.M ? p.M : b);
        found[0] = z >= 0 && z < p.bank ? z : p.bank;  // bank: none
      }
    }
    __syncthreads();
    if (found[0] < 0) return false;
    first = found[1];
    last = found[2];
    if (p.few > 0 && last - first > p.few) {
      o->next = last;
      return false;
    }
    o->z = found[0] < p.bank ? found[0] : -1;
    if (p.scales != nullptr && o->z >= 0) o->scale = p.scales[o->z];
  }
  // One or kRows, not a number of the launch's: with that float32 takes 71
  // registers, not 63, and three CTAs fit an SM, not four.
  const int step = p.alone ? 1 : kRows;
  if ((t - first) % step != 0) return false;
  o->count = min(step, last - t);
  o->next = t + o->count;
  return true;
}

template <class T>
__device__ __forceinline__ void store(const P &p, int row, int n, float v, const Rows &o) {
  v *= o.scale;
  if (p.add != nullptr && row >= o.add0 && row < o.add1) {
    const long long at = row * p.add_ld + n;
    if (index_ok(kSitePartialRead, at, 1, p.add_extent)) v += p.add[at];
  }
  const long long at = row * p.c_ld + n;
  if (!index_ok(kSiteCStore, at, 1, p.c_extent)) return;
  if (p.c_f32) {
    static_cast<float *>(p.C)[at] = v;
    return;
  }
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  static_cast<__nv_bfloat16 *>(p.C)[at] = h;
  if (p.C_lo != nullptr) {
    const long long lo = row * p.c_lo_ld + n;
    if (index_ok(kSitePartialWrite, lo, 1, p.c_lo_extent))
      static_cast<__nv_bfloat16 *>(p.C_lo)[lo] = second_term(v, h);
  }
}

// CTAs an SM that the compiler plans registers for. bf16: with two (three for B
// stored N x K) it holds the loads of two rounds (one row of 4096 x 4096 12 -> 8
// us, 20 -> 11). float32 is left to it (0): four CTAs of one round are faster
// than two of two (9 against 12 us); in a loop over rows (SPAN) it has to be told.
template <class T, int BF16, bool SPAN>
constexpr int kCtas = Vec<T>::n == 4 ? (SPAN ? 4 : 0) : BF16;

// This CTA's rows, one product after another: f(t, rows). SPAN: more than one.
template <bool SPAN, class F>
__device__ __forceinline__ void for_rows(const P &p, const F &f) {
  Rows o;
  if constexpr (SPAN) {
    const int t0 = static_cast<int>(blockIdx.y) * p.span, end = min(t0 + p.span, p.M);
    for (int t = t0; t < end; t = o.next) {
      if (t > t0) __syncthreads();  // shared memory of the one before is read
      if (rows_of(p, t, &o)) f(t, o);
    }
  } else if (rows_of(p, static_cast<int>(blockIdx.y), &o)) {
    f(static_cast<int>(blockIdx.y), o);
  }
}

// B stored K x N. TX threads of 16 bytes across the CTA's columns, DEEP rows of
// B in flight a thread.
template <class T, int TX, int kDeep, bool SPAN>
__global__ void __launch_bounds__(kThreads, kCtas<T, 2, SPAN>) seg_rows_kn_kernel(const P p) {
  constexpr int V = Vec<T>::n, TY = kThreads / TX, NT = TX * V;
  __shared__ float sums[TY * NT], as[kStaged];
  float *const total = as;  // in the end: [count][NT]
  static_assert(kRows * NT <= kStaged, "totals in A's place");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for_rows<SPAN>(p, [&](int t, const Rows &o) {
    const int count = o.count, z = o.z;
    const int n0 = blockIdx.x * NT;
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, n = n0 + tx * V;
    // This CTA's k, a multiple of 16 but for the last one's end.
    const int slice = (p.K / 16 + p.slices - 1) / p.slices * 16;
    const int k_lo = min(static_cast<int>(blockIdx.z) * slice, p.K);
    const int k_hi = static_cast<int>(blockIdx.z) + 1 == p.slices ? p.K : min(k_lo + slice, p.K);
    float acc[kRows][V] = {};
    if (z >= 0) {
      const T *B = static_cast<const T *>(p.B) + z * p.b_stride;
      const long long extent = p.b_extent - z * p.b_stride;
      const int chunk = chunk_of(count);
      for (int c0 = k_lo; c0 < k_hi; c0 += chunk) {
        const int c1 = min(chunk, k_hi - c0);
        if (c0 > k_lo) __syncthreads();
        stage_a<T>(p, as, t, count, c0, k_hi, chunk);
        __syncthreads();
#pragma unroll 2
        for (int k = ty * kDeep; k < c1; k += TY * kDeep) {
          uint4 w[kDeep];
#pragma unroll
          for (int j = 0; j < kDeep; ++j)
            w[j] = load16<T>(B, static_cast<long long>(c0 + k + j) * p.b_ld + n,
                             k + j < c1 ? p.N - n : 0, kSiteLoadB, extent);
          float b[kDeep][V];
#pragma unroll
          for (int j = 0; j < kDeep; ++j) unpack<T>(w[j], b[j]);
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (r < count) {
#pragma unroll
              for (int j = 0; j < kDeep; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                  acc[r][v] = fmaf(as[r * chunk + k + j], b[j][v], acc[r][v]);
            }
        }
      }
    }
    // Two steps: groups of threads add TY / G of a column's sums, then one the
    // groups'.
    constexpr int G = NT < kThreads ? kThreads / NT : 1, PER = TY / G > 0 ? TY / G : 1;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r >= count) break;
#pragma unroll
      for (int v = 0; v < V; ++v) sums[ty * NT + tx * V + v] = acc[r][v];
      __syncthreads();
      if constexpr (G > 1 && TY % G == 0) {
        const int c = threadIdx.x % NT, group = threadIdx.x / NT;
        float s = 0.0f;
#pragma unroll
        for (int y = 0; y < PER; ++y) s += sums[(group * PER + y) * NT + c];
        __syncthreads();
        sums[group * NT + c] = s;
        __syncthreads();
        if (group == 0) {
          s = 0.0f;
#pragma unroll
          for (int y = 0; y < G; ++y) s += sums[y * NT + c];
          total[r * NT + c] = s;
        }
      } else {
        for (int c = threadIdx.x; c < NT; c += kThreads) {
          float s = 0.0f;
#pragma unroll
          for (int y = 0; y < TY; ++y) s += sums[y * NT + c];
          total[r * NT + c] = s;
        }
      }
      __syncthreads();
    }
    if (p.slices > 1) cluster_sync();  // every CTA's totals are there
    if (blockIdx.z == 0) {
      for (int i = threadIdx.x; i < count * NT; i += kThreads) {
        const int r = i / NT, c = i % NT;
        float s = total[i];
        for (int q = 1; q < p.slices; ++q) {
          uint32_t at;
          float v;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                       : "=r"(at)
                       : "r"(smem_addr(total + i)), "r"(q));
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
          s += v;
        }
        if (n0 + c < p.N) store<T>(p, t + r, n0 + c, s, o);
      }
    }
    if (p.slices > 1) cluster_sync();  // and stay until they are read
  });
}

// B stored N x K. A warp takes kWarpN columns.
template <class T, bool SPAN>
__global__ void __launch_bounds__(kThreads, kCtas<T, 3, SPAN>) seg_rows_nk_kernel(const P p) {
  constexpr int V = Vec<T>::n;
  __shared__ __align__(16) float as[kStaged];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for_rows<SPAN>(p, [&](int t, const Rows &o) {
    const int count = o.count, z = o.z;
    const int lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kWarpN;
    float acc[kRows][kWarpN] = {};
    if (z >= 0) {
      const T *B = static_cast<const T *>(p.B) + z * p.b_stride;
      const long long extent = p.b_extent - z * p.b_stride;
      const int chunk = chunk_of(count);
      for (int c0 = 0; c0 < p.K; c0 += chunk) {
        const int c1 = min(chunk, p.K - c0);
        if (c0 > 0) __syncthreads();
        stage_a<T>(p, as, t, count, c0, p.K, chunk);
        __syncthreads();
#pragma unroll 2
        for (int k = lane * V; k < c1; k += 32 * V) {
          uint4 w[kWarpN];
#pragma unroll
          for (int j = 0; j < kWarpN; ++j)
            w[j] = load16<T>(B, static_cast<long long>(n0 + j) * p.b_ld + c0 + k,
                             n0 + j < p.N ? c1 - k : 0, kSiteLoadB, extent);
          float b[kWarpN][V];
#pragma unroll
          for (int j = 0; j < kWarpN; ++j) unpack<T>(w[j], b[j]);
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (r < count) {
#pragma unroll
              for (int v = 0; v < V; v += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(as + r * chunk + k + v);
#pragma unroll
                for (int j = 0; j < kWarpN; ++j) {
                  acc[r][j] = fmaf(x.x, b[j][v], acc[r][j]);
                  acc[r][j] = fmaf(x.y, b[j][v + 1], acc[r][j]);
                  acc[r][j] = fmaf(x.z, b[j][v + 2], acc[r][j]);
                  acc[r][j] = fmaf(x.w, b[j][v + 3], acc[r][j]);
                }
              }
            }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r < count) {
#pragma unroll
        for (int j = 0; j < kWarpN; ++j) {
          float s = acc[r][j];
#pragma unroll
          for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
          if (lane == 0 && n0 + j < p.N) store<T>(p, t + r, n0 + j, s, o);
        }
      }
  });
}

long long extent_of(const SegMatrix &m) {
  return (m.count - 1) * m.stride + matrix_extent(m.rows, m.cols, m.ld);
}

// CTAs of a launch with a row each.
long long ctas_of(const P &p, int columns) {
  return static_cast<long long>((p.N + columns - 1) / columns) * p.M * p.slices;
}

// Rows a CTA looks at. Where segments may be left to the tensor cores, CTAs that
// find nothing to do are the cost: 65536 of them (512 rows x 1024 x 1024 float32,
// all in one segment) take 77 us of the GPU. Then 64 CTAs an SM share the rows
// (that case 341 us evenly routed and 59 in one segment with 160 CTAs an SM, 344
// and 45 with 64; 16 an SM no longer balance, 381 us). Up to 192 an SM a row
// each is faster (32 rows, 16 segments, 4096 x 4096: 191 against 209 us).
int span_of(const P &p, int columns, int sms) {
  const long long ctas = ctas_of(p, columns);
  if (p.few == 0 || ctas <= 192LL * sms) return 1;
  return static_cast<int>((ctas + 64LL * sms - 1) / (64LL * sms));
}

template <class K>
int launch(K kernel, P p, int columns, int sms, cudaStream_t stream) {
  // Rows together read their matrix once; where there are too few CTAs to fill
  // the GPU, one row each is faster (8 x 512 x 512 bf16: 7.0 -> 4.7 us).
  p.alone = ctas_of(p, columns) <= 2LL * sms;
  const int rows = (p.M + p.span - 1) / p.span;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + columns - 1) / columns),
                     static_cast<unsigned>(rows), static_cast<unsigned>(p.slices));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = static_cast<unsigned>(p.slices);
  cfg.attrs = attr;
  cfg.numAttrs = p.slices > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? kOk : kErrLaunch;
}

template <class T, int TX>
int launch_kn(P p, int sms, cudaStream_t stream) {
  constexpr int kColumns = TX * Vec<T>::n;
  p.span = span_of(p, kColumns, sms);
  return p.span > 1 ? launch(seg_rows_kn_kernel<T, TX, 8, true>, p, kColumns, sms, stream)
                    : launch(seg_rows_kn_kernel<T, TX, 8, false>, p, kColumns, sms, stream);
}

template <class T>
int launch_type(P p, int transb, int sms, cudaStream_t stream) {
  constexpr int V = Vec<T>::n, kColumns = kThreads / 32 * kWarpN;
  p.slices = !transb && p.K >= kSliceK ? kSlices : 1;
  if (transb) {
    p.span = span_of(p, kColumns, sms);
    return p.span > 1 ? launch(seg_rows_nk_kernel<T, true>, p, kColumns, sms, stream)
                      : launch(seg_rows_nk_kernel<T, false>, p, kColumns, sms, stream);
  }
  // A short contraction has no work for many threads along k; a narrow result
  // none for many along n.
  if (p.K <= 16 && p.N >= 512 * V) return launch_kn<T, 128>(p, sms, stream);
  if (p.K <= 64) return launch_kn<T, 32>(p, sms, stream);
  if (p.N <= 2 * V) return launch_kn<T, 2>(p, sms, stream);
  return launch_kn<T, 8>(p, sms, stream);
}

}  // namespace

GEMM_INDEX_FAULT_TAKE(seg_rows_index_fault_take)

bool seg_rows_fits(const SegArgs &a) {
  // All rows together few, or the segments' (about two each, at most).
  if (a.wgrad || a.R > 0 || a.K <= 0) return false;
  const int64_t fours = (a.M + kRows - 1) / kRows;
  if (a.M > 2 * kRows && (a.dense || a.M > 2 * a.groups || a.M > 512)) return false;
  // float32: 8 rows of 4096 x 11008 take 87 us here, 114 on the tensor cores.
  if (!a.bf16 || a.K <= kShortK) return true;
  // bf16: what grows with the CTAs (of four rows of a segment, at most) and
  // with the rows is limited: 4 rows of 4096 x 4096 take 13 us here and 19 on
  // the tensor cores, 8 rows 25 and 19; a row of each of four segments 39 and
  // 33, of two 15 and 23; one row of 4096 x 11008 24 and 29, four 38 and 29.
  const int64_t ctas = a.dense ? fours : (a.M < a.groups - 1 + fours ? a.M : a.groups - 1 + fours);
  return a.N * (a.M + 2 * ctas) <= kMostBf16;
}

// The host knows the rows' average, not where they are: 512 rows of 256 experts
// may all have chosen one. Its matrix of 1024 x 1024 float32 was then read 128
// times (240 us; the tensor cores' one product 31), one of 128 x 11008 bf16 as
// often (508 against 14). Past kMostSkewed segments of more than eight rows are
// left to the tensor cores, in a launch of their own (45 and 34 us). Where all
// have few rows that launch costs 6 us (32 rows, 16 segments, 4096 x 4096
// float32: 184 -> 191); below, the worst case takes no longer than the even one
// (64 rows, 64 segments, 1024 x 1024: 33 us in one segment, 71 in all).
int seg_rows_few(const SegArgs &a) {
  const double work = static_cast<double>(a.M) * static_cast<double>(a.N * a.K);
  return a.dense || a.M <= 2 * kRows || work <= kMostSkewed ? 0 : 2 * kRows;
}

int seg_rows_launch(const SegArgs &a, int sm_count, cudaStream_t stream) {
  P p = {};
  p.A = a.A.p;
  p.A_lo = a.A_lo.p;
  p.B = a.B.p;
  p.C = const_cast<void *>(a.C.p);
  p.C_lo = const_cast<void *>(a.C_lo.p);
  p.add = static_cast<const float *>(a.add.p);
  p.scales = a.scales;
  p.offsets = !a.dense || a.add.p != nullptr ? a.offsets : nullptr;
  p.index = a.index;
  p.a_ld = a.A.ld;
  p.a_lo_ld = a.A_lo.ld;
  p.b_ld = a.B.ld;
  p.b_stride = a.B.stride;
  p.c_ld = a.C.ld;
  p.c_lo_ld = a.C_lo.ld;
  p.add_ld = a.add.ld;
  p.a_extent = extent_of(a.A);
  p.a_lo_extent = extent_of(a.A_lo);
  p.b_extent = extent_of(a.B);
  p.c_extent = extent_of(a.C);
  p.c_lo_extent = extent_of(a.C_lo);
  p.add_extent = extent_of(a.add);
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.groups = static_cast<int>(a.groups);
  p.bank = static_cast<int>(a.bank);
  p.dense = a.dense;
  p.few = a.few;
  p.c_f32 = !a.bf16 || a.c_f32;
  return a.bf16 ? launch_type<__nv_bfloat16>(p, a.transb, sm_count, stream)
                : launch_type<float>(p, a.transb, sm_count, stream);
}

}  // namespace gemm
