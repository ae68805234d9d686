// clip.cu -- the norm of many tensors together, and their clipping by it.
//
//   norm = sqrt(sum over all tensors of x^2),  y = x min(1, limit / (norm + 1e-6))
//
// Two passes over memory that nothing can join: every factor waits for the last
// element. The first sums squares, 32 KB of a tensor a CTA at a time, the next
// ones under way meanwhile; the second scales, from the end backwards, since what the
// first pass read last is still in L2 (128 MB of bf16 53 us, forwards 60; 332 MB 165
// and 170), and ends at once where the factor is 1, in place. The sums of the first pass's CTAs (a double each, two CTAs an SM) are
// added by a warp of every CTA of the second by itself, in one order, in place of a
// launch between them. (By all threads, root and quotient too, the FP64 units took a
// fifth of the pass.)
//
// Squares of fp32 leave fp32's range from 1.8e19 on and lose bits below 1e-19.
// A thread adds the squares of its 32 to 64 values of a chunk in fp32, and where
// their sum is not between 2^-100 and 2^100 (and not of zeros alone), again in 64
// bits; chunks are added in 64 bits. The FP64 units take one addition of 64
// elements, which hides behind the loads.
//
// Measured (24 bf16 tensors of 332 MB in all, launches by themselves): norm 52 us (6.4
// TB/s), scale 99 us (6.7 TB/s). Two CTAs an SM: 360 MB 178 us, with one 215, three
// 191, four 182 (both passes). 48 tensors of 8192 fp32: 4.7 + 5.7 us, launches and their
// chains of loads.
//
// The list of tensors travels as the kernels' argument (100 of them, or 1000 a
// launch), so a captured graph holds it and nothing is copied to the device.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "clip.h"
#include "ptx.cuh"

namespace gemm {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kLoads = 8;
constexpr int kChunkBytes = kThreads * 16 * kLoads;
constexpr int kFew = 100, kMany = 1000;  // tensors of a launch

struct Entry {
  const void *src;
  void *dst;
  long long n;
  int chunk;  // the tensor's first of the launch's chunks
  int flags;
};
constexpr int kBf16 = 1, kScalar = 2, kInPlace = 4;

template <int CAP>
struct List {
  double *partials;
  float *norm;      // scale: written by the launch's first CTA (or null)
  long long slots;  // partials of all launches
  long long first;  // norm: this launch's first partial
  float limit;
  int count, chunks;
  int in_place;  // all of them
  Entry e[CAP];
};

// The tensor of chunk c.
template <int CAP>
__device__ __forceinline__ int entry_of(const List<CAP> &p, int c) {
  int lo = 0, hi = p.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.e[mid].chunk <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Elements before the first 16-byte boundary.
__device__ __forceinline__ int head_of(const Entry &e, int elem) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(e.src) & 15);
  const long long h = off == 0 ? 0 : (16 - off) / elem;
  return static_cast<int>(h < e.n ? h : e.n);
}

template <class T>
__device__ __forceinline__ void unpack(const uint4 &w, float *v) {
  const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      v[i] = __uint_as_float(u[i]);
    } else {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ double squares(const float *v, int n) {
  double s = 0.0;
  for (int i = 0; i < n; ++i) s = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), s);
  return s;
}

// A chunk's vectors, this thread's: 16-byte loads, kThreads apart.
struct Chunk {
  const Entry *e;  // null: none
  int c;           // of the tensor's chunks
  uint4 w[kLoads];
};

template <class T>
__device__ __forceinline__ void load_vectors(const Entry &e, int c, uint4 (&w)[kLoads]) {
  constexpr int kVec = 16 / sizeof(T);
  const T *x = static_cast<const T *>(e.src);
  const int head = head_of(e, sizeof(T));
  const long long vecs = (e.n - head) / kVec;
  const long long v0 = static_cast<long long>(c) * (kThreads * kLoads) + threadIdx.x;
  const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const long long at = v0 + i * kThreads;
    w[i] = at < vecs && index_ok(kSiteReduceIn, head + at * kVec, kVec, e.n)
               ? xv[at] : make_uint4(0, 0, 0, 0);
  }
}

template <int CAP>
__device__ __forceinline__ Chunk load_chunk(const List<CAP> &p, int c, bool there) {
  Chunk k;
  k.e = nullptr;
  if (!there) return k;
  k.e = &p.e[entry_of(p, c)];
  k.c = c - k.e->chunk;
  if (k.e->flags & kBf16) load_vectors<__nv_bfloat16>(*k.e, k.c, k.w);
  else load_vectors<float>(*k.e, k.c, k.w);
  return k;
}

// Squares of a chunk, this thread's.
template <class T>
__device__ __forceinline__ double chunk_squares(const Chunk &k) {
  constexpr int kVec = 16 / sizeof(T);
  const Entry &e = *k.e;
  float local = 0.0f;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    float v[kVec], s = 0.0f;
    unpack<T>(k.w[i], v);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s = fmaf(v[j], v[j], s);
    local += s;
  }
  double sum = local;
  if (!(local >= 0x1p-100f && local <= 0x1p100f)) {
    unsigned any = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) any |= k.w[i].x | k.w[i].y | k.w[i].z | k.w[i].w;
    sum = 0.0;
    if (any != 0) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        float v[kVec];
        unpack<T>(k.w[i], v);
        sum += squares(v, kVec);
      }
    }
  }
  // the first chunk takes the elements around the vectors too
  if (k.c == 0) {
    const T *x = static_cast<const T *>(e.src);
    const int head = head_of(e, sizeof(T));
    const long long tail = head + (e.n - head) / kVec * kVec;
    const int ends = head + static_cast<int>(e.n - tail);
    if (static_cast<int>(threadIdx.x) < ends) {
      const int t = threadIdx.x;
      const long long at = t < head ? t : tail + (t - head);
      if (index_ok(kSiteReduceIn, at, 1, e.n)) {
        const float v = static_cast<float>(x[at]);
        sum += squares(&v, 1);
      }
    }
  }
  return sum;
}

// Sum over the CTA, in thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kWarps];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w];
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ List<CAP> p) {
  grid_dependency_wait();
  grid_launch_dependents();
  double sum = 0.0;
  const int step = static_cast<int>(gridDim.x);
  Chunk now = load_chunk(p, blockIdx.x, static_cast<int>(blockIdx.x) < p.chunks);
  for (int c = blockIdx.x; c < p.chunks; c += step) {
    const Chunk next = load_chunk(p, c + step, p.chunks - c > step);
    sum += now.e->flags & kBf16 ? chunk_squares<__nv_bfloat16>(now) : chunk_squares<float>(now);
    now = next;
  }
  sum = block_sum(sum);
  const long long at = p.first + blockIdx.x;
  if (threadIdx.x == 0 && index_ok(kSiteReducePartial, at, 1, p.slots)) p.partials[at] = sum;
}

template <class T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

template <class T>
__device__ __forceinline__ void scale_chunk(const Chunk &k, float f) {
  constexpr int kVec = 16 / sizeof(T);
  const Entry &e = *k.e;
  const T *x = static_cast<const T *>(e.src);
  T *y = static_cast<T *>(e.dst);
  const int head = head_of(e, sizeof(T));
  const long long vecs = (e.n - head) / kVec, tail = head + vecs * kVec;
  const long long first = static_cast<long long>(k.c) * (kThreads * kLoads);
  if (e.flags & kScalar) {  // the two lie on boundaries of their own
    const long long last = min(first + kThreads * kLoads, vecs);
    for (long long i = head + first * kVec + threadIdx.x; i < head + last * kVec; i += kThreads)
      if (index_ok(kSiteReduceIn, i, 1, e.n)) y[i] = rounded<T>(static_cast<float>(x[i]) * f);
  } else {
    uint4 *yv = reinterpret_cast<uint4 *>(y + head);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const long long at = first + threadIdx.x + i * kThreads;
      if (!(at < vecs && index_ok(kSiteReduceOut, head + at * kVec, kVec, e.n))) continue;
      float v[kVec];
      unpack<T>(k.w[i], v);
      unsigned u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (sizeof(T) == 4) {
          u[j] = __float_as_uint(v[j] * f);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j] * f, v[2 * j + 1] * f);
          u[j] = *reinterpret_cast<const unsigned *>(&h);
        }
      }
      __stcs(yv + at, make_uint4(u[0], u[1], u[2], u[3]));  // beside what is still to be read
    }
  }
  if (k.c == 0) {
    const int ends = head + static_cast<int>(e.n - tail), t = threadIdx.x;
    if (t < ends) {
      const long long at = t < head ? t : tail + (t - head);
      if (index_ok(kSiteReduceOut, at, 1, e.n)) y[at] = rounded<T>(static_cast<float>(x[at]) * f);
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ List<CAP> p) {
  __shared__ float factor;
  grid_dependency_wait();
  grid_launch_dependents();
  // A thread reads no element that another one writes (a tensor in place is its own
  // operand, element by element), so the first ones may be on their way.
  const int step = static_cast<int>(gridDim.x);
  Chunk now = load_chunk(p, p.chunks - 1 - static_cast<int>(blockIdx.x),
                         static_cast<int>(blockIdx.x) < p.chunks);
  if (threadIdx.x < 32) {
    double sum = 0.0;
#pragma unroll 4
    for (long long i = threadIdx.x; i < p.slots; i += 32)
      if (index_ok(kSiteReducePartial, i, 1, p.slots)) sum += p.partials[i];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (threadIdx.x == 0) {
      const double norm = sqrt(sum), ratio = static_cast<double>(p.limit) / (norm + 1e-6);
      if (blockIdx.x == 0 && p.norm != nullptr) *p.norm = static_cast<float>(norm);
      factor = ratio > 1.0 ? 1.0f : static_cast<float>(ratio);  // a NaN stays one
    }
  }
  __syncthreads();
  const float f = factor;
  if (f == 1.0f && p.in_place) return;  // nothing to read or write
  for (int i = blockIdx.x; i < p.chunks; i += step) {
    const Chunk next = load_chunk(p, p.chunks - 1 - i - step, p.chunks - i > step);
    if (!(f == 1.0f && (now.e->flags & kInPlace))) {
      if (now.e->flags & kBf16) scale_chunk<__nv_bfloat16>(now, f);
      else scale_chunk<float>(now, f);
    }
    now = next;
  }
}

template <class K, class L>
int launch(K kernel, const L &p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? kOk : kErrLaunch;
}

// Tensors [i0, *next) as a list, as many as fit in it and in 2^31 chunks.
template <int CAP>
void fill(const ClipArgs &a, int64_t i0, int64_t *next, List<CAP> *p) {
  p->count = p->chunks = 0;
  p->in_place = 1;
  int64_t i = i0;
  for (; i < a.count && p->count < CAP; ++i) {
    const int64_t n = a.n[i];
    if (n == 0) continue;
    const int elem = a.bf16(i) ? 2 : 4;
    const int64_t chunks = (n * elem + kChunkBytes - 1) / kChunkBytes;
    if (p->chunks + chunks > 0x70000000LL) break;
    Entry &e = p->e[p->count++];
    e.src = a.x[i];
    e.dst = a.y != nullptr ? a.y[i] : const_cast<void *>(a.x[i]);
    e.n = n;
    e.chunk = p->chunks;
    e.flags = (elem == 2 ? kBf16 : 0) | (e.dst == e.src ? kInPlace : 0) |
              ((reinterpret_cast<uintptr_t>(e.dst) - reinterpret_cast<uintptr_t>(e.src)) % 16 != 0
                   ? kScalar : 0);
    p->in_place &= e.dst == e.src;
    p->chunks += static_cast<int>(chunks);
  }
  *next = i;
}

int grid_of(int chunks, int sms) {
  const int most = 2 * (sms > 0 ? sms : 1);
  return chunks < most ? (chunks > 0 ? chunks : 1) : most;
}

template <int CAP>
int run(const ClipArgs &a, int64_t launches, int sms, cudaStream_t stream) {
  // Tens of KB at most, and gone with the call: the launches copy it.
  List<CAP> p;
  std::memset(&p, 0, offsetof(List<CAP>, e));
  int64_t *start = static_cast<int64_t *>(malloc(static_cast<size_t>(launches + 1) * sizeof(int64_t)));
  if (start == nullptr) return kErrLaunch;
  int64_t slots = 0, n = 0;
  for (int64_t i = 0; i < a.count; ++n) {
    start[n] = i;
    fill<CAP>(a, i, &i, &p);
    slots += grid_of(p.chunks, sms);
  }
  void *ws = nullptr;
  int st = pool_alloc(&ws, static_cast<size_t>(slots > 0 ? slots : 1) * sizeof(double), stream);
  if (st == kOk) {
    p.partials = static_cast<double *>(ws);
    p.slots = slots;
    p.limit = a.limit;
    for (int64_t l = 0; st == kOk && l < n; ++l) {
      int64_t next;
      fill<CAP>(a, start[l], &next, &p);
      const int grid = grid_of(p.chunks, sms);
      st = launch(norm_kernel<CAP>, p, grid, stream);
      p.first += grid;
    }
    p.norm = a.norm;
    if (!a.scale || n == 0) {
      p.count = p.chunks = 0;
      if (st == kOk) st = launch(scale_kernel<CAP>, p, 1, stream);
    } else {
      for (int64_t l = n - 1; st == kOk && l >= 0; --l) {
        int64_t next;
        fill<CAP>(a, start[l], &next, &p);
        st = launch(scale_kernel<CAP>, p, grid_of(p.chunks, sms), stream);
        p.norm = nullptr;
      }
    }
    const int fst = pool_free(ws, stream);
    if (st == kOk) st = fst;
  }
  free(start);
  return st;
}

}  // namespace

GEMM_INDEX_FAULT_TAKE(clip_index_fault_take)

int clip_launch(const ClipArgs &a, int sm_count, cudaStream_t stream) {
  // A list is cut where it is full, or near 2^31 chunks (a tensor has 2^28 at most).
  const int64_t launches = 2 + a.count / 4;
  return a.count <= kFew ? run<kFew>(a, launches, sm_count, stream)
                         : run<kMany>(a, launches, sm_count, stream);
}

}  // namespace gemm
