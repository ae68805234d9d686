// route_rows.cu -- rows to the experts and back: copies of each token's row at
// its places, the weighted sum of a token's rows, and its gradients.
//
//   dispatch   Y[places[t][j]] = X[t]
//   combine    O[t] = sum_j w[t][j] Y[places[t][j]]
//   backward   dY[places[t][j]] = w[t][j] dO[t],  dw[t][j] = dO[t] . Y[places[t][j]]
//
// All three are bound by memory: a token's row is read once (or written once),
// each expert's row once, whichever order they lie in. Up to eight warps share a
// token's row, each a piece of 1 KB of it at a time through all its places, with the
// loads of up to four places in flight. Rows are read and written 16 bytes a lane
// where their starts and widths allow it.
//
// Measured (8192 tokens of 4096 bf16, two places each, launches by themselves):
// dispatch 29 to 31 us (201 MB: 6.4 to 6.9 TB/s), combine 28 us (7.1 TB/s), backward 54
// us (336 MB: 6.2 TB/s); a plain copy has 6.8. 1531 tokens of 777 fp32 (rows on no 16 bytes), three
// places: 5.6, 6.9 and 7.8 us.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "route.h"

namespace gemm {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct P {
  const void *token, *expert;
  void *out;
  const int32_t *places;
  const float *weights;
  float *dweights;
  long long ld_token, ld_expert, ld_out;
  long long token_extent, expert_extent, out_extent;
  long long rows;
  int T, D, k;    // D in loads (kElems elements each)
  int pieces;     // of a row
  int per_token;  // warps of a token: 1, 2, 4 or 8
};

// A lane's share of a row at a time: U loads of kElems elements, 32 loads apart.
template <class T, bool VEC>
struct Row {
  using Load = T;
  static constexpr int kElems = 1, U = 8;
  static __device__ __forceinline__ Load zero() { return Load(0.0f); }
  static __device__ __forceinline__ void unpack(const Load &l, float (&v)[kElems]) {
    v[0] = static_cast<float>(l);
  }
  static __device__ __forceinline__ Load pack(const float (&v)[kElems]) { return static_cast<T>(v[0]); }
};
template <>
struct Row<float, true> {
  using Load = float4;
  static constexpr int kElems = 4, U = 2;
  static __device__ __forceinline__ Load zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ void unpack(const Load &l, float (&v)[kElems]) {
    v[0] = l.x;
    v[1] = l.y;
    v[2] = l.z;
    v[3] = l.w;
  }
  static __device__ __forceinline__ Load pack(const float (&v)[kElems]) {
    return make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Row<__nv_bfloat16, true> {
  using Load = uint4;
  static constexpr int kElems = 8, U = 2;
  static __device__ __forceinline__ Load zero() { return make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void unpack(const Load &l, float (&v)[kElems]) {
    const unsigned u[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Load pack(const float (&v)[kElems]) {
    unsigned u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const unsigned *>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// Loads [c, c + 32 U) of a row, this lane's.
template <class R>
__device__ __forceinline__ void load_row(const void *base, long long row_at, int c, int D, int site,
                                         long long extent, typename R::Load (&v)[R::U]) {
  const typename R::Load *p =
      reinterpret_cast<const typename R::Load *>(static_cast<const char *>(base));
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    const int i = c + 32 * u;
    v[u] = i < D && index_ok(site, row_at + static_cast<long long>(i) * R::kElems, R::kElems, extent)
               ? __ldcs(p + row_at / R::kElems + i)  // read once
               : R::zero();
  }
}
template <class R>
__device__ __forceinline__ void store_row(void *base, long long row_at, int c, int D,
                                          long long extent, const typename R::Load (&v)[R::U]) {
  typename R::Load *p = reinterpret_cast<typename R::Load *>(static_cast<char *>(base));
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    const int i = c + 32 * u;
    if (i < D && index_ok(kSiteCStore, row_at + static_cast<long long>(i) * R::kElems, R::kElems,
                          extent))
      p[row_at / R::kElems + i] = v[u];
  }
}

__device__ __forceinline__ long long place_of(const P &p, long long s) {
  const long long at = index_ok(kSiteLoadB, s, 1, static_cast<long long>(p.T) * p.k) ? p.places[s] : -1;
  return at >= 0 && at < p.rows ? at : -1;
}

__device__ __forceinline__ float weight_of(const P &p, long long s) {
  return p.weights != nullptr && index_ok(kSiteLoadB, s, 1, static_cast<long long>(p.T) * p.k)
             ? p.weights[s] : 1.0f;
}

// Calls of f(token, piece) for this warp's pieces.
template <class F>
__device__ __forceinline__ void for_pieces(const P &p, F f) {
  const int warp = static_cast<int>(threadIdx.x >> 5), per = p.per_token;
  const int tokens = kWarps / per, sub = warp % per;
  const long long step = static_cast<long long>(gridDim.x) * tokens;
  for (long long t = static_cast<long long>(blockIdx.x) * tokens + warp / per; t < p.T; t += step)
    for (int piece = sub; piece < p.pieces; piece += per) f(t, piece);
}

template <class T, bool VEC, int PLACES>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const P p) {
  using R = Row<T, VEC>;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  for_pieces(p, [&](long long t, int piece) {
    const int c = piece * 32 * R::U + lane;
    typename R::Load v[R::U];
    load_row<R>(p.token, t * p.ld_token, c, p.D, kSiteCopySrc, p.token_extent, v);
    for (int j0 = 0; j0 < p.k; j0 += PLACES) {
      long long at[PLACES];
#pragma unroll
      for (int j = 0; j < PLACES; ++j) at[j] = j0 + j < p.k ? place_of(p, t * p.k + j0 + j) : -1;
#pragma unroll
      for (int j = 0; j < PLACES; ++j)
        if (at[j] >= 0) store_row<R>(p.out, at[j] * p.ld_out, c, p.D, p.out_extent, v);
    }
  });
}

// CTAs an SM, and so registers. 8192 tokens of 4096 bf16, two places: 29 us with four,
// 33 with three or five; 4096 tokens, six places: 38 with three, 43 with two, 65 with
// four (spills).
constexpr int combine_ctas(int places) { return places == 2 ? 4 : 3; }

template <class T, bool VEC, int PLACES>
__global__ void __launch_bounds__(kThreads, combine_ctas(PLACES)) combine_kernel(const P p) {
  using R = Row<T, VEC>;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  for_pieces(p, [&](long long t, int piece) {
    const int c = piece * 32 * R::U + lane;
    float sum[R::U][R::kElems] = {};
    for (int j0 = 0; j0 < p.k; j0 += PLACES) {
      typename R::Load v[PLACES][R::U];
      long long at[PLACES];
      float w[PLACES];
#pragma unroll
      for (int j = 0; j < PLACES; ++j) {
        const long long s = t * p.k + j0 + j;
        at[j] = j0 + j < p.k ? place_of(p, s) : -1;
        w[j] = j0 + j < p.k ? weight_of(p, s) : 1.0f;
      }
#pragma unroll
      for (int j = 0; j < PLACES; ++j)
        if (at[j] >= 0)
          load_row<R>(p.expert, at[j] * p.ld_expert, c, p.D, kSiteLoadA, p.expert_extent, v[j]);
#pragma unroll
      for (int j = 0; j < PLACES; ++j) {
        if (at[j] < 0) continue;
#pragma unroll
        for (int u = 0; u < R::U; ++u) {
          float y[R::kElems];
          R::unpack(v[j][u], y);
#pragma unroll
          for (int e = 0; e < R::kElems; ++e) sum[u][e] = fmaf(w[j], y[e], sum[u][e]);
        }
      }
    }
    typename R::Load o[R::U];
#pragma unroll
    for (int u = 0; u < R::U; ++u) o[u] = R::pack(sum[u]);
    store_row<R>(p.out, t * p.ld_out, c, p.D, p.out_extent, o);
  });
}

// CTAs an SM, and so registers. 8192 tokens of 4096 bf16, two places: 57 us with four,
// 65 with three, 81 with five (spills); 4096 tokens, six places: 82 with two, 95 with
// three; element by element (1531 tokens of 777, fp32, three places): 7.8 with three,
// 11.4 with two.
constexpr int backward_ctas(bool vec, int places) { return !vec ? 3 : (places == 2 ? 4 : 2); }

// `per_token` warps share a token's pieces; their sums of dw meet in shared
// memory, in the order of the warps.
template <class T, bool VEC, int PLACES>
__global__ void __launch_bounds__(kThreads, backward_ctas(VEC, PLACES)) backward_kernel(const P p) {
  using R = Row<T, VEC>;
  __shared__ float part[kWarps][32][33];  // warp, slot, lane
  __shared__ float dots[kWarps][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = static_cast<int>(threadIdx.x >> 5);
  const int tokens = kWarps / p.per_token, mine = warp / p.per_token, sub = warp % p.per_token;
  for (long long t0 = static_cast<long long>(blockIdx.x) * tokens; t0 < p.T;
       t0 += static_cast<long long>(gridDim.x) * tokens) {
    const long long t = t0 + mine;
    if (t < p.T) {
      for (int j = 0; j < p.k; ++j) part[warp][j][lane] = 0.0f;
      for (int piece = sub; piece < p.pieces; piece += p.per_token) {
        const int c = piece * 32 * R::U + lane;
        typename R::Load d[R::U];
        load_row<R>(p.token, t * p.ld_token, c, p.D, kSiteLoadA, p.token_extent, d);
        for (int j0 = 0; j0 < p.k; j0 += PLACES) {
          typename R::Load v[PLACES][R::U];
          long long at[PLACES];
          float wj[PLACES];
#pragma unroll
          for (int j = 0; j < PLACES; ++j) {
            const long long s = t * p.k + j0 + j;
            at[j] = j0 + j < p.k ? place_of(p, s) : -1;
            wj[j] = j0 + j < p.k ? weight_of(p, s) : 1.0f;
          }
#pragma unroll
          for (int j = 0; j < PLACES; ++j) {
            if (at[j] >= 0 && p.dweights != nullptr)
              load_row<R>(p.expert, at[j] * p.ld_expert, c, p.D, kSiteLoadB, p.expert_extent, v[j]);
          }
#pragma unroll
          for (int j = 0; j < PLACES; ++j) {
            if (at[j] < 0) continue;
            const float w = wj[j];
            float dot = 0.0f;
            typename R::Load o[R::U];
#pragma unroll
            for (int u = 0; u < R::U; ++u) {
              float g[R::kElems], y[R::kElems];
              R::unpack(d[u], g);
              if (p.dweights != nullptr) {
                R::unpack(v[j][u], y);
#pragma unroll
                for (int e = 0; e < R::kElems; ++e) dot = fmaf(g[e], y[e], dot);
              }
#pragma unroll
              for (int e = 0; e < R::kElems; ++e) g[e] *= w;
              o[u] = R::pack(g);
            }
            if (p.out != nullptr)
              store_row<R>(p.out, at[j] * p.ld_out, c, p.D, p.out_extent, o);
            if (p.dweights != nullptr) part[warp][j0 + j][lane] += dot;
          }
        }
      }
      if (p.dweights != nullptr) {
        // lane j: the sum of slot j's 32 parts
        __syncwarp();
        float sum = 0.0f;
        if (lane < p.k)
#pragma unroll 8
          for (int l = 0; l < 32; ++l) sum += part[warp][lane][l];
        dots[warp][lane] = sum;
      }
    }
    if (p.dweights == nullptr) continue;
    __syncthreads();
    if (t < p.T && sub == 0 && lane < p.k) {
      float sum = 0.0f;
      for (int w = 0; w < p.per_token; ++w) sum += dots[warp + w][lane];
      if (index_ok(kSiteCStore, t * p.k + lane, 1, static_cast<long long>(p.T) * p.k)) p.dweights[t * p.k + lane] = sum;
    }
    __syncthreads();
  }
}

// -------------------------------------------------------------------- host --

template <class K>
int launch(K kernel, const P &p, long long blocks, int sms, cudaStream_t stream) {
  const long long most = 8LL * (sms > 0 ? sms : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? (blocks < 1 ? 1 : blocks) : most), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? kOk : kErrLaunch;
}

bool wide(const void *base, int64_t ld, int elem) {
  return base == nullptr || (reinterpret_cast<uintptr_t>(base) % 16 == 0 && ld * elem % 16 == 0);
}

// Rows in 16-byte loads?
bool fill(const RowsArgs &a, P *p) {
  const int elem = a.bf16 ? 2 : 4;
  const bool vec = a.D * elem % 16 == 0 && wide(a.token, a.ld_token, elem) &&
                   wide(a.expert, a.ld_expert, elem) && wide(a.out, a.ld_out, elem);
  *p = P{};
  p->token = a.token;
  p->expert = a.expert;
  p->out = a.out;
  p->places = a.places;
  p->weights = a.weights;
  p->dweights = a.dweights;
  p->ld_token = a.ld_token;
  p->ld_expert = a.ld_expert;
  p->ld_out = a.ld_out;
  p->token_extent = matrix_extent(a.T, a.D, a.ld_token);
  p->expert_extent = matrix_extent(a.rows, a.D, a.ld_expert);
  p->rows = a.rows;
  p->T = static_cast<int>(a.T);
  p->k = static_cast<int>(a.k);
  const int elems = vec ? 16 / elem : 1, u = vec ? 2 : 8;
  p->D = static_cast<int>(a.D / elems);
  p->pieces = (p->D + 32 * u - 1) / (32 * u);
  // As many warps a token as it has pieces: 64 tokens of 4096 bf16, six places,
  // dispatch, combine, backward with up to eight warps 9, 9, 11 us, with one 16, 24, 34;
  // of 8192 tokens the same but for dispatch (38 against 42; cold).
  p->per_token = 1;
  while (p->per_token < kWarps && p->per_token < p->pieces) p->per_token *= 2;
  return vec;
}

template <template <class, bool, int> class K, bool VEC, int PLACES>
int pick_type(bool bf16, const P &p, int sms, cudaStream_t s) {
  const int tokens = kWarps / p.per_token;
  const long long blocks = (static_cast<long long>(p.T) + tokens - 1) / tokens;
  return bf16 ? launch(K<__nv_bfloat16, VEC, PLACES>::kernel(), p, blocks, sms, s)
              : launch(K<float, VEC, PLACES>::kernel(), p, blocks, sms, s);
}

// Places in flight: what a token has, up to four (few registers, and so more
// warps, where it has one or two: combine of 8192 tokens of 4096 bf16 40 us, by the
// kernel of four 44, backward 71 and 82; cold).
template <template <class, bool, int> class K>
int pick(bool bf16, bool vec, const P &p, int sms, cudaStream_t s) {
  if (vec) return p.k <= 2 ? pick_type<K, true, 2>(bf16, p, sms, s) : pick_type<K, true, 4>(bf16, p, sms, s);
  return p.k <= 2 ? pick_type<K, false, 2>(bf16, p, sms, s) : pick_type<K, false, 4>(bf16, p, sms, s);
}

template <class T, bool VEC, int PLACES>
struct Dispatch {
  static auto kernel() { return dispatch_kernel<T, VEC, PLACES>; }
};
template <class T, bool VEC, int PLACES>
struct Combine {
  static auto kernel() { return combine_kernel<T, VEC, PLACES>; }
};
template <class T, bool VEC, int PLACES>
struct Backward {
  static auto kernel() { return backward_kernel<T, VEC, PLACES>; }
};

}  // namespace

GEMM_INDEX_FAULT_TAKE(rows_index_fault_take)

int rows_dispatch_launch(const RowsArgs &a, int sm_count, cudaStream_t stream) {
  P p;
  const bool vec = fill(a, &p);
  p.out_extent = matrix_extent(a.rows, a.D, a.ld_out);
  return pick<Dispatch>(a.bf16, vec, p, sm_count, stream);
}

int rows_combine_launch(const RowsArgs &a, int sm_count, cudaStream_t stream) {
  P p;
  const bool vec = fill(a, &p);
  p.out_extent = matrix_extent(a.T, a.D, a.ld_out);
  return pick<Combine>(a.bf16, vec, p, sm_count, stream);
}

int rows_backward_launch(const RowsArgs &a, int sm_count, cudaStream_t stream) {
  P p;
  const bool vec = fill(a, &p);
  p.out_extent = matrix_extent(a.rows, a.D, a.ld_out);
  // Warps of one token meet at its end: no more of them than fill the GPU (8192
  // tokens of 4096 bf16: 71 us, with eight warps a token 75; 1024: 18.6 and 17.5).
  while (p.per_token > 1 && a.T * p.per_token >= 32LL * sm_count) p.per_token /= 2;
  return pick<Backward>(a.bf16, vec, p, sm_count, stream);
}

}  // namespace gemm
