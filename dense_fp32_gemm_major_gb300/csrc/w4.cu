// w4.cu -- products of few rows with weights in 4 bits.
//
//   C[t, n] = sum_k A[t, k] W[n, k],   W[n, k] = s[n, k / group] (q[n, k] - z[n, k / group])
//
// With few rows the product is a reading of the weights: half a byte each, and
// its time that of memory as long as nothing else takes longer. What the kernel
// does about that:
//
//   * Weights come by TMA, 64 rows of 128 bytes (256 k) a stage, swizzled so that
//     the eight rows of a fragment lie in eight different groups of four banks.
//   * q - z is an integer that bf16 holds exactly. It is made by two logic
//     operations and one subtraction for two values: the nibbles q of a word, in
//     pairs 16 bits apart, become 128 + q by setting the bits above them, and 128
//     + z is taken away. mma.sync multiplies them with A (16 n by 8 rows by 16 k),
//     exactly, adding in fp32; the scales meet the sums, not the weights: at the
//     end of each group, at most 128 k, in fp32 registers. So no rounding of a
//     weight enters, and sums in the tensor core, which truncate, stay short.
//   * tcgen05 has nothing to give here: its smallest tile of lanes is 128 n, its
//     operands would have to go back to shared memory as bf16, four times the
//     bytes that came, and with eight rows an MMA of 16 x 8 x 16 a warp is enough
//     (one for every 2.7 KB that memory delivers).
//   * A stands in shared memory in the order of the fragments, which is that of
//     the nibbles: k in blocks of 32, lane j of four holding 8 neighbours as the
//     pairs (0, 4), (1, 5), (2, 6), (3, 7). fp32 values are three bf16 terms.
//   * Few tiles: the CTAs of a cluster share k, and add their sums from each
//     other's shared memory in the order of their ranks.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "ptx.cuh"
#include "w4.h"

namespace gemm {
namespace {

constexpr int kTileN = 64, kBlockK = 256, kStages = 4;
constexpr int kStageBytes = kTileN * kBlockK / 2;
constexpr int kConsumers = 128, kThreads = kConsumers + 32;
constexpr int kMaxSplit = 8;

__device__ int g_w4_status;  // first error recorded by a kernel of this unit

// A as fragments: for each tile of 8 rows and each block of 256 k, `terms` bf16
// terms and the 8 rows' factors. A segment's tiles follow each other from
// tile r0 / 8 + g on (r0: its first row, g: its number), which no two share.
struct Prep {
  const void *A;
  uint8_t *to;
  const int64_t *offsets;
  long long lda, a_extent, to_extent;
  int M, K, blocks, a_vec;
};

struct P {
  const uint8_t *A;  // Prep::to
  const void *scales;
  const uint8_t *zeros;
  void *C;
  const int64_t *offsets;
  long long a_extent, lds, strides, s_extent, ldz, stridez, z_extent, ldc, c_extent;
  int M, N, K, row_groups;
  int blocks, split;  // of k; CTAs that share them
  int per_group;      // times that the scales are applied to a group
  int z_step;         // 0: one matrix for all segments
  unsigned long long timeout_ns;
};

struct Shared {
  uint64_t full[kStages], empty[kStages];
  int abort, drain_abort;
};

// 1-D copy into this CTA's shared memory.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// D += A B: A 16 x 16, B 16 x 8, bf16, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nibbles i and i + 4 of a word, less z, as two bf16.
template <int I>
__device__ __forceinline__ uint32_t pair_of(uint32_t w, uint32_t zero) {
  const uint32_t v = (w >> (4 * I) & 0x000f000fu) | 0x43004300u;  // 128 + q
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&zero));
  return *reinterpret_cast<const uint32_t *>(&d);
}

__device__ __forceinline__ float read_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

// A's values from 2^113 on (and infinities, NaN) could leave fp32's range in a sum
// of 256 products with up to 15, although their products with the weights do
// not. A row's block of k with such values is taken 2^-16 times, and its sums
// 2^16 times.
constexpr float kShrink = 0x1p-16f, kGrow = 0x1p16f;

// Whether a word's two bf16 (or its fp32: the upper) have an exponent of 240 or more.
__device__ __forceinline__ uint32_t large(uint32_t u) {
  const uint32_t t = u & u << 1;
  return t & t << 2;
}

// Eight neighbouring k of a row, in the fragments' order, term by term; *shrink:
// kShrink times, for one of the warp's 256 is large.
template <class T>
__device__ __forceinline__ void load8(const Prep &p, long long at, int left, bool *shrink,
                                      uint4 (&out)[sizeof(T) == 2 ? 1 : 3]) {
  const T *a = static_cast<const T *>(p.A) + at;
  if constexpr (sizeof(T) == 2) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (left >= 8 && p.a_vec) {
      if (index_ok(kSiteLoadA, at, 8, p.a_extent)) v = __ldg(reinterpret_cast<const uint4 *>(a));
    } else {
      uint32_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        h[i] = i < left && index_ok(kSiteLoadA, at + i, 1, p.a_extent) ? bits(a[i]) : 0u;
      v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    const uint32_t big = large(v.x) | large(v.y) | large(v.z) | large(v.w);
    *shrink = __any_sync(0xffffffffu, (big & 0x40004000u) != 0);
    if (*shrink) {
      const __nv_bfloat162 f = __float2bfloat162_rn(kShrink);
      uint32_t *u = &v.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(u + i), f);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    out[0] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                        __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
  } else {
    float v[8];
    if (left >= 8 && p.a_vec) {
      float4 f[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      if (index_ok(kSiteLoadA, at, 8, p.a_extent)) {
        f[0] = __ldg(reinterpret_cast<const float4 *>(a));
        f[1] = __ldg(reinterpret_cast<const float4 *>(a) + 1);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[4 * i] = f[i].x;
        v[4 * i + 1] = f[i].y;
        v[4 * i + 2] = f[i].z;
        v[4 * i + 3] = f[i].w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = i < left && index_ok(kSiteLoadA, at + i, 1, p.a_extent) ? a[i] : 0.0f;
    }
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) big |= large(__float_as_uint(v[i]));
    *shrink = __any_sync(0xffffffffu, (big & 0x40000000u) != 0);
    if (*shrink)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= kShrink;
    uint32_t h[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // Of an infinite value there is no second term. (What is finite is far from
      // bf16's end: shrunk, if it was not.)
      const __nv_bfloat16 t0 = __float2bfloat16_rn(v[i]);
      const float r1 = isinf(v[i]) ? 0.0f : v[i] - __bfloat162float(t0);
      const __nv_bfloat16 t1 = __float2bfloat16_rn(r1);
      const __nv_bfloat16 t2 = __float2bfloat16_rn(r1 - __bfloat162float(t1));
      h[0][i] = bits(t0);
      h[1][i] = bits(t1);
      h[2][i] = bits(t2);
    }
#pragma unroll
    for (int t = 0; t < 3; ++t)
      out[t] = make_uint4(h[t][0] | h[t][4] << 16, h[t][1] | h[t][5] << 16,
                          h[t][2] | h[t][6] << 16, h[t][3] | h[t][7] << 16);
  }
}

template <class T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

__host__ __device__ constexpr int terms_of(int elem) { return elem == 2 ? 1 : 3; }
// Bytes of A for a tile of 8 rows and a block of k, and from one to the next.
__host__ __device__ constexpr int a_bytes(int elem) { return kBlockK * 8 * 2 * terms_of(elem) + 32; }
__host__ __device__ constexpr int a_step(int elem) { return a_bytes(elem) + 96; }

__device__ __forceinline__ long long held(long long a, long long m) {
  return a < 0 ? 0 : (a > m ? m : a);
}

__device__ __forceinline__ void segment_of(const int64_t *offsets, int g, int M, long long *r0,
                                           long long *r1) {
  *r0 = 0;
  *r1 = M;
  if (offsets != nullptr) {
    *r0 = held(offsets[g], M);
    *r1 = held(offsets[g + 1], M);
  }
}

constexpr int kPrepWarps = 4;

// A warp takes a block of k of a row: once for all CTAs that will read it.
template <class T>
__global__ void __launch_bounds__(32 * kPrepWarps) w4_prep_kernel(const Prep p) {
  constexpr int kTerms = terms_of(sizeof(T));
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, g = blockIdx.y;
  long long r0, r1;
  segment_of(p.offsets, g, p.M, &r0, &r1);
  if (r0 >= r1) return;
  const long long rows = (r1 - r0 + 7) / 8 * 8;  // the last tile's absent rows are zero
  for (long long u = static_cast<long long>(blockIdx.x) * kPrepWarps + threadIdx.x / 32;
       u < rows * p.blocks; u += static_cast<long long>(gridDim.x) * kPrepWarps) {
    const long long r = u / p.blocks;
    const int b = static_cast<int>(u - r * p.blocks), token = static_cast<int>(r & 7);
    const long long k = static_cast<long long>(b) * kBlockK + lane * 8;
    const long long left = r0 + r < r1 ? p.K - k : 0;
    uint4 v[kTerms];
    bool shrink;
    load8<T>(p, (r0 + r) * p.lda + k, left < 8 ? static_cast<int>(left) : 8, &shrink, v);
    const long long to = ((r0 / 8 + g + r / 8) * p.blocks + b) * a_step(sizeof(T));
    if (!index_ok(kSitePartialWrite, to, a_bytes(sizeof(T)), p.to_extent)) continue;
#pragma unroll
    for (int i = 0; i < kTerms; ++i)
      *reinterpret_cast<uint4 *>(p.to + to +
                                 ((lane / 4 * kTerms + i) * 32 + token * 4 + lane % 4) * 16) = v[i];
    if (lane == 0)
      *reinterpret_cast<float *>(p.to + to + kTerms * 4096 + token * 4) = shrink ? kGrow : 1.0f;
  }
}

// NT tiles of 8 rows at a time; the scales meet the sums every PERIOD steps of 32 k.
template <class T, int NT, int PERIOD>
__global__ void __launch_bounds__(kThreads)
    w4_kernel(const __grid_constant__ CUtensorMap map, const P p) {
  constexpr int kTerms = terms_of(sizeof(T)), kABytes = a_bytes(sizeof(T)), kAStep = a_step(sizeof(T));
  constexpr int kTimes = 8 / PERIOD;  // of a block
  extern __shared__ uint8_t raw[];
  uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
  uint8_t *as = stages + kStages * kStageBytes;  // kStages x NT tiles
  float *sums = reinterpret_cast<float *>(as + kStages * NT * kAStep);
  __shared__ Shared sh;

  const int warp = static_cast<int>(warp_index()), lane = threadIdx.x & 31;
  const int tile = static_cast<int>(blockIdx.x) / p.split, rank = static_cast<int>(blockIdx.x) % p.split;
  const int g = blockIdx.y, n0 = tile * kTileN;
  // What this launch reads but A was there before the one that makes A began
  // (each launch lets the next one in behind its own wait).
  long long r0, r1;
  segment_of(p.offsets, g, p.M, &r0, &r1);
  if (r0 >= r1) return;  // the whole cluster: it shares the segment
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kConsumers / 32);
    }
    sh.abort = sh.drain_abort = 0;
    fence_barrier_init();
    tma_prefetch_map(&map);
  }
  __syncthreads();
  const int b0 = static_cast<int>(static_cast<long long>(p.blocks) * rank / p.split);
  const int b1 = static_cast<int>(static_cast<long long>(p.blocks) * (rank + 1) / p.split);

  int stage = 0;
  uint32_t parity = 0;
  auto next = [&] {
    if (++stage == kStages) {
      stage = 0;
      parity ^= 1u;
    }
  };
  bool first = true;

  for (long long t0 = r0; t0 < r1; t0 += 8 * NT) {
    const int used = static_cast<int>(r1 - t0 >= 8 * NT ? NT : (r1 - t0 + 7) / 8);  // tiles
    if (warp == kConsumers / 32) {
      if (lane == 0) {
        auto load_w = [&](int b) {
          mbar_arrive_expect_tx(&sh.full[stage], kStageBytes + used * kABytes);
          tma_load_3d(stages + stage * kStageBytes, &map, &sh.full[stage], b * (kBlockK / 2), n0,
                      g * p.z_step);
        };
        auto load_a = [&](int b) {
          const long long at = ((r0 / 8 + g + (t0 - r0) / 8) * p.blocks + b) * kAStep;
          for (int i = 0; i < used; ++i) {
            const long long from = at + static_cast<long long>(i) * p.blocks * kAStep;
            bulk_load(as + (stage * NT + i) * kAStep, p.A + from, kABytes, &sh.full[stage]);
          }
        };
        int b = b0, issued = 0;
        if (first) {
          // The first weights are on their way while A is being made.
          for (; b < b1 && issued < kStages; ++b, ++issued) {
            load_w(b);
            next();
          }
          grid_dependency_wait();
          grid_launch_dependents();
          stage = 0;
          parity = 0;
          for (b = b0, issued = 0; b < b1 && issued < kStages; ++b, ++issued) {
            load_a(b);
            next();
          }
        }
        for (; b < b1; ++b, ++issued) {
          if (!mbar_wait_bounded(&sh.empty[stage], parity ^ 1u, p.timeout_ns, &sh.abort,
                                 &g_w4_status))
            break;
          load_w(b);
          load_a(b);
          next();
        }
        if (sh.abort) {
          // Given up: the copies under way land before anyone leaves.
          for (int i = issued < kStages ? issued : kStages; i > 0; --i) {
            const int at = (stage - i + kStages) % kStages;
            const uint32_t ph = stage - i < 0 ? parity ^ 1u : parity;
            mbar_wait_bounded(&sh.full[at], ph, p.timeout_ns, &sh.drain_abort, &g_w4_status);
          }
        }
      }
      __syncwarp();
      stage = __shfl_sync(0xffffffffu, stage, 0);
      parity = __shfl_sync(0xffffffffu, parity, 0);
    } else {
      const int row = warp * 16 + lane / 4, j = lane % 4, swz = row & 7;
      // Scales and zeros of two rows, a block ahead of their use. (Rows and groups
      // behind the last take its values: their products are not kept, or zero.)
      const long long n_lo = min(n0 + row, p.N - 1), n_hi = min(n0 + row + 8, p.N - 1);
      float s_next[kTimes][2];
      uint32_t z_next[kTimes][2];
      auto fetch = [&](int b) {
#pragma unroll
        for (int c = 0; c < kTimes; ++c) {
          const unsigned at = static_cast<unsigned>(b) * kTimes + c;
          const int gi = min(static_cast<int>(p.per_group == 1 ? at : at / p.per_group), p.row_groups - 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const long long n = h == 0 ? n_lo : n_hi;
            const long long i = g * p.strides + n * p.lds + gi;
            s_next[c][h] = index_ok(kSiteLoadB, i, 1, p.s_extent)
                               ? static_cast<float>(__ldg(static_cast<const T *>(p.scales) + i)) : 0.0f;
            z_next[c][h] = 8;
            if (p.zeros != nullptr) {
              const long long iz = g * p.stridez + n * p.ldz + gi;
              if (index_ok(kSiteLoadB, iz, 1, p.z_extent)) z_next[c][h] = __ldg(p.zeros + iz) & 15u;
            }
          }
        }
      };
      float sum[NT][4] = {};
      if (b0 < b1) fetch(b0);
      for (int b = b0; b < b1; ++b) {
        float s[kTimes][2];
        uint32_t z[kTimes][2];
#pragma unroll
        for (int c = 0; c < kTimes; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s[c][h] = s_next[c][h];
            z[c][h] = 0x43004300u | z_next[c][h] | z_next[c][h] << 16;
          }
        if (b + 1 < b1) fetch(b + 1);
        mbar_wait_bounded(&sh.full[stage], parity, p.timeout_ns, &sh.abort, &g_w4_status);
        const uint8_t *w0 = stages + stage * kStageBytes + row * 128 + j * 4;
        const uint8_t *ab = as + stage * NT * kAStep;
        float2 grow[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          grow[nt] = *reinterpret_cast<const float2 *>(ab + nt * kAStep + kTerms * 4096 + j * 8);
#pragma unroll
        for (int c = 0; c < kTimes; ++c) {
          float part[NT][2][4] = {};  // two sums, so that one's MMA need not wait for the other's
#pragma unroll
          for (int i = c * PERIOD; i < (c + 1) * PERIOD; ++i) {
            const uint32_t lo = *reinterpret_cast<const uint32_t *>(w0 + ((i ^ swz) << 4));
            const uint32_t hi = *reinterpret_cast<const uint32_t *>(w0 + 8 * 128 + ((i ^ swz) << 4));
            const uint32_t f0[4] = {pair_of<0>(lo, z[c][0]), pair_of<0>(hi, z[c][1]),
                                    pair_of<1>(lo, z[c][0]), pair_of<1>(hi, z[c][1])};
            const uint32_t f1[4] = {pair_of<2>(lo, z[c][0]), pair_of<2>(hi, z[c][1]),
                                    pair_of<3>(lo, z[c][0]), pair_of<3>(hi, z[c][1])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (nt >= used) continue;
#pragma unroll
              for (int t = kTerms - 1; t >= 0; --t) {  // small terms first
                const uint4 x = *reinterpret_cast<const uint4 *>(ab + nt * kAStep +
                                                                 (i * kTerms + t) * 512 + lane * 16);
                mma(part[nt][0], f0, x.x, x.y);
                mma(part[nt][1], f1, x.z, x.w);
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (nt >= used) continue;
            const float(&a)[4] = part[nt][0], (&d)[4] = part[nt][1];
            sum[nt][0] = fmaf(s[c][0] * grow[nt].x, a[0] + d[0], sum[nt][0]);
            sum[nt][1] = fmaf(s[c][0] * grow[nt].y, a[1] + d[1], sum[nt][1]);
            sum[nt][2] = fmaf(s[c][1] * grow[nt].x, a[2] + d[2], sum[nt][2]);
            sum[nt][3] = fmaf(s[c][1] * grow[nt].y, a[3] + d[3], sum[nt][3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);
        next();
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float *to = sums + (nt * 8 + 2 * j) * kTileN + row;
        to[0] = sum[nt][0];
        to[kTileN] = sum[nt][1];
        to[8] = sum[nt][2];
        to[kTileN + 8] = sum[nt][3];
      }
    }
    if (first) grid_dependency_wait();
    first = false;
    // All parts of the tile are there (cluster); this CTA's share of them.
    if (p.split > 1) cluster_sync();
    else __syncthreads();
    const int all = 8 * used * kTileN;
    const int e0 = all * rank / p.split, e1 = all * (rank + 1) / p.split;
    for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += kThreads) {
      const long long t = t0 + e / kTileN;
      const int n = n0 + e % kTileN;
      if (t >= r1 || n >= p.N) continue;
      float v;
      if (p.split == 1) {
        v = sums[e];
      } else {
        v = 0.0f;
        const uint32_t a = smem_addr(sums + e);
        for (int r = 0; r < p.split; ++r) v += read_cluster(a, static_cast<uint32_t>(r));
      }
      const long long at = t * p.ldc + n;
      if (index_ok(kSiteCStore, at, 1, p.c_extent)) static_cast<T *>(p.C)[at] = rounded<T>(v);
    }
    // nobody's sums are written again, or gone, before all are read
    if (p.split > 1) cluster_sync();
    else __syncthreads();
  }
}

// ------------------------------------------------- copies of the weights --

struct Copy {
  const uint8_t *src;
  uint8_t *dst;
  long long lds, strides, extent, ldd, strided, dst_extent;
  long long rows, count, bytes;
  const int64_t *offsets;
  long long M;
};

// A warp takes a row, a lane four bytes of it.
__global__ void __launch_bounds__(256) w4_pack_kernel(const Copy p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long words = p.ldd / 4;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32; i < p.rows * p.count;
       i += static_cast<long long>(gridDim.x) * 8) {
    const long long z = i / p.rows, row = i - z * p.rows;
    if (p.offsets != nullptr && held(p.offsets[z], p.M) >= held(p.offsets[z + 1], p.M)) continue;
    const long long from = z * p.strides + row * p.lds, to = z * p.strided + row * p.ldd;
    for (long long w = lane; w < words; w += 32) {
      uint32_t v = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (w * 4 + b < p.bytes && index_ok(kSiteCopySrc, from + w * 4 + b, 1, p.extent))
          v |= static_cast<uint32_t>(p.src[from + w * 4 + b]) << (8 * b);
      if (index_ok(kSiteCopyDst, to + w * 4, 4, p.dst_extent))
        *reinterpret_cast<uint32_t *>(p.dst + to + w * 4) = v;
    }
  }
}

struct Expand {
  const uint8_t *q, *zeros;
  const void *scales;
  void *hi, *lo;
  long long ldq, strideq, q_extent, lds, strides, s_extent, ldz, stridez, z_extent, ldd, d_extent;
  long long n0, rows, count;
  int K, group;
  const int64_t *offsets;
  long long M;
};

// A thread takes a byte: two neighbours of a row.
template <class T>
__global__ void __launch_bounds__(256) w4_expand_kernel(const Expand p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int half = (p.K + 1) / 2;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32; i < p.rows * p.count;
       i += static_cast<long long>(gridDim.x) * 8) {
    const long long z = i / p.rows, row = i - z * p.rows, n = p.n0 + row;
    if (p.offsets != nullptr && held(p.offsets[z], p.M) >= held(p.offsets[z + 1], p.M)) continue;
    const long long from = z * p.strideq + n * p.ldq, to = i * p.ldd;
    for (int b = lane; b < half; b += 32) {
      if (!index_ok(kSiteCopySrc, from + b, 1, p.q_extent)) continue;
      const int q = p.q[from + b], k = 2 * b, at = k / p.group;  // group is even
      const long long is = z * p.strides + n * p.lds + at, iz = z * p.stridez + n * p.ldz + at;
      if (!index_ok(kSiteLoadB, is, 1, p.s_extent)) continue;
      const float s = static_cast<float>(static_cast<const T *>(p.scales)[is]);
      int zero = 8;
      if (p.zeros != nullptr && index_ok(kSiteLoadB, iz, 1, p.z_extent)) zero = p.zeros[iz] & 15;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (k + e >= p.K || !index_ok(kSiteCopyDst, to + k + e, 1, p.d_extent)) continue;
        // exact but for fp32 scales of more than 20 bits
        const float w = s * static_cast<float>((q >> (4 * e) & 15) - zero);
        if constexpr (sizeof(T) == 4) {
          static_cast<float *>(p.hi)[to + k + e] = w;
        } else {
          const __nv_bfloat16 h = __float2bfloat16_rn(w);
          const float first = __bfloat162float(h);
          static_cast<__nv_bfloat16 *>(p.hi)[to + k + e] = h;
          static_cast<__nv_bfloat16 *>(p.lo)[to + k + e] =
              __float2bfloat16_rn(isinf(first) ? 0.0f : w - first);
        }
      }
    }
  }
}

// -------------------------------------------------------------------- host --

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

long long extent_of(int64_t count, int64_t stride, int64_t rows, int64_t cols, int64_t ld) {
  return (count - 1) * stride + matrix_extent(rows, cols, ld);
}

template <class K, class... A>
int launch(K kernel, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
           const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  // Above the 48 KiB default: kept by the current device, set where it is needed.
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return kErrLaunch;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? kOk : kErrLaunch;
}

template <class T, int NT, int PERIOD>
int launch_period(const CUtensorMap &map, const P &p, int groups, cudaStream_t stream) {
  const int tiles = (p.N + kTileN - 1) / kTileN;
  const size_t smem = 1024 + kStages * (kStageBytes + NT * a_step(sizeof(T))) + 8 * NT * kTileN * 4;
  return launch(w4_kernel<T, NT, PERIOD>,
                dim3(static_cast<unsigned>(tiles * p.split), static_cast<unsigned>(groups), 1), kThreads,
                smem, p.split, stream, map, p);
}

template <class T, int NT>
int launch_nt(const CUtensorMap &map, const P &p, int groups, int64_t group, cudaStream_t stream) {
  if (group % 256 == 0) return launch_period<T, NT, 8>(map, p, groups, stream);
  if (group % 128 == 0) return launch_period<T, NT, 4>(map, p, groups, stream);
  if (group % 64 == 0) return launch_period<T, NT, 2>(map, p, groups, stream);
  return launch_period<T, NT, 1>(map, p, groups, stream);
}

}  // namespace

GEMM_INDEX_FAULT_TAKE(w4_index_fault_take)

int w4_poll_status(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return kErrLaunch;
  int h = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&h, g_w4_status, sizeof(int)) != cudaSuccess) return kErrLaunch;
  if (h != 0 && cudaMemcpyToSymbol(g_w4_status, &zero, sizeof(int)) != cudaSuccess)
    return kErrLaunch;
  return h;
}

bool w4_readable(const W4Args &a) {
  return reinterpret_cast<uintptr_t>(a.Q) % 16 == 0 && a.ldq % 16 == 0 &&
         (a.groups <= 1 || a.strideq % 16 == 0);
}

int w4_launch(const W4Args &a, int sm_count, cudaStream_t stream) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return kErrLaunch;
  CUtensorMap map;
  const bool stack = a.groups > 1 && a.strideq > 0;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>((a.K + 1) / 2), static_cast<cuuint64_t>(a.N),
                              static_cast<cuuint64_t>(stack ? a.groups : 1)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.ldq),
                                 static_cast<cuuint64_t>(stack ? a.strideq : a.ldq)};
  const cuuint32_t box[3] = {kBlockK / 2, kTileN, 1}, step[3] = {1, 1, 1};
  if (fn(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(a.Q), dims, strides, box,
         step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return kErrLaunch;
  const int elem = a.bf16 ? 2 : 4;
  P p = {};
  p.row_groups = static_cast<int>((a.K + a.group - 1) / a.group);
  p.scales = a.scales;
  p.lds = a.lds;
  p.strides = a.strides;
  p.s_extent = extent_of(a.groups, a.strides, a.N, p.row_groups, a.lds);
  p.zeros = a.zeros;
  p.ldz = a.ldz;
  p.stridez = a.stridez;
  p.z_extent = extent_of(a.groups, a.stridez, a.N, p.row_groups, a.ldz);
  p.C = a.C;
  p.ldc = a.ldc;
  p.c_extent = matrix_extent(a.M, a.N, a.ldc);
  p.offsets = a.offsets;
  p.z_step = stack ? 1 : 0;
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.blocks = static_cast<int>((a.K + kBlockK - 1) / kBlockK);
  int period = 8;
  while (a.group % (32 * period) != 0) period /= 2;
  p.per_group = static_cast<int>(a.group / (32 * period));
  p.timeout_ns = 2000000000ull + 2000ull * static_cast<unsigned long long>(a.K);
  const int64_t tiles = (a.N + kTileN - 1) / kTileN;
  const int64_t used = a.groups < a.M ? a.groups : a.M;  // segments with rows, at most
  p.split = 1;
  while (p.split < kMaxSplit && 8 * p.split <= p.blocks && tiles * used * p.split < 4 * sm_count)
    p.split *= 2;

  Prep q = {};
  q.A = a.A;
  q.lda = a.lda;
  q.a_extent = matrix_extent(a.M, a.K, a.lda);
  q.a_vec = reinterpret_cast<uintptr_t>(a.A) % 16 == 0 && a.lda * elem % 16 == 0;
  q.offsets = a.offsets;
  q.M = p.M;
  q.K = p.K;
  q.blocks = p.blocks;
  q.to_extent = (a.M / 8 + a.groups + 1) * p.blocks * a_step(elem);
  void *ws = nullptr;
  int st = pool_alloc(&ws, static_cast<size_t>(q.to_extent), stream);
  if (st != kOk) return st;
  q.to = static_cast<uint8_t *>(ws);
  p.A = q.to;
  p.a_extent = q.to_extent;
  const int64_t average = (a.M + a.groups - 1) / a.groups;
  const int64_t prep = (average + 7) / 8 * 8 * p.blocks / kPrepWarps + 1;
  const dim3 grid(static_cast<unsigned>(prep < 4096 ? prep : 4096), static_cast<unsigned>(a.groups), 1);
  st = a.bf16 ? launch(w4_prep_kernel<__nv_bfloat16>, grid, 32 * kPrepWarps, 0, 1, stream, q)
              : launch(w4_prep_kernel<float>, grid, 32 * kPrepWarps, 0, 1, stream, q);
  // Rows at a time: what a segment has on average, or (few more instructions) twice
  // that; others take several turns.
  const int groups = static_cast<int>(a.groups);
  if (st == kOk) {
    if (a.bf16)
      st = a.M <= 8 || average <= 2 ? launch_nt<__nv_bfloat16, 1>(map, p, groups, a.group, stream)
           : average <= 12          ? launch_nt<__nv_bfloat16, 2>(map, p, groups, a.group, stream)
                                    : launch_nt<__nv_bfloat16, 4>(map, p, groups, a.group, stream);
    else
      st = a.M <= 8 || average <= 2 ? launch_nt<float, 1>(map, p, groups, a.group, stream)
                                    : launch_nt<float, 2>(map, p, groups, a.group, stream);
  }
  const int fst = pool_free(ws, stream);
  return st != kOk ? st : fst;
}

int w4_pack_launch(const W4Args &a, uint8_t *dst, int64_t ldd, int64_t strided, int sm_count,
                   cudaStream_t stream) {
  Copy p = {};
  p.src = a.Q;
  p.dst = dst;
  p.lds = a.ldq;
  p.strides = a.strideq;
  p.rows = a.N;
  p.count = a.strideq == 0 ? 1 : a.groups;
  p.bytes = (a.K + 1) / 2;
  p.extent = extent_of(p.count, a.strideq, a.N, p.bytes, a.ldq);
  p.ldd = ldd;
  p.strided = strided;
  p.dst_extent = extent_of(p.count, strided, a.N, ldd, ldd);
  p.offsets = p.count > 1 ? a.offsets : nullptr;
  p.M = a.M;
  const int64_t blocks = (p.rows * p.count + 7) / 8, most = 8LL * sm_count;
  return launch(w4_pack_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most), 1, 1),
                256, 0, 1, stream, p);
}

int w4_expand_launch(const W4Args &a, int64_t n0, int64_t rows, void *hi, void *lo, int64_t ldd,
                     int sm_count, cudaStream_t stream) {
  Expand p = {};
  const int64_t row_groups = (a.K + a.group - 1) / a.group;
  p.q = a.Q;
  p.zeros = a.zeros;
  p.scales = a.scales;
  p.hi = hi;
  p.lo = lo;
  p.ldq = a.ldq;
  p.strideq = a.strideq;
  p.q_extent = extent_of(a.groups, a.strideq, a.N, (a.K + 1) / 2, a.ldq);
  p.lds = a.lds;
  p.strides = a.strides;
  p.s_extent = extent_of(a.groups, a.strides, a.N, row_groups, a.lds);
  p.ldz = a.ldz;
  p.stridez = a.stridez;
  p.z_extent = extent_of(a.groups, a.stridez, a.N, row_groups, a.ldz);
  p.ldd = ldd;
  p.d_extent = a.groups * rows * ldd;
  p.n0 = n0;
  p.rows = rows;
  p.count = a.groups;
  p.K = static_cast<int>(a.K);
  p.group = static_cast<int>(a.group);
  p.offsets = a.offsets;
  p.M = a.M;
  const int64_t blocks = (rows * a.groups + 7) / 8, most = 8LL * sm_count;
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most), 1, 1);
  return a.bf16 ? launch(w4_expand_kernel<__nv_bfloat16>, grid, 256, 0, 1, stream, p)
                : launch(w4_expand_kernel<float>, grid, 256, 0, 1, stream, p);
}

}  // namespace gemm
