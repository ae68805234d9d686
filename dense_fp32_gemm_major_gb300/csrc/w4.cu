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

constexpr int kTileN = 64, kBlockK = 256, kStages = 6;
constexpr int kStageBytes = kTileN * kBlockK / 2;
constexpr int kConsumers = 128, kThreads = kConsumers + 32;
constexpr int kMaxSplit = 8;

__device__ int g_w4_status;  // first error recorded by a kernel of this unit

struct P {
  const void *A, *scales;
  const uint8_t *zeros;
  void *C;
  const int64_t *offsets;
  long long lda, a_extent, lds, strides, s_extent, ldz, stridez, z_extent, ldc, c_extent;
  int groups, M, N, K, group, row_groups;
  int split;      // CTAs that share a tile's k
  int phase;      // blocks of k whose A and scales stand in shared memory together
  int period;     // 32-k steps between two times the scales are applied
  int a_vec;      // A's rows in 16-byte loads
  int step_groups;  // groups that a phase may touch
  int z_step;       // 0: one matrix for all segments
  unsigned long long timeout_ns;
};

struct Shared {
  uint64_t full[kStages], empty[kStages];
  int abort, drain_abort;
};

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
// of 128 products with up to 15, although their products with the weights do
// not. Rows with such values are taken 2^-16 times, and their sums 2^16 times.
constexpr float kShrink = 0x1p-16f, kGrow = 0x1p16f;

// Whether a word's two bf16 (or its fp32: the upper) have an exponent of 240 or more.
__device__ __forceinline__ uint32_t large(uint32_t u) {
  const uint32_t t = u & u << 1;
  return t & t << 2;
}

// Eight neighbouring k of a row, in the fragments' order, term by term; whether
// one is large. `shrink`: kShrink times.
template <class T>
__device__ __forceinline__ bool load8(const P &p, long long at, int left, bool shrink,
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
    if (shrink) {
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
    return (big & 0x40004000u) != 0;
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
    for (int i = 0; i < 8; ++i) {
      big |= large(__float_as_uint(v[i]));
      if (shrink) v[i] *= kShrink;
    }
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
    return (big & 0x40000000u) != 0;
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
// Bytes of A in a block of k, for NT tiles of 8 rows.
__host__ __device__ constexpr int a_block_bytes(int nt, int elem) {
  return kBlockK * 8 * 2 * nt * terms_of(elem);
}

__device__ __forceinline__ long long held(long long a, long long m) {
  return a < 0 ? 0 : (a > m ? m : a);
}

// NT tiles of 8 rows at a time.
template <class T, int NT>
__global__ void __launch_bounds__(kThreads)
    w4_kernel(const __grid_constant__ CUtensorMap map, const P p) {
  constexpr int kTerms = terms_of(sizeof(T));
  extern __shared__ uint8_t raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) / 1024 * 1024);
  uint8_t *stages = base;
  uint8_t *as = stages + kStages * kStageBytes;
  float *sums = reinterpret_cast<float *>(as + p.phase * a_block_bytes(NT, sizeof(T)));
  float *scales = sums + 8 * NT * kTileN;                        // step_groups x 64
  uint32_t *zeros = reinterpret_cast<uint32_t *>(scales + p.step_groups * kTileN);
  __shared__ Shared sh;
  __shared__ int shrunk[8 * NT];  // rows whose A is taken kShrink times

  const int warp = static_cast<int>(warp_index()), lane = threadIdx.x & 31;
  const int tile = static_cast<int>(blockIdx.x) / p.split, rank = static_cast<int>(blockIdx.x) % p.split;
  const int g = blockIdx.y, n0 = tile * kTileN;
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
  grid_dependency_wait();
  grid_launch_dependents();

  long long r0 = 0, r1 = p.M;
  if (p.offsets != nullptr) {
    r0 = held(p.offsets[g], p.M);
    r1 = held(p.offsets[g + 1], p.M);
  }
  if (r0 >= r1) return;  // the whole cluster: it shares the segment
  const int blocks = (p.K + kBlockK - 1) / kBlockK;
  const int b0 = static_cast<int>(static_cast<long long>(blocks) * rank / p.split);
  const int b1 = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / p.split);

  int stage = 0;
  uint32_t parity = 0;
  auto next = [&] {
    if (++stage == kStages) {
      stage = 0;
      parity ^= 1u;
    }
  };

  for (long long t0 = r0; t0 < r1; t0 += 8 * NT) {
    if (warp == kConsumers / 32) {
      if (lane == 0) {
        int issued = 0;
        for (int b = b0; b < b1; ++b) {
          if (!mbar_wait_bounded(&sh.empty[stage], parity ^ 1u, p.timeout_ns, &sh.abort,
                                 &g_w4_status))
            break;
          mbar_arrive_expect_tx(&sh.full[stage], kStageBytes);
          tma_load_3d(stages + stage * kStageBytes, &map, &sh.full[stage], b * (kBlockK / 2), n0,
                      g * p.z_step);
          next();
          ++issued;
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
      float sum[NT][4] = {};
      for (int ph0 = b0; ph0 < b1; ph0 += p.phase) {
        const int ph1 = min(ph0 + p.phase, b1);
        named_barrier_sync(1, kConsumers);  // the phase before is read
        // A: rows t0 .. t0 + 8 NT, as fragments
        const int units = (ph1 - ph0) * 32;
        // (again: only the rows that are shrunk, or to see which are)
        auto stage_a = [&](bool again, bool look) {
          bool over = false;
          for (int u = threadIdx.x; u < units * 8 * NT; u += kConsumers) {
            const int token = u / units, k8 = u - token * units;  // k8: eight k
            const long long t = t0 + token;
            const long long k = static_cast<long long>(ph0) * kBlockK + k8 * 8;
            if (again && !look && !shrunk[token]) continue;
            uint4 v[kTerms];
#pragma unroll
            for (int i = 0; i < kTerms; ++i) v[i] = make_uint4(0, 0, 0, 0);
            if (t < r1 && k < p.K) {
              const long long left = p.K - k;
              const bool big = load8<T>(p, t * p.lda + k, left < 8 ? static_cast<int>(left) : 8,
                                        again && !look, v);
              over |= big;
              if (look && big) shrunk[token] = 1;
            }
            if (look) continue;
#pragma unroll
            for (int i = 0; i < kTerms; ++i)
              *reinterpret_cast<uint4 *>(
                  as + (((k8 / 4 * NT + token / 8) * kTerms + i) * 32 + token % 8 * 4 + k8 % 4) * 16) = v[i];
          }
          return over;
        };
        const bool over = stage_a(false, false);
        // scales and zeros of the groups that the phase meets
        const int g0 = ph0 * kBlockK / p.group;
        const int count = min((ph1 * kBlockK - 1) / p.group + 1, p.row_groups) - g0;
        for (int u = threadIdx.x; u < p.step_groups * kTileN; u += kConsumers) {
          const int r = u % kTileN, at = u / kTileN;
          float s = 0.0f;
          uint32_t z = 8;
          if (at < count && n0 + r < p.N) {
            const long long i = g * p.strides + (n0 + r) * p.lds + g0 + at;
            if (index_ok(kSiteLoadB, i, 1, p.s_extent))
              s = static_cast<float>(static_cast<const T *>(p.scales)[i]);
            if (p.zeros != nullptr) {
              const long long iz = g * p.stridez + (n0 + r) * p.ldz + g0 + at;
              if (index_ok(kSiteLoadB, iz, 1, p.z_extent)) z = p.zeros[iz] & 15u;
            }
          }
          scales[u] = s;
          zeros[u] = 0x43004300u | z | z << 16;
        }
        const bool plain = named_barrier_and(1, kConsumers, !over);
        if (!plain) {
          if (threadIdx.x < 8 * NT) shrunk[threadIdx.x] = 0;
          named_barrier_sync(1, kConsumers);
          stage_a(true, true);
          named_barrier_sync(1, kConsumers);
          stage_a(true, false);
          named_barrier_sync(1, kConsumers);
        }
        const int per_group = p.group / 32;
        int at_group = 0, in_group = ph0 * 8 - g0 * per_group;
        for (int b = ph0; b < ph1; ++b) {
          mbar_wait_bounded(&sh.full[stage], parity, p.timeout_ns, &sh.abort, &g_w4_status);
          const uint8_t *w0 = stages + stage * kStageBytes + row * 128 + j * 4;
          const uint8_t *ab = as + (b - ph0) * a_block_bytes(NT, sizeof(T)) + lane * 16;
          float part[NT][4] = {};
          int since = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t lo = *reinterpret_cast<const uint32_t *>(w0 + ((i ^ swz) << 4));
            const uint32_t hi = *reinterpret_cast<const uint32_t *>(w0 + 8 * 128 + ((i ^ swz) << 4));
            const uint32_t zlo = zeros[at_group * kTileN + row];
            const uint32_t zhi = zeros[at_group * kTileN + row + 8];
            const uint32_t f0[4] = {pair_of<0>(lo, zlo), pair_of<0>(hi, zhi), pair_of<1>(lo, zlo),
                                    pair_of<1>(hi, zhi)};
            const uint32_t f1[4] = {pair_of<2>(lo, zlo), pair_of<2>(hi, zhi), pair_of<3>(lo, zlo),
                                    pair_of<3>(hi, zhi)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int t = kTerms - 1; t >= 0; --t) {  // small terms first
                const uint4 x = *reinterpret_cast<const uint4 *>(ab + ((i * NT + nt) * kTerms + t) * 512);
                mma(part[nt], f0, x.x, x.y);
                mma(part[nt], f1, x.z, x.w);
              }
            if (++since == p.period) {
              const float s0 = scales[at_group * kTileN + row], s1 = scales[at_group * kTileN + row + 8];
              if (!plain) {
                // rows that are shrunk; the others as ever
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 2; ++c)
                    if (shrunk[nt * 8 + 2 * j + c]) {
                      sum[nt][c] = fmaf(s0 * part[nt][c], kGrow, sum[nt][c]);
                      sum[nt][c + 2] = fmaf(s1 * part[nt][c + 2], kGrow, sum[nt][c + 2]);
                      part[nt][c] = part[nt][c + 2] = 0.0f;
                    }
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                sum[nt][0] = fmaf(s0, part[nt][0], sum[nt][0]);
                sum[nt][1] = fmaf(s0, part[nt][1], sum[nt][1]);
                sum[nt][2] = fmaf(s1, part[nt][2], sum[nt][2]);
                sum[nt][3] = fmaf(s1, part[nt][3], sum[nt][3]);
                part[nt][0] = part[nt][1] = part[nt][2] = part[nt][3] = 0.0f;
              }
              since = 0;
            }
            if (++in_group == per_group) {
              in_group = 0;
              ++at_group;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.empty[stage]);
          next();
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float *s = sums + (nt * 8 + 2 * j) * kTileN + row;
        s[0] = sum[nt][0];
        s[kTileN] = sum[nt][1];
        s[8] = sum[nt][2];
        s[kTileN + 8] = sum[nt][3];
      }
    }
    // All parts of the tile are there (cluster); this CTA's share of them.
    if (p.split > 1) cluster_sync();
    else __syncthreads();
    const int all = 8 * NT * kTileN;
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

template <class T, int NT>
int launch_nt(const CUtensorMap &map, P &p, int sms, cudaStream_t stream) {
  const int tiles = (p.N + kTileN - 1) / kTileN, blocks = (p.K + kBlockK - 1) / kBlockK;
  const int used = p.groups < p.M ? p.groups : p.M;  // segments with rows, at most
  p.split = 1;
  while (p.split < kMaxSplit && 4 * p.split <= blocks &&
         static_cast<int64_t>(tiles) * used * p.split < 2 * sms)
    p.split *= 2;
  const int own = (blocks + p.split - 1) / p.split;
  const int room = 32 * 1024 / a_block_bytes(NT, sizeof(T));
  p.phase = own < room ? own : (room < 1 ? 1 : room);
  p.step_groups = (p.phase * kBlockK + p.group - 1) / p.group + 1;
  const size_t smem = 1024 + kStages * kStageBytes +
                      static_cast<size_t>(p.phase) * a_block_bytes(NT, sizeof(T)) +
                      8 * NT * kTileN * 4 + static_cast<size_t>(p.step_groups) * kTileN * 8;
  return launch(w4_kernel<T, NT>, dim3(static_cast<unsigned>(tiles * p.split), static_cast<unsigned>(p.groups), 1),
                kThreads, smem, p.split, stream, map, p);
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
  p.A = a.A;
  p.lda = a.lda;
  p.a_extent = matrix_extent(a.M, a.K, a.lda);
  p.a_vec = reinterpret_cast<uintptr_t>(a.A) % 16 == 0 && a.lda * elem % 16 == 0;
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
  p.groups = static_cast<int>(a.groups);
  p.z_step = stack ? 1 : 0;
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.group = static_cast<int>(a.group);
  p.period = a.group % 128 == 0 ? 4 : (a.group % 64 == 0 ? 2 : 1);
  p.timeout_ns = 2000000000ull + 2000ull * static_cast<unsigned long long>(a.K);
  // Rows at a time: what a segment has on average; others take several turns.
  const int64_t average = (a.M + a.groups - 1) / a.groups;
  if (a.bf16) {
    if (average <= 8) return launch_nt<__nv_bfloat16, 1>(map, p, sm_count, stream);
    if (average <= 16) return launch_nt<__nv_bfloat16, 2>(map, p, sm_count, stream);
    return launch_nt<__nv_bfloat16, 4>(map, p, sm_count, stream);
  }
  if (average <= 8) return launch_nt<float, 1>(map, p, sm_count, stream);
  return launch_nt<float, 2>(map, p, sm_count, stream);
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
