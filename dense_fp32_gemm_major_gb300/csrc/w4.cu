// w4.cu -- products of few rows with weights in 4 bits.
//
//   C[t, n] = sum_k A[t, k] W[n, k],   W[n, k] = s[n, k / group] (q[n, k] - z[n, k / group])
//
// With few rows the product is a reading of the weights: half a byte each, and
// its time that of memory as long as nothing else takes longer. Two things could:
// making operands of nibbles, and multiplying them.
//
//   * 128 rows of W are the lanes of a tcgen05 tile, the rows of A its columns.
//     (mma.sync multiplies 256 products a clock of an SM here, measured: at 8 rows
//     a third less than memory delivers; the first form of this kernel spent 83 %
//     of its time in it.)
//   * A bf16 whose upper eight bits are zero is its lower eight times 2^-133 (the
//     subnormals and the first normal values are one line). So the nibbles of a
//     word, in pairs 16 bits apart and moved to bits 4 to 7 of each half, are operands
//     16 q 2^-133: seven operations of the integer lanes for eight weights (memory at
//     full speed brings 47 weights a clock of an SM, its integer lanes do 64
//     operations). Not to bits 0 to 3, where four of them need no move: the tensor core
//     aligns the products of 16 k by their operands' exponents, which for subnormals is
//     that of 2^-126, and drops what lies 25 bits below the largest. So it keeps
//     products to 2^-22 of the largest |a| (to 2^-18 with q 2^-133, where sums of few or
//     very different values were off by up to nine times their bound). A is scaled by
//     2^106, to meet them in the middle of fp32's range; rows with values from 2^16 on by
//     less.
//   * sum s (q - z) a = s (sum q a - z sum a): the sums of A are made with A, a
//     term each, and are about as exact as the tensor core's, so that where q = z
//     nearly nothing is left.
//   * A thread makes a row's operands out of shared memory and stores them to TMEM,
//     where the tensor core reads them; shared memory would be written and read at
//     4 times the bytes.
//   * Scales and zeros meet the sums, in fp32, at the end of each group, at most
//     128 k: no weight is rounded, and sums in the tensor core, which truncate,
//     stay short. They are a value a thread.
//   * Two warpgroups take 128 k in turn, each with its own operand and accumulator
//     in TMEM: one makes operands while the other's are multiplied.
//   * A comes as the tensor core reads it (w4_prep_kernel, once a call; of one or two
//     rows the producer's warp makes it, a launch less): its k in
//     the order of the nibble pairs (0, 4), (1, 5), (2, 6), (3, 7); fp32 values as
//     three bf16 terms, each a column.
//   * Weights come by TMA, 128 rows of 256 k a stage, A by plain bulk copies.
//     Few tiles: the CTAs of a cluster share k, and add their sums from each
//     other's shared memory in the order of their ranks.
//
// Measured (launches by themselves with cold caches, group 128): one bf16 row of 4096 x
// 11008 17.5 us (23 MB: 1.3 TB/s; back to back, the weights in L2, 13.1), 64 rows of 8
// experts, 6 of them used, 54 us (142 MB: 2.7 TB/s of 6.8; back to back 53). Neither
// memory nor a pipe is what bounds it (integer lanes 39 %, tensor core 8 %), but the chain of a block: 128 k of operands are made and stored (about 700
// clocks), multiplied by eight dependent MMAs (118 clocks each), and read out (600),
// with four such chains an SM; and the MMAs of one thread start no closer than about
// 100 clocks, so that two CTAs an SM give 1600 clocks a block each at best, of 2500
// measured. Not kept: mma.sync 76 us; operands of 64 k, double buffered, 58; with two
// chains of accumulators 56; a warpgroup that reads sums for one that makes operands
// 64 to 66; two issuing threads 53; bigger hand-overs 87 (spills).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "seg_ptx.cuh"
#include "w4.h"

namespace gemm {
namespace {

constexpr int kTileN = 128, kBlockK = 256;
constexpr int kWBytes = kTileN * kBlockK / 2;  // of a stage
constexpr int kGroups = 2, kMakers = 128 * kGroups, kMakerWarps = kMakers / 32;  // make operands
constexpr int kProducer = kMakerWarps, kMma = kMakerWarps + 1;         // warps
constexpr int kThreads = kMakers + 64;
constexpr int kMaxSplit = 8;

__device__ int g_w4_status;  // first error recorded by a kernel of this unit

// A as operands: for each tile of rows and each block of 256 k, four panels of 64
// k (a line of 128 bytes for each row and term, swizzled); a byte a row, terms8's
// exponent; and the sums of the row's terms between two times that scales are
// applied.
struct Prep {
  const void *A;
  uint8_t *to;
  const int64_t *offsets;
  long long lda, a_extent, to_extent;
  int M, K, blocks, a_vec;
  int by_rows;  // see first_tile
};

// A segment's tiles follow each other from here on, which no two segments share (r0:
// its first row, g: its number): M / rows + groups of them, or M where that is less.
__host__ __device__ __forceinline__ long long first_tile(bool by_rows, long long r0, int rows, int g) {
  return by_rows ? r0 : r0 / rows + g;
}

struct P {
  const uint8_t *A;  // Prep::to
  const void *scales;
  const uint8_t *zeros;
  void *C;
  const int64_t *offsets;
  long long lds, strides, s_extent, ldz, stridez, z_extent, ldc, c_extent;
  int M, N, K, row_groups;
  int blocks, split;  // of k; CTAs that share them
  int per_group;      // times that the scales are applied to a group
  int z_step;         // 0: one matrix for all segments
  int by_rows;
  unsigned long long timeout_ns;
  Prep prep;  // A itself
};

struct Shared {
  uint64_t full_w[4], full_a[4], empty[4];  // stages, at most
  uint64_t made[kGroups], multiplied[kGroups], drain;
  uint32_t tmem;
  int abort, drain_abort;
};

// As mbar_wait_bounded, but asleep between looks (up to kNap ns each) instead of
// looking again at once: what waits here leaves the issue slots to the warps that
// make operands.
constexpr uint32_t kNap = 20000;
__device__ __forceinline__ bool nap_wait(uint64_t *bar, uint32_t parity, uint64_t timeout_ns,
                                         volatile int *abort, int *status) {
  const uint32_t a = smem_addr(bar);
  auto look = [&] {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(a), "r"(parity), "r"(kNap)
        : "memory");
    return done != 0;
  };
  if (look()) return true;
  const uint64_t t0 = global_timer_ns();
  while (!look()) {
    if (*abort) return false;
    if (global_timer_ns() - t0 > timeout_ns) {
      *abort = 1;
      atomicCAS(status, 0, kStatusTimeout);
      return false;
    }
  }
  return true;
}

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

// Loads that stay where they are written: ahead of their use, which the compiler
// would move them back to.
__device__ __forceinline__ float load_ahead(const float *p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ __nv_bfloat16 load_ahead(const __nv_bfloat16 *p) {
  unsigned short v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return __ushort_as_bfloat16(v);
}
__device__ __forceinline__ uint32_t load_ahead(const uint8_t *p) {
  uint32_t v;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// D[tmem] (+)= A[tmem] B[smem]^T, kind::f16 with bf16 operands, 128 lanes.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f16: D fp32 (bits 4-5 = 1), A and B bf16 (bits
// 7-9 and 10-12 = 1), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t m, uint32_t n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

__device__ __forceinline__ float read_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

// Exponents of A's scaling (powers of two): kScale as long as a row's 256 values
// are below 2^16 (biased exponent kLargest); else, that of the largest of them
// above kLargest less. fp32 values that are all below 2^-60 (kSmallest) kMore more:
// their products' last bits, of the third term, would be below 2^-149 from 2^-102 on.
// Sums are of units of 2^-129, a weight's (16 2^-133).
constexpr int kScale = 106, kUnit = 129, kLargest = 127 + 15, kSmallest = 127 - 60, kMore = 16;
constexpr float kLargeScale = 0x1p104f;

__device__ __forceinline__ float power(int e) {  // 2^e, e in -126 .. 127
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

__host__ __device__ constexpr int terms_of(int elem) { return elem == 2 ? 1 : 3; }

// Eight neighbouring k of a row, `left` of which there are.
template <class T>
__device__ __forceinline__ void load8(const Prep &p, long long at, long long left, float (&v)[8]) {
  const T *a = static_cast<const T *>(p.A) + at;
  if (left >= 8 && p.a_vec && index_ok(kSiteLoadA, at, 8, p.a_extent)) {
    if constexpr (sizeof(T) == 2) {
      const uint4 w = __ldg(reinterpret_cast<const uint4 *>(a));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(a) + i);
        v[4 * i] = f.x;
        v[4 * i + 1] = f.y;
        v[4 * i + 2] = f.z;
        v[4 * i + 3] = f.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = i < left && index_ok(kSiteLoadA, at + i, 1, p.a_extent) ? static_cast<float>(a[i]) : 0.0f;
  }
}

// They as operands, term by term, and their sums, those of A's scaled values times
// 2^-kUnit; returns how much less than by kScale the warp's 256 values are scaled.
template <class T>
__device__ __forceinline__ int terms8(const float (&v)[8], uint4 (&out)[terms_of(sizeof(T))],
                                      float (&sum)[terms_of(sizeof(T))]) {
  constexpr int kTerms = terms_of(sizeof(T));
  unsigned e = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) e = max(e, __float_as_uint(v[i]) >> 23 & 0xffu);
  e = __reduce_max_sync(0xffffffffu, e);
  int less = static_cast<int>(e) > kLargest ? static_cast<int>(e) - kLargest : 0;
  if constexpr (kTerms > 1)
    if (e != 0 && e < kSmallest) less = -kMore;
  const float scale = power(kScale - less);
#pragma unroll
  for (int t = 0; t < kTerms; ++t) sum[t] = 0.0f;
  uint32_t h[kTerms][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float rest = v[i] * scale;
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
      const __nv_bfloat16 term = __float2bfloat16_rn(rest);
      const float f = __bfloat162float(term);
      sum[t] += f * 0x1p-100f;
      h[t][i] = __bfloat16_as_ushort(term);
      rest = isinf(f) ? 0.0f : rest - f;  // of infinity there is no second term
    }
  }
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    sum[t] *= 0x1p-29f;
    out[t] = make_uint4(h[t][0] | h[t][4] << 16, h[t][1] | h[t][5] << 16, h[t][2] | h[t][6] << 16,
                        h[t][3] | h[t][7] << 16);
  }
  return less;
}

template <class T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// A tile of rows: COLS columns of the tensor core (a multiple of 16), a column for
// each term of a row; the scales are applied every PERIOD steps of 32 k.
template <class T, int COLS, int PERIOD>
struct Tile {
  static constexpr int kTerms = terms_of(sizeof(T)), kRows = COLS / kTerms;
  static constexpr int kTimes = 8 / PERIOD;  // of a block of 256 k
  static constexpr int kPanel = COLS * 128;
  static constexpr int kFlags = 4 * kPanel, kSums = kFlags + (kRows <= 16 ? 16 : kRows);
  static constexpr int kBytes = kSums + (kTimes * kTerms * kRows * 4 + 15) / 16 * 16;  // of a block
  static constexpr int kStep = (kBytes + 1023) / 1024 * 1024;  // from one to the next
};

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

// A row of a tile's block, by a warp with 8 values a lane.
template <class T, class A, int PERIOD>
__device__ __forceinline__ void put_row(const float (&v)[8], uint8_t *to, int row) {
  const int lane = threadIdx.x & 31;
  uint4 w[A::kTerms];
  float sum[A::kTerms];
  const int less = terms8<T>(v, w, sum);
#pragma unroll
  for (int i = 0; i < A::kTerms; ++i)
#pragma unroll
    for (int d = 1; d < 4 * PERIOD; d *= 2) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], d);
  uint8_t *panel = to + lane / 8 * A::kPanel;
  float *sums = reinterpret_cast<float *>(to + A::kSums);
#pragma unroll
  for (int i = 0; i < A::kTerms; ++i) {
    const int line = i * A::kRows + row;
    *reinterpret_cast<uint4 *>(panel + line * 128 + ((lane % 8 ^ (line & 7)) << 4)) = w[i];
    if (lane % (4 * PERIOD) == 0) sums[(lane / (4 * PERIOD) * A::kTerms + i) * A::kRows + row] = sum[i];
  }
  if (lane == 0) to[A::kFlags + row] = static_cast<uint8_t>(less);
}

constexpr int kPrepWarps = 4;

// A warp takes a block of k of a row: once for all CTAs that will read it. (3 to 4 us, a
// launch; without it every CTA made its own: 64 rows of 8 experts took 268 us, not 66.)
template <class T, int COLS, int PERIOD>
__global__ void __launch_bounds__(32 * kPrepWarps) w4_prep_kernel(const Prep p) {
  using A = Tile<T, COLS, PERIOD>;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, g = blockIdx.y;
  long long r0, r1;
  segment_of(p.offsets, g, p.M, &r0, &r1);
  if (r0 >= r1) return;
  const long long rows = (r1 - r0 + A::kRows - 1) / A::kRows * A::kRows;  // absent rows are zero
  for (long long u = static_cast<long long>(blockIdx.x) * kPrepWarps + threadIdx.x / 32;
       u < rows * p.blocks; u += static_cast<long long>(gridDim.x) * kPrepWarps) {
    const long long r = u / p.blocks;
    const int b = static_cast<int>(u - r * p.blocks), row = static_cast<int>(r % A::kRows);
    const long long k = static_cast<long long>(b) * kBlockK + lane * 8;
    const long long left = r0 + r < r1 ? p.K - k : 0;
    float v[8];
    load8<T>(p, (r0 + r) * p.lda + k, left, v);
    const long long to = ((first_tile(p.by_rows, r0, A::kRows, g) + r / A::kRows) * p.blocks + b) * A::kStep;
    if (index_ok(kSitePartialWrite, to, A::kBytes, p.to_extent)) put_row<T, A, PERIOD>(v, p.to + to, row);
  }
}

// Columns of TMEM: an operand (128 k, two a column) for each warpgroup, and its
// accumulators, one for each time that the scales are applied.
__host__ __device__ constexpr int tmem_columns(int cols, int times) {
  return kGroups * (64 + cols * times) <= 256 ? 256 : 512;
}

// Stages: what shared memory has room for, twice an SM up to 32 columns.
__host__ __device__ constexpr int stages_of(int cols) { return cols == 32 || cols == 96 ? 3 : 4; }

// Rows of a call up to which the kernel makes A's operands itself, in the producer's
// warp of every CTA (fp32: one, three terms). Of 4096 x 11008, one launch | two, GPU
// time of bf16: 1 row 16.5 | 16.6 us, 2 rows 16.8 | 16.8, 4 rows 22.6 | 17.1; of fp32:
// 1 row 16.6 | 16.7, 2 rows 19.5 | 16.7. The launch and its workspace that this saves
// are 4 us of the host, of 19 from Python.
constexpr int kMakeRows = 2;
constexpr int make_rows(int elem) { return elem == 2 ? kMakeRows : 1; }

// The scales meet the sums every PERIOD steps of 32 k. MAKE: of up to make_rows rows.
template <class T, int COLS, int PERIOD, bool MAKE>
__global__ void __launch_bounds__(kThreads, COLS <= 32 && tmem_columns(COLS, 4 / PERIOD) == 256 ? 2 : 1)
    w4_kernel(const __grid_constant__ CUtensorMap map, const P p) {
  using A = Tile<T, COLS, PERIOD>;
  constexpr int kTimes = A::kTimes / kGroups, kColumns = tmem_columns(COLS, kTimes), kStages = stages_of(COLS);
  extern __shared__ uint8_t raw[];
  uint8_t *ws = raw + (-smem_addr(raw) & 1023u);  // (an offset: the compiler still sees shared memory)
  uint8_t *as = ws + kStages * kWBytes;
  // the warpgroups' sums of a tile, when all stages have been used
  float *sums = reinterpret_cast<float *>(ws);
  __shared__ Shared sh;

  const int warp = static_cast<int>(warp_index()), lane = threadIdx.x & 31;
  const int tile = static_cast<int>(blockIdx.x) / p.split, rank = static_cast<int>(blockIdx.x) % p.split;
  const int g = blockIdx.y, n0 = tile * kTileN;
  if constexpr (MAKE) {
    grid_dependency_wait();
    grid_launch_dependents();
  }
  // (Else: what this launch reads but A was there before the one that makes A began;
  // each launch lets the next one in behind its own wait.)
  long long r0, r1;
  segment_of(p.offsets, g, p.M, &r0, &r1);
  if (r0 >= r1) {  // the whole cluster: it shares the segment
    // A launch behind this one counts on this one's end being that of the one before.
    if constexpr (!MAKE) grid_dependency_wait();
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full_w[i], 1);
      mbar_init(&sh.full_a[i], 1);
      mbar_init(&sh.empty[i], kMakerWarps + 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&sh.made[i], 4);
      mbar_init(&sh.multiplied[i], 1);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = sh.drain_abort = 0;
    fence_barrier_init();
    tma_prefetch_map(&map);
  }
  if (warp == kMma) {
    tmem_alloc<1>(&sh.tmem, kColumns);
    tmem_relinquish<1>();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const int b0 = static_cast<int>(static_cast<long long>(p.blocks) * rank / p.split);
  const int b1 = static_cast<int>(static_cast<long long>(p.blocks) * (rank + 1) / p.split);

  int stage = 0;
  uint32_t parity = 0, phase = 0;  // of the stages, and of made and multiplied
  auto next = [&] {
    if (++stage == kStages) {
      stage = 0;
      parity ^= 1u;
    }
  };
  auto wait = [&](uint64_t *bar, uint32_t ph) {
    return nap_wait(bar, ph, p.timeout_ns, &sh.abort, &g_w4_status);
  };
  bool first = true;

  for (long long t0 = r0; t0 < r1; t0 += A::kRows) {
    if (warp == kProducer && MAKE) {
      const int used = static_cast<int>(min(static_cast<long long>(A::kRows), r1 - t0));
      int ahead = stage, b_w = b0;  // lane 0's weights, up to kStages blocks ahead
      uint32_t ahead_parity = parity;
      auto load_w = [&] {
        if (!wait(&sh.empty[ahead], ahead_parity ^ 1u)) return false;
        mbar_arrive_expect_tx(&sh.full_w[ahead], kWBytes);
        tma_load_3d(ws + ahead * kWBytes, &map, &sh.full_w[ahead], b_w * (kBlockK / 2), n0, g * p.z_step);
        ++b_w;
        if (++ahead == kStages) {
          ahead = 0;
          ahead_parity ^= 1u;
        }
        return true;
      };
      if (lane == 0)
        while (b_w < b1 && b_w - b0 < kStages && load_w()) {}
      __syncwarp();
      // rows that are not there are zero, in all stages
      for (int i = lane; i < kStages * A::kStep / 16; i += 32)
        reinterpret_cast<uint4 *>(as)[i] = make_uint4(0, 0, 0, 0);
      __syncwarp();
      for (int b = b0; b < b1; ++b) {
        bool ok = true;
        if (b - b0 >= kStages) {
          if (lane == 0) ok = load_w();  // (and the stage is empty)
          ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok) break;
        __syncwarp();
        uint8_t *to = as + stage * A::kStep;
        const long long k = static_cast<long long>(b) * kBlockK + lane * 8;
        float v[kMakeRows][8];
#pragma unroll
        for (int i = 0; i < kMakeRows; ++i)
          if (i < used) load8<T>(p.prep, (t0 + i) * p.prep.lda + k, p.K - k, v[i]);
#pragma unroll
        for (int i = 0; i < kMakeRows; ++i)
          if (i < used) put_row<T, A, PERIOD>(v[i], to, i);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full_a[stage]);
        next();
      }
      if (lane == 0 && sh.abort) {
        // Given up: the copies under way land before anyone leaves.
        for (int i = min(b_w - b0, kStages); i > 0; --i)
          mbar_wait_bounded(&sh.full_w[(ahead - i + kStages) % kStages],
                            ahead - i < 0 ? ahead_parity ^ 1u : ahead_parity, p.timeout_ns,
                            &sh.drain_abort, &g_w4_status);
      }
      __syncwarp();
    } else if (warp == kProducer) {
      if (lane == 0) {
        const long long at = (first_tile(p.by_rows, r0, A::kRows, g) + (t0 - r0) / A::kRows) * p.blocks;
        auto load_w = [&](int b) {
          mbar_arrive_expect_tx(&sh.full_w[stage], kWBytes);
          tma_load_3d(ws + stage * kWBytes, &map, &sh.full_w[stage], b * (kBlockK / 2), n0,
                      g * p.z_step);
        };
        auto load_a = [&](int b) {
          mbar_arrive_expect_tx(&sh.full_a[stage], A::kBytes);
          bulk_load(as + stage * A::kStep, p.A + (at + b) * A::kStep, A::kBytes, &sh.full_a[stage]);
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
          if (!wait(&sh.empty[stage], parity ^ 1u)) break;
          load_w(b);
          load_a(b);
          next();
        }
        if (sh.abort) {
          // Given up: the copies under way land before anyone leaves.
          for (int i = issued < kStages ? issued : kStages; i > 0; --i) {
            const int s = (stage - i + kStages) % kStages;
            const uint32_t ph = stage - i < 0 ? parity ^ 1u : parity;
            mbar_wait_bounded(&sh.full_w[s], ph, p.timeout_ns, &sh.drain_abort, &g_w4_status);
            mbar_wait_bounded(&sh.full_a[s], ph, p.timeout_ns, &sh.drain_abort, &g_w4_status);
          }
        }
      }
      __syncwarp();
      stage = __shfl_sync(0xffffffffu, stage, 0);
      parity = __shfl_sync(0xffffffffu, parity, 0);
    } else if (warp == kMma) {
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_bf16(kTileN, COLS);
        bool ok = true;
        for (int b = b0; ok && b < b1; ++b) {
          ok = wait(&sh.full_a[stage], parity);
          const uint64_t desc = smem_desc(smem_addr(as + stage * A::kStep), 16, 1024, 2);
#pragma unroll
          for (int h = 0; h < kGroups; ++h) {
            // the operand is there, and the accumulators have been read
            ok = ok && wait(&sh.made[h], phase);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t a = tmem + h * 64, d = tmem + kGroups * 64 + h * COLS * kTimes;
#pragma unroll
            for (int i = 0; i < 8; ++i)  // steps of 16 k
              mma_bf16_ts(d + i / (2 * PERIOD) * COLS, a + i * 8,
                          desc + (((h * 2 + i / 4) * A::kPanel + i % 4 * 32) >> 4), idesc,
                          i % (2 * PERIOD) != 0);
            mma_commit(&sh.multiplied[h]);
          }
          if (ok) mma_commit(&sh.empty[stage]);
          phase ^= 1u;
          next();
        }
        if (sh.abort) {
          // Given up: the MMAs under way end before TMEM is freed.
          mma_commit(&sh.drain);
          mbar_wait_bounded(&sh.drain, 0, p.timeout_ns, &sh.drain_abort, &g_w4_status);
        }
      }
      __syncwarp();
      stage = __shfl_sync(0xffffffffu, stage, 0);
      parity = __shfl_sync(0xffffffffu, parity, 0);
      phase = __shfl_sync(0xffffffffu, phase, 0);
    } else {
      const int h = warp / 4, row = warp % 4 * 32 + lane;
      const uint32_t lanes = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16);
      const uint32_t a_tmem = lanes + h * 64, d_tmem = lanes + kGroups * 64 + h * COLS * kTimes;
      // The row's scales and zeros, a block ahead of their use. (A row or a group
      // behind the last takes its values: its products are not kept, or zero.)
      const long long n = min(n0 + row, p.N - 1);
      const long long s_at = g * p.strides + n * p.lds, z_at = g * p.stridez + n * p.ldz;
      T s_next[kTimes];
      uint32_t z_next[kTimes];
      auto fetch = [&](int b) {
#pragma unroll
        for (int c = 0; c < kTimes; ++c) {
          const unsigned at = (static_cast<unsigned>(b) * kGroups + h) * kTimes + c;
          const int gi = min(static_cast<int>(p.per_group == 1 ? at : at / p.per_group), p.row_groups - 1);
          s_next[c] = index_ok(kSiteLoadB, s_at + gi, 1, p.s_extent)
                          ? load_ahead(static_cast<const T *>(p.scales) + s_at + gi) : T(0.0f);
          z_next[c] = 8;
          if (p.zeros != nullptr && index_ok(kSiteLoadB, z_at + gi, 1, p.z_extent))
            z_next[c] = load_ahead(p.zeros + z_at + gi);
        }
      };
      float sum[A::kRows] = {}, s_now[kTimes], z_now[kTimes];

      // Adds the accumulators of the block before, which stands in stage `at`, to
      // the sums: u = sum q a - z sum a for every row, in units of 2^(kScale - kUnit).
      auto drain_as = [&](auto is_large, const uint8_t *at) {
        constexpr bool LARGE = decltype(is_large)::value;
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < kTimes; ++c) {
          uint32_t v[COLS / 16][16];
#pragma unroll
          for (int i = 0; i < COLS / 16; ++i) tmem_load_16cols(d_tmem + c * COLS + i * 16, v[i]);
          tmem_load_wait();
#pragma unroll
          for (int i = 0; i < COLS / 16; ++i) tmem_regs_ready(v[i]);
          const float *asums =
              reinterpret_cast<const float *>(at + A::kSums) + (h * kTimes + c) * A::kTerms * A::kRows;
          // From 2^104 on a scale and the unit of the sums are two factors.
          const bool apart = LARGE && !(fabsf(s_now[c]) < kLargeScale);
          const float s = apart ? s_now[c] : s_now[c] * power(kUnit - kScale);
          [[maybe_unused]] const float unit = apart ? power(kUnit - kScale) : 1.0f;
          [[maybe_unused]] float as4[4];
#pragma unroll
          for (int t = 0; t < A::kRows; ++t) {
            float u;
            if constexpr (A::kTerms == 1) {
              if (t % 4 == 0) {
                const float4 f = *reinterpret_cast<const float4 *>(asums + t);
                as4[0] = f.x;
                as4[1] = f.y;
                as4[2] = f.z;
                as4[3] = f.w;
              }
              u = fmaf(-z_now[c], as4[t % 4], __uint_as_float(v[t / 16][t % 16]));
            } else {
              u = 0.0f;
#pragma unroll
              for (int i = A::kTerms - 1; i >= 0; --i) {  // small terms first
                const int col = i * A::kRows + t;
                u += fmaf(-z_now[c], asums[col], __uint_as_float(v[col / 16][col % 16]));
              }
            }
            // (exact: A is scaled by that much less; by more, the scale is, lest u leaves
            // the normal numbers)
            if constexpr (LARGE && A::kTerms > 1) {
              const int less = static_cast<int8_t>(at[A::kFlags + t]);
              const float f = power(less);
              sum[t] = fmaf(less < 0 ? s * f : s, (less < 0 ? u : u * f) * unit, sum[t]);
              continue;
            }
            if constexpr (LARGE) u = u * power(at[A::kFlags + t]) * unit;
            sum[t] = fmaf(s, u, sum[t]);
          }
        }
        tc_fence_before_sync();
      };
      auto drain = [&](int of, uint32_t ph) {
        wait(&sh.multiplied[h], phase ^ 1u);
        wait(&sh.full_a[of], ph);  // (long since)
        const uint8_t *at = as + of * A::kStep;
        const uint32_t *flags = reinterpret_cast<const uint32_t *>(at + A::kFlags);
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < A::kRows / 4; ++i) any |= flags[i];
        if constexpr (A::kRows % 4 != 0) any |= flags[A::kRows / 4] & ((1u << (A::kRows % 4 * 8)) - 1u);
        bool large = any != 0;
#pragma unroll
        for (int c = 0; c < kTimes; ++c) large |= !(fabsf(s_now[c]) < kLargeScale);
        // (the warp's choice: all its lanes read TMEM together)
        if (__any_sync(0xffffffffu, large)) drain_as(std::true_type{}, at);
        else drain_as(std::false_type{}, at);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[of]);
      };
      if (b0 < b1) fetch(b0);
      int before = 0;  // the stage of the block before, and its parity
      uint32_t before_parity = 0;
      for (int b = b0; b < b1; ++b) {
        float s[kTimes], z[kTimes];
#pragma unroll
        for (int c = 0; c < kTimes; ++c) {
          s[c] = static_cast<float>(s_next[c]);
          z[c] = static_cast<float>(z_next[c] & 15u);
        }
        if (b + 1 < b1) fetch(b + 1);
        wait(&sh.full_w[stage], parity);
        __syncwarp();  // together again, for TMEM
        const uint8_t *line = ws + stage * kWBytes + row * 128;
        // 64 k of the line: 32 columns of the operand
        auto make = [&](int q, uint32_t (&v)[32]) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int chunk = h * 4 + q * 2 + c;  // 32 k
            const uint4 w = *reinterpret_cast<const uint4 *>(line + ((chunk ^ (row & 7)) << 4));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[c * 16 + i * 4] = u[i] << 4 & 0x00f000f0u;
              v[c * 16 + i * 4 + 1] = u[i] & 0x00f000f0u;
              v[c * 16 + i * 4 + 2] = u[i] >> 4 & 0x00f000f0u;
              v[c * 16 + i * 4 + 3] = u[i] >> 8 & 0x00f000f0u;
            }
          }
        };
        uint32_t v[32];
        make(0, v);
        if (b > b0) drain(before, before_parity);
#pragma unroll
        for (int c = 0; c < kTimes; ++c) {
          s_now[c] = s[c];
          z_now[c] = z[c];
        }
        tmem_store_32cols(a_tmem, v);
        make(1, v);
        tmem_store_32cols(a_tmem + 32, v);
        tmem_store_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.made[h]);
        before = stage;
        before_parity = parity;
        phase ^= 1u;
        next();
      }
      if (b0 < b1) drain(before, before_parity);
      // Every copy has landed and been used: the other warpgroup's too, once it
      // is here.
      named_barrier_sync(1, kMakers);
#pragma unroll
      for (int t = 0; t < A::kRows; ++t) sums[(h * A::kRows + t) * kTileN + row] = sum[t];
    }
    if (first) grid_dependency_wait();
    first = false;
    // All parts of the tile are there (cluster); this CTA's share of them.
    if (p.split > 1) cluster_sync();
    else __syncthreads();
    const int used = static_cast<int>(min(static_cast<long long>(A::kRows), r1 - t0));
    const int all = used * kTileN;
    const int e0 = all * rank / p.split, e1 = all * (rank + 1) / p.split;
    for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += kThreads) {
      const int n = n0 + e % kTileN;
      if (n >= p.N) continue;
      float v = 0.0f;
      if (p.split == 1) {
        v = sums[e] + sums[A::kRows * kTileN + e];
      } else {
        const uint32_t a = smem_addr(sums + e);
        for (int r = 0; r < p.split; ++r)
          v += read_cluster(a, static_cast<uint32_t>(r)) +
               read_cluster(a + A::kRows * kTileN * 4, static_cast<uint32_t>(r));
      }
      const long long at = (t0 + e / kTileN) * p.ldc + n;
      if (index_ok(kSiteCStore, at, 1, p.c_extent)) static_cast<T *>(p.C)[at] = rounded<T>(v);
    }
    // Nobody's sums are gone, or overwritten by copies, before all are read.
    fence_proxy_async_smem();
    if (p.split > 1) cluster_sync();
    else __syncthreads();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after_sync();
    tmem_dealloc<1>(tmem, kColumns);
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

// A warp takes a row, a lane four bytes of it. (1531 x 389 bytes: 4.7 us, of which a
// launch is most.)
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
  int K, group, words;  // q in words of four bytes?
  const int64_t *offsets;
  long long M;
};

// A warp takes 2048 k of a row, a lane eight neighbours at a time: four bytes of q,
// and 16 of each result (whose rows have room for whole eights). 4096 x 11008 to two
// bf16 terms: 47 us, 203 MB at 4.3 TB/s (54 % of the integer lanes); fp32 43 us.
constexpr int kExpandK = 2048;
template <class T>
__global__ void __launch_bounds__(256) w4_expand_kernel(const Expand p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int half = (p.K + 1) / 2, pieces = (p.K + kExpandK - 1) / kExpandK;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32; i < p.rows * p.count * pieces;
       i += static_cast<long long>(gridDim.x) * 8) {
    const long long line = i / pieces, z = line / p.rows, n = p.n0 + line - z * p.rows;
    if (p.offsets != nullptr && held(p.offsets[z], p.M) >= held(p.offsets[z + 1], p.M)) continue;
    const long long from = z * p.strideq + n * p.ldq, to = line * p.ldd;
    const long long s_at = z * p.strides + n * p.lds, z_at = z * p.stridez + n * p.ldz;
    const int k0 = static_cast<int>(i - line * pieces) * kExpandK;
#pragma unroll 4
    for (int c = 0; c < kExpandK / 256; ++c) {
      const int k = k0 + c * 256 + lane * 8, b = k / 2;
      if (k >= p.K) break;
      uint32_t q = 0;
      if (p.words && b + 4 <= half && index_ok(kSiteCopySrc, from + b, 4, p.q_extent)) {
        q = __ldcs(reinterpret_cast<const uint32_t *>(p.q + from + b));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (b + j < half && index_ok(kSiteCopySrc, from + b + j, 1, p.q_extent))
            q |= static_cast<uint32_t>(p.q[from + b + j]) << (8 * j);
      }
      const int at = k / p.group;  // of a multiple of 32
      if (!index_ok(kSiteLoadB, s_at + at, 1, p.s_extent)) continue;
      const float s = static_cast<float>(static_cast<const T *>(p.scales)[s_at + at]);
      float zero = 8.0f;
      if (p.zeros != nullptr && index_ok(kSiteLoadB, z_at + at, 1, p.z_extent))
        zero = static_cast<float>(p.zeros[z_at + at] & 15);
      float w[8];
      // 2^23 + q less 2^23 + z; the product is exact but for fp32 scales of more
      // than 20 bits
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = s * (__uint_as_float(0x4b000000u | (q >> (4 * j) & 15u)) - (0x1p23f + zero));
      if (!index_ok(kSiteCopyDst, to + k, 8, p.d_extent)) continue;
      if constexpr (sizeof(T) == 4) {
        float4 *out = reinterpret_cast<float4 *>(static_cast<float *>(p.hi) + to + k);
        out[0] = make_float4(w[0], w[1], w[2], w[3]);
        out[1] = make_float4(w[4], w[5], w[6], w[7]);
      } else {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(w[2 * j], w[2 * j + 1]);
          const float2 f = __bfloat1622float2(h);
          const __nv_bfloat162 l = __floats2bfloat162_rn(isinf(f.x) ? 0.0f : w[2 * j] - f.x,
                                                         isinf(f.y) ? 0.0f : w[2 * j + 1] - f.y);
          hi[j] = *reinterpret_cast<const uint32_t *>(&h);
          lo[j] = *reinterpret_cast<const uint32_t *>(&l);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.hi) + to + k) =
            make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.lo) + to + k) =
            make_uint4(lo[0], lo[1], lo[2], lo[3]);
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

long long up16(long long x) { return (x + 15) / 16 * 16; }

// Whether TMA can read Q as it lies.
bool readable(const W4Args &a) {
  return reinterpret_cast<uintptr_t>(a.Q) % 16 == 0 && a.ldq % 16 == 0 &&
         (a.groups <= 1 || a.strideq % 16 == 0);
}

// Q's rows to rows that it can: dst has pitch ldd and stride strided.
int pack(const W4Args &a, uint8_t *dst, int64_t ldd, int64_t strided, int sm_count,
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

int encode(const W4Args &a, CUtensorMap *map) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return kErrLaunch;
  const bool stack = a.groups > 1 && a.strideq > 0;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>((a.K + 1) / 2), static_cast<cuuint64_t>(a.N),
                              static_cast<cuuint64_t>(stack ? a.groups : 1)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.ldq),
                                 static_cast<cuuint64_t>(stack ? a.strideq : a.ldq)};
  const cuuint32_t box[3] = {kBlockK / 2, kTileN, 1}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(a.Q), dims, strides, box,
            step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? kOk : kErrLaunch;
}

// A's operands, and the products.
template <class T, int COLS, int PERIOD, bool MAKE>
int launch_both(const W4Args &a, P p, const Prep &prep, int sm_count, cudaStream_t stream) {
  using A = Tile<T, COLS, PERIOD>;
  const int groups = static_cast<int>(a.groups);
  const int tiles = (p.N + kTileN - 1) / kTileN;
  constexpr int kStages = stages_of(COLS);
  static_assert(kGroups * A::kRows * kTileN * 4 <= kStages * kWBytes, "sums stand where weights did");
  size_t smem = 1024 + kStages * (kWBytes + A::kStep);
  // Shared memory keeps an SM to the CTAs that its TMEM has room for: two of 256
  // columns or one of 512, and none beside a dense or a segmented product's (512
  // columns). One more would wait in its allocation for another to leave, and, on
  // two streams, clusters could wait for each other.
  const size_t least = tmem_columns(COLS, 4 / PERIOD) == 512 ? 128 * 1024 : 100 * 1024;
  if (smem < least) smem = least;
  Prep q = prep;
  const long long most = static_cast<long long>(p.M) / A::kRows + groups;
  p.by_rows = q.by_rows = p.M < most;
  q.to_extent = MAKE ? 0 : (p.by_rows ? p.M : most) * p.blocks * A::kStep;
  // One workspace: the operands, and behind them Q where it has to be copied.
  W4Args from = a;
  const bool copied = !readable(a);
  if (copied) {
    from.ldq = up16((a.K + 1) / 2);
    from.strideq = a.strideq == 0 ? 0 : a.N * from.ldq;
  }
  const int64_t copy = copied ? (a.strideq == 0 ? 1 : a.groups) * a.N * from.ldq : 0;
  void *to = nullptr;
  int st = kOk;
  if (q.to_extent + copy > 0) st = pool_alloc(&to, static_cast<size_t>(q.to_extent + copy), stream);
  if (st != kOk) return st;
  q.to = static_cast<uint8_t *>(to);
  p.A = q.to;
  p.prep = q;
  CUtensorMap map;
  if (copied) {
    uint8_t *dst = q.to + q.to_extent;
    from.Q = dst;
    st = pack(a, dst, from.ldq, from.strideq, sm_count, stream);
  }
  if (st == kOk) st = encode(from, &map);
  const int64_t average = (p.M + groups - 1) / groups;
  const int64_t units = (average + A::kRows - 1) / A::kRows * A::kRows * p.blocks;
  const int64_t blocks = (units + kPrepWarps - 1) / kPrepWarps;
  if constexpr (!MAKE)
    if (st == kOk)
      st = launch(w4_prep_kernel<T, COLS, PERIOD>,
                  dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096), static_cast<unsigned>(groups), 1),
                  32 * kPrepWarps, 0, 1, stream, q);
  if (st == kOk)
    st = launch(w4_kernel<T, COLS, PERIOD, MAKE>,
                dim3(static_cast<unsigned>(tiles * p.split), static_cast<unsigned>(groups), 1), kThreads,
                smem, p.split, stream, map, p);
  const int fst = to != nullptr ? pool_free(to, stream) : kOk;
  return st != kOk ? st : fst;
}

template <class T, int COLS, bool MAKE = false>
int launch_cols(const W4Args &a, const P &p, const Prep &q, int period, int sms, cudaStream_t stream) {
  if (period == 4) return launch_both<T, COLS, 4, MAKE>(a, p, q, sms, stream);
  if (period == 2) return launch_both<T, COLS, 2, MAKE>(a, p, q, sms, stream);
  // (more columns' accumulators of groups of 32 are more than TMEM holds)
  return launch_both<T, (COLS < 48 ? COLS : (sizeof(T) == 2 ? 32 : 48)), 1, MAKE>(a, p, q, sms, stream);
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

int w4_launch(const W4Args &a, int sm_count, cudaStream_t stream) {
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
  p.z_step = a.groups > 1 && a.strideq > 0 ? 1 : 0;
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.blocks = static_cast<int>((a.K + kBlockK - 1) / kBlockK);
  int period = 4;
  while (a.group % (32 * period) != 0) period /= 2;
  p.per_group = static_cast<int>(a.group / (32 * period));
  p.timeout_ns = 2000000000ull + 2000ull * static_cast<unsigned long long>(a.K);
  const int64_t tiles = (a.N + kTileN - 1) / kTileN;
  const int64_t used = a.groups < a.M ? a.groups : a.M;  // segments with rows, at most
  // CTAs of a tile: as many as an SM has two of at a time (a third would wait for a
  // round of its own: 4096 x 11008, 86 tiles), and two blocks each.
  int64_t split = 2 * static_cast<int64_t>(sm_count) / (tiles * used);
  if (split > p.blocks / 2) split = p.blocks / 2;
  if (split > kMaxSplit) split = kMaxSplit;
  p.split = split < 1 ? 1 : static_cast<int>(split);

  Prep q = {};
  q.A = a.A;
  q.lda = a.lda;
  q.a_extent = matrix_extent(a.M, a.K, a.lda);
  q.a_vec = reinterpret_cast<uintptr_t>(a.A) % 16 == 0 && a.lda * elem % 16 == 0;
  q.offsets = a.offsets;
  q.M = p.M;
  q.K = p.K;
  q.blocks = p.blocks;
  // Rows at a time: twice what a segment has on average, for segments differ;
  // longer ones take several turns. (11008 x 4096 in bf16, 16 | 32 | 64 rows in one
  // turn: 19 | 21 | 33 us; 96 in two of 64: 56.)
  const int64_t rows = a.groups > 1 ? 2 * ((a.M + a.groups - 1) / a.groups) : a.M;
  if (a.bf16) {
    if (a.M <= make_rows(2)) return launch_cols<__nv_bfloat16, 16, true>(a, p, q, period, sm_count, stream);
    if (rows <= 16) return launch_cols<__nv_bfloat16, 16>(a, p, q, period, sm_count, stream);
    if (rows <= 32) return launch_cols<__nv_bfloat16, 32>(a, p, q, period, sm_count, stream);
    return launch_cols<__nv_bfloat16, 64>(a, p, q, period, sm_count, stream);
  }
  if (a.M <= make_rows(4)) return launch_cols<float, 16, true>(a, p, q, period, sm_count, stream);
  if (rows <= 5) return launch_cols<float, 16>(a, p, q, period, sm_count, stream);
  if (rows <= 16) return launch_cols<float, 48>(a, p, q, period, sm_count, stream);
  return launch_cols<float, 96>(a, p, q, period, sm_count, stream);
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
  p.words = reinterpret_cast<uintptr_t>(a.Q) % 4 == 0 && a.ldq % 4 == 0 && a.strideq % 4 == 0;
  p.offsets = a.offsets;
  p.M = a.M;
  const int64_t pieces = (a.K + kExpandK - 1) / kExpandK;
  const int64_t blocks = (rows * a.groups * pieces + 7) / 8, most = 8LL * sm_count;
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most), 1, 1);
  return a.bf16 ? launch(w4_expand_kernel<__nv_bfloat16>, grid, 256, 0, 1, stream, p)
                : launch(w4_expand_kernel<float>, grid, 256, 0, 1, stream, p);
}

}  // namespace gemm
