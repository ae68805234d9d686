// seg_tc.cu -- segmented matrix products on the tensor cores of sm_103a.
//
// A tile of the result is computed transposed, D = L Q^T, on a CTA pair
// (tcgen05 cta_group::2): 256 lanes n (columns of the result, 128 a CTA) by up
// to 256 columns q,
//
//   rows:   D[n, t] = sum_k B_z[k, n] A[t, k]      q = rows t of one segment
//   wgrad:  D[n, i] = sum_t B[t, n] A[t, i]        t = rows of the segment
//
// so a segment with few rows needs few columns (N of the MMA is the tile's own
// row count, rounded up to 32): the weights then stream through at the rate of
// memory whatever the other 240 columns would have cost. Lanes are consecutive
// in the result's rows.
//
// Tiles of all segments form one list, dealt round-robin to persistent pairs;
// every role walks it by itself from a table of the segments' first tiles,
// which each CTA makes from the device's offsets at its start. Operands stand
// in shared memory as lines of 64 contiguous elements (128 bytes, 128-byte
// swizzle), K-major or MN-major as they lie in memory: no transposed copy.
//
// bf16 operands come by TMA, 64 k of 128 + 128 lines a stage, and go to
// kind::f16 MMAs as they are. float32 operands, and bf16 ones that TMA cannot
// read as given, are loaded by eight warps; a float32 value, 32 k a stage, is
// split into three bf16 terms on the way,
//
//   x = h + m + l,   h = bf16(x), m = bf16(x - h), l = bf16(x - h - m),
//
// exact for finite x (24 bits in three terms of 8; Henry, Tang and Heinecke,
// "Leveraging the bfloat16 artificial intelligence datatype for
// higher-precision computations", ARITH 2019). The products hh, hm, mh, mm,
// hl, lh are summed; those left out are below 2^-24 of |x y|.
//
// The tensor core truncates as it adds to an accumulator: sums of K products
// drift by about 2^-24 per MMA (measured: 4.4e-6 of the result's norm after
// 256 bf16 MMAs of one accumulator, against 1.1e-6 of an FP32 FMA chain). For
// float32 each accumulator therefore holds 64 k only, a stage's small products
// first, and the epilogue warps add it to sums in registers, rounded to
// nearest, while the next one fills.
//
// Every barrier wait is bounded; on a timeout the pair lets its copies and
// MMAs finish (bounded), frees TMEM and exits, and the host reads the status.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "ptx.cuh"
#include "segments.h"

namespace gemm {

__device__ int g_seg_status;  // first error recorded by a kernel of this unit

namespace {

constexpr int kLanes = 256;     // result columns per tile (MMA M, of the pair)
constexpr int kCols = 256;      // most rows per tile (MMA N)
constexpr int kHalf = 128;      // lanes, and columns at most, of one CTA of the pair
constexpr int kColStep = 32;    // granularity of the MMA's N
constexpr int kRasterM = 8;     // row tiles per raster group
constexpr uint32_t kTmemCols = 512;

struct SegOperand {
  const void *p[2];  // one or two terms of the operand
  long long ld, zs, extent;
  int vec;           // 8 elements at a multiple of 8 are one aligned load
};

struct SegTc {
  int wgrad, dense;
  int groups, M, N, K, bank;
  int passes;        // terms summed of a two-term operand: 1 or 2
  int tiles_n;
  int q_box;         // TMA: lines per copy of Q (rows kind)
  int l_whole, q_whole;  // TMA: an MN-major operand comes as one 4-D copy
  SegOperand L, Q;   // plain loads
  const int64_t *offsets;
  const int32_t *index;
  const float *scales;
  const float *add;  // dense: fp32 addend of the rows that the segments hold
  long long add_ld, add_extent;
  void *C, *C_lo;    // C_lo: the result's second term
  int c_f32;
  int c_rows;        // rows of the result can leave as 16-byte pieces
  long long c_ld, c_lo_ld, c_stride, c_extent, c_lo_extent;
  unsigned long long timeout_ns;
};

template <class T, bool TMA>
struct Cfg {
  static constexpr bool kSplit = std::is_same<T, float>::value;  // three-term operands
  static constexpr int kTerms = kSplit ? 3 : 1;
  // k per stage: 128-byte lines of bf16, or 64-byte ones of each float32 term
  // (two stages of three terms leave room for the values in flight).
  static constexpr int kBK = kSplit ? 32 : 64;
  // k of one accumulator, float32 (two stages).
  static constexpr int kChunk = kSplit ? 64 : kBK;
  static constexpr int kOpBytes = kHalf * kBK * 2;  // one term of one operand
  static constexpr int kStageBytes = 2 * kTerms * kOpBytes;
  static constexpr int kStages = kSplit ? 2 : 6;
  // Float32 values on their way: lines of 32 (128 bytes, 128-byte swizzle),
  // 128 of either operand a stage.
  static constexpr int kRawOpBytes = kHalf * 128;
  static constexpr int kRawStages = kSplit ? 3 : 1;
  static constexpr int kRawBytes = kSplit ? kRawStages * 2 * kRawOpBytes : 0;
  // Results on their way out, per 128 columns of the tile: two pieces of 16
  // rows of 128 bf16, or one of float32.
  static constexpr int kOutBytes = 8192;
  static constexpr bool kLoaders = kSplit || !TMA;  // warps that fill the stages
  static constexpr int kMmaWarp = 1;
  static constexpr int kFixWarp = 2;
  static constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
  static constexpr int kLoadWarp0 = 12, kLoadWarps = 8;
  static constexpr int kThreads = 32 * (kLoaders ? kLoadWarp0 + kLoadWarps : kLoadWarp0);
  static constexpr int kCopyWarps = 3;  // float32 without TMA: warps 0, 2 and 3
  
};

template <int STAGES, int RAW>
struct Shared {
  uint64_t full[STAGES], empty[STAGES], part[STAGES];
  uint64_t raw_full[RAW], raw_empty[RAW];
  uint64_t acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  int abort;
};

// One tile of the list, as every role sees it.
struct Tile {
  int g, z;       // segment; its matrix (-1: none)
  int n0;         // first lane (result column)
  int q0, qn;     // first column and how many are in the result
  int k0, klen;   // first row of the contraction (wgrad) and its length
  int row0;       // rows kind: row of the result of column 0 is q0 (absolute)
};

struct Table {
  int *first;     // [groups + 1] tiles of the segments before
  int *row;       // [groups + 1] offsets, held to the rows there are
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ bool tile_at(const SegTc &p, const Table &tab, int t, Tile &o) {
  const int groups = p.dense ? 1 : p.groups;
  if (t >= tab.first[groups]) return false;
  int lo = 0, hi = groups;  // the segment whose tiles hold t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.first[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int idx = t - tab.first[lo];
  const int2 rows = make_int2(tab.row[lo], max(tab.row[lo], tab.row[lo + 1]));
  const int height = p.wgrad ? p.K : rows.y - rows.x;
  const int tm = cdiv(height, kCols);
  // Groups of kRasterM row tiles, lane tiles in the outer loop, so that the
  // pairs at work at one time share operand tiles in L2.
  const int group = idx / (kRasterM * p.tiles_n);
  const int m_first = group * kRasterM;
  const int width = min(kRasterM, tm - m_first);
  const int rem = idx - group * kRasterM * p.tiles_n;
  const int mi = m_first + rem % width, ni = rem / width;
  o.g = lo;
  // The segment's rows in tm equal parts (in steps of kColStep), not whole
  // tiles and a rest: the pairs end together, and no tile is all operand
  // traffic and no work.
  const int step = p.wgrad ? 128 : kColStep;
  const int width_q = cdiv(cdiv(height, tm), step) * step;
  o.n0 = ni * kLanes;
  o.qn = min(width_q, height - mi * width_q);
  if (p.wgrad) {
    o.z = 0;
    o.q0 = mi * width_q;
    o.k0 = rows.x;
    o.klen = rows.y - rows.x;
  } else {
    o.z = lo;
    if (p.dense) {
      o.z = 0;
    } else if (p.index != nullptr) {
      o.z = p.index[lo];
      if (o.z < 0 || o.z >= p.bank) o.z = -1;
    } else if (o.z >= p.bank) {
      o.z = -1;
    }
    o.q0 = rows.x + mi * width_q;
    o.k0 = 0;
    o.klen = o.z < 0 ? 0 : p.K;
  }
  return true;
}

// MMA columns of a tile: its own, in steps the operand's layout allows (an
// MN-major Q comes in lines of 64, one per CTA at least).
template <bool QMN>
__device__ __forceinline__ int mma_cols(const Tile &t) {
  constexpr int step = QMN ? 128 : kColStep;
  return cdiv(t.qn, step) * step;
}

// One try that suspends the thread for up to 20 us: a role that polls in a
// tight loop (eight epilogue warps do most of the time) takes shared-memory
// cycles from the copies and the MMAs.
template <bool CLUSTER>
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t done;
  if (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
  return done != 0;
}

// Wait for the phase; gives up (false) after the launch's limit, recording a
// timeout, or when another role of the CTA has given up.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const SegTc &p,
                                     volatile int *abort) {
  const uint32_t a = smem_addr(bar);
  if (try_wait_long<CLUSTER>(a, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  while (!try_wait_long<CLUSTER>(a, parity)) {
    if (*abort) return false;
    if (global_timer_ns() - t0 > p.timeout_ns) {
      *abort = 1;
      atomicCAS(&g_seg_status, 0, kStatusTimeout);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const SegTc &p,
                                          volatile int *abort) {
  const bool ok = wait(bar, parity, p, abort);
  return __all_sync(0xffffffffu, ok);
}

// Spin (bounded, ignoring the abort flag) until the phase completes.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity, uint64_t timeout_ns) {
  const uint32_t a = smem_addr(bar);
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (global_timer_ns() - t0 > timeout_ns) break;
  }
}

template <int STAGES>
struct Ring {
  uint32_t idx = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++idx == STAGES) {
      idx = 0;
      phase ^= 1;
    }
  }
};

// ------------------------------------------------------------ instructions --

// D[tmem] (+)= A[smem] B[smem]^T, kind::f16 with bf16 operands, on the pair.
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f16: D fp32 (bits 4-5 = 1), A and B bf16
// (bits 7-9 and 10-12 = 1), MN-major operands (bits 15 and 16), N >> 3 in bits
// 17-22, M >> 4 in bits 24-28.
__device__ __forceinline__ uint32_t idesc_bf16(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         ((n >> 3) << 17) | ((m >> 4) << 24);
}

// Descriptor of an operand's first 16 k. K-major: lines are rows of BK k, 8-line
// atoms one after another, 16 k are 32 bytes along the line. MN-major: lines are
// k, BK lines to a chunk of 64 elements, 16 k are 16 lines.
template <bool MN, int BK>
__device__ __forceinline__ uint64_t line_desc(uint32_t base) {
  if (MN) return smem_desc(base, BK * 128, 1024, 2);
  return smem_desc(base, 16, BK * 16, BK == 64 ? 2 : 4);
}

// Arrive on the barrier at the shared::cluster address (the even CTA's). What
// it announces never crosses the pair: lines that the odd CTA's threads wrote to
// its own shared memory, fenced for its own tensor core, or its own TMEM read
// out. A release at CTA scope is therefore enough; one at cluster scope cost
// 280 ns of every float32 stage (4096 x 4864 x 4096: 672 against 530 us).
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Store the box at (x, y, z) of the map from shared memory, asynchronously.
__device__ __forceinline__ void store_box(const CUtensorMap *map, uint32_t src, int x, int y,
                                          int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Copy `bytes` (a multiple of 16) from shared to global memory, asynchronously.
__device__ __forceinline__ void store_bulk(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
}

// ------------------------------------------------------------- plain loads --

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Bf16 elements [x, x + 8) of the line at `row` (element offset), those at or
// past `limit` zero.
__device__ __forceinline__ uint4 load_eight(const SegOperand &o, const __nv_bfloat16 *p, int site,
                                            long long row, int x, int limit) {
  const long long off = row + x;
  if (o.vec && x + 8 <= limit && index_ok(site, off, 8, o.extent))
    return __ldg(reinterpret_cast<const uint4 *>(p + off));
  const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    e[i] = x + i < limit && index_ok(site, off + i, 1, o.extent) ? __ldg(h + off + i) : 0;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

// Copy a float from global to shared memory, asynchronously; `bytes` 0: zero.
__device__ __forceinline__ void copy_float(uint32_t dst, const float *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// Eight float32 values as three bf16 terms (`term` bytes apart).
__device__ __forceinline__ void store_terms(uint8_t *dst, int term, float (&v)[8]) {
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      if (t < 2) {  // what the term leaves, exactly
        v[2 * i] -= __uint_as_float(w[i] << 16);
        v[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
      }
    }
    *reinterpret_cast<uint4 *>(dst + t * term) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Registers of a role's warps, float32: the epilogue warps hold 128 sums each.
// 128 x 40 + 256 x 152 + 256 x 64 registers, within the launch's 640 x 96
// (checked by the host). Stated where each role begins: the compiler then
// allots by role.
template <bool SPLIT, int R>
__device__ __forceinline__ void set_registers() {
  if constexpr (SPLIT && R > 96)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
  else if constexpr (SPLIT)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// ------------------------------------------------------------------ kernel --

// LMN, QMN: the operand lies with its lane (column) index contiguous.
template <class T, bool TMA, bool LMN, bool QMN>
__global__ void __launch_bounds__(Cfg<T, TMA>::kThreads, 1)
    seg_tc_kernel(const __grid_constant__ CUtensorMap map_l0,
                  const __grid_constant__ CUtensorMap map_l1,
                  const __grid_constant__ CUtensorMap map_q0,
                  const __grid_constant__ CUtensorMap map_q1,
                  const __grid_constant__ CUtensorMap map_c, const SegTc p) {
  using C = Cfg<T, TMA>;
  constexpr int STAGES = C::kStages, kBK = C::kBK, kOpBytes = C::kOpBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *stages = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *raw = stages + STAGES * C::kStageBytes;
  using Sh = Shared<STAGES, C::kRawStages>;
  uint8_t *out = raw + C::kRawBytes;
  Sh *sh = reinterpret_cast<Sh *>(out + 2 * C::kOutBytes);
  Table tab;
  const int groups = p.dense ? 1 : p.groups;
  tab.row = reinterpret_cast<int *>(sh + 1);
  tab.first = tab.row + groups + 1;
  volatile int *abort = &sh->abort;

  const uint32_t warp = warp_index();
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  // Arrivals that fill a stage. Copies straight to it: the even CTA's (both
  // CTAs' bytes), or for weight gradients one arrival from each CTA's copies or
  // masks. Else one from each CTA's load warps.
  constexpr int kFullCount = C::kLoaders || QMN ? 2 : 1;
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh->full[s], kFullCount);
      mbar_init(&sh->empty[s], 1);
      mbar_init(&sh->part[s], 1);  // this CTA's bytes of a stage that is masked before use
    }
    for (int s = 0; s < C::kRawStages; ++s) {
      mbar_init(&sh->raw_full[s], TMA ? 1 : 32 * C::kCopyWarps);
      mbar_init(&sh->raw_empty[s], C::kLoadWarps);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sh->acc_full[a], 1);
      mbar_init(&sh->acc_empty[a], 2);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_barrier_init();
  }
  if (TMA && warp == 0 && lane == 0) {
    tma_prefetch_map(&map_l0);
    tma_prefetch_map(&map_q0);
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc<2>(&sh->tmem_base, kTmemCols);
    tmem_relinquish<2>();
  }
  grid_dependency_wait();
  // The table of segments: their rows, and the tiles before each.
  for (int g = threadIdx.x; g <= groups; g += C::kThreads) {
    const long long a = p.dense ? (g ? p.M : 0) : p.offsets[g];
    tab.row[g] = static_cast<int>(a < 0 ? 0 : (a > p.M ? p.M : a));
  }
  __syncthreads();
  for (int g = threadIdx.x; g < groups; g += C::kThreads)
    tab.first[g] =
        cdiv(p.wgrad ? p.K : max(tab.row[g + 1] - tab.row[g], 0), kCols) * p.tiles_n;
  __syncthreads();
  if (warp == 0) {
    int sum = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int g = g0 + static_cast<int>(lane);
      const int own = g < groups ? tab.first[g] : 0;
      int v = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, d);
        if (static_cast<int>(lane) >= d) v += w;
      }
      if (g < groups) tab.first[g] = sum + v - own;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) tab.first[groups] = sum;
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // barriers and TMEM of both CTAs are set up
  tc_fence_after_sync();
  const uint32_t tmem = sh->tmem_base;
  grid_launch_dependents();

  const bool epilogue = warp >= C::kEpiWarp0 && warp < C::kEpiWarp0 + C::kEpiWarps;
  const bool loader = C::kLoaders && warp >= C::kLoadWarp0;

  Tile t;
  if (TMA && !C::kSplit && warp == 0) {
    // ------------------------------------------------------------- copies --
    if (lane == 0) {
      Ring<STAGES> r;
      uint32_t part_phase = 0, parts = 0;  // stages that went to part[], by phase and at all
      int issued = 0;
      bool ok = true;
      const uint32_t full0 = mbar_cluster_addr(&sh->full[0], 0);
      for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
        const int half = mma_cols<QMN>(t) / 2;
        const int ln = t.n0 + static_cast<int>(rank) * kHalf;
        const int qn = t.q0 + static_cast<int>(rank) * half;
        const int copies = QMN ? half / 64 : cdiv(half, p.q_box);
        const uint32_t bytes =
            kOpBytes + static_cast<uint32_t>(copies) * (QMN ? 8192u : 128u * p.q_box);
        for (int pass = 0; ok && pass < p.passes; ++pass) {
          const CUtensorMap *ml = pass ? &map_l1 : &map_l0, *mq = pass ? &map_q1 : &map_q0;
          for (int kk = 0; kk < t.klen; kk += kBK) {
            if (!wait(&sh->empty[r.idx], r.phase ^ 1, p, abort)) {
              ok = false;
              break;
            }
            uint8_t *st = stages + r.idx * C::kStageBytes;
            uint32_t bar = full0 + r.idx * 8;
            parts &= ~(1u << r.idx);
            if (QMN && t.klen - kk < kBK && (t.klen - kk) % 16 != 0) {
              // This CTA's own barrier; the mask warp passes it on.
              bar = smem_addr(&sh->part[r.idx]);
              mbar_arrive_expect_tx(&sh->part[r.idx], bytes);
              parts |= 1u << r.idx;
              part_phase ^= 1u << r.idx;
            } else if (rank == 0) {
              mbar_arrive_expect_tx(&sh->full[r.idx], 2 * bytes);
              if (QMN) mbar_arrive(&sh->full[r.idx]);
            }
            if (!LMN) {
              tma_load_3d_pair(st, ml, bar, kk, ln, t.z);
            } else if (p.l_whole) {
              tma_load_4d_pair(st, ml, bar, 0, t.k0 + kk, ln / 64, t.z);
            } else {
              tma_load_3d_pair(st, ml, bar, ln, t.k0 + kk, t.z);
              tma_load_3d_pair(st + 8192, ml, bar, ln + 64, t.k0 + kk, t.z);
            }
            if (QMN && p.q_whole) {
              tma_load_4d_pair(st + kOpBytes, mq, bar, 0, t.k0 + kk, qn / 64, 0);
            } else {
              for (int c = 0; c < copies; ++c) {
                if (QMN)
                  tma_load_3d_pair(st + kOpBytes + c * 8192, mq, bar, qn + c * 64, t.k0 + kk, 0);
                else
                  tma_load_3d_pair(st + kOpBytes + c * p.q_box * 128, mq, bar, kk,
                                   qn + c * p.q_box, 0);
              }
            }
            ++issued;
            r.next();
          }
        }
      }
      // On a timeout let the copies that were started land: those of the last
      // stages issued, one phase back where the ring has wrapped since.
      if (!ok)
        for (int s = 0; s < STAGES && s < issued; ++s) {
          r.phase ^= r.idx == 0 ? 1u : 0u;
          r.idx = r.idx == 0 ? STAGES - 1 : r.idx - 1;
          if (parts >> r.idx & 1u)
            drain_wait(&sh->part[r.idx], (part_phase >> r.idx & 1u) ^ 1u, p.timeout_ns);
          else if (rank == 0)
            drain_wait(&sh->full[r.idx], r.phase, p.timeout_ns);
        }
    }
    __syncwarp();
  } else if (TMA && !C::kSplit && QMN && warp == C::kFixWarp) {
    // -------------------------------------------------------------- masks --
    // The last stage of a segment whose rows end inside a step of 16: zero
    // both operands' lines from its end to the step's, which hold the next
    // segment's rows (whatever they are: NaN times zero is NaN).
    Ring<STAGES> r;
    uint32_t part_phase = 0;
    bool ok = true;
    for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
      const int half = mma_cols<QMN>(t) / 2;
      const int blocks = cdiv(t.klen, kBK);
      for (int kb = 0; kb < blocks * p.passes; ++kb) {
        const int kk = (kb >= blocks ? kb - blocks : kb) * kBK;
        const int tail = t.klen - kk;
        if (tail < kBK && tail % 16 != 0) {
          if (!warp_wait(&sh->part[r.idx], part_phase >> r.idx & 1u, p, abort)) {
            ok = false;
            break;
          }
          part_phase ^= 1u << r.idx;
          uint8_t *st = stages + r.idx * C::kStageBytes;
          const int end = (tail + 15) / 16 * 16;
          const int chunks = 2 + half / 64;  // of L, then of Q
          for (int e = static_cast<int>(lane); e < chunks * (end - tail) * 8; e += 32) {
            const int c = e / ((end - tail) * 8), w = e % ((end - tail) * 8);
            *reinterpret_cast<uint4 *>(st + c * 8192 + (tail + w / 8) * 128 + w % 8 * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(mbar_cluster_addr(&sh->full[r.idx], 0));
        }
        r.next();
      }
    }
  } else if (C::kSplit && TMA && warp == 0) {
    // ------------------------------------------------ float32 by TMA --
    set_registers<C::kSplit, 40>();
    if (lane == 0) {
      Ring<C::kRawStages> r;
      int issued = 0;
      bool ok = true;
      for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
        const int half = mma_cols<QMN>(t) / 2;
        const int ln = t.n0 + static_cast<int>(rank) * kHalf;
        const int qn = t.q0 + static_cast<int>(rank) * half;
        const int copies = QMN ? half / 32 : cdiv(half, p.q_box);
        const uint32_t bytes = C::kRawOpBytes +
                               static_cast<uint32_t>(copies) * (QMN ? 4096u : 128u * p.q_box);
        for (int kk = 0; kk < t.klen; kk += kBK) {
          if (!wait(&sh->raw_empty[r.idx], r.phase ^ 1, p, abort)) {
            ok = false;
            break;
          }
          uint8_t *l = raw + r.idx * 2 * C::kRawOpBytes, *q = l + C::kRawOpBytes;
          const uint32_t bar = smem_addr(&sh->raw_full[r.idx]);
          mbar_arrive_expect_tx(&sh->raw_full[r.idx], bytes);
          if (!LMN) {
            tma_load_3d_pair(l, &map_l0, bar, kk, ln, t.z);
          } else if (p.l_whole) {
            tma_load_4d_pair(l, &map_l0, bar, 0, t.k0 + kk, ln / 32, t.z);
          } else {
            for (int c = 0; c < 4; ++c)
              tma_load_3d_pair(l + c * 4096, &map_l0, bar, ln + c * 32, t.k0 + kk, t.z);
          }
          if (QMN && p.q_whole) {
            tma_load_4d_pair(q, &map_q0, bar, 0, t.k0 + kk, qn / 32, 0);
          } else {
            for (int c = 0; c < copies; ++c) {
              if (QMN)
                tma_load_3d_pair(q + c * 4096, &map_q0, bar, qn + c * 32, t.k0 + kk, 0);
              else
                tma_load_3d_pair(q + c * p.q_box * 128, &map_q0, bar, kk, qn + c * p.q_box, 0);
            }
          }
          ++issued;
          r.next();
        }
      }
      if (!ok)  // let the copies that were started land
        for (int s = 0; s < C::kRawStages && s < issued; ++s) {
          r.phase ^= r.idx == 0 ? 1u : 0u;
          r.idx = r.idx == 0 ? C::kRawStages - 1 : r.idx - 1;
          drain_wait(&sh->raw_full[r.idx], r.phase, p.timeout_ns);
        }
    }
    __syncwarp();
  } else if (C::kSplit && !TMA && warp < C::kEpiWarp0 && warp != C::kMmaWarp) {
    // ------------------------------- float32 of any pitch and alignment --
    set_registers<C::kSplit, 40>();
    // A line of 32 values a warp and copy, eight lines at a time; the warps
    // take the groups of eight in turn.
    const int cw = warp == 0 ? 0 : static_cast<int>(warp) - 1;
    const int ln31 = static_cast<int>(lane);
    Ring<C::kRawStages> r;
    bool ok = true;
    for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
      const int half = mma_cols<QMN>(t) / 2;
      const int ln = t.n0 + static_cast<int>(rank) * kHalf;
      const int qn = static_cast<int>(rank) * half;
      for (int kk = 0; kk < t.klen; kk += kBK) {
        if (!warp_wait(&sh->raw_empty[r.idx], r.phase ^ 1, p, abort)) {
          ok = false;
          break;
        }
        const uint32_t base = smem_addr(raw) + r.idx * 2 * C::kRawOpBytes;
        for (int g = cw; g < 32; g += C::kCopyWarps) {  // sixteen groups of L, then of Q
          const bool is_l = g < 16, mn = is_l ? LMN : QMN;
          const SegOperand &o = is_l ? p.L : p.Q;
          const int line0 = (g & 15) * 8;  // K-major: the row; MN-major: chunk * 32 + k
          long long off;
          int first, last, x, end;  // lines [first, last) and values x < end exist
          if (mn) {
            const int k = kk + (line0 & 31), lane0 = (is_l ? ln : t.q0 + qn) + (line0 >> 5) * 32;
            off = static_cast<long long>(t.k0 + k) * o.ld + lane0;
            first = k;
            last = is_l || (line0 >> 5) * 32 < half ? t.klen : 0;
            x = lane0;
            end = is_l ? p.N : p.K;
          } else {
            const int m = (is_l ? ln : qn) + line0;
            off = static_cast<long long>(is_l ? m : t.q0 + m) * o.ld + kk;
            first = m;
            last = is_l ? p.N : (line0 < half ? t.qn : 0);
            x = kk;
            end = p.K;
          }
          if (!is_l && first >= last) continue;  // no columns here: never read
          if (is_l) off += t.z * o.zs;
          const float *src = static_cast<const float *>(o.p[0]);
          const uint32_t dst = base + (g * 8) * 128 + (ln31 & 3) * 4;
          const bool in = x + ln31 < end;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const long long at = off + e * o.ld + ln31;
            const bool take = in && first + e < last &&
                              index_ok(is_l ? kSiteLoadB : kSiteLoadA, at, 1, o.extent);
            copy_float(dst + e * 128 + ((ln31 >> 2) ^ e) * 16, take ? src + at : src, take ? 4 : 0);
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_addr(&sh->raw_full[r.idx]))
                     : "memory");
        r.next();
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == C::kMmaWarp) {
    set_registers<C::kSplit, 40>();
    if (rank == 0 && lane == 0) {
      // --------------------------------------------------- MMA (even CTA) --
      Ring<STAGES> r;
      Ring<2> acc;
      bool ok = true;
      // Descriptors of the first stage; others are a number of 16-byte units on.
      const uint32_t base = smem_addr(stages);
      const uint64_t l0 = line_desc<LMN, C::kBK>(base);
      const uint64_t q0 = line_desc<QMN, C::kBK>(base + C::kTerms * C::kOpBytes);
      constexpr uint32_t kTerm = C::kOpBytes >> 4, kl = LMN ? 128 : 2, kq = QMN ? 128 : 2;
      for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
        const uint32_t idesc = idesc_bf16(kLanes, static_cast<uint32_t>(mma_cols<QMN>(t)), LMN, QMN);
        uint32_t more = 0;  // 0: the next MMA starts its accumulator
        for (int pass = 0; ok && pass < p.passes; ++pass)
          for (int kk0 = 0; kk0 < t.klen; kk0 += kBK) {
            if (more == 0) {
              // Both CTAs' epilogues have drained the accumulator.
              if (!wait<true>(&sh->acc_empty[acc.idx], acc.phase ^ 1, p, abort)) {
                ok = false;
                break;
              }
            }
            // Copies alone complete a stage of the rows form; other stages
            // have arrivals of the odd CTA's warps (acquire at cluster scope).
            if (!wait<C::kLoaders || QMN>(&sh->full[r.idx], r.phase, p, abort)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const int left = t.klen - kk0;
            const uint64_t l = l0 + r.idx * (C::kStageBytes >> 4);
            const uint64_t q = q0 + r.idx * (C::kStageBytes >> 4);
            const uint32_t d = tmem + acc.idx * kCols;
            auto products = [&](auto steps) {
              if constexpr (C::kSplit) {
                // Small products first: mm, hl, lh, hm, mh, then hh.
                constexpr uint32_t tl[6] = {1, 0, 2, 0, 1, 0}, tq[6] = {1, 2, 0, 1, 0, 0};
#pragma unroll
                for (int c = 0; c < 6; ++c)
#pragma unroll
                  for (int kk = 0; kk < steps(); ++kk) {
                    mma_bf16_pair(d, l + tl[c] * kTerm + kk * kl, q + tq[c] * kTerm + kk * kq,
                                  idesc, c + kk > 0 ? 1u : more);
                  }
              } else {
#pragma unroll
                for (int kk = 0; kk < steps(); ++kk)
                  mma_bf16_pair(d, l + kk * kl, q + kk * kq, idesc, kk > 0 ? 1u : more);
              }
            };
            if (left > kBK - 16)
              products([] { return kBK / 16; });
            else
              products([left] { return (left + 15) / 16; });
            mma_commit_multicast<2>(&sh->empty[r.idx], 3);
            more = 1;
            if ((C::kSplit && (kk0 + kBK) % C::kChunk == 0) ||
                (kk0 + kBK >= t.klen && pass + 1 == p.passes)) {
              mma_commit_multicast<2>(&sh->acc_full[acc.idx], 3);
              acc.next();
              more = 0;
            }
            r.next();
          }
      }
      // Every MMA issued completes before TMEM is released.
      mma_commit_multicast<2>(&sh->drain, 1);
      drain_wait(&sh->drain, 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (epilogue) {
    // ----------------------------------------------------------- epilogue --
    set_registers<C::kSplit, 152>();
    const uint32_t quad = warp & 3, part = (warp - C::kEpiWarp0) >> 2;
    const uint32_t tlane = tmem + ((quad * 32) << 16) + part * 128;
    const int c0 = static_cast<int>(part) * 128;  // this warp's first column
    Ring<2> acc;
    int add0 = 0, add1 = 0;  // rows with an addend
    if (p.add != nullptr) {
      const long long a = p.offsets[0], b = p.offsets[p.groups];
      add0 = static_cast<int>(a < 0 ? 0 : (a > p.M ? p.M : a));
      add1 = static_cast<int>(b < 0 ? 0 : (b > p.M ? p.M : b));
    }
    // The accumulator can be refilled: one arrival for all the CTA's epilogue
    // warps (a release at cluster scope from each costs more than the barrier
    // that gathers them). False if one of them gave up on its wait; every warp
    // comes here once for each accumulator.
    auto drained = [&](uint32_t a, bool ok) {
      tc_fence_before_sync();
      ok = named_barrier_and(1, 32 * C::kEpiWarps, ok);
      if (ok && threadIdx.x == 32 * C::kEpiWarp0)
        mbar_arrive_at(mbar_cluster_addr(&sh->acc_empty[a], 0));
      return ok;
    };
    for (int i = pair; tile_at(p, tab, i, t); i += pairs) {
      const int blocks = cdiv(t.klen, C::kChunk) * p.passes;
      const int n = t.n0 + static_cast<int>(rank * 128 + quad * 32 + lane);
      bool ok = true;
      if constexpr (C::kSplit) {
        // Sum the accumulators of 64 k each in registers; the sums go back to
        // TMEM in the place of the last one, so that float32 and bf16 results
        // leave through the same short loop.
        float sum[128];
#pragma unroll
        for (int c = 0; c < 128; ++c) sum[c] = 0.0f;
        for (int kb = 0; kb < blocks; ++kb) {
          ok = warp_wait(&sh->acc_full[acc.idx], acc.phase, p, abort);
          tc_fence_after_sync();
#pragma unroll
          for (int c = 0; c < 128; c += 16)
            if (ok && c0 + c < t.qn) {
              uint32_t v[16];
              tmem_load_16cols(tlane + acc.idx * kCols + c, v);
              tmem_load_wait();
              tmem_regs_ready(v);
#pragma unroll
              for (int k = 0; k < 16; ++k) sum[c + k] += __uint_as_float(v[k]);
            }
          if (kb + 1 == blocks) break;
          ok = drained(acc.idx, ok);
          if (!ok) break;
          acc.next();
        }
        if (blocks > 1 && ok) {
#pragma unroll
          for (int c = 0; c < 128; c += 16)
            if (c0 + c < t.qn) {
              uint32_t v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(sum[c + k]);
              tmem_store_16cols(tlane + acc.idx * kCols + c, v);
            }
          tmem_store_wait();
        }
      } else if (blocks > 0) {
        ok = warp_wait(&sh->acc_full[acc.idx], acc.phase, p, abort);
        tc_fence_after_sync();
      }
      // All warps go on together from here, or none does.
      if (!named_barrier_and(1, 32 * C::kEpiWarps, ok)) break;
      const float scale =
          !p.wgrad && !p.dense && p.scales != nullptr && t.z >= 0 ? p.scales[t.z] : 1.0f;
      const long long row0 = t.q0 + c0;
      const long long at = (p.wgrad ? t.g * p.c_stride : 0) + row0 * p.c_ld + n;
      const int count = n < p.N ? t.qn - c0 : 0;  // this lane's columns
#pragma unroll 1
      for (int c = 0; c < 128 && c0 + c < t.qn; c += 16) {
        float f[16];
        if (blocks > 0) {
          uint32_t v[16];
          tmem_load_16cols(tlane + acc.idx * kCols + c, v);
          tmem_load_wait();
          tmem_regs_ready(v);
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] = scale * __uint_as_float(v[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] = 0.0f;
        }
        if (p.add != nullptr) {  // sixteen loads in flight
          const long long from = row0 * p.add_ld + n;
          float a[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int row = t.q0 + c0 + c + k;
            const long long off = from + (c + k) * p.add_ld;
            a[k] = c + k < count && row >= add0 && row < add1 &&
                           index_ok(kSitePartialRead, off, 1, p.add_extent)
                       ? __ldg(p.add + off)
                       : 0.0f;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] += a[k];
        }
        if (p.c_rows) {
          // Sixteen rows of this CTA's 128 lanes meet in shared memory and
          // leave as whole pieces of their rows.
          const int elem = p.c_f32 ? 4 : 2, row_bytes = kHalf * elem;
          const uint32_t to = smem_addr(out) + part * C::kOutBytes +
                              (p.c_f32 ? 0 : (c >> 4 & 1) * (C::kOutBytes / 2));
          const uint32_t at_lane = to + (quad * 32 + lane) * elem;
          if (quad == 0) {  // the copies that last read this piece are done with it
            if (p.c_f32)
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            else
              asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          }
          named_barrier_sync(3 + part, 128);
          if (p.c_f32) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(at_lane + k * row_bytes), "f"(f[k])
                           : "memory");
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(at_lane + k * row_bytes),
                           "h"(__bfloat16_as_ushort(__float2bfloat16_rn(f[k])))
                           : "memory");
          }
          fence_proxy_async_smem();
          named_barrier_sync(3 + part, 128);
          if (quad == 0) {
            const int n_cta = t.n0 + static_cast<int>(rank) * kHalf;
            const int width = min(kHalf, p.N - n_cta);
            if (c0 + c + 16 <= t.qn) {
              // One box of sixteen rows (as a copy for each row, 256 bytes at
              // a time, results left at 2 TB/s).
              if (lane == 0 && width > 0)
                store_box(&map_c, to, n_cta, t.q0 + c0 + c, p.wgrad ? t.g : 0);
            } else {  // the segment ends here
              const int row = c + static_cast<int>(lane);
              const long long off = at - n + n_cta + row * p.c_ld;
              if (lane < 16 && c0 + row < t.qn && width > 0 &&
                  index_ok(kSiteCStore, off, width, p.c_extent))
                store_bulk(static_cast<uint8_t *>(p.C) + off * elem, to + lane * row_bytes,
                           static_cast<uint32_t>(width * elem));
            }
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else if (p.c_f32) {
          float *dst = static_cast<float *>(p.C);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const long long off = at + (c + k) * p.c_ld;
            if (c + k < count && index_ok(kSiteCStore, off, 1, p.c_extent)) dst[off] = f[k];
          }
        } else {
          __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.C);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const long long off = at + (c + k) * p.c_ld;
            if (c + k < count && index_ok(kSiteCStore, off, 1, p.c_extent))
              dst[off] = __float2bfloat16_rn(f[k]);
          }
          if (p.C_lo != nullptr) {
            __nv_bfloat16 *lo = static_cast<__nv_bfloat16 *>(p.C_lo);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const long long off = (row0 + c + k) * p.c_lo_ld + n;
              if (c + k < count && index_ok(kSitePartialWrite, off, 1, p.c_lo_extent))
                lo[off] = __float2bfloat16_rn(
                    f[k] - static_cast<float>(__float2bfloat16_rn(f[k])));
            }
          }
        }
      }
      if (blocks > 0) {
        drained(acc.idx, true);
        acc.next();
      }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (loader) {
    // -------------------------------------------------------- plain loads --
    set_registers<C::kSplit, 64>();
    // Both operands are masked here, by row and by column.
    const int lw = static_cast<int>(warp) - C::kLoadWarp0;
    Ring<STAGES> r;
    bool ok = true;
    // The CTA's part of a stage is written: one release at cluster scope for
    // all its load warps (a thread of the odd CTA that waited for their
    // arrivals and passed them on was 375 ns of every stage's way).
    const uint32_t full0 = mbar_cluster_addr(&sh->full[0], 0);
    // False if a warp gave up on a wait; each comes here once a stage.
    auto filled = [&](uint32_t s, bool ok) {
      fence_proxy_async_smem();
      ok = named_barrier_and(2, 32 * C::kLoadWarps, ok);
      if (ok && threadIdx.x == 32 * C::kLoadWarp0) mbar_arrive_at(full0 + s * 8);
      return ok;
    };
    if constexpr (C::kSplit) {
      // Split the values that have arrived: eight a lane, four lanes to a line
      // of 32. Lanes 4 to 7 of each eight take the line 5 away (k ^ 5), whose
      // swizzled pieces lie in the other banks, as read and as written.
      const int g = static_cast<int>(lane) >> 2, j = static_cast<int>(lane) & 3;
      const int k8 = (g >> 1) ^ ((g & 1) * 5);  // line within eight
      Ring<C::kRawStages> a;
      for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
        const int half = mma_cols<QMN>(t) / 2;
        for (int kk = 0; kk < t.klen; kk += kBK) {
          ok = warp_wait(&sh->raw_full[a.idx], a.phase, p, abort) &&
               warp_wait(&sh->empty[r.idx], r.phase ^ 1, p, abort);
          const uint8_t *from = raw + a.idx * 2 * C::kRawOpBytes;
          uint8_t *to = stages + r.idx * C::kStageBytes;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const bool mn = u < 2 ? LMN : QMN;
            const int line = ((u & 1) * 8 + lw) * 8 + k8;  // MN-major: chunk * 32 + k
            // K-major Q: rows; MN-major: chunks of 32 columns.
            if (!ok || (u >= 2 && (QMN ? line : line & ~7) >= half)) continue;
            const uint8_t *src = from + (u < 2 ? 0 : C::kRawOpBytes) + line * 128;
            float v[8];
            *reinterpret_cast<float4 *>(v) =
                *reinterpret_cast<const float4 *>(src + ((2 * j) ^ k8) * 16);
            *reinterpret_cast<float4 *>(v + 4) =
                *reinterpret_cast<const float4 *>(src + ((2 * j + 1) ^ k8) * 16);
            if (QMN && kk + (line & 31) >= t.klen) {  // the next segment's row
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            }
            uint8_t *dst = to + (u < 2 ? 0 : C::kTerms * kOpBytes);
            if (mn)  // line k of a chunk of 64, in its first or second half
              dst += (line >> 6) * (kBK * 128) + (line & 31) * 128 +
                     ((((line >> 5 & 1) * 4 + j) ^ k8) * 16);
            else
              dst += line * 64 + ((j ^ (k8 >> 1 & 3)) * 16);
            store_terms(dst, kOpBytes, v);
          }
          ok = filled(r.idx, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive(&sh->raw_empty[a.idx]);
          a.next();
          r.next();
        }
      }
    } else if constexpr (!TMA) {
      // Eight lanes to a line of 64 elements, four lines a warp and load.
      const int sub = static_cast<int>(lane) >> 3, j = static_cast<int>(lane) & 7;
      for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
        const int half = mma_cols<QMN>(t) / 2;
        const int ln = t.n0 + static_cast<int>(rank) * kHalf;
        const int qn = static_cast<int>(rank) * half;  // within the tile
        const int blocks = cdiv(t.klen, kBK);
        for (int kb = 0; kb < blocks * p.passes; ++kb) {
          const int second = kb >= blocks, kk = (second ? kb - blocks : kb) * kBK;
          uint8_t *st = stages + r.idx * C::kStageBytes;
#pragma unroll
          for (int op = 0; op < 2; ++op) {
            const SegOperand &o = op == 0 ? p.L : p.Q;
            const bool mn = op == 0 ? LMN : QMN;
            const T *src = static_cast<const T *>(second ? o.p[1] : o.p[0]);
            const int site = op == 0 ? kSiteLoadB : kSiteLoadA;
            const long long z = op == 0 ? t.z * o.zs : 0;
            uint4 e[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const int line = s * 32 + lw * 4 + sub;
              long long row;
              int x, limit;
              if (mn) {  // line: k; elements: lanes or columns
                const int k = kk + (line & 63);
                x = (op == 0 ? ln : t.q0 + qn) + (line >> 6) * 64 + j * 8;
                limit = k < t.klen ? (op == 0 ? p.N : p.K) : 0;
                if (op == 1 && (line >> 6) * 64 >= half) limit = 0;
                row = z + static_cast<long long>(t.k0 + k) * o.ld;
              } else {
                const int m = op == 0 ? ln + line : qn + line;
                x = kk + j * 8;
                limit = (op == 0 ? m < p.N : line < half && m < t.qn) ? p.K : 0;
                row = z + static_cast<long long>(op == 0 ? m : t.q0 + m) * o.ld;
              }
              e[s] = load_eight(o, src, site, row, x, limit);
            }
            if (op == 0) ok = warp_wait(&sh->empty[r.idx], r.phase ^ 1, p, abort);
#pragma unroll
            for (int s = 0; ok && s < 4; ++s) {
              const int line = s * 32 + lw * 4 + sub;
              if (op == 1 && !mn && line >= half) continue;  // no MMA column
              *reinterpret_cast<uint4 *>(st + op * kOpBytes + line * 128 + (j ^ (line & 7)) * 16) =
                  e[s];
            }
          }
          ok = filled(r.idx, ok);
          if (!ok) break;
          r.next();
        }
      }
    }
  } else {
    set_registers<C::kSplit, 40>();
  }

  // Neither CTA frees its TMEM or leaves while the pair's MMAs, copies or
  // arrivals may still reach it.
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == C::kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc<2>(tmem, kTmemCols);
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

// Map over a stack of row-major matrices, zero outside each: lines of 128 bytes
// (64 bf16 or 32 float32 columns), `lines` rows a copy; chunks > 1: the same
// seen as chunks of one line's columns (a multiple of them, so that no chunk
// leaves its row), that many a copy.
bool encode_lines(const SegMatrix &m, const void *ptr, bool bf16, int lines, int chunks,
                  CUtensorMap *out) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t elem = bf16 ? 2 : 4;
  const cuuint32_t line = bf16 ? 64 : 32;
  const bool stack = m.count > 1 && m.stride > 0;
  const cuuint64_t pitch = static_cast<cuuint64_t>(m.ld) * elem;
  const cuuint64_t next = stack ? static_cast<cuuint64_t>(m.stride) * elem : pitch;
  const cuuint64_t count = static_cast<cuuint64_t>(stack ? m.count : 1);
  const cuuint64_t rows = static_cast<cuuint64_t>(m.rows), cols = static_cast<cuuint64_t>(m.cols);
  const cuuint32_t height = static_cast<cuuint32_t>(lines);
  cuuint64_t dims[4] = {cols, rows, count, 1}, strides[3] = {pitch, next, 0};
  cuuint32_t box[4] = {line, height, 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  if (chunks > 1) {
    dims[0] = line;
    dims[2] = cols / line;
    dims[3] = count;
    strides[1] = 128;
    strides[2] = next;
    box[2] = static_cast<cuuint32_t>(chunks);
  }
  return fn(out, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
            chunks > 1 ? 4 : 3, const_cast<void *>(ptr), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of the results: boxes of 128 columns by 16 rows, not swizzled.
bool encode_result(const SegMatrix &m, bool f32, CUtensorMap *out) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t elem = f32 ? 4 : 2, pitch = static_cast<cuuint64_t>(m.ld) * elem;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(m.cols), static_cast<cuuint64_t>(m.rows),
                              static_cast<cuuint64_t>(m.count)};
  const cuuint64_t strides[2] = {
      pitch, m.count > 1 ? static_cast<cuuint64_t>(m.stride) * elem : pitch};
  const cuuint32_t box[3] = {kHalf, 16, 1}, step[3] = {1, 1, 1};
  return fn(out, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void *>(m.p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// TMA reads 16-byte aligned rows; a stride of zero (one matrix for all) is not
// a stride of its maps.
bool tma_ok(const SegMatrix &m, const void *p, int elem) {
  const int per16 = 16 / elem;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && m.ld % per16 == 0 && m.stride % per16 == 0 &&
         (m.count <= 1 || m.stride > 0);
}

long long extent_of(const SegMatrix &m) {
  return (m.count - 1) * m.stride + matrix_extent(m.rows, m.cols, m.ld);
}

SegOperand operand_of(const SegMatrix &m, const void *second, int elem) {
  SegOperand o;
  o.p[0] = m.p;
  o.p[1] = second != nullptr ? second : m.p;
  o.ld = m.ld;
  o.zs = m.stride;
  o.extent = extent_of(m);
  const uintptr_t at = reinterpret_cast<uintptr_t>(o.p[0]) | reinterpret_cast<uintptr_t>(o.p[1]);
  const int per16 = 16 / elem;
  o.vec = at % 16 == 0 && m.ld % per16 == 0 && m.stride % per16 == 0;
  return o;
}

template <class T, bool TMA, bool LMN, bool QMN>
int launch(const CUtensorMap (&maps)[5], const SegTc &p, int sm_count, cudaStream_t stream) {
  using C = Cfg<T, TMA>;
  auto *kernel = seg_tc_kernel<T, TMA, LMN, QMN>;
  const int groups = p.dense ? 1 : p.groups;
  const int fixed = C::kStages * C::kStageBytes + C::kRawBytes + 2 * C::kOutBytes +
                    static_cast<int>(sizeof(Shared<C::kStages, C::kRawStages>)) + 1024;
  const int smem = fixed + groups * 8 + 8;
  static std::once_flag once;
  static bool ready = false;
  std::call_once(once, [&] {
    cudaFuncAttributes at;
    ready = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 fixed + kMaxSegments * 8 + 8) == cudaSuccess &&
            cudaFuncGetAttributes(&at, kernel) == cudaSuccess &&
            // the register split draws on the launch's registers
            (!C::kSplit || at.numRegs * C::kThreads >= 128 * 40 + 256 * 152 + 256 * 64);
  });
  if (!ready) return kErrLaunch;
  // Tiles at most: every segment may end in a part tile.
  const long long height = p.wgrad ? p.K : p.M;
  long long tiles = p.wgrad ? static_cast<long long>(groups) * ((height + kCols - 1) / kCols)
                            : height / kCols + (p.dense ? 1 : groups);
  tiles *= p.tiles_n;
  if (tiles > 0x7fffffffLL) return kErrInvalidArg;
  long long pairs = sm_count / 2;
  if (pairs > tiles) pairs = tiles;
  if (pairs < 1) pairs = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], maps[4], p) == cudaSuccess
             ? kOk
             : kErrLaunch;
}

template <class T, bool TMA>
int launch_layout(bool lmn, bool qmn, const CUtensorMap (&maps)[5], const SegTc &p, int sm_count,
                  cudaStream_t stream) {
  if (qmn) return launch<T, TMA, true, true>(maps, p, sm_count, stream);
  if (lmn) return launch<T, TMA, true, false>(maps, p, sm_count, stream);
  return launch<T, TMA, false, false>(maps, p, sm_count, stream);
}

}  // namespace

GEMM_INDEX_FAULT_TAKE(seg_tc_index_fault_take)

int seg_tc_poll_status(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return kErrLaunch;
  int h = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&h, g_seg_status, sizeof(int)) != cudaSuccess) return kErrLaunch;
  if (h != 0 && cudaMemcpyToSymbol(g_seg_status, &zero, sizeof(int)) != cudaSuccess)
    return kErrLaunch;
  return h;
}

int seg_tc_launch(const SegArgs &a, int sm_count, cudaStream_t stream) {
  SegTc p = {};
  p.wgrad = a.wgrad;
  p.dense = a.dense;
  p.groups = static_cast<int>(a.groups);
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.bank = static_cast<int>(a.bank);
  p.passes = a.A_lo != nullptr || a.B_lo != nullptr ? 2 : 1;
  p.tiles_n = static_cast<int>((a.N + kLanes - 1) / kLanes);
  p.offsets = a.offsets;
  p.index = a.index;
  p.scales = a.scales;
  p.add = static_cast<const float *>(a.add.p);
  p.add_ld = a.add.ld;
  p.add_extent = extent_of(a.add);
  p.C = const_cast<void *>(a.C.p);
  p.c_f32 = !a.bf16 || a.c_f32;
  const int64_t c_elem = p.c_f32 ? 4 : 2;
  p.c_rows = a.C_lo.p == nullptr && reinterpret_cast<uintptr_t>(a.C.p) % 16 == 0 &&
             a.C.ld * c_elem % 16 == 0 && a.C.stride * c_elem % 16 == 0 && a.N * c_elem % 16 == 0;
  p.c_ld = a.C.ld;
  p.c_stride = a.C.stride;
  p.c_extent = extent_of(a.C);
  p.C_lo = const_cast<void *>(a.C_lo.p);
  p.c_lo_ld = a.C_lo.ld;
  p.c_lo_extent = extent_of(a.C_lo);
  // 2 s, and 2 us for each k of the longest contraction.
  p.timeout_ns = 2000000000ull + 2000ull * static_cast<unsigned long long>(a.wgrad ? a.M : a.K);
  // Lines per copy of Q: about half a tile's rows, as the average segment has
  // them, so that small segments do not read their neighbours' rows.
  const long long average = p.dense ? a.M : a.M / (a.groups > 0 ? a.groups : 1);
  p.q_box = average <= 64 ? 32 : (average <= 128 ? 64 : 128);
  const bool lmn = a.wgrad || !a.transb, qmn = a.wgrad;
  const int elem = a.bf16 ? 2 : 4;
  p.L = operand_of(a.B, a.B_lo, elem);
  p.Q = operand_of(a.A, a.A_lo, elem);
  CUtensorMap maps[5];
  std::memset(maps, 0, sizeof(maps));
  const bool empty = a.K == 0 || a.M == 0;  // no operand is read
  const bool tma = !empty && tma_ok(a.B, p.L.p[0], elem) && tma_ok(a.B, p.L.p[1], elem) &&
                   tma_ok(a.A, p.Q.p[0], elem) && tma_ok(a.A, p.Q.p[1], elem);
  if (tma) {
    const int line = 128 / elem, bk = a.bf16 ? 64 : 32;
    const int l_lines = lmn ? bk : kHalf, q_lines = qmn ? bk : p.q_box;
    // One copy of all chunks, where every tile has them all: lanes always do.
    p.l_whole = lmn && a.N % line == 0;
    p.q_whole = qmn && a.K % kCols == 0;
    const int lc = p.l_whole ? kHalf / line : 1, qc = p.q_whole ? kHalf / line : 1;
    if (!encode_lines(a.B, p.L.p[0], a.bf16, l_lines, lc, &maps[0]) ||
        !encode_lines(a.A, p.Q.p[0], a.bf16, q_lines, qc, &maps[2]))
      return kErrLaunch;
    maps[1] = maps[0];
    maps[3] = maps[2];
    if ((a.B_lo != nullptr && !encode_lines(a.B, a.B_lo, a.bf16, l_lines, lc, &maps[1])) ||
        (a.A_lo != nullptr && !encode_lines(a.A, a.A_lo, a.bf16, q_lines, qc, &maps[3])))
      return kErrLaunch;
  }
  if (p.c_rows && !encode_result(a.C, p.c_f32, &maps[4])) return kErrLaunch;
  if (a.bf16)
    return tma ? launch_layout<__nv_bfloat16, true>(lmn, qmn, maps, p, sm_count, stream)
               : launch_layout<__nv_bfloat16, false>(lmn, qmn, maps, p, sm_count, stream);
  return tma ? launch_layout<float, true>(lmn, qmn, maps, p, sm_count, stream)
             : launch_layout<float, false>(lmn, qmn, maps, p, sm_count, stream);
}

}  // namespace gemm
