// seg_tc.cu -- segmented matrix products on the tensor cores of sm_103a.
//
// A tile of the result is computed transposed, D = L Q^T, on a CTA pair
// (tcgen05 cta_group::2): 256 lanes n (columns of the result, 128 a CTA) by up
// to 256 columns q,
//
//   rows:    D[n, t] = sum_k B_z[k, n] A[t, k]     q = rows t of one segment
//   adapted: D[n, t] = sum_k B[k, n] A[t, k] + sum_r L_a[r, n] U[t, r]
//   wgrad:   D[n, i] = sum_t B[t, n] A[t, i]       t = rows of the segment
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
// Both types come by TMA. bf16 operands, 64 k of 128 + 128 lines a stage, go to
// kind::f16 MMAs as they are. float32 values, 32 k a stage, are split by eight
// warps into three bf16 terms on the way,
//
//   x = h + m + l,   h = bf16(x), m = bf16(x - h), l = bf16(x - h - m),
//
// exact for |x| from 2^-110 to the largest finite value (24 bits in three terms
// of 8; Henry, Tang and Heinecke, "Leveraging the bfloat16 artificial
// intelligence datatype for higher-precision computations", ARITH 2019). h is
// rounded to the largest finite bf16, not to infinity (|x| >= 3.3962e38); m is
// then 2^-8 of x as elsewhere. Below 2^-110 the last bits fall under bf16's
// smallest value: x is held to 2^-134. Of an infinite x the terms are finite,
// infinite and NaN. The products hh, hm, mh, mm, hl, lh are summed; those left
// out are below 2^-24 of |x y|.
//
// The tensor core truncates as it adds to an accumulator: sums of K products
// drift by about 2^-24 per MMA (measured: 4.4e-6 of the result's norm after
// 256 bf16 MMAs of one accumulator, against 1.1e-6 of an FP32 FMA chain). For
// float32 each accumulator therefore holds 64 k only, a stage's small products
// first, and the epilogue warps add it to sums in registers, rounded to
// nearest, while the next one fills (3.3e-7 whatever K; with 128 k 7.5e-7).
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

#include "seg_ptx.cuh"
#include "seg_terms.cuh"
#include "segments.h"

namespace gemm {

__device__ int g_seg_status;  // first error recorded by a kernel of this unit

namespace {

constexpr int kLanes = 256;     // result columns per tile (MMA M, of the pair)
constexpr int kCols = 256;      // most rows per tile (MMA N)
constexpr int kHalf = 128;      // lanes, and columns at most, of one CTA of the pair
constexpr int kColStep = 32;    // granularity of the MMA's N
constexpr int kRasterM = 8;     // row tiles per raster group
constexpr int kBlock = 64;      // k of a block: a bf16 stage, or a float32 accumulator
constexpr int kMaxSplits = 16;
// Splitting a tile along k costs about 4 us (the sums' way through memory, and
// the counters' zeros before the launch); blocks take 0.3 us (bf16) and up to 2
// us (float32). Fewest blocks of an item, and of a contraction worth splitting.
constexpr int kItemBlocksBf16 = 8, kItemBlocksF32 = 3, kSplitBlocksBf16 = 32, kSplitBlocksF32 = 8;
constexpr uint32_t kTmemCols = 512;

enum Form : int { kRows = 0, kDense = 1, kAdapted = 2, kWgrad = 3 };

struct SegTc {
  int form;
  int groups;        // segments
  int entries;       // of the table: groups; dense 1; adapted groups + 2
  int M, N, K, R, bank;
  int z_step, a_step;  // 0: one matrix for every segment, one L for every adapter
  // Passes over the operands of a tile: one, or two with a two-term operand;
  // adapted: A and B, then U (its terms) and the adapter's L.
  int passes;
  int tiles_n;
  int q_box, q_shift;  // lines per copy of a K-major Q: 1 << q_shift
  int q_whole;       // wgrad, one pass: maps.q[2] brings all chunks of Q in one copy
  int l_whole, l_whole1;  // the MN-major L of pass 0, of the others, comes as one 4-D copy
  const int64_t *offsets;
  const int32_t *index;
  const float *scales;
  const float *add;  // dense: fp32 addend of the rows that the segments hold
  long long add_ld, add_extent;
  void *C, *C_lo;    // C_lo: the result's second term
  int c_f32;
  int c_rows;        // rows of the result can leave by TMA
  long long c_ld, c_lo_ld, c_stride, c_extent, c_lo_extent;
  // Few tiles: the blocks of each go to several pairs, which leave their sums
  // in slots (one a work item, at most as many as pairs, 2 x 256 x 128 floats); the last one adds them.
  float *slots;
  unsigned *arrived;  // [2 tile + rank] of the split tiles, zero
  long long slot_extent;
  // > 0: so many rows and segments that offsets which claim rows again and again
  // could make more tiles than 32 bits count: the tiles there are at most
  // otherwise.
  int most_tiles;
  int few;            // rows: segments of up to this many are another launch's
  int ahead;          // starts before the launch before it has ended (SegArgs::ahead)
  unsigned long long timeout_ns;
};

template <class T>
struct Cfg {
  static constexpr bool kSplit = std::is_same<T, float>::value;  // three-term operands
  static constexpr int kTerms = kSplit ? 3 : 1;
  // k per stage: 128-byte lines of bf16, or 64-byte ones of each float32 term
  // (two stages of three terms leave room for the values in flight).
  static constexpr int kBK = kSplit ? 32 : 64;
  static constexpr int kOpBytes = kHalf * kBK * 2;  // one term of one operand
  static constexpr int kStageBytes = 2 * kTerms * kOpBytes;
  static constexpr int kStages = kSplit ? 2 : 6;
  // Float32 values on their way: lines of 32 (128 bytes, 128-byte swizzle),
  // 128 of either operand a stage.
  static constexpr int kRawOpBytes = kHalf * 128;
  static constexpr int kRawStages = kSplit ? 3 : 1;
  static constexpr int kRawBytes = kSplit ? kRawStages * 2 * kRawOpBytes : 0;
  // Results on their way out, for each four epilogue warps: 16 rows of 128 (8
  // float32 rows of a bf16 product).
  static constexpr int kOutBytes = kSplit ? 8192 : 4096;
  static constexpr int kMmaWarp = 1;
  static constexpr int kFixWarp = 2;
  // Epilogue warps. bf16: 8192 x 11008 x 4096 takes 444 us with eight, 415 with
  // sixteen; float32 has registers for eight. Those of a quarter of the lanes
  // take sixteen columns each in turn, kEpiStep apart, so that they share narrow
  // tiles too: with a run of columns for each, 2048 x 16 x 2048 in float32 takes
  // 43 us, not 35.5.
  static constexpr int kEpiWarp0 = 4, kEpiWarps = kSplit ? 8 : 16;
  static constexpr int kEpiStep = 16 * (kEpiWarps / 4);
  static constexpr int kLoadWarp0 = 12, kLoadWarps = 8;
  static constexpr int kThreads = 32 * (kSplit ? kLoadWarp0 + kLoadWarps : kEpiWarp0 + kEpiWarps);
};

template <int STAGES, int RAW>
struct Shared {
  uint64_t full[STAGES], empty[STAGES], part[STAGES];
  uint64_t raw_full[RAW], raw_empty[RAW];
  uint64_t acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  int abort;
  int tiles[3];  // of width 256, 128, 64
  int longest;   // rows of the longest segment
  int cut[3];    // Table::shift, whole, splits
  int last;      // this CTA's sums complete a split tile
};

// One work item -- a tile of the list, or a part of its blocks -- as every role
// sees it.
struct Tile {
  int over, tile;   // split tiles: item and tile past the whole ones
  int g, z;         // segment; its matrix
  int a;            // adapted: the segment's adapter
  int n0;           // first lane (result column)
  int q0, qn;       // first column (rows form: row of the result), and how many
  int k0;           // wgrad: first row of the contraction
  int klen, xlen;   // k of the first pass, of each of the others
  int b0, b1;       // blocks to sum, counted through the passes
  bool split;       // others sum other blocks of the tile
};

struct SegMaps {
  CUtensorMap l[3], q[3], c;  // by pass; of the results
};

struct Table {
  int *first;     // [entries + 1] tiles of the entries before
  int *row;       // [entries + 1] offsets, held to the rows there are
  int shift;      // most columns of a tile: 1 << shift
  int whole;      // tiles that are one work item each; the others are
  int splits;     // this many
};

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// a / b for a >= 0, b > 0: the integer divisions of a tile's place in the list
// would be half a microsecond in every role's way.
__device__ __forceinline__ int quotient(int a, int b) {
  if (a >= 1 << 22) return a / b;
  const int q = static_cast<int>(__fdividef(static_cast<float>(a) + 0.5f, static_cast<float>(b)));
  return q - (q * b > a) + ((q + 1) * b <= a);
}

// An offset, held to the rows there are.
__device__ __forceinline__ int held(long long offset, int rows) {
  return static_cast<int>(offset < 0 ? 0 : (offset > rows ? rows : offset));
}

// Rows of an entry, none where they are another launch's.
__device__ __forceinline__ int rows_of(const SegTc &p, const Table &tab, int g) {
  const int rows = tab.row[g + 1] - tab.row[g];
  return rows > p.few ? rows : 0;
}

__device__ __forceinline__ int matrix_of(const SegTc &p, int g) {
  const int z = p.index != nullptr ? p.index[g] : g;
  return z >= 0 && z < p.bank ? z : -1;
}

// Passes of a tile in blocks: f(pass, length, first k, last k) for each pass
// that has some of the item's blocks; false stops.
template <class F>
__device__ __forceinline__ bool for_passes(const SegTc &p, const Tile &t, const F &f) {
  int base = 0;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int len = pass == 0 ? t.klen : t.xlen, n = cdiv(len, kBlock);
    const int lo = max(t.b0 - base, 0), hi = min(t.b1 - base, n);
    if (lo < hi && !f(pass, len, lo * kBlock, min(hi * kBlock, len))) return false;
    base += n;
  }
  return true;
}

__device__ __forceinline__ bool tile_at(const SegTc &p, const Table &tab, int item, Tile &o) {
  const int over = item - tab.whole;
  const int t = over < 0 ? item : tab.whole + quotient(over, tab.splits);
  if (t >= tab.first[p.entries]) return false;
  int lo = 0, hi = p.entries;  // the entry whose tiles hold t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.first[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int idx = t - tab.first[lo];
  const int r0 = tab.row[lo], rows = rows_of(p, tab, lo);
  const int height = p.form == kWgrad ? p.K : rows;
  const int tm = (height + (1 << tab.shift) - 1) >> tab.shift;
  // Groups of kRasterM row tiles, lane tiles in the outer loop, so that the
  // pairs at work at one time share operand tiles in L2.
  const int group = quotient(idx, kRasterM * p.tiles_n);
  const int m_first = group * kRasterM;
  const int across = min(kRasterM, tm - m_first);
  const int rem = idx - group * kRasterM * p.tiles_n;
  const int ni = quotient(rem, across), mi = m_first + rem - ni * across;
  // The segment's rows in tm equal parts (in steps the MMA allows), not whole
  // tiles and a rest: the pairs end together, and no tile is all operand
  // traffic and no work.
  const int step = p.form == kWgrad ? 128 : kColStep;  // a power of two
  const int part = (quotient(height + tm - 1, tm) + step - 1) & ~(step - 1);
  o.over = over;
  o.tile = t - tab.whole;
  o.g = lo;
  o.n0 = ni * kLanes;
  o.qn = min(part, height - mi * part);
  o.q0 = mi * part;
  o.k0 = 0;
  o.z = 0;
  o.a = -1;
  o.klen = o.xlen = p.K;
  if (p.form == kWgrad) {
    o.k0 = r0;
    o.klen = o.xlen = rows;
  } else {
    o.q0 += r0;
    if (p.form == kRows) {
      o.z = matrix_of(p, lo);
      if (o.z < 0) o.klen = o.xlen = 0;
    } else if (p.form == kAdapted) {
      o.a = lo > 0 && lo <= p.groups ? matrix_of(p, lo - 1) : -1;
      o.xlen = o.a >= 0 ? p.R : 0;
    }
  }
  const int blocks = cdiv(o.klen, kBlock) + (p.passes - 1) * cdiv(o.xlen, kBlock);
  o.split = over >= 0 && tab.splits > 1;
  if (o.split) {
    const int s = over - (t - tab.whole) * tab.splits;
    o.b0 = quotient(blocks * s, tab.splits);
    o.b1 = quotient(blocks * (s + 1), tab.splits);
  } else {
    o.b0 = 0;
    o.b1 = blocks;
  }
  return true;
}

// How the list is cut, from its tiles at each width (every CTA finds the same):
// by the time it should take, in microseconds.
//
// A block of 64 k takes nearly the same at every width (256, 128, 64 columns:
// bf16 0.302, 0.282, 0.275, float32 1.99, 1.72, 1.55), so narrower tiles pay
// only where they fill pairs that would be idle. Tiles past the last full round
// can be split along k where that leaves every pair at most one item; the item
// that completes a tile reads the others' sums, bound by their way through L2
// (256 columns, 128 KB a CTA: about 2.1 us an item), so the best number of items
// is the root of the tile's time over that, and few columns allow many.
// A whole warp: lane i looks at width 256 >> i.
template <bool SPLIT>
__device__ __forceinline__ void choose_cut(const SegTc &p, const int *tiles, int longest, int pairs,
                                           int lane, Table &tab) {
  constexpr float kBlockUs = SPLIT ? 2.0f : 0.3f, kFixedCols = SPLIT ? 640.0f : 1800.0f;
  constexpr float kItemUs = SPLIT ? 9.0f : 5.0f;  // an item's start and end
  constexpr float kPerCol = kBlockUs / (kCols + kFixedCols);
  const int blocks = p.passes * cdiv(p.form == kWgrad ? longest : p.K, kBlock);
  const int rows = p.form == kWgrad ? p.K : longest;
  const int i = lane < (p.form == kWgrad ? 2 : 3) ? lane : 0;
  const int n = tiles[i], width = kCols >> i;
  const int rounds = quotient(n, pairs), rest = n - rounds * pairs;
  const float tile = blocks * (width + kFixedCols) * kPerCol;
  const float item = 2.1f / kCols * static_cast<float>(min(width, rows));  // its sums' reading
  int splits = 1;
  if (rest > 0 && p.slots != nullptr) {
    splits = min(static_cast<int>(sqrtf(__fdividef(tile, item))), quotient(pairs, rest));
    splits = min(min(splits, kMaxSplits), blocks / (SPLIT ? kItemBlocksF32 : kItemBlocksBf16));
    splits = max(splits, 1);
  }
  const float last =
      rest == 0 ? 0.0f
                : (splits > 1 ? __fdividef(tile, static_cast<float>(splits)) + splits * item + kItemUs
                              : tile);
  float time = static_cast<float>(rounds) * tile + last;
  int best = 0;
#pragma unroll
  for (int q = 1; q < 3; ++q) {  // wider ones first: a tie is theirs
    const float other = __shfl_sync(0xffffffffu, time, q), mine = __shfl_sync(0xffffffffu, time, best);
    if (other < mine) best = q;
  }
  tab.shift = 8 - best;
  tab.splits = __shfl_sync(0xffffffffu, splits, best);
  tab.whole = __shfl_sync(0xffffffffu, splits > 1 ? n - rest : n, best);
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

// From L2, and behind grid_dependency_wait(): the grid before may have written
// it while this one ran, so it is no constant of this grid's.
__device__ __forceinline__ float load_added(const float *p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

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

// Arrivals on a barrier of the even CTA (its shared::cluster address), for a
// thread of that CTA that waits with acquire at cluster scope.
//
// Of lines in shared memory, which both CTAs' tensor core reads: every thread
// that wrote some has fenced them for the asynchronous proxy and met this one.
// A release at cluster scope of shared memory alone: a full one also waits for
// whatever else is under way and took 280 ns of every float32 stage (4096 rows,
// 2048 x 2048 in 8 segments: 158 us with this one, 184 with that).
__device__ __forceinline__ void mbar_arrive_filled(uint32_t bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
      : "memory");
}

// Of TMEM that has been read out: tcgen05's own fences, before this arrival and
// behind the wait, order the loads before the next MMAs.
__device__ __forceinline__ void mbar_arrive_drained(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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

// ----------------------------------------------------------- float32 terms --

// Two values rounded to nearest; FINITE: past the largest value, to it.
template <bool FINITE>
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t w;
  if constexpr (FINITE)
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// Eight float32 values as three bf16 terms (`term` bytes apart).
__device__ __forceinline__ void store_terms(uint8_t *dst, int term, float (&v)[8]) {
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = t == 0 ? pack_bf16<true>(v[2 * i], v[2 * i + 1]) : pack_bf16<false>(v[2 * i], v[2 * i + 1]);
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
template <class T, bool LMN, bool QMN>
__global__ void __launch_bounds__(Cfg<T>::kThreads, 1)
    seg_tc_kernel(const __grid_constant__ SegMaps maps, const __grid_constant__ SegTc p) {
  using C = Cfg<T>;
  constexpr int STAGES = C::kStages, kBK = C::kBK, kOpBytes = C::kOpBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *stages = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *raw = stages + STAGES * C::kStageBytes;
  uint8_t *out = raw + C::kRawBytes;
  using Sh = Shared<STAGES, C::kRawStages>;
  Sh *sh = reinterpret_cast<Sh *>(out + C::kEpiWarps / 4 * C::kOutBytes);
  Table tab;
  tab.row = reinterpret_cast<int *>(sh + 1);
  tab.first = tab.row + p.entries + 1;
  volatile int *abort = &sh->abort;

  const uint32_t warp = warp_index();
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  // Arrivals that fill a stage. Copies straight to it: the even CTA's (both
  // CTAs' bytes), or for weight gradients one arrival from each CTA's copies or
  // masks. float32: one from each CTA's load warps.
  constexpr int kFullCount = C::kSplit || QMN ? 2 : 1;
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);

  if (p.few > 0) {
    // Nothing to do where all segments are the launch before's, behind whose
    // end this one ends (for the launches that count on that).
    int any = 0;
    for (int g = threadIdx.x; g < p.groups; g += C::kThreads)
      any |= held(p.offsets[g + 1], p.M) - held(p.offsets[g], p.M) > p.few;
    if (!__syncthreads_or(any)) {
      grid_dependency_wait();
      return;
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh->full[s], kFullCount);
      mbar_init(&sh->empty[s], 1);
      mbar_init(&sh->part[s], 1);  // this CTA's bytes of a stage that is masked before use
    }
    for (int s = 0; s < C::kRawStages; ++s) {
      mbar_init(&sh->raw_full[s], 1);
      mbar_init(&sh->raw_empty[s], C::kLoadWarps);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sh->acc_full[a], 1);
      mbar_init(&sh->acc_empty[a], 2);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    sh->tiles[0] = sh->tiles[1] = sh->tiles[2] = sh->longest = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&maps.l[0]);
    tma_prefetch_map(&maps.q[0]);
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc<2>(&sh->tmem_base, kTmemCols);
    tmem_relinquish<2>();
  }
  // The arguments into the constant cache while the previous grid ends: the
  // roles' first looks at them would each wait for memory.
  for (uint32_t i = threadIdx.x; i < sizeof(SegTc) / 4; i += C::kThreads) {
    const int touched = reinterpret_cast<const int *>(&p)[i];
    asm volatile("" ::"r"(touched));
  }
  // ahead: what is read from here on was there before the previous grid began;
  // the copies wait for it before they read U, the epilogue before it writes.
  if (!p.ahead) grid_dependency_wait();
  // The table of segments: their rows, and the tiles before each.
  for (int g = threadIdx.x; g <= p.entries; g += C::kThreads) {
    long long a;
    if (p.form == kDense)
      a = g ? p.M : 0;
    else if (p.form == kAdapted)  // rows before and behind the segments, too
      a = g == 0 ? 0 : (g == p.entries ? p.M : p.offsets[g - 1]);
    else
      a = p.offsets[g];
    tab.row[g] = held(a, p.M);
  }
  __syncthreads();
  if (p.most_tiles > 0) {
    // Such offsets get no tiles (their rows' results are unspecified).
    if (threadIdx.x == 0) {
      long long sum = 0;
      for (int g = 0; g < p.entries; ++g)
        sum += static_cast<long long>(cdiv(rows_of(p, tab, g), kCols / 4)) * p.tiles_n;
      sh->longest = sum > p.most_tiles ? -1 : 0;
    }
    __syncthreads();
    const bool none = sh->longest < 0;
    __syncthreads();
    for (int g = threadIdx.x; none && g <= p.entries; g += C::kThreads) tab.row[g] = 0;
    if (threadIdx.x == 0) sh->longest = 0;
    __syncthreads();
  }
  for (int g = threadIdx.x; g < p.entries; g += C::kThreads) {
    const int rows = rows_of(p, tab, g);
    const int height = p.form == kWgrad ? p.K : rows;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (height > 0) atomicAdd(&sh->tiles[i], cdiv(height, kCols >> i) * p.tiles_n);
    atomicMax(&sh->longest, rows);
  }
  __syncthreads();
  if (warp == 0) {
    choose_cut<C::kSplit>(p, sh->tiles, sh->longest, pairs, static_cast<int>(lane), tab);
    if (lane == 0) {
      sh->cut[0] = tab.shift;
      sh->cut[1] = tab.whole;
      sh->cut[2] = tab.splits;
    }
    int sum = 0;
    for (int g0 = 0; g0 < p.entries; g0 += 32) {
      const int g = g0 + static_cast<int>(lane);
      int own = 0;
      if (g < p.entries)
        own = cdiv(p.form == kWgrad ? p.K : rows_of(p, tab, g), 1 << tab.shift) * p.tiles_n;
      int v = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, d);
        if (static_cast<int>(lane) >= d) v += w;
      }
      if (g < p.entries) tab.first[g] = sum + v - own;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) tab.first[p.entries] = sum;
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // barriers and TMEM of both CTAs are set up
  tc_fence_after_sync();
  const uint32_t tmem = sh->tmem_base;
  tab.shift = sh->cut[0];
  tab.whole = sh->cut[1];
  tab.splits = sh->cut[2];
  // Only behind the wait: when a grid starts, all but the last one before it
  // are then complete, which is what an `ahead` grid builds on.
  if (!p.ahead) grid_launch_dependents();

  const bool epilogue = warp >= C::kEpiWarp0 && warp < C::kEpiWarp0 + C::kEpiWarps;
  Tile t;
  if (warp == 0) {
    // ------------------------------------------------------------- copies --
    // bf16: into the stages, both CTAs' bytes on the even CTA's barrier.
    // float32: into this CTA's ring of raw values.
    set_registers<C::kSplit, 40>();
    constexpr int kLine = C::kSplit ? 32 : 64;          // elements of a line
    constexpr int kChunk = kBK * 128;                   // bytes of an MN-major chunk
    constexpr int RING = C::kSplit ? C::kRawStages : STAGES;
    constexpr int kSlot = C::kSplit ? 2 * C::kRawOpBytes : C::kStageBytes;
    uint8_t *const ring = C::kSplit ? raw : stages;
    if (lane == 0) {
      uint64_t *const ring_empty = C::kSplit ? sh->raw_empty : sh->empty;
      uint64_t *const ring_full = C::kSplit ? sh->raw_full : sh->full;
      Ring<RING> r;
      uint32_t part_phase = 0, parts = 0;  // stages that went to part[], by phase and at all
      int issued = 0;
      bool ok = true;
      const uint32_t full0 = C::kSplit ? smem_addr(sh->raw_full) : mbar_cluster_addr(sh->full, 0);
      for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
        const int half = mma_cols<QMN>(t) / 2;
        const int ln = t.n0 + static_cast<int>(rank) * kHalf;
        const int qn = t.q0 + static_cast<int>(rank) * half;
        const int copies = QMN ? half / kLine : (half + p.q_box - 1) >> p.q_shift;
        const uint32_t bytes =
            static_cast<uint32_t>(kHalf * 128 + copies * (QMN ? kChunk : 128 * p.q_box));
        ok = for_passes(p, t, [&](int pass, int len, int k_lo, int k_hi) {
          const CUtensorMap *ml = &maps.l[pass], *mq = &maps.q[pass];
          const int lz = p.form == kAdapted && pass > 0 ? t.a * p.a_step : t.z * p.z_step;
          const bool whole = pass > 0 && p.form == kAdapted ? p.l_whole1 : p.l_whole;
          if (p.ahead && pass > 0 && p.form == kAdapted) {  // U is the previous grid's
            grid_dependency_wait();
            asm volatile("fence.proxy.async;" ::: "memory");
          }
          for (int kk = k_lo; kk < k_hi; kk += kBK) {
            if (!wait(&ring_empty[r.idx], r.phase ^ 1, p, abort)) return false;
            uint8_t *l = ring + r.idx * kSlot;
            uint8_t *q = l + kHalf * 128;
            uint32_t bar = full0 + r.idx * 8;
            parts &= ~(1u << r.idx);
            if (C::kSplit) {
              mbar_arrive_expect_tx(&ring_full[r.idx], bytes);
            } else if (QMN && len - kk < kBK && (len - kk) % 16 != 0) {
              // This CTA's own barrier; the mask warp passes it on.
              bar = smem_addr(&sh->part[r.idx]);
              mbar_arrive_expect_tx(&sh->part[r.idx], bytes);
              parts |= 1u << r.idx;
              part_phase ^= 1u << r.idx;
            } else if (rank == 0) {
              mbar_arrive_expect_tx(&ring_full[r.idx], 2 * bytes);
              if (QMN) mbar_arrive(&ring_full[r.idx]);
            }
            if (!LMN) {
              tma_load_3d_pair(l, ml, bar, kk, ln, lz);
            } else if (whole) {
              tma_load_4d_pair(l, ml, bar, 0, t.k0 + kk, ln / kLine, lz);
            } else {
#pragma unroll
              for (int c = 0; c < kHalf / kLine; ++c)
                tma_load_3d_pair(l + c * kChunk, ml, bar, ln + c * kLine, t.k0 + kk, lz);
            }
            if (QMN && p.q_whole && half == kHalf) {
              tma_load_4d_pair(q, &maps.q[2], bar, 0, t.k0 + kk, qn / kLine, 0);
              ++issued;
              r.next();
              continue;
            }
            for (int c = 0; c < copies; ++c) {
              if (QMN)
                tma_load_3d_pair(q + c * kChunk, mq, bar, qn + c * kLine, t.k0 + kk, 0);
              else
                tma_load_3d_pair(q + c * p.q_box * 128, mq, bar, kk, qn + c * p.q_box, 0);
            }
            ++issued;
            r.next();
          }
          return true;
        });
      }
      // On a timeout let the copies that were started land: those of the last
      // stages issued, one phase back where the ring has wrapped since.
      if (!ok)
        for (int s = 0; s < RING && s < issued; ++s) {
          r.phase ^= r.idx == 0 ? 1u : 0u;
          r.idx = r.idx == 0 ? RING - 1 : r.idx - 1;
          if (parts >> r.idx & 1u)
            drain_wait(&sh->part[r.idx], (part_phase >> r.idx & 1u) ^ 1u, p.timeout_ns);
          else if (C::kSplit || rank == 0)
            drain_wait(&ring_full[r.idx], r.phase, p.timeout_ns);
        }
    }
    __syncwarp();
  } else if (!C::kSplit && QMN && warp == C::kFixWarp) {
    // -------------------------------------------------------------- masks --
    // The last stage of a segment whose rows end inside a step of 16: zero
    // both operands' lines from its end to the step's, which hold the next
    // segment's rows (whatever they are: NaN times zero is NaN).
    Ring<STAGES> r;
    uint32_t part_phase = 0;
    bool ok = true;
    for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
      const int half = mma_cols<QMN>(t) / 2;
      ok = for_passes(p, t, [&](int, int len, int k_lo, int k_hi) {
        for (int kk = k_lo; kk < k_hi; kk += kBK) {
          const int tail = len - kk;
          if (tail < kBK && tail % 16 != 0) {
            if (!warp_wait(&sh->part[r.idx], part_phase >> r.idx & 1u, p, abort)) return false;
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
            if (lane == 0) mbar_arrive_filled(mbar_cluster_addr(&sh->full[r.idx], 0));
          }
          r.next();
        }
        return true;
      });
    }
  } else if (warp == C::kMmaWarp) {
    set_registers<C::kSplit, 40>();
    if (rank == 0 && lane == 0) {
      // --------------------------------------------------- MMA (even CTA) --
      Ring<STAGES> r;
      Ring<2> acc;
      bool ok = true;
      // Descriptors of the first stage; others are a number of 16-byte units on.
      const uint32_t base = smem_addr(stages);
      const uint64_t l0 = line_desc<LMN, kBK>(base);
      const uint64_t q0 = line_desc<QMN, kBK>(base + C::kTerms * kOpBytes);
      constexpr uint32_t kTerm = kOpBytes >> 4, kl = LMN ? 128 : 2, kq = QMN ? 128 : 2;
      for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
        const uint32_t idesc = idesc_bf16(kLanes, static_cast<uint32_t>(mma_cols<QMN>(t)), LMN, QMN);
        uint32_t more = 0;  // 0: the next MMA starts its accumulator
        ok = for_passes(p, t, [&](int, int len, int k_lo, int k_hi) {
          for (int kk0 = k_lo; kk0 < k_hi; kk0 += kBK) {
            // Both CTAs' epilogues have drained the accumulator.
            if (more == 0 && !wait<true>(&sh->acc_empty[acc.idx], acc.phase ^ 1, p, abort))
              return false;
            // Copies alone complete a bf16 stage of the rows form; others have
            // arrivals of the odd CTA's warps (acquire at cluster scope).
            if (!wait<C::kSplit || QMN>(&sh->full[r.idx], r.phase, p, abort)) return false;
            tc_fence_after_sync();
            const int left = len - kk0;
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
                  for (int kk = 0; kk < steps(); ++kk)
                    mma_bf16_pair(d, l + tl[c] * kTerm + kk * kl, q + tq[c] * kTerm + kk * kq,
                                  idesc, c + kk > 0 ? 1u : more);
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
            if (C::kSplit && ((kk0 + kBK) % kBlock == 0 || kk0 + kBK >= k_hi)) {
              mma_commit_multicast<2>(&sh->acc_full[acc.idx], 3);
              acc.next();
              more = 0;
            }
            r.next();
          }
          return true;
        });
        if (!C::kSplit && ok && more) {
          mma_commit_multicast<2>(&sh->acc_full[acc.idx], 3);
          acc.next();
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
    const uint32_t tlane = tmem + ((quad * 32) << 16) + part * 16;
    const int c0 = static_cast<int>(part) * 16;  // this warp's first column
    Ring<2> acc;
    int add0 = 0, add1 = 0;  // rows with an addend
    if (p.add != nullptr) {
      add0 = held(p.offsets[0], p.M);
      add1 = held(p.offsets[p.groups], p.M);
    }
    // The accumulator can be refilled: one arrival for all the CTA's epilogue
    // warps. False if one of them gave up on its wait; every warp comes here
    // once for each accumulator.
    auto drained = [&](uint32_t a, bool ok) {
      tc_fence_before_sync();
      ok = named_barrier_and(1, 32 * C::kEpiWarps, ok);
      if (ok && threadIdx.x == 32 * C::kEpiWarp0)
        mbar_arrive_drained(mbar_cluster_addr(&sh->acc_empty[a], 0));
      return ok;
    };
    // Nothing is written, nor `add` read, before the previous grid has ended.
    bool held = p.ahead;
    auto let_go = [&] {
      if (held) {
        grid_dependency_wait();
        grid_launch_dependents();
      }
      held = false;
    };
    for (int i = pair; tile_at(p, tab, i, t); i += pairs) {
      const int blocks = t.b1 - t.b0;
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
            if (ok && c0 + c / 16 * C::kEpiStep < t.qn) {
              uint32_t v[16];
              tmem_load_16cols(tlane + acc.idx * kCols + c / 16 * C::kEpiStep, v);
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
            if (c0 + c / 16 * C::kEpiStep < t.qn) {
              uint32_t v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(sum[c + k]);
              tmem_store_16cols(tlane + acc.idx * kCols + c / 16 * C::kEpiStep, v);
            }
          tmem_store_wait();
        }
      } else if (blocks > 0) {
        ok = warp_wait(&sh->acc_full[acc.idx], acc.phase, p, abort);
        tc_fence_after_sync();
      }
      // All warps go on together from here, or none does.
      if (!named_barrier_and(1, 32 * C::kEpiWarps, ok)) break;
      let_go();
      const float scale = p.form == kRows && p.scales != nullptr && t.z >= 0 ? p.scales[t.z] : 1.0f;
      const long long row0 = t.q0 + c0;
      const long long at = (p.form == kWgrad ? t.g * p.c_stride : 0) + row0 * p.c_ld + n;
      const int count = n < p.N ? t.qn - c0 : 0;  // this lane's columns

      // Sixteen columns from TMEM.
      auto load = [&](int c, float (&f)[16]) {
        if (blocks > 0) {
          uint32_t v[16];
          tmem_load_16cols(tlane + acc.idx * kCols + c, v);
          tmem_load_wait();
          tmem_regs_ready(v);
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] = __uint_as_float(v[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] = 0.0f;
        }
      };
      // Sixteen columns of the result, from c of this warp's on.
      auto finish = [&](int c, float (&f)[16]) {
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] *= scale;
        if (p.add != nullptr) {  // sixteen loads in flight
          const long long from = row0 * p.add_ld + n;
          float a[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int row = t.q0 + c0 + c + k;
            const long long off = from + (c + k) * p.add_ld;
            a[k] = c + k < count && row >= add0 && row < add1 &&
                           index_ok(kSitePartialRead, off, 1, p.add_extent)
                       ? load_added(p.add + off)
                       : 0.0f;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] += a[k];
        }
        if (p.c_rows) {
          // Rows of this CTA's 128 lanes meet in shared memory and leave as
          // whole pieces of their rows.
          const int elem = p.c_f32 ? 4 : 2, row_bytes = kHalf * elem;
          const int rows = C::kOutBytes / row_bytes;  // 16, or 8
          const uint32_t to = smem_addr(out) + part * C::kOutBytes;
          const uint32_t at_lane = to + (quad * 32 + lane) * elem;
          const int n_cta = t.n0 + static_cast<int>(rank) * kHalf;
          const int width = min(kHalf, p.N - n_cta);
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            if (h == 8 && rows == 16) break;
            // The copies that last read the piece are done with it.
            if (quad == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            named_barrier_sync(3 + part, 128);
            if (p.c_f32) {
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (k >= h && k < h + rows)
                  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at_lane + (k - h) * row_bytes),
                               "f"(f[k])
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
              if (c0 + c + h + rows <= t.qn) {
                // One box (as a copy for each row, 256 bytes at a time, results
                // left at 2 TB/s).
                if (lane == 0 && width > 0)
                  store_box(&maps.c, to, n_cta, t.q0 + c0 + c + h, p.form == kWgrad ? t.g : 0);
              } else {  // the segment ends here
                const int row = c + h + static_cast<int>(lane);
                const long long off = at - n + n_cta + row * p.c_ld;
                if (static_cast<int>(lane) < rows && c0 + row < t.qn && width > 0 &&
                    index_ok(kSiteCStore, off, width, p.c_extent))
                  store_bulk(static_cast<uint8_t *>(p.C) + off * elem, to + lane * row_bytes,
                             static_cast<uint32_t>(width * elem));
              }
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
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
                lo[off] = second_term(f[k], __float2bfloat16_rn(f[k]));
            }
          }
        }
      };

      const int c_end = t.qn - c0;
      bool write = true;
      if (t.split) {
        // This item's sums to its slot: four columns of a lane together, lanes
        // side by side. The item that completes the tile adds them all, always
        // in the same order. Warps past the result's last column have none.
        constexpr long long kSlotCta = static_cast<long long>(kCols) * kHalf;
        const bool lanes = n - static_cast<int>(lane) < p.N;
        const long long mine =
            static_cast<long long>(rank) * kSlotCta +
            (static_cast<long long>(c0 / 4) * kHalf + quad * 32 + lane) * 4;
        auto slot = [&](int s, int c) {
          return (static_cast<long long>(t.tile) * tab.splits + s) * 2 * kSlotCta + mine +
                 static_cast<long long>(c) * kHalf;
        };
        const int own = t.over - t.tile * tab.splits;
#pragma unroll 1
        for (int c = 0; lanes && c < c_end; c += C::kEpiStep) {
          float f[16];
          load(c, f);
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            if (index_ok(kSitePartialWrite, slot(own, c + k), 4, p.slot_extent))
              *reinterpret_cast<float4 *>(p.slots + slot(own, c + k)) =
                  make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
        }
        __threadfence();
        named_barrier_sync(1, 32 * C::kEpiWarps);
        if (threadIdx.x == 32 * C::kEpiWarp0) {
          const unsigned before = atomicAdd(&p.arrived[t.tile * 2 + static_cast<int>(rank)], 1u);
          sh->last = before + 1 == static_cast<unsigned>(tab.splits);
        }
        named_barrier_sync(1, 32 * C::kEpiWarps);
        write = sh->last != 0;
        if (write) {
          __threadfence();
#pragma unroll 1
          for (int c = 0; c < c_end; c += C::kEpiStep) {
            float f[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) f[k] = 0.0f;
#pragma unroll 4
            for (int s = 0; s < (lanes ? tab.splits : 0); ++s)
#pragma unroll
              for (int k = 0; k < 16; k += 4)
                if (index_ok(kSitePartialRead, slot(s, c + k), 4, p.slot_extent)) {
                  const float4 v =
                      __ldcg(reinterpret_cast<const float4 *>(p.slots + slot(s, c + k)));
                  f[k] += v.x;
                  f[k + 1] += v.y;
                  f[k + 2] += v.z;
                  f[k + 3] += v.w;
                }
            finish(c, f);
          }
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < c_end; c += C::kEpiStep) {
          float f[16];
          load(c, f);
          finish(c, f);
        }
      }
      if (blocks > 0) {
        drained(acc.idx, true);
        acc.next();
      }
    }
    let_go();
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (C::kSplit && warp >= C::kLoadWarp0) {
    // -------------------------------------------------- float32 to terms --
    // Split the values that have arrived: eight a lane, four lanes to a line
    // of 32. Lanes 4 to 7 of each eight take the line 5 away (k ^ 5), whose
    // swizzled pieces lie in the other banks, as read and as written.
    set_registers<C::kSplit, 64>();
    if constexpr (C::kSplit) {
      const int lw = static_cast<int>(warp) - C::kLoadWarp0;
      const int g = static_cast<int>(lane) >> 2, j = static_cast<int>(lane) & 3;
      const int k8 = (g >> 1) ^ ((g & 1) * 5);  // line within eight
      Ring<STAGES> r;
      Ring<C::kRawStages> a;
      const uint32_t full0 = mbar_cluster_addr(&sh->full[0], 0);
      bool ok = true;
      for (int i = pair; ok && tile_at(p, tab, i, t); i += pairs) {
        const int half = mma_cols<QMN>(t) / 2;
        ok = for_passes(p, t, [&](int, int len, int k_lo, int k_hi) {
          for (int kk = k_lo; kk < k_hi; kk += kBK) {
            bool ready = warp_wait(&sh->raw_full[a.idx], a.phase, p, abort) &&
                         warp_wait(&sh->empty[r.idx], r.phase ^ 1, p, abort);
            const uint8_t *from = raw + a.idx * 2 * C::kRawOpBytes;
            uint8_t *to = stages + r.idx * C::kStageBytes;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const bool mn = u < 2 ? LMN : QMN;
              const int line = ((u & 1) * 8 + lw) * 8 + k8;  // MN-major: chunk * 32 + k
              // K-major Q: rows; MN-major: chunks of 32 columns.
              if (!ready || (u >= 2 && (QMN ? line : line & ~7) >= half)) continue;
              const uint8_t *src = from + (u < 2 ? 0 : C::kRawOpBytes) + line * 128;
              float v[8];
              *reinterpret_cast<float4 *>(v) =
                  *reinterpret_cast<const float4 *>(src + ((2 * j) ^ k8) * 16);
              *reinterpret_cast<float4 *>(v + 4) =
                  *reinterpret_cast<const float4 *>(src + ((2 * j + 1) ^ k8) * 16);
              if (QMN && kk + (line & 31) >= len) {  // the next segment's row
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
            // The CTA's part of the stage is written: one release for all its
            // load warps (a thread of the odd CTA that waited for their
            // arrivals and passed them on was 375 ns of every stage's way).
            // Each warp comes here once a stage; false if one gave up.
            fence_proxy_async_smem();
            if (!named_barrier_and(2, 32 * C::kLoadWarps, ready)) return false;
            if (threadIdx.x == 32 * C::kLoadWarp0) mbar_arrive_filled(full0 + r.idx * 8);
            if (lane == 0) mbar_arrive(&sh->raw_empty[a.idx]);
            a.next();
            r.next();
          }
          return true;
        });
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

// Map over a stack of row-major matrices (one, where its matrices are the same),
// zero outside each: boxes of `box0` columns by `box1` rows; chunks > 1: the
// same seen as chunks of box0 columns (a multiple of them, so that no chunk
// leaves its row), that many a box.
bool encode(const SegMatrix &m, bool bf16, int box0, int box1, int chunks,
            bool swizzle, CUtensorMap *out) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t elem = bf16 ? 2 : 4;
  const bool stack = m.count > 1 && m.stride > 0;
  const cuuint64_t pitch = static_cast<cuuint64_t>(m.ld) * elem;
  const cuuint64_t next = stack ? static_cast<cuuint64_t>(m.stride) * elem : pitch;
  const cuuint64_t count = static_cast<cuuint64_t>(stack ? m.count : 1);
  const cuuint64_t rows = static_cast<cuuint64_t>(m.rows), cols = static_cast<cuuint64_t>(m.cols);
  cuuint64_t dims[4] = {cols, rows, count, 1}, strides[3] = {pitch, next, 0};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(box0), static_cast<cuuint32_t>(box1), 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  if (chunks > 1) {
    dims[0] = box[0];
    dims[2] = cols / box[0];
    dims[3] = count;
    strides[1] = 128;
    strides[2] = next;
    box[2] = static_cast<cuuint32_t>(chunks);
  }
  return fn(out, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
            chunks > 1 ? 4 : 3, const_cast<void *>(m.p), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

long long extent_of(const SegMatrix &m) {
  return (m.count - 1) * m.stride + matrix_extent(m.rows, m.cols, m.ld);
}

template <class T, bool LMN, bool QMN>
int launch(const SegMaps &maps, const SegTc &p, int pairs, cudaStream_t stream) {
  using C = Cfg<T>;
  auto *kernel = seg_tc_kernel<T, LMN, QMN>;
  const int fixed = C::kStages * C::kStageBytes + C::kRawBytes + C::kEpiWarps / 4 * C::kOutBytes +
                    static_cast<int>(sizeof(Shared<C::kStages, C::kRawStages>)) + 1024;
  auto smem = [fixed](int entries) { return fixed + 8 * entries + 8; };
  // Shared memory above the 48 KiB default is enabled once per device.
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return kErrLaunch;
  static bool attr_set[64] = {};
  static std::mutex attr_mu;
  {
    std::lock_guard<std::mutex> g(attr_mu);
    if (!attr_set[dev]) {
      cudaFuncAttributes at;
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               smem(kMaxSegments + 2)) != cudaSuccess ||
          cudaFuncGetAttributes(&at, kernel) != cudaSuccess ||
          // the register split draws on the launch's registers
          (C::kSplit && at.numRegs * C::kThreads < 128 * 40 + 256 * 152 + 256 * 64))
        return kErrLaunch;
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem(p.entries));
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
  return cudaLaunchKernelEx(&cfg, kernel, maps, p) == cudaSuccess ? kOk : kErrLaunch;
}

template <class T>
int launch_layout(bool lmn, bool qmn, const SegMaps &maps, const SegTc &p, int pairs,
                  cudaStream_t stream) {
  if (qmn) return launch<T, true, true>(maps, p, pairs, stream);
  if (lmn) return launch<T, true, false>(maps, p, pairs, stream);
  return launch<T, false, false>(maps, p, pairs, stream);
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

bool seg_tc_readable(const SegMatrix &m, bool bf16) {
  const int per16 = bf16 ? 8 : 4;
  return reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld % per16 == 0 &&
         (m.count <= 1 || m.stride % per16 == 0);
}

bool seg_tc_splits(const SegArgs &a, int terms) {
  const int64_t blocks = ((a.wgrad ? a.M : a.K) + kBlock - 1) / kBlock *
                         (a.A_lo.p != nullptr || a.B_lo.p != nullptr ? 2 : terms);
  return blocks >= (a.bf16 ? kSplitBlocksBf16 : kSplitBlocksF32);
}

int64_t seg_tc_slots(int sm_count) {
  return static_cast<int64_t>(sm_count > 1 ? sm_count / 2 : 1) * 2 * kCols * kHalf;
}

int seg_tc_launch(const SegArgs &a, int sm_count, cudaStream_t stream) {
  SegTc p = {};
  const bool adapted = a.R > 0;
  p.form = a.wgrad ? kWgrad : (adapted ? kAdapted : (a.dense ? kDense : kRows));
  p.groups = static_cast<int>(a.groups);
  p.entries = p.form == kDense ? 1 : p.groups + (adapted ? 2 : 0);
  p.M = static_cast<int>(a.M);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.R = static_cast<int>(a.R);
  p.bank = static_cast<int>(a.bank);
  p.z_step = a.B.count > 1 && a.B.stride == 0 ? 0 : 1;
  p.a_step = a.L.count > 1 && a.L.stride == 0 ? 0 : 1;
  const bool two_terms = a.A_lo.p != nullptr || a.B_lo.p != nullptr;
  p.passes = adapted ? (a.U_lo.p != nullptr ? 3 : 2) : (two_terms ? 2 : 1);
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
  p.few = a.few;
  p.ahead = a.ahead;
  p.c_ld = a.C.ld;
  p.c_stride = a.C.stride;
  p.c_extent = extent_of(a.C);
  p.C_lo = const_cast<void *>(a.C_lo.p);
  p.c_lo_ld = a.C_lo.ld;
  p.c_lo_extent = extent_of(a.C_lo);
  // 2 s, and 2 us for each k of the longest contraction.
  p.timeout_ns = 2000000000ull + 2000ull * static_cast<unsigned long long>(a.wgrad ? a.M : a.K);

  // The tiles there are at most (every segment may end in a part tile, and the
  // narrowest is 64 columns), and at least, if the segments hold all rows.
  const long long height = a.wgrad ? a.K : a.M;
  const long long most = ((a.wgrad ? p.entries * ((height + 127) / 128) : height / 64 + p.entries)) *
                         p.tiles_n;
  const long long least =
      (a.wgrad ? p.entries : 1) * ((height + kCols - 1) / kCols) * p.tiles_n;
  if (most > 0x7fff0000LL) return kErrInvalidArg;  // an item's number and the pairs, < 2^31
  const long long claimed = p.entries * ((height + 63) / 64) * p.tiles_n;
  p.most_tiles = !a.wgrad && claimed > 0x7fff0000LL ? static_cast<int>(most) : 0;
  int pairs = sm_count / 2;
  if (pairs < 1) pairs = 1;
  // Lines per copy of a K-major Q: about half a tile's rows, so that small
  // segments and narrow tiles do not read their neighbours' rows.
  const long long average = p.form == kRows ? a.M / (a.groups > 0 ? a.groups : 1) : a.M;
  p.q_shift = average <= 64 ? 5 : (average <= 128 || least < pairs ? 6 : 7);
  p.q_box = 1 << p.q_shift;

  const bool lmn = a.wgrad || !a.transb, qmn = a.wgrad;
  const int line = a.bf16 ? 64 : 32, bk = a.bf16 ? 64 : 32;
  SegMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  auto encode_l = [&](const SegMatrix &m, int *whole, CUtensorMap *out) {
    // One copy of all chunks of the lanes' operand where no chunk leaves its row.
    *whole = lmn && m.cols % line == 0;
    return encode(m, a.bf16, line, lmn ? bk : kHalf, *whole ? kHalf / line : 1, true, out);
  };
  auto encode_q = [&](const SegMatrix &m, CUtensorMap *out) {
    return encode(m, a.bf16, line, qmn ? bk : p.q_box, 1, true, out);
  };
  if (a.K > 0 && a.M > 0) {  // else no operand is read
    if (!seg_tc_readable(a.A, a.bf16) || !seg_tc_readable(a.B, a.bf16)) return kErrInvalidArg;
    bool ok = encode_l(a.B, &p.l_whole, &maps.l[0]) && encode_q(a.A, &maps.q[0]);
    if (adapted) {
      ok = ok && encode_l(a.L, &p.l_whole1, &maps.l[1]) &&
           encode_q(a.U, &maps.q[1]);
      maps.l[2] = maps.l[1];
      if (ok && a.U_lo.p != nullptr) ok = encode_q(a.U_lo, &maps.q[2]);
    } else if (two_terms) {
      maps.l[1] = maps.l[0];
      maps.q[1] = maps.q[0];
      if (ok && a.B_lo.p != nullptr) ok = encode_l(a.B_lo, &p.l_whole1, &maps.l[1]);
      if (ok && a.A_lo.p != nullptr) ok = encode_q(a.A_lo, &maps.q[1]);
    }
    if (ok && qmn && !two_terms && a.A.cols % line == 0) {
      p.q_whole = 1;
      ok = encode(a.A, a.bf16, line, bk, kHalf / line, true, &maps.q[2]);
    }
    if (!ok) return kErrLaunch;
  }
  if (p.c_rows && !encode(a.C, !p.c_f32, kHalf, a.bf16 && p.c_f32 ? 8 : 16, 1, false, &maps.c)) return kErrLaunch;

  if (a.slots != nullptr && seg_tc_splits(a)) {
    p.slots = a.slots;
    p.arrived = a.arrived;
    p.slot_extent = static_cast<long long>(seg_tc_slots(sm_count));
  } else if (pairs > most) {
    pairs = most > 0 ? static_cast<int>(most) : 1;
  }
  return a.bf16 ? launch_layout<__nv_bfloat16>(lmn, qmn, maps, p, pairs, stream)
                : launch_layout<float>(lmn, qmn, maps, p, pairs, stream);
}

}  // namespace gemm
