// route.cu -- the router of a mixture of experts: scores, the best experts of
// every token, their weights, the plan that sorts the tokens' slots by expert,
// and the gradient of the logits.
//
// Choice. A warp takes a token; lane l holds the V = ceil(E / 32) neighbouring
// experts from l V on. Keys are fp32 values mapped to unsigned integers of the
// same order, so that one redux finds the warp's largest and the lowest lane
// that holds it is that of the lowest expert. Up to 256 experts every lane sorts
// its keys (a network of minima and maxima), with its experts in place of their
// lowest bits, and k rounds take the largest of the lanes' heads. Keys that differ
// in those bits alone are seen where they stand next to each other, and the token
// is chosen again by whole keys. (Looking for the expert in every round, and for
// the lane's next one, was half of all instructions.)
//
// Comparisons. Without bias and sums over groups the logits are the keys: both
// scores ascend with them. Otherwise the keys are s + bias in fp32, which is off
// by rounding; where two keys whose order matters are closer than the bound of
// that (close() below), the token is chosen again in 64 bits (choose_wide): with
// fp32 logits about one token of a thousand (256 experts), so that the slow
// FP64 units are off the path.
//
// Plan. A stable counting sort: each CTA of the router counts its chunk's slots
// by expert, sums the counts of the chunks before its own and ranks its slots, a
// warp 32 at a time by matching experts. Up to 24 tokens one CTA does it all, up to
// 192 the CTAs of a cluster, which read each other's counts in shared memory; of
// more, a second launch (a programmatic dependent) takes the counts from global
// memory. Counts are integers: their order of addition does not show.
//
// Measured (one GB300, all figures of this file: calls back to back in a graph, so that
// logits below some 100 MB are in L2; in brackets by themselves with cold caches, as
// ncu times them). 1 token of 8 experts 3.6 us, 64 of 256 in groups 8.9 (12.7): chains
// of dependent steps of a few warps. 4095 of 64, bf16, softmax, 6 slots: choice 4.0,
// plan 7.5. 32768 of 256, fp32, 8 slots: softmax 34, with a bias 54; sigmoid with a
// bias 47, in 8 groups 56, of these a fifth masked 49 (58); and 16 (17) for the plan;
// against 5 us of memory for the logits: the choice is bound by instructions, 1080 warp
// instructions a token (47 % of the integer lanes' rate). Softmax of one slot takes 23
// us, each further slot 1.5, a bias 6 (one slot) to 20 (eight: of more pairs some are
// too close, and a 64-bit choice at a CTA's end shows as 8). The plan's time is the
// counts of all chunks, which every CTA sums, and two passes over its slots; the
// gradient's 11 us there (15; 64 experts, 4095 tokens: 4.6) are 33 MB written, a row's
// zeros and then its slots; softmax that is not renormalised, three reads of the row
// more, 23.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ptx.cuh"
#include "route.h"

namespace gemm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxSlots = 32;  // of a token
constexpr float kUnit = 5.9604645e-8f;  // 2^-24

struct P {
  const void *logits;
  long long ldx, x_extent;
  const float *bias;
  const uint8_t *mask;
  int32_t *experts;
  float *weights;
  int *hist;  // chunks x E counts (several CTAs)
  int64_t *offsets;
  int32_t *order, *places;
  int T, E, k;
  int sigmoid, renormalise, compare_scores, vec;
  int groups, top_groups, group_best, per_group, group_lanes, group_shift;  // lanes: 1 << shift
  int lanes_hold_groups;  // every lane's experts are of one group, a group's of group_lanes lanes
  float scale;
  int chunk, chunks;  // tokens of a CTA, CTAs
  int plan, plan_warps;
};

// Integers a warp stages: E keys where groups are looked through, and its slots.
__host__ __device__ __forceinline__ int staged_ints(const P &p) {
  return (p.groups > 1 ? p.E : 0) + kMaxSlots;
}

// ------------------------------------------------------------------- values --

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ float load_logit(const P &p, long long t, int e) {
  const long long at = t * p.ldx + e;
  return index_ok(kSiteLoadA, at, 1, p.x_extent) ? as_float(static_cast<const T *>(p.logits)[at])
                                                 : 0.0f;
}

__device__ __forceinline__ float load_bias(const P &p, int e) {
  return p.bias != nullptr && index_ok(kSiteLoadB, e, 1, p.E) ? __ldg(p.bias + e) : 0.0f;
}

// Unsigned integers in the order of the values; 0: not available, 1: NaN. The
// zeros are one value.
__device__ __forceinline__ unsigned key_of(float f) {
  if (f != f) return 1u;
  const unsigned u = __float_as_uint(__fadd_rn(f, 0.0f));
  return u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
  return __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ unsigned long long key_of(double f) {
  if (f != f) return 1ull;
  const unsigned long long u =
      static_cast<unsigned long long>(__double_as_longlong(__dadd_rn(f, 0.0)));
  return u ^ (static_cast<unsigned long long>(static_cast<long long>(u) >> 63) |
              0x8000000000000000ull);
}
__device__ __forceinline__ double value_of(unsigned long long key) {
  return __longlong_as_double(
      static_cast<long long>(key ^ (key >> 63 ? 0x8000000000000000ull : ~0ull)));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, m));
  return v;
}
template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(kFull, v, m);
  return v;
}
__device__ __forceinline__ unsigned warp_best(unsigned v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ unsigned long long warp_best(unsigned long long v) {
  const unsigned high = static_cast<unsigned>(v >> 32), best = __reduce_max_sync(kFull, high);
  const unsigned low = __reduce_max_sync(kFull, high == best ? static_cast<unsigned>(v) : 0u);
  return static_cast<unsigned long long>(best) << 32 | low;
}

__device__ __forceinline__ float sigmoid(float x) {
  const float z = expf(-fabsf(x));
  return (x < 0.0f ? z : 1.0f) / (1.0f + z);
}
__device__ __forceinline__ double sigmoid(double x) {
  const double z = exp(-fabs(x));
  return (x < 0.0 ? z : 1.0) / (1.0 + z);
}

// The two largest of both pairs (a1 >= a2, b1 >= b2).
template <class U>
__device__ __forceinline__ void merge_best(U &a1, U &a2, U b1, U b2) {
  const U low = a1 < b1 ? a1 : b1, second = a2 > b2 ? a2 : b2;
  a1 = a1 < b1 ? b1 : a1;
  a2 = low > second ? low : second;
}

// A group's key from those of its best experts: their sum, of one where it has
// no second.
template <class U>
__device__ __forceinline__ U group_key(U b1, U b2, int best) {
  if (b1 < 2) return b1;
  if (best == 1 || b2 == 0) return b1;
  if (b2 == 1) return 1;
  return key_of(value_of(b1) + value_of(b2));
}

// The `top` largest of a key a lane (0: none), the lowest lane first, as a mask.
template <class U>
__device__ __forceinline__ unsigned choose_lanes(U key, int top) {
  unsigned chosen = 0;
  for (int i = 0; i < top; ++i) {
    const U best = warp_best(key);
    if (best == 0) break;
    const int lane = __ffs(__ballot_sync(kFull, key == best)) - 1;
    chosen |= 1u << lane;
    if ((threadIdx.x & 31) == lane) key = 0;
  }
  return chosen;
}

// Lane r's choice: the r-th best of the keys, -1 where there is none; *last its
// key.
template <int V, class U>
__device__ __forceinline__ int choose_experts(U (&key)[V], int k, U *won) {
  const int lane = threadIdx.x & 31;
  U local = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) local = key[i] > local ? key[i] : local;
  int mine = -1;
  *won = 0;
  for (int r = 0; r < k; ++r) {
    const U best = warp_best(local);
    if (best == 0) break;
    const int from = __ffs(__ballot_sync(kFull, local == best)) - 1;
    int e = 0;
    if (lane == from) {
      // the lowest of its experts with this key goes
      bool found = false;
      local = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!found && key[i] == best) {
          found = true;
          e = lane * V + i;
          key[i] = 0;
        }
        local = key[i] > local ? key[i] : local;
      }
    }
    e = __shfl_sync(kFull, e, from);
    if (lane == r) {
      mine = e;
      *won = best;
    }
  }
  return mine;
}

// -------------------------------------------------------- choice in 64 bits --

// Lane r's choice by keys of 64 bits. A sigmoid is computed again only for those
// of a lane's experts that can matter: those not below `least` (the last of the chosen)
// and, with groups, its best two (which a group's may be); of the others fp32 tells
// enough. Where the groups themselves may be others (`regroup`) their experts can be
// far below `least`: the groups are chosen by the lanes' best two, and behind that
// the experts not below the last that those have. One token of this is some 8 us, beside
// the CTA's other warps. (All scores of a token at once: 32768 tokens of 256 experts in
// groups, with the gradient, 79 -> 83 us, for CTAs end with one.)
template <int V, class T>
__device__ __noinline__ int choose_wide(const P &p, long long t, float least, float err, bool regroup) {
  const int lane = threadIdx.x & 31;
  unsigned long long key[V];
  // Keys of groups that are not chosen are 0 behind this.
  auto keep_groups = [&] {
    if (p.groups <= 1) return;
    if (p.lanes_hold_groups) {  // as choose()
      unsigned long long b1 = 0, b2 = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) merge_best(b1, b2, key[i], 0ull);
      for (int d = p.group_lanes / 2; d > 0; d >>= 1) {
        const unsigned long long o1 = __shfl_xor_sync(kFull, b1, d);
        const unsigned long long o2 = __shfl_xor_sync(kFull, b2, d);
        merge_best(b1, b2, o1, o2);
      }
      const int first = lane & ~(p.group_lanes - 1);
      const unsigned kept =
          choose_lanes(lane == first ? group_key(b1, b2, p.group_best) : 0ull, p.top_groups);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!(kept >> first & 1u)) key[i] = 0;
    } else {
      unsigned long long mine = 0;
      for (int g = 0; g < p.groups; ++g) {
        unsigned long long b1 = 0, b2 = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if ((lane * V + i) / p.per_group == g) merge_best(b1, b2, key[i], 0ull);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          const unsigned long long o1 = __shfl_xor_sync(kFull, b1, d);
          const unsigned long long o2 = __shfl_xor_sync(kFull, b2, d);
          merge_best(b1, b2, o1, o2);
        }
        if (lane == g) mine = group_key(b1, b2, p.group_best);
      }
      const unsigned kept = choose_lanes(mine, p.top_groups);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int g = (lane * V + i) / p.per_group;
        if (g > 31 || !(kept >> g & 1u)) key[i] = 0;
      }
    }
  };
  if (p.sigmoid) {
    float f[V];
    unsigned done[(V + 31) / 32] = {};  // of a lane's experts, by their places
    float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      const float x = e < p.E ? load_logit<T>(p, t, e) : -INFINITY;
      const float b = e < p.E ? load_bias(p, e) : 0.0f;
      const bool there = x != -INFINITY && b != -INFINITY;
      f[i] = there ? sigmoid(x) + b : -INFINITY;
      key[i] = there ? key_of(static_cast<double>(f[i])) : 0;
      const float v = f[i] != f[i] ? -INFINITY : f[i];  // (a NaN is behind all others)
      b2 = fmaxf(b2, fminf(b1, v));
      b1 = fmaxf(b1, v);
    }
    auto refine = [&](float from) {
      const float low = from - 4.0f * (err + kUnit * fabsf(from));
#pragma unroll
      for (int i0 = 0; i0 < V; i0 += 32) {
        unsigned again = 0;
#pragma unroll
        for (int i = i0; i < V && i < i0 + 32; ++i)
          if (key[i] > 1 && !(f[i] < low)) again |= 1u << (i - i0);
        again &= ~done[i0 / 32];
        done[i0 / 32] |= again;
        while (__any_sync(kFull, again != 0)) {
          const int at = __ffs(again) - 1;
          unsigned long long wide = 0;
          if (at >= 0) {
            const int e = lane * V + i0 + at;
            wide = key_of(sigmoid(static_cast<double>(load_logit<T>(p, t, e))) +
                          static_cast<double>(load_bias(p, e)));
            again &= again - 1;
          }
#pragma unroll
          for (int i = i0; i < V && i < i0 + 32; ++i)
            if (at == i - i0) key[i] = wide;
        }
      }
    };
    // (A lane of experts of several groups: all of them. Many experts a lane, too,
    // for want of registers.)
    constexpr bool kTwice = V <= 8;
    if (p.groups > 1 && (p.per_group % V != 0 || (regroup && !kTwice))) refine(-INFINITY);
    else refine(p.groups == 1 ? least : (regroup ? b2 : fminf(least, b2)));
    keep_groups();
    if (kTwice && regroup) {
      unsigned narrow[V], won32;
#pragma unroll
      for (int i = 0; i < V; ++i) narrow[i] = key[i] > 1 ? key_of(f[i]) : static_cast<unsigned>(key[i]);
      choose_experts<V>(narrow, p.k, &won32);
      won32 = __shfl_sync(kFull, won32, p.k - 1);
      refine(won32 > 1 ? value_of(won32) : -INFINITY);
    }
  } else {
    double f[V], m = -INFINITY, sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      f[i] = e < p.E ? static_cast<double>(load_logit<T>(p, t, e)) : -INFINITY;
      key[i] = f[i] == -INFINITY ? 0 : 2;
      m = fmax(m, f[i]);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, s));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f[i] = key[i] != 0 ? exp(f[i] - m) : 0.0;
      sum += f[i];
    }
    const double part = 1.0 / warp_sum(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f[i] *= part;
      if (key[i] != 0 && p.bias != nullptr) {
        const float b = load_bias(p, lane * V + i);
        if (b == -INFINITY) key[i] = 0;
        f[i] += static_cast<double>(b);
      }
      if (key[i] != 0) key[i] = key_of(f[i]);
    }
    keep_groups();
  }
  unsigned long long won;
  return choose_experts<V>(key, p.k, &won);
}

// ------------------------------------------------------------------- router --

// The bound of a score's error in a comparison, in units of 2^-24 of the largest
// score. ex2.approx is off by 2^-22, its argument by 2^-24 |x|, which times
// exp(-|x|), or for a sigmoid s (1 - s), stays below 5 units (1.3); rcp.approx by
// two; the sum by as many roundings as it has steps, and its terms.
template <int V>
__device__ __forceinline__ float score_error(const P &p, float sum) {
  return p.sigmoid ? 10.0f * kUnit : (V + 24.0f) * kUnit * (sum > 0.0f ? 1.0f / sum : 0.0f);
}

__device__ __forceinline__ float fast_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float fast_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Descending, by Batcher's odd-even merge.
template <int V>
__device__ __forceinline__ void sort_keys(unsigned (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int j = d % p; j + d < V; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d; ++i)
          if (i + j + d < V && (i + j) / (2 * p) == (i + j + d) / (2 * p)) {
            const unsigned a = k[i + j], b = k[i + j + d];
            k[i + j] = a > b ? a : b;
            k[i + j + d] = a > b ? b : a;
          }
}

struct Choice {
  int expert;     // lane r: of slot r (-1: none)
  unsigned won;   // lane r: its key
  unsigned next;  // the largest key left
};

// The k best of up to 8 keys a lane: heads sorted, the lowest bits of each V - 1
// less the expert's place in the lane. Keys come back without those bits.
template <int V>
__device__ __forceinline__ Choice choose_sorted(unsigned (&head)[V], int k, int *slots) {
  const int lane = threadIdx.x & 31;
  const unsigned before = (1u << lane) - 1u;
  Choice c = {-1, 0u, 0u};
  int r = 0;
  for (; r < k; ++r) {
    const unsigned mine = head[0] & ~(V - 1u), best = warp_best(mine);
    if (best == 0) break;
    const unsigned equal = __ballot_sync(kFull, mine == best);
    const bool first = mine == best && (equal & before) == 0;
    if (first) slots[r] = lane * V + (V - 1) - static_cast<int>(head[0] & (V - 1u));
#pragma unroll
    for (int i = 0; i < V; ++i) head[i] = first ? (i + 1 < V ? head[i + 1] : 0u) : head[i];
    c.won = lane == r ? best : c.won;
  }
  c.next = warp_best(head[0] & ~(V - 1u));
  __syncwarp();
  if (lane < r) c.expert = slots[lane];
  __syncwarp();
  return c;
}

// The same of many, looked through in every round.
template <int V>
__device__ __forceinline__ Choice choose_any(unsigned (&key)[V], int k) {
  Choice c;
  c.expert = choose_experts<V>(key, k, &c.won);
  unsigned local = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) local = key[i] > local ? key[i] : local;
  c.next = warp_best(local);
  return c;
}

// Lane r: the expert of slot r (-1: none). *m, *sum: softmax's, where it is
// needed; *bad: softmax of a NaN or of +infinity. `staged`: E integers and 32 of
// the warp's own.
template <int V, class T>
__device__ __forceinline__ int choose(const P &p, long long t, const float (&bias)[V], unsigned *staged,
                                      float *m_out, float *sum_out, bool *bad_out) {
  constexpr int kVec = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  float x[V];
  if (V % kVec == 0 && p.vec) {
#pragma unroll
    for (int i = 0; i < V; i += kVec) {
      const int e = lane * V + i;  // E is a multiple of kVec here
      uint4 w = make_uint4(0, 0, 0, 0);
      const long long at = t * p.ldx + e;
      if (e < p.E && index_ok(kSiteLoadA, at, kVec, p.x_extent))
        w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.logits) + at));
      const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float v = sizeof(T) == 4 ? __uint_as_float(u[j * sizeof(T) / 4])
                                       : __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u
                                                               : u[j / 2] << 16);
        x[i + j] = e < p.E ? v : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      x[i] = e < p.E ? load_logit<T>(p, t, e) : -INFINITY;
    }
  }
  float m = -INFINITY, sum = 0.0f;
  bool bad = false;
  const bool stats = !p.sigmoid && (p.compare_scores || !p.renormalise);
  if (!p.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) bad |= !(x[i] < INFINITY);
    bad = __any_sync(kFull, bad);
  }
  if (stats) {
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (x[i] > -INFINITY) sum += expf(x[i] - m);
    sum = warp_sum(sum);
  }
  *m_out = m;
  *sum_out = sum;
  *bad_out = bad;

  unsigned key[V];
  const float part = p.sigmoid ? 0.0f : (bad ? NAN : fast_inverse(sum));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f = x[i];
    if (p.compare_scores) {
      f = p.sigmoid ? fast_inverse(1.0f + fast_exp(-f)) : fast_exp(f - m) * part;
      f += bias[i];
    }
    // a logit or a bias of -infinity: not available, or past the last expert
    key[i] = x[i] != -INFINITY && bias[i] != -INFINITY ? key_of(f) : 0u;
  }
  const float err = score_error<V>(p, sum);
  bool unsure = false;

  constexpr bool kSort = V <= 8;
  [[maybe_unused]] unsigned head[V] = {};
  auto sort = [&] {
#pragma unroll
    for (int i = 0; i < V; ++i) head[i] = key[i] == 0 ? 0u : (key[i] & ~(V - 1u)) | (V - 1 - i);
    sort_keys<V>(head);
  };
  if constexpr (kSort) sort();
  if (p.groups > 1) {
    // The best two of each group, by group_lanes lanes.
    const int g = lane >> p.group_shift, sub = lane & (p.group_lanes - 1);
    unsigned b1 = 0, b2 = 0;
    if (kSort && p.lanes_hold_groups) {
#pragma unroll
      for (int i = 0; i < V; ++i) merge_best(b1, b2, key[i], 0u);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane * V + i < p.E) staged[lane * V + i] = key[i];
      __syncwarp();
      if (g < p.groups)
        for (int j = sub; j < p.per_group; j += p.group_lanes)
          merge_best(b1, b2, staged[g * p.per_group + j], 0u);
    }
    for (int s = p.group_lanes / 2; s > 0; s >>= 1) {
      const unsigned o1 = __shfl_xor_sync(kFull, b1, s), o2 = __shfl_xor_sync(kFull, b2, s);
      merge_best(b1, b2, o1, o2);
    }
    __syncwarp();
    const unsigned mine = sub == 0 ? group_key(b1, b2, p.group_best) : 0u;
    const unsigned kept = choose_lanes(mine, p.top_groups);
    if (p.compare_scores) {
      // the lowest chosen group against each that is not
      const bool in = kept >> lane & 1u;
      float off = 0.0f;  // what this group's sum may be off by
      if (mine > 1)
        off = 2.0f * err + kUnit * (fabsf(value_of(b1)) + (b2 > 1 ? fabsf(value_of(b2)) : 0.0f) +
                                    fabsf(value_of(mine)));
      const unsigned low = __reduce_min_sync(kFull, in ? mine : kFull);
      const float off_in = __uint_as_float(
          __reduce_max_sync(kFull, in ? __float_as_uint(off) : 0u));
      if (!in && mine > 1 && low > 1 && low != kFull)
        unsure = value_of(low) - value_of(mine) <= off + off_in;
    }
    if (kSort && p.lanes_hold_groups) {
      if (!(kept >> (g * p.group_lanes) & 1u)) {
#pragma unroll
        for (int i = 0; i < V; ++i) head[i] = key[i] = 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int of = (lane * V + i) / p.per_group;
        if (of >= p.groups || !(kept >> (of * p.group_lanes) & 1u)) key[i] = 0;
      }
      if constexpr (kSort) sort();
    }
  }

  int *slots = reinterpret_cast<int *>(staged + staged_ints(p) - kMaxSlots);
  Choice c;
  if constexpr (kSort) c = choose_sorted<V>(head, p.k, slots);
  else c = choose_any<V>(key, p.k);
  const unsigned next = __shfl_down_sync(kFull, c.won, 1);
  const unsigned last = __shfl_sync(kFull, c.won, p.k - 1);
  // Neighbours of the chosen that may stand the other way round, and the last of
  // them and what is left: closer than the error, or equal but for the bits that
  // the sort left out (`cut`), which bring the smaller key up to as many steps of
  // fp32 closer. (A NaN's key, 1, loses to those bits: whole keys again.)
  auto close = [&](unsigned a, unsigned b, unsigned cut) {
    if (a == b) return true;
    if (!p.compare_scores || b <= 8) return false;
    const float u = value_of(a), v = value_of(b | cut);
    return u - v <= 2.0f * err + kUnit * (fabsf(u) + fabsf(v));
  };
  bool look = false;
  if (sizeof(T) == 4 || p.compare_scores) {  // (bf16 logits have nothing in those bits)
    constexpr unsigned kCut = kSort ? V - 1u : 0u;
    look = lane + 1 < p.k && next != 0 && close(c.won, next, kCut);
    look |= lane == p.k - 1 && last != 0 && c.next != 0 && close(last, c.next, kCut);
  }
  if (kSort) {
#pragma unroll
    for (int i = 0; i < V; ++i) look |= key[i] == 1u;
  }
  if (!__any_sync(kFull, look | unsure)) return c.expert;

  // By whole keys, and whether equal ones are of equal logits and biases.
  const bool regroup = __any_sync(kFull, unsure);
  float least = INFINITY;
  if constexpr (kSort) c = choose_any<V>(key, p.k);
  if (p.compare_scores) {
    auto same = [&](int a, int b) {
      return load_logit<T>(p, t, a) == load_logit<T>(p, t, b) &&
             load_bias(p, a) == load_bias(p, b);
    };
    const unsigned next_key = __shfl_down_sync(kFull, c.won, 1);
    const int next_e = __shfl_down_sync(kFull, c.expert, 1);
    if (lane + 1 < p.k && next_key > 1 && close(c.won, next_key, 0u)) unsure |= !same(c.expert, next_e);
    const unsigned last_key = __shfl_sync(kFull, c.won, p.k - 1);
    const int last_e = __shfl_sync(kFull, c.expert, p.k - 1);
    if (last_key > 1) {
      least = value_of(last_key);
#pragma unroll
      for (int i = 0; i < V; ++i)  // those that are left
        if (key[i] > 1 && close(last_key, key[i], 0u)) unsure |= !same(last_e, lane * V + i);
    }
    if (__any_sync(kFull, unsure))
      return choose_wide<V, T>(p, t, least == INFINITY ? -INFINITY : least, err, regroup);
  }
  return c.expert;
}

// Lane r: the weight of its expert.
template <class T>
__device__ __forceinline__ float weight_of(const P &p, long long t, int e, float m, float sum,
                                           bool bad) {
  const bool there = e >= 0;
  const float x = there ? load_logit<T>(p, t, e) : -INFINITY;
  float w;
  if (!p.renormalise) {
    w = p.sigmoid ? sigmoid(x) : expf(x - m) / sum;
  } else {
    // Scores relative to the largest one's, so that they may all be tiny.
    float top = warp_max(x);
    float part;
    if (p.sigmoid) {
      top = fminf(top, 0.0f);
      part = (x < 0.0f ? expf(x - top) : 1.0f) / (1.0f + expf(-fabsf(x)));
    } else {
      part = expf(x - top);
    }
    if (!there) part = 0.0f;
    w = part / warp_sum(part);
  }
  if (bad) w = NAN;
  return there ? w * p.scale : 0.0f;
}

// -------------------------------------------------------------------- plan --

// start[e] = sum of count[< e], and the sum of all in start[E], by one warp.
__device__ __forceinline__ void scan_experts(const int *count, int *start, int E) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane, v = e < E ? count[e] : 0;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, s, d);
      if (lane >= d) s += o;
    }
    if (e < E) start[e] = carry + s - v;
    carry += __shfl_sync(kFull, s, 31);
  }
  if (lane == 0) start[E] = carry;
}

struct PlanShared {
  int *count;  // E: the chunk's, or all slots', counts
  int *start;  // E + 1: first row of each expert
  int *base;   // E: first row of each expert's slots of this chunk
  int *warp;   // plan_warps x E
};

__device__ __forceinline__ PlanShared plan_shared(int *smem, int E) {
  return PlanShared{smem, smem + E, smem + 2 * E + 1, smem + 3 * E + 1};
}
__host__ __device__ constexpr int plan_ints(int E, int warps) { return (3 + warps) * E + 1; }

__device__ __forceinline__ int read_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// Rows of slots [s0, s1), whose experts' first rows are in sh.base. All threads.
__device__ void rank_slots(const P &p, const PlanShared &sh, int s0, int s1, long long slots) {
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31, E = p.E;
  for (int i = threadIdx.x; i < p.plan_warps * E; i += blockDim.x) sh.warp[i] = 0;
  __syncthreads();
  const int each = ((s1 - s0 + p.plan_warps - 1) / p.plan_warps + 31) / 32 * 32;
  const long long from = s0 + static_cast<long long>(warp) * each;
  const long long to = from + each < s1 ? from + each : s1;
  const bool works = warp < p.plan_warps;
  int *count = sh.warp + (works ? warp : 0) * E;
  auto expert_of = [&](long long s) {
    const int e = index_ok(kSiteLoadB, s, 1, slots) ? p.experts[s] : -1;
    return e >= 0 && e < E ? e : -1;
  };
  if (works)
    for (long long s = from + lane; s < to; s += 32) {
      const int e = expert_of(s);
      if (e >= 0) atomicAdd(&count[e], 1);
    }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int at = sh.base[e];
    for (int w = 0; w < p.plan_warps; ++w) {
      const int n = sh.warp[w * E + e];
      sh.warp[w * E + e] = at;
      at += n;
    }
  }
  __syncthreads();
  if (works)
    for (long long s0w = from; s0w < to; s0w += 32) {
      const long long s = s0w + lane;
      const int e = s < to ? expert_of(s) : -2;
      const unsigned same = __match_any_sync(kFull, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      if (e >= 0) {
        const int row = count[e] + rank;
        if (index_ok(kSiteCStore, row, 1, slots)) p.order[row] = static_cast<int>(s);
        if (index_ok(kSiteCStore, s, 1, slots)) p.places[s] = row;
      } else if (e == -1 && index_ok(kSiteCStore, s, 1, slots)) {
        p.places[s] = -1;
      }
      __syncwarp();
      if (e >= 0 && rank == 0) count[e] += __popc(same);
      __syncwarp();
    }
}

// Chunk c of the plan: counts of all chunks are in p.hist, or (one chunk) this
// CTA's own in sh.count.
__device__ void plan_chunk(const P &p, const PlanShared &sh, int c, long long slots) {
  const int E = p.E, tid = threadIdx.x;
  if (p.chunks > 1 && p.hist == nullptr) {  // the cluster's
    cluster_sync();
    for (int e = tid; e < E; e += blockDim.x) {
      int before = 0, all = 0;
      for (int j = 0; j < p.chunks; ++j) {
        const int n = read_cluster(smem_addr(sh.count + e), static_cast<unsigned>(j));
        all += n;
        before += j < c ? n : 0;
      }
      sh.base[e] = before;
      sh.warp[e] = all;
    }
    cluster_sync();  // all counts are read
    for (int e = tid; e < E; e += blockDim.x) sh.count[e] = sh.warp[e];
  } else if (p.chunks > 1) {
    for (int e = tid; e < E; e += blockDim.x) sh.count[e] = sh.base[e] = 0;
    __syncthreads();
    // several threads an expert, each over a part of the chunks
    int parts = static_cast<int>(blockDim.x) / E;
    parts = parts < 1 ? 1 : (parts > p.chunks ? p.chunks : parts);
    const int each = (p.chunks + parts - 1) / parts;
    for (int i = tid; i < E * parts; i += blockDim.x) {
      const int e = i % E, c0 = i / E * each, c1 = min(c0 + each, p.chunks);
      int before = 0, all = 0;
#pragma unroll 8
      for (int j = c0; j < c1; ++j) {
        const long long at = static_cast<long long>(j) * E + e;
        const int n = index_ok(kSitePartialRead, at, 1, static_cast<long long>(p.chunks) * E)
                          ? __ldcg(p.hist + at) : 0;
        all += n;
        before += j < c ? n : 0;
      }
      if (all != 0) atomicAdd(&sh.count[e], all);
      if (before != 0) atomicAdd(&sh.base[e], before);
    }
  }
  __syncthreads();
  if (tid < 32) scan_experts(sh.count, sh.start, E);
  __syncthreads();
  for (int e = tid; e <= E; e += blockDim.x) {
    if (e < E) sh.base[e] = sh.start[e] + (p.chunks > 1 ? sh.base[e] : 0);
    if (c == 0 && index_ok(kSiteCStore, e, 1, E + 1)) p.offsets[e] = sh.start[e];
  }
  // rows of no slot
  const long long used = sh.start[E];
  for (long long r = used + static_cast<long long>(c) * blockDim.x + tid; r < slots;
       r += static_cast<long long>(p.chunks) * blockDim.x)
    if (index_ok(kSiteCStore, r, 1, slots)) p.order[r] = -1;
  const long long s0 = static_cast<long long>(c) * p.chunk * p.k;
  const long long s1 = s0 + static_cast<long long>(p.chunk) * p.k;
  rank_slots(p, sh, static_cast<int>(s0), static_cast<int>(s1 < slots ? s1 : slots), slots);
}

// As many warps as registers leave room for without spills that count: the choice of
// 32768 tokens, 8 slots, by a sigmoid with a bias in groups (softmax), 256 experts (V =
// 8): 768 threads 56 us (34), 512 70 (46), 384 82 (53); 64 experts: 1024 37 (23), 768 37
// (22), 512 55 (36); 512 experts: 512 (72), 384 (84).
constexpr int route_threads(int V) { return V <= 4 ? 1024 : (V == 8 ? 768 : (V == 16 ? 512 : 256)); }

template <int V, class T>
__global__ void __launch_bounds__(route_threads(V)) route_kernel(const P p) {
  extern __shared__ int smem[];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int warps = static_cast<int>(blockDim.x >> 5);
  const PlanShared sh = plan_shared(smem, p.E);
  // groups' keys stand where the plan's counts of a warp will
  unsigned *staged = reinterpret_cast<unsigned *>(p.plan ? sh.base : smem) + warp * staged_ints(p);
  const long long slots = static_cast<long long>(p.T) * p.k;
  __shared__ int taken;  // tokens of the chunk, behind the warps' first
  if (threadIdx.x == 0) taken = warps;
  if (p.plan)
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) sh.count[e] = 0;
  __syncthreads();
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    bias[i] = lane * V + i < p.E ? load_bias(p, lane * V + i) : 0.0f;
  // A warp takes the next token when it is done with one: masked ones take no time, and
  // those of choose_wide much.
  const long long t0 = static_cast<long long>(blockIdx.x) * p.chunk;
  const int count = static_cast<int>(min(static_cast<long long>(p.T) - t0, static_cast<long long>(p.chunk)));
  for (int i = warp; i < count;) {
    const long long t = t0 + i;
    if (lane == 0) i = atomicAdd(&taken, 1);
    int e = -1;
    float w = 0.0f;
    if (p.mask == nullptr || (index_ok(kSiteLoadB, t, 1, p.T) && p.mask[t] != 0)) {
      float m, sum;
      bool bad;
      e = choose<V, T>(p, t, bias, staged, &m, &sum, &bad);
      w = weight_of<T>(p, t, e, m, sum, bad);
    }
    if (lane < p.k) {
      const long long s = t * p.k + lane;
      if (index_ok(kSiteCStore, s, 1, slots)) {
        p.experts[s] = e;
        p.weights[s] = w;
      }
      if (p.plan && e >= 0) atomicAdd(&sh.count[e], 1);
    }
    i = __shfl_sync(kFull, i, 0);
  }
  if (!p.plan) return;
  __syncthreads();
  if (p.hist != nullptr) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      const long long at = static_cast<long long>(blockIdx.x) * p.E + e;
      if (index_ok(kSitePartialWrite, at, 1, static_cast<long long>(p.chunks) * p.E))
        p.hist[at] = sh.count[e];
    }
  } else {
    plan_chunk(p, sh, blockIdx.x, slots);  // reads the experts behind the barrier above
  }
}

// The plan of 32768 tokens of 256 experts, 8 slots: 16 us, with 512 threads 21, 256 34;
// 8192 of 1024: 29, 51, 65; 500 of 256: 7.5, 7.4, 8.7.
constexpr int kPlanThreads = 1024;

// Counts of a chunk of given experts.
__global__ void __launch_bounds__(kPlanThreads) count_kernel(const P p) {
  extern __shared__ int smem[];
  grid_dependency_wait();
  grid_launch_dependents();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) smem[e] = 0;
  __syncthreads();
  const long long slots = static_cast<long long>(p.T) * p.k;
  const long long s0 = static_cast<long long>(blockIdx.x) * p.chunk * p.k;
  const long long s1 = min(slots, s0 + static_cast<long long>(p.chunk) * p.k);
  for (long long s = s0 + threadIdx.x; s < s1; s += blockDim.x) {
    const int e = index_ok(kSiteLoadB, s, 1, slots) ? p.experts[s] : -1;
    if (e >= 0 && e < p.E) atomicAdd(&smem[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    const long long at = static_cast<long long>(blockIdx.x) * p.E + e;
    if (index_ok(kSitePartialWrite, at, 1, static_cast<long long>(p.chunks) * p.E))
      p.hist[at] = smem[e];
  }
}

// The plan of a chunk; one chunk: its counts too.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const P p) {
  extern __shared__ int smem[];
  grid_dependency_wait();
  grid_launch_dependents();
  const PlanShared sh = plan_shared(smem, p.E);
  const long long slots = static_cast<long long>(p.T) * p.k;
  if (p.chunks == 1) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) sh.count[e] = 0;
    __syncthreads();
    for (long long s = threadIdx.x; s < slots; s += blockDim.x) {
      const int e = index_ok(kSiteLoadB, s, 1, slots) ? p.experts[s] : -1;
      if (e >= 0 && e < p.E) atomicAdd(&sh.count[e], 1);
    }
  }
  plan_chunk(p, sh, static_cast<int>(blockIdx.x), slots);
}

// ---------------------------------------------------------------- gradient --

struct B {
  const float *dweights, *weights;
  const void *logits;
  const int32_t *experts;
  void *dlogits;
  long long ldx, x_extent, lddx, dx_extent;
  int T, E, k, sigmoid, renormalise, vec;
  float inv_scale;
};

constexpr int kBackThreads = 256;

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// A warp takes a token: its row goes out without the slots' terms (zero, or what
// softmax's sum gives to all experts), and behind that the slots' experts.
template <class T>
__global__ void __launch_bounds__(kBackThreads) route_backward_kernel(const B p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31, E = p.E;
  const T *x = static_cast<const T *>(p.logits);
  T *dx = static_cast<T *>(p.dlogits);
  const long long slots = static_cast<long long>(p.T) * p.k;
  const long long warps = static_cast<long long>(gridDim.x) * (kBackThreads / 32);
  constexpr int kVec = 16 / sizeof(T);
  for (long long t = static_cast<long long>(blockIdx.x) * (kBackThreads / 32) + warp; t < p.T;
       t += warps) {
    const long long at = t * p.ldx, s = t * p.k + lane, out = t * p.lddx;
    auto logit = [&](int j) {
      return index_ok(kSiteLoadA, at + j, 1, p.x_extent) ? as_float(x[at + j]) : 0.0f;
    };
    int e = -1;
    float w = 0.0f, g = 0.0f;
    if (lane < p.k && index_ok(kSiteLoadB, s, 1, slots)) {
      e = p.experts[s];
      w = p.weights[s];
      g = p.dweights[s];
    }
    if (e < 0 || e >= E) e = -1;
    const bool there = e >= 0;
    const float l = there && (p.sigmoid || !p.renormalise) ? logit(e) : 0.0f;
    const float total = warp_sum(there ? g * w : 0.0f);
    float d = p.renormalise ? w * (g - total * p.inv_scale) : w * g;
    if (p.sigmoid) d *= sigmoid(-l);
    // of an expert that stands in several slots, the sum by its first
    unsigned same = 0;
    for (int r = 0; r < p.k; ++r)
      if (__shfl_sync(kFull, e, r) == e) same |= 1u << r;
    if (!there) same = 0;
    bool writes = there;
    if (__any_sync(kFull, __popc(same) > 1)) {
      float both = 0.0f;
      for (int r = 0; r < p.k; ++r) {
        const float v = __shfl_sync(kFull, d, r);
        if (same >> r & 1u) both += v;
      }
      d = both;
      writes = there && __ffs(same) - 1 == lane;
    }
    if (!p.sigmoid && !p.renormalise && __any_sync(kFull, there)) {
      float m = -INFINITY;
      for (int j = lane; j < E; j += 32) m = fmaxf(m, logit(j));
      m = warp_max(m);
      float sum = 0.0f;
      for (int j = lane; j < E; j += 32) {
        const float v = logit(j);
        sum += v != -INFINITY ? expf(v - m) : 0.0f;
      }
      const float factor = total / warp_sum(sum);
      auto share = [&](float v) { return v != -INFINITY ? -expf(v - m) * factor : 0.0f; };
      d += share(l);
      for (int j = lane; j < E; j += 32)
        if (index_ok(kSiteCStore, out + j, 1, p.dx_extent)) dx[out + j] = from_float<T>(share(logit(j)));
    } else if (p.vec) {  // E is a multiple of kVec
      for (int j = lane * kVec; j < E; j += 32 * kVec)
        if (index_ok(kSiteCStore, out + j, kVec, p.dx_extent))
          *reinterpret_cast<uint4 *>(dx + out + j) = make_uint4(0, 0, 0, 0);
    } else {
      for (int j = lane; j < E; j += 32)
        if (index_ok(kSiteCStore, out + j, 1, p.dx_extent)) dx[out + j] = from_float<T>(0.0f);
    }
    __syncwarp();
    if (writes && index_ok(kSiteCStore, out + e, 1, p.dx_extent)) dx[out + e] = from_float<T>(d);
  }
}

// -------------------------------------------------------------------- host --

template <class K, class A>
int launch(K kernel, const A &p, unsigned grid, int threads, size_t smem, cudaStream_t stream,
           unsigned cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  // Above the 48 KiB default: set on the current device, which keeps it (every
  // call, where it is needed; it takes no launch).
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return kErrLaunch;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? kOk : kErrLaunch;
}

// Warps of a CTA that rank slots: as many as have room for their counts.
int plan_warps_of(int64_t E, int warps) {
  const int64_t room = (46 * 1024 / 4 - 1) / E - 3;
  return static_cast<int>(room < warps ? (room < 1 ? 1 : room) : warps);
}

size_t smem_of(const P &p, int threads) {
  const size_t plan = p.plan ? static_cast<size_t>(plan_ints(p.E, p.plan_warps)) * 4 : 0;
  const size_t keys =
      static_cast<size_t>((p.plan ? 2 * p.E + 1 : 0) + threads / 32 * staged_ints(p)) * 4;
  return plan > keys ? plan : keys;
}

template <int V, class T>
int launch_v(P &p, cudaStream_t stream) {
  p.lanes_hold_groups = p.per_group % V == 0 && p.per_group / V == p.group_lanes;
  int threads = route_threads(V);
  const int64_t want = 32LL * p.chunk;
  if (threads > want) threads = static_cast<int>((want + 127) / 128 * 128);
  p.plan_warps = plan_warps_of(p.E, threads / 32 < 16 ? threads / 32 : 16);
  return launch(route_kernel<V, T>, p, static_cast<unsigned>(p.chunks), threads, smem_of(p, threads),
                stream, p.plan && p.hist == nullptr ? static_cast<unsigned>(p.chunks) : 1u);
}

template <class T>
int launch_route(P &p, cudaStream_t stream) {
  if (p.E <= 32) return launch_v<1, T>(p, stream);
  if (p.E <= 64) return launch_v<2, T>(p, stream);
  if (p.E <= 128) return launch_v<4, T>(p, stream);
  if (p.E <= 256) return launch_v<8, T>(p, stream);
  if (p.E <= 512) return launch_v<16, T>(p, stream);
  if (p.E <= 1024) return launch_v<32, T>(p, stream);
  return launch_v<64, T>(p, stream);
}

int launch_plan(P p, cudaStream_t stream) {
  p.plan_warps = plan_warps_of(p.E, kPlanThreads / 32);
  return launch(plan_kernel, p, static_cast<unsigned>(p.chunks), kPlanThreads,
                static_cast<size_t>(plan_ints(p.E, p.plan_warps)) * 4, stream);
}

// Tokens of a CTA: at least `least`, and no more CTAs than SMs.
void cut(P &p, int64_t tokens, int least, int sms) {
  int64_t chunks = (tokens + least - 1) / least;
  if (chunks > sms) chunks = sms;
  if (chunks < 1) chunks = 1;
  const int64_t chunk = (tokens + chunks - 1) / chunks;
  p.chunk = static_cast<int>(chunk);
  p.chunks = static_cast<int>((tokens + chunk - 1) / chunk);
}

}  // namespace

GEMM_INDEX_FAULT_TAKE(route_index_fault_take)

int route_launch(const RouteArgs &a, int sm_count, cudaStream_t stream) {
  P p = {};
  p.logits = a.logits;
  p.ldx = a.ldx;
  p.x_extent = matrix_extent(a.T, a.E, a.ldx);
  p.bias = a.bias;
  p.mask = a.mask;
  p.experts = a.experts;
  p.weights = a.weights;
  p.offsets = a.offsets;
  p.order = a.order;
  p.places = a.places;
  p.T = static_cast<int>(a.T);
  p.E = static_cast<int>(a.E);
  p.k = static_cast<int>(a.k);
  p.sigmoid = a.sigmoid;
  p.renormalise = a.renormalise;
  p.groups = a.groups;
  p.top_groups = a.top_groups;
  p.group_best = a.group_best;
  p.per_group = static_cast<int>(a.E / a.groups);
  p.group_shift = 5;
  while (32 >> p.group_shift < a.groups) --p.group_shift;
  p.group_lanes = 1 << p.group_shift;
  p.compare_scores = a.bias != nullptr || (a.groups > 1 && a.group_best > 1);
  const int elem = a.bf16 ? 2 : 4, per16 = 16 / elem;
  p.vec = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.ldx % per16 == 0 && a.E % per16 == 0;
  p.scale = a.scale;
  p.plan = a.offsets != nullptr;
  // Up to 24 tokens one CTA does all (a warp each); more, eight tokens a CTA: 64
  // tokens of 256 experts, with the plan, 13.4 us (cold), in one CTA 25.7. Up to 192 the CTAs
  // of a cluster, one launch: 64 tokens 13.4 against 16.5 to 18.6 in two launches, 192
  // tokens 17.5 against 18.6, and 256 21.6 against 16.5.
  constexpr int kCluster = 8;
  const bool together = a.T <= 24 * kCluster;
  cut(p, a.T, a.T <= 24 ? 24 : 8, together ? kCluster : sm_count);
  void *ws = nullptr;
  if (p.plan && !together) {
    const int st = pool_alloc(&ws, static_cast<size_t>(p.chunks) * a.E * sizeof(int), stream);
    if (st != kOk) return st;
    p.hist = static_cast<int *>(ws);
  }
  int st = a.bf16 ? launch_route<__nv_bfloat16>(p, stream) : launch_route<float>(p, stream);
  if (ws != nullptr) {
    if (st == kOk) st = launch_plan(p, stream);
    const int fst = pool_free(ws, stream);
    if (st == kOk) st = fst;
  }
  return st;
}

int route_plan_launch(int64_t slots, int64_t E, const int32_t *experts, int64_t *offsets,
                      int32_t *order, int32_t *places, int sm_count, cudaStream_t stream) {
  P p = {};
  p.experts = const_cast<int32_t *>(experts);  // read here
  p.offsets = offsets;
  p.order = order;
  p.places = places;
  p.T = static_cast<int>(slots);
  p.E = static_cast<int>(E);
  p.k = 1;
  p.plan = 1;
  cut(p, slots, 4096, sm_count);
  if (p.chunks == 1) return launch_plan(p, stream);
  void *ws = nullptr;
  int st = pool_alloc(&ws, static_cast<size_t>(p.chunks) * E * sizeof(int), stream);
  if (st != kOk) return st;
  p.hist = static_cast<int *>(ws);
  st = launch(count_kernel, p, static_cast<unsigned>(p.chunks), kPlanThreads,
              static_cast<size_t>(E) * sizeof(int), stream);
  if (st == kOk) st = launch_plan(p, stream);
  const int fst = pool_free(ws, stream);
  return st != kOk ? st : fst;
}

int route_backward_launch(const RouteBackwardArgs &a, int sm_count, cudaStream_t stream) {
  B p = {};
  p.dweights = a.dweights;
  p.weights = a.weights;
  p.logits = a.logits;
  p.experts = a.experts;
  p.dlogits = a.dlogits;
  p.ldx = a.ldx;
  p.x_extent = matrix_extent(a.T, a.E, a.ldx);
  p.lddx = a.lddx;
  p.dx_extent = matrix_extent(a.T, a.E, a.lddx);
  p.T = static_cast<int>(a.T);
  p.E = static_cast<int>(a.E);
  p.k = static_cast<int>(a.k);
  p.sigmoid = a.sigmoid;
  p.renormalise = a.renormalise;
  p.inv_scale = 1.0f / a.scale;
  const int elem = a.bf16 ? 2 : 4, per16 = 16 / elem;
  p.vec = reinterpret_cast<uintptr_t>(a.dlogits) % 16 == 0 && a.lddx % per16 == 0 &&
          a.E % per16 == 0;
  const int64_t blocks = (a.T + kBackThreads / 32 - 1) / (kBackThreads / 32);
  const int64_t most = 8LL * (sm_count > 0 ? sm_count : 1);
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  return a.bf16 ? launch(route_backward_kernel<__nv_bfloat16>, p, grid, kBackThreads, 0, stream)
                : launch(route_backward_kernel<float>, p, grid, kBackThreads, 0, stream);
}

}  // namespace gemm
