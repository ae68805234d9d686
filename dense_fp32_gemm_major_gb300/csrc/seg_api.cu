// seg_api.cu -- the C ABI of the segmented products (declared in
// include/segment_gemm_f32.h): argument validation and kernel launches.

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/segment_gemm_f32.h"
#include "segments.h"

namespace {

using gemm::SegArgs;
using gemm::SegMatrix;

constexpr int64_t kMaxDim = 0x7fffffffLL;       // sizes and pitches < 2^31
constexpr int64_t kMaxSpan = int64_t{1} << 44;  // elements one stack may span

struct Range {
  uintptr_t lo = 0, hi = 0;
};

bool overlap(const Range &a, const Range &b) { return a.lo < b.hi && b.lo < a.hi; }

bool dim_ok(int64_t x) { return x >= 0 && x <= kMaxDim; }

// A stack of matrices the call may touch: its pitch and stride, and (unless it
// is empty) its pointer. `disjoint`: a result, whose matrices must not share
// elements.
bool stack_ok(const SegMatrix &m, int elem, bool disjoint, Range *range) {
  if (m.ld < (m.cols > 1 ? m.cols : 1) || m.ld > kMaxDim || m.stride < 0) return false;
  const int64_t one = gemm::matrix_extent(m.rows, m.cols, m.ld);
  if (one == 0 || m.count == 0) return true;
  if (one > kMaxSpan || (m.count > 1 && m.stride > kMaxSpan / (m.count - 1))) return false;
  const int64_t span = (m.count - 1) * m.stride + one;
  if (span > kMaxSpan) return false;
  if (disjoint && m.count > 1 && m.stride < one) return false;
  const uintptr_t p = reinterpret_cast<uintptr_t>(m.p);
  if (p == 0 || p % static_cast<uintptr_t>(elem) != 0) return false;
  range->lo = p;
  range->hi = p + static_cast<uintptr_t>(span) * elem;
  return true;
}

// `count` values of `elem` bytes at p (null allowed where optional).
bool array_ok(const void *p, int64_t count, int elem, bool optional, Range *range) {
  if (p == nullptr) return optional || count == 0;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (a % static_cast<uintptr_t>(elem) != 0) return false;
  range->lo = a;
  range->hi = a + static_cast<uintptr_t>(count) * elem;
  return true;
}

bool op_ok(int op) { return op == GEMM_OP_N || op == GEMM_OP_T; }

bool common_ok(int type, int64_t groups) {
  return (type == GEMM_F32_TYPE_F32 || type == GEMM_F32_TYPE_BF16) && groups >= 0 &&
         groups <= GEMM_F32_MAX_SEGMENTS;
}

int launch(const SegArgs &a, int sms, cudaStream_t stream) {
  return gemm::seg_simt_launch(a, sms, stream);
}

}  // namespace

extern "C" {

int gemm_f32_grouped(int type, int transb, int64_t groups, int64_t M, int64_t N, int64_t K,
                     const void *A, int64_t lda, const void *B, int64_t ldb, int64_t strideb,
                     void *C, int64_t ldc, const int64_t *offsets, void *stream) {
  if (!common_ok(type, groups) || !op_ok(transb) || !dim_ok(M) || !dim_ok(N) || !dim_ok(K))
    return GEMM_ERR_INVALID_ARG;
  const int elem = type == GEMM_F32_TYPE_BF16 ? 2 : 4;
  SegArgs a;
  a.bf16 = type == GEMM_F32_TYPE_BF16;
  a.groups = a.bank = groups;
  a.M = M;
  a.N = N;
  a.K = K;
  a.transb = transb;
  a.A = SegMatrix{A, lda, 0, M, K, 1};
  a.B = SegMatrix{B, ldb, strideb, transb ? N : K, transb ? K : N, groups};
  a.C = SegMatrix{C, ldc, 0, M, N, 1};
  a.offsets = offsets;
  Range ra, rb, rc, ro;
  if (!stack_ok(a.A, elem, false, &ra) || !stack_ok(a.B, elem, false, &rb) ||
      !stack_ok(a.C, elem, true, &rc) || !array_ok(offsets, groups + 1, 8, groups == 0, &ro))
    return GEMM_ERR_INVALID_ARG;
  if (groups == 0 || M == 0 || N == 0) return GEMM_OK;
  if (overlap(rc, ra) || overlap(rc, rb) || overlap(rc, ro)) return GEMM_ERR_ALIAS;
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  return launch(a, sms, static_cast<cudaStream_t>(stream));
}

int gemm_f32_grouped_wgrad(int type, int64_t groups, int64_t M, int64_t N, int64_t K,
                           const void *A, int64_t lda, const void *D, int64_t ldd, void *C,
                           int64_t ldc, int64_t stridec, const int64_t *offsets, void *stream) {
  if (!common_ok(type, groups) || !dim_ok(M) || !dim_ok(N) || !dim_ok(K))
    return GEMM_ERR_INVALID_ARG;
  const int elem = type == GEMM_F32_TYPE_BF16 ? 2 : 4;
  SegArgs a;
  a.bf16 = type == GEMM_F32_TYPE_BF16;
  a.wgrad = true;
  a.groups = groups;
  a.M = M;
  a.N = N;
  a.K = K;
  a.A = SegMatrix{A, lda, 0, M, K, 1};
  a.B = SegMatrix{D, ldd, 0, M, N, 1};
  a.C = SegMatrix{C, ldc, stridec, K, N, groups};
  a.offsets = offsets;
  Range ra, rd, rc, ro;
  if (!stack_ok(a.A, elem, false, &ra) || !stack_ok(a.B, elem, false, &rd) ||
      !stack_ok(a.C, elem, true, &rc) || !array_ok(offsets, groups + 1, 8, groups == 0, &ro))
    return GEMM_ERR_INVALID_ARG;
  if (groups == 0 || N == 0 || K == 0) return GEMM_OK;
  if (overlap(rc, ra) || overlap(rc, rd) || overlap(rc, ro)) return GEMM_ERR_ALIAS;
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  return launch(a, sms, static_cast<cudaStream_t>(stream));
}

int gemm_f32_lora(int type, int transw, int transl, int64_t segments, int64_t bank, int64_t M,
                  int64_t N, int64_t K, int64_t R, const void *X, int64_t ldx, const void *W,
                  int64_t ldw, const void *A, int64_t lda, int64_t stridea, const void *B,
                  int64_t ldb, int64_t strideb, const int64_t *offsets, const int32_t *index,
                  const float *scales, void *U, int64_t ldu, void *Y, int64_t ldy, void *stream) {
  if (!common_ok(type, segments) || !op_ok(transw) || !op_ok(transl) || !dim_ok(M) || !dim_ok(N) ||
      !dim_ok(K) || !dim_ok(R) || !dim_ok(bank))
    return GEMM_ERR_INVALID_ARG;
  const int elem = type == GEMM_F32_TYPE_BF16 ? 2 : 4;
  const bool adapted = R > 0 && bank > 0 && segments > 0 && M > 0;
  SegArgs y;
  y.bf16 = type == GEMM_F32_TYPE_BF16;
  y.dense = true;
  y.groups = adapted ? segments : 0;
  y.bank = bank;
  y.M = M;
  y.N = N;
  y.K = K;
  y.R = adapted ? R : 0;
  y.transb = transw;
  y.transl = transl;
  y.A = SegMatrix{X, ldx, 0, M, K, 1};
  y.B = SegMatrix{W, ldw, 0, transw ? N : K, transw ? K : N, 1};
  y.C = SegMatrix{Y, ldy, 0, M, N, 1};
  y.L = SegMatrix{B, ldb, strideb, transl ? N : R, transl ? R : N, bank};
  y.offsets = offsets;
  y.index = index;
  SegArgs u = y;  // U = s (X A)
  u.dense = false;
  u.N = R;
  u.R = 0;
  u.transb = transl;
  u.scales = scales;
  u.B = SegMatrix{A, lda, stridea, transl ? R : K, transl ? K : R, bank};
  u.C = SegMatrix{U, ldu, 0, M, R, 1};
  Range rx, rw, ra, rb, ro, ri, rs, ru, ry;
  if (!stack_ok(y.A, elem, false, &rx) || !stack_ok(y.B, elem, false, &rw) ||
      !stack_ok(y.C, elem, true, &ry))
    return GEMM_ERR_INVALID_ARG;
  if (adapted &&
      (!stack_ok(u.B, elem, false, &ra) || !stack_ok(y.L, elem, false, &rb) ||
       !array_ok(offsets, segments + 1, 8, false, &ro) ||
       !array_ok(index, segments, 4, true, &ri) || !array_ok(scales, bank, 4, true, &rs) ||
       (U != nullptr && !stack_ok(u.C, elem, true, &ru))))
    return GEMM_ERR_INVALID_ARG;
  const Range in[] = {rx, rw, ra, rb, ro, ri, rs};
  for (const Range &r : in)
    if (overlap(r, ry) || overlap(r, ru)) return GEMM_ERR_ALIAS;
  if (overlap(ru, ry)) return GEMM_ERR_ALIAS;
  if (M == 0 || (N == 0 && (!adapted || U == nullptr))) return GEMM_OK;
  int dev = 0, sms = 0;
  int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void *work = nullptr;
  if (adapted) {
    if (U == nullptr) {
      u.C.ld = (R + 7) / 8 * 8;
      st = gemm::pool_alloc(&work, static_cast<size_t>(M) * u.C.ld * elem, s);
      if (st != gemm::kOk) return st;
      u.C.p = work;
    }
    y.U = u.C;
    st = launch(u, sms, s);
  }
  if (st == gemm::kOk && N > 0) st = launch(y, sms, s);
  if (work != nullptr) {
    const int fst = gemm::pool_free(work, s);
    if (st == gemm::kOk) st = fst;
  }
  return st;
}

}  // extern "C"
