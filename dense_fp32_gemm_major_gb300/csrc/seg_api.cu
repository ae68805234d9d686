// seg_api.cu -- the C ABI of the segmented products (declared in
// include/segment_gemm_f32.h): argument validation and kernel launches.

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/segment_gemm_f32.h"
#include "segments.h"

namespace {

using gemm::SegArgs;
using gemm::SegMatrix;

constexpr int64_t kMaxPitch = 0x7fffffffLL;     // pitches and banks < 2^31
constexpr int64_t kMaxSpan = int64_t{1} << 44;  // elements one stack may span

struct Range {
  uintptr_t lo = 0, hi = 0;
};

bool overlap(const Range &a, const Range &b) { return a.lo < b.hi && b.lo < a.hi; }

bool dim_ok(int64_t x) { return x >= 0 && x <= GEMM_F32_MAX_SEGMENT_SIZE; }

// A stack of matrices the call may touch: its pitch and stride, and (unless it
// is empty) its pointer. `disjoint`: a result, whose matrices must not share
// elements.
bool stack_ok(const SegMatrix &m, int elem, bool disjoint, Range *range) {
  if (m.ld < (m.cols > 1 ? m.cols : 1) || m.ld > kMaxPitch || m.stride < 0) return false;
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

// The workspace of a call, from the library's pool: copies of operands that the
// kernels cannot read as they lie, and what its products hand to one another.
class Workspace {
 public:
  Workspace(bool bf16, const int64_t *offsets, int64_t groups, int64_t M)
      : bf16_(bf16), offsets_(offsets), groups_(groups), rows_(M) {}

  // Have m copied, unless it is readable or empty. by_segment: matrix g is
  // used only where segment g has rows.
  void readable(SegMatrix &m, bool by_segment = false) {
    if (m.rows == 0 || m.cols == 0 || m.count == 0 || gemm::seg_tc_readable(m, bf16_)) return;
    gemm::SegCopy &c = copies_[copy_count_];
    c.src = m;
    if (m.stride == 0) c.src.count = 1;
    if (by_segment && m.stride != 0) {
      c.offsets = offsets_;
      c.groups = groups_;
      c.M = rows_;
      c.by_matrix = true;
    }
    target_[copy_count_++] = &m;
    matrix(m, m.rows, m.cols, bf16_ ? 2 : 4, m.stride == 0 ? 1 : m.count);
  }

  // A new stack of matrices with readable rows.
  void matrix(SegMatrix &m, int64_t rows, int64_t cols, int elem, int64_t count = 1) {
    const int64_t per16 = 16 / elem;
    m.rows = rows;
    m.cols = cols;
    m.ld = (cols + per16 - 1) / per16 * per16;
    if (count > 1) m.stride = rows * m.ld;
    placed_[placed_count_] = &m;
    at_[placed_count_++] = bytes_;
    bytes_ += static_cast<size_t>((count * rows * m.ld * elem + 255) / 256 * 256);
  }

  // Room for splitting the tiles of a product of this shape.
  void splits(const SegArgs &a, int terms = 1) {
    if (gemm::seg_tc_splits(a, terms) && !(gemm::seg_rows_fits(a) && gemm::seg_rows_few(a) == 0))
      split_ = true;
  }

  // Allocate, place, zero the split tiles' counters, and copy.
  int take(int sms, cudaStream_t s) {
    sms_ = sms;
    const size_t counters = static_cast<size_t>(kProducts) * sms * sizeof(unsigned);
    const size_t slots = split_ ? static_cast<size_t>(gemm::seg_tc_slots(sms)) * sizeof(float) : 0;
    if (bytes_ + slots == 0) return gemm::kOk;
    const int st = gemm::pool_alloc(&p_, bytes_ + slots + (split_ ? counters : 0), s);
    if (st != gemm::kOk) return st;
    if (split_) {
      slots_ = reinterpret_cast<float *>(static_cast<uint8_t *>(p_) + bytes_);
      arrived_ = reinterpret_cast<unsigned *>(static_cast<uint8_t *>(p_) + bytes_ + slots);
      if (cudaMemsetAsync(arrived_, 0, counters, s) != cudaSuccess) return gemm::kErrLaunch;
    }
    for (int i = 0; i < placed_count_; ++i) placed_[i]->p = static_cast<uint8_t *>(p_) + at_[i];
    for (int i = 0; i < copy_count_; ++i) {
      copies_[i].dst = *target_[i];
      const int cst = gemm::seg_pack_launch(copies_[i], bf16_, sms, s);
      if (cst != gemm::kOk) return cst;
    }
    return gemm::kOk;
  }

  // One product, with the scratch it may want.
  int launch(SegArgs &a, cudaStream_t s) {
    if (gemm::seg_rows_fits(a)) {
      a.few = gemm::seg_rows_few(a);
      const int st = gemm::seg_rows_launch(a, sms_, s);
      if (st != gemm::kOk || a.few == 0) return st;
      a.ahead = true;  // other rows of the same operands
    }
    if (split_) {
      a.slots = slots_;
      a.arrived = arrived_ + static_cast<size_t>(products_++ % kProducts) * sms_;
    }
    return gemm::seg_tc_launch(a, sms_, s);
  }

  // Rows of the segments, from here to the caller's matrix.
  int hand_back(const SegMatrix &from, const SegMatrix &to, cudaStream_t s) {
    gemm::SegCopy c;
    c.src = from;
    c.dst = to;
    c.offsets = offsets_;
    c.groups = groups_;
    c.M = rows_;
    return gemm::seg_pack_launch(c, bf16_, sms_, s);
  }

  int give_back(int st, cudaStream_t s) {
    if (p_ == nullptr) return st;
    const int fst = gemm::pool_free(p_, s);
    return st != gemm::kOk ? st : fst;
  }

 private:
  static constexpr int kMost = 12, kProducts = 5;
  bool bf16_;
  const int64_t *offsets_;
  int64_t groups_, rows_;
  void *p_ = nullptr;
  size_t bytes_ = 0;
  gemm::SegCopy copies_[kMost];
  SegMatrix *target_[kMost], *placed_[kMost];
  size_t at_[kMost];
  int copy_count_ = 0, placed_count_ = 0;
  bool split_ = false;
  float *slots_ = nullptr;
  unsigned *arrived_ = nullptr;
  int sms_ = 0, products_ = 0;
};

// Y = X op(W) + U op(B_a), U = s_a (X op(A_a)).
struct Lora {
  bool bf16 = false, adapted = false;
  bool zero_u = false;       // no adapters at all: U's rows are zero
  int transw = 0, transl = 0;
  int64_t segments = 0, bank = 0, M = 0, N = 0, K = 0, R = 0;
  SegMatrix X, W, A, B, Y;
  SegMatrix user_u;          // the caller's, or none
  SegMatrix u, u_lo, sum;    // U, its second term (bf16), and U B in fp32
  const int64_t *offsets = nullptr;
  const int32_t *index = nullptr;
  const float *scales = nullptr;
  bool fused = false, ahead = false;

  // U B in the projection's own accumulators, or a product of its own that the
  // projection's tiles add? An MMA over rows of several segments would let one
  // adapter's NaN or infinity into the others' rows (0 * inf), so the fused
  // form's tiles are the segments' own: each segment reads W again, from L2.
  // With 128 rows a segment and more that costs less than U B's way through
  // memory (8192 rows, nine segments, 4096 x 4096, rank 64 bf16: 259 -> 219 us;
  // 1531 rows, seven segments, 1000 x 2048, rank 24: 131 -> 107 us with its
  // backward pass) -- but a round of float32 tiles more, which the segments'
  // part tiles can make, costs more where there are few (2048 rows, four
  // segments, 2048 x 2048: 105 -> 130 us); 32 rows in 32 segments would read W
  // 32 times.
  void prepare(Workspace &w, int sms) {
    const int64_t tiles = (M + 255) / 256 * ((N + 255) / 256);
    fused = adapted && K > 0 && transw == transl && M >= 128 * segments &&
            (bf16 || tiles >= sms);
    // The projection starts on the SMs that U = s X A, or U B, leaves free (1531
    // rows, 1000 x 2048, rank 24, with its backward pass: 94 -> 85 us, 2048 x
    // 4096 x 4096: 74 -> 70). In the fused form U takes few SMs, the pairs start
    // far apart, and over more than two rounds of tiles they no longer meet in
    // L2 (8192 rows, 2048 x 2048 bf16: 83 -> 88 us).
    ahead = !fused || tiles <= sms;
    w.readable(X);
    w.readable(W);
    SegArgs shape;
    shape.bf16 = bf16;
    shape.dense = true;
    shape.M = M;
    shape.N = N;
    shape.K = K;
    w.splits(shape);
    if (!adapted) return;
    shape.dense = false;
    shape.groups = segments;
    shape.N = R;
    w.splits(shape);
    w.readable(A);
    w.readable(B);
    // bf16: U is an operand of the second product, and rounded to one bf16 it
    // would add an error as large as the result's own rounding: two terms.
    const int elem = bf16 ? 2 : 4;
    if (user_u.p != nullptr && gemm::seg_tc_readable(user_u, bf16))
      u = user_u;
    else
      w.matrix(u, M, R, elem);
    if (bf16) w.matrix(u_lo, M, R, elem);
    if (!fused) w.matrix(sum, M, N, 4);
  }

  int run(Workspace &w, cudaStream_t s) {
    SegArgs y;
    y.bf16 = bf16;
    y.M = M;
    y.bank = bank;
    y.offsets = offsets;
    y.groups = adapted ? segments : 0;
    if (zero_u) {
      SegArgs z = y;  // a product without a contraction
      z.groups = segments;
      z.N = R;
      z.C = user_u;
      const int st = w.launch(z, s);
      if (st != gemm::kOk) return st;
    }
    if (adapted) {
      SegArgs p = y;  // U = s (X A)
      p.index = index;
      p.N = R;
      p.K = K;
      p.A = X;
      p.B = A;
      p.transb = transl;
      p.scales = scales;
      p.C = u;
      p.C_lo = u_lo;
      int st = w.launch(p, s);
      if (st == gemm::kOk && user_u.p != nullptr && u.p != user_u.p)
        st = w.hand_back(u, user_u, s);
      if (st != gemm::kOk) return st;
    }
    y.dense = true;
    y.N = N;
    y.K = K;
    y.A = X;
    y.B = W;
    y.transb = transw;
    y.C = Y;
    if (N == 0) return gemm::kOk;  // no Y
    if (!adapted) return w.launch(y, s);
    y.ahead = ahead;
    if (fused) {
      y.index = index;
      y.R = R;
      y.U = u;
      y.U_lo = u_lo;
      y.L = B;
      return w.launch(y, s);
    }
    SegArgs e = y;  // U B
    e.ahead = false;
    e.dense = false;
    e.index = index;
    e.K = R;
    e.A = u;
    e.A_lo = u_lo;
    e.B = B;
    e.transb = transl;
    e.C = sum;
    e.c_f32 = true;
    int st = w.launch(e, s);
    if (st != gemm::kOk) return st;
    y.add = sum;
    return w.launch(y, s);
  }
};

// One product, its operands copied where they have to be.
int launch(SegArgs &a, int sms, cudaStream_t s) {
  Workspace w(a.bf16, a.offsets, a.groups, a.M);
  if (a.M > 0 && (a.wgrad || a.K > 0)) {
    w.readable(a.A);
    w.readable(a.B, !a.wgrad);
    w.splits(a);
  }
  int st = w.take(sms, s);
  if (st == gemm::kOk) st = w.launch(a, s);
  return w.give_back(st, s);
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
      !dim_ok(K) || !dim_ok(R) || bank < 0 || bank > kMaxPitch)
    return GEMM_ERR_INVALID_ARG;
  const int elem = type == GEMM_F32_TYPE_BF16 ? 2 : 4;
  Lora l;
  l.bf16 = type == GEMM_F32_TYPE_BF16;
  l.transw = transw;
  l.transl = transl;
  const bool rows = R > 0 && segments > 0 && M > 0;  // that an adapter may have
  l.adapted = rows && bank > 0;
  l.zero_u = rows && bank == 0 && U != nullptr;
  l.segments = segments;
  l.bank = bank;
  l.M = M;
  l.N = N;
  l.K = K;
  l.R = R;
  l.X = SegMatrix{X, ldx, 0, M, K, 1};
  l.W = SegMatrix{W, ldw, 0, transw ? N : K, transw ? K : N, 1};
  l.A = SegMatrix{A, lda, stridea, transl ? R : K, transl ? K : R, bank};
  l.B = SegMatrix{B, ldb, strideb, transl ? N : R, transl ? R : N, bank};
  l.user_u = SegMatrix{U, ldu, 0, M, R, 1};
  l.Y = SegMatrix{Y, ldy, 0, M, N, 1};
  l.offsets = offsets;
  l.index = index;
  l.scales = scales;
  Range rx, rw, ra, rb, ro, ri, rs, ru, ry;
  if (!stack_ok(l.X, elem, false, &rx) || !stack_ok(l.W, elem, false, &rw) ||
      !stack_ok(l.Y, elem, true, &ry))
    return GEMM_ERR_INVALID_ARG;
  if (l.adapted &&
      (!stack_ok(l.A, elem, false, &ra) || !stack_ok(l.B, elem, false, &rb) ||
       !array_ok(index, segments, 4, true, &ri) || !array_ok(scales, bank, 4, true, &rs)))
    return GEMM_ERR_INVALID_ARG;
  if ((l.adapted || l.zero_u) && (!array_ok(offsets, segments + 1, 8, false, &ro) ||
                                  (U != nullptr && !stack_ok(l.user_u, elem, true, &ru))))
    return GEMM_ERR_INVALID_ARG;
  const Range in[] = {rx, rw, ra, rb, ro, ri, rs};
  for (const Range &r : in)
    if (overlap(r, ry) || overlap(r, ru)) return GEMM_ERR_ALIAS;
  if (overlap(ru, ry)) return GEMM_ERR_ALIAS;
  if (M == 0 || (N == 0 && ((!l.adapted && !l.zero_u) || U == nullptr))) return GEMM_OK;
  int dev = 0, sms = 0;
  int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Workspace work(l.bf16, offsets, segments, M);
  l.prepare(work, sms);
  st = work.take(sms, s);
  if (st == gemm::kOk) st = l.run(work, s);
  return work.give_back(st, s);
}

int gemm_f32_lora_backward(int type, int transw, int transl, int64_t segments, int64_t M,
                           int64_t N, int64_t K, int64_t R, const void *dY, int64_t lddy,
                           const void *X, int64_t ldx, const void *U, int64_t ldu, const void *W,
                           int64_t ldw, const void *A, int64_t lda, int64_t stridea,
                           const void *B, int64_t ldb, int64_t strideb, const int64_t *offsets,
                           const float *scales, void *dX, int64_t lddx, void *dA, int64_t ldda,
                           int64_t strideda, void *dB, int64_t lddb, int64_t stridedb,
                           void *stream) {
  if (!common_ok(type, segments) || !op_ok(transw) || !op_ok(transl) || !dim_ok(M) || !dim_ok(N) ||
      !dim_ok(K) || !dim_ok(R))
    return GEMM_ERR_INVALID_ARG;
  const int elem = type == GEMM_F32_TYPE_BF16 ? 2 : 4;
  // dX = dY op(W)^T + s (dY B^T) A^T: the forward with N and K, and the
  // factors, exchanged, every matrix read the other way round.
  Lora l;
  l.bf16 = type == GEMM_F32_TYPE_BF16;
  l.transw = transw ? GEMM_OP_N : GEMM_OP_T;
  l.transl = transl ? GEMM_OP_N : GEMM_OP_T;
  l.adapted = R > 0 && segments > 0 && M > 0;
  l.segments = l.bank = segments;
  l.M = M;
  l.N = K;
  l.K = N;
  l.R = R;
  l.X = SegMatrix{dY, lddy, 0, M, N, 1};
  l.W = SegMatrix{W, ldw, 0, transw ? N : K, transw ? K : N, 1};
  l.A = SegMatrix{B, ldb, strideb, transl ? N : R, transl ? R : N, segments};
  l.B = SegMatrix{A, lda, stridea, transl ? R : K, transl ? K : R, segments};
  l.Y = SegMatrix{dX, lddx, 0, M, K, 1};
  l.offsets = offsets;
  l.scales = scales;
  SegMatrix x{X, ldx, 0, M, K, 1}, u{U, ldu, 0, M, R, 1};
  const SegMatrix da{dA, ldda, strideda, transl ? R : K, transl ? K : R, segments};
  const SegMatrix db{dB, lddb, stridedb, transl ? N : R, transl ? R : N, segments};
  Range rdy, rx, ru, rw, ra, rb, ro, rs, rdx, rda, rdb;
  if (!stack_ok(l.X, elem, false, &rdy) || !stack_ok(l.W, elem, false, &rw) ||
      !stack_ok(l.Y, elem, true, &rdx) || !stack_ok(da, elem, true, &rda) ||
      !stack_ok(db, elem, true, &rdb))
    return GEMM_ERR_INVALID_ARG;
  if (segments > 0 && !array_ok(offsets, segments + 1, 8, false, &ro)) return GEMM_ERR_INVALID_ARG;
  if (l.adapted &&
      (!stack_ok(x, elem, false, &rx) || !stack_ok(u, elem, false, &ru) ||
       !stack_ok(l.A, elem, false, &rb) || !stack_ok(l.B, elem, false, &ra) ||
       !array_ok(scales, segments, 4, true, &rs)))
    return GEMM_ERR_INVALID_ARG;
  const Range in[] = {rdy, rx, ru, rw, ra, rb, ro, rs}, out[] = {rdx, rda, rdb};
  for (int i = 0; i < 3; ++i) {
    for (const Range &r : in)
      if (overlap(r, out[i])) return GEMM_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(out[j], out[i])) return GEMM_ERR_ALIAS;
  }
  // No dX, and neither dA nor dB.
  if ((M == 0 || K == 0) && (segments == 0 || R == 0 || (K == 0 && N == 0))) return GEMM_OK;
  int dev = 0, sms = 0;
  int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Workspace work(l.bf16, offsets, segments, M);
  if (M > 0) {
    SegArgs shape;  // of the gradients
    shape.bf16 = l.bf16;
    shape.wgrad = true;
    shape.M = M;
    work.splits(shape);
    // dA's V has two terms in bf16: half the rows are as long. Asked of the
    // segments' average, since zeroing the counters takes 5 us (1531 rows in one
    // segment, 2048 x 1000, rank 24: 55.5 -> 52 us; in seven, 48 -> 53).
    if (l.bf16 && l.adapted) {
      shape.M = M / segments;
      work.splits(shape, 2);
    }
    l.prepare(work, sms);
    if (l.adapted) {
      work.readable(x);
      work.readable(u);
    }
  }
  st = work.take(sms, s);
  if (st == gemm::kOk && M > 0) st = l.run(work, s);
  // dA = X^T V (stored R x K: V^T X) and dB = U^T dY (stored N x R: dY^T U).
  SegArgs g;
  g.bf16 = l.bf16;
  g.wgrad = true;
  g.groups = segments;
  g.M = M;
  g.offsets = offsets;
  const SegMatrix &v = l.u;
  if (st == gemm::kOk && segments > 0 && R > 0 && K > 0) {
    g.A = transl ? v : x;
    g.B = transl ? x : v;
    g.A_lo = transl ? l.u_lo : SegMatrix{};
    g.B_lo = transl ? SegMatrix{} : l.u_lo;
    g.C = da;
    g.K = da.rows;
    g.N = da.cols;
    g.ahead = M > 0;  // V was made before dX
    st = work.launch(g, s);
  }
  if (st == gemm::kOk && segments > 0 && R > 0 && N > 0) {
    g.A = transl ? l.X : u;
    g.B = transl ? u : l.X;
    g.A_lo = g.B_lo = SegMatrix{};
    g.C = db;
    g.K = db.rows;
    g.N = db.cols;
    g.ahead = M > 0;  // reads what the caller gave
    st = work.launch(g, s);
  }
  return work.give_back(st, s);
}

}  // extern "C"
