// w4_api.cu -- the C ABI of products with 4-bit weights (declared in
// include/w4_gemm_f32.h): argument validation and launches.

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/w4_gemm_f32.h"
#include "args.h"
#include "w4.h"

namespace {

using gemm::array_ok;
using gemm::dim_ok;
using gemm::overlap;
using gemm::Range;
using gemm::SegArgs;
using gemm::SegMatrix;
using gemm::stack_ok;
using gemm::W4Args;

// Rows a segment from which on the weights are expanded once for the tensor-core
// kernels of the segmented products: measured, w4_launch | many_rows in us at group
// 128, cold caches, a call in a graph,
//   rows                       128        256        512        2048
//   bf16  4096 x 11008       66 | 103  115 | 105  217 | 140   819 | 256
//   bf16  32 x 1408 x 2048  113 | 186  205 | 191  391 | 221  1514 | 514
//   fp32  4096 x 11008      107 | 170  197 | 191  377 | 326  1478 | 731
//   fp32  32 x 1408 x 2048  189 | 271  356 | 311  696 | 464  2719 | 1460
// The host knows their average alone. Where one segment has most of the rows, that one's
// turns follow each other; with 8 of 10 rows in the last segment, the others equal,
//   rows, average              128        256
//   bf16  8 x 4096 x 11008  426 | 787   752 | 897  (equal: 240 | 758, 457 | 766)
//   bf16  32 x 1408 x 2048  707 | 199  1337 | 227
//   fp32  8 x 4096 x 11008  754 | 1389 1383 | 1768 (equal: 455 | 1354, 891 | 1460)
//   fp32  32 x 1408 x 2048 1235 | 318  2383 | 416
// so that many small matrices with most rows in one take up to six times as long as
// expanded ones would.
constexpr int64_t kManyRows = 256;
// Bytes of expanded weights at a time: more than 4096 x 11008 have, for a part of
// them has fewer tiles than the GPU SMs (at 128 MB that one took 247 us in place of
// 149; 256 MB and 1 GB are within 6 % of each other).
constexpr int64_t kExpanded = int64_t{512} << 20;

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Many rows: the weights as matrices of the type (bf16: as the sum of two, which
// holds s (q - z) exactly), so many at a time as kExpanded holds, through the
// segmented products' kernel.
int many_rows(const W4Args &a, int sms, cudaStream_t s) {
  const int elem = a.bf16 ? 2 : 4, terms = a.bf16 ? 2 : 1;
  const int64_t ld = up(a.K, 8), line = ld * elem * terms;
  int64_t rows = kExpanded / line / 256 * 256;
  if (rows < 256) rows = 256;
  if (rows > a.N) rows = a.N;
  int64_t slab = kExpanded / (rows * line);
  if (slab < 1) slab = 1;
  if (slab > a.groups) slab = a.groups;
  const int64_t one = up(slab * rows * ld * elem, 256);
  SegMatrix x{a.A, a.lda, 0, a.M, a.K, 1};
  const bool copy = !gemm::seg_tc_readable(x, a.bf16);
  const int64_t ldx = up(a.K, 8);
  uint8_t *ws = nullptr;
  int st = gemm::pool_alloc(reinterpret_cast<void **>(&ws),
                            static_cast<size_t>(one * terms + (copy ? a.M * ldx * elem : 0)), s);
  if (st != gemm::kOk) return st;
  if (copy) {
    gemm::SegCopy c;
    c.src = x;
    c.dst = x;
    c.dst.p = ws + one * terms;
    c.dst.ld = ldx;
    st = gemm::seg_pack_launch(c, a.bf16, sms, s);
    x = c.dst;
  }
  for (int64_t g0 = 0; st == gemm::kOk && g0 < a.groups; g0 += slab) {
    W4Args w = a;
    w.groups = a.groups - g0 < slab ? a.groups - g0 : slab;
    w.Q += g0 * a.strideq;
    w.scales = static_cast<const uint8_t *>(a.scales) + g0 * a.strides * elem;
    if (w.zeros != nullptr) w.zeros += g0 * a.stridez;
    if (w.offsets != nullptr) w.offsets += g0;
    for (int64_t n0 = 0; st == gemm::kOk && n0 < a.N; n0 += rows) {
      const int64_t now = a.N - n0 < rows ? a.N - n0 : rows;
      st = gemm::w4_expand_launch(w, n0, now, ws, ws + one, ld, sms, s);
      if (st != gemm::kOk) break;
      SegArgs p;
      p.bf16 = a.bf16;
      p.dense = a.offsets == nullptr;
      p.groups = p.dense ? 0 : w.groups;
      p.bank = w.groups;
      p.M = a.M;
      p.N = now;
      p.K = a.K;
      p.A = x;
      p.B = SegMatrix{ws, ld, now * ld, now, a.K, w.groups};
      if (a.bf16) {
        p.B_lo = p.B;
        p.B_lo.p = ws + one;
      }
      p.transb = GEMM_OP_T;
      p.C = SegMatrix{static_cast<uint8_t *>(a.C) + n0 * elem, a.ldc, 0, a.M, now, 1};
      p.offsets = w.offsets;
      st = gemm::seg_tc_launch(p, sms, s);
    }
  }
  const int fst = gemm::pool_free(ws, s);
  return st != gemm::kOk ? st : fst;
}

}  // namespace

extern "C" int gemm_f32_w4(int type, int64_t groups, int64_t M, int64_t N, int64_t K,
                           int64_t group, const void *A, int64_t lda, const uint8_t *Q,
                           int64_t ldq, int64_t strideq, const void *scales, int64_t lds,
                           int64_t strides, const uint8_t *zeros, int64_t ldz, int64_t stridez,
                           void *C, int64_t ldc, const int64_t *offsets, void *stream) {
  if ((type != GEMM_F32_TYPE_F32 && type != GEMM_F32_TYPE_BF16) || groups < 0 ||
      groups > GEMM_F32_MAX_SEGMENTS || !dim_ok(M) || !dim_ok(N) || !dim_ok(K) || group < 32 ||
      group % 32 != 0 || !dim_ok(group) || (offsets == nullptr && groups > 1))
    return GEMM_ERR_INVALID_ARG;
  const int elem = type == GEMM_F32_TYPE_BF16 ? 2 : 4;
  const int64_t row_groups = (K + group - 1) / group;
  Range ra, rq, rs, rz, rc, ro;
  if (!stack_ok(SegMatrix{A, lda, 0, M, K, 1}, elem, false, &ra) ||
      !stack_ok(SegMatrix{Q, ldq, strideq, N, (K + 1) / 2, groups}, 1, false, &rq) ||
      !stack_ok(SegMatrix{scales, lds, strides, N, row_groups, groups}, elem, false, &rs) ||
      (zeros != nullptr &&
       !stack_ok(SegMatrix{zeros, ldz, stridez, N, row_groups, groups}, 1, false, &rz)) ||
      !stack_ok(SegMatrix{C, ldc, 0, M, N, 1}, elem, true, &rc) ||
      !array_ok(offsets, groups + 1, 8, true, &ro))
    return GEMM_ERR_INVALID_ARG;
  if (groups == 0 || M == 0 || N == 0) return GEMM_OK;
  const Range in[] = {ra, rq, rs, rz, ro};
  for (const Range &r : in)
    if (overlap(r, rc)) return GEMM_ERR_ALIAS;
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) {  // empty sums
    if (offsets != nullptr)
      return gemm_f32_grouped(type, GEMM_OP_T, groups, M, N, 0, A, lda, Q, 1, 0, C, ldc, offsets,
                              stream);
    return cudaMemset2DAsync(C, static_cast<size_t>(ldc) * elem, 0, static_cast<size_t>(N) * elem,
                             static_cast<size_t>(M), s) == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
  }
  W4Args a;
  a.bf16 = type == GEMM_F32_TYPE_BF16;
  a.groups = groups;
  a.M = M;
  a.N = N;
  a.K = K;
  a.group = group;
  a.A = A;
  a.lda = lda;
  a.Q = Q;
  a.ldq = ldq;
  a.strideq = strideq;
  a.scales = scales;
  a.lds = lds;
  a.strides = strides;
  a.zeros = zeros;
  a.ldz = ldz;
  a.stridez = stridez;
  a.C = C;
  a.ldc = ldc;
  a.offsets = offsets;
  return M >= kManyRows * groups ? many_rows(a, sms, s) : gemm::w4_launch(a, sms, s);
}
