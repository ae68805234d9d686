/*
 * segment_gemm_f32.h -- C ABI of libgemm_f32.so, part 3: matrix products over
 * segments of rows on an NVIDIA GB300 (sm_103a): products grouped by expert
 * with ragged sizes, their weight gradients, and low-rank adapters of many
 * requests beside a shared projection.
 *
 * Segments. The rows (tokens) of a row-major matrix lie sorted by segment:
 * segment g is rows offsets[g] .. offsets[g + 1] - 1. `offsets` holds
 * segments + 1 int64 values in DEVICE memory, non-decreasing, from 0 to at
 * most M; the host never reads them, so a router's output on the same stream
 * can be passed on without a synchronisation. Segments may be empty; rows
 * before offsets[0] and from offsets[segments] on belong to none. Values
 * outside [0, M] are held to it and a decreasing one makes its segment empty,
 * so that no access leaves the matrices. Where two segments claim a row, or
 * offsets decrease in a call with adapters, results are unspecified. At most
 * GEMM_F32_MAX_SEGMENTS segments a call.
 *
 * Types. `type` is that of every matrix of the call (a gemm_f32_type). The
 * "f32" of the names is the type of the sums: products are exact to fp32 or
 * better and accumulated in fp32, whatever the operands' type.
 *   GEMM_F32_TYPE_F32   fp32 operands and results, FP32 class: |C - AB| <=
 *                       2 K 2^-24 (|A| |B|), as GEMM_F32_EXACT, for operands
 *                       that are zero or from 2^-110 in magnitude to the
 *                       largest finite value, and results of 2^-126 and more
 *                       that pass no infinity on the way. Smaller operands are
 *                       held to 2^-134 each. Results of an infinite or NaN
 *                       operand are not finite (NaN where fp32 arithmetic may
 *                       have infinity; which one depends on the sizes).
 *   GEMM_F32_TYPE_BF16  bf16 operands, fp32 sums, results rounded once to bf16
 *                       (nearest even). The tensor cores truncate as they add
 *                       to a sum: up to about 1e-9 K of it, half a rounding to
 *                       bf16 at a million products of one sign.
 * A row of one segment never reaches the results of another: NaN and
 * infinities stay in the rows (and, in gradients, in the segments) that hold
 * them.
 *
 * Streams, ownership, errors and thread safety are those of gemm_f32.h.
 * Results do not depend on timing: the same call gives the same bits.
 */
#ifndef SEGMENT_GEMM_F32_H
#define SEGMENT_GEMM_F32_H

#include <stdint.h>

#include "gemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GEMM_F32_TYPE_F32 = 0,
    GEMM_F32_TYPE_BF16 = 1
} gemm_f32_type;

#define GEMM_F32_MAX_SEGMENTS 2048
/* M, N, K and R at most: 2^31 - 2^26, so that sums of a size, a tile and the
 * number of tiles stay below 2^31. */
#define GEMM_F32_MAX_SEGMENT_SIZE 0x7c000000

/*
 * gemm_f32_grouped -- C_g = A_g op(B_g) for every segment (expert) g: rows of A
 * times the segment's own matrix, into the same rows of C.
 *   groups    segments, 0 .. GEMM_F32_MAX_SEGMENTS
 *   M, N, K   A is M x K, op(B_g) K x N, C is M x N
 *   transb    GEMM_OP_N: B_g stored K x N (ldb >= max(1, N)); GEMM_OP_T: N x K
 *             (ldb >= max(1, K)) -- also the gradient of the inputs of a
 *             product with GEMM_OP_N
 *   B         B_g starts strideb elements after B_(g-1); strideb >= 0 (0: one
 *             matrix for all)
 *   C         rows of no segment are not written; must not overlap A, B or
 *             offsets (GEMM_ERR_ALIAS)
 * Pointers are device pointers aligned to their element (offsets to 8 bytes).
 * K == 0 sets the segments' rows to zero. Leading dimensions and spans as for
 * gemm_f32; sizes up to GEMM_F32_MAX_SEGMENT_SIZE.
 */
int gemm_f32_grouped(int type, int transb, int64_t groups, int64_t M, int64_t N, int64_t K,
                     const void *A, int64_t lda,
                     const void *B, int64_t ldb, int64_t strideb,
                     void *C, int64_t ldc,
                     const int64_t *offsets, void *stream);

/*
 * gemm_f32_grouped_wgrad -- C_g = A_g^T D_g for every segment g: the gradient
 * of B_g in C = A B (D: the gradient of the product's result).
 *   M, N, K   A is M x K, D is M x N, every C_g K x N
 *   C         C_g starts stridec elements after C_(g-1); stridec >= (K - 1) ldc
 *             + N. An empty segment's C_g is set to zero.
 */
int gemm_f32_grouped_wgrad(int type, int64_t groups, int64_t M, int64_t N, int64_t K,
                           const void *A, int64_t lda,
                           const void *D, int64_t ldd,
                           void *C, int64_t ldc, int64_t stridec,
                           const int64_t *offsets, void *stream);

/*
 * gemm_f32_lora -- a shared projection with a low-rank adapter for each
 * segment (request):
 *
 *     U = s_a (X A_a),   Y = X op(W) + U B_a,   a = index[segment of the row]
 *
 *   segments  0 .. GEMM_F32_MAX_SEGMENTS
 *   bank      adapters held in A, B and scales
 *   M, N, K, R  X is M x K, op(W) K x N, A_a K x R, B_a R x N, U M x R, Y M x N
 *   transw    W stored K x N (GEMM_OP_N) or N x K (GEMM_OP_T)
 *   transl    GEMM_OP_N: A_a stored K x R and B_a R x N; GEMM_OP_T: A_a R x K
 *             and B_a N x R. With dY for X, W and the factors exchanged and
 *             both flags flipped the same call is the gradient of X, and U
 *             the second operand of the gradient of A.
 *   A, B      adapter a starts stridea (strideb) elements after a - 1 (0: one
 *             factor shared by all)
 *   index     device int32, one adapter for each segment; NULL: adapter g for
 *             segment g. A value outside [0, bank) means none: such rows, and
 *             rows of no segment, get X op(W) alone.
 *   scales    device float, s_a for each adapter; NULL: 1
 *   U, ldu    receives U (rows of no segment are not written, those of a
 *             segment without adapter are zero), rounded to the type: what
 *             gemm_f32_lora_backward takes: in bf16 half the memory between the
 *             passes, at 1.4 times the error of a dB rounded once (2.35e-3 of
 *             its norm against 1.66e-3). NULL: not returned. The second product
 *             takes U unrounded (bf16: as the sum of two bf16 terms).
 *   Y         all M rows are written; Y and U must not overlap anything else
 *             (GEMM_ERR_ALIAS)
 * R == 0 is the projection alone. U's terms and U B (M x N fp32) stand in a
 * workspace from the library's stream-ordered pool meanwhile.
 */
int gemm_f32_lora(int type, int transw, int transl, int64_t segments, int64_t bank,
                  int64_t M, int64_t N, int64_t K, int64_t R,
                  const void *X, int64_t ldx,
                  const void *W, int64_t ldw,
                  const void *A, int64_t lda, int64_t stridea,
                  const void *B, int64_t ldb, int64_t strideb,
                  const int64_t *offsets, const int32_t *index, const float *scales,
                  void *U, int64_t ldu,
                  void *Y, int64_t ldy, void *stream);

/*
 * gemm_f32_lora_backward -- gradients of gemm_f32_lora on a frozen W, with
 * adapter g for segment g (rows sorted by adapter):
 *
 *     V = s_g (dY B_g^T),   dX = dY op(W)^T + V A_g^T,
 *     dA_g = X^T V,         dB_g = U^T dY        over the rows of segment g
 *
 *   U         the forward's U, M x R
 *   dA, dB    as A and B are stored (transl), pitches ldda, lddb and strides
 *             strideda, stridedb; empty segments' are zero
 *   others    as for gemm_f32_lora
 */
int gemm_f32_lora_backward(int type, int transw, int transl, int64_t segments,
                           int64_t M, int64_t N, int64_t K, int64_t R,
                           const void *dY, int64_t lddy,
                           const void *X, int64_t ldx,
                           const void *U, int64_t ldu,
                           const void *W, int64_t ldw,
                           const void *A, int64_t lda, int64_t stridea,
                           const void *B, int64_t ldb, int64_t strideb,
                           const int64_t *offsets, const float *scales,
                           void *dX, int64_t lddx,
                           void *dA, int64_t ldda, int64_t strideda,
                           void *dB, int64_t lddb, int64_t stridedb, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SEGMENT_GEMM_F32_H */
