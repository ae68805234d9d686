/*
 * reduce_f32.h -- C ABI of libgemm_f32.so, part 2: the sum of a fp32 vector,
 * and the norm of many tensors together and their clipping by it, on an NVIDIA
 * GB300 (sm_103a).
 *
 * Operation. out[0] = sum_{i < n} x[i], computed as in "GPU compute shaders"
 * ("How it works", step 6, and the reduce routine under "Code"): `groups`
 * groups each walk x with a grid stride and reduce their threads' sums by a
 * tree to one partial sum; a second dispatch adds the partials. Status codes
 * are those of gemm_f32.h.
 *
 * Determinism: for the same n, groups, device and 16-byte alignment of x,
 * every addition happens in the same order, so reruns give bit-identical
 * results (the page's "Pitfalls": a float sum is reproducible only when the
 * group count and the order are fixed).
 *
 * Accuracy: with G groups, |out - sum x| <= h 2^-24 sum |x| (to first order),
 * h = ceil(n / (1024 G)) + ceil(G / 256) + 24: each element passes through at
 * most h fp32 roundings.
 */
#ifndef REDUCE_F32_H
#define REDUCE_F32_H

#include <stdint.h>

#include "segment_gemm_f32.h"  /* gemm_f32_type */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * reduce_f32_sum -- *out = sum of x[0, n), stream ordered.
 *   n       elements, 0 <= n <= 2^40; n == 0 sets *out = 0.
 *   x       device pointer to n fp32 values, 4-byte aligned (16-byte aligned
 *           x takes 128-bit loads).
 *   out     device pointer to one fp32, 4-byte aligned, outside x
 *           (GEMM_ERR_ALIAS otherwise).
 *   groups  number of partial sums, 1 .. 65535, or 0 for the default (four
 *           per SM). It fixes the summation order.
 *   stream  cudaStream_t as void* (NULL = the legacy default stream).
 * The partial sums live in a workspace of `groups` floats taken from the
 * library's stream-ordered memory pool on `stream` and returned behind the
 * second kernel. Argument errors are reported before anything is enqueued.
 * Returns a gemm_f32_status.
 */
int reduce_f32_sum(int64_t n, const float *x, float *out, int groups, void *stream);

/*
 * reduce_f32_norm -- *norm = sqrt(sum of x^2 over all elements of all tensors).
 * reduce_f32_clip -- y = x min(1, limit / (*norm + 1e-6)) for every tensor: the
 * clipping of gradients by their global norm.
 *   count   tensors, 0 .. 2^20 (none: the norm is 0)
 *   x, y    HOST arrays of `count` device pointers, each to the n[i] elements of
 *           a dense tensor, aligned to its element; y NULL, or y[i] = x[i]: in
 *           place (which nothing is written to where the factor is 1). No result
 *           may overlap another, the norm, or an operand but its own in the same
 *           place (GEMM_ERR_ALIAS): a tensor that is listed twice cannot be
 *           clipped in place.
 *   n       HOST array, elements of each tensor, 0 .. 2^40
 *   type    HOST array, a gemm_f32_type for each tensor (x[i] and y[i])
 *   limit   >= 0 (infinity: no tensor changes unless the norm is not finite)
 *   norm    device pointer to one fp32
 * The arrays are read before the call returns. Squares are added by 32 to 64 in
 * fp32 (in 64 bits where their sum is below 2^-100 or above 2^100), those sums in 64
 * bits: the norm is within 2^-20 of its value over the whole range of the types. The
 * order is fixed by the tensors' sizes and alignment, the device and the order of
 * the list: reruns are bit-identical.
 * The factor is computed in 64 bits and rounded to fp32 (2^-24; below 2^-126 to
 * 2^-150), the products once to the type. An infinite element makes the norm infinite,
 * the factor 0 (NaN with an infinite limit) and infinite elements NaN; a NaN makes every
 * result NaN. A finite norm above fp32's range is given as infinity, with the factor
 * of its value. Workspace: 8 bytes a CTA from the library's pool.
 *   A launch takes up to 100 tensors of a shorter list, 1000 of a longer one. Each of
 * the clipping's launches adds the partial sums of all of the norm's: 10000 tensors of
 * 100 elements take 0.35 ms, 100000 9 ms (the norm alone 1.5), 2^20 0.76 s (16 ms).
 */
int reduce_f32_norm(int64_t count, const void *const *x, const int64_t *n, const int *type,
                    float *norm, void *stream);
int reduce_f32_clip(int64_t count, const void *const *x, void *const *y, const int64_t *n,
                    const int *type, float limit, float *norm, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* REDUCE_F32_H */
