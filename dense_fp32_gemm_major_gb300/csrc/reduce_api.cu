// reduce_api.cu -- the C ABI of the norm of many tensors and of their clipping
// (declared in include/reduce_f32.h): argument validation and launches.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include "../../include/reduce_f32.h"
#include "clip.h"

namespace {

constexpr int64_t kMaxTensors = int64_t{1} << 20, kMaxElements = int64_t{1} << 40;

struct Span {
  uintptr_t lo, hi;
  int64_t i;  // whose result (-1: an operand's)
};

bool tensor_ok(const void *p, int64_t n, int type) {
  if ((type != GEMM_F32_TYPE_F32 && type != GEMM_F32_TYPE_BF16) || n < 0 || n > kMaxElements)
    return false;
  const uintptr_t elem = type == GEMM_F32_TYPE_BF16 ? 2 : 4;
  return n == 0 || (p != nullptr && reinterpret_cast<uintptr_t>(p) % elem == 0);
}

bool lists_ok(int64_t count, const void *const *x, const int64_t *n, const int *type) {
  if (count < 0 || count > kMaxTensors) return false;
  if (count > 0 && (x == nullptr || n == nullptr || type == nullptr)) return false;
  for (int64_t i = 0; i < count; ++i)
    if (!tensor_ok(x[i], n[i], type[i])) return false;
  return true;
}

uintptr_t bytes_of(int64_t n, int type) {
  return static_cast<uintptr_t>(n) * (type == GEMM_F32_TYPE_BF16 ? 2 : 4);
}

// Results that share memory with each other, or with an operand that is not
// their own in the same place. kOk, kErrAlias, or kErrLaunch without memory.
int check_aliases(const gemm::ClipArgs &a) {
  std::unique_ptr<Span[]> out(new (std::nothrow) Span[static_cast<size_t>(a.count + 1)]);
  if (!out) return gemm::kErrLaunch;
  int64_t outs = 0;
  const uintptr_t at_norm = reinterpret_cast<uintptr_t>(a.norm);
  out[outs++] = Span{at_norm, at_norm + 4, -1};
  for (int64_t i = 0; i < a.count; ++i) {
    if (a.n[i] == 0) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.y != nullptr ? a.y[i] : a.x[i]);
    out[outs++] = Span{p, p + bytes_of(a.n[i], a.type[i]), i};
  }
  std::sort(out.get(), out.get() + outs, [](const Span &l, const Span &r) { return l.lo < r.lo; });
  for (int64_t i = 1; i < outs; ++i)
    if (out[i].lo < out[i - 1].hi) return gemm::kErrAlias;
  if (a.y == nullptr) return gemm::kOk;
  for (int64_t i = 0; i < a.count; ++i) {
    if (a.n[i] == 0) continue;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(a.x[i]), hi = lo + bytes_of(a.n[i], a.type[i]);
    // disjoint results in ascending order: the first that ends behind lo
    int64_t f = std::partition_point(out.get(), out.get() + outs,
                                     [lo](const Span &s) { return s.hi <= lo; }) - out.get();
    for (; f < outs && out[f].lo < hi; ++f)
      if (out[f].i != i || out[f].lo != lo) return gemm::kErrAlias;
  }
  return gemm::kOk;
}

// The norm beside its operands.
int check_norm(const gemm::ClipArgs &a) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.norm);
  for (int64_t i = 0; i < a.count; ++i) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(a.x[i]), hi = lo + bytes_of(a.n[i], a.type[i]);
    if (a.n[i] > 0 && at < hi && lo < at + 4) return gemm::kErrAlias;
  }
  return gemm::kOk;
}

bool result_ok(const float *norm) {
  return norm != nullptr && reinterpret_cast<uintptr_t>(norm) % 4 == 0;
}

int run(const gemm::ClipArgs &a, void *stream) {
  int dev = 0, sms = 0;
  const int st = gemm::current_device_info(&dev, &sms);
  if (st != gemm::kOk) return st;
  return gemm::clip_launch(a, sms, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int reduce_f32_norm(int64_t count, const void *const *x, const int64_t *n, const int *type,
                    float *norm, void *stream) {
  if (!lists_ok(count, x, n, type) || !result_ok(norm)) return GEMM_ERR_INVALID_ARG;
  gemm::ClipArgs a;
  a.count = count;
  a.x = x;
  a.n = n;
  a.type = type;
  a.norm = norm;
  const int st = check_norm(a);
  return st != gemm::kOk ? st : run(a, stream);
}

int reduce_f32_clip(int64_t count, const void *const *x, void *const *y, const int64_t *n,
                    const int *type, float limit, float *norm, void *stream) {
  if (!lists_ok(count, x, n, type) || !result_ok(norm) || !(limit >= 0.0f))
    return GEMM_ERR_INVALID_ARG;
  if (y != nullptr)
    for (int64_t i = 0; i < count; ++i)
      if (!tensor_ok(y[i], n[i], type[i])) return GEMM_ERR_INVALID_ARG;
  gemm::ClipArgs a;
  a.count = count;
  a.x = x;
  a.y = y;
  a.n = n;
  a.type = type;
  a.limit = limit;
  a.norm = norm;
  a.scale = true;
  const int st = check_aliases(a);
  return st != gemm::kOk ? st : run(a, stream);
}

}  // extern "C"
