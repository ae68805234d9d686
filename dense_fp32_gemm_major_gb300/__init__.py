"""Python binding of libgemm_f32.so: dense row-major fp32 GEMM on GB300.

Argument marshalling only. Every step of the product runs in the library's
CUDA kernels; there is no CPU or PyTorch fallback. Importing the package does
not need a GPU, but it does need the built library: if libgemm_f32.so is
missing the import fails loudly (build it with ``__graft_entry__.build()`` or
``python -m dense_fp32_gemm_major_gb300._build``).

The entry points mirror include/gemm_f32.h one to one (same names, same
argument order; pointers are plain integers, streams are ``cudaStream_t``
values as integers, 0 = the legacy default stream). ``matmul`` and ``gemm``
are convenience wrappers over ``gemm_f32_ex`` and ``gemm_f32_general`` for
torch CUDA tensors; ``grouped_matmul``, ``grouped_wgrad``, ``lora_matmul`` and
``lora_backward`` those of the products over segments of rows
(include/segment_gemm_f32.h), for float32 and bfloat16 tensors. Around those:
the router ``route``, ``route_backward`` and ``route_plan``, the rows' way to the
experts and back ``dispatch``, ``combine`` and ``combine_backward``
(include/route_f32.h), products with 4-bit weights ``w4_matmul``
(include/w4_gemm_f32.h), and the gradients' ``grad_norm`` and ``clip_grads``
(include/reduce_f32.h).

``checked_library()`` loads libgemm_f32_checked.so, the same library built
with device-side index checks (see include/gemm_f32.h, "The checked build");
its handle has the same functions, and the wrappers below take it as ``lib``.
"""

from __future__ import annotations

import array
import collections
import ctypes
import operator
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgemm_f32.so")
LIB_CHECKED_PATH = os.path.join(_PKG, "libgemm_f32_checked.so")
INCLUDE_DIR = os.path.join(os.path.dirname(_PKG), "include")
HEADER_PATH = os.path.join(INCLUDE_DIR, "gemm_f32.h")
HEADERS = [HEADER_PATH, os.path.join(INCLUDE_DIR, "reduce_f32.h"),
           os.path.join(INCLUDE_DIR, "segment_gemm_f32.h"),
           os.path.join(INCLUDE_DIR, "route_f32.h"),
           os.path.join(INCLUDE_DIR, "w4_gemm_f32.h")]

# gemm_f32_mode
EXACT, TF32, EXACT_SIMT = 0, 1, 2
MODES = {"exact": EXACT, "tf32": TF32, "exact_simt": EXACT_SIMT}
# gemm_f32_status
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_DEVICE, ERR_LAUNCH, ERR_TIMEOUT, ERR_ALIAS, ERR_INDEX = range(7)
# index-check sites (gemm_f32_take_index_fault)
SITE_C_STORE, SITE_PARTIAL_WRITE, SITE_PARTIAL_READ, SITE_COUNTER, SITE_BAND = range(1, 6)
SITE_LOAD_A, SITE_LOAD_B, SITE_COPY_SRC, SITE_COPY_DST = range(6, 10)
SITE_REDUCE_IN, SITE_REDUCE_PARTIAL, SITE_REDUCE_OUT = range(10, 13)
# fixed scratch of gemm_f32_noalloc
NOALLOC_SCRATCH_BYTES = 40 * 1024 * 1024
# gemm_f32_kernel
KERNEL_AUTO, KERNEL_SIMT, KERNEL_TC_TMA, KERNEL_TC_LSU = range(4)
KERNELS = {"auto": KERNEL_AUTO, "simt": KERNEL_SIMT, "tc_tma": KERNEL_TC_TMA, "tc_lsu": KERNEL_TC_LSU}
# gemm_f32_order, gemm_f32_op
ROW_MAJOR, COL_MAJOR = 0, 1
OP_N, OP_T = 0, 1
# gemm_f32_type
TYPE_F32, TYPE_BF16 = 0, 1
MAX_SEGMENTS, MAX_SEGMENT_SIZE = 2048, 0x7c000000
# gemm_f32_score
SCORES = {"softmax": 0, "sigmoid": 1}
MAX_ROUTE_SLOTS = 32


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = "gemm_f32"):
        self.status = status
        super().__init__(f"{what} failed: {gemm_f32_status_string(status)} ({status})")


_lib = None
_lib_checked = None


def _open(path):
    if not os.path.exists(path):
        raise RuntimeError(
            f"{os.path.basename(path)} is not built ({path}); run __graft_entry__.build(). "
            "There is no fallback implementation.")
    lib = ctypes.CDLL(path)
    i64, i32, p = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    sig = [i64, i64, i64, p, i64, p, i64, p, i64]
    lib.gemm_f32.argtypes = sig + [i32, p]
    lib.gemm_f32.restype = i32
    lib.gemm_f32_ex.argtypes = sig + [i32, i32, p]
    lib.gemm_f32_ex.restype = i32
    lib.gemm_f32_select.argtypes = sig + [i32, i32]
    lib.gemm_f32_select.restype = i32
    lib.gemm_f32_host.argtypes = sig + [i32]
    lib.gemm_f32_host.restype = i32
    lib.gemm_f32_noalloc.argtypes = sig + [i32, p]
    lib.gemm_f32_noalloc.restype = i32
    f32 = ctypes.c_float
    lib.gemm_f32_general.argtypes = [i32, i32, i32, i64, i64, i64, f32, p, i64, p, i64, f32, p,
                                     i64, i32, i32, p]
    lib.gemm_f32_general.restype = i32
    lib.reduce_f32_sum.argtypes = [i64, p, p, i32, p]
    lib.reduce_f32_sum.restype = i32
    lib.gemm_f32_grouped.argtypes = [i32, i32, i64, i64, i64, i64, p, i64, p, i64, i64, p, i64, p, p]
    lib.gemm_f32_grouped.restype = i32
    lib.gemm_f32_grouped_wgrad.argtypes = [i32, i64, i64, i64, i64, p, i64, p, i64, p, i64, i64, p, p]
    lib.gemm_f32_grouped_wgrad.restype = i32
    lib.gemm_f32_lora.argtypes = ([i32, i32, i32] + [i64] * 6 + [p, i64, p, i64, p, i64, i64,
                                  p, i64, i64, p, p, p, p, i64, p, i64, p])
    lib.gemm_f32_lora.restype = i32
    lib.gemm_f32_lora_backward.argtypes = ([i32, i32, i32] + [i64] * 5 + [p, i64] * 4
                                           + [p, i64, i64] * 2 + [p, p, p, i64]
                                           + [p, i64, i64] * 2 + [p])
    lib.gemm_f32_lora_backward.restype = i32
    lib.gemm_f32_route.argtypes = ([i32, i32, i64, i64, i64, p, i64, p, p, i64, i64, i64, i32, f32]
                                   + [p] * 6)
    lib.gemm_f32_route.restype = i32
    lib.gemm_f32_route_backward.argtypes = [i32, i32, i64, i64, i64, p, p, i64, p, p, i32, f32, p,
                                            i64, p]
    lib.gemm_f32_route_backward.restype = i32
    lib.gemm_f32_route_plan.argtypes = [i64, i64, p, p, p, p, p]
    lib.gemm_f32_route_plan.restype = i32
    lib.gemm_f32_dispatch.argtypes = [i32, i64, i64, i64, i64, p, i64, p, p, i64, p]
    lib.gemm_f32_dispatch.restype = i32
    lib.gemm_f32_combine.argtypes = [i32, i64, i64, i64, i64, p, i64, p, p, p, i64, p]
    lib.gemm_f32_combine.restype = i32
    lib.gemm_f32_combine_backward.argtypes = [i32, i64, i64, i64, i64, p, i64, p, i64, p, p, p, i64,
                                              p, p]
    lib.gemm_f32_combine_backward.restype = i32
    lib.gemm_f32_w4.argtypes = [i32] + [i64] * 5 + [p, i64] + [p, i64, i64] * 3 + [p, i64, p, p]
    lib.gemm_f32_w4.restype = i32
    lib.reduce_f32_norm.argtypes = [i64, p, p, p, p, p]
    lib.reduce_f32_norm.restype = i32
    lib.reduce_f32_clip.argtypes = [i64, p, p, p, p, f32, p, p]
    lib.reduce_f32_clip.restype = i32
    lib.gemm_f32_status_string.argtypes = [i32]
    lib.gemm_f32_status_string.restype = ctypes.c_char_p
    lib.gemm_f32_measure_peaks.argtypes = [ctypes.POINTER(ctypes.c_double)] * 4
    lib.gemm_f32_measure_peaks.restype = i32
    lib.gemm_f32_poll_device_status.argtypes = [p]
    lib.gemm_f32_poll_device_status.restype = i32
    lib.gemm_f32_selftest_wait_timeout.argtypes = [i64, p]
    lib.gemm_f32_selftest_wait_timeout.restype = i32
    lib.gemm_f32_selftest_stalled_gemm.argtypes = sig + [i32, i64, p]
    lib.gemm_f32_selftest_stalled_gemm.restype = i32
    lib.gemm_f32_selftest_host_missing_block.argtypes = sig + [i64]
    lib.gemm_f32_selftest_host_missing_block.restype = i32
    lib.gemm_f32_schedule_check.argtypes = [i64, i64, i64, i64, i32, ctypes.POINTER(ctypes.c_int64)]
    lib.gemm_f32_schedule_check.restype = i32
    lib.gemm_f32_checked_build.argtypes = []
    lib.gemm_f32_checked_build.restype = i32
    ll = ctypes.POINTER(ctypes.c_longlong)
    lib.gemm_f32_take_index_fault.argtypes = [p, ll, ctypes.POINTER(i32), ll, ll]
    lib.gemm_f32_take_index_fault.restype = i32
    lib.gemm_f32_index_site_name.argtypes = [i32]
    lib.gemm_f32_index_site_name.restype = ctypes.c_char_p
    lib.gemm_f32_selftest_index_check.argtypes = sig + [i32, i32, p]
    lib.gemm_f32_selftest_index_check.restype = i32
    return lib


def _load():
    global _lib
    if _lib is None:
        _lib = _open(LIB_PATH)
    return _lib


def reload():
    """Drop the cached handles (after a rebuild) and load the library again."""
    global _lib, _lib_checked
    _lib = None
    _lib_checked = None
    return _load()


def library():
    return _load()


def checked_library():
    """The index-checked build (libgemm_f32_checked.so): same functions as
    library(); slower, for debugging and the index-check tests."""
    global _lib_checked
    if _lib_checked is None:
        _lib_checked = _open(LIB_CHECKED_PATH)
    return _lib_checked


def declared_symbols() -> list[str]:
    """Function names declared in the public headers (include/*.h)."""
    names = set()
    for path in HEADERS:
        with open(path) as f:
            text = f.read()
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        names.update(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*((?:gemm|reduce)_f32\w*)\s*\(",
                                text, flags=re.M))
    return sorted(names)


# ------------------------------------------------------------ raw C ABI --

def gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, mode, stream=0) -> int:
    return _load().gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, mode, stream or None)


def gemm_f32_ex(M, N, K, A, lda, B, ldb, C, ldc, mode, kernel, stream=0) -> int:
    return _load().gemm_f32_ex(M, N, K, A, lda, B, ldb, C, ldc, mode, kernel, stream or None)


def gemm_f32_general(order, transa, transb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, mode,
                     kernel=KERNEL_AUTO, stream=0) -> int:
    """C = alpha * op(A) op(B) + beta * C (see include/gemm_f32.h)."""
    return _load().gemm_f32_general(order, transa, transb, M, N, K, alpha, A, lda, B, ldb, beta,
                                    C, ldc, mode, kernel, stream or None)


def gemm_f32_select(M, N, K, A, lda, B, ldb, C, ldc, mode, kernel=KERNEL_AUTO) -> int:
    return _load().gemm_f32_select(M, N, K, A, lda, B, ldb, C, ldc, mode, kernel)


def gemm_f32_host(M, N, K, A, lda, B, ldb, C, ldc, mode) -> int:
    return _load().gemm_f32_host(M, N, K, A, lda, B, ldb, C, ldc, mode)


def gemm_f32_noalloc(M, N, K, A, lda, B, ldb, C, ldc, mode, stream=0) -> int:
    """gemm_f32 that allocates no device memory (workspace in a fixed
    NOALLOC_SCRATCH_BYTES array; see include/gemm_f32.h)."""
    return _load().gemm_f32_noalloc(M, N, K, A, lda, B, ldb, C, ldc, mode, stream or None)


def reduce_f32_sum(n, x, out, groups=0, stream=0) -> int:
    """*out = sum of x[0, n) (device pointers; see include/reduce_f32.h)."""
    return _load().reduce_f32_sum(n, x, out, groups, stream or None)


def gemm_f32_grouped(type, transb, groups, M, N, K, A, lda, B, ldb, strideb, C, ldc, offsets,
                     stream=0) -> int:
    """C_g = A_g op(B_g) for every segment g (see include/segment_gemm_f32.h)."""
    return _load().gemm_f32_grouped(type, transb, groups, M, N, K, A, lda, B, ldb, strideb, C, ldc,
                                    offsets, stream or None)


def gemm_f32_grouped_wgrad(type, groups, M, N, K, A, lda, D, ldd, C, ldc, stridec, offsets,
                           stream=0) -> int:
    """C_g = A_g^T D_g for every segment g (see include/segment_gemm_f32.h)."""
    return _load().gemm_f32_grouped_wgrad(type, groups, M, N, K, A, lda, D, ldd, C, ldc, stridec,
                                          offsets, stream or None)


def gemm_f32_lora(type, transw, transl, segments, bank, M, N, K, R, X, ldx, W, ldw, A, lda, stridea,
                  B, ldb, strideb, offsets, index, scales, U, ldu, Y, ldy, stream=0) -> int:
    """Y = X op(W) + s (X A_a) B_a, a the adapter of the row's segment (see
    include/segment_gemm_f32.h)."""
    return _load().gemm_f32_lora(type, transw, transl, segments, bank, M, N, K, R, X, ldx, W, ldw,
                                 A, lda, stridea, B, ldb, strideb, offsets, index or None,
                                 scales or None, U or None, ldu, Y, ldy, stream or None)


def gemm_f32_lora_backward(type, transw, transl, segments, M, N, K, R, dY, lddy, X, ldx, U, ldu, W,
                           ldw, A, lda, stridea, B, ldb, strideb, offsets, scales, dX, lddx, dA,
                           ldda, strideda, dB, lddb, stridedb, stream=0) -> int:
    """Gradients of gemm_f32_lora (see include/segment_gemm_f32.h)."""
    return _load().gemm_f32_lora_backward(type, transw, transl, segments, M, N, K, R, dY, lddy, X,
                                          ldx, U, ldu, W, ldw, A, lda, stridea, B, ldb, strideb,
                                          offsets, scales or None, dX, lddx, dA, ldda, strideda, dB,
                                          lddb, stridedb, stream or None)


def gemm_f32_route(type, score, T, E, k, logits, ldx, bias, mask, groups, top_groups, group_best,
                   renormalise, scale, experts, weights, offsets, order, places, stream=0) -> int:
    """The k best experts of every token, their weights, and the plan (see
    include/route_f32.h)."""
    return _load().gemm_f32_route(type, score, T, E, k, logits, ldx, bias or None, mask or None,
                                  groups, top_groups, group_best, renormalise, scale, experts,
                                  weights, offsets or None, order or None, places or None,
                                  stream or None)


def gemm_f32_route_backward(type, score, T, E, k, dweights, logits, ldx, experts, weights,
                            renormalise, scale, dlogits, lddx, stream=0) -> int:
    """Gradient of the logits (see include/route_f32.h)."""
    return _load().gemm_f32_route_backward(type, score, T, E, k, dweights, logits, ldx, experts,
                                           weights, renormalise, scale, dlogits, lddx, stream or None)


def gemm_f32_route_plan(slots, E, experts, offsets, order, places, stream=0) -> int:
    """The plan of given experts (see include/route_f32.h)."""
    return _load().gemm_f32_route_plan(slots, E, experts, offsets, order, places, stream or None)


def gemm_f32_dispatch(type, T, D, k, rows, X, ldx, places, Y, ldy, stream=0) -> int:
    """Each token's row to all of its places (see include/route_f32.h)."""
    return _load().gemm_f32_dispatch(type, T, D, k, rows, X, ldx, places, Y, ldy, stream or None)


def gemm_f32_combine(type, T, D, k, rows, Y, ldy, places, weights, O, ldo, stream=0) -> int:
    """The weighted sum of each token's rows (see include/route_f32.h)."""
    return _load().gemm_f32_combine(type, T, D, k, rows, Y, ldy, places, weights or None, O, ldo,
                                    stream or None)


def gemm_f32_combine_backward(type, T, D, k, rows, dO, lddo, Y, ldy, places, weights, dY, lddy,
                              dweights, stream=0) -> int:
    """Gradients of gemm_f32_combine (see include/route_f32.h)."""
    return _load().gemm_f32_combine_backward(type, T, D, k, rows, dO, lddo, Y, ldy, places,
                                             weights or None, dY or None, lddy, dweights or None,
                                             stream or None)


def gemm_f32_w4(type, groups, M, N, K, group, A, lda, Q, ldq, strideq, scales, lds, strides, zeros,
                ldz, stridez, C, ldc, offsets, stream=0) -> int:
    """C = A W^T with weights in 4 bits (see include/w4_gemm_f32.h)."""
    return _load().gemm_f32_w4(type, groups, M, N, K, group, A, lda, Q, ldq, strideq, scales, lds,
                               strides, zeros or None, ldz, stridez, C, ldc, offsets or None,
                               stream or None)


def reduce_f32_norm(count, x, n, type, norm, stream=0) -> int:
    """The norm of many tensors together; x, n, type: ctypes arrays (see
    include/reduce_f32.h)."""
    return _load().reduce_f32_norm(count, x, n, type, norm, stream or None)


def reduce_f32_clip(count, x, y, n, type, limit, norm, stream=0) -> int:
    """Tensors clipped by their norm (see include/reduce_f32.h)."""
    return _load().reduce_f32_clip(count, x, y, n, type, limit, norm, stream or None)


def gemm_f32_status_string(status: int) -> str:
    return _load().gemm_f32_status_string(status).decode()


def gemm_f32_measure_peaks():
    """(status, tf32_tflops, fp32_tflops, tf32_sm_mhz, fp32_sm_mhz) from the
    MMA-only and FFMA-only probe kernels on the current device: each rate and
    the median SM clock its kernel ran at."""
    t, f = ctypes.c_double(0.0), ctypes.c_double(0.0)
    tc, fc = ctypes.c_double(0.0), ctypes.c_double(0.0)
    st = _load().gemm_f32_measure_peaks(ctypes.byref(t), ctypes.byref(f), ctypes.byref(tc),
                                        ctypes.byref(fc))
    return st, t.value, f.value, tc.value, fc.value


def gemm_f32_poll_device_status(stream=0) -> int:
    return _load().gemm_f32_poll_device_status(stream or None)


def gemm_f32_selftest_wait_timeout(timeout_ns: int, stream=0) -> int:
    return _load().gemm_f32_selftest_wait_timeout(timeout_ns, stream or None)


def gemm_f32_selftest_stalled_gemm(M, N, K, A, lda, B, ldb, C, ldc, mode, timeout_ns,
                                   stream=0) -> int:
    return _load().gemm_f32_selftest_stalled_gemm(M, N, K, A, lda, B, ldb, C, ldc, mode,
                                                  timeout_ns, stream or None)


def gemm_f32_checked_build(lib=None) -> int:
    return (lib or _load()).gemm_f32_checked_build()


def gemm_f32_take_index_fault(stream=0, lib=None):
    """(status, count, site, offset, extent): the index-check record since the
    last call, reset (checked build; count is always 0 in the regular one)."""
    count, off, ext = ctypes.c_longlong(0), ctypes.c_longlong(0), ctypes.c_longlong(0)
    site = ctypes.c_int(0)
    st = (lib or _load()).gemm_f32_take_index_fault(stream or None, ctypes.byref(count),
                                                   ctypes.byref(site), ctypes.byref(off),
                                                   ctypes.byref(ext))
    return st, count.value, site.value, off.value, ext.value


def gemm_f32_index_site_name(site: int, lib=None) -> str:
    return (lib or _load()).gemm_f32_index_site_name(site).decode()


def gemm_f32_selftest_index_check(M, N, K, A, lda, B, ldb, C, ldc, mode, kernel=KERNEL_AUTO,
                                  stream=0, lib=None) -> int:
    return (lib or _load()).gemm_f32_selftest_index_check(M, N, K, A, lda, B, ldb, C, ldc, mode,
                                                         kernel, stream or None)


def gemm_f32_selftest_host_missing_block(M, N, K, A, lda, B, ldb, C, ldc, timeout_ns) -> int:
    return _load().gemm_f32_selftest_host_missing_block(M, N, K, A, lda, B, ldb, C, ldc,
                                                        timeout_ns)


SCHEDULE_KINDS = {"exact_pair": 0, "tf32_pair": 1, "exact_lsu": 2, "tf32_lsu": 3}
SCHEDULE_STATS = ("tiles", "k_blocks", "whole_tiles", "sk_share", "sk_clusters", "splits",
                  "max_parts", "clusters", "cluster_split")


def gemm_f32_schedule_check(m: int, n: int, k: int, workers: int, kind):
    """Host-only check of the tile schedule (no GPU): (status, stats dict)."""
    stats = (ctypes.c_int64 * len(SCHEDULE_STATS))()
    kind = SCHEDULE_KINDS[kind] if isinstance(kind, str) else int(kind)
    st = _load().gemm_f32_schedule_check(m, n, k, workers, kind, stats)
    return st, dict(zip(SCHEDULE_STATS, list(stats)))


# ---------------------------------------------------------- conveniences --

def _mode(mode) -> int:
    return MODES[mode] if isinstance(mode, str) else int(mode)


def _kernel(kernel) -> int:
    return KERNELS[kernel] if isinstance(kernel, str) else int(kernel)


def _check_rows(shape, row_stride, col_stride, name):
    """A matrix the library can address as (pointer, leading dimension): unit
    column stride and rows that do not overlap (strides in elements). Views
    that break either rule (expanded, transposed or reversed ones) would make
    the library read or write outside the matrix, so they are refused."""
    rows, cols = int(shape[0]), int(shape[1])
    if rows == 0 or cols == 0:
        return
    if cols > 1 and col_stride != 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    if rows > 1 and row_stride < cols:
        raise ValueError(f"{name} has overlapping or reversed rows (row stride {row_stride} "
                         f"for {cols} columns)")


def _check_operand(t, name, device=None):
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D float32 CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    _check_rows(t.shape, t.stride(0), t.stride(1), name)


def _ld(t) -> int:
    return max(int(t.stride(0)), int(t.shape[1]), 1) if t.shape[0] > 1 else max(int(t.shape[1]), 1)


def matmul(a, b, mode="exact", out=None, kernel="auto", stream=None):
    """C = A x B for row-major float32 CUDA tensors (stream ordered).

    ``a`` is M x K, ``b`` K x N; ``out`` (M x N, row-major, may have a padded
    row stride) is overwritten and returned. ``stream`` defaults to torch's
    current stream.
    """
    import torch

    _check_operand(a, "a")
    _check_operand(b, "b", a.device)
    m, k = a.shape
    k2, n = b.shape
    if k != k2:
        raise ValueError(f"inner dimensions differ: {tuple(a.shape)} x {tuple(b.shape)}")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=a.device)
    else:
        _check_operand(out, "out", a.device)
        if tuple(out.shape) != (m, n):
            raise ValueError("out has the wrong shape")
    if stream is None:
        stream = torch.cuda.current_stream(a.device).cuda_stream
    with torch.cuda.device(a.device):
        st = gemm_f32_ex(m, n, k, a.data_ptr(), _ld(a), b.data_ptr(), _ld(b), out.data_ptr(),
                         _ld(out), _mode(mode), _kernel(kernel), stream)
    if st != OK:
        raise GemmError(st)
    return out


def gemm(a, b, out=None, alpha=1.0, beta=0.0, transa=False, transb=False, mode="exact",
         kernel="auto", stream=None):
    """out = alpha * op(a) op(b) + beta * out for row-major float32 CUDA tensors.

    ``a`` is stored M x K, or K x M with ``transa``; ``b`` K x N, or N x K
    with ``transb``. ``out`` (M x N) is read only when beta != 0 and is
    required then. Stream ordered on ``stream`` (default: torch's current
    stream); returns ``out``.
    """
    import torch

    _check_operand(a, "a")
    _check_operand(b, "b", a.device)
    m, k = (a.shape[1], a.shape[0]) if transa else tuple(a.shape)
    k2, n = (b.shape[1], b.shape[0]) if transb else tuple(b.shape)
    if k != k2:
        raise ValueError(f"inner dimensions differ: op(a) is {m} x {k}, op(b) is {k2} x {n}")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs out")
        out = torch.empty((m, n), dtype=torch.float32, device=a.device)
    else:
        _check_operand(out, "out", a.device)
        if tuple(out.shape) != (m, n):
            raise ValueError("out has the wrong shape")
    if stream is None:
        stream = torch.cuda.current_stream(a.device).cuda_stream
    with torch.cuda.device(a.device):
        st = gemm_f32_general(ROW_MAJOR, OP_T if transa else OP_N, OP_T if transb else OP_N, m, n,
                              k, float(alpha), a.data_ptr(), _ld(a), b.data_ptr(), _ld(b),
                              float(beta), out.data_ptr(), _ld(out), _mode(mode), _kernel(kernel),
                              stream)
    if st != OK:
        raise GemmError(st, "gemm_f32_general")
    return out


def vector_sum(x, groups=0, out=None, stream=None):
    """Sum of a 1-D float32 CUDA tensor through reduce_f32_sum; returns a
    one-element float32 CUDA tensor (stream ordered)."""
    import torch

    if (not isinstance(x, torch.Tensor) or x.dtype != torch.float32 or not x.is_cuda
            or x.dim() != 1 or (x.numel() > 1 and x.stride(0) != 1)):
        raise TypeError("x must be a contiguous 1-D float32 CUDA tensor")
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    elif (not isinstance(out, torch.Tensor) or out.dtype != torch.float32
          or out.device != x.device or out.numel() < 1):
        raise TypeError("out must be a float32 tensor of at least one element on x's device")
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    with torch.cuda.device(x.device):
        st = reduce_f32_sum(x.numel(), x.data_ptr(), out.data_ptr(), int(groups), stream)
    if st != OK:
        raise GemmError(st, "reduce_f32_sum")
    return out


# Operands of the segmented products. The checks run on every call, before
# microseconds of work, so each tensor's attributes are read once.

def _segment_type(t, name):
    """The library's type code of a float32 or bfloat16 CUDA tensor."""
    import torch

    if isinstance(t, torch.Tensor) and t.is_cuda:
        if t.dtype is torch.bfloat16:
            return TYPE_BF16
        if t.dtype is torch.float32:
            return TYPE_F32
    raise TypeError(f"{name} must be a float32 or bfloat16 CUDA tensor")


def _addressing(shape, strides, name):
    """(leading dimension, stride of the stack) of a matrix or a stack of them
    that the library can address; the rules are those of _check_rows."""
    rows, cols = shape[-2], shape[-1]
    ld, unit = strides[-2], strides[-1]
    if (unit != 1 and cols > 1) or (rows > 1 and ld < cols):
        _check_rows((rows, cols), ld, unit, name)
    return (ld if rows > 1 and cols else cols) or 1, (
        strides[0] if len(shape) == 3 and shape[0] > 1 else 0)


def _matrices(t, name, dim, kind, device):
    """(shape, pointer, leading dimension, stride of the stack) of a `dim`-D
    tensor of the type and device."""
    if _segment_type(t, name) != kind or t.get_device() != device:
        raise ValueError(f"{name} is {t.dtype} on {t.device}, unlike the first operand")
    shape = t.shape
    if len(shape) != dim:
        raise TypeError(f"{name} must have {dim} dimensions, not {len(shape)}")
    ld, stride = _addressing(shape, t.stride(), name)
    return shape, t.data_ptr(), ld, stride


def _result(out, name, shape, like, kind, device, stream):
    """out, or a new tensor of the shape in memory of the call's stream (on
    another than torch's current one the call runs ahead of work that may still
    read what the current one's memory held), and its (pointer, ld, stride)."""
    if out is None:
        import torch

        if stream is None or stream == torch._C._cuda_getCurrentRawStream(device):
            out = torch.empty(shape, dtype=like.dtype, device=device)
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
                out = torch.empty(shape, dtype=like.dtype, device=device)
        return out, out.data_ptr(), shape[-1] or 1, (shape[1] * shape[2] if len(shape) == 3 else 0)
    got, ptr, ld, stride = _matrices(out, name, len(shape), kind, device)
    if tuple(got) != shape:
        raise ValueError(f"{name} has the wrong shape: {tuple(got)}, not {shape}")
    if len(shape) == 3 and shape[0] > 1 and out.numel() and stride < (shape[1] - 1) * ld + shape[2]:
        raise ValueError(f"{name}'s matrices overlap")
    return out, ptr, ld, stride


def _offsets(offsets, device):
    """(segments, pointer)"""
    import torch

    if (not isinstance(offsets, torch.Tensor) or offsets.dtype is not torch.int64
            or offsets.dim() != 1 or not offsets.is_cuda or offsets.get_device() != device
            or not offsets.is_contiguous() or offsets.shape[0] < 1):
        raise TypeError("offsets must be a contiguous 1-D int64 tensor of segments + 1 values on "
                        "the operands' device")
    segments = offsets.shape[0] - 1
    if segments > MAX_SEGMENTS:
        raise ValueError(f"{segments} segments: at most {MAX_SEGMENTS} a call")
    return segments, offsets.data_ptr()


def _array(t, name, dtype, count, device):
    import torch

    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda
            or t.get_device() != device or t.dim() != 1 or t.shape[0] != count
            or not t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous {dtype} tensor of {count} values on the "
                        "operands' device")
    return t.data_ptr()


def _call(name, device, stream, *args):
    import torch

    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    function = getattr(_lib or _load(), name)
    if torch._C._cuda_getDevice() == device:
        st = function(*args, stream or None)
    else:
        with torch.cuda.device(device):
            st = function(*args, stream or None)
    if st != OK:
        raise GemmError(st, name)


def grouped_matmul(a, b, offsets, transb=False, out=None, stream=None):
    """Products grouped by expert: out[t] = a[t] @ op(b[g]) for the rows t of
    segment g, offsets[g] <= t < offsets[g + 1].

    ``a`` is M x K, float32 or bfloat16; ``b`` G x K x N, or G x N x K with
    ``transb`` (which also is the gradient of the inputs: ``grouped_matmul(dy,
    b, offsets, transb=True)``); ``offsets`` G + 1 int64 values on the device,
    never read by the host. ``out`` (M x N) is returned; rows of no segment are
    not written. Stream ordered on ``stream`` (default: torch's current one); a
    new result stands in that stream's memory (``record_stream`` before it is
    dropped while another stream may still read it).

    As of all functions here, results are no part of an autograd graph: the
    gradients are calls of their own (above, and grouped_wgrad).
    """
    kind = _segment_type(a, "a")
    dev = a.get_device()
    (m, k), pa, lda, _ = _matrices(a, "a", 2, kind, dev)
    (count, k2, n), pb, ldb, strideb = _matrices(b, "b", 3, kind, dev)
    groups, po = _offsets(offsets, dev)
    if transb:
        k2, n = n, k2
    if count != groups:
        raise ValueError(f"{count} matrices for {groups} segments")
    if k != k2:
        raise ValueError(f"inner dimensions differ: a is {m} x {k}, op(b) {k2} x {n}")
    out, pc, ldc, _ = _result(out, "out", (m, n), a, kind, dev, stream)
    _call("gemm_f32_grouped", dev, stream, kind, OP_T if transb else OP_N, groups, m, n, k, pa, lda,
          pb, ldb, strideb, pc, ldc, po)
    return out


def grouped_wgrad(a, d, offsets, out=None, stream=None):
    """Weight gradients of grouped_matmul: out[g] = a[rows of g]^T @ d[rows of
    g], zero where segment g is empty. ``a`` is M x K, ``d`` M x N, ``out`` G x
    K x N (returned)."""
    kind = _segment_type(a, "a")
    dev = a.get_device()
    (m, k), pa, lda, _ = _matrices(a, "a", 2, kind, dev)
    (m2, n), pd, ldd, _ = _matrices(d, "d", 2, kind, dev)
    groups, po = _offsets(offsets, dev)
    if m != m2:
        raise ValueError(f"a has {m} rows, d {m2}")
    out, pc, ldc, stridec = _result(out, "out", (groups, k, n), a, kind, dev, stream)
    _call("gemm_f32_grouped_wgrad", dev, stream, kind, groups, m, n, k, pa, lda, pd, ldd, pc, ldc,
          stridec, po)
    return out


def lora_matmul(x, w, lora_a, lora_b, offsets, adapters=None, scales=None, transw=False,
                transl=False, out=None, shrink_out=None, stream=None):
    """A shared projection with a low-rank adapter for each segment of rows:
    out = x @ op(w) + u @ op(lora_b[i]), u = scales[i] * (x @ op(lora_a[i])),
    i = adapters[segment of the row].

    ``x`` is M x K; ``w`` K x N (N x K with ``transw``); ``lora_a`` a bank of
    K x R and ``lora_b`` of R x N matrices (R x K and N x R with ``transl``);
    ``offsets`` segments + 1 int64 values, ``adapters`` int32, one for each
    segment (a value outside the bank: no adapter; None: adapter g for segment
    g), ``scales`` float32, one for each adapter (None: 1), all on the device.
    ``shrink_out`` (M x R, of x's type, u rounded to it), if given, receives u
    for lora_backward. Returns ``out`` (M x N). Factors may be shared: an
    expanded ``lora_a`` or ``lora_b``.
    """
    import torch

    kind = _segment_type(x, "x")
    dev = x.get_device()
    (m, k), px, ldx, _ = _matrices(x, "x", 2, kind, dev)
    (k2, n), pw, ldw, _ = _matrices(w, "w", 2, kind, dev)
    (bank, ka, r), pa, lda, stridea = _matrices(lora_a, "lora_a", 3, kind, dev)
    (bank2, rb, nb), pb, ldb, strideb = _matrices(lora_b, "lora_b", 3, kind, dev)
    segments, po = _offsets(offsets, dev)
    if transw:
        k2, n = n, k2
    if transl:
        ka, r, rb, nb = r, ka, nb, rb
    if k != k2:
        raise ValueError(f"inner dimensions differ: x is {m} x {k}, op(w) {k2} x {n}")
    if ka != k or rb != r or nb != n or bank2 != bank:
        raise ValueError(f"op(lora_a) is {bank} of {ka} x {r} and op(lora_b) {bank2} of {rb} x {nb} "
                         f"beside a {k} x {n} projection")
    if adapters is None and segments > bank:
        raise ValueError(f"{segments} segments, {bank} adapters and no choice of adapters")
    pi = None if adapters is None else _array(adapters, "adapters", torch.int32, segments, dev)
    ps = None if scales is None else _array(scales, "scales", torch.float32, bank, dev)
    out, py, ldy, _ = _result(out, "out", (m, n), x, kind, dev, stream)
    pu, ldu = None, r or 1
    if shrink_out is not None:
        _, pu, ldu, _ = _result(shrink_out, "shrink_out", (m, r), x, kind, dev, stream)
    _call("gemm_f32_lora", dev, stream, kind, OP_T if transw else OP_N, OP_T if transl else OP_N,
          segments, bank, m, n, k, r, px, ldx, pw, ldw, pa, lda, stridea, pb, ldb, strideb, po, pi,
          ps, pu, ldu, py, ldy)
    return out


def lora_backward(dy, x, shrink, w, lora_a, lora_b, offsets, scales=None, transw=False,
                  transl=False, stream=None):
    """Gradients of lora_matmul with one adapter for each segment (adapters
    None; rows sorted by adapter) on a frozen ``w``: (dx, d lora_a, d lora_b).
    ``shrink`` is the forward's shrink_out: for bfloat16, d lora_b is that of u
    as it was rounded. Factors of empty segments get zero; of factors shared by
    several segments (expanded) each segment's gradient is returned.
    """
    import torch

    kind = _segment_type(dy, "dy")
    dev = dy.get_device()
    (m, n), pdy, lddy, _ = _matrices(dy, "dy", 2, kind, dev)
    (m2, k), px, ldx, _ = _matrices(x, "x", 2, kind, dev)
    (m3, r), pu, ldu, _ = _matrices(shrink, "shrink", 2, kind, dev)
    wshape, pw, ldw, _ = _matrices(w, "w", 2, kind, dev)
    ashape, pa, lda, stridea = _matrices(lora_a, "lora_a", 3, kind, dev)
    bshape, pb, ldb, strideb = _matrices(lora_b, "lora_b", 3, kind, dev)
    segments, po = _offsets(offsets, dev)
    if m2 != m or m3 != m:
        raise ValueError(f"dy has {m} rows, x {m2} and shrink {m3}")
    if (tuple(wshape) != ((n, k) if transw else (k, n))
            or tuple(ashape) != ((segments, r, k) if transl else (segments, k, r))
            or tuple(bshape) != ((segments, n, r) if transl else (segments, r, n))):
        raise ValueError(f"w {tuple(wshape)}, lora_a {tuple(ashape)} and lora_b {tuple(bshape)} are "
                         f"not those of {segments} segments, a {k} x {n} projection and rank {r}")
    ps = None if scales is None else _array(scales, "scales", torch.float32, segments, dev)
    dx, pdx, lddx, _ = _result(None, "dx", (m, k), dy, kind, dev, stream)
    da, pda, ldda, strideda = _result(None, "da", tuple(ashape), dy, kind, dev, stream)
    db, pdb, lddb, stridedb = _result(None, "db", tuple(bshape), dy, kind, dev, stream)
    _call("gemm_f32_lora_backward", dev, stream, kind, OP_T if transw else OP_N,
          OP_T if transl else OP_N, segments, m, n, k, r, pdy, lddy, px, ldx, pu, ldu, pw, ldw, pa,
          lda, stridea, pb, ldb, strideb, po, ps, pdx, lddx, pda, ldda, strideda, pdb, lddb,
          stridedb)
    return dx, da, db


def _empty(shape, dtype, device, stream):
    """A new tensor in memory of the call's stream."""
    import torch

    if stream is None or stream == torch._C._cuda_getCurrentRawStream(device):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        return torch.empty(shape, dtype=dtype, device=device)


_codes = {}  # a tensor type's gemm_f32_type; filled at first use


def _matrix(t, name, kind=None, device=None):
    """(type code, device, rows, columns, pointer, leading dimension) of a 2-D
    float32 or bfloat16 CUDA tensor, of the type and device where they are given."""
    if not _codes:
        import torch

        _codes.update({torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16})
    try:
        code, dev, (rows, cols), (ld, unit) = _codes[t.dtype], t.get_device(), t.shape, t.stride()
        pointer = t.data_ptr()
    except (AttributeError, KeyError, ValueError):
        _segment_type(t, name)
        raise TypeError(f"{name} must have 2 dimensions") from None
    if dev < 0:
        _segment_type(t, name)
    if kind is not None and (code != kind or dev != device):
        raise ValueError(f"{name} is {t.dtype} on {t.device}, unlike the first operand")
    if rows > 1:
        if (unit != 1 and cols > 1) or ld < cols:
            _check_rows((rows, cols), ld, unit, name)
        return code, dev, rows, cols, pointer, (ld if cols else cols) or 1
    if unit != 1 and cols > 1:
        _check_rows((rows, cols), ld, unit, name)
    return code, dev, rows, cols, pointer, cols or 1


def _dense(t, name, dtype, shape, device):
    """The pointer of a contiguous tensor of the type, shape and device."""
    import torch

    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != device
            or t.shape != shape or not t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on the "
                        "operands' device")
    return t.data_ptr()


def _slots(t, name, device):
    """(T, k, pointer) of a contiguous T x k int32 tensor."""
    import torch

    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.dim() != 2
            or t.get_device() != device or not t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous 2-D int32 tensor on the operands' device")
    count, k = t.shape
    if not 1 <= k <= MAX_ROUTE_SLOTS:
        raise ValueError(f"{name} has {k} slots a token: 1 to {MAX_ROUTE_SLOTS}")
    return count, k, t.data_ptr()


def _score(score):
    if score not in SCORES:
        raise ValueError(f"score must be one of {', '.join(SCORES)}, not {score!r}")
    return SCORES[score]


Routing = collections.namedtuple("Routing", "experts weights offsets order places")


def _new_routing(t, e, k, device):
    # (five pieces of memory: 7 us of the host; views into one, 13)
    import torch

    empty = torch.empty
    experts = empty((t, k), dtype=torch.int32, device=device)
    return Routing(experts, empty((t, k), dtype=torch.float32, device=device),
                   empty((e + 1,), dtype=torch.int64, device=device),
                   empty((t * k,), dtype=torch.int32, device=device), torch.empty_like(experts))


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_best=2,
          renormalise=True, scale=1.0, mask=None, stream=None):
    """The router of a mixture of experts: the ``k`` experts of every token with
    the largest score + bias, their weights, and the plan that sorts the tokens'
    slots by expert, as a ``Routing``:

      experts   T x k int32, best first, ties to the lowest index; -1: none
      weights   T x k float32: scale * score, with ``renormalise`` over the sum of
                the token's scores; 0 where there is no expert
      offsets   E + 1 int64, as the products over segments take them
      order     T k int32: the slot t k + j of each sorted row; -1 behind the last
      places    T x k int32: the row of each slot, or -1

    ``logits`` is T x E, float32 or bfloat16; ``score`` "softmax" or "sigmoid";
    ``bias`` E float32, for the choice alone. ``groups`` > 1: the experts are that
    many groups of neighbours, and the ``top_groups`` (None: all) groups with the
    largest sum of their ``group_best`` (1 or 2) best are chosen from. ``mask``, T
    bool: tokens with False take no part. Logits or biases of -infinity make an
    expert unavailable. Scores are compared as real numbers are (see
    include/route_f32.h). Nothing is read by the host.
    """
    import torch

    kind, dev, t, e, px, ldx = _matrix(logits, "logits")
    if not 1 <= e <= MAX_SEGMENTS:
        raise ValueError(f"{e} experts: 1 to {MAX_SEGMENTS}")
    if not 1 <= k <= min(e, MAX_ROUTE_SLOTS):
        raise ValueError(f"{k} slots a token: 1 to {MAX_ROUTE_SLOTS}, and to the {e} experts")
    if top_groups is None:
        top_groups = groups
    if not 1 <= groups <= 32 or e % groups or not 1 <= top_groups <= groups or group_best not in (1, 2):
        raise ValueError(f"{e} experts in {groups} groups, {top_groups} chosen by their best "
                         f"{group_best}: up to 32 equal groups, by one or two")
    pb = None if bias is None else _dense(bias, "bias", torch.float32, (e,), dev)
    pm = None if mask is None else _dense(mask, "mask", torch.bool, (t,), dev)
    if stream is None or stream == torch._C._cuda_getCurrentRawStream(dev):
        r = _new_routing(t, e, k, dev)
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev)):
            r = _new_routing(t, e, k, dev)
    _call("gemm_f32_route", dev, stream, kind, _score(score), t, e, k, px, ldx, pb, pm, groups,
          top_groups, group_best, 1 if renormalise else 0, float(scale),
          *[x.data_ptr() for x in r])
    return r


def route_backward(dweights, logits, experts, weights, score="softmax", renormalise=True, scale=1.0,
                   out=None, stream=None):
    """Gradient of ``route``'s logits from that of its weights, ``dweights`` (T x
    k float32), the choice held fixed. ``experts`` and ``weights`` are the
    forward's; ``score``, ``renormalise`` and ``scale`` as there. Returns T x E of
    the logits' type."""
    import torch

    kind, dev, t, e, px, ldx = _matrix(logits, "logits")
    t2, k, pe = _slots(experts, "experts", dev)
    if t2 != t:
        raise ValueError(f"logits has {t} tokens, experts {t2}")
    if not 1 <= e <= MAX_SEGMENTS:
        raise ValueError(f"{e} experts: 1 to {MAX_SEGMENTS}")
    pw = _dense(weights, "weights", torch.float32, (t, k), dev)
    pg = _dense(dweights, "dweights", torch.float32, (t, k), dev)
    out, po, ldo, _ = _result(out, "out", (t, e), logits, kind, dev, stream)
    _call("gemm_f32_route_backward", dev, stream, kind, _score(score), t, e, k, pg, px, ldx, pe, pw,
          1 if renormalise else 0, float(scale), po, ldo)
    return out


def route_plan(experts, count, stream=None):
    """The plan of experts that were chosen otherwise: (offsets, order, places) as
    ``route`` returns them, for ``experts``, T x k int32 (any value outside [0,
    count): none)."""
    import torch

    if not isinstance(experts, torch.Tensor) or not experts.is_cuda:
        raise TypeError("experts must be a contiguous 2-D int32 CUDA tensor")
    dev = experts.get_device()
    t, k, pe = _slots(experts, "experts", dev)
    if not 1 <= count <= MAX_SEGMENTS:
        raise ValueError(f"{count} experts: 1 to {MAX_SEGMENTS}")
    offsets = _empty((count + 1,), torch.int64, dev, stream)
    order = _empty((t * k,), torch.int32, dev, stream)
    places = _empty((t, k), torch.int32, dev, stream)
    _call("gemm_f32_route_plan", dev, stream, t * k, count, pe, offsets.data_ptr(),
          order.data_ptr(), places.data_ptr())
    return offsets, order, places


def dispatch(x, places, out=None, stream=None):
    """Each token's row to all of its places: out[places[t, j]] = x[t]. ``x`` is T
    x D, float32 or bfloat16, ``places`` T x k int32 (``route``'s; outside out's
    rows: none). ``out`` is T k x D where it is not given; rows that no place names
    are not written. Its gradient is ``combine`` without weights."""
    kind, dev, t, d, px, ldx = _matrix(x, "x")
    t2, k, pp = _slots(places, "places", dev)
    if t2 != t:
        raise ValueError(f"x has {t} tokens, places {t2}")
    if out is None:
        shape = (t * k, d)
    elif getattr(out, "dim", lambda: 0)() == 2:
        shape = (out.shape[0], d)
    else:
        raise TypeError("out must be a 2-D tensor")
    out, po, ldo, _ = _result(out, "out", shape, x, kind, dev, stream)
    _call("gemm_f32_dispatch", dev, stream, kind, t, d, k, shape[0], px, ldx, pp, po, ldo)
    return out


def combine(y, places, weights=None, out=None, stream=None):
    """The weighted sum of each token's rows: out[t] = sum_j weights[t, j] *
    y[places[t, j]], in fp32, rounded once; zero where a token has no place.
    ``y`` is rows x D, float32 or bfloat16, ``places`` T x k int32, ``weights`` T x
    k float32 (None: 1, which is the gradient of ``dispatch``)."""
    import torch

    kind, dev, rows, d, py, ldy = _matrix(y, "y")
    t, k, pp = _slots(places, "places", dev)
    pw = None if weights is None else _dense(weights, "weights", torch.float32, (t, k), dev)
    out, po, ldo, _ = _result(out, "out", (t, d), y, kind, dev, stream)
    _call("gemm_f32_combine", dev, stream, kind, t, d, k, rows, py, ldy, pp, pw, po, ldo)
    return out


def combine_backward(dout, y, places, weights=None, out=None, stream=None):
    """Gradients of ``combine``: (dy, dweights), dy[places[t, j]] = weights[t, j] *
    dout[t] (``out`` where it is given; rows that no place names are not written)
    and dweights[t, j] = dout[t] . y[places[t, j]], float32, 0 without a place."""
    import torch

    kind, dev, t, d, pd, ldd = _matrix(dout, "dout")
    _, _, rows, d2, py, ldy = _matrix(y, "y", kind, dev)
    t2, k, pp = _slots(places, "places", dev)
    if t2 != t or d2 != d:
        raise ValueError(f"dout is {t} x {d}, places has {t2} tokens and y {d2} columns")
    pw = None if weights is None else _dense(weights, "weights", torch.float32, (t, k), dev)
    out, po, ldo, _ = _result(out, "out", (rows, d), y, kind, dev, stream)
    dweights = _empty((t, k), torch.float32, dev, stream)
    _call("gemm_f32_combine_backward", dev, stream, kind, t, d, k, rows, pd, ldd, py, ldy, pp, pw,
          po, ldo, dweights.data_ptr())
    return out, dweights


def _w4_matrices(t, name, dtype, dim, device):
    """As _matrices, of a type of its own."""
    if t.dtype is not dtype or not t.is_cuda or t.get_device() != device:
        raise TypeError(f"{name} must be a {dtype} tensor on x's device")
    if t.dim() != dim:
        raise TypeError(f"{name} must have {dim} dimensions, not {t.dim()}")
    ld, stride = _addressing(t.shape, t.stride(), name)
    return t.shape, t.data_ptr(), ld, stride


def w4_matmul(x, q, scales, group, zeros=None, offsets=None, out=None, stream=None):
    """Products with weights in 4 bits: out = x @ w.T, w[n, k] = scales[n, k //
    group] * (q[n, k] - zeros[n, k // group]).

    ``x`` is M x K, float32 or bfloat16. ``q`` is N x ceil(K / 2) uint8, two
    neighbouring k a byte, the even one in the low four bits; ``scales`` N x
    ceil(K / group) of x's type; ``zeros`` the same shape, uint8, of which the low
    four bits count (None: 8). ``group`` is a multiple of 32. With ``offsets``
    (segments + 1 int64 on the device) all three are stacks of a matrix for each
    segment of rows, as for ``grouped_matmul``. Few rows (single tokens, decoding
    steps) take the time of reading ``q``; rows of ``q`` should start on 16 bytes,
    others are copied first. Returns ``out`` (M x N).
    """
    import torch

    kind, dev, m, k, px, ldx = _matrix(x, "x")
    dim, groups, po = 2, 1, None
    if offsets is not None:
        dim = 3
        groups, po = _offsets(offsets, dev)
    for t, name in ((q, "q"), (scales, "scales"), (zeros, "zeros")):
        if not isinstance(t, torch.Tensor) and not (t is None and name == "zeros"):
            raise TypeError(f"{name} must be a tensor")
    qs, pq, ldq, strideq = _w4_matrices(q, "q", torch.uint8, dim, dev)
    ss, ps, lds, strides = _matrices(scales, "scales", dim, kind, dev)
    if group < 32 or group % 32:
        raise ValueError(f"groups of {group}: a multiple of 32")
    n = qs[-2]
    stack = (groups,) if dim == 3 else ()
    row = stack + (n, -(-k // group))
    if tuple(qs) != stack + (n, (k + 1) // 2) or tuple(ss) != row:
        raise ValueError(f"q {tuple(qs)} and scales {tuple(ss)} are not those of {groups} matrices of "
                         f"{n} rows of {k} values in groups of {group}")
    pz, ldz, stridez = None, row[-1] or 1, 0
    if zeros is not None:
        zs, pz, ldz, stridez = _w4_matrices(zeros, "zeros", torch.uint8, dim, dev)
        if tuple(zs) != row:
            raise ValueError(f"zeros {tuple(zs)} for scales {tuple(ss)}")
    out, pc, ldc, _ = _result(out, "out", (m, n), x, kind, dev, stream)
    _call("gemm_f32_w4", dev, stream, kind, groups, m, n, k, group, px, ldx, pq, ldq, strideq, ps,
          lds, strides, pz, ldz, stridez, pc, ldc, po)
    return out


def _tensor_list(tensors, name, device):
    """(device, pointers, sizes, types) of dense tensors on one device. An attribute
    at a time: there may be hundreds of them before microseconds of work."""
    import torch

    types = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16}
    try:
        kinds = list(map(types.__getitem__, map(operator.attrgetter("dtype"), tensors)))
        devices = set(map(torch.Tensor.get_device, tensors))
        if not devices:
            return device, [], [], []
        if min(devices) < 0:
            raise KeyError
    except (AttributeError, KeyError, TypeError):
        raise TypeError(f"{name} must be float32 or bfloat16 CUDA tensors") from None
    if device is not None:
        devices.add(device)
    if len(devices) > 1:
        raise ValueError(f"{name} are not all on one device")
    if not all(map(torch.Tensor.is_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    return (devices.pop(), list(map(torch.Tensor.data_ptr, tensors)),
            list(map(torch.Tensor.numel, tensors)), kinds)


def _arrays(pointers, sizes, kinds):
    # (ctypes arrays of 48 tensors take 12 us of the host, these 2)
    return array.array("Q", pointers), array.array("q", sizes), array.array("i", kinds)


def _address(values):
    return values.buffer_info()[0] or None


def grad_norm(tensors, stream=None):
    """The norm of all tensors together, sqrt(sum of x^2), as a one-element float32
    CUDA tensor. ``tensors``: contiguous float32 and bfloat16 CUDA tensors (of one
    device; none: 0, on the current one)."""
    import torch

    dev, pointers, sizes, kinds = _tensor_list(list(tensors), "tensors", None)
    if dev is None:
        dev = torch.cuda.current_device()
    norm = _empty((1,), torch.float32, dev, stream)
    x, n, kind = _arrays(pointers, sizes, kinds)
    _call("reduce_f32_norm", dev, stream, len(sizes), _address(x), _address(n), _address(kind),
          norm.data_ptr())
    return norm


def clip_grads(tensors, limit, out=None, stream=None):
    """Gradients clipped by their norm: every tensor times min(1, limit / (norm +
    1e-6)), into ``out`` (tensors of the same types and sizes; None: in place).
    Returns the norm before, as grad_norm does; nothing is read by the host. No
    result may overlap another tensor of the call, but its own operand."""
    import torch

    limit = float(limit)
    if not limit >= 0.0:
        raise ValueError(f"limit must be zero or more, not {limit}")
    tensors = list(tensors)
    dev, pointers, sizes, kinds = _tensor_list(tensors, "tensors", None)
    x, n, kind = _arrays(pointers, sizes, kinds)
    y = None
    if out is not None:
        dev, to, to_sizes, to_kinds = _tensor_list(list(out), "out", dev)
        if to_sizes != sizes or to_kinds != kinds:
            raise ValueError("out does not have the tensors' types and sizes")
        y = array.array("Q", to)
    if dev is None:
        dev = torch.cuda.current_device()
    norm = _empty((1,), torch.float32, dev, stream)
    _call("reduce_f32_clip", dev, stream, len(sizes), _address(x), None if y is None else _address(y),
          _address(n), _address(kind), limit, norm.data_ptr())
    return norm


def _check_host(x, name):
    import numpy as np

    if not isinstance(x, np.ndarray) or x.dtype != np.float32 or x.ndim != 2:
        raise TypeError(f"{name} must be a 2-D float32 numpy array")
    if x.strides[0] % 4 or x.strides[1] % 4:
        raise ValueError(f"{name}'s strides are not whole elements")
    _check_rows(x.shape, x.strides[0] // 4, x.strides[1] // 4, name)


def matmul_host(a, b, mode="exact", out=None):
    """C = A x B for host numpy float32 arrays through gemm_f32_host (blocking)."""
    import numpy as np

    _check_host(a, "a")
    _check_host(b, "b")
    m, k = a.shape
    k2, n = b.shape
    if k != k2:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = np.empty((m, n), dtype=np.float32)
    else:
        _check_host(out, "out")
        if out.shape != (m, n):
            raise ValueError("out has the wrong shape")
        if not out.flags.writeable:
            raise ValueError("out is read-only")
    ld = lambda x: max(x.strides[0] // 4, x.shape[1], 1) if x.shape[0] > 1 else max(x.shape[1], 1)
    st = gemm_f32_host(m, n, k, a.ctypes.data, ld(a), b.ctypes.data, ld(b), out.ctypes.data,
                       ld(out), _mode(mode))
    if st != OK:
        raise GemmError(st, "gemm_f32_host")
    return out
