"""The router and the rows' way to the experts (include/route_f32.h), products
with 4-bit weights (include/w4_gemm_f32.h) and the norm of many tensors
(include/reduce_f32.h), what needs no GPU: the entry points refuse bad arguments
before any CUDA call, and the Python wrappers what the library cannot address."""

import ctypes
import math

import pytest
import torch

import dense_fp32_gemm_major_gb300 as g

# Fake, never dereferenced, 256-byte aligned "device" addresses.
P = [0x10000000 * i for i in range(16)]
NO_GPU = (g.ERR_LAUNCH, g.ERR_UNSUPPORTED_DEVICE)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is present")


def route(**kw):
    a = dict(type=0, score=0, T=64, E=32, k=4, logits=P[1], ldx=32, bias=P[2], mask=P[3], groups=4,
             top_groups=2, group_best=2, renormalise=1, scale=1.0, experts=P[4], weights=P[5],
             offsets=P[6], order=P[7], places=P[8])
    a.update(kw)
    return g.gemm_f32_route(*a.values())


def backward(**kw):
    a = dict(type=0, score=0, T=64, E=32, k=4, dweights=P[1], logits=P[2], ldx=32, experts=P[3],
             weights=P[4], renormalise=1, scale=1.0, dlogits=P[5], lddx=32)
    a.update(kw)
    return g.gemm_f32_route_backward(*a.values())


def plan(**kw):
    a = dict(slots=64, E=32, experts=P[1], offsets=P[2], order=P[3], places=P[4])
    a.update(kw)
    return g.gemm_f32_route_plan(*a.values())


def dispatch(**kw):
    a = dict(type=0, T=16, D=48, k=2, rows=32, X=P[1], ldx=48, places=P[2], Y=P[3], ldy=48)
    a.update(kw)
    return g.gemm_f32_dispatch(*a.values())


def combine(**kw):
    a = dict(type=0, T=16, D=48, k=2, rows=32, Y=P[1], ldy=48, places=P[2], weights=P[4], O=P[3],
             ldo=48)
    a.update(kw)
    return g.gemm_f32_combine(*a.values())


def combine_backward(**kw):
    a = dict(type=0, T=16, D=48, k=2, rows=32, dO=P[1], lddo=48, Y=P[2], ldy=48, places=P[3],
             weights=P[4], dY=P[5], lddy=48, dweights=P[6])
    a.update(kw)
    return g.gemm_f32_combine_backward(*a.values())


def w4(**kw):
    a = dict(type=0, groups=4, M=16, N=64, K=96, group=32, A=P[1], lda=96, Q=P[2], ldq=48,
             strideq=64 * 48, scales=P[3], lds=3, strides=192, zeros=P[4], ldz=3, stridez=192, C=P[5],
             ldc=64, offsets=P[6])
    a.update(kw)
    return g.gemm_f32_w4(*a.values())


def lists(x, n, kinds):
    c = len(n)
    return (ctypes.c_void_p * c)(*x), (ctypes.c_int64 * c)(*n), (ctypes.c_int * c)(*kinds)


def norm(x=(P[1], P[2]), n=(100, 7), kinds=(0, 1), out=P[9]):
    x, n, kinds = lists(x, n, kinds)
    return g.reduce_f32_norm(len(n), x, n, kinds, out)


def clip(x=(P[1], P[2]), y=None, n=(100, 7), kinds=(0, 1), limit=1.0, out=P[9]):
    y = None if y is None else (ctypes.c_void_p * len(y))(*y)
    x, n, kinds = lists(x, n, kinds)
    return g.reduce_f32_clip(len(n), x, y, n, kinds, limit, out)


BIG = 1 << 31
REFUSED = [
    (route, [dict(type=2), dict(score=2), dict(score=-1), dict(T=-1), dict(E=0), dict(E=2049, ldx=2049),
             dict(k=0), dict(k=33), dict(E=2, ldx=2, groups=1, top_groups=1, k=3), dict(ldx=31),
             dict(groups=0), dict(groups=3), dict(groups=64), dict(top_groups=0), dict(top_groups=5),
             dict(group_best=0), dict(group_best=3), dict(renormalise=2), dict(scale=math.nan),
             dict(logits=0), dict(logits=P[1] + 2), dict(bias=P[2] + 2), dict(experts=0),
             dict(weights=0), dict(weights=P[5] + 1), dict(offsets=0), dict(order=0), dict(places=0),
             dict(offsets=P[6] + 4), dict(T=1 << 30)]),
    (backward, [dict(type=2), dict(score=2), dict(T=-1), dict(E=0), dict(E=4096, ldx=4096, lddx=4096),
                dict(k=0), dict(k=33), dict(ldx=31), dict(lddx=31), dict(scale=0.0),
                dict(scale=math.nan), dict(dweights=0), dict(logits=0), dict(experts=0),
                dict(weights=0), dict(dlogits=0), dict(dlogits=P[5] + 2), dict(renormalise=-1)]),
    (plan, [dict(slots=-1), dict(slots=BIG), dict(E=0), dict(E=2049), dict(experts=0), dict(offsets=0),
            dict(order=0), dict(places=0), dict(places=P[4] + 2)]),
    (dispatch, [dict(type=2), dict(T=-1), dict(D=-1), dict(k=0), dict(k=33), dict(rows=-1),
                dict(ldx=47), dict(ldy=47), dict(X=0), dict(Y=0), dict(places=0), dict(Y=P[3] + 2),
                dict(rows=BIG), dict(T=BIG - 1)]),
    (combine, [dict(type=-1), dict(T=-1), dict(D=-1), dict(k=0), dict(k=33), dict(ldy=47),
               dict(ldo=47), dict(Y=0), dict(O=0), dict(places=0), dict(weights=P[4] + 2)]),
    (combine_backward, [dict(type=2), dict(k=33), dict(lddo=47), dict(ldy=47), dict(lddy=47),
                        dict(dO=0), dict(Y=0), dict(places=0), dict(dY=0, dweights=0),
                        dict(dweights=P[6] + 2)]),
    (w4, [dict(type=2), dict(groups=-1), dict(groups=2049), dict(M=-1), dict(N=-1), dict(K=-1),
          dict(group=0), dict(group=16), dict(group=48), dict(group=-32), dict(lda=95), dict(ldq=47),
          dict(lds=2), dict(ldz=2), dict(ldc=63), dict(strideq=-1), dict(offsets=0), dict(A=0),
          dict(Q=0), dict(scales=0), dict(C=0), dict(A=P[1] + 2), dict(offsets=P[6] + 4),
          dict(scales=P[3] + 2)]),
    (norm, [dict(x=(P[1], 0)), dict(x=(P[1] + 2, P[2])), dict(x=(P[1], P[2] + 1)), dict(n=(100, -1)),
            dict(kinds=(0, 2)), dict(out=0), dict(out=P[9] + 2), dict(n=(100, 1 << 41))]),
    (clip, [dict(x=(P[1], 0)), dict(kinds=(-1, 1)), dict(out=0), dict(limit=-1.0),
            dict(limit=math.nan), dict(y=(P[3], 0)), dict(y=(P[3] + 2, P[4]))]),
]


@pytest.mark.parametrize("call, kw", [(c, kw) for c, kws in REFUSED for kw in kws],
                         ids=lambda v: v.__name__ if callable(v) else str(v))
def test_refuses(call, kw):
    assert call(**kw) == g.ERR_INVALID_ARG


ALIASES = [
    (route, [dict(experts=P[1]), dict(weights=P[4]), dict(order=P[7], places=P[7] + 64), dict(offsets=P[3]),
             dict(weights=P[2] + 124)]),
    (backward, [dict(dlogits=P[2]), dict(dlogits=P[1] + 1020), dict(dlogits=P[4])]),
    (plan, [dict(order=P[1]), dict(places=P[3]), dict(offsets=P[4])]),
    (dispatch, [dict(Y=P[1]), dict(Y=P[2])]),
    (combine, [dict(O=P[1]), dict(O=P[4] - 64)]),
    (combine_backward, [dict(dY=P[2]), dict(dY=P[1]), dict(dweights=P[5] + 8), dict(dweights=P[4])]),
    (w4, [dict(C=P[1]), dict(C=P[2] + 4), dict(C=P[3]), dict(C=P[4]), dict(C=P[6])]),
    (norm, [dict(out=P[1] + 396), dict(out=P[2] + 12)]),
    (clip, [dict(x=(P[1], P[1] + 200)), dict(x=(P[1], P[1]), kinds=(0, 0)), dict(y=(P[3], P[3] + 4)),
            dict(y=(P[2], P[4])), dict(y=(P[1] + 4, P[4])), dict(out=P[1]), dict(y=(P[3], P[4]), out=P[4]),
            dict(y=(P[3], P[4]), out=P[2])]),
]


@pytest.mark.parametrize("call, kw", [(c, kw) for c, kws in ALIASES for kw in kws],
                         ids=lambda v: v.__name__ if callable(v) else str(v))
def test_aliases_are_refused(call, kw):
    assert call(**kw) == g.ERR_ALIAS


def test_nothing_to_do_makes_no_cuda_call():
    assert route(T=0, logits=0, experts=0, weights=0, offsets=0, order=0, places=0) == g.OK
    assert backward(T=0, dweights=0, logits=0, experts=0, weights=0, dlogits=0) == g.OK
    assert dispatch(T=0, X=0, places=0) == g.OK and dispatch(D=0, X=0, Y=0) == g.OK
    assert combine(T=0, O=0, places=0) == g.OK and combine(D=0, Y=0, O=0) == g.OK
    assert combine_backward(T=0, dO=0, places=0, dweights=0) == g.OK
    assert w4(M=0, A=0, C=0) == g.OK and w4(N=0, Q=0, scales=0, zeros=0, C=0) == g.OK
    assert w4(groups=0, Q=0, scales=0, offsets=0) == g.OK


@no_gpu
def test_valid_calls_fail_cleanly_without_a_gpu():
    assert route() in NO_GPU
    assert route(bias=0, mask=0, groups=1, top_groups=1, offsets=0, order=0, places=0) in NO_GPU
    assert route(T=0, logits=0, experts=0, weights=0, order=0, places=0) in NO_GPU  # offsets
    assert backward(type=1, score=1, renormalise=0, scale=0.0) in NO_GPU
    assert plan() in NO_GPU and plan(slots=0, experts=0, order=0, places=0) in NO_GPU  # offsets
    assert dispatch(type=1) in NO_GPU and combine(weights=0) in NO_GPU
    assert combine_backward(dY=0) in NO_GPU and combine_backward(dweights=0, Y=0) in NO_GPU
    assert combine_backward(D=0, dO=0, Y=0, dY=0) in NO_GPU  # zeros
    assert w4() in NO_GPU and w4(groups=1, offsets=0, zeros=0) in NO_GPU
    assert w4(K=0, A=0, Q=0, scales=0, zeros=0) in NO_GPU and w4(strideq=0, strides=0, stridez=0) in NO_GPU
    assert norm() in NO_GPU and norm((), (), ()) in NO_GPU
    assert clip() in NO_GPU and clip(y=(P[1], P[2])) in NO_GPU and clip(y=(P[3], P[4])) in NO_GPU
    assert clip(x=(P[1], 0), n=(100, 0), limit=math.inf) in NO_GPU


def test_wrappers_refuse_what_is_not_on_a_gpu():
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: g.route(x, 2), lambda: g.route_backward(x, x, i, x),
                 lambda: g.route_plan(i, 8), lambda: g.dispatch(x, i), lambda: g.combine(x, i),
                 lambda: g.combine_backward(x, x, i),
                 lambda: g.w4_matmul(x, torch.zeros(4, 4, dtype=torch.uint8), x, 32),
                 lambda: g.grad_norm([x]), lambda: g.clip_grads([x], 1.0)):
        with pytest.raises(TypeError):
            call()
    for limit in (-1.0, math.nan):
        with pytest.raises(ValueError):
            g.clip_grads([], limit)
