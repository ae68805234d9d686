"""Segmented products (include/segment_gemm_f32.h), what needs no GPU: the
entry points refuse bad arguments before any CUDA call, and the Python
wrappers refuse tensors the library cannot address."""

import pytest
import torch

import dense_fp32_gemm_major_gb300 as g

# Fake, never dereferenced, 256-byte aligned "device" addresses.
PA, PB, PC, PO, PU, PW, PI = (0x10000000 * i for i in range(1, 8))
# what a valid call returns without a GPU
NO_GPU = (g.ERR_LAUNCH, g.ERR_UNSUPPORTED_DEVICE)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is present")


def grouped(**kw):
    a = dict(type=0, transb=0, groups=4, M=64, N=32, K=48, A=PA, lda=48, B=PB, ldb=32,
             strideb=48 * 32, C=PC, ldc=32, offsets=PO)
    a.update(kw)
    return g.gemm_f32_grouped(*a.values())


def wgrad(**kw):
    a = dict(type=0, groups=4, M=64, N=32, K=48, A=PA, lda=48, D=PB, ldd=32, C=PC, ldc=32,
             stridec=48 * 32, offsets=PO)
    a.update(kw)
    return g.gemm_f32_grouped_wgrad(*a.values())


def lora(**kw):
    a = dict(type=0, transw=0, transl=0, segments=4, bank=6, M=64, N=32, K=48, R=8, X=PA, ldx=48,
             W=PW, ldw=32, A=PB, lda=8, stridea=48 * 8, B=PB + (1 << 20), ldb=32, strideb=8 * 32,
             offsets=PO, index=PI, scales=PI + 4096, U=PU, ldu=8, Y=PC, ldy=32)
    a.update(kw)
    return g.gemm_f32_lora(*a.values())


@pytest.mark.parametrize("kw", [
    dict(type=2), dict(type=-1), dict(transb=2), dict(groups=-1), dict(groups=g.MAX_SEGMENTS + 1),
    dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(lda=47), dict(ldb=31), dict(ldc=31),
    dict(transb=1, ldb=47), dict(strideb=-1), dict(A=0), dict(B=0), dict(C=0), dict(offsets=0),
    dict(A=PA + 2), dict(C=PC + 1), dict(type=1, B=PB + 1), dict(offsets=PO + 4),
    dict(M=(1 << 31) - 1, lda=(1 << 31) - 1), dict(strideb=1 << 44),
])
def test_grouped_refuses(kw):
    assert grouped(**kw) == g.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(type=7), dict(groups=-1), dict(M=-1), dict(lda=47), dict(ldd=31), dict(ldc=31),
    dict(stridec=47 * 32 + 31), dict(A=0), dict(D=0), dict(C=0), dict(offsets=0), dict(D=PB + 2),
])
def test_wgrad_refuses(kw):
    assert wgrad(**kw) == g.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(type=7), dict(transw=3), dict(transl=-1), dict(segments=g.MAX_SEGMENTS + 1),
    dict(bank=-1), dict(R=-1), dict(ldx=47), dict(ldw=31), dict(lda=7), dict(ldb=31), dict(ldu=7),
    dict(ldy=31), dict(transl=1, lda=47), dict(X=0), dict(W=0), dict(A=0), dict(B=0), dict(Y=0),
    dict(offsets=0), dict(index=PI + 2), dict(scales=PI + 1), dict(U=PU + 2), dict(stridea=-8),
])
def test_lora_refuses(kw):
    assert lora(**kw) == g.ERR_INVALID_ARG


@pytest.mark.parametrize("call, kw", [
    (grouped, dict(C=PA)), (grouped, dict(C=PB + 4 * (4 * 48 * 32 - 1))), (grouped, dict(C=PO + 32)),
    (wgrad, dict(C=PB)), (wgrad, dict(C=PA + 4)), (wgrad, dict(C=PO - 4 * 48 * 32 * 4 + 4)),
    (lora, dict(Y=PU)), (lora, dict(U=PA)), (lora, dict(U=PW)), (lora, dict(Y=PI)),
    (lora, dict(Y=PB + 16)), (lora, dict(U=PI + 4096)),
])
def test_aliases_are_refused(call, kw):
    assert call(**kw) == g.ERR_ALIAS


def test_nothing_to_do_makes_no_cuda_call():
    assert grouped(M=0, A=0, C=0) == g.OK
    assert grouped(N=0, B=0, C=0, ldb=1, ldc=1) == g.OK
    assert grouped(groups=0, B=0, offsets=0) == g.OK
    assert wgrad(groups=0, C=0, offsets=0) == g.OK
    assert wgrad(N=0, D=0, C=0, ldd=1, ldc=1) == g.OK
    assert lora(M=0, X=0, Y=0, U=0) == g.OK


@no_gpu
def test_valid_calls_fail_cleanly_without_a_gpu():
    assert grouped() in NO_GPU
    assert grouped(type=1, transb=1, ldb=48, A=PA + 2) in NO_GPU
    assert grouped(strideb=0) in NO_GPU
    assert grouped(K=0, A=0, B=0) in NO_GPU  # zeros
    assert wgrad(M=0, A=0, D=0) in NO_GPU    # zeros
    assert lora(index=0, scales=0) in NO_GPU
    assert lora(R=0, A=0, B=0, U=0) in NO_GPU
    assert lora(segments=0, offsets=0, index=0) in NO_GPU


def test_wrappers_refuse_what_is_not_on_a_gpu():
    x, w, o = torch.zeros(4, 8), torch.zeros(2, 8, 4), torch.tensor([0, 2, 4])
    with pytest.raises(TypeError):
        g.grouped_matmul(x, w, o)
    with pytest.raises(TypeError):
        g.grouped_wgrad(x, x, o)
    with pytest.raises(TypeError):
        g.lora_matmul(x, w[0], w, w, o)
    with pytest.raises(TypeError):
        g.lora_backward(x, x, x, w[0], w, w, o)


def test_stack_addressing():
    at = lambda t: g._addressing(t.shape, t.stride(), "t")
    t = torch.zeros(3, 5, 8)
    assert at(t) == (8, 40) and at(t[0]) == (8, 0)
    assert at(t[:, :, :3]) == (8, 40)
    assert at(t[:, :1]) == (8, 40) and at(t[:1]) == (8, 0) and at(t[1:, :1, :3]) == (3, 40)
    assert at(torch.zeros(5, 8).expand(3, 5, 8)) == (8, 0)
    assert at(torch.zeros(0, 8)) == (8, 0) and at(torch.zeros(4, 0)) == (1, 0)
    for bad in (torch.zeros(5, 8).t(), torch.zeros(1, 8).expand(5, 8),
                torch.zeros(64).as_strided((2, 5, 8), (0, 4, 1))):
        with pytest.raises(ValueError):
            at(bad)
