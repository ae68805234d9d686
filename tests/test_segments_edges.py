"""Segmented products, what needs no GPU: sizes and arguments at the edges of
what the entry points take."""

from test_segments import NO_GPU, PA, PB, PC, PI, PO, PU, PW, g, lora, no_gpu


def test_a_bank_without_adapters_checks_the_shrink_it_writes():
    empty = dict(bank=0, A=0, B=0, scales=0)
    assert lora(**empty, U=PU + 2) == g.ERR_INVALID_ARG
    assert lora(**empty, ldu=7) == g.ERR_INVALID_ARG
    assert lora(**empty, offsets=0) == g.ERR_INVALID_ARG
    for taken in (PA, PC, PO):
        assert lora(**empty, U=taken) == g.ERR_ALIAS
    assert lora(**empty, U=0, offsets=0, N=0, ldw=1, ldy=1) == g.OK  # nothing to write


@no_gpu
def test_a_bank_without_adapters_has_a_shrink_to_write():
    assert lora(bank=0, A=0, B=0, scales=0) in NO_GPU
    assert lora(bank=0, A=0, B=0, scales=0, N=0, ldw=1, ldy=1) in NO_GPU


def lora_backward(**kw):
    a = dict(type=0, transw=0, transl=0, segments=4, M=64, N=32, K=48, R=8, dY=PC, lddy=32, X=PA,
             ldx=48, U=PU, ldu=8, W=PW, ldw=32, A=PB, lda=8, stridea=48 * 8, B=PB + (1 << 20), ldb=32,
             strideb=8 * 32, offsets=PO, scales=PI, dX=PA + (1 << 20), lddx=48, dA=PA + (2 << 20),
             ldda=8, strideda=48 * 8, dB=PA + (3 << 20), lddb=32, stridedb=8 * 32)
    a.update(kw)
    return g.gemm_f32_lora_backward(*a.values())


def test_gradients_without_elements_make_no_cuda_call():
    none = dict(K=0, X=0, W=0, A=0, dX=0, dA=0)
    assert lora_backward(**none, R=0, U=0, B=0, dB=0) == g.OK
    assert lora_backward(**none, segments=0, offsets=0, U=0, B=0, dB=0, scales=0) == g.OK
    assert lora_backward(**none, N=0, dY=0, B=0, dB=0) == g.OK
    assert lora_backward(M=0, R=0, X=0, dY=0, U=0, A=0, B=0, dX=0, dA=0, dB=0) == g.OK


@no_gpu
def test_gradients_with_elements_are_computed():
    assert lora_backward() in NO_GPU
    assert lora_backward(K=0, X=0, W=0, A=0, dX=0, dA=0) in NO_GPU  # dB
    assert lora_backward(N=0, dY=0, W=0, B=0, dB=0) in NO_GPU       # dX, dA: zeros
    assert lora_backward(M=0, X=0, dY=0, U=0, dX=0) in NO_GPU       # dA, dB: zeros
