"""Segmented products, what needs no GPU: sizes and arguments at the edges of
what the entry points take."""

import pytest

from test_segments import NO_GPU, PA, PB, PC, PI, PO, PU, PW, g, grouped, lora, no_gpu, wgrad


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


# One size at a time, the others 1; huge matrices lie apart in the address space.
TOP = g.MAX_SEGMENT_SIZE
FAR = 1 << 44


def sized(call, size, value):
    """The call with this value for one size, its matrices without padding."""
    d = dict(M=1, N=1, K=1, R=1)
    d[size] = value
    columns = {grouped: dict(A="K", B="N", C="N"), wgrad: dict(A="K", D="N", C="N"),
               lora: dict(X="K", W="N", A="R", B="N", U="R", Y="N"),
               lora_backward: dict(dY="N", X="K", U="R", W="N", A="R", B="N", dX="K", dA="R", dB="N")}
    args = {}
    for i, (name, cols) in enumerate(columns[call].items()):
        args[name], args["ld" + name.lower()] = (i + 1) * FAR, d[cols]
    args.update({grouped: dict(groups=1, strideb=0), wgrad: dict(groups=1, stridec=0),
                 lora: dict(segments=1, bank=1, stridea=0, strideb=0),
                 lora_backward: dict(segments=1)}[call])
    if call in (grouped, wgrad):
        d.pop("R")
    return call(**args, **d)


@pytest.mark.parametrize("call", [grouped, wgrad, lora, lora_backward])
def test_sizes_stay_clear_of_32_bits(call):
    # sums of a size, a tile and the number of tiles are 32-bit
    for size in "MNKR" if call in (lora, lora_backward) else "MNK":
        for value in (TOP + 1, (1 << 31) - 1, 1 << 31):
            assert sized(call, size, value) == g.ERR_INVALID_ARG, (size, value)


@no_gpu
@pytest.mark.parametrize("call", [grouped, wgrad, lora, lora_backward])
def test_the_largest_sizes_are_taken(call):
    for size in "MNKR" if call in (lora, lora_backward) else "MNK":
        assert sized(call, size, TOP) in NO_GPU, size


def test_no_sum_of_the_kernels_passes_32_bits():
    # a size, the widest tile, the most tiles of it there are (64 rows each), and
    # the longest stretch of a contraction that is staged at a time
    assert TOP + TOP // 64 + 256 < 1 << 31 and TOP + 8192 < 1 << 31
    # blocks of three passes, times the most items that one tile is split into
    assert 3 * (TOP // 64 + 1) * 16 < 1 << 31
