"""Segmented products, what needs no GPU: sizes and arguments at the edges of
what the entry points take."""

from test_segments import NO_GPU, PA, PC, PO, PU, g, lora, no_gpu


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
