"""Many calls on the same inputs give the same bits. A copy that refills shared
memory before the last reads of it are done, or a use of a value before it has
arrived, shows in a few calls of hundreds: single calls of a test pass."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g(gemm_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return gemm_lib


def uniform(shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, generator=gen, device="cuda") * 2 - 1


def differing(call, out, calls):
    """Of `calls` calls that write out, how many gave other bits than the first."""
    call()
    first, count = out.clone(), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(calls):
        out.fill_(float("nan"))
        call()
        count += (out.view(torch.int32) != first.view(torch.int32)).any()
    return int(count)


@pytest.mark.parametrize("m, n, k, calls", [(4096, 4096, 4096, 1500), (2048, 2048, 2048, 1000),
                                            (1000, 1531, 777, 1000), (512, 512, 512, 500)], ids=str)
@pytest.mark.parametrize("transa, transb", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("mode", ["exact", "tf32"])
def test_gemm_repeats_its_bits(g, mode, transa, transb, m, n, k, calls):
    a = uniform((k, m) if transa else (m, k), 1)
    b = uniform((n, k) if transb else (k, n), 2)
    out = torch.empty(m, n, device="cuda")
    assert differing(lambda: g.gemm(a, b, out=out, transa=transa, transb=transb, mode=mode),
                     out, calls if mode == "exact" else calls // 5) == 0
    c64 = (a.t() if transa else a)[:64].double() @ (b.t() if transb else b).double()
    s64 = (a.t() if transa else a)[:64].double().abs() @ (b.t() if transb else b).double().abs()
    bound = 2 * k * 2.0 ** -24 if mode == "exact" else 2 * k * 2.0 ** -11
    assert ((out[:64].double() - c64).abs() <= bound * s64).all()


@pytest.mark.parametrize("calls", [1500])
def test_scaled_gemm_repeats_its_bits(g, calls):
    a, b, c0 = uniform((4096, 4096), 3), uniform((4096, 4096), 4), uniform((4096, 4096), 5)
    out = torch.empty_like(c0)

    def call():
        out.copy_(c0)
        g.gemm(a, b, out=out, alpha=1.25, beta=-0.5, transb=True)

    assert differing(call, out, calls) == 0


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("k", [777, 2048])
def test_segmented_products_repeat_their_bits(g, dt, k):
    m, n, r = 2048, 2048, 16
    off = torch.tensor([0, 500, 500, 1531, 2048], device="cuda")
    x, dy, w = uniform((m, k), 6).to(dt), uniform((m, n), 7).to(dt), uniform((4, k, n), 8).to(dt)
    wt = w.transpose(1, 2).contiguous()
    a, b = uniform((4, k, r), 9).to(dt), uniform((4, r, n), 10).to(dt)
    as_bits = lambda t: t.view(torch.int32 if dt == torch.float32 else torch.int16)
    u = torch.empty(m, r, dtype=dt, device="cuda")
    for call in (lambda: (g.grouped_matmul(x, w, off),), lambda: (g.grouped_matmul(x, wt, off, True),),
                 lambda: (g.grouped_wgrad(x, dy, off),),
                 lambda: (g.lora_matmul(x, w[0], a, b, off, shrink_out=u),),
                 lambda: g.lora_backward(dy, x, u, w[0], a, b, off)):
        first = call()
        count = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(400):
            for c, ref in zip(call(), first):
                count += (as_bits(c) != as_bits(ref)).any()
        assert int(count) == 0
