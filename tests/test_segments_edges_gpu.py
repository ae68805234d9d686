"""Segmented products on the GPU at the edges of what they take: factors shared
by all adapters, the ends of the types' range, banks without adapters, routing
that sends every row one way. Checks and tolerances are those of
test_segments_gpu.py."""

import pytest
import torch

from test_segments_gpu import TYPES, check, ids, lora_64, normal, offsets_of, product, rounding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g(gemm_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return gemm_lib


# 128 rows a segment and more: the adapter's half in the projection's own
# accumulators (float32 where the tiles fill the GPU once: 2560 columns at 4096
# rows); few rows a segment: a product of its own; eight rows: plain FMAs.
SHARED = [([300, 200, 157, 300], 136, 264, 24), ([1500, 700, 0, 1900], 200, 2560, 40),
          ([40, 30, 3, 9], 72, 131, 16), ([1, 2, 0, 3], 512, 264, 8)]


@pytest.mark.parametrize("shared", ["a", "b", "both"])
@pytest.mark.parametrize("sizes, k, n, r", SHARED, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_lora_with_a_factor_shared_by_all_adapters(g, sizes, k, n, r, shared, trans, dt):
    m, bank = sum(sizes), len(sizes)
    off, o = offsets_of(sizes)
    x, w = normal((m, k), 1, dt), normal((n, k) if trans else (k, n), 2, dt)
    a = normal((bank, r, k) if trans else (bank, k, r), 3, dt)
    b = normal((bank, n, r) if trans else (bank, r, n), 4, dt)
    if shared != "b":
        a = a[:1].expand_as(a)
    if shared != "a":
        b = b[:1].expand_as(b)
    scales = torch.rand(bank, device="cuda") + 0.5
    at, bt = [t.t() if trans else t for t in a], [t.t() if trans else t for t in b]
    u = torch.empty(m, r, dtype=dt, device="cuda")
    y = g.lora_matmul(x, w, a, b, off, None, scales, trans, trans, shrink_out=u)
    y64, ty, _, _ = lora_64(x, w.t() if trans else w, at, bt, o, range(bank), scales)
    check(y, y64, ty, "y")
    dy = normal((m, n), 5, dt)
    dx = g.lora_backward(dy, x, u, w, a, b, off, scales, trans, trans)[0]
    x64, tx, _, _ = lora_64(dy, w if trans else w.t(), [t.t() for t in bt], [t.t() for t in at], o,
                            range(bank), scales)
    check(dx, x64, tx, "dx")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_every_device_of_a_process(g, dt):
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    for d in range(2):
        with torch.cuda.device(d):
            off, o = offsets_of([40, 50])
            a, b = normal((90, 64), 31, dt), normal((2, 64, 80), 32, dt)
            c64, s64 = product(a[:40], b[0])
            c = g.grouped_matmul(a, b, off)
            check(c[:40], c64, rounding(c64, s64, 64, dt))
            g.grouped_wgrad(a, c, off)
