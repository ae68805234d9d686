"""Segmented products on the GPU against the sums' definition in 64 bits.

Tolerances, per element, from the operators' statements (S: the sum of the
absolute products behind an element; K: its length):

  float32    2 K 2^-24 S                     FP32 class; one more rounding of
             2^-24 |C| for sums of one or two products
  bfloat16   2^-8 |C| + (K + 2) 2^-23 S      one rounding to bf16 (unit roundoff
             2^-9, doubled where C itself is off) of an fp32 sum, whose adds may
             truncate

An adapter's term passes through U = s (x A): its error, bounded the same way
(s is one more product), reaches the result times |B|.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]
ids = {torch.float32: "f32", torch.bfloat16: "bf16"}.get


@pytest.fixture(scope="module")
def g(gemm_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return gemm_lib


def normal(shape, seed, dt, pad=0, lead=0):
    """A tensor of the shape whose rows are `pad` elements apart beyond their
    width and whose data starts `lead` elements into its buffer; the gaps hold
    NaN."""
    gen = torch.Generator().manual_seed(seed)
    rows, cols = 1, shape[-1]
    for s in shape[:-1]:
        rows *= s
    buf = torch.full((rows * (cols + pad) + lead,), float("nan"), dtype=dt, device="cuda")
    t = buf[lead:].view(rows, cols + pad)[:, :cols].view(shape) if pad == 0 else \
        buf[lead:].view(*shape[:-1], cols + pad)[..., :cols]
    t.copy_(torch.randn(shape, generator=gen).cuda().to(dt))
    return t


def offsets_of(sizes, first=0):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int64, device="cuda"), o


def rounding(c64, s64, k, dt):
    if dt == torch.float32:
        return 2 * k * 2.0 ** -24 * s64 + 2.0 ** -24 * c64.abs()
    return 2.0 ** -8 * c64.abs() + (k + 2) * 2.0 ** -23 * s64


def check(c, c64, tol, what=""):
    err = (c.double() - c64).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
        f"{bad.nonzero()[0].tolist()}: {c[bad][0].item()} for {c64[bad][0].item()}")


def product(a, b):
    a, b = a.double(), b.double()
    return a @ b, a.abs() @ b.abs()


def check_grouped(c, a, b, o, transb, dt):
    for i in range(len(o) - 1):
        r = slice(o[i], o[i + 1])
        if o[i + 1] > o[i]:
            c64, s64 = product(a[r], b[i].t() if transb else b[i])
            check(c[r], c64, rounding(c64, s64, a.shape[1], dt), f"segment {i}")


SEGMENTS = [
    ([1], 1, 1), ([1], 16, 8), ([0, 3, 0], 64, 64), ([5, 0, 130, 1], 40, 72), ([0, 0], 8, 8),
    ([256, 255, 257], 64, 256), ([1, 2, 3, 31, 32, 33, 64, 65, 127, 128, 129], 96, 40),
    ([700, 300], 777, 301), ([17] * 70, 128, 136), ([64, 64], 2048, 520), ([3, 200], 1000, 1531),
]


@pytest.mark.parametrize("sizes, k, n", SEGMENTS, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_grouped(g, sizes, k, n, transb, dt):
    m = sum(sizes)
    off, o = offsets_of(sizes)
    a = normal((m, k), 1, dt)
    b = normal((len(sizes),) + ((n, k) if transb else (k, n)), 2, dt)
    c = g.grouped_matmul(a, b, off, transb)
    check_grouped(c, a, b, o, transb, dt)
    assert torch.equal(c, g.grouped_matmul(a, b, off, transb))


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("pad, lead", [(8, 0), (16, 8), (1, 0), (0, 1), (3, 5), (4, 4)])
def test_grouped_pitches_and_alignment(g, dt, transb, pad, lead):
    sizes, k, n = [33, 0, 100], 88, 104
    off, o = offsets_of(sizes)
    a = normal((133, k), 3, dt, pad, lead)
    b = normal((3,) + ((n, k) if transb else (k, n)), 4, dt, pad, lead)
    c = normal((133, n), 5, dt, pad, lead)
    gaps = c._base.isnan().sum().item()
    assert g.grouped_matmul(a, b, off, transb, out=c) is c
    check_grouped(c, a, b, o, transb, dt)
    assert c._base.isnan().sum().item() == gaps == c._base.numel() - c.numel()  # pitch and lead untouched


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_grouped_stack_strides(g, dt):
    off, o = offsets_of([40, 0, 50])
    a = normal((90, 64), 6, dt)
    every = normal((6, 64, 96), 7, dt)
    for b in (every[::2], every[:1].expand(3, 64, 96), every[1:4, :, 8:72]):
        check_grouped(g.grouped_matmul(a, b, off), a, b, o, False, dt)
    b = every[:3, 8:40]  # 32 x 96, read transposed
    x = normal((90, 96), 8, dt)
    check_grouped(g.grouped_matmul(x, b, off, True), x, b, o, True, dt)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_grouped_rows_of_no_segment_are_left_alone(g, dt):
    a, b = normal((100, 64), 9, dt), normal((2, 64, 80), 10, dt)
    c = torch.full((100, 80), 7.0, dtype=dt, device="cuda")
    off, o = offsets_of([30, 41], first=11)
    g.grouped_matmul(a, b, off, out=c)
    check_grouped(c, a, b, o, False, dt)
    assert (c[:11] == 7).all() and (c[82:] == 7).all()
    # offsets outside the rows are held to them
    wild = torch.tensor([-5, 20, 1 << 40], dtype=torch.int64, device="cuda")
    c = g.grouped_matmul(a, b, wild)
    check_grouped(c, a, b, [0, 20, 100], False, dt)
    falling = torch.tensor([50, 20, 60], dtype=torch.int64, device="cuda")
    c.fill_(7.0)
    g.grouped_matmul(a, b, falling, out=c)
    c64, s64 = product(a[20:60], b[1])
    check(c[20:60], c64, rounding(c64, s64, 64, dt))
    assert (c[:20] == 7).all() and (c[60:] == 7).all()


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_grouped_keeps_nan_and_infinity_where_they_are(g, dt, bad):
    sizes, k, n = [37, 90, 20], 130, 70
    off, o = offsets_of(sizes)
    a, b = normal((147, k), 11, dt), normal((3, k, n), 12, dt)
    a[50] = bad
    b[2, 5, 9] = bad
    c = g.grouped_matmul(a, b, off)
    assert not c[50].isfinite().any() and not c[127:, 9].isfinite().any()
    c[50], a[50] = 0, 0
    c[127:, 9], b[2, :, 9] = 0, 0
    check_grouped(c, a, b, o, False, dt)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_grouped_without_a_contraction_is_zero(g, dt):
    off, _ = offsets_of([2, 3])
    a = torch.empty(6, 0, dtype=dt, device="cuda")
    b = torch.empty(2, 0, 9, dtype=dt, device="cuda")
    c = torch.full((6, 9), 7.0, dtype=dt, device="cuda")
    g.grouped_matmul(a, b, off, out=c)
    assert (c[:5] == 0).all() and (c[5:] == 7).all()
    assert g.grouped_matmul(a[:0], b, offsets_of([0, 0])[0]).shape == (0, 9)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("sizes, k, n", [([1], 9000, 24), ([2, 0, 1], 8200, 70), ([4, 1], 4200, 512),
                                         ([0, 7], 2100, 33), ([1, 1, 0, 1], 6, 700)],
                         ids=lambda v: str(v))
def test_grouped_few_rows(g, sizes, k, n, transb, dt):
    # single tokens and a few more, contractions longer than what is staged
    off, o = offsets_of(sizes)
    a = normal((o[-1], k), 73, dt)
    b = normal((len(sizes),) + ((n, k) if transb else (k, n)), 74, dt)
    c = g.grouped_matmul(a, b, off, transb)
    check_grouped(c, a, b, o, transb, dt)
    assert torch.equal(c, g.grouped_matmul(a, b, off, transb))


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_as_many_segments_as_a_call_takes(g, dt):
    sizes = [i % 4 + (i % 97 == 0) * 30 for i in range(g.MAX_SEGMENTS)]
    off, o = offsets_of(sizes)
    a, b = normal((o[-1], 72), 75, dt), normal((g.MAX_SEGMENTS, 72, 24), 76, dt)
    c = g.grouped_matmul(a, b, off)
    rows = torch.repeat_interleave(torch.arange(g.MAX_SEGMENTS), torch.tensor(sizes)).cuda()
    c64 = torch.einsum("tk,tkn->tn", a.double(), b.double()[rows])
    s64 = torch.einsum("tk,tkn->tn", a.double().abs(), b.double().abs()[rows])
    check(c, c64, rounding(c64, s64, 72, dt))
    d = normal((o[-1], 24), 77, dt)
    w = g.grouped_wgrad(a, d, off)
    for i in (0, 1, 97, 1000, 2046, 2047):
        c64, s64 = product(a[o[i]:o[i + 1]].t(), d[o[i]:o[i + 1]])
        check(w[i], c64, rounding(c64, s64, sizes[i], dt))
    assert (w[4] == 0).all() and (w[2044] == 0).all()  # empty segments


@pytest.mark.parametrize("k", [256, 4096, 16384])
def test_long_sums_are_as_exact_as_fp32(g, k):
    # Each of K adds rounded to nearest is off by at most 2^-24 of the running
    # sum, which grows as the root of its length: in the 2-norm, over many
    # results, sqrt(K) 2^-24 / sqrt(6) = 0.82 sqrt(K) 2^-25. Sums that truncate
    # drift as K and leave that behind from K of a few thousand on.
    a, b = normal((96, k), 13, torch.float32), normal((1, k, 128), 14, torch.float32)
    off, _ = offsets_of([96])
    c64, _ = product(a, b[0])
    err = (g.grouped_matmul(a, b, off).double() - c64).norm() / c64.norm()
    assert err <= k ** 0.5 * 2.0 ** -25


def test_fp32_range(g):
    # products of large and small magnitudes keep the FP32 class
    a, b = normal((70, 96), 15, torch.float32), normal((1, 96, 64), 16, torch.float32)
    a *= 2.0 ** torch.arange(-40, 56, device="cuda").float()
    b[0] *= 2.0 ** -torch.arange(-40, 56, device="cuda").float()[:, None]
    off, o = offsets_of([70])
    check_grouped(g.grouped_matmul(a, b, off), a, b, o, False, torch.float32)


def test_results_beyond_32_bit_offsets(g):
    # 2.4e9 results of bf16: element offsets pass 2^31
    m, n, k = 60_000, 40_000, 16
    a, b = normal((m, k), 17, torch.bfloat16), normal((2, k, n), 18, torch.bfloat16)
    off, o = offsets_of([100, m - 100])
    c = g.grouped_matmul(a, b, off)
    for r in (slice(0, 40), slice(90, 110), slice(m - 70, m)):
        for i in (0, 1):
            q = slice(max(r.start, o[i]), min(r.stop, o[i + 1]))
            if q.start < q.stop:
                c64, s64 = product(a[q], b[i])
                check(c[q], c64, rounding(c64, s64, k, torch.bfloat16))


@pytest.mark.parametrize("sizes, k, n", SEGMENTS, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_wgrad(g, sizes, k, n, dt):
    m = sum(sizes)
    off, o = offsets_of(sizes)
    a, d = normal((m, k), 21, dt), normal((m, n), 22, dt)
    c = g.grouped_wgrad(a, d, off)
    assert c.shape == (len(sizes), k, n)
    for i, s in enumerate(sizes):
        c64, s64 = product(a[o[i]:o[i + 1]].t(), d[o[i]:o[i + 1]])
        check(c[i], c64, rounding(c64, s64, s, dt), f"segment {i}")
    assert torch.equal(c, g.grouped_wgrad(a, d, off))


@pytest.mark.parametrize("sizes, k, n", [([3001, 50], 64, 96), ([2500, 2100], 300, 520),
                                         ([5000], 24, 17)], ids=lambda v: str(v))
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_wgrad_long_segments(g, sizes, k, n, dt):
    # few tiles and long sums: several work items a tile
    off, o = offsets_of(sizes)
    a, d = normal((o[-1], k), 26, dt), normal((o[-1], n), 27, dt)
    c = g.grouped_wgrad(a, d, off)
    for i, s in enumerate(sizes):
        c64, s64 = product(a[o[i]:o[i + 1]].t(), d[o[i]:o[i + 1]])
        check(c[i], c64, rounding(c64, s64, s, dt), f"segment {i}")
    assert torch.equal(c, g.grouped_wgrad(a, d, off))


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("pad, lead", [(8, 0), (1, 0), (0, 1), (3, 5), (4, 4)])
def test_wgrad_pitches_and_neighbours(g, dt, pad, lead):
    # NaN and infinity in the rows beside a segment stay out of its sums
    sizes, k, n = [21, 0, 77, 16], 72, 136
    off, o = offsets_of(sizes, first=3)
    a, d = normal((120, k), 23, dt, pad, lead), normal((120, n), 24, dt, pad, lead)
    a[:3], d[:3], a[117:], d[117:] = float("nan"), float("inf"), float("inf"), float("nan")
    a[30] = float("nan")
    d[40] = float("inf")
    c = normal((4, k, n), 25, dt, pad, lead)
    gaps = c._base.isnan().sum().item()
    g.grouped_wgrad(a, d, off, out=c)
    assert (c[1] == 0).all() and not c[2].isfinite().any()
    for i in (0, 3):
        c64, s64 = product(a[o[i]:o[i + 1]].t(), d[o[i]:o[i + 1]])
        check(c[i], c64, rounding(c64, s64, sizes[i], dt))
    c[2] = 0
    assert c._base.isnan().sum().item() == gaps


def lora_64(x, w, a, b, o, which, scales):
    """(y, its tolerance's parts) of lora_matmul in 64 bits; a, b: lists of K x R and R x N."""
    y, sy = product(x, w)
    extra = torch.zeros_like(y)
    u = torch.zeros(x.shape[0], a[0].shape[1], dtype=torch.float64, device="cuda")
    tu = torch.zeros_like(u)
    for i, z in enumerate(which):
        if not 0 <= z < len(a) or o[i + 1] <= o[i]:
            continue
        r = slice(o[i], o[i + 1])
        f = scales[z].item()
        u64, s64 = product(x[r], a[z])
        u[r] = f * u64
        tu[r] = rounding(f * u64, abs(f) * s64, x.shape[1] + 1, x.dtype)
        y64, sl = product(u[r], b[z])
        y[r] += y64
        sy[r] += sl
        extra[r] = tu[r] @ b[z].double().abs()
    return y, rounding(y, sy, x.shape[1] + u.shape[1], x.dtype) + extra, u, tu


LORA = [  # sizes, adapters (None: one each), bank, K, N, R
    ([1], [0], 1, 16, 8, 4), ([1], [2], 4, 512, 512, 8), ([0, 5], None, 2, 64, 64, 16),
    ([1] * 33, [i % 7 - 1 for i in range(33)], 5, 256, 264, 16),
    ([100, 0, 157, 300], [3, 1, -1, 3], 4, 136, 520, 64), ([40, 30], None, 2, 77, 131, 3),
    ([64, 64, 128, 256, 1], [0, 1, 2, 1, 9], 3, 128, 256, 200), ([129], [0], 1, 1000, 301, 1),
    ([7] * 60, [i % 9 for i in range(60)], 9, 96, 72, 24),
    ([1500, 700, 0, 1900], [1, -1, 0, 2], 3, 200, 2560, 40), ([900, 1100], None, 2, 1000, 264, 130),
]


@pytest.mark.parametrize("sizes, which, bank, k, n, r", LORA, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("trans", ["nn", "tn", "nt", "tt"])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_lora(g, sizes, which, bank, k, n, r, trans, dt):
    m = sum(sizes) + 3  # the last rows belong to no segment
    off, o = offsets_of(sizes)
    transw, transl = trans[0] == "t", trans[1] == "t"
    x, w = normal((m, k), 31, dt), normal((n, k) if transw else (k, n), 32, dt)
    a = normal((bank, r, k) if transl else (bank, k, r), 33, dt)
    b = normal((bank, n, r) if transl else (bank, r, n), 34, dt)
    scales = torch.rand(bank, device="cuda") + 0.5
    index = None if which is None else torch.tensor(which, dtype=torch.int32, device="cuda")
    u = torch.full((m, r), 7.0, dtype=dt, device="cuda")
    y = g.lora_matmul(x, w, a, b, off, index, scales, transw, transl, shrink_out=u)
    y64, ty, u64, tu = lora_64(x, w.t() if transw else w, [t.t() if transl else t for t in a],
                               [t.t() if transl else t for t in b], o,
                               which or list(range(len(sizes))), scales)
    check(y, y64, ty, "y")
    check(u[:o[-1]], u64[:o[-1]], tu[:o[-1]], "u")
    assert (u[o[-1]:] == 7).all()
    # without shrink_out the same sums, bit for bit
    assert torch.equal(y, g.lora_matmul(x, w, a, b, off, index, scales, transw, transl))


@pytest.mark.parametrize("sizes, first, m, k, n, r", [
    ([1, 3], 2, 8, 1024, 2048, 16), ([3, 0, 4], 0, 8, 640, 4400, 8), ([1] * 6, 1, 8, 4096, 1000, 24),
    ([5], 1, 8, 200, 11008, 3), ([1, 0, 1], 1, 3, 1500, 1531, 40), ([2], 0, 2, 130, 9000, 16)],
    ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_lora_few_rows(g, sizes, first, m, k, n, r, trans, dt):
    # rows before and behind the segments share CTAs with rows in them
    off, o = offsets_of(sizes, first)
    x, w = normal((m, k), 91, dt), normal((n, k) if trans else (k, n), 92, dt)
    a = normal((len(sizes), r, k) if trans else (len(sizes), k, r), 93, dt)
    b = normal((len(sizes), n, r) if trans else (len(sizes), r, n), 94, dt)
    one = torch.ones(len(sizes), device="cuda")
    y = g.lora_matmul(x, w, a, b, off, transw=trans, transl=trans)
    y64, ty, _, _ = lora_64(x, w.t() if trans else w, [t.t() if trans else t for t in a],
                            [t.t() if trans else t for t in b], o, list(range(len(sizes))), one)
    check(y, y64, ty, "y")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_lora_without_adapters_is_the_projection(g, dt):
    x, w = normal((50, 64), 35, dt), normal((64, 72), 36, dt)
    y64, s64 = product(x, w)
    none = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    off, _ = offsets_of([20, 25])
    a, b = normal((3, 64, 8), 37, dt), normal((3, 8, 72), 38, dt)
    a.fill_(float("nan"))  # never read
    for y in (g.lora_matmul(x, w, a, b, off, none),
              g.lora_matmul(x, w, a, b, offsets_of([])[0]),
              g.lora_matmul(x, w, a[:0], b[:0], off, none),
              g.lora_matmul(x, w, a[:, :, :0], b[:, :0], off, none)):
        check(y, y64, rounding(y64, s64, 64, dt))


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_lora_keeps_segments_apart(g, dt):
    # a NaN in one request's rows, or in an adapter of its own, reaches no other
    sizes, which = [3, 40, 1, 30], [0, 1, 2, 0]
    off, o = offsets_of(sizes)
    x, w = normal((74, 96), 41, dt), normal((96, 80), 42, dt)
    a, b = normal((3, 96, 16), 43, dt), normal((3, 16, 80), 44, dt)
    scales = torch.ones(3, device="cuda")
    x[10], b[2, 3] = float("nan"), float("inf")
    index = torch.tensor(which, dtype=torch.int32, device="cuda")
    y = g.lora_matmul(x, w, a, b, off, index)
    assert y[10].isnan().all() and not y[43].isfinite().any()
    keep = [i for i in range(74) if i not in (10, 43)]
    x[10], b[2, 3] = 0, 0
    y64, ty, _, _ = lora_64(x, w, a, b, o, which, scales)
    check(y[keep], y64[keep], ty[keep])


BACKWARD = [([1], 16, 8, 4), ([0, 5], 64, 64, 16), ([100, 0, 157, 30], 136, 260, 24),
            ([300, 41], 77, 131, 3), ([64, 64, 128], 128, 256, 64)]


@pytest.mark.parametrize("sizes, k, n, r", BACKWARD, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("trans", ["nn", "tt"])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_lora_backward(g, sizes, k, n, r, trans, dt):
    t = trans[0] == "t"
    m, bank = sum(sizes), len(sizes)
    off, o = offsets_of(sizes)
    x, dy = normal((m, k), 51, dt), normal((m, n), 52, dt)
    w = normal((n, k) if t else (k, n), 53, dt)
    a = normal((bank, r, k) if t else (bank, k, r), 54, dt)
    b = normal((bank, n, r) if t else (bank, r, n), 55, dt)
    scales = torch.rand(bank, device="cuda") + 0.5
    u = torch.empty(m, r, dtype=dt, device="cuda")
    g.lora_matmul(x, w, a, b, off, None, scales, t, t, shrink_out=u)
    dx, da, db = g.lora_backward(dy, x, u, w, a, b, off, scales, t, t)
    at, bt = [z.t() if t else z for z in a], [z.t() if t else z for z in b]
    x64, tx, v64, tv = lora_64(dy, w if t else w.t(), [z.t() for z in bt], [z.t() for z in at], o,
                               range(bank), scales)
    check(dx, x64, tx, "dx")
    assert da.shape == a.shape and db.shape == b.shape
    for i in range(bank):
        s = slice(o[i], o[i + 1])
        da64, sa = product(x[s].t(), v64[s])
        ta = rounding(da64, sa, sizes[i], dt) + x[s].double().abs().t() @ tv[s]
        check(da[i].t() if t else da[i], da64, ta, "da")
        db64, sb = product(u[s].t(), dy[s])  # of the U that the forward returned
        check(db[i].t() if t else db[i], db64, rounding(db64, sb, sizes[i], dt), "db")


def test_gradients_against_differences(g):
    # L = sum(y * dy) is bilinear in every factor, so central differences along
    # a direction are exact up to the sums' own rounding (2-norm bound: 1e-4 of
    # the terms' magnitude for these lengths)
    dt, sizes, k, n, r = torch.float32, [30, 0, 45], 64, 96, 8
    off, _ = offsets_of(sizes)
    x, w = normal((75, k), 61, dt), normal((k, n), 62, dt)
    a, b, dy = normal((3, k, r), 63, dt), normal((3, r, n), 64, dt), normal((75, n), 65, dt)
    scales = torch.tensor([0.5, 2.0, 1.5], device="cuda")
    u = torch.empty(75, r, device="cuda")
    g.lora_matmul(x, w, a, b, off, None, scales, shrink_out=u)
    grads = g.lora_backward(dy, x, u, w, a, b, off, scales)

    def loss(x, a, b):
        y = g.lora_matmul(x, w, a, b, off, None, scales)
        return (y.double() * dy.double()).sum(), (y.double() * dy.double()).abs().sum()

    for i, grad in enumerate(grads):
        step = torch.randn(grad.shape, generator=torch.Generator().manual_seed(66 + i)).cuda()
        up, down = [x, a, b], [x, a, b]
        up[i], down[i] = up[i] + step, down[i] - step
        (lu, su), (ld, sd) = loss(*up), loss(*down)
        assert abs((lu - ld) / 2 - (grad.double() * step.double()).sum()) <= 1e-4 * (su + sd)

    e = normal((3, k, n), 67, dt)
    c = lambda e: (g.grouped_matmul(x, e, off).double() * dy.double())
    step = normal((3, k, n), 68, dt)
    up, down = c(e + step), c(e - step)
    got = (g.grouped_wgrad(x, dy, off).double() * step.double()).sum()
    assert abs((up.sum() - down.sum()) / 2 - got) <= 1e-4 * (up.abs().sum() + down.abs().sum())


def test_graph_capture_and_replay(g):
    # the workspace and its zeros are part of the capture
    off, o = offsets_of([40, 0, 25])
    x, w = normal((65, 2048), 71, torch.bfloat16), normal((2048, 96), 72, torch.bfloat16)
    a, b = normal((3, 2048, 16), 73, torch.bfloat16), normal((3, 16, 96), 74, torch.bfloat16)
    ref = g.lora_matmul(x, w, a, b, off)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.lora_matmul(x, w, a, b, off, out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(out, ref)
    x.mul_(2)  # exact in every rounding
    graph.replay()
    assert torch.equal(out, 2 * ref)


CHAINS = [([400, 0, 300, 324], 1024, 520, 16), ([200, 311, 190], 1000, 2048, 24),
          ([1] * 32, 2048, 1024, 16), ([2, 1, 0, 1], 512, 512, 8), ([900, 1100], 2048, 2048, 64)]


@pytest.mark.parametrize("sizes, k, n, r", CHAINS, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_launches_of_a_step_keep_their_order(g, sizes, k, n, r, dt):
    """Launches of a call may overlap; what one makes and the next reads, and
    the inputs that are overwritten right behind the call, keep their order: the
    same bits as one step at a time."""
    m, s = sum(sizes), len(sizes)
    off, _ = offsets_of(sizes)
    w = normal((k, n), 1, dt)
    jobs = [(normal((m, k), 10 + i, dt), normal((m, n), 20 + i, dt), normal((s, k, r), 30 + i, dt),
             normal((s, r, n), 40 + i, dt)) for i in range(4)]
    held = [t.clone() for t in jobs[0]]
    u = torch.empty((m, r), dtype=dt, device="cuda")

    def step(i, wait):
        for to, t in zip(held, jobs[i]):
            to.copy_(t)
        wait()
        x, dy, a, b = held
        y = g.lora_matmul(x, w, a, b, off, shrink_out=u)
        wait()
        out = (y,) + tuple(g.lora_backward(dy, x, u, w, a, b, off))
        wait()
        for t in held + [u]:
            t.fill_(float("nan"))
        return out

    refs = [step(i, torch.cuda.synchronize) for i in range(len(jobs))]
    outs = [(i, step(i, lambda: None)) for _ in range(8) for i in range(len(jobs))]
    for i, out in outs:
        for c, ref in zip(out, refs[i]):
            assert torch.equal(c, ref)


def test_concurrent_streams(g):
    off, o = offsets_of([64, 64])
    jobs = [(normal((128, 4096), 80 + i, torch.float32), normal((2, 4096, 192), 90 + i, torch.float32))
            for i in range(4)]
    refs = [g.grouped_matmul(a, b, off) for a, b in jobs]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in jobs], []
    for _ in range(5):
        for s, (a, b) in zip(streams, jobs):
            with torch.cuda.stream(s):
                outs.append(g.grouped_matmul(a, b, off))
    torch.cuda.synchronize()
    for i, c in enumerate(outs):
        assert torch.equal(c, refs[i % 4])


def test_streams(g):
    # offsets made on the same side stream, right before the call
    a, b = normal((400, 256), 71, torch.bfloat16), normal((4, 256, 512), 72, torch.bfloat16)
    ref = g.grouped_matmul(a, b, offsets_of([100, 100, 100, 100])[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        off = torch.arange(5, device="cuda", dtype=torch.int64) * 100
        c = g.grouped_matmul(a, b, off)
    side.synchronize()
    assert torch.equal(c, ref)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_every_access_is_inside_the_declared_extents(g, checked_lib, dt):
    lib, kind = checked_lib, g.TYPE_BF16 if dt == torch.bfloat16 else g.TYPE_F32
    s = torch.cuda.current_stream().cuda_stream
    for pad, lead in ((0, 0), (3, 1)):
        m, k, n, r = 301, 72, 137, 20
        off, _ = offsets_of([100, 0, 150, 31], first=7)
        x, d = normal((m, k), 81, dt, pad, lead), normal((m, n), 82, dt, pad, lead)
        b, w = normal((4, k, n), 83, dt, pad, lead), normal((k, n), 84, dt, pad, lead)
        la, lb = normal((4, k, r), 85, dt, pad, lead), normal((4, r, n), 86, dt, pad, lead)
        y, u = normal((m, n), 87, dt, pad, lead), normal((m, r), 88, dt, pad, lead)
        ptr = lambda t: t.data_ptr()
        ld = lambda t: g._addressing(t.shape, t.stride(), "t")[0]
        st = lambda t: g._addressing(t.shape, t.stride(), "t")[1]
        assert lib.gemm_f32_grouped(kind, 0, 4, m, n, k, ptr(x), ld(x), ptr(b), ld(b), st(b), ptr(y),
                                    ld(y), ptr(off), s) == g.OK
        assert lib.gemm_f32_grouped_wgrad(kind, 4, m, n, k, ptr(x), ld(x), ptr(d), ld(d), ptr(b),
                                          ld(b), st(b), ptr(off), s) == g.OK
        assert lib.gemm_f32_lora(kind, 0, 0, 4, 4, m, n, k, r, ptr(x), ld(x), ptr(w), ld(w), ptr(la),
                                 ld(la), st(la), ptr(lb), ld(lb), st(lb), ptr(off), None, None,
                                 ptr(u), ld(u), ptr(y), ld(y), s) == g.OK
        status, count, site, at, extent = g.gemm_f32_take_index_fault(s, lib=lib)
        assert (status, count) == (g.OK, 0), (g.gemm_f32_index_site_name(site), at, extent)


def test_wrappers_refuse(g):
    f, h = torch.float32, torch.bfloat16
    x, b = normal((8, 16), 91, f), normal((2, 16, 24), 92, f)
    off, _ = offsets_of([3, 5])
    for call, exc in [
        (lambda: g.grouped_matmul(x.half(), b, off), TypeError),
        (lambda: g.grouped_matmul(x, b.to(h), off), ValueError),
        (lambda: g.grouped_matmul(x, b[0], off), TypeError),
        (lambda: g.grouped_matmul(x, b, off[:2]), ValueError),
        (lambda: g.grouped_matmul(x, b, off.int()), TypeError),
        (lambda: g.grouped_matmul(x, b, off.cpu()), TypeError),
        (lambda: g.grouped_matmul(x, b, off, transb=True), ValueError),
        (lambda: g.grouped_matmul(x.t().contiguous().t(), b, off), ValueError),
        (lambda: g.grouped_matmul(x, b, off, out=x), ValueError),
        (lambda: g.grouped_wgrad(x, x[:5], off), ValueError),
        (lambda: g.grouped_wgrad(x, x, off, out=x.new_empty(16, 16).expand(2, 16, 16)), ValueError),
        (lambda: g.lora_matmul(x, b[0], b, b, off), ValueError),
        (lambda: g.lora_matmul(x, b[0], x.new_ones(1, 16, 4), x.new_ones(1, 4, 24), off), ValueError),
        (lambda: g.lora_matmul(x, b[0], x.new_ones(2, 16, 4), x.new_ones(2, 4, 24), off,
                               scales=x.new_ones(3)), TypeError),
        (lambda: g.lora_matmul(x, b[0], x.new_ones(2, 16, 4), x.new_ones(2, 4, 24), off,
                               adapters=off[:2]), TypeError),
        (lambda: g.lora_backward(x, x, x, b[0], b[:1], b[:1], off), ValueError),
    ]:
        with pytest.raises(exc):
            call()
    with pytest.raises(g.GemmError):  # the result on its own operand
        g.grouped_matmul(x, b[:, :, :16], off, out=x)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_example_learns(g, dt):
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_adapters.py")
    spec = importlib.util.spec_from_file_location("expert_adapters", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(dt, steps=12, tokens=700, width=128, hidden=256)
    assert all(a == a for a in losses) and losses[-1] < 0.9 * losses[0]
