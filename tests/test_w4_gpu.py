"""Products with 4-bit weights on the GPU against their definition in 64 bits.

Tolerances, per element (S: the sum of the absolute products behind an element,
K: its length), as for the other products over segments:

  float32    2 K 2^-24 S + 2^-24 |C|
  bfloat16   2^-8 |C| + (K + 2) 2^-23 S
"""

import math

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


def case(m, n, k, group, dt, zeros, groups=None, seed=1):
    gen = torch.Generator().manual_seed(seed)
    stack = () if groups is None else (groups,)
    row = stack + (n, -(-k // group))
    x = torch.randn(m, k, generator=gen).to(dt).cuda()
    q = torch.randint(256, stack + (n, (k + 1) // 2), generator=gen).to(torch.uint8).cuda()
    s = ((torch.rand(row, generator=gen) + 0.5) * torch.randn(row, generator=gen).sign() / 16).to(dt).cuda()
    z = torch.randint(256, row, generator=gen).to(torch.uint8).cuda() if zeros else None
    return x, q, s, z


def weights_64(q, s, z, k, group):
    at = torch.arange(k, device=q.device)
    v = q.long()[..., at // 2] >> (4 * (at % 2)) & 15
    zero = 8 if z is None else (z.long() & 15)[..., at // group]
    return (v - zero).double() * s.double()[..., at // group]


def check(c, x, w, dt, what="", least=0.0):
    k = x.shape[1]
    c64, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    if dt == torch.float32:
        tol = 2 * k * 2.0 ** -24 * size + 2.0 ** -24 * c64.abs()
    else:
        tol = 2.0 ** -8 * c64.abs() + (k + 2) * 2.0 ** -23 * size
    bad = ~((c.double() - c64).abs() <= tol + least)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"


SIZES = [(1, 1, 1, 32), (1, 64, 32, 32), (1, 512, 512, 128), (3, 70, 100, 32), (8, 129, 256, 64),
         (9, 64, 288, 96), (13, 301, 777, 32), (16, 200, 1000, 256), (17, 96, 640, 320), (33, 65, 520, 128), (150, 70, 300, 32),
         (70, 192, 2048, 4096), (2, 1531, 4096, 128), (5, 40, 11008, 128), (1, 8, 30000, 64)]


@pytest.mark.parametrize("m, n, k, group", SIZES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_w4(g, m, n, k, group, zeros, dt):
    x, q, s, z = case(m, n, k, group, dt, zeros)
    c = g.w4_matmul(x, q, s, group, zeros=z)
    check(c, x, weights_64(q, s, z, k, group), dt)
    assert torch.equal(c, g.w4_matmul(x, q, s, group, zeros=z))


@pytest.mark.parametrize("m, n, k, group", [(256, 64, 64, 32), (300, 301, 777, 64), (400, 700, 1024, 128)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_w4_of_many_rows(g, m, n, k, group, zeros, dt):
    x, q, s, z = case(m, n, k, group, dt, zeros)
    check(g.w4_matmul(x, q, s, group, zeros=z), x, weights_64(q, s, z, k, group), dt)


SEGMENTS = [[1], [0, 3, 0], [5, 0, 30, 1], [1] * 20, [64, 0, 9], [0, 0], [2, 7, 8, 9, 15, 16, 17, 40],
            [300, 0, 150], [900, 0, 150], [2000, 3, 0, 1]]


@pytest.mark.parametrize("sizes", SEGMENTS, ids=str)
@pytest.mark.parametrize("n, k, group", [(130, 512, 128), (65, 777, 32)])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_w4_by_segment(g, sizes, n, k, group, dt):
    m, starts = sum(sizes) + 3, [2]
    for size in sizes:
        starts.append(starts[-1] + size)
    x, q, s, z = case(m, n, k, group, dt, True, len(sizes))
    x[:2] = math.nan  # rows of no segment
    x[m - 1:] = math.nan
    out = torch.full((m, n), 7.0, dtype=dt, device="cuda")
    assert g.w4_matmul(x, q, s, group, zeros=z, offsets=torch.tensor(starts).cuda(), out=out) is out
    assert (out[:2] == 7).all() and (out[m - 1:] == 7).all()
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        check(out[a:b], x[a:b], weights_64(q[i], s[i], z[i], k, group), dt, f"segment {i}")


@pytest.mark.parametrize("m", [6, 1000])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_offsets_outside_the_rows_are_held_to_them(g, dt, m):
    x, q, s, _ = case(m, 40, 128, 32, dt, False, 3)
    wild = torch.tensor([-(1 << 62), 2, 1, 1 << 62]).cuda()
    out = torch.full((m, 40), 7.0, dtype=dt, device="cuda")
    g.w4_matmul(x, q, s, 32, offsets=wild, out=out)
    check(out[:1], x[:1], weights_64(q[0], s[0], None, 128, 32), dt)
    # (row 1 is claimed by two segments)
    check(out[2:], x[2:], weights_64(q[2], s[2], None, 128, 32), dt)


@pytest.mark.parametrize("m", [1, 2, 5, 600])
@pytest.mark.parametrize("pad, lead", [(16, 0), (16, 16), (3, 0), (0, 1), (8, 8)])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_pitches_and_alignment(g, dt, m, pad, lead):
    n, k, group = 100, 256, 64
    x, q, s, z = case(m, n, k, group, dt, True, 2)

    def spread(t, fill):
        cols = t.shape[-1]
        rows = t.numel() // cols
        buf = torch.full((rows * (cols + pad) + lead,), fill, dtype=t.dtype, device="cuda")
        v = buf[lead:].view(*t.shape[:-1], cols + pad)[..., :cols]
        v.copy_(t)
        return v

    off = torch.tensor([0, m // 3, m]).cuda()
    out = spread(torch.zeros(m, n, dtype=dt, device="cuda"), math.nan)
    gaps = int(out._base.isnan().sum())
    got = g.w4_matmul(spread(x, math.nan), spread(q, 255), spread(s, math.nan), group,
                      zeros=spread(z, 255), offsets=off, out=out)
    for i, (a, b) in enumerate([(0, m // 3), (m // 3, m)]):
        check(got[a:b], x[a:b], weights_64(q[i], s[i], z[i], k, group), dt)
    assert int(out._base.isnan().sum()) == gaps


@pytest.mark.parametrize("m", [4, 900])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_one_matrix_for_all_segments(g, dt, m):
    x, q, s, z = case(m, 72, 160, 32, dt, True)
    off = torch.tensor([0, 1, m // 2, m]).cuda()
    got = g.w4_matmul(x, q.expand(3, -1, -1), s.expand(3, -1, -1), 32, zeros=z.expand(3, -1, -1), offsets=off)
    check(got, x, weights_64(q, s, z, 160, 32), dt)


@pytest.mark.parametrize("m", [3, 300])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_nan_and_infinities_stay_where_they_are(g, dt, m):
    x, q, s, z = case(m, 80, 300, 32, dt, True)
    want = g.w4_matmul(x, q, s, 32, zeros=z)
    x[1, 299] = math.nan
    s[7, 3] = math.inf
    s[9, 9] = math.nan
    got = g.w4_matmul(x, q, s, 32, zeros=z)
    assert got[1].isnan().all() and not got[:, 7].isfinite().any() and not got[:, 9].isfinite().any()
    rows = [r for r in range(m) if r != 1]
    cols = [c for c in range(80) if c not in (7, 9)]
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])
    x[1, 299] = 0.0
    x[0, 5] = math.inf
    got = g.w4_matmul(x, q, s, 32, zeros=z)
    assert not got[0].isfinite().any() and got[2, cols].isfinite().all()


def test_fp32_from_the_smallest_to_the_largest(g):
    x, q, s, z = case(4, 64, 128, 32, torch.float32, True)
    w = weights_64(q, s, z, 128, 32)
    top = torch.finfo(torch.float32).max
    x[0] = 0.0
    x[0, 3] = top
    x[1] *= 2.0 ** -100
    x[2] *= 2.0 ** 100
    got = g.w4_matmul(x, q, s * 2.0 ** -8, 32, zeros=z)
    check(got, x, w * 2.0 ** -8, torch.float32)


@pytest.mark.parametrize("m", [1, 2, 4, 14, 300])
@pytest.mark.parametrize("k", [1, 3, 40, 600])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_small_values_have_all_their_bits(g, dt, m, k):
    # from 2^-110 on; in other rows and blocks of k larger ones
    n, group = 70, 32
    x, q, s, _ = case(m, n, k, group, dt, False)
    z = torch.zeros(n, -(-k // group), dtype=torch.uint8, device="cuda")
    gen = torch.Generator().manual_seed(7)
    size = torch.randint(-110, -95, (m, k), generator=gen).double().exp2()
    size[:, 256:] = torch.randint(-70, -40, size[:, 256:].shape, generator=gen).double().exp2()
    x = ((1 + torch.rand(m, k, generator=gen).double()) * size).to(dt).cuda()
    x[1::4] *= 2.0 ** 90
    x[2::4, k // 2:] = 0.0
    got = g.w4_matmul(x, q, s, group, zeros=z)
    check(got, x, weights_64(q, s, z, k, group), dt)


@pytest.mark.parametrize("m", [1, 4, 14, 300])
@pytest.mark.parametrize("large", [1.0, 2.0 ** 40])
def test_small_values_beside_large_ones_of_no_weight(g, m, large):
    # what is lost of a small value then: 2^-121 of q - z, below 2^16 so much more of it
    n, k, group = 70, 300, 32
    x, q, s, _ = case(m, n, k, group, torch.float32, False)
    z = torch.zeros(n, -(-k // group), dtype=torch.uint8, device="cuda")
    x *= torch.randint(-108, -80, (m, k), generator=torch.Generator().manual_seed(8)).double().exp2().float().cuda()
    x[:, 1::64] = large
    q[:, ::32] &= 15  # (q of the odd k)
    got = g.w4_matmul(x, q, s, group, zeros=z)
    w = weights_64(q, s, z, k, group)
    lost = k * 2.0 ** -121 * max(1.0, large * 2.0 ** -16) * s.double().abs().max()
    check(got, x, w, torch.float32, least=float(lost))


@pytest.mark.parametrize("m", [1, 2, 14, 60, 300])
@pytest.mark.parametrize("k", [2, 3, 5, 16, 33, 200])
@pytest.mark.parametrize("zeros", [0, 1, 8])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_small_values_beside_large_ones(g, dt, m, k, zeros):
    # products of few and very different values, relative to the sum of |s| (q + z) |a|
    n, group = 200, 32
    gen = torch.Generator().manual_seed(k)
    low = 2 - min(zeros, 2)  # q + z of 2 at least
    q4 = torch.randint(low, 16, (n, k + k % 2), generator=gen)
    q4[:, k:] = 0
    q = (q4[:, ::2] | q4[:, 1::2] << 4).to(torch.uint8).cuda()
    s = ((torch.rand(n, -(-k // group), generator=gen) + 0.5) / 16).to(dt).cuda()
    z = torch.full((n, -(-k // group)), zeros, dtype=torch.uint8, device="cuda")
    size = torch.randint(-26, -6, (m, k), generator=gen)
    size[torch.arange(m), torch.randint(k, (m,), generator=gen)] = 0
    sign = torch.randint(0, 2, (m, k), generator=gen) * 2 - 1
    x = (sign * (1 + torch.rand(m, k, generator=gen).double()) * size.double().exp2()).to(dt).cuda()
    got = g.w4_matmul(x, q, s, group, zeros=z).double()
    w = weights_64(q, s, z, k, group)
    all_s = s.double().abs().repeat_interleave(group, 1)[:, :k]
    c64 = x.double() @ w.t()
    size = x.double().abs() @ (all_s * (q4[:, :k].cuda() + zeros)).t()
    step = 2 * k * 2.0 ** -24 if dt == torch.float32 else (k + 2) * 2.0 ** -23
    tol = step * size + (2.0 ** -24 if dt == torch.float32 else 2.0 ** -8) * c64.abs()
    bad = ~((got - c64).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float(((got - c64).abs() / tol).max()):.3g} of the bound"


@pytest.mark.parametrize("m", [3, 300])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_large_scales(g, dt, m):
    x, q, s, z = case(m, 70, 300, 32, dt, True)
    s[::3] *= 2.0 ** 127  # 1.5 2^123 at most: 15 of them are finite
    s[1::3] *= 2.0 ** 104
    s[2::3] *= 2.0 ** -30
    x *= 2.0 ** -100
    x[2] *= 2.0 ** 100
    assert s.isfinite().all()
    w = weights_64(q, s, z, 300, 32)
    got = g.w4_matmul(x, q, s, 32, zeros=z)
    rows = [r for r in range(m) if r != 2]
    # Results of 2^-130 x: a rounding below the smallest normal value, 2^-126, is off by
    # half the smallest value of the type, and K sums of fp32 by half of 2^-149 each.
    least = torch.finfo(dt).eps * 2.0 ** -127 + 300 * 2.0 ** -150
    check(got[rows], x[rows], w, dt, least=least)
    x[2] *= 2.0 ** 17  # above 2^16, where A is scaled by less
    got = g.w4_matmul(x, q, s, 32, zeros=z)
    check(got[:, 1::3], x, w[1::3], dt)
    check(got[:, 2::3], x, w[2::3], dt, least=least)


@pytest.mark.parametrize("m", [4, 300])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_weights_near_their_zeros(g, dt, m):
    # s (sum q a - z sum a): the error is relative to the sum of |s| (q + z) |a|, the
    # products that are summed.
    n, k, group = 64, 512, 128
    x, q, s, _ = case(m, n, k, group, dt, False)
    z = torch.full((n, k // group), 15, dtype=torch.uint8, device="cuda")
    q.fill_(255)
    q[:, 7::64] = 0xEF
    got = g.w4_matmul(x, q, s, group, zeros=z)
    w = weights_64(q, s, z, k, group)
    c64 = x.double() @ w.t()
    size = x.double().abs() @ (30 * s.double().abs().repeat_interleave(group, 1)).t()
    step = 2 * k * 2.0 ** -24 if dt == torch.float32 else (k + 2) * 2.0 ** -23
    tol = step * size + (2.0 ** -24 if dt == torch.float32 else 2.0 ** -8) * c64.abs()
    assert ((got.double() - c64).abs() <= tol).all()


@pytest.mark.parametrize("sizes", [[0] * 40 + [1, 0, 2] + [0] * 20, [1] + [0] * 500 + [1]], ids=["63", "502"])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_many_segments_of_few_rows(g, dt, sizes):
    n, k, group = 70, 300, 32
    m, starts = sum(sizes), [0]
    for size in sizes:
        starts.append(starts[-1] + size)
    x, q, s, z = case(m, n, k, group, dt, True, len(sizes))
    got = g.w4_matmul(x, q, s, group, zeros=z, offsets=torch.tensor(starts).cuda())
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        check(got[a:b], x[a:b], weights_64(q[i], s[i], z[i], k, group), dt, f"segment {i}")


@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_offsets_that_change_behind_a_call_without_rows(g, dt, m):
    # nothing of a call without rows reads the offsets that the next launch writes
    n, k, group = 200, 512, 128
    x, q, s, z = case(m, n, k, group, dt, True, 3)
    experts = (torch.arange(m, device="cuda").view(m, 1) % 3).int()
    off, want = torch.zeros(4, dtype=torch.int64, device="cuda"), g.route_plan(experts, 3)[0]
    order, places = (torch.empty(m, dtype=torch.int32, device="cuda") for _ in range(2))
    stream = torch.cuda.current_stream().cuda_stream
    out = torch.full((m, n), 7.0, dtype=dt, device="cuda")
    for _ in range(20):
        off.zero_()
        g.w4_matmul(x, q, s, group, zeros=z, offsets=off, out=out)
        st = g.gemm_f32_route_plan(m, 3, experts.data_ptr(), off.data_ptr(), order.data_ptr(), places.data_ptr(), stream)
        assert st == g.OK
        got = g.w4_matmul(x, q, s, group, zeros=z, offsets=off)
    assert torch.equal(off, want) and (out == 7).all()
    starts = want.tolist()
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        check(got[a:b], x[a:b], weights_64(q[i], s[i], z[i], k, group), dt, f"segment {i}")


@pytest.mark.parametrize("m", [1, 2])
@pytest.mark.parametrize("n, k, group", [(130, 30000, 64), (1, 33, 32), (300, 2304, 96), (11008, 4096, 128)])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_single_tokens(g, dt, n, k, group, m):
    x, q, s, z = case(m, n, k, group, dt, True)
    got = g.w4_matmul(x, q, s, group, zeros=z)
    check(got, x, weights_64(q, s, z, k, group), dt)
    for first in (0, 1, m):  # one row a segment, or both, or none
        off = torch.tensor([0, first, first, m]).cuda()
        mine = g.w4_matmul(x, q.expand(3, -1, -1), s.expand(3, -1, -1), group, zeros=z.expand(3, -1, -1), offsets=off)
        check(mine, x, weights_64(q, s, z, k, group), dt)
    x[0, k - 1] = math.inf
    if m == 2:
        x[1] *= 2.0 ** 30
        mine = g.w4_matmul(x, q, s, group, zeros=z)
        check(mine[1:], x[1:], weights_64(q, s, z, k, group), dt)
        assert not mine[0].isfinite().any()


# Weights of more than 512 MB in 4 bytes each are expanded in parts: of the matrices, and
# of a matrix.
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_weights_expanded_in_parts(g, dt):
    n, k, group, groups = 1024, 1024, 128, 140
    sizes = [260] * groups
    sizes[3], sizes[131], sizes[139] = 0, 700, 1
    starts = [0]
    for size in sizes:
        starts.append(starts[-1] + size)
    assert starts[-1] >= 256 * groups
    x, q, s, z = case(starts[-1], n, k, group, dt, True, groups)
    got = g.w4_matmul(x, q, s, group, zeros=z, offsets=torch.tensor(starts).cuda())
    for i in (0, 2, 3, 127, 128, 131, 138, 139):
        rows = slice(starts[i], starts[i + 1])
        check(got[rows], x[rows], weights_64(q[i], s[i], z[i], k, group), dt, f"segment {i}")
    n, k = 8200, 16384
    x, q, s, z = case(256, n, k, group, dt, True)
    got = g.w4_matmul(x, q, s, group, zeros=z)
    for i in (0, 4096, 8104):
        rows = slice(i, i + 96)
        check(got[:, rows], x, weights_64(q[rows], s[rows], z[rows], k, group), dt, f"rows from {i}")


@pytest.mark.parametrize("m", [1, 150])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_without_a_contraction(g, dt, m):
    x = torch.zeros(m, 0, dtype=dt, device="cuda")
    q, s = torch.zeros(24, 0, dtype=torch.uint8, device="cuda"), torch.zeros(24, 0, dtype=dt, device="cuda")
    assert not g.w4_matmul(x, q, s, 32).any()
    out = torch.full((m, 24), 7.0, dtype=dt, device="cuda")
    off = torch.tensor([0, 1, 1]).cuda()
    g.w4_matmul(x, q.expand(2, -1, -1), s.expand(2, -1, -1), 32, offsets=off, out=out)
    assert not out[0].any() and (out[1:] == 7).all()


def test_refusals(g):
    x, q, s, z = case(4, 64, 128, 32, torch.float32, True)
    for bad in (lambda: g.w4_matmul(x, q, s, 16), lambda: g.w4_matmul(x, q, s, 64),
                lambda: g.w4_matmul(x, q[:, 1:], s, 32), lambda: g.w4_matmul(x, q, s, 32, zeros=z[:, :2]),
                lambda: g.w4_matmul(x, q, s[:60], 32), lambda: g.w4_matmul(x, q.t(), s, 32),
                lambda: g.w4_matmul(x, q, s, 32, out=torch.zeros(4, 63, device="cuda")),
                lambda: g.w4_matmul(x, q, s.bfloat16(), 32)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: g.w4_matmul(x, q.int(), s, 32), lambda: g.w4_matmul(x, q.cpu(), s, 32),
                lambda: g.w4_matmul(x, q, s, 32, offsets=torch.tensor([0, 4]).cuda()),
                lambda: g.w4_matmul(x, q, None, 32), lambda: g.w4_matmul(x.half(), q, s, 32)):
        with pytest.raises(TypeError):
            bad()
