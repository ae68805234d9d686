"""The norm of many tensors and their clipping by it, on the GPU against the
definition in 64 bits.

The squares of at most 64 values are added in fp32 (each through 16 roundings of
2^-24, half of which show in the root), everything else in 64 bits, and the norm is
rounded once: below 18 2^-24 of it. The factor is as good, and rounded once; a product is rounded once
to its type (finfo.eps / 2), below the type's normal numbers to half of its
smallest one.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def g(gemm_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return gemm_lib


def tensors(sizes, types=(F32, BF16), scale=1.0, seed=1):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * scale).to(types[i % len(types)]).cuda()
            for i, n in enumerate(sizes)]


def norm_64(ts):
    return math.sqrt(sum(float((t.double().cpu() ** 2).sum()) for t in ts))


def check_norm(norm, ts):
    want = norm_64(ts)
    assert norm.dtype == F32 and norm.shape == (1,)
    assert abs(float(norm) - want) <= 18 * U * want


def check_clip(g, ts, limit, place):
    before = [t.clone() for t in ts]
    out = None if place else [torch.full_like(t, math.nan) for t in ts]
    norm = g.clip_grads(ts, limit, out=out)
    check_norm(norm, before)
    want = norm_64(before)
    factor = min(1.0, limit / (want + 1e-6))
    for t, b, o in zip(ts, before, ts if place else out):
        w = b.double() * factor
        tol = (torch.finfo(b.dtype).eps / 2 + 20 * U) * w.abs() + torch.finfo(b.dtype).smallest_normal * torch.finfo(b.dtype).eps
        assert ((o.double() - w).abs() <= tol).all()
        if factor == 1.0 and limit > 1.01 * want:
            assert torch.equal(o, b)
        if not place:
            assert torch.equal(t, b)
    return norm


LISTS = [[], [0], [1], [7, 0, 9], [4096, 4097, 4095], [16384] * 3, [1, 2, 3] * 40, [5] * 250, [33] * 1001,
         [100, 1 << 20, 3], [3000000, 1]]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("types", [(F32,), (BF16,), (F32, BF16)], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("place", [False, True])
def test_clip(g, sizes, types, place):
    ts = tensors(sizes, types)
    check_norm(g.grad_norm(ts), ts)
    check_clip(g, ts, 0.25, place)
    check_clip(g, tensors(sizes, types), 1e9, place)


def test_no_tensors(g):
    assert float(g.grad_norm([])) == 0.0 and float(g.clip_grads([], 1.0)) == 0.0
    assert float(g.clip_grads([torch.zeros(9, device="cuda")], 0.0)) == 0.0


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lead", [1, 2, 3, 5])
@pytest.mark.parametrize("n", [1, 2, 6, 40, 5000])
def test_alignment(g, dt, lead, n):
    buf = tensors([n + lead + 9], (dt,))[0]
    t = buf[lead:lead + n]
    rest = buf.clone()
    check_norm(g.grad_norm([t]), [t])
    for shift in (0, 1, 4, lead):  # results that start elsewhere
        out = torch.full((n + 16,), 7.0, dtype=dt, device="cuda")
        o = out[shift:shift + n]
        g.clip_grads([t], 0.5, out=[o])
        w = t.double() * min(1.0, 0.5 / (norm_64([t]) + 1e-6))
        assert ((o.double() - w).abs() <= (torch.finfo(dt).eps / 2 + 20 * U) * w.abs()).all()
        assert (out[:shift] == 7).all() and (out[shift + n:] == 7).all()
    check_clip(g, [t], 0.5, True)
    assert torch.equal(buf[:lead], rest[:lead]) and torch.equal(buf[lead + n:], rest[lead + n:])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-30, 1e-20, 1e-15, 1e-9, 1e15, 1e19, 1e30, 1e37])
def test_the_whole_range_of_the_types(g, dt, scale):
    ts = [(torch.randn(5000, generator=torch.Generator().manual_seed(2)).double() * scale).to(dt).cuda(),
          torch.zeros(3000, dtype=dt, device="cuda")]
    check_norm_range(g.grad_norm(ts), ts)
    # small values beside large ones, in one chunk and in others
    ts[0][::7] *= 1e-3
    ts += [torch.full((100,), 1e-3, dtype=dt, device="cuda")]
    check_norm_range(g.grad_norm(ts), ts)


def check_norm_range(norm, ts):
    want = norm_64(ts)
    if want > torch.finfo(F32).max:  # 5000 values of 1e37: 70 1e37 > 3.4e38
        assert float(norm) == math.inf
    else:
        assert abs(float(norm) - want) <= 18 * U * want + 2.0 ** -150


@pytest.mark.parametrize("dt", [F32, BF16])
def test_infinity_and_nan(g, dt):
    ts = tensors([100, 5000, 30], (dt,))
    ts[1][4321] = math.inf
    ts[2][3] = torch.finfo(dt).max
    out = [torch.empty_like(t) for t in ts]
    assert float(g.clip_grads(ts, 1.0, out=out)) == math.inf
    assert out[1][4321].isnan() and not out[0].any() and not out[2].any()
    ts[0][0] = math.nan
    assert math.isnan(float(g.grad_norm(ts)))
    assert math.isnan(float(g.clip_grads(ts, 1.0, out=out))) and all(o.isnan().all() for o in out)
    big = [torch.full((1000,), torch.finfo(dt).max, dtype=dt, device="cuda")]
    assert float(g.grad_norm(big)) == math.inf  # of 64 bits, above fp32's
    assert float(g.clip_grads(big, math.inf)) == math.inf


def test_reruns_are_equal_and_zero_limit(g):
    ts = tensors([3000, 70000, 11, 500000])
    assert torch.equal(g.grad_norm(ts), g.grad_norm(ts))
    g.clip_grads(ts, 0.0)
    assert not any(t.any() for t in ts)


def test_shapes_and_refusals(g):
    a, b = torch.randn(8, 16, device="cuda"), torch.randn(4, 4, 4, device="cuda")
    check_norm(g.grad_norm([a, b]), [a, b])
    for bad in (lambda: g.grad_norm([a.t()]), lambda: g.grad_norm([a[:, :3]]), lambda: g.clip_grads([a], -1.0),
                lambda: g.clip_grads([a], 1.0, out=[b]), lambda: g.clip_grads([a, b], 1.0, out=[a]),
                lambda: g.clip_grads([a], 1.0, out=[a.bfloat16()])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: g.grad_norm([a.double()]), lambda: g.grad_norm([a, None]), lambda: g.grad_norm([a.cpu()])):
        with pytest.raises(TypeError):
            bad()
    for ts, out in (([a, a], None), ([a, a.view(-1)[5:]], None), ([a, b], [b, a]), ([a], [a.view(-1)[:128]])):
        if out is not None and out[0] is not a and out[0].data_ptr() == a.data_ptr():
            g.clip_grads(ts, 1.0, out=out)  # the same memory in the same place
            continue
        if out is not None and [o.shape for o in out] != [t.shape for t in ts]:
            continue
        with pytest.raises(g.GemmError) as e:
            g.clip_grads(ts, 1.0, out=out)
        assert e.value.status == g.ERR_ALIAS
    # listed twice, results apart
    out = [torch.empty_like(a), torch.empty_like(a)]
    g.clip_grads([a, a], 0.5, out=out)
    assert torch.equal(out[0], out[1])


def test_results_in_the_place_of_operands(g):
    # refused but for a tensor's own place, whatever the shape that it is seen in there
    a, b = torch.randn(8, 16, device="cuda"), torch.randn(8, 16, device="cuda")
    before, both = a.clone(), torch.cat([a.view(-1), b.view(-1)])
    want = before.double() * (0.5 / (norm_64([a]) + 1e-6))
    for ts, out in (([a, b], [b, a]), ([a, a], None), ([a, a.view(-1)[5:]], None), ([a, a], [a, b]),
                    ([both[:128], both[128:]], [both[1:129], b.view(-1)]),
                    ([both[:128], a.view(-1)], [both[64:192], both[:128]])):
        kept = [t.clone() for t in ts]
        with pytest.raises(g.GemmError) as e:
            g.clip_grads(ts, 0.5, out=out)
        assert e.value.status == g.ERR_ALIAS
        assert all(torch.equal(t, k) for t, k in zip(ts, kept))
    g.clip_grads([a], 0.5, out=[a.view(-1)])
    assert ((a.double() - want).abs() <= 21 * U * want.abs()).all()
    x = torch.randn(100, device="cuda")
    y = x.clone()
    g.clip_grads([x, b], 0.5, out=[x, both[:128].view(8, 16)])  # one in place, one elsewhere
    assert ((x.double() - y.double() * (0.5 / (norm_64([y, b]) + 1e-6))).abs() <= 21 * U * y.double().abs()).all()


def test_norms_beyond_fp32_and_infinite_limits(g):
    x = torch.full((1000,), 1e38, device="cuda")
    out = [torch.empty_like(x)]
    assert float(g.clip_grads([x], 1.0, out=out)) == math.inf  # 3.2e39
    want = x.double() / norm_64([x])
    # a factor of 3e-40 is rounded to 2^-149: 2^-150 / 3.1e-40 of it
    assert ((out[0].double() - want).abs() <= (2.0 ** -150 / 3.1e-40 + U) * want).all()
    x[7] = math.inf
    assert float(g.clip_grads([x], math.inf, out=out)) == math.inf and out[0].isnan().all()
    assert float(g.clip_grads([x], 1.0, out=out)) == math.inf
    assert out[0][7].isnan() and not out[0][:7].any()
