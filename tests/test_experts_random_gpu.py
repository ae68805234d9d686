"""Random cases of the router and of 4-bit products over their whole ranges: values
next to each other, infinities, NaN, scales and sizes far apart, odd strides; against
the definitions in 64 bits, with the bounds of test_route_gpu.py and test_w4_gpu.py."""

import math
import random

import pytest
import torch

import test_route_gpu as route_tests

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def g(gemm_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return gemm_lib


def logits_of(rng, gen, shape, dt):
    kind = rng.choice(["normal", "wide", "ties", "steps", "steps", "tiny", "flat", "huge"])
    x = torch.randn(shape, generator=gen)
    if kind == "ties":
        x = torch.randint(-3, 4, shape, generator=gen).float()
    elif kind == "steps":  # a few steps of fp32 from each other
        x = rng.choice([0.5, 3.0, 4.0, -2.0, 10.0, -9.0]) + torch.randint(-6, 7, shape, generator=gen) * 2.0 ** -22
    elif kind == "flat":
        x = x * 5 + rng.choice([20.0, 40.0, -40.0, -90.0])
    else:
        x *= {"normal": 1.5, "wide": 30.0, "tiny": 1e-6, "huge": 1e30}[kind]
    x = x.float().to(dt)
    if rng.random() < 0.3:
        where = torch.rand(shape, generator=gen)
        x[where < 0.15] = -math.inf
        for at, value in ((0.5, math.nan), (0.6, math.inf), (0.7, torch.finfo(dt).min)):
            if rng.random() < 0.3:
                x[(where > at) & (where < at + 0.03)] = value
    return x


def bias_of(rng, gen, e):
    size = rng.choice([0.0, 1e-8, 0.1, 1.0, 3.0, 10.0, 100.0, 1e4, 1e30])
    b = torch.randn(e, generator=gen) * (rng.choice([1e-7, 0.01, 1.0]) * size) + size * rng.choice([1, -1, 0])
    for value in (-math.inf, math.inf, math.nan):
        if rng.random() < 0.1:
            b[torch.rand(e, generator=gen) < 0.07] = value
    return b


def test_routers(g):
    rng = random.Random(1)
    for case in range(400):
        groups, per = rng.choice([1, 1, 1, 2, 3, 4, 8, 16, 32]), rng.choice([1, 2, 3, 5, 8, 16, 20, 32, 33, 64, 100, 256])
        e = groups * per
        if e > 2048:
            continue
        t, dt, score = rng.choice([1, 3, 7, 20, 26]), rng.choice([F32, F32, BF16]), rng.choice(["softmax", "sigmoid"])
        gen = torch.Generator().manual_seed(case)
        x, k = logits_of(rng, gen, (t, e), dt), rng.randint(1, min(32, e))
        kw = dict(groups=groups, top_groups=rng.randint(1, groups), group_best=rng.choice([1, 2]), score=score,
                  renormalise=rng.random() < 0.5, scale=2.5, bias=bias_of(rng, gen, e) if rng.random() < 0.7 else None)
        r = g.route(x.cuda(), k, **(kw | {"bias": None if kw["bias"] is None else kw["bias"].cuda()}))
        experts, w = route_tests.route_64(x, k, score, kw["bias"], groups, kw["top_groups"], kw["group_best"],
                                          kw["renormalise"], 2.5, None)
        got = r.experts.cpu().long()
        same = (got == experts).all(1)
        if not same.all():  # keys that are one in 64 bits, but for its own rounding
            key = torch.stack([route_tests.score_of(v.double(), score) for v in x])
            key = key if kw["bias"] is None else key + kw["bias"].double()
            for i in (~same).nonzero().flatten().tolist():
                j = int((got[i] != experts[i]).nonzero()[0])
                a, b = int(experts[i, j]), int(got[i, j])
                assert a >= 0 and b >= 0, f"case {case}, token {i}"
                assert abs(key[i, a] - key[i, b]) <= 2.0 ** -51 * abs(key[i, a]), f"case {case}, token {i}"
        tol = (e / 32 + 40 + 2 * min(route_tests.spread_of(x), 1e4)) * route_tests.U * w.abs() + 2.0 ** -126
        weights = r.weights.cpu().double()
        assert torch.equal(weights.isnan()[same], w.isnan()[same]), f"case {case}"
        assert ((weights - w).abs() <= tol)[same[:, None] & ~w.isnan()].all(), f"case {case}"


def spread(t, pad, lead):
    cols = t.shape[-1]
    buf = torch.full((t.numel() // cols * (cols + pad) + lead,), 77, dtype=t.dtype, device="cuda")
    v = buf[lead:].view(*t.shape[:-1], cols + pad)[..., :cols]
    v.copy_(t)
    return v


def between(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def test_products_with_4_bit_weights(g):
    # Bound: that of test_w4_gpu.py relative to the sum of |s| (q + z) |a|, twice for
    # fp32 (the largest of 16 values may meet q + z = 1), and the smallest numbers.
    rng = random.Random(2)
    for case in range(100):
        dt, k, n = rng.choice([F32, BF16]), between(rng, 1, 1500), between(rng, 1, 300)
        group, groups = rng.choice([32, 64, 96, 128, 160, 256, 4096]), rng.choice([None, None, 1, 2, 3, 8, 40])
        if groups is None:
            stack, starts, m = (), [0], between(rng, 1, 700)
            starts.append(m)
        else:
            stack, starts = (groups,), [rng.randint(0, 3)]
            for _ in range(groups):
                starts.append(starts[-1] + rng.choice([0, 0, 1, 2, 3, 5, 9, 17, 33, 70]))
            m = starts[-1] + rng.randint(1, 3)
        gen = torch.Generator(device="cuda").manual_seed(case)
        rand = lambda *s: torch.rand(s, generator=gen, device="cuda")
        x = torch.randn(m, k, generator=gen, device="cuda", dtype=torch.float64)
        kind = rng.choice(["normal", "normal", "small", "large", "mixed", "zeros"])
        if kind in ("small", "large"):
            x *= 2.0 ** rng.randint(*{"small": (-100, -20), "large": (5, 100)}[kind])
        elif kind == "mixed":  # by blocks of 256 k
            x *= torch.randint(-100, 100, (m, -(-k // 256)), generator=gen, device="cuda").double().exp2().repeat_interleave(256, 1)[:, :k]
        elif kind == "zeros":
            x[rand(m, k) < 0.7] = 0.0
        x = x.to(dt)
        row = stack + (n, -(-k // group))
        size = rng.choice([0, 0, -4, -30] + ([-100, 60, 104, 110] if kind not in ("large", "mixed") else []))
        s = ((rand(*row).double() + 0.5) * torch.where(rand(*row) < 0.5, -1.0, 1.0) * 2.0 ** size).to(dt)
        q = torch.randint(256, stack + (n, (k + 1) // 2), generator=gen, device="cuda").to(torch.uint8)
        z = torch.randint(256, row, generator=gen, device="cuda").to(torch.uint8) if rng.random() < 0.6 else None
        how = rng.choice([(0, 0), (0, 0), (16, 0), (3, 1), (8, 16), (0, 1)])
        out = torch.full((m, n), 7.0, dtype=dt, device="cuda")
        g.w4_matmul(spread(x, *how), spread(q, *how), spread(s, *how), group, out=out,
                    zeros=None if z is None else spread(z, *how),
                    offsets=None if groups is None else torch.tensor(starts, device="cuda"))
        if groups is not None:
            assert (out[:starts[0]] == 7).all() and (out[starts[-1]:] == 7).all(), f"case {case}"
        at = torch.arange(k, device="cuda")
        for i, (a, b) in enumerate(zip(starts, starts[1:])):
            pick = lambda v: v if groups is None else v[i]
            v = pick(q).long()[:, at // 2] >> (4 * (at % 2)) & 15
            zero = 8 if z is None else (pick(z).long() & 15)[:, at // group]
            s64, x64 = pick(s).double()[:, at // group], x[a:b].double()
            c64 = x64 @ ((v - zero).double() * s64).t()
            terms = x64.abs() @ ((v + zero).double() * s64.abs()).t()
            if dt == F32:
                tol = 4 * k * 2.0 ** -24 * terms + 2.0 ** -24 * c64.abs()
            else:
                tol = 2.0 ** -8 * c64.abs() + (k + 2) * 2.0 ** -23 * terms
            tol += torch.finfo(dt).eps * 2.0 ** -127 + k * 2.0 ** -149
            bad = ~((out[a:b].double() - c64).abs() <= tol) & (c64.abs() < 0.99 * torch.finfo(dt).max)
            assert not bad.any(), f"case {case}, segment {i}: {bad.nonzero()[0].tolist()}"
