"""The router, its plan and gradient, and the rows' way to the experts and back,
on the GPU against their definitions in 64 bits, token by token on the CPU.

Tolerances, from the roundings that a value goes through (u = 2^-24):

  weights     (E / 32 + 40 + 2 max |x - max x|) u of the value: expf's two units
              and its argument's rounding, the sum of E terms (E / 32 a lane, five
              steps between lanes), division and scale
  gradients   the same of a weight or score, and k + 20 more for the sum over the
              slots, on w |g| + (w / scale or s) sum |g w|; a sigmoid 8 u
  sums        (terms + 1) u of the sum of absolute terms
  rounding    finfo(type).eps / 2 of the value

Whole numbers are equal.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16]
ids = {torch.float32: "f32", torch.bfloat16: "bf16"}.get


@pytest.fixture(scope="module")
def g(gemm_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return gemm_lib


def step_of(dt):
    return torch.finfo(dt).eps / 2


def randn(shape, seed, scale=1.0, dt=torch.float32):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dt)


# ------------------------------------------------------------------ definition --

def score_of(x, score):
    if score == "sigmoid":
        z = torch.exp(-x.abs())
        return torch.where(x < 0, z, torch.ones_like(z)) / (1 + z)
    e = torch.exp(x - x.max())
    return torch.where(x == -math.inf, 0.0, e / e.sum())


def rank(keys, among):
    """Indices `among` from the best down: numbers, then NaN; ties to the lowest."""
    return sorted(among, key=lambda i: (math.isnan(keys[i]), 0.0 if math.isnan(keys[i]) else -keys[i], i))


def route_64(logits, k, score, bias, groups, top, best, renormalise, scale, mask):
    t, e = logits.shape
    experts, weights = torch.full((t, k), -1), torch.zeros(t, k, dtype=torch.float64)
    for r in range(t):
        if mask is not None and not mask[r]:
            continue
        x = logits[r].double()
        s = score_of(x, score)
        compare = bias is not None or (groups > 1 and best > 1)
        key = (s if compare else x).clone()
        there = x != -math.inf
        if bias is not None:
            key += bias.double()
            there &= bias != -math.inf
        key, there = key.tolist(), [i for i in range(e) if there[i]]
        if groups > 1:
            per, sums = e // groups, {}
            for q in range(groups):
                first = rank(key, [i for i in there if i // per == q])[:best]
                if first:
                    sums[q] = sum(key[i] for i in first)
            kept = set(rank(sums, list(sums))[:top])
            there = [i for i in there if i // per in kept]
        got = rank(key, there)[:k]
        experts[r, :len(got)] = torch.tensor(got, dtype=experts.dtype)
        if got:
            w = s[got]
            if renormalise:
                if score == "sigmoid":  # in proportion, where all are tiny
                    m = min(float(x[got].max()), 0.0)
                    w = torch.where(x[got] < 0, torch.exp(x[got] - m) / (1 + torch.exp(x[got])), w)
                elif not w.isnan().any():
                    w = torch.exp(x[got] - x[got].max())
                w = w / w.sum()
            weights[r, :len(got)] = w * scale
    return experts, weights


def plan_64(experts, e):
    flat = experts.flatten().tolist()
    slots = [[s for s, x in enumerate(flat) if x == i] for i in range(e)]
    order = [s for of in slots for s in of]
    offsets = [0]
    for of in slots:
        offsets.append(offsets[-1] + len(of))
    places = [-1] * len(flat)
    for r, s in enumerate(order):
        places[s] = r
    return offsets, order + [-1] * (len(flat) - len(order)), places


def check_plan(offsets, order, places, experts, e):
    want = plan_64(experts, e)
    assert offsets.tolist() == want[0]
    assert order.tolist() == want[1]
    assert places.flatten().tolist() == want[2]


def spread_of(logits):
    x = torch.where(logits.double().isfinite(), logits.double(), 0.0)
    return float((x.max(1).values - x.min(1).values).max()) if x.numel() else 0.0


def check_route(r, logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_best=2,
                renormalise=True, scale=1.0, mask=None):
    t, e = logits.shape
    bias = None if bias is None else bias.cpu()
    experts, weights = route_64(logits.cpu(), k, score, bias, groups, top_groups or groups, group_best,
                                renormalise, scale, None if mask is None else mask.cpu())
    assert torch.equal(r.experts.cpu().long(), experts), (r.experts.cpu() != experts).nonzero()[:4]
    got = r.weights.cpu().double()
    tol = (e / 32 + 40 + 2 * min(spread_of(logits.cpu()), 1e4)) * U * weights.abs() + 2.0 ** -126
    assert torch.equal(got.isnan(), weights.isnan())
    assert ((got - weights).abs() <= tol)[~weights.isnan()].all()
    check_plan(r.offsets, r.order, r.places, experts, e)


def call(g, logits, k, **kw):
    r = g.route(logits, k, **kw)
    check_route(r, logits, k, **kw)
    again = g.route(logits, k, **kw)
    assert all(torch.equal(a, b) for a, b in zip(r, again) if a.dtype != torch.float32)
    assert torch.equal(r.weights.view(torch.int32), again.weights.view(torch.int32))
    return r


# ----------------------------------------------------------------------- router --

SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (64, 64, 6), (65, 33, 4), (130, 160, 8), (37, 256, 8),
         (7, 300, 10), (5, 777, 3), (4, 1024, 32), (3, 2048, 32), (3, 2047, 1), (500, 16, 4)]


@pytest.mark.parametrize("t, e, k", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_route(g, t, e, k, score, renormalise, dt):
    logits = randn((t, e), 1, 1.5, dt).cuda()
    call(g, logits, k, score=score, renormalise=renormalise, scale=2.5)
    bias = randn((e,), 2, 0.2).cuda()
    call(g, logits, k, score=score, renormalise=renormalise, bias=bias)


@pytest.mark.parametrize("e, groups, top, best", [
    (8, 8, 3, 1), (8, 2, 1, 2), (64, 8, 4, 2), (160, 8, 3, 1), (160, 20, 5, 2), (256, 8, 4, 2), (256, 32, 7, 2),
    (96, 3, 2, 2), (1024, 16, 3, 2), (2048, 32, 2, 1), (6, 3, 3, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_route_in_groups(g, e, groups, top, best, score, biased, dt):
    logits = randn((70, e), 3, 1.5, dt).cuda()
    bias = randn((e,), 4, 0.3).cuda() if biased else None
    k = min(8, e // groups * top)
    call(g, logits, k, score=score, bias=bias, groups=groups, top_groups=top, group_best=best, scale=2.5)
    # more slots than the chosen groups have experts
    call(g, logits, min(e, 32), score=score, bias=bias, groups=groups, top_groups=1, group_best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_ties_go_to_the_lowest_index(g, score, groups, dt):
    logits = torch.randint(-2, 3, (200, 64), generator=torch.Generator().manual_seed(5)).to(dt).cuda()
    logits[:3] = 0.0
    logits[3] = -0.0
    logits[4, ::2] = -0.0
    for bias in (None, torch.zeros(64).cuda(), (torch.arange(64) % 3 - 1).float().cuda()):
        call(g, logits, 6, score=score, groups=groups, top_groups=max(1, groups // 2), bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups, best", [(1, 1), (8, 2), (8, 1)])
def test_scores_closer_than_fp32_tells(g, score, groups, best):
    # a bias that takes away all of the score that fp32 holds: what is left is
    # below 2^-25, in an order that only more bits show
    logits = randn((40, 64), 6)
    s = torch.stack([score_of(r.double(), score) for r in logits])
    for r in range(4):
        bias = (0.5 - s[r]).float().cuda()
        call(g, logits.cuda()[r:r + 1], 8, score=score, groups=groups, top_groups=max(1, groups // 2),
             group_best=best, bias=bias)
    # neighbours in fp32, whose sigmoids are one fp32 value where they are flat
    x = torch.full((3, 64), 4.0)
    x[:, 1:] += torch.arange(63).float() * 2.0 ** -20
    call(g, x.cuda(), 9, score=score, groups=groups, top_groups=max(1, groups // 2), group_best=best,
         bias=torch.zeros(64).cuda())
    # far apart in logits, one in fp32 scores
    x = torch.arange(30, 94).float().repeat(2, 1)
    call(g, x.cuda(), 9, score=score, groups=groups, top_groups=max(1, groups // 2), group_best=best)


def pairs_around(e, near, score, t, seed):
    """Logits of two available experts a token, and biases, such that both sums s +
    b lie within 1e-7 or so of a border between two fp32 numbers: the one below a
    multiple of eight steps of fp32, `near` in size, and that multiple."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *n: torch.rand(*n, generator=gen, dtype=torch.float64)
    step = 2.0 ** (math.floor(math.log2(near)) - 23)
    logit = lambda s: torch.log(s / (1 - s))
    x, rows = torch.full((t, e), -math.inf), torch.arange(t)
    if score == "sigmoid":
        bias = (near - 0.3 - 0.4 * rand(e)).float()
        border = (torch.round((near - 0.2 + 0.4 * rand(t)) / (8 * step)) * 8 - 0.5) * step
        first = torch.randint(e, (t,), generator=gen)
        second = (first + torch.randint(1, e, (t,), generator=gen)) % e
        for at in (first, second):
            s = border - bias.double()[at] + (rand(t) - 0.5) * 2e-7
            x[rows, at] = logit(s).float()
    else:  # two scores are 1 in sum, and so each pair of experts has a border of its own
        perm, n = torch.randperm(e, generator=gen), e // 2
        high = torch.round((near - 0.2 + 0.4 * rand(n)) / (8 * step)) * 8 * step
        part = torch.round((0.2 + 0.6 * rand(n)) / step) * step
        bias = torch.zeros(e, dtype=torch.float64)
        bias[perm[:n]], bias[perm[n:2 * n]] = high - part, high - step - 1 + part
        pair = torch.randint(n, (t,), generator=gen)
        s = part[pair] - step / 2 + (rand(t) - 0.5) * 2e-7
        low = (rand(t) - 0.5).float()
        x[rows, perm[:n][pair]] = (low.double() + logit(s)).float()
        x[rows, perm[n:2 * n][pair]] = low
        assert torch.equal(bias, bias.float().double())
    return x, bias.float()


@pytest.mark.parametrize("e, near", [(48, 17.0), (64, 20.0), (80, 5.0), (80, 9.0), (128, 9.0), (200, 3.5), (200, 9.0),
                                     (256, 3.5), (256, 5.0), (256, 100.0), (300, 3.5), (256, -3.5), (256, -9.0)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 2])
def test_sums_on_both_sides_of_a_rounding(g, e, near, score, k):
    # fp32 sums may stand the wrong way round, one step apart, and where keys lose
    # their lowest bits eight steps
    t = 30000
    x, bias = pairs_around(e, abs(near), score, t, 50)
    if near < 0:
        bias = bias - 2 * abs(near) - (1 if score == "sigmoid" else 0)
    d = x.double().cuda()
    s = torch.sigmoid(d) if score == "sigmoid" else torch.softmax(d, 1)
    key = torch.where(x.cuda() == -math.inf, -math.inf, s + bias.double().cuda())
    top = key.sort(dim=1, descending=True, stable=True)
    r = g.route(x.cuda(), k, score=score, bias=bias.cuda())
    clear = top.values[:, 0] - top.values[:, 1] > 1e-13 * abs(near)  # (64 bits have their own)
    wrong = (r.experts != top.indices[:, :k].int()).any(1) & clear
    assert clear.sum() > t // 2 and not wrong.any(), f"{int(wrong.sum())} of {t}"


@pytest.mark.parametrize("e, groups", [(256, 8), (256, 4), (64, 4), (512, 8), (1024, 8)])
def test_experts_of_a_group_that_only_64_bits_choose(g, e, groups):
    # Two groups whose sums are one in fp32: the later one's is larger. Its experts
    # behind the best two are below those that the first group would give, and so close
    # that fp32 has one score for several of them; the highest index is the best.
    t, per = 48, e // groups
    gen = torch.Generator().manual_seed(51)
    x = torch.full((t, e), -5.0)
    for r in range(t):
        a, b = sorted(torch.randperm(groups, generator=gen)[:2].tolist())
        x[r, a * per:(a + 1) * per] = 4.0
        x[r, b * per:(b + 1) * per] = 3.0 + torch.arange(per).float() * 2.0 ** -22
        for of, best in ((a, 5.0), (b, 5.0 + (r % 3 + 1) * 2.0 ** -21)):
            x[r, of * per + torch.randperm(per, generator=gen)[:2]] = torch.tensor([5.0, best])
    for k in (4, 8):
        call(g, x.cuda(), k, score="sigmoid", groups=groups, top_groups=1, group_best=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_masks_infinities_and_nan(g, score, renormalise, biased, groups):
    e, inf = 32, math.inf
    x = randn((14, e), 7)
    x[0] = -inf                                   # nothing
    x[1, 3:] = -inf                               # less than k
    x[2] = torch.finfo(torch.float32).min         # a mask of the lowest value everywhere
    x[3, 1:] = torch.finfo(torch.float32).min
    x[4, 5] = math.nan
    x[5, 5:] = math.nan
    x[6] = math.nan
    x[7, 9] = inf
    x[8, ::2] = -inf
    x[9] = -1000.0 - torch.arange(e)              # scores below fp32's range
    x[10] = 200.0 + torch.arange(e)
    x[11, 8:16] = -inf                            # a group without experts
    x[12, 1:8] = -inf                             # one with a single one
    x[13, 0] = torch.finfo(torch.float32).max
    bias = None
    if biased:
        bias = randn((e,), 8, 0.1)
        bias[7] = -inf
        bias = bias.cuda()
    mask = torch.ones(14, dtype=torch.bool)
    mask[8] = False
    for m in (None, mask.cuda()):
        call(g, x.cuda(), 6, score=score, renormalise=renormalise, bias=bias, groups=groups,
             top_groups=max(1, groups // 2), mask=m)
    none = torch.zeros(14, dtype=torch.bool, device="cuda")
    r = call(g, x.cuda(), 6, score=score, mask=none)
    assert (r.experts == -1).all() and not r.weights.any() and not r.offsets.any()


def test_nan_stays_in_its_token(g):
    x = randn((300, 64), 9).cuda()
    want = g.route(x, 4)
    x[17, 3] = math.nan
    got = g.route(x, 4)
    others = torch.arange(300, device="cuda") != 17
    assert torch.equal(got.experts[others], want.experts[others])
    assert torch.equal(got.weights[others], want.weights[others])
    assert got.weights[17].isnan().all()


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("e, pad, lead", [(64, 8, 0), (64, 0, 1), (64, 3, 0), (61, 3, 0), (40, 24, 8)])
def test_route_pitches_and_alignment(g, dt, e, pad, lead):
    buf = torch.full((100 * (e + pad) + lead,), math.nan, dtype=dt, device="cuda")
    x = buf[lead:].view(100, e + pad)[:, :e]
    x.copy_(randn((100, e), 10).to(dt))
    r = call(g, x, 5)
    dw = randn((100, 5), 11).cuda()
    out = torch.full_like(buf, 7.0)[lead:].view(100, e + pad)[:, :e]
    d = g.route_backward(dw, x, r.experts, r.weights, out=out)
    assert d is out
    assert torch.equal(d, g.route_backward(dw, x.contiguous(), r.experts, r.weights))
    if pad:
        assert (out._base.view(-1)[lead:].view(100, e + pad)[:, e:] == 7).all()


@pytest.mark.parametrize("t, e, k", [(1000, 8, 2), (4095, 64, 6), (2500, 256, 8), (129, 2048, 4), (20000, 16, 1)])
def test_long_batches(g, t, e, k):
    # many CTAs; experts of uneven popularity, a padded tail
    logits = (randn((t, e), 12) + randn((e,), 13, 2.0)).cuda()
    mask = torch.arange(t, device="cuda") < t - t // 5
    kw = dict(score="sigmoid", bias=randn((e,), 14, 0.1).cuda(), mask=mask)
    r = g.route(logits, k, **kw)
    key = torch.sigmoid(logits.double()) + kw["bias"].double()
    want = key.sort(dim=1, descending=True, stable=True).indices[:, :k].int()
    want[~mask] = -1
    assert torch.equal(r.experts, want)
    check_plan(r.offsets, r.order, r.places, want, e)
    for a, b in zip(g.route_plan(r.experts, e), (r.offsets, r.order, r.places)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("t", [23, 24, 25, 191, 192, 193, 5000])
def test_padded_batches_route_as_their_tokens_do(g, t):
    # whole stretches of the batch masked, as padding is
    e, k = 256, 8
    gen = torch.Generator().manual_seed(t)
    x, b = torch.randn(t, e, generator=gen).cuda(), torch.randn(e, generator=gen).cuda()
    mask = torch.ones(t, dtype=torch.bool)
    mask[t // 3:t // 2] = False
    mask[t - t // 5:] = False
    kw = dict(score="sigmoid", bias=b, groups=8, top_groups=4)
    r, every = g.route(x, k, mask=mask.cuda(), **kw), g.route(x, k, **kw)
    there = mask.cuda()[:, None]
    assert torch.equal(r.experts, torch.where(there, every.experts, -1))
    assert torch.equal(r.weights, torch.where(there, every.weights, 0.0))
    flat = r.experts.flatten().long()
    used = int((flat >= 0).sum())
    order = torch.sort(torch.where(flat < 0, e, flat), stable=True).indices
    assert torch.equal(r.order[:used].long(), order[:used]) and (r.order[used:] == -1).all()
    counts = torch.bincount(flat[flat >= 0], minlength=e)
    assert torch.equal(r.offsets, torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
    assert torch.equal(r.places.flatten()[order[:used]].long(), torch.arange(used, device="cuda"))
    assert torch.equal(r.places < 0, r.experts < 0)
    again = g.route(x, k, mask=mask.cuda(), **kw)
    assert all(torch.equal(u, v) for u, v in zip(r, again))


@pytest.mark.parametrize("slots, e", [(1, 1), (31, 5), (4096, 3), (4097, 7), (70000, 200), (10000, 2048)])
def test_plan_of_given_experts(g, slots, e):
    gen = torch.Generator().manual_seed(15)
    x = torch.randint(-2, e + 3, (slots, 1), generator=gen).int()
    x[0, 0] = -(1 << 31)
    x[-1, 0] = (1 << 31) - 1
    offsets, order, places = g.route_plan(x.cuda(), e)
    check_plan(offsets, order, places, torch.where((x < 0) | (x >= e), -1, x), e)
    one = torch.full((slots, 1), e - 1, dtype=torch.int32)  # all to one
    check_plan(*g.route_plan(one.cuda(), e), one, e)


def test_no_tokens(g):
    x = torch.zeros(0, 8, device="cuda")
    r = g.route(x, 2)
    assert r.experts.shape == (0, 2) and r.offsets.tolist() == [0] * 9
    assert g.route_backward(r.weights, x, r.experts, r.weights).shape == (0, 8)
    assert g.route_plan(r.experts, 8)[0].tolist() == [0] * 9
    assert g.dispatch(x, r.places).shape == (0, 8) and g.combine(x, r.places).shape == (0, 8)
    y = torch.ones(3, 8, device="cuda")
    dy, dw = g.combine_backward(x, y, r.places)
    assert dy.shape == (3, 8) and dw.shape == (0, 2)


# --------------------------------------------------------------------- gradient --

def backward_64(dw, logits, experts, weights, score, renormalise, scale):
    """The gradient and the scale of its errors."""
    t, e = logits.shape
    x, g64, w = logits.double(), dw.double(), weights.double()
    d, a = torch.zeros(t, e, dtype=torch.float64), torch.zeros(t, e, dtype=torch.float64)
    for r in range(t):
        slots = [j for j in range(experts.shape[1]) if 0 <= experts[r, j] < e]
        total = sum(float(g64[r, j] * w[r, j]) for j in slots)
        size = sum(abs(float(g64[r, j] * w[r, j])) for j in slots)
        s = score_of(x[r], score)
        for j in slots:
            i = int(experts[r, j])
            wj, gj = float(w[r, j]), float(g64[r, j])
            part = wj * (gj - total / scale) if renormalise else wj * gj
            bound = abs(wj * gj) + (abs(wj / scale) * size if renormalise else 0.0)
            if score == "sigmoid":
                part *= float(score_of(-x[r, i], score))
            d[r, i] += part
            a[r, i] += bound
        if score == "softmax" and not renormalise and slots:
            d[r] -= s * total
            a[r] += s * size
    return d, a


@pytest.mark.parametrize("t, e, k", [(1, 1, 1), (3, 5, 5), (70, 64, 6), (33, 256, 8), (5, 777, 3), (3, 2048, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_gradient(g, t, e, k, score, renormalise, dt):
    logits = randn((t, e), 16, 1.5, dt)
    mask = torch.rand(t, generator=torch.Generator().manual_seed(17)) < 0.8
    kw = dict(score=score, renormalise=renormalise, scale=2.5)
    r = g.route(logits.cuda(), k, bias=randn((e,), 18, 0.2).cuda(), mask=mask.cuda(), **kw)
    dw = randn((t, k), 19)
    d = g.route_backward(dw.cuda(), logits.cuda(), r.experts, r.weights, **kw)
    assert d.dtype == dt
    d64, size = backward_64(dw, logits, r.experts.cpu(), r.weights.cpu(), **kw)
    tol = (e / 32 + 60 + k + 2 * spread_of(logits)) * U * size + step_of(dt) * d64.abs() + 2.0 ** -126
    assert ((d.cpu().double() - d64).abs() <= tol).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_is_that_of_differences(g, score, renormalise):
    # in 64 bits: the weights as functions of the logits, the choice held
    logits, dw = randn((20, 16), 20), randn((20, 4), 21).double()
    kw = dict(score=score, renormalise=renormalise, scale=1.5)
    r = g.route(logits.cuda(), 4, **kw)
    d = g.route_backward(dw.float().cuda(), logits.cuda(), r.experts, r.weights, **kw).cpu().double()

    def value(x):
        s = torch.stack([score_of(row, score) for row in x]).gather(1, r.experts.cpu().long())
        s = s / s.sum(1, keepdim=True) if renormalise else s
        return (s * 1.5 * dw.float().double()).sum(1)

    h = 1e-5
    for i in range(16):
        up, down = logits.double().clone(), logits.double().clone()
        up[:, i] += h
        down[:, i] -= h
        slope = (value(up) - value(down)) / (2 * h)
        # differences: h^2 times a third derivative below 10; 1e-16 / h; the gradient 1e-5
        assert ((d[:, i] - slope).abs() <= 1e-5).all()


def test_gradient_of_experts_chosen_twice_and_of_none(g):
    logits, dw = randn((9, 8), 22), randn((9, 4), 23)
    experts = torch.tensor([[1, 1, 3, 1], [0, -1, 9, 0], [-1] * 4] * 3, dtype=torch.int32)
    w = torch.rand(9, 4, generator=torch.Generator().manual_seed(24))
    w[1, 1] = dw[1, 2] = math.nan  # of slots without an expert
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            d = g.route_backward(dw.cuda(), logits.cuda(), experts.cuda(), w.cuda(), score, renormalise)
            d64, size = backward_64(dw, logits, experts, w, score, renormalise, 1.0)
            assert ((d.cpu().double() - d64).abs() <= 80 * U * size).all()


# ------------------------------------------------------------------------- rows --

def rows_case(t, d, k, e, dt, seed, none=0.1):
    gen = torch.Generator().manual_seed(seed)
    experts = torch.rand(t, e, generator=gen).topk(k, 1).indices.int()
    experts[torch.rand(t, k, generator=gen) < none] = -1
    w = torch.rand(t, k, generator=gen) - 0.3
    return (experts, w, randn((t, d), seed + 1, dt=dt), randn((t * k, d), seed + 2, dt=dt),
            randn((t, d), seed + 3, dt=dt))


def padded(t, pad, lead):
    """The same values in rows that lie pad elements apart, from an element off."""
    buf = torch.full((t.shape[0] * (t.shape[1] + pad) + lead,), math.nan, dtype=t.dtype, device="cuda")
    v = buf[lead:].view(t.shape[0], -1)[:, :t.shape[1]]
    v.copy_(t)
    return v


ROWS = [(1, 1, 1), (1, 4096, 2), (5, 64, 3), (32, 512, 8), (40, 777, 3), (3, 9000, 32), (700, 136, 2),
        (17, 8, 1), (9, 1000, 5)]


@pytest.mark.parametrize("t, d, k", ROWS)
@pytest.mark.parametrize("pad, lead", [(0, 0), (8, 0), (5, 0), (0, 1)])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_rows(g, t, d, k, pad, lead, dt):
    e = max(k, 8)
    experts, w, x, y, dout = rows_case(t, d, k, e, dt, 30)
    offsets, order, places = g.route_plan(experts.cuda(), e)
    n, order = int(offsets[-1]), order.cpu()
    at = [padded(v, pad, lead) for v in (x, y, dout)]
    at[1][n:] = math.nan  # rows of no slot are not read
    out = padded(torch.full((t * k, d), 7.0, dtype=dt), pad, lead)
    gaps = int(out._base.isnan().sum()) if out._base is not None else 0
    assert g.dispatch(at[0], places, out=out) is out
    token = order[:n].long() // k
    assert torch.equal(out[:n].cpu(), x[token]) and (out[n:] == 7).all()
    if out._base is not None:
        assert int(out._base.isnan().sum()) == gaps

    p, y64, w64 = places.cpu().long(), y.double(), w.double()
    there = (p >= 0).double()
    terms = y64[p.clamp(min=0)] * there[:, :, None]
    for weights in (w, None):
        f = (w64 if weights is not None else torch.ones_like(w64))[:, :, None]
        o = g.combine(at[1], places, None if weights is None else weights.cuda())
        o64, size = (terms * f).sum(1), (terms * f).abs().sum(1)
        assert ((o.cpu().double() - o64).abs() <= (k + 1) * U * size + step_of(dt) * o64.abs()).all()

        dy = torch.full((t * k, d), 7.0, dtype=dt, device="cuda")
        dy2, dw = g.combine_backward(at[2], at[1], places, None if weights is None else weights.cuda(), out=dy)
        assert dy2 is dy and (dy[n:] == 7).all()
        d64 = dout.double()[token] * (f.expand(t, k, 1).reshape(-1, 1)[order[:n].long()])
        assert ((dy[:n].cpu().double() - d64).abs() <= (U + step_of(dt)) * d64.abs() + 2.0 ** -133).all()
        dw64 = (terms * dout.double()[:, None]).sum(2)
        size = (terms * dout.double()[:, None]).abs().sum(2)
        assert ((dw.cpu().double() - dw64).abs() <= (d + 1) * U * size).all()
        assert not dw.cpu()[p < 0].any()


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_places_outside_the_rows_are_none(g, dt):
    x, y = randn((4, 40), 40, dt=dt).cuda(), randn((6, 40), 41, dt=dt).cuda()
    places = torch.tensor([[0, 6], [-1, 3], [1 << 30, -(1 << 31)], [5, 2]], dtype=torch.int32).cuda()
    w = torch.tensor([[2.0, math.nan], [math.inf, 3.0], [math.nan, 1.0], [0.5, -1.0]]).cuda()
    out = torch.full((6, 40), 7.0, dtype=dt, device="cuda")
    g.dispatch(x, places, out=out)
    assert torch.equal(out, torch.stack([x[0], out[1], x[3], x[1], out[4], x[3]])) and (out[[1, 4]] == 7).all()
    o = g.combine(y, places, w).double()
    want = torch.stack([2 * y[0].double(), 3 * y[3].double(), 0 * y[0].double(),
                        0.5 * y[5].double() - y[2].double()])
    assert ((o - want).abs() <= step_of(dt) * want.abs() + 2 * U * 8).all()
    dy, dw = g.combine_backward(x, y, places, w, out=torch.full_like(out, 7.0))
    assert (dy[[1, 4]] == 7).all() and dw[0, 1] == 0 and not dw[2].any() and dw[1, 0] == 0


def test_nan_and_infinity_stay_in_their_rows(g):
    y = randn((8, 32), 42).cuda()
    y[3] = math.nan
    y[5, 4] = math.inf
    places = torch.arange(8, dtype=torch.int32).view(4, 2).cuda()
    o = g.combine(y, places, torch.rand(4, 2).cuda())
    assert o[1].isnan().all() and o[[0, 3]].isfinite().all() and o[2].isinf().sum() == 1
    dw = g.combine_backward(torch.ones(4, 32, device="cuda"), y, places)[1]
    assert dw[1, 1].isnan() and dw[2, 1].isinf() and dw[1, 0].isfinite()


def test_rows_of_more_than_32_bits_of_elements(g):
    # the last row of 2.2 billion elements, in a buffer of 4.4 GB
    rows, d = 70000, 32000
    buf = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    x = randn((2, d), 43, dt=torch.bfloat16).cuda()
    places = torch.tensor([[rows - 1], [0]], dtype=torch.int32).cuda()
    g.dispatch(x, places, out=buf)
    assert torch.equal(buf[rows - 1], x[0]) and torch.equal(buf[0], x[1])
    assert torch.equal(g.combine(buf, places), x)
    dy, dw = g.combine_backward(x, buf, places, out=torch.empty_like(buf))
    assert torch.equal(dy[rows - 1], x[0])
    want = (x.double() ** 2).sum(1)
    assert ((dw[:, 0].double() - want).abs() <= (d + 1) * U * want).all()
