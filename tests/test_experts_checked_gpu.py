"""The router, the rows' way to the experts and back, 4-bit products, norm and
clipping through the checked build: every access lies inside the extents that the
call declared (nothing is recorded), and what comes out is bit for bit what the
regular build gives."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]
ids = {torch.float32: "f32", torch.bfloat16: "bf16"}.get


@pytest.fixture
def both(gemm_lib, checked_lib, monkeypatch):
    """A call with the regular build, and again with the checked one."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g, stream = gemm_lib, torch.cuda.current_stream().cuda_stream
    regular = g.library()
    g.gemm_f32_take_index_fault(stream, lib=checked_lib)

    def run(call):
        monkeypatch.setattr(g, "_lib", regular)
        want = call(g)
        monkeypatch.setattr(g, "_lib", checked_lib)
        got = call(g)
        monkeypatch.setattr(g, "_lib", regular)
        assert len(got) == len(want)
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"result {i}"
        return want

    yield run
    status, count, site, at, extent = g.gemm_f32_take_index_fault(stream, lib=checked_lib)
    assert (status, count) == (g.OK, 0), (g.gemm_f32_index_site_name(site), at, extent)
    assert checked_lib.gemm_f32_poll_device_status(stream or None) == g.OK


def randn(*shape, seed=1, dt=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dt).cuda()


def apart(t, pad, lead):
    """The same values in rows that lie pad elements further apart, from `lead` on."""
    cols = t.shape[-1]
    buf = torch.full((t.numel() // cols * (cols + pad) + lead,), 77, dtype=t.dtype, device="cuda")
    v = buf[lead:].view(*t.shape[:-1], cols + pad)[..., :cols]
    v.copy_(t)
    return v


# one CTA, a cluster, two launches; lanes of one, few and many experts
@pytest.mark.parametrize("t, e, k, groups", [(1, 8, 2, 1), (24, 33, 4, 3), (25, 64, 6, 8), (150, 256, 8, 8), (192, 48, 3, 4),
                                             (193, 100, 4, 5), (3000, 256, 8, 8), (700, 77, 5, 7), (400, 777, 9, 3),
                                             (300, 2048, 32, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("pad, lead", [(0, 0), (3, 1)])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_router(both, t, e, k, groups, score, pad, lead, dt):
    x = apart(randn(t, e, dt=dt), pad, lead)
    x[::7, ::3] = -math.inf
    bias, mask = randn(e, seed=2) * 0.3, torch.rand(t, generator=torch.Generator().manual_seed(3)).cuda() < 0.8
    dw = randn(t, k, seed=4)
    for kw in (dict(), dict(bias=bias, mask=mask), dict(bias=bias + 3.0, groups=groups, top_groups=max(1, groups // 2)),
               dict(renormalise=False, groups=groups, group_best=1)):
        r = both(lambda g: g.route(x, k, score=score, **kw))
        renormalise = kw.get("renormalise", True)
        both(lambda g: (g.route_backward(dw, x, r[0], r[1], score, renormalise,
                                         out=apart(torch.zeros_like(x), pad, lead)).contiguous(),))
        both(lambda g: g.route_plan(r[0], e))


@pytest.mark.parametrize("t, d, k", [(1, 1, 1), (1, 4096, 2), (40, 777, 3), (3, 9000, 32), (700, 136, 2), (9, 1000, 5)])
@pytest.mark.parametrize("pad, lead", [(0, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_rows(both, t, d, k, pad, lead, dt):
    gen = torch.Generator().manual_seed(5)
    places = torch.randperm(t * k, generator=gen).int().view(t, k)
    places[torch.rand(t, k, generator=gen) < 0.2] = -1
    places = places.cuda()
    x, y = apart(randn(t, d, seed=6, dt=dt), pad, lead), apart(randn(t * k, d, seed=7, dt=dt), pad, lead)
    for w in (randn(t, k, seed=8), None):
        both(lambda g: (g.dispatch(x, places, out=apart(torch.zeros_like(y), pad, lead)).contiguous(),
                        g.combine(y, places, w, out=apart(torch.zeros_like(x), pad, lead)).contiguous()))
        new = lambda: apart(torch.zeros_like(y), pad, lead)
        both(lambda g: [v.contiguous() for v in g.combine_backward(x, y, places, w, out=new())])


# A made by the kernel, by a launch of its own (one turn and several), expanded weights
@pytest.mark.parametrize("sizes", [1, 5, 40, 300, [1], [0, 2, 0], [5, 0, 30, 1], [9] * 20, [300, 0, 150], [900, 0, 150]],
                         ids=str)
@pytest.mark.parametrize("n, k, group", [(130, 512, 128), (65, 777, 32), (1, 33, 64)])
@pytest.mark.parametrize("pad, lead", [(0, 0), (16, 16), (3, 1)])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_w4(both, sizes, n, k, group, pad, lead, dt):
    m, stack, off = sizes, (), None
    if isinstance(sizes, list):
        off = torch.tensor([2] + sizes).cumsum(0).cuda()
        m, stack = int(off[-1]) + 3, (len(sizes),)
    gen = torch.Generator().manual_seed(9)
    row = stack + (n, -(-k // group))
    q = apart(torch.randint(256, stack + (n, (k + 1) // 2), generator=gen).to(torch.uint8).cuda(), pad, lead)
    z = apart(torch.randint(256, row, generator=gen).to(torch.uint8).cuda(), pad, lead)
    s = apart((torch.rand(row, generator=gen) / 16).to(dt).cuda(), pad, lead)
    x = apart(randn(m, k, seed=10, dt=dt), pad, lead)
    for zeros in (z, None):
        both(lambda g: (g.w4_matmul(x, q, s, group, zeros=zeros, offsets=off,
                                    out=apart(torch.zeros(m, n, dtype=dt, device="cuda"), pad, lead)).contiguous(),))


@pytest.mark.parametrize("sizes", [[], [0], [1], [7, 0, 9], [4096, 4097, 4095], [5] * 250, [33] * 1001, [3000000, 1]],
                         ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_norm_and_clip(both, sizes, lead, shift, dt):
    ts = [randn(n + lead, seed=i, dt=dt)[lead:] for i, n in enumerate(sizes)]

    def call(g):
        out = [torch.zeros(n + shift, dtype=dt, device="cuda")[shift:] for n in sizes]
        place = [t.clone() for t in ts]
        return [g.grad_norm(ts), g.clip_grads(ts, 0.25, out=out), *out, g.clip_grads(place, 0.25), *place]

    both(call)
