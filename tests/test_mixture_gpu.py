"""A mixture-of-experts layer out of the router, the rows' way to the experts and
back, the products over segments, 4-bit products and the clipping, as they are used
together: in training and serving, on other streams, in graphs and from threads.

Errors are of the norm of what 64 bits give: float32 steps are good to some 1e-6
each (2e-5 for all of them); in bfloat16 each of the roundings on the way adds at most
2^-8 of the value (finfo.eps / 2).
"""

import math
import threading

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


class Layer:
    """y[t] = sum_j w[t, j] silu(x[t] up[e]) down[e], e the experts of token t."""

    def __init__(self, dt, tokens=150, width=72, hidden=104, experts=8, k=2, seed=1, **kw):
        gen = torch.Generator().manual_seed(seed)
        n = lambda *s, scale=1.0: (torch.randn(*s, generator=gen) * scale).cuda()
        self.x = n(tokens, width).to(dt)
        self.dy = n(tokens, width).to(dt)
        self.router = n(width, experts, scale=width ** -0.5)
        self.bias = n(experts, scale=0.05)
        self.up = n(experts, width, hidden, scale=width ** -0.5).to(dt)
        self.down = n(experts, hidden, width, scale=hidden ** -0.5).to(dt)
        self.mask = (torch.rand(tokens, generator=gen) < 0.9).cuda()
        self.k, self.kw = k, dict(score="sigmoid", scale=1.5) | kw

    def forward(self, g):
        logits = self.x.float() @ self.router
        r = g.route(logits, self.k, bias=self.bias, mask=self.mask, **self.kw)
        xs = g.dispatch(self.x, r.places)
        z = g.grouped_matmul(xs, self.up, r.offsets)
        act = torch.nn.functional.silu(z.float()).to(z.dtype)
        ys = g.grouped_matmul(act, self.down, r.offsets)
        return g.combine(ys, r.places, r.weights), (logits, r, xs, z, act, ys)

    def backward(self, g, saved):
        logits, r, xs, z, act, ys = saved
        dys, dw = g.combine_backward(self.dy, ys, r.places, r.weights)
        ddown = g.grouped_wgrad(act, dys, r.offsets)
        dact = g.grouped_matmul(dys, self.down, r.offsets, transb=True).float()
        s = torch.sigmoid(z.float())
        dz = (dact * s * (1 + z.float() * (1 - s))).to(z.dtype)
        dup = g.grouped_wgrad(xs, dz, r.offsets)
        dx = g.combine(g.grouped_matmul(dz, self.up, r.offsets, transb=True), r.places)
        kw = {n: v for n, v in self.kw.items() if n != "groups" and n != "top_groups"}
        dlogits = g.route_backward(dw, logits, r.experts, r.weights, **kw)
        dx = (dx.float() + dlogits @ self.router.t()).to(dx.dtype)
        return dx, dup, ddown, self.x.float().t() @ dlogits

    def step(self, g):
        y, saved = self.forward(g)
        grads = self.backward(g, saved)
        clipped = [torch.empty_like(t) for t in grads]
        return (y, *grads, *clipped, g.clip_grads(grads, 0.5, out=clipped))

    def step_64(self, experts):
        """By autograd, the choice of experts given."""
        d = lambda t: t.double().cpu()
        x, router, up, down = (d(t).requires_grad_() for t in (self.x, self.router, self.up, self.down))
        logits = x @ router
        score = torch.sigmoid(logits) if self.kw["score"] == "sigmoid" else torch.softmax(logits, 1)
        e = experts.cpu().long()
        there = e >= 0
        s = score.gather(1, e.clamp(min=0))
        w = self.kw["scale"] * s / s.sum(1, keepdim=True) if self.kw.get("renormalise", True) else self.kw["scale"] * s
        y = torch.zeros_like(x)
        for i in range(x.shape[0]):
            for j in range(self.k):
                if there[i, j]:
                    z = x[i] @ up[e[i, j]]
                    y[i] = y[i] + w[i, j] * ((z * torch.sigmoid(z)) @ down[e[i, j]])
        grads = torch.autograd.grad(y, (x, up, down, router), d(self.dy))
        norm = math.sqrt(sum(float((t ** 2).sum()) for t in grads))
        factor = min(1.0, 0.5 / (norm + 1e-6))
        return (y.detach(), *grads, *[t * factor for t in grads], torch.tensor([norm], dtype=torch.float64))


@pytest.mark.parametrize("kw", [dict(), dict(renormalise=False), dict(score="softmax"),
                                dict(score="softmax", renormalise=False), dict(groups=4, top_groups=2)], ids=str)
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_a_training_step(g, dt, kw):
    layer = Layer(dt, **kw)
    got = layer.step(g)
    want = layer.step_64(layer.forward(g)[1][1].experts)
    tol = 2e-5 if dt == torch.float32 else 10 * 2.0 ** -8
    for i, (a, b) in enumerate(zip(got, want)):
        assert a.shape == b.shape
        err = float((a.double().cpu() - b).norm() / b.norm())
        assert err <= tol, f"output {i}: {err:.3g} of the norm"


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("tokens", [1, 7, 40])
def test_serving_with_4_bit_experts(g, dt, tokens):
    gen = torch.Generator().manual_seed(2)
    e, width, hidden, group, k = 8, 256, 320, 64, 2
    x = torch.randn(tokens, width, generator=gen).to(dt).cuda()
    logits = torch.randn(tokens, e, generator=gen).cuda()

    def bank(n, kk):
        q = torch.randint(256, (e, n, kk // 2), generator=gen).to(torch.uint8).cuda()
        s = ((torch.rand(e, n, kk // group, generator=gen) + 0.5) * kk ** -0.5 / 4).to(dt).cuda()
        low = torch.stack([q & 15, q >> 4], 3).view(e, n, kk)
        return q, s, (low.double() - 8) * s.double().repeat_interleave(group, 2)

    (q1, s1, w1), (q2, s2, w2) = bank(hidden, width), bank(width, hidden)
    r = g.route(logits, k)
    xs = g.dispatch(x, r.places)
    h = g.w4_matmul(xs, q1, s1, group, offsets=r.offsets)
    y = g.combine(g.w4_matmul(h, q2, s2, group, offsets=r.offsets), r.places, r.weights)
    want = torch.zeros(tokens, width, dtype=torch.float64, device="cuda")
    for t in range(tokens):
        for j in range(k):
            i = int(r.experts[t, j])
            want[t] += r.weights[t, j].double() * ((x[t].double() @ w1[i].t()) @ w2[i].t())
    tol = 1e-5 if dt == torch.float32 else 3 * 2.0 ** -8
    assert float((y.double() - want).norm() / want.norm()) <= tol


def equal(a, b):
    return all(torch.equal(p.view(torch.uint8) if p.dtype != torch.bool else p, q.view(torch.uint8)
                           if q.dtype != torch.bool else q) for p, q in zip(a, b))


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_steps_in_graphs(g, dt):
    # two graphs of different layers, replayed in turn and on two streams at once
    layers = [Layer(dt, seed=s, tokens=t) for s, t in ((3, 150), (4, 700))]
    want = [layer.step(g) for layer in layers]
    graphs, got = [], []
    for layer in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(layer.step(g))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(equal(a, b) for a, b in zip(got, want))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all(equal(a, b) for a, b in zip(got, want))
    # other inputs in the same memory
    other = Layer(dt, seed=5, tokens=150)
    layers[0].x.copy_(other.x)
    layers[0].dy.copy_(other.dy)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert equal(got[0], layers[0].step(g))


def calls(g, dt):
    """A call of every entry point, of inputs that it overwrites right behind it."""
    gen = torch.Generator().manual_seed(6)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()
    x, logits, places = n(300, 264).to(dt), n(300, 40), torch.randperm(900, generator=gen).int().view(300, 3).cuda()
    rows, w, q = n(900, 264).to(dt), n(300, 3), torch.randint(256, (96, 132), generator=gen).to(torch.uint8).cuda()
    s = (n(96, 9) / 16).to(dt)
    experts = torch.randint(-1, 40, (300, 3), generator=gen).int().cuda()
    odd = torch.randint(256, (96, 131), generator=gen).to(torch.uint8).cuda()
    grads = [n(5000).to(dt), n(300, 264)]
    return [
        ((logits,), lambda l: g.route(l, 3, bias=w.view(-1)[:40].contiguous(), score="sigmoid")),
        ((logits[:20],), lambda l: g.route(l, 3)),
        ((w, logits), lambda d, l: (g.route_backward(d, l, experts, w),)),
        ((experts,), lambda e: g.route_plan(e, 40)),
        ((x,), lambda v: (g.dispatch(v, places),)),
        ((rows, w), lambda y, v: (g.combine(y, places, v),)),
        ((x, rows), lambda d, y: g.combine_backward(d, y, places, w)),
        ((x[:9], q), lambda v, b: (g.w4_matmul(v, b, s, 32),)),
        ((x[:40, :262].contiguous(), odd), lambda v, b: (g.w4_matmul(v, b, s, 32),)),
        ((x, q), lambda v, b: (g.w4_matmul(v, b, s, 32),)),
        (tuple(grads), lambda *t: (g.grad_norm(t),)),
        (tuple(grads), lambda *t: (g.clip_grads(t, 0.1, out=[o.clone() for o in t]),)),
    ]


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_calls_in_a_row_on_another_stream(g, dt):
    # no launch starts before what it reads is there, or reads what comes behind it
    todo = calls(g, dt)
    want = [f(*[t.clone() for t in a]) for a, f in todo]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        copies = [[torch.zeros_like(t) for t in a] for a, _ in todo]
        side.wait_stream(torch.cuda.current_stream())
        got = []
        with torch.cuda.stream(side):
            for (a, f), c in zip(todo, copies):
                for t, v in zip(a, c):
                    v.copy_(t)
                got.append(f(*c))
                for v in c:
                    v.zero_()
        side.synchronize()
        for i, (p, q) in enumerate(zip(got, want)):
            assert equal(p, q), f"call {i}"


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_streams_by_their_handle(g, dt):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, logits = torch.randn(60, 64, device="cuda").to(dt), torch.randn(60, 8, device="cuda")
    q, s = torch.randint(256, (40, 32), device="cuda").to(torch.uint8), torch.ones(40, 2, device="cuda").to(dt)
    torch.cuda.synchronize()
    r = g.route(logits, 2, stream=side.cuda_stream)
    xs = g.dispatch(x, r.places, stream=side.cuda_stream)
    o = g.combine(xs, r.places, r.weights, stream=side.cuda_stream)
    dy, dw = g.combine_backward(x, xs, r.places, r.weights, stream=side.cuda_stream)
    dl = g.route_backward(dw, logits, r.experts, r.weights, stream=side.cuda_stream)
    c = g.w4_matmul(x, q, s, 32, stream=side.cuda_stream)
    norm = g.grad_norm([dy, dl], stream=side.cuda_stream)
    plan = g.route_plan(r.experts, 8, stream=side.cuda_stream)
    side.synchronize()
    t = g.route(logits, 2)
    xs2 = g.dispatch(x, t.places)
    dy2, dw2 = g.combine_backward(x, xs2, t.places, t.weights)
    dl2 = g.route_backward(dw2, logits, t.experts, t.weights)
    assert equal((*r, xs, o, dy, dw, dl, c, norm, *plan),
                 (*t, xs2, g.combine(xs2, t.places, t.weights), dy2, dw2, dl2, g.w4_matmul(x, q, s, 32),
                  g.grad_norm([dy2, dl2]), *g.route_plan(t.experts, 8)))


def test_threads(g):
    todo = calls(g, torch.float32)
    want = [f(*a) for a, f in todo]
    torch.cuda.synchronize()
    wrong = []

    def work(seed):
        with torch.cuda.stream(torch.cuda.Stream()):
            for i in range(30):
                n = (seed + i) % len(todo)
                got = todo[n][1](*todo[n][0])
                torch.cuda.current_stream().synchronize()
                if not equal(got, want[n]):
                    wrong.append(n)

    threads = [threading.Thread(target=work, args=(3 * i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert g.gemm_f32_poll_device_status(0) == g.OK


def test_another_device(g):
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    want = [f(*a) for a, f in calls(g, torch.bfloat16)]
    with torch.cuda.device(1):
        todo = calls(g, torch.bfloat16)
    for (a, f), w in zip(todo, want):
        assert equal([t.cpu() for t in f(*a)], [t.cpu() for t in w])


def test_products_of_both_kinds_on_two_streams(g):
    # tensor-core kernels of all of TMEM beside those of half of it
    a, b = torch.randn(700, 512, device="cuda"), torch.randn(512, 600, device="cuda")
    todo = calls(g, torch.bfloat16)
    v, q = todo[7][0]
    want = [g.matmul(a, b), todo[7][1](v, q)[0], todo[9][1](*todo[9][0])[0]]
    torch.cuda.synchronize()
    one, two, three = (torch.cuda.Stream() for _ in range(3))
    for _ in range(20):
        got = []
        for stream, f in ((one, lambda: g.matmul(a, b)), (two, lambda: todo[7][1](v, q)[0]),
                          (three, lambda: todo[9][1](*todo[9][0])[0])):
            with torch.cuda.stream(stream):
                for _ in range(5):
                    r = f()
            got.append(r)
        torch.cuda.synchronize()
        assert equal(got, want)
    assert g.gemm_f32_poll_device_status(0) == g.OK
