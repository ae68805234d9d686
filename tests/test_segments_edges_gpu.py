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


@pytest.mark.parametrize("rows", [4, 8, 9, 70])
@pytest.mark.parametrize("transb", [False, True])
def test_fp32_up_to_the_largest_finite_value(g, rows, transb):
    # float32 operands within 0.2 % of the largest finite value round to
    # infinity in bfloat16; results are held to the FP32 class all the same
    top = torch.finfo(torch.float32).max
    off, o = offsets_of([rows])
    a, b = normal((rows, 64), 6, torch.float32), normal((1, 64, 96), 7, torch.float32)
    near = top * (1 - torch.arange(64, device="cuda") * 2.0 ** -13).float()
    signs = a.sign()
    for big, small in ((near * signs, b * 2.0 ** -10), (torch.full_like(a, -top), b * 2.0 ** -10),
                       (signs * top * (b[0, :, :1].t() > 0), b * 2.0 ** -10)):
        s64 = big.double().abs() @ small[0].double().abs()
        c64 = big.double() @ small[0].double()
        c = g.grouped_matmul(big, small.transpose(1, 2).contiguous() if transb else small, off, transb)
        check(c, c64, rounding(c64, s64, 64, torch.float32))
    # the other operand at the top
    w = (near[:, None] * b[0].sign())[None]
    x = a * 2.0 ** -10
    c64, s64 = product(x, w[0])
    c = g.grouped_matmul(x, w.transpose(1, 2).contiguous() if transb else w, off, transb)
    check(c, c64, rounding(c64, s64, 64, torch.float32))
    # and in a weight gradient
    d = normal((rows, 40), 8, torch.float32) * 2.0 ** -10
    c64, s64 = product((near * signs).t(), d)
    check(g.grouped_wgrad(near * signs, d, off)[0], c64, rounding(c64, s64, rows, torch.float32))


@pytest.mark.parametrize("rows", [4, 8, 9, 70])
def test_fp32_down_to_the_smallest_value(g, rows):
    # Values below 2^-110 are held to 2^-134 each (their last bits lie below
    # bfloat16's smallest value): that much of the other operand's sum beside
    # the FP32 class. From 2^-110 on nothing is lost.
    off, o = offsets_of([rows])
    b = normal((1, 64, 96), 9, torch.float32) * 2.0 ** 100
    for low, high, lost in ((-110, -90, 0.0), (-149, -100, 2.0 ** -134)):
        power = torch.linspace(low, high, 64, device="cuda").round().double()
        a = ((1 + torch.rand(rows, 64, generator=torch.Generator().manual_seed(10)).cuda().double())
             * 2.0 ** power).float()
        c64, s64 = product(a, b[0])
        tol = rounding(c64, s64, 64, torch.float32) + lost * b[0].double().abs().sum(0)
        check(g.grouped_matmul(a, b, off), c64, tol)


@pytest.mark.parametrize("rows", [3, 40, 300])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_shrink_of_a_bank_without_adapters_is_zero(g, rows, dt):
    off, o = offsets_of([rows, 0, 2], first=1)
    x, w = normal((rows + 5, 64), 11, dt), normal((64, 72), 12, dt)
    none = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    a, b = torch.empty(0, 64, 8, dtype=dt, device="cuda"), torch.empty(0, 8, 72, dtype=dt, device="cuda")
    for u in (torch.full((rows + 5, 8), 7.0, dtype=dt, device="cuda"),
              torch.full((rows + 5, 11), 7.0, dtype=dt, device="cuda")[:, 1:9]):  # an odd pitch
        y = g.lora_matmul(x, w, a, b, off, none, shrink_out=u)
        y64, s64 = product(x, w)
        check(y, y64, rounding(y64, s64, 64, dt))
        assert (u[1:rows + 3] == 0).all() and (u[:1] == 7).all() and (u[rows + 3:] == 7).all()


@pytest.mark.parametrize("rows", [5, 60])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_lora_backward_of_a_projection_without_inputs(g, rows, dt):
    # no columns of X: there is no dX, and with rank 0 or no segment nothing else
    off, _ = offsets_of([rows])
    dy = normal((rows, 24), 13, dt)
    x, w = torch.empty(rows, 0, dtype=dt, device="cuda"), torch.empty(0, 24, dtype=dt, device="cuda")
    for r, o in ((0, off), (4, off[:1])):
        u = normal((rows, max(r, 1)), 14, dt)[:, :r]
        s = o.numel() - 1
        dx, da, db = g.lora_backward(dy, x, u, w, torch.empty(s, 0, r, dtype=dt, device="cuda"),
                                     torch.empty(s, r, 24, dtype=dt, device="cuda"), o)
        assert dx.shape == (rows, 0) and da.shape == (s, 0, r) and db.shape == (s, r, 24)
    u, b = normal((rows, 4), 14, dt), normal((1, 4, 24), 15, dt)
    dx, da, db = g.lora_backward(dy, x, u, w, torch.empty(1, 0, 4, dtype=dt, device="cuda"), b, off)
    c64, s64 = product(u.t(), dy)
    check(db[0], c64, rounding(c64, s64, rows, dt))


# rows, segments, contraction, columns: as many rows as the segments' average of
# two allows, and products whose matrices are many times what one CTA reads
SKEW = [(512, 256, 1024, 1024), (64, 64, 512, 2048), (200, 100, 96, 1040), (512, 300, 128, 2050),
        (40, 24, 333, 1531), (9, 5, 4096, 1024)]


@pytest.mark.parametrize("m, groups, k, n", SKEW, ids=str)
@pytest.mark.parametrize("route", ["one", "few", "even", "ends"])
@pytest.mark.parametrize("transb", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_skewed_routing(g, m, groups, k, n, route, transb, dt):
    sizes = [0] * groups
    for i in range(m):
        sizes[{"one": groups // 2, "few": i % 3 * (groups // 3), "even": i % groups,
               "ends": (i % 7 > 0) * (groups - 1)}[route]] += 1
    off, o = offsets_of(sizes)
    a = normal((m, k), 20, dt)
    b = normal((1,) + ((n, k) if transb else (k, n)), 21, dt)
    scale = 2.0 ** (torch.arange(groups, device="cuda") % 5 - 2)  # every segment's own, exactly
    b = (b * scale[:, None, None]).to(dt)
    c = g.grouped_matmul(a, b, off, transb)
    of_row = torch.repeat_interleave(scale.double(), torch.tensor(sizes, device="cuda"))[:, None]
    c64, s64 = product(a, b[2].t() if transb else b[2])  # scale 1
    check(c, c64 * of_row, rounding(c64 * of_row, s64 * of_row, k, dt))
    assert torch.equal(c, g.grouped_matmul(a, b, off, transb))


@pytest.mark.parametrize("dt, m, groups, k, n", [(torch.float32, 512, 256, 1024, 1024),
                                                 (torch.float32, 128, 64, 2048, 4096),
                                                 (torch.bfloat16, 512, 256, 128, 11008)], ids=str)
def test_skewed_routing_costs_no_more_than_one_product(g, dt, m, groups, k, n):
    # All rows to one of many experts is the product of one matrix: read once
    # for every few rows it took 5 to 20 times as long (here: up to 3 times,
    # with what it takes to look for the others' rows).
    a, b = normal((m, k), 22, dt), torch.zeros(groups, k, n, dtype=dt, device="cuda")
    off, _ = offsets_of([0] * (groups // 2) + [m] + [0] * (groups - groups // 2 - 1))
    alone, _ = offsets_of([m])

    def time(b, off):
        out, best = torch.empty(m, n, dtype=dt, device="cuda"), float("inf")
        for _ in range(8):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(200_000)  # the calls queue up behind it
            start.record()
            for _ in range(4):
                g.grouped_matmul(a, b, off, out=out)
            end.record()
            end.synchronize()
            best = min(best, start.elapsed_time(end))
        return best

    skewed, one = time(b, off), time(b[:1], alone)
    assert skewed <= 3 * one, (skewed, one)


@pytest.mark.parametrize("route", ["one", "few", "even"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_skewed_requests_of_adapters(g, route, trans, dt):
    # the products of U and with U each shared by two launches, between others
    m, segments, k, n, r = 400, 200, 2048, 4400, 96
    sizes = [0] * segments
    for i in range(m):
        sizes[{"one": 77, "few": i % 3 * 50, "even": i // 2}[route]] += 1
    off, o = offsets_of(sizes)
    which = [i % 6 - 1 for i in range(segments)]
    index = torch.tensor(which, dtype=torch.int32, device="cuda")
    w = normal((n, k) if trans else (k, n), 33, dt)
    a = normal((5, r, k) if trans else (5, k, r), 34, dt)
    b = normal((5, n, r) if trans else (5, r, n), 35, dt)
    scales = torch.rand(5, device="cuda") + 0.5
    jobs = [normal((m, k), 36 + i, dt) for i in range(3)]
    x, u = torch.empty_like(jobs[0]), torch.empty(m, r, dtype=dt, device="cuda")

    def step(i, wait):
        x.copy_(jobs[i])
        u.fill_(float("nan"))
        wait()
        y = g.lora_matmul(x, w, a, b, off, index, scales, trans, trans, shrink_out=u)
        x.fill_(float("nan"))
        return y, u.clone()

    refs = [step(i, torch.cuda.synchronize) for i in range(3)]
    at, bt = [t.t() if trans else t for t in a], [t.t() if trans else t for t in b]
    y64, ty, u64, tu = lora_64(jobs[0], w.t() if trans else w, at, bt, o, which, scales)
    check(refs[0][0], y64, ty, "y")
    check(refs[0][1], u64, tu, "u")
    outs = [(i, step(i, lambda: None)) for _ in range(4) for i in range(3)]
    for i, out in outs:
        assert torch.equal(out[0], refs[i][0]) and torch.equal(out[1], refs[i][1])


@pytest.mark.parametrize("sizes, k, n", [([2, 2], 64, 264), ([30, 20], 64, 264), ([256, 300], 128, 520)],
                         ids=lambda v: str(v))
def test_infinite_shrink_of_bf16_stays_infinite(g, sizes, k, n):
    # U, held as two terms, is infinite in one row: so is the row's result, not
    # NaN (every factor of that row's sums is positive)
    dt = torch.bfloat16
    off, o = offsets_of(sizes)
    x, w = normal((o[-1], k), 16, dt), normal((k, n), 17, dt).abs()
    a, b = normal((2, k, 8), 18, dt).abs(), normal((2, 8, n), 19, dt).abs() + 0.5
    w[0], a[:, 0] = 1, 1
    for value in (float("inf"), 3.3e38):  # the second: sums that pass the largest value
        x[1] = 1
        x[1, 0] = value
        if value != float("inf"):
            a[:, 0] = 4
        u = torch.empty(o[-1], 8, dtype=dt, device="cuda")
        y = g.lora_matmul(x, w, a, b, off, shrink_out=u)
        assert (u[1] == float("inf")).all()
        assert (y[1] == float("inf")).all()
        keep = [t for t in range(o[-1]) if t != 1]
        one = torch.ones(2, device="cuda")
        x[1] = 0
        y64, ty, _, _ = lora_64(x, w, a, b, o, range(2), one)
        check(y[keep], y64[keep], ty[keep])


def test_more_claimed_tiles_than_32_bits_count(g):
    # 2048 segments that could each claim all of 2^34 results: offsets in order
    # give each row its own; offsets that claim all rows 1024 times write
    # nothing outside the matrix and end
    m, n, k, segments = 1 << 18, 1 << 16, 16, g.MAX_SEGMENTS
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB")
    dt = torch.bfloat16
    a, b = normal((m, k), 40, dt), normal((1, k, n), 41, dt).expand(segments, k, n)
    buf = torch.full((m + 2, n), 7.0, dtype=dt, device="cuda")
    c = buf[1:-1]
    sizes = [100 + i % 57 for i in range(segments)]
    off, o = offsets_of(sizes, first=5)
    g.grouped_matmul(a, b, off, out=c)
    for i in (0, 1, 1000, segments - 1):
        r = slice(o[i], o[i + 1])
        c64, s64 = product(a[r], b[i])
        check(c[r], c64, rounding(c64, s64, k, dt))
    assert (buf[:6] == 7).all() and (c[o[-1]:o[-1] + 300] == 7).all() and (buf[-1] == 7).all()
    again = torch.tensor([0, m] * (segments // 2) + [0], dtype=torch.int64, device="cuda")
    g.grouped_matmul(a, b, again, out=c)
    assert g.gemm_f32_poll_device_status(torch.cuda.current_stream().cuda_stream) == g.OK
    assert (buf[0] == 7).all() and (buf[-1] == 7).all()


def nodes_of(call):
    """Names of the work that a call puts on its stream, captured and not run."""
    import ctypes

    cu = ctypes.CDLL("libcuda.so.1")
    stream, graph, count = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_size_t(0)
    handle = ctypes.c_void_p(stream.cuda_stream)
    with torch.cuda.stream(stream):
        call()  # its results' memory is there when it is captured
        stream.synchronize()
        assert cu.cuStreamBeginCapture_v2(handle, 2) == 0
        try:
            call()
        finally:
            assert cu.cuStreamEndCapture(handle, ctypes.byref(graph)) == 0
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(count)) == 0
    nodes, kind = (ctypes.c_void_p * count.value)(), ctypes.c_int()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(count)) == 0
    names = []
    for n in nodes:
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(n), ctypes.byref(kind)) == 0
        names.append({0: "kernel", 2: "memset", 10: "alloc", 11: "free"}.get(kind.value, "other"))
    assert cu.cuGraphDestroy(graph) == 0
    return names


@pytest.mark.parametrize("dt, rows, segments, split", [
    (torch.bfloat16, 900, 1, 0), (torch.bfloat16, 1100, 1, 1), (torch.bfloat16, 1500, 7, 0),
    (torch.bfloat16, 2100, 1, 1), (torch.float32, 400, 1, 0), (torch.float32, 600, 1, 1)], ids=str)
@pytest.mark.parametrize("trans", [False, True])
def test_gradient_of_two_terms_may_be_split_by_its_own_length(g, dt, rows, segments, split, trans):
    # dA reads V in two bf16 terms: 32 blocks of 64 rows, from which on tiles may
    # be split, are 1024 rows. The counters of split tiles are zeroed first.
    k, n, r = 264, 136, 16
    off, _ = offsets_of([rows // segments] * (segments - 1) + [rows - rows // segments * (segments - 1)])
    x, dy, w = normal((rows, k), 23, dt), normal((rows, n), 24, dt), normal((k, n), 25, dt)
    a = normal((segments, r, k) if trans else (segments, k, r), 26, dt)
    b = normal((segments, n, r) if trans else (segments, r, n), 27, dt)
    u = normal((rows, r), 28, dt)
    names = nodes_of(lambda: g.lora_backward(dy, x, u, w, a, b, off, transl=trans))
    assert names.count("memset") == split, names


@pytest.mark.parametrize("call", ["grouped_matmul", "grouped_wgrad", "lora_matmul", "lora_backward"])
def test_results_of_a_call_on_another_stream_have_memory_of_its_own(g, call):
    # `stream` runs ahead of torch's current one: a result must not stand in
    # memory that work still queued on the current stream reads.
    m, n, dt = 512, 512, torch.float32
    x, w = normal((m, n), 29, dt), normal((1, n, n), 30, dt)
    off, _ = offsets_of([m])
    f = {"grouped_matmul": lambda **kw: g.grouped_matmul(x, w, off, **kw),
         "grouped_wgrad": lambda **kw: g.grouped_wgrad(x, x, off, **kw),
         "lora_matmul": lambda **kw: g.lora_matmul(x, w[0], w, w, off, **kw),
         "lora_backward": lambda **kw: g.lora_backward(x, x, x, w[0], w, w, off, **kw)}[call]
    want = f()
    want = want if isinstance(want, tuple) else (want,)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.ones(m, n, device="cuda") for _ in range(6)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # about 10 ms
        kept = [t + 0 for t in old]  # read only then
        del old
        got = f(stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert all((t == 1).all() for t in kept)
        got = got if isinstance(got, tuple) else (got,)
        assert all(torch.equal(c, ref) for c, ref in zip(got, want))
        del got, kept


def test_streams_by_their_handle(g):
    # the legacy default stream (0) from another one, and the current one by name
    x, w = normal((300, 128), 42, torch.bfloat16), normal((3, 128, 264), 43, torch.bfloat16)
    off, _ = offsets_of([100, 0, 200])
    want = g.grouped_matmul(x, w, off)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for s in (0, side.cuda_stream, torch.cuda.default_stream().cuda_stream):
            c = g.grouped_matmul(x, w, off, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(c, want)
        assert torch.cuda.current_stream() == side


@pytest.fixture
def checked(g, checked_lib, monkeypatch):
    """The wrappers on the checked build; its record is looked at in the end."""
    monkeypatch.setattr(g, "_lib", checked_lib)
    yield g
    s = torch.cuda.current_stream().cuda_stream
    status, count, site, at, extent = g.gemm_f32_take_index_fault(s, lib=checked_lib)
    assert (status, count) == (g.OK, 0), (g.gemm_f32_index_site_name(site), at, extent)
    assert checked_lib.gemm_f32_poll_device_status(s or None) == g.OK


# Single tokens, over a cluster along k and not; routing shared by two launches;
# few tiles of long sums (slots); whole tiles; each as it lies and at an odd pitch.
CHECKED = [([1], 1100, 40), ([2, 0, 3], 1040, 520), ([1, 1, 6], 96, 2100), ([5], 20, 4200),
           ([0] * 30 + [60] + [0] * 9 + [1] * 20, 1024, 2100), ([1, 9] * 8 + [0] * 50, 1030, 2050),
           ([40], 8200, 72), ([300, 20], 4200, 264), ([256, 255, 257], 200, 512)]


@pytest.mark.parametrize("sizes, k, n", CHECKED, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("pad, lead", [(0, 0), (3, 1)])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_accesses_of_grouped_products(checked, sizes, k, n, pad, lead, trans, dt):
    off, o = offsets_of(sizes, first=1)
    a = normal((o[-1] + 2, k), 44, dt, pad, lead)
    b = normal((len(sizes),) + ((n, k) if trans else (k, n)), 45, dt, pad, lead)
    c = normal((o[-1] + 2, n), 46, dt, pad, lead)
    checked.grouped_matmul(a, b, off, trans, out=c)
    for i, s in enumerate(sizes):
        if s:
            c64, s64 = product(a[o[i]:o[i + 1]], b[i].t() if trans else b[i])
            check(c[o[i]:o[i + 1]], c64, rounding(c64, s64, k, dt))


@pytest.mark.parametrize("sizes, k, n", [([5000], 24, 17), ([2500, 0, 2100], 300, 520), ([3], 64, 40)],
                         ids=lambda v: str(v))
@pytest.mark.parametrize("pad, lead", [(0, 0), (3, 1)])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_accesses_of_weight_gradients(checked, sizes, k, n, pad, lead, dt):
    off, o = offsets_of(sizes, first=1)
    a, d = normal((o[-1] + 2, k), 47, dt, pad, lead), normal((o[-1] + 2, n), 48, dt, pad, lead)
    c = checked.grouped_wgrad(a, d, off, out=normal((len(sizes), k, n), 49, dt, pad, lead))
    for i, s in enumerate(sizes):
        c64, s64 = product(a[o[i]:o[i + 1]].t(), d[o[i]:o[i + 1]])
        check(c[i], c64, rounding(c64, s64, s, dt))


# Tokens (addend of U B among plain FMAs); few rows a segment; the fused form;
# long sums; few rows of many segments, one of which has most.
ADAPTERS = [([1], 1100, 520, 16), ([3, 0, 4], 640, 1100, 24), ([40, 30], 72, 137, 20),
            ([300, 200, 157, 300], 136, 264, 24), ([1500, 700, 0, 1900], 200, 2560, 40),
            ([90, 60], 4200, 300, 130), ([150] + [1] * 99, 1030, 2600, 70)]


@pytest.mark.parametrize("sizes, k, n, r", ADAPTERS, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("pad, lead", [(0, 0), (3, 1)])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_accesses_of_adapters(checked, sizes, k, n, r, pad, lead, trans, dt):
    m, bank = sum(sizes) + 3, len(sizes)
    off, o = offsets_of(sizes, first=2)
    x, dy = normal((m, k), 50, dt, pad, lead), normal((m, n), 51, dt, pad, lead)
    w = normal((n, k) if trans else (k, n), 52, dt, pad, lead)
    a = normal((bank, r, k) if trans else (bank, k, r), 53, dt, pad, lead)
    b = normal((bank, n, r) if trans else (bank, r, n), 54, dt, pad, lead)
    scales = torch.rand(bank, device="cuda") + 0.5
    u, y = normal((m, r), 55, dt, pad, lead), normal((m, n), 56, dt, pad, lead)
    checked.lora_matmul(x, w, a, b, off, None, scales, trans, trans, out=y, shrink_out=u)
    at, bt = [t.t() if trans else t for t in a], [t.t() if trans else t for t in b]
    y64, ty, _, _ = lora_64(x, w.t() if trans else w, at, bt, o, range(bank), scales)
    check(y, y64, ty, "y")
    dx, da, db = checked.lora_backward(dy, x, u, w, a, b, off, scales, trans, trans)
    x64, tx, v64, tv = lora_64(dy, w if trans else w.t(), [t.t() for t in bt], [t.t() for t in at], o,
                               range(bank), scales)
    check(dx, x64, tx, "dx")
    for i in range(min(bank, 4)):
        s = slice(o[i], o[i + 1])
        da64, sa = product(x[s].t(), v64[s])
        ta = rounding(da64, sa, sizes[i], dt) + x[s].double().abs().t() @ tv[s]
        check(da[i].t() if trans else da[i], da64, ta, "da")
        db64, sb = product(u[s].t(), dy[s])
        check(db[i].t() if trans else db[i], db64, rounding(db64, sb, sizes[i], dt), "db")


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_without_rows_or_contractions(g, dt):
    # no rows: gradients are zero; no contraction: the adapter's half is all, and U is zero
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    new = lambda *shape: torch.full(shape, 3.0, dtype=dt, device="cuda")
    assert g.grouped_matmul(new(0, 64), new(3, 64, 40), off).shape == (0, 40)
    assert (g.grouped_wgrad(new(0, 64), new(0, 40), off) == 0).all()
    assert g.lora_matmul(new(0, 64), new(64, 40), new(3, 64, 8), new(3, 8, 40), off).shape == (0, 40)
    dx, da, db = g.lora_backward(new(0, 40), new(0, 64), new(0, 8), new(64, 40), new(3, 64, 8),
                                 new(3, 8, 40), off)
    assert dx.shape == (0, 64) and (da == 0).all() and (db == 0).all()
    assert da.shape == (3, 64, 8) and db.shape == (3, 8, 40)
    for rows in (3, 70, 600):
        off, _ = offsets_of([rows])
        u = new(rows, 8)
        y = g.lora_matmul(new(rows, 0), new(0, 40), new(1, 0, 8), new(1, 8, 40), off, shrink_out=u)
        assert (y == 0).all() and (u == 0).all()
        # no columns of dY: dX and dA are zero, dB is empty
        dx, da, db = g.lora_backward(new(rows, 0), new(rows, 64), new(rows, 8), new(64, 0),
                                     new(1, 64, 8), new(1, 8, 0), off)
        assert (dx == 0).all() and (da == 0).all() and db.shape == (1, 8, 0)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_offsets_at_the_ends_of_their_type(g, dt):
    # held to the rows there are, by both launches of a product that is shared
    m, groups, k, n = 512, 256, 128, 2560
    a, b = normal((m, k), 60, dt), normal((1, k, n), 61, dt).expand(groups, k, n)
    off = torch.full((groups + 1,), -(1 << 63), dtype=torch.int64, device="cuda")
    off[groups // 2:] = (1 << 63) - 1
    c64, s64 = product(a, b[0])
    check(g.grouped_matmul(a, b, off), c64, rounding(c64, s64, k, dt))
    off[groups // 2:] = 300
    c = torch.full((m, n), 7.0, dtype=dt, device="cuda")
    g.grouped_matmul(a, b, off, out=c)
    check(c[:300], c64[:300], rounding(c64, s64, k, dt)[:300])
    assert (c[300:] == 7).all()
