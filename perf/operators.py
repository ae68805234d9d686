"""Cases that measure the segmented matrix products: products grouped by
expert, their weight gradients, and low-rank adapters of many requests beside
a shared projection, forward and backward.

Rows (tokens) lie sorted by segment: `offsets` (segments + 1 whole numbers on
the GPU) says where each one starts, and segments may be empty. `run` computes
one pass, in plain torch operations in fp32 (`own` false) or through the
package's operators (`own` true). Sizes follow the repository's own workloads
(512 to 4096, 1000 x 1531 x 777, 8192 x 11008 x 4096) and odd ones drawn from
the same range.
"""

import random

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # A single sequence's next token, sent to two of eight small experts.
        {"name": "experts token bf16", "op": "grouped", "type": "bf16", "T": 2, "G": 8, "K": 1024, "N": 2048, "split": 1},
        # One decoding step of a batch of 32 sequences, two experts each, at the
        # repository's largest projection.
        {"name": "experts decode bf16", "op": "grouped", "type": "bf16", "T": 64, "G": 8, "K": 4096, "N": 11008, "split": 2},
        # A prompt chunk through the same experts: the largest product.
        {"name": "experts prompt bf16", "op": "grouped", "type": "bf16", "T": 8192, "G": 8, "K": 4096, "N": 11008, "split": 3},
        # The ragged workload in full precision: odd pitches, odd segments.
        {"name": "experts ragged f32", "op": "grouped", "type": "f32", "T": 1000, "G": 5, "K": 777, "N": 1531, "split": 4},
        # Gradient of the experts' inputs in training (weights read transposed).
        {"name": "experts dinput f32", "op": "grouped_t", "type": "f32", "T": 4096, "G": 8, "K": 2048, "N": 2048, "split": 5},
        # Gradients of the experts' weights: long ragged sums, large outputs.
        {"name": "experts dweight bf16", "op": "wgrad", "type": "bf16", "T": 8192, "G": 8, "K": 2048, "N": 4096, "split": 6},
        {"name": "experts dweight ragged f32", "op": "wgrad", "type": "f32", "T": 1531, "G": 6, "K": 777, "N": 1000, "split": 7},
        # One request, one token, a small projection: latency.
        {"name": "adapters token f32", "op": "lora", "type": "f32", "T": 1, "G": 1, "K": 512, "N": 512, "R": 8, "bank": 4, "split": 8},
        # A decoding step of 32 requests, most with an adapter of their own.
        {"name": "adapters decode bf16", "op": "lora", "type": "bf16", "T": 32, "G": 32, "K": 4096, "N": 4096, "R": 16, "bank": 64, "split": 9},
        # Prompts of nine requests side by side.
        {"name": "adapters prompt bf16", "op": "lora", "type": "bf16", "T": 8192, "G": 9, "K": 4096, "N": 4096, "R": 64, "bank": 16, "split": 10},
        # A fine-tuning step of several adapters on one frozen projection:
        # forward, then the gradients of the input and of both factors.
        {"name": "adapters step f32", "op": "lora_step", "type": "f32", "T": 2048, "G": 4, "K": 2048, "N": 2048, "R": 16, "split": 11},
        {"name": "adapters step ragged bf16", "op": "lora_step", "type": "bf16", "T": 1531, "G": 7, "K": 1000, "N": 2048, "R": 24, "split": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_t", "wgrad", "lora", "lora_step"])
    while True:
        c = {"op": op, "type": rng.choice(["f32", "bf16"]), "T": _log_int(rng, 1, 8192),
             "G": _log_int(rng, 1, 64), "K": _log_int(rng, 32, 4096), "N": _log_int(rng, 32, 11008),
             "split": rng.randrange(1 << 20)}
        if rng.random() < 0.6:  # most programs' widths are multiples of 64; the others stay odd
            c["K"], c["N"] = -(-c["K"] // 64) * 64, -(-c["N"] // 64) * 64
        if op.startswith("lora"):
            c["R"] = rng.choice([4, 8, 16, 32, 64, 128, _log_int(rng, 1, 128)])
            if op == "lora":
                c["bank"] = _log_int(rng, 1, 64)
        banks = c["G"] * c["K"] * c["N"] if op in ("grouped", "grouped_t", "wgrad") else c["K"] * c["N"]
        passes = 3 if op == "lora_step" else 1
        if banks <= 8 * 4096 * 11008 and passes * c["T"] * c["K"] * c["N"] <= 8192 * 4096 * 11008:
            return c


def _sizes(c):
    """Rows of each segment: uneven, some empty, T in all; given by the case alone."""
    r = random.Random(c["split"])
    weight = [r.random() + 0.15 if r.random() > 0.1 else 0.0 for _ in range(c["G"])]
    if not sum(weight):
        weight[r.randrange(c["G"])] = 1.0
    if c["T"] <= 2 * c["G"]:  # few rows: each one picks its segment
        sizes = [0] * c["G"]
        for g in r.choices(range(c["G"]), weight, k=c["T"]):
            sizes[g] += 1
        return sizes
    sizes = [int(c["T"] * w / sum(weight)) for w in weight]
    sizes[max(range(c["G"]), key=lambda g: weight[g])] += c["T"] - sum(sizes)
    return sizes


def _adapters(c):
    """The adapter of each segment; about one in eight has none (-1)."""
    if "bank" not in c:
        return list(range(c["G"]))
    r = random.Random(c["split"] + 1)
    got = [r.randrange(c["bank"]) if r.random() > 0.12 else -1 for _ in range(c["G"])]
    got[0] = max(got[0], 0)
    return got


def prepare(case, seed):
    dt, dev = _TYPES[case["type"]], "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    T, G, K, N = (case[k] for k in "TGKN")
    sizes = _sizes(case)
    starts = [0]
    for s in sizes:
        starts.append(starts[-1] + s)
    st = {"op": case["op"], "type": dt, "longest": max(sizes),
          "offsets": torch.tensor(starts, dtype=torch.int64, device=dev)}
    if case["op"] == "grouped":
        st |= {"x": normal(T, K), "w": normal(G, K, N, scale=K ** -0.5)}
    elif case["op"] == "grouped_t":
        st |= {"x": normal(T, K), "w": normal(G, N, K, scale=K ** -0.5)}
    elif case["op"] == "wgrad":
        st |= {"x": normal(T, K), "dy": normal(T, N)}
    else:
        bank = case.get("bank", G)
        st |= {"x": normal(T, K), "w": normal(K, N, scale=K ** -0.5),
               "a": normal(bank, K, case["R"], scale=K ** -0.5),
               "b": normal(bank, case["R"], N, scale=case["R"] ** -0.5),
               "scales": torch.rand(bank, generator=gen, device=dev) + 0.5,
               "adapters": torch.tensor(_adapters(case), dtype=torch.int32, device=dev)}
        if case["op"] == "lora_step":
            st |= {"dy": normal(T, N)}
    return st


# ------------------------------------------------------------- plain forms --

def _places(s, rows):
    """Each row's segment, and its place in it."""
    row = torch.arange(rows, device=s["offsets"].device)
    seg = torch.searchsorted(s["offsets"][1:], row, right=True)
    return seg, row - s["offsets"][seg]


def _padded(s, x, at):
    """Rows of x by segment: segments x the longest's rows, with zeros behind the shorter ones."""
    out = torch.zeros(s["offsets"].numel() - 1, s["longest"], x.shape[1], device=x.device)
    out[at] = x.float()
    return out


def _plain_lora(s, x, w, a, b, at):
    """(x w + scale (x a) b, scale (x a)) in fp32; a and b hold one factor for each segment."""
    u = torch.matmul(_padded(s, x, at), a.float()) * s["scale"]
    return x.float() @ w.float() + torch.matmul(u, b.float())[at], u


def _plain(s):
    dt = s["type"]
    at = _places(s, s["x"].shape[0])
    if s["op"] == "grouped":
        return torch.matmul(_padded(s, s["x"], at), s["w"].float())[at].to(dt)
    if s["op"] == "grouped_t":
        return torch.matmul(_padded(s, s["x"], at), s["w"].float().transpose(1, 2))[at].to(dt)
    if s["op"] == "wgrad":
        return torch.matmul(_padded(s, s["x"], at).transpose(1, 2), _padded(s, s["dy"], at)).to(dt)
    which = s["adapters"].long()
    none = which < 0
    which = which.clamp(min=0)
    s = s | {"scale": torch.where(none, 0.0, s["scales"][which])[:, None, None]}
    a, b = s["a"][which], s["b"][which]
    y, u = _plain_lora(s, s["x"], s["w"], a, b, at)
    if s["op"] == "lora":
        return y.to(dt)
    dx, v = _plain_lora(s, s["dy"], s["w"].t(), b.transpose(1, 2), a.transpose(1, 2), at)
    da = torch.matmul(_padded(s, s["x"], at).transpose(1, 2), v)
    db = torch.matmul(u.transpose(1, 2), _padded(s, s["dy"], at))
    return {"y": y.to(dt), "dx": dx.to(dt), "da": da.to(dt), "db": db.to(dt)}


# ---------------------------------------------------- the package's operators --

def _own(s):
    import dense_fp32_gemm_major_gb300 as g

    if s["op"] == "grouped":
        return g.grouped_matmul(s["x"], s["w"], s["offsets"])
    if s["op"] == "grouped_t":
        return g.grouped_matmul(s["x"], s["w"], s["offsets"], transb=True)
    if s["op"] == "wgrad":
        return g.grouped_wgrad(s["x"], s["dy"], s["offsets"])
    if s["op"] == "lora":
        return g.lora_matmul(s["x"], s["w"], s["a"], s["b"], s["offsets"], adapters=s["adapters"],
                             scales=s["scales"])
    u = torch.empty(s["x"].shape[0], s["a"].shape[2], dtype=s["type"], device=s["x"].device)
    y = g.lora_matmul(s["x"], s["w"], s["a"], s["b"], s["offsets"], scales=s["scales"], shrink_out=u)
    dx, da, db = g.lora_backward(s["dy"], s["x"], u, s["w"], s["a"], s["b"], s["offsets"],
                                 scales=s["scales"])
    return {"y": y, "dx": dx, "da": da, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- figures --

def work(case):
    T, G, K, N = (case[k] for k in "TGKN")
    size = 4 if case["type"] == "f32" else 2
    used = sum(1 for s in _sizes(case) if s)
    if case["op"] in ("grouped", "grouped_t"):
        return {"bytes": size * (T * K + used * K * N + T * N) + 8 * (G + 1), "flops": 2 * T * K * N}
    if case["op"] == "wgrad":
        return {"bytes": size * (T * K + T * N + G * K * N) + 8 * (G + 1), "flops": 2 * T * K * N}
    R = case["R"]
    rows = {}
    for s, a in zip(_sizes(case), _adapters(case)):
        if s and a >= 0:
            rows[a] = rows.get(a, 0) + s
    low = 2 * sum(rows.values()) * R * (K + N)
    factors = len(rows) * R * (K + N)
    if case["op"] == "lora":
        return {"bytes": size * (T * K + K * N + factors + T * N), "flops": 2 * T * K * N + low}
    # forward, input gradient and the factors' gradients: x, dy, w and the
    # factors are read, y, dx and the gradients written
    return {"bytes": size * (2 * T * K + 2 * T * N + K * N + factors + G * R * (K + N)),
            "flops": 4 * T * K * N + 3 * low}


def exact(case, seed):
    """The outputs in 64 bits, from the sums' definition, segment by segment."""
    s = prepare(case, seed)
    starts = s["offsets"].tolist()
    spans = list(zip(starts[:-1], starts[1:]))
    x = s["x"].double()
    if case["op"] in ("grouped", "grouped_t"):
        form = "tk,kn->tn" if case["op"] == "grouped" else "tk,nk->tn"
        return torch.cat([torch.einsum(form, x[i:j], s["w"][g].double()) for g, (i, j) in enumerate(spans)])
    if case["op"] == "wgrad":
        return torch.stack([torch.einsum("tk,tn->kn", x[i:j], s["dy"][i:j].double()) for i, j in spans])
    w, which = s["w"].double(), s["adapters"].tolist()
    y = torch.einsum("tk,kn->tn", x, w)
    dy = s["dy"].double() if "dy" in s else None
    dx = torch.einsum("tn,kn->tk", dy, w) if dy is not None else None
    da, db = [], []
    for (i, j), k in zip(spans, which):
        if k < 0:
            continue
        a, b, f = s["a"][k].double(), s["b"][k].double(), float(s["scales"][k])
        u = torch.einsum("tk,kr->tr", x[i:j], a)
        y[i:j] += f * torch.einsum("tr,rn->tn", u, b)
        if dy is not None:
            v = torch.einsum("tn,rn->tr", dy[i:j], b)
            dx[i:j] += f * torch.einsum("tr,kr->tk", v, a)
            da.append(f * torch.einsum("tk,tr->kr", x[i:j], v))
            db.append(f * torch.einsum("tr,tn->rn", u, dy[i:j]))
    if dy is None:
        return y
    return {"y": y, "dx": dx, "da": torch.stack(da), "db": torch.stack(db)}
