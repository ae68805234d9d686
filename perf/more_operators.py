"""Cases that measure what stands around the products over segments in a
mixture of experts: the router, the way of rows to the experts and back,
products with 4-bit weights, and the clipping of all gradients by their norm.

`run` computes one pass, in plain torch operations in fp32 (`own` false; in 64
bits where experts are compared) or through the package's operators (`own`
true). Sizes follow the repository's own workloads (512 to 4096, 1000 x 1531 x
777, 8192 x 11008 x 4096; 8 experts) and generic ones, odd ones among them.

The operators:

  route      scores of T x E logits by softmax or sigmoid; the k best experts of
             every token by score + bias, within the best groups of experts where
             there are groups (ties to the lowest index); their scores as
             weights, renormalised and scaled; and the plan: tokens' slots sorted
             by expert (offsets, order) and each slot's row (places)
  rows       a copy of every token for each of its experts, sorted by expert; and
             back: the weighted sum of a token's rows
  w4         x W_g^T with W = scale (q - zero), q in 4 bits, a scale and a zero for
             each `group` values of k
  clip       all gradients times min(1, most / (norm + 1e-6)), norm the root of
             the sum of their squares
"""

import random

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SOFTMAX = {"score": "softmax", "bias": False, "groups": 1, "top": 1, "best": 1}
_GROUPED = {"score": "sigmoid", "bias": True, "groups": 8, "top": 4, "best": 2}


def listed():
    return [
        # One token, two of eight experts: latency.
        {"name": "route token f32", "op": "route", "type": "f32", "T": 1, "E": 8, "k": 2, "renormalise": True, "scale": 1.0, "padded": False, **_SOFTMAX},
        # A decoding step of a padded batch through many small experts in groups.
        {"name": "route decode f32", "op": "route", "type": "f32", "T": 64, "E": 256, "k": 8, "renormalise": True, "scale": 2.5, "padded": True, **_GROUPED},
        # A training step's router, its logits a product in bf16, and its gradient.
        {"name": "route step bf16", "op": "route_step", "type": "bf16", "T": 4095, "E": 64, "k": 6, "renormalise": False, "scale": 1.0, "padded": False, **_SOFTMAX},
        # The largest: a long batch through 256 experts in groups, and the gradient.
        {"name": "route step long f32", "op": "route_step", "type": "f32", "T": 32768, "E": 256, "k": 8, "renormalise": True, "scale": 2.5, "padded": True, **_GROUPED},
        # A decoding step's tokens to two of eight experts each, and back.
        {"name": "rows decode bf16", "op": "rows", "type": "bf16", "T": 32, "D": 4096, "E": 8, "k": 2},
        # A training step's: there, back, and the gradients of both.
        {"name": "rows step bf16", "op": "rows_step", "type": "bf16", "T": 8192, "D": 4096, "E": 8, "k": 2},
        # Odd sizes in full precision: rows that start on no 16 bytes.
        {"name": "rows step ragged f32", "op": "rows_step", "type": "f32", "T": 1531, "D": 777, "E": 5, "k": 3},
        # The next token of one sequence through the largest projection.
        {"name": "w4 token bf16", "op": "w4", "type": "bf16", "T": 1, "G": 1, "K": 4096, "N": 11008, "group": 128, "zeros": False, "split": 1},
        # A decoding step of 32 sequences, two experts each.
        {"name": "w4 experts decode bf16", "op": "w4", "type": "bf16", "T": 64, "G": 8, "K": 4096, "N": 11008, "group": 128, "zeros": True, "split": 2},
        # A few tokens in full precision, odd sizes, a last group that is short.
        {"name": "w4 ragged f32", "op": "w4", "type": "f32", "T": 13, "G": 1, "K": 777, "N": 1531, "group": 32, "zeros": True, "split": 3},
        # The adapters' gradients of a small fine-tuning step: many small tensors.
        {"name": "clip adapters f32", "op": "clip", "type": "f32", "tensors": 48, "most": 512 * 16, "least": 512 * 16, "split": 4},
        # The gradients of the largest experts, and of small tensors around them.
        {"name": "clip experts bf16", "op": "clip", "type": "bf16", "tensors": 24, "most": 4096 * 11008, "least": 777, "split": 5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["route", "route_step", "rows", "rows_step", "w4", "w4", "w4", "clip"])
    c = {"op": op, "type": rng.choice(["f32", "bf16"])}
    if op.startswith("route"):
        groups = rng.choice([1, 1, 2, 4, 8])
        c["E"] = groups * max(2, _log_int(rng, 4, 320) // groups)
        c |= {"T": _log_int(rng, 1, 16384), "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
              "groups": groups, "top": rng.randint(1, groups), "best": rng.choice([1, 2]),
              "scale": rng.choice([1.0, 1.0, 2.5]), "padded": rng.random() < 0.3}
        c["k"] = rng.randint(1, min(10, c["E"] // groups * c["top"]))
        c["renormalise"] = c["k"] > 1 and rng.random() < 0.6  # one expert alone keeps its score
    elif op.startswith("rows"):
        c |= {"T": _log_int(rng, 1, 8192), "D": _log_int(rng, 64, 4096), "E": _log_int(rng, 2, 64)}
        if rng.random() < 0.6:  # most widths are multiples of 64; the others stay odd
            c["D"] = -(-c["D"] // 64) * 64
        c["k"] = rng.randint(1, min(4, c["E"]))
        while c["T"] * c["D"] * c["k"] > 8192 * 4096 * 2:
            c["T"] = c["T"] // 2
    elif op == "w4":
        c |= {"T": _log_int(rng, 1, 64), "G": rng.choice([1, 1, _log_int(rng, 2, 16)]), "K": _log_int(rng, 64, 4096),
              "N": _log_int(rng, 64, 11008), "group": rng.choice([32, 64, 128, 128, 256]), "zeros": rng.random() < 0.5,
              "split": rng.randrange(1 << 20)}
        if rng.random() < 0.7:
            c["K"], c["N"] = -(-c["K"] // 64) * 64, -(-c["N"] // 64) * 64
        while c["G"] * c["K"] * c["N"] > 8 * 4096 * 11008:
            c["G"] = c["G"] // 2
    else:
        c |= {"tensors": _log_int(rng, 1, 400), "least": _log_int(rng, 1, 1024), "split": rng.randrange(1 << 20)}
        c["most"] = _log_int(rng, c["least"], 4096 * 4096)
        while sum(_lengths(c)) * (2 if c["type"] == "f32" else 1) > 24 * 4096 * 11008 // 4:
            c["tensors"] = c["tensors"] // 2 or 1
    return c


def _lengths(c):
    """Elements of each tensor: spread over the logarithm; given by the case alone."""
    r = random.Random(c["split"])
    n = [_log_int(r, c["least"], c["most"]) for _ in range(c["tensors"])]
    n[0] = c["most"]
    return n


def _starts(c):
    """Rows of each expert: uneven, some empty, T in all; given by the case alone."""
    r = random.Random(c["split"])
    weight = [r.random() + 0.15 if r.random() > 0.1 else 0.0 for _ in range(c["G"])]
    if not sum(weight):
        weight[r.randrange(c["G"])] = 1.0
    starts = [0] * (c["G"] + 1)
    for g in r.choices(range(c["G"]), weight, k=c["T"]):
        starts[g + 1] += 1
    for g in range(c["G"]):
        starts[g + 1] += starts[g]
    return starts


def prepare(case, seed):
    dt, dev = _TYPES[case["type"]], "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    def whole(n, *shape):
        return torch.randint(n, shape, generator=gen, device=dev)

    st = dict(case)
    if case["op"].startswith("route"):
        T, E = case["T"], case["E"]
        # some experts are asked for more than others, and the bias leans against that
        lean = torch.randn(E, generator=gen, device=dev) * 0.5
        st["logits"] = (torch.randn(T, E, generator=gen, device=dev) * 1.5 + lean).to(dt)
        st["bias"] = (lean * -0.05).float() if case["bias"] else None
        st["mask"] = uniform(T) > 0.2 if case["padded"] else None
        st["dweights"] = torch.randn(T, case["k"], generator=gen, device=dev)
    elif case["op"].startswith("rows"):
        T, E, k = case["T"], case["E"], case["k"]
        experts = (torch.randn(T, E, generator=gen, device=dev)
                   + torch.randn(E, generator=gen, device=dev) * 0.5).topk(k, dim=1).indices
        order = experts.flatten().sort(stable=True).indices
        places = torch.empty_like(order)
        places[order] = torch.arange(T * k, device=dev)
        w = uniform(T, k) + 0.1
        st |= {"x": normal(T, case["D"]), "y": normal(T * k, case["D"]), "order": order.int(),
               "places": places.view(T, k).int(), "weights": w / w.sum(1, keepdim=True)}
        if case["op"] == "rows_step":
            st |= {"dout": normal(T, case["D"]), "drows": normal(T * k, case["D"])}
    elif case["op"] == "w4":
        T, G, K, N = (case[n] for n in "TGKN")
        per_row = -(-K // case["group"])
        st |= {"x": normal(T, K), "q": whole(256, G, N, -(-K // 2)).to(torch.uint8),
               "scales": ((uniform(G, N, per_row) + 0.5) * (K ** -0.5 / 4)).to(dt),
               "zeros": (whole(8, G, N, per_row) + 4).to(torch.uint8) if case["zeros"] else None,
               "offsets": torch.tensor(_starts(case), dtype=torch.int64, device=dev)}
    else:
        lengths = _lengths(case)
        st["grads"] = [normal(n, scale=10.0 ** -(i % 4)) for i, n in enumerate(lengths)]
        st["out"] = [torch.empty_like(t) for t in st["grads"]]
        st["limit"] = 1.0
    return st


# ------------------------------------------------------------- plain forms --

def _scores(s, logits):
    return _softmax(logits) if s["score"] == "softmax" else 1 / (1 + torch.exp(-logits))


def _softmax(x):
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    T, E, k = s["T"], s["E"], s["k"]
    dev = s["logits"].device
    logits = s["logits"].float()
    # Scores are compared in 64 bits: two that are close may change places in 32.
    # Without bias or sums the logits compare as their scores do, exactly.
    key = logits.double()
    if s["bias"] is not None or (s["groups"] > 1 and s["best"] > 1):
        key = _scores(s, key)
        if s["bias"] is not None:
            key = key + s["bias"].double()
    if s["groups"] > 1:
        per = E // s["groups"]
        best = key.view(T, s["groups"], per).sort(dim=2, descending=True).values[:, :, :s["best"]].sum(2)
        top = best.sort(dim=1, descending=True, stable=True).indices[:, :s["top"]]
        kept = torch.zeros(T, s["groups"], dtype=torch.bool, device=dev).scatter_(1, top, True)
        key = torch.where(kept.repeat_interleave(per, 1), key, -torch.inf)
    experts = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    weights = _scores(s, logits).gather(1, experts)
    if s["renormalise"]:
        weights = weights / weights.sum(1, keepdim=True)
    weights = weights * s["scale"]
    if s["mask"] is not None:
        experts = torch.where(s["mask"][:, None], experts, -1)
        weights = torch.where(s["mask"][:, None], weights, 0.0)
    flat = experts.flatten()
    by, order = torch.where(flat < 0, E, flat).sort(stable=True)
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=dev))
    used = torch.arange(T * k, device=dev) < offsets[E]
    places = torch.empty_like(order)
    places[order] = torch.where(used, torch.arange(T * k, device=dev), -1)
    return (experts.int(), weights, offsets, torch.where(used, order, -1).int(), places.view(T, k).int())


def _plain_route_backward(s, experts, weights):
    logits = s["logits"].float()
    at = experts.long().clamp(min=0)
    g = torch.where(experts >= 0, s["dweights"], 0.0)
    total = (g * weights).sum(1, keepdim=True)
    if s["renormalise"]:
        total = total / s["scale"]
    if s["score"] == "sigmoid":
        part = weights * (g - total if s["renormalise"] else g) / (1 + torch.exp(logits.gather(1, at)))
    elif s["renormalise"]:
        part = weights * (g - total)
    else:
        part = weights * g
    d = torch.zeros_like(logits).scatter_add_(1, at, torch.where(experts >= 0, part, 0.0))
    if s["score"] == "softmax" and not s["renormalise"]:
        d = d - _softmax(logits) * total
    return d.to(s["logits"].dtype)


def _plain_rows(s):
    dt, k = _TYPES[s["type"]], s["k"]
    order, places = s["order"].long(), s["places"].long()
    rows = s["x"][order // k]
    y = s["y"].float()
    back = (y[places] * s["weights"][:, :, None]).sum(1).to(dt)
    if s["op"] == "rows":
        return {"rows": rows, "back": back}
    dout = s["dout"].float()
    return {"rows": rows, "back": back,
            "dy": (dout[order // k] * s["weights"].flatten()[order][:, None]).to(dt),
            "dweights": (y[places] * dout[:, None]).sum(2),
            "dx": s["drows"].float()[places].sum(1).to(dt)}


def _plain_w4(s):
    G, K, N = s["G"], s["K"], s["N"]
    q = torch.stack([s["q"] & 15, s["q"] >> 4], 3).view(G, N, -1)[:, :, :K].float()
    zeros = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(s["group"], 2)[:, :, :K]
    w = (q - zeros) * s["scales"].float().repeat_interleave(s["group"], 2)[:, :, :K]
    x = s["x"].float()
    if G == 1:
        return (x @ w[0].t()).to(s["x"].dtype)
    # every row with its own expert's weights, as a batch of products
    row = torch.arange(s["T"], device=x.device)
    expert = torch.searchsorted(s["offsets"][1:], row, right=True)
    rows = torch.zeros(G, s["T"], K, device=x.device)
    rows[expert, row] = x
    return torch.matmul(rows, w.transpose(1, 2))[expert, row].to(s["x"].dtype)


def _plain_clip(s):
    total = torch.stack([t.double().square().sum() for t in s["grads"]]).sum()  # a long sum
    norm = total.sqrt().float()
    factor = (s["limit"] / (norm + 1e-6)).clamp(max=1.0)
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * factor)
    return {"norm": norm.view(1), "grads": s["out"]}


def _plain(s):
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "route_step":
        r = _plain_route(s)
        return (*r, _plain_route_backward(s, r[0], r[1]))
    if s["op"] == "w4":
        return _plain_w4(s)
    return _plain_clip(s) if s["op"] == "clip" else _plain_rows(s)


# ---------------------------------------------------- the package's operators --

def _own(s):
    import dense_fp32_gemm_major_gb300 as g

    if s["op"].startswith("route"):
        r = g.route(s["logits"], s["k"], score=s["score"], bias=s["bias"], groups=s["groups"], top_groups=s["top"],
                    group_best=s["best"], renormalise=s["renormalise"], scale=s["scale"], mask=s["mask"])
        if s["op"] == "route":
            return tuple(r)
        return (*r, g.route_backward(s["dweights"], s["logits"], r.experts, r.weights, score=s["score"],
                                     renormalise=s["renormalise"], scale=s["scale"]))
    if s["op"].startswith("rows"):
        rows = g.dispatch(s["x"], s["places"])
        back = g.combine(s["y"], s["places"], s["weights"])
        if s["op"] == "rows":
            return {"rows": rows, "back": back}
        dy, dweights = g.combine_backward(s["dout"], s["y"], s["places"], s["weights"])
        return {"rows": rows, "back": back, "dy": dy, "dweights": dweights,
                "dx": g.combine(s["drows"], s["places"])}
    if s["op"] == "w4":
        if s["G"] == 1:
            zeros = None if s["zeros"] is None else s["zeros"][0]
            return g.w4_matmul(s["x"], s["q"][0], s["scales"][0], s["group"], zeros=zeros)
        return g.w4_matmul(s["x"], s["q"], s["scales"], s["group"], zeros=s["zeros"], offsets=s["offsets"])
    return {"norm": g.clip_grads(s["grads"], s["limit"], out=s["out"]), "grads": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- figures --

def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"].startswith("route"):
        T, E, k = case["T"], case["E"], case["k"]
        # logits in; experts, weights, order and places (4 bytes each) and offsets
        # out; a score is some four operations, its comparisons k or so
        nbytes, flops = size * T * E + 16 * T * k + 8 * (E + 1) + (4 * E if case["bias"] else 0), T * E * (4 + k)
        if case["op"] == "route_step":  # weights' gradients in, logits' out
            nbytes, flops = nbytes + 4 * T * k + size * T * E, flops + T * (E + 8 * k)
        return {"bytes": nbytes, "flops": flops}
    if case["op"].startswith("rows"):
        T, D, k = case["T"], case["D"], case["k"]
        cells = T * D + T * k * D + T * k * D + T * D  # x, rows; y, back
        flops = 2 * T * k * D
        if case["op"] == "rows_step":  # dout, (y again,) dy; drows, dx
            cells += T * D + T * k * D + T * k * D + T * D
            flops += 4 * T * k * D
        return {"bytes": size * cells + 12 * T * k, "flops": flops}
    if case["op"] == "w4":
        T, G, K, N = (case[n] for n in "TGKN")
        starts = _starts(case)
        used = sum(1 for a, b in zip(starts, starts[1:]) if b > a)
        per_row = -(-K // case["group"])
        weights = N * (-(-K // 2) + per_row * (size + (1 if case["zeros"] else 0)))
        return {"bytes": size * T * (K + N) + used * weights, "flops": 2 * T * K * N}
    n = sum(_lengths(case))
    return {"bytes": 2 * size * n, "flops": 3 * n}


def exact(case, seed):
    """The outputs in 64 bits, from the definitions."""
    s = prepare(case, seed)
    if case["op"].startswith("route"):
        return _exact_route(case, s)
    if case["op"].startswith("rows"):
        T, k = case["T"], case["k"]
        slot = torch.empty(T * k, dtype=torch.int64, device="cuda")
        slot[s["places"].flatten().long()] = torch.arange(T * k, device="cuda")
        token = torch.div(slot, k, rounding_mode="floor")
        rows = s["x"].index_select(0, token)
        back = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda")
        back.index_add_(0, token, s["y"].double() * s["weights"].double().flatten()[slot][:, None])
        if case["op"] == "rows":
            return {"rows": rows, "back": back}
        dx = torch.zeros_like(back).index_add_(0, token, s["drows"].double())
        dtoken = s["dout"].double().index_select(0, token)
        dw = torch.empty(T * k, dtype=torch.float64, device="cuda")
        dw[slot] = torch.einsum("rd,rd->r", dtoken, s["y"].double())
        return {"rows": rows, "back": back, "dy": dtoken * s["weights"].double().flatten()[slot][:, None],
                "dweights": dw.view(T, k), "dx": dx}
    if case["op"] == "w4":
        K, group = case["K"], case["group"]
        starts = s["offsets"].tolist()
        out = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
        index = torch.arange(K, device="cuda")
        for e, (i, j) in enumerate(zip(starts, starts[1:])):
            if j > i:
                q = s["q"][e].int()[:, index // 2] >> (4 * (index % 2)) & 15
                z = s["zeros"][e].int()[:, index // group] if case["zeros"] else 8
                w = (q - z).double() * s["scales"][e].double()[:, index // group]
                out[i:j] = torch.einsum("tk,nk->tn", s["x"][i:j].double(), w)
        return out
    norm = sum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in s["grads"]) ** 0.5
    factor = min(1.0, s["limit"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            "grads": [t.double() * factor for t in s["grads"]]}


def _exact_route(case, s):
    """Token by token where it is chosen, in the order of the definition: one
    expert after another."""
    T, E, k = case["T"], case["E"], case["k"]
    x = s["logits"].double()
    score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    # sigmoid and softmax ascend: without a bias or a sum the logits decide
    plain = not case["bias"] and (case["groups"] == 1 or case["best"] == 1)
    left = x.clone() if plain else score + (s["bias"].double() if case["bias"] else 0)
    if case["groups"] > 1:
        per = E // case["groups"]
        of_group = left.view(T, case["groups"], per).topk(case["best"], 2).values.sum(2)
        drop = torch.ones(T, case["groups"], dtype=torch.bool, device="cuda")
        for _ in range(case["top"]):
            first = (of_group == of_group.amax(1, keepdim=True)).int().argmax(1, keepdim=True)
            of_group.scatter_(1, first, -torch.inf)
            drop.scatter_(1, first, False)
        left.view(T, case["groups"], per)[drop] = -torch.inf
    chosen = []
    for _ in range(k):
        first = (left == left.amax(1, keepdim=True)).int().argmax(1, keepdim=True)
        left.scatter_(1, first, -torch.inf)
        chosen.append(first)
    experts = torch.cat(chosen, 1)
    picked = score.gather(1, experts)
    total = picked.sum(1, keepdim=True) if case["renormalise"] else 1.0
    weights = picked / total * case["scale"]
    there = s["mask"][:, None].expand(T, k) if case["padded"] else torch.ones_like(experts, dtype=torch.bool)
    weights = weights * there
    flat = torch.where(there, experts, E).flatten().cpu()
    count = torch.bincount(flat, minlength=E + 1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), count[:E].cumsum(0)])
    # slot after slot to its expert's next row
    order, places, at = [-1] * (T * k), [-1] * (T * k), offsets.tolist()
    for slot, e in enumerate(flat.tolist()):
        if e < E:
            order[at[e]], places[slot] = slot, at[e]
            at[e] += 1
    ints = {"dtype": torch.int32, "device": "cuda"}
    result = (torch.where(there, experts, -1).int(), weights, offsets.cuda(), torch.tensor(order, **ints),
              torch.tensor(places, **ints).view(T, k))
    if case["op"] == "route":
        return result
    # the derivative of sum(weights * dweights) by the logits, by the chain rule
    # from weights to scores to logits
    g = s["dweights"].double() * there * case["scale"]
    dpicked = (g - (g * picked / total).sum(1, keepdim=True)) / total if case["renormalise"] else g
    dpicked = dpicked * there
    dscore = torch.zeros_like(x).scatter_(1, experts, dpicked)
    if case["score"] == "sigmoid":
        return (*result, dscore * score * torch.sigmoid(-x))
    return (*result, score * (dscore - (dscore * score).sum(1, keepdim=True)))
