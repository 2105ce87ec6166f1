"""What is measured of the expert layer's operators and of gradient clipping:
cases over their range, the operators in plain torch operations (32-bit,
rounded once at the end), the calls a user makes of the library, and their
definitions in 64 bits.

The expert layer: the plan that groups a batch's tokens by the experts chosen
for them, the products of each group with its expert's weight, their
gradients, and the weighted sum that brings the experts' rows back to their
tokens, with its gradient.  Clipping: the norm over all gradients that an
AllReduce left, and the gradients scaled by it.
"""
import math

import torch

own = False

F32, BF16 = "float32", "bfloat16"
SIZE = {F32: 4, BF16: 2, "int32": 4, "int64": 8}
TYPE = {F32: torch.float32, BF16: torch.bfloat16, "int32": torch.int32, "int64": torch.int64}


def listed():
    return [
        # the gradients of a small model: nothing but latency
        _clip("clip_4x256", 4, 256, 1000, F32, F32),
        # 16-bit gradients as the AllReduce left them, into the 32-bit ones that the optimizer reads, odd sizes
        _clip("clip_24x1001_bf16_to_fp32", 24, 1001, 32003, BF16, F32),
        # the 32-bit gradients of a larger model
        _clip("clip_16x4096", 16, 4096, 65536, F32, F32),
        # the groups of a short prompt
        _plan("plan_64x2_of_8", 64, 2, 8, "int64"),
        # the groups of a training batch over many small experts
        _plan("plan_65536x8_of_256", 65536, 8, 256, "int32"),
        # one new token through two of eight experts: their weights are read once
        _matmul("matmul_1x2_of_8_1024x4096", 1, 2, 8, 1024, 4096, BF16),
        # a mid-sized batch of odd sizes
        _matmul("matmul_2503x2_of_16_1001x2003", 2503, 2, 16, 1001, 2003, BF16),
        # a training batch
        _matmul("matmul_16384x2_of_16_4096x2048", 16384, 2, 16, 4096, 2048, BF16),
        # the gradients of a small 32-bit model, odd sizes, dense weight gradients
        _matmul("matmul_grad_509x1_of_4_1001x509", 509, 1, 4, 1001, 509, F32, grad=True, weight_grad=F32),
        # those of a training batch, added to the 32-bit gradients that earlier micro-batches left
        _matmul("matmul_grad_16384x2_of_16_4096x2048", 16384, 2, 16, 4096, 2048, BF16, grad=True, weight_grad=F32,
                accumulate=True),
        # back from the experts to a few tokens, and the gradients, 32-bit, odd sizes
        _combine("combine_33x2x1001", 33, 2, 1001, F32, F32),
        # the same for a training batch with eight experts a token
        _combine("combine_16384x8x2048", 16384, 8, 2048, BF16, F32),
    ]


def _clip(name, layers, dim, vocab, dtype, out):
    return {"name": name, "op": "clip", "layers": layers, "dim": dim, "vocab": vocab, "dtype": dtype, "out": out,
            "max_norm": 0.25, "scale": 0.125, "eps": 1e-6}


def _plan(name, tokens, top, experts, ids, local=None, first=0):
    return {"name": name, "op": "plan", "tokens": tokens, "top": top, "experts": experts, "ids": ids,
            "local": local or experts, "first": first}


def _matmul(name, tokens, top, experts, inner, outer, dtype, grad=False, weight_grad=BF16, accumulate=False):
    return {"name": name, "op": "matmul_grad" if grad else "matmul", "tokens": tokens, "top": top, "experts": experts,
            "in": inner, "out": outer, "dtype": dtype, "weight_grad": weight_grad, "accumulate": accumulate}


def _combine(name, tokens, top, dim, dtype, weights):
    return {"name": name, "op": "combine", "tokens": tokens, "top": top, "experts": max(8, top), "dim": dim,
            "dtype": dtype, "weights": weights}


def draw(rng):
    """A case of the same kinds: sizes log-uniform over the listed ones'
    range, about half of them odd."""
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n if rng.random() < 0.5 else max(lo, n // 8 * 8)

    kind = rng.choice(["clip", "plan", "matmul", "matmul", "matmul_grad", "matmul_grad", "combine"])
    while True:
        dtype, wide = rng.choice([BF16, BF16, BF16, F32]), rng.choice([BF16, F32])
        top = rng.choice([1, 2, 2, 4, 6, 8])
        if kind == "clip":
            c = _clip("", size(1, 32), size(64, 4096), size(1000, 65536), rng.choice([BF16, F32]), wide)
        elif kind == "plan":
            experts = max(2 * top, size(4, 256))
            local, first = experts, 0
            if experts >= 8 and rng.random() < 0.3:
                local = experts // 4
                first = rng.randrange(0, experts - local + 1)
            c = _plan("", size(16, 65536), top, experts, rng.choice(["int32", "int64"]), local, first)
        elif kind.startswith("matmul"):
            c = _matmul("", size(1, 16384), top, max(top, size(1, 128)), size(64, 4096), size(64, 4096), dtype,
                        kind == "matmul_grad", wide, rng.random() < 0.5)
        else:
            c = _combine("", size(1, 32768), top, size(64, 4096), dtype, wide)
        del c["name"]
        w = work(c)
        if w["bytes"] > (4.3e9 if kind == "clip" else 1.6e9):
            continue
        if kind.startswith("matmul") and (w["flops"] > (5.5e11 if dtype == BF16 else 6e10)
                                          or c["experts"] * c["in"] * c["out"] > 1.4e8):
            continue
        return c


def _shapes(c):
    """Elements of the gradients of a model of one product, two norm weights
    and a gate a layer, and a table."""
    d = c["dim"]
    return [c["vocab"] * d] + [d * d, d, d, d] * c["layers"]


def work(case):
    c = case
    if c["op"] == "clip":
        n = sum(_shapes(c))
        return {"bytes": n * (SIZE[c["dtype"]] + SIZE[c["out"]]) + 8, "flops": 3 * n}
    n = c["tokens"] * c["top"]
    if c["op"] == "plan":
        return {"bytes": n * (SIZE[c["ids"]] + 8) + 4 * (c["local"] + 1), "flops": 0}
    es = SIZE[c["dtype"]]
    if c["op"] == "combine":
        d = c["dim"]
        out = c["tokens"] * d * es
        extra = n * (4 + SIZE[c["weights"]])
        return {"bytes": n * d * es + out + extra + 2 * n * d * es + out + extra + n * SIZE[c["weights"]],
                "flops": 5 * n * d}
    used = c["experts"] * (1 - (1 - 1 / c["experts"]) ** n)
    weight = used * c["in"] * c["out"]
    rows = n * (c["in"] + c["out"]) * es
    if c["op"] == "matmul":
        return {"bytes": rows + weight * es, "flops": 2 * n * c["in"] * c["out"]}
    every = c["experts"] * c["in"] * c["out"]
    return {"bytes": rows + weight * es + n * c["in"] * es
            + (2 * weight if c["accumulate"] else every) * SIZE[c["weight_grad"]],
            "flops": 4 * n * c["in"] * c["out"]}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, dtype=F32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(TYPE[dtype])

    s = {"case": c}
    if c["op"] == "clip":
        sizes = _shapes(c)
        # one flat vector that an AllReduce works on; the gradients are views of it
        s["flat"] = normal(sum(sizes), dtype=c["dtype"], std=1e-2)
        s["flat_out"] = torch.empty(sum(sizes), dtype=TYPE[c["out"]], device="cuda")
        s["grads"], s["outs"] = list(s["flat"].split(sizes)), list(s["flat_out"].split(sizes))
        return s
    T, K, E = c["tokens"], c["top"], c["experts"]
    # the router: some experts are liked more than others, no token takes one twice
    liking = normal(E, std=0.5)
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    ids = (liking + noise).topk(K, dim=1).indices
    if T > 1:  # about 1 token in 100 is padding: no expert
        ids[torch.rand(T, generator=g, device="cuda") < 0.01] = -1
    if c["op"] == "plan":
        s["ids"] = ids.to(TYPE[c["ids"]])
        return s
    offsets, _, slots = _plan_of(ids, E, 0)
    s["offsets"], s["slots"] = offsets, slots
    R = T * K
    if c["op"] == "combine":
        s["y"] = normal(R, c["dim"], dtype=c["dtype"])
        s["weights"] = torch.softmax(normal(T, K), dim=1).to(TYPE[c["weights"]])
        s["grad_out"] = normal(T, c["dim"], dtype=c["dtype"], std=1e-2)
        s["grad_y"] = torch.zeros_like(s["y"])  # rows of no token stay as they are
        return s
    counts = (offsets[1:] - offsets[:-1]).long()
    s["most"] = max(1, int(counts.max()))  # rows of the largest group, for the plain form
    i, o = c["in"], c["out"]
    s["weight"] = normal(E, o, i, dtype=c["dtype"], std=i ** -0.5)
    s["x"] = normal(R, i, dtype=c["dtype"])
    if c["op"] == "matmul":
        s["out"] = torch.zeros(R, o, dtype=TYPE[c["dtype"]], device="cuda")  # rows behind the last group stay as they are
    else:
        s["grad_out"] = normal(R, o, dtype=c["dtype"], std=1e-2)
        s["grad_x"] = torch.zeros(R, i, dtype=TYPE[c["dtype"]], device="cuda")
        s["grad_weight"] = normal(E, o, i, dtype=c["weight_grad"], std=1e-1) if c["accumulate"] else \
            torch.empty(E, o, i, dtype=TYPE[c["weight_grad"]], device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        if "calls" not in state:  # bound on the first pass, repeated on the same buffers
            state["calls"], state["outputs"] = _bind(state)
        for call in state["calls"]:
            call()
        return state["outputs"]
    return PLAIN[state["case"]["op"]](state)


def _bind(s):
    """The calls a training program binds once to its buffers and repeats
    every step, and their outputs."""
    import collective_communication_algorithms_gb300 as hc
    c = s["case"]
    if c["op"] == "clip":
        a = hc.bind_clip_grads(s["grads"], c["max_norm"], out=s["outs"], scale=c["scale"], eps=c["eps"])
        return [a], {"norm": a.outputs["norm"], "grads": s["flat_out"]}
    if c["op"] == "plan":
        a = hc.bind_expert_plan(s["ids"], c["local"], first_expert=c["first"])
        return [a], {k: a.outputs[k] for k in ("offsets", "tokens", "slots")}
    if c["op"] == "matmul":
        a = hc.bind_expert_matmul(s["x"], s["weight"], s["offsets"], out=s["out"])
        return [a], {"out": s["out"]}
    if c["op"] == "matmul_grad":
        a = hc.bind_expert_matmul_grad(s["grad_out"], s["offsets"], x=s["x"], weight=s["weight"], grad_x=s["grad_x"],
                                       grad_weight=s["grad_weight"], accumulate=c["accumulate"])
        return [a], {"grad_x": s["grad_x"], "grad_weight": s["grad_weight"]}
    a = hc.bind_expert_combine(s["y"], s["slots"], weights=s["weights"])
    b = hc.bind_expert_combine_grad(s["grad_out"], s["slots"], y=s["y"], weights=s["weights"], grad_y=s["grad_y"])
    return [a, b], {"out": a.outputs["out"], "grad_y": s["grad_y"], "grad_weights": b.outputs["grad_weights"]}


def _plain_clip(s):
    c = s["case"]
    g = s["flat"].float()
    norm = torch.sqrt((g * g).sum()) * abs(c["scale"])
    factor = (c["max_norm"] / (norm + c["eps"])).clamp(max=1.0) * c["scale"]
    s["flat_out"].copy_(g * factor)
    return {"norm": norm.reshape(1), "grads": s["flat_out"]}


def _plan_of(ids, local, first):
    T, K = ids.shape
    at = ids.reshape(-1).long() - first
    at = torch.where((at >= 0) & (at < local), at, local)
    place, order = torch.sort(at, stable=True)
    counts = torch.zeros(local + 1, dtype=torch.long, device=ids.device).index_add_(0, at, torch.ones_like(at))
    offsets = torch.cat([counts.new_zeros(1), counts[:local].cumsum(0)]).int()
    here = place < local
    tokens = torch.where(here, order // K, -1).int()
    slots = torch.empty(T * K, dtype=torch.int32, device=ids.device)
    slots[order] = torch.where(here, torch.arange(T * K, device=ids.device), -1).int()
    return offsets, tokens, slots.view(T, K)


def _plain_plan(s):
    offsets, tokens, slots = _plan_of(s["ids"], s["case"]["local"], s["case"]["first"])
    return {"offsets": offsets, "tokens": tokens, "slots": slots}


def _groups(s):
    """Places of every expert's rows, as many as the largest group has, and
    which of them are its own."""
    start, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
    at = start[:, None] + torch.arange(s["most"], device="cuda")
    return at.clamp(max=s["x"].shape[0] - 1), at < end[:, None]


def _padded(rows, at, here):
    return torch.where(here[:, :, None], rows[at].float(), 0.0)


def _back(padded, here, out):
    """The padded groups' rows, one group after the other, in out's first rows."""
    rows = padded[here]
    out[:rows.shape[0]] = rows.to(out.dtype)
    return out


def _plain_matmul(s):
    at, here = _groups(s)
    y = torch.bmm(_padded(s["x"], at, here), s["weight"].float().transpose(1, 2))
    return {"out": _back(y, here, s["out"])}


def _plain_matmul_grad(s):
    at, here = _groups(s)
    g = _padded(s["grad_out"], at, here)
    gw = torch.bmm(g.transpose(1, 2), _padded(s["x"], at, here))
    if s["case"]["accumulate"]:
        gw += s["grad_weight"].float()
    s["grad_weight"].copy_(gw)
    return {"grad_x": _back(torch.bmm(g, s["weight"].float()), here, s["grad_x"]), "grad_weight": s["grad_weight"]}


def _plain_combine(s):
    c = s["case"]
    here = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    rows = torch.where(here[:, :, None], s["y"][at].float(), 0.0)
    w, g = s["weights"].float(), s["grad_out"].float()
    out = (rows * w[:, :, None]).sum(dim=1)
    grad_w = (rows * g[:, None, :]).sum(dim=2)
    grad = w[:, :, None] * g[:, None, :]
    s["grad_y"][s["slots"][here].long()] = grad[here].to(TYPE[c["dtype"]])
    return {"out": out.to(TYPE[c["dtype"]]), "grad_y": s["grad_y"], "grad_weights": grad_w.to(TYPE[c["weights"]])}


PLAIN = {"clip": _plain_clip, "plan": _plain_plan, "matmul": _plain_matmul, "matmul_grad": _plain_matmul_grad,
         "combine": _plain_combine}


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    D = torch.float64
    if c["op"] == "clip":
        total = sum(float(p.to(D).pow(2).sum()) for p in s["flat"].split(1 << 26))
        norm = math.sqrt(total) * abs(c["scale"])
        factor = min(1.0, c["max_norm"] / (norm + c["eps"])) * c["scale"]
        return {"norm": torch.tensor([norm], dtype=D, device="cuda"), "grads": s["flat"].to(D).mul_(factor)}
    if c["op"] == "plan":
        ids, K = s["ids"].reshape(-1).long() - c["first"], c["top"]
        slots = torch.full_like(ids, -1)
        tokens = torch.full_like(ids, -1)
        ends = [0]
        for e in range(c["local"]):
            mine = (ids == e).nonzero()[:, 0]
            a, b = ends[-1], ends[-1] + mine.numel()
            slots[mine] = torch.arange(a, b, device="cuda")
            tokens[a:b] = torch.div(mine, K, rounding_mode="floor")
            ends.append(b)
        return {"offsets": torch.tensor(ends, device="cuda").int(), "tokens": tokens.int(),
                "slots": slots.int().view(s["ids"].shape)}
    if c["op"] == "combine":
        y, w, g = s["y"].to(D), s["weights"].to(D), s["grad_out"].to(D)
        out, grad_w, grad_y = torch.zeros_like(g), torch.zeros_like(w), torch.zeros_like(y)
        for j in range(c["top"]):
            t = (s["slots"][:, j] >= 0).nonzero()[:, 0]
            r = s["slots"][t, j].long()
            out[t] += w[t, j, None] * y[r]
            grad_w[t, j] = torch.linalg.vecdot(g[t], y[r])
            grad_y[r] = w[t, j, None] * g[t]
        return {"out": out, "grad_y": grad_y, "grad_weights": grad_w}
    ends = s["offsets"].tolist()
    if c["op"] == "matmul":
        out = torch.zeros(s["x"].shape[0], c["out"], dtype=D, device="cuda")
        for e in range(c["experts"]):
            out[ends[e]:ends[e + 1]] = s["x"][ends[e]:ends[e + 1]].to(D) @ s["weight"][e].to(D).T
        return {"out": out}
    grad_x = torch.zeros(s["x"].shape, dtype=D, device="cuda")
    grad_w = s["grad_weight"].to(D) if c["accumulate"] else torch.zeros(s["weight"].shape, dtype=D, device="cuda")
    for e in range(c["experts"]):
        a, b = ends[e], ends[e + 1]
        g = s["grad_out"][a:b].to(D)
        grad_x[a:b] = g @ s["weight"][e].to(D)
        grad_w[e] += g.T @ s["x"][a:b].to(D)
    return {"grad_x": grad_x, "grad_weight": grad_w}
