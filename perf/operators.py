"""What is measured of the training operators: cases over their range, the
operators in plain torch operations (32-bit, rounded once at the end), the
calls a user makes of the library, and their definitions in 64 bits.

The operators are those of one training step around the collectives: the
embedding lookup and its gradient, the norms and the gate at a block's
boundary with their gradient, and the distillation loss on a teacher's top
logits with its gradient.
"""
import math

import torch

own = False

F32, BF16 = "float32", "bfloat16"
SIZE = {F32: 4, BF16: 2, "int32": 4, "int64": 8}
TYPE = {F32: torch.float32, BF16: torch.bfloat16, "int32": torch.int32, "int64": torch.int64}


def listed():
    return [
        # the embedding of one new token: nothing but latency
        _embedding("embedding_1x1024", 1, 32768, 1024, BF16, BF16, "int64"),
        # a training batch of tokens, fp32 master table, bf16 activations
        _embedding("embedding_16384x4096", 16384, 131072, 4096, F32, BF16, "int64"),
        # the gradient of a short fine-tuning prompt, added to what earlier micro-batches left
        _embedding_grad("embedding_grad_33x1024", 33, 32768, 1024, BF16, F32, "int64", accumulate=True),
        # the gradient of one rank's rows of a vocabulary split over four ranks, odd sizes, 16-bit gradients
        _embedding_grad("embedding_grad_16411x1000_shard", 16411, 32003, 1000, BF16, BF16, "int32", rows=8001,
                        first=500, accumulate=True),
        # a training batch's dense gradient, ready for an AllReduce over the data-parallel ranks
        _embedding_grad("embedding_grad_65536x2048", 65536, 131072, 2048, BF16, F32, "int64"),
        # the block boundary of one new token
        _norm("block_norm_1x4096", 1, 4096, BF16, BF16, 1),
        # the block boundary of a training batch of eight sequences, a gate for each
        _norm("block_norm_16384x4096", 16384, 4096, BF16, BF16, 8),
        # its gradient on a small fp32 model with a gate for every token, odd sizes
        _norm("block_norm_grad_509x1001", 509, 1001, F32, F32, 509, grad=True),
        # its gradient on a training batch
        _norm("block_norm_grad_16384x4096", 16384, 4096, BF16, F32, 8, grad=True),
        # the loss and its gradient on a few answer tokens of a small vocabulary
        _distill("distill_8x32768", 8, 32768, 16, BF16, "int64"),
        # the loss for the log and, later, its gradient, fp32 logits of an odd vocabulary
        _distill("distill_509x50021_split", 509, 50021, 33, F32, "int32", split=True),
        # the loss and its gradient over a training batch's logits
        _distill("distill_4096x131072", 4096, 131072, 64, BF16, "int64"),
    ]


def _embedding(name, tokens, vocab, dim, table, out, ids, rows=None, first=0):
    return {"name": name, "op": "embedding", "tokens": tokens, "vocab": vocab, "rows": rows or vocab, "first": first,
            "dim": dim, "table": table, "out": out, "ids": ids, "scale": math.sqrt(dim)}


def _embedding_grad(name, tokens, vocab, dim, out, table, ids, rows=None, first=0, accumulate=False):
    return {"name": name, "op": "embedding_grad", "tokens": tokens, "vocab": vocab, "rows": rows or vocab,
            "first": first, "dim": dim, "table": table, "out": out, "ids": ids, "scale": math.sqrt(dim),
            "padding": 3, "accumulate": accumulate}


def _norm(name, tokens, dim, dtype, weight, gates, grad=False):
    return {"name": name, "op": "block_norm_grad" if grad else "block_norm", "tokens": tokens, "dim": dim,
            "dtype": dtype, "weight": weight, "gates": gates, "residual_scale": 0.75, "eps": 1e-6}


def _distill(name, tokens, vocab, top, dtype, ids, split=False):
    return {"name": name, "op": "distill", "tokens": tokens, "vocab": vocab, "top": top, "dtype": dtype, "ids": ids,
            "split": split, "temperature": 2.0, "scale": 1.0 / tokens}


def draw(rng):
    """A case of the same kinds: sizes log-uniform over the listed ones'
    range, about half of them odd, at most about 0.8 GB of work."""
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n if rng.random() < 0.5 else max(lo, n // 8 * 8)

    kind = rng.choice(["embedding", "embedding_grad", "embedding_grad", "block_norm", "block_norm_grad", "distill",
                       "distill"])
    most = 0.8e9
    while True:
        dtype, wide = rng.choice([BF16, BF16, F32]), rng.choice([BF16, F32])
        ids = rng.choice(["int32", "int64"])
        if kind in ("embedding", "embedding_grad"):
            tokens, vocab, dim = size(1, 65536), size(1000, 131072), size(64, 8192)
            rows, first = vocab, 0
            if tokens >= 256 and rng.random() < 0.3:
                rows = max(1, vocab // 4)
                first = rng.randrange(0, vocab - rows + 1)
            if kind == "embedding":
                c = _embedding("", tokens, vocab, dim, wide, dtype, ids, rows, first)
            else:
                c = _embedding_grad("", tokens, vocab, dim, dtype, wide, ids, rows, first, rng.random() < 0.5)
        elif kind.startswith("block_norm"):
            gates = rng.choice([1, 2, 4, 8, 0])
            tokens = size(1, 32768)
            if gates == 0:
                gates = tokens
            tokens = max(1, tokens // gates) * gates
            c = _norm("", tokens, size(64, 8192), dtype, wide, gates, kind == "block_norm_grad")
        else:
            c = _distill("", size(1, 4096), size(1000, 131072), size(1, 128), dtype, ids, rng.random() < 0.4)
        del c["name"]
        if work(c)["bytes"] <= most and c.get("rows", 0) * c["dim" if "dim" in c else "vocab"] * 4 <= 2.0e9:
            return c


def _distinct(c):
    """Distinct rows of this rank expected among the tokens' ids."""
    r = torch.arange(c["first"] + 1, c["first"] + c["rows"] + 1, dtype=torch.float64)
    p = torch.log1p(1 / r) / math.log(c["vocab"] + 1)
    return float((1 - torch.exp(c["tokens"] * torch.log1p(-p))).sum())


def work(case):
    c = case
    if c["op"].startswith("embedding"):
        T, d, share = c["tokens"], c["dim"], _share(c)
        distinct = _distinct(c)
        ids = T * SIZE[c["ids"]]
        if c["op"] == "embedding":
            return {"bytes": ids + distinct * d * SIZE[c["table"]] + T * d * SIZE[c["out"]], "flops": T * share * d}
        rows = 2 * distinct if c["accumulate"] else c["rows"]
        return {"bytes": ids + T * share * d * SIZE[c["out"]] + rows * d * SIZE[c["table"]], "flops": 2 * T * share * d}
    if c["op"] == "block_norm":
        n = c["tokens"] * c["dim"]
        return {"bytes": 4 * n * SIZE[c["dtype"]] + (2 + c["gates"]) * c["dim"] * SIZE[c["weight"]] + 8 * c["tokens"],
                "flops": 11 * n}
    if c["op"] == "block_norm_grad":
        n = c["tokens"] * c["dim"]
        return {"bytes": 6 * n * SIZE[c["dtype"]] + 2 * (2 + c["gates"]) * c["dim"] * SIZE[c["weight"]]
                + 8 * c["tokens"], "flops": 28 * n}
    n = c["tokens"] * c["vocab"]
    top = c["tokens"] * c["top"] * (4 + SIZE[c["ids"]])
    passes = 3 if c["split"] else 2
    return {"bytes": passes * n * SIZE[c["dtype"]] + top * (2 if c["split"] else 1) + 16 * c["tokens"],
            "flops": 8 * n}


def _share(c):
    """Share of the tokens whose row is on this rank (1/rank frequencies)."""
    return (math.log(c["first"] + c["rows"] + 1) - math.log(c["first"] + 1)) / math.log(c["vocab"] + 1)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, dtype=F32, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(TYPE[dtype])

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    T = c["tokens"]
    s = {"case": c}
    if c["op"].startswith("embedding"):
        # word frequencies fall as 1/rank; about 1 in 50 tokens is padding (-1, or the padding id)
        u = uniform(T).double()
        ids = (torch.exp(u * math.log(c["vocab"] + 1)).long() - 1).clamp_(0, c["vocab"] - 1)
        if T > 1:
            v = uniform(T)
            ids = torch.where(v < 0.01, -1, ids)
            ids = torch.where(v > 0.99, 3, ids)
        s["ids"] = ids.to(TYPE[c["ids"]])
        if c["op"] == "embedding":
            s["table"] = normal(c["rows"], c["dim"], dtype=c["table"], std=0.02)
        else:
            s["grad_out"] = normal(T, c["dim"], dtype=c["out"], std=1e-2)
            # the buffer the gradient goes to; when adding to it, what earlier micro-batches left
            s["grad_table"] = normal(c["rows"], c["dim"], dtype=c["table"], std=1e-1) if c["accumulate"] else \
                torch.empty(c["rows"], c["dim"], dtype=TYPE[c["table"]], device="cuda")
    elif c["op"].startswith("block_norm"):
        d, G = c["dim"], c["gates"]
        s["y"] = normal(T, d, dtype=c["dtype"], std=2.0)
        s["x"] = normal(T, d, dtype=c["dtype"], std=4.0)
        s["post_weight"] = (1 + normal(d, std=0.1)).to(TYPE[c["weight"]])
        s["pre_weight"] = (1 + normal(d, std=0.1)).to(TYPE[c["weight"]])
        s["gate"] = normal(G, d, dtype=c["weight"], std=0.5)
        if c["op"] == "block_norm_grad":
            s["grad_r"] = normal(T, d, dtype=c["dtype"], std=1e-2)
            s["grad_z"] = normal(T, d, dtype=c["dtype"], std=1e-2)
            _, _, s["post_rstd"], s["pre_rstd"] = _norm_parts(s)  # what the forward pass kept
    else:
        V, K = c["vocab"], c["top"]
        s["logits"] = normal(T, V, dtype=c["dtype"], std=2.0)
        pad = V // 100  # the vocabulary is padded: its last columns are masked off
        if pad:
            s["logits"][:, V - pad:] = -math.inf
        s["teacher_logits"] = (normal(T, K) * 3).sort(dim=1, descending=True).values
        tid = torch.randint(0, V - pad, (T, K), generator=g, device="cuda")
        # some teacher rows hold fewer than K entries
        have = torch.randint(max(1, K // 2), K + 1, (T, 1), generator=g, device="cuda")
        tid = torch.where(torch.arange(K, device="cuda")[None, :] < have, tid, -1)
        s["teacher_ids"] = tid.to(TYPE[c["ids"]])
        # prompt tokens carry no loss
        s["row_weight"] = (uniform(T) < 0.9).float() if T > 1 else torch.ones(1, device="cuda")
    if own:
        _bind(s)
    return s


def _bind(s):
    """The calls a training program binds once to its buffers and repeats every
    step, and the output buffers and scratch it keeps for them."""
    import collective_communication_algorithms_gb300 as hc
    c = s["case"]
    if c["op"] == "embedding":
        s["calls"] = [hc.bind_embedding(s["table"], s["ids"], scale=c["scale"], first_id=c["first"],
                                        out_dtype=TYPE[c["out"]])]
        s["outputs"] = {"out": s["calls"][0].outputs["out"]}
    elif c["op"] == "embedding_grad":
        s["calls"] = [hc.bind_embedding_grad(s["grad_out"], s["ids"], s["grad_table"], scale=c["scale"],
                                             first_id=c["first"], padding_id=c["padding"],
                                             accumulate=c["accumulate"])]
        s["outputs"] = {"grad_table": s["grad_table"]}
    elif c["op"] == "block_norm":
        s["calls"] = [hc.bind_block_norm(s["y"], s["x"], post_weight=s["post_weight"], gate=s["gate"],
                                         pre_weight=s["pre_weight"], residual_scale=c["residual_scale"],
                                         eps=c["eps"])]
        o = s["calls"][0].outputs
        s["outputs"] = {k: o[k] for k in ("r", "z", "post_rstd", "pre_rstd")}
    elif c["op"] == "block_norm_grad":
        s["calls"] = [hc.bind_block_norm_grad(s["grad_r"], s["grad_z"], s["y"], s["x"], s["post_rstd"],
                                              s["pre_rstd"], post_weight=s["post_weight"], gate=s["gate"],
                                              pre_weight=s["pre_weight"], residual_scale=c["residual_scale"])]
        o = s["calls"][0].outputs
        s["outputs"] = {k: o[k] for k in ("grad_y", "grad_x", "grad_post_weight", "grad_gate", "grad_pre_weight")}
    elif c["split"]:
        a = hc.bind_distill(s["logits"], s["teacher_logits"], s["teacher_ids"], row_weight=s["row_weight"],
                            grad=False, temperature=c["temperature"], scale=c["scale"])
        b = hc.bind_distill_grad(s["logits"], s["teacher_logits"], s["teacher_ids"], a.outputs["stats"],
                                 row_weight=s["row_weight"], temperature=c["temperature"], scale=c["scale"])
        s["calls"] = [a, b]
        s["outputs"] = {"loss": a.outputs["loss"], "stats": a.outputs["stats"], "grad": b.outputs["grad"]}
    else:
        a = hc.bind_distill(s["logits"], s["teacher_logits"], s["teacher_ids"], row_weight=s["row_weight"],
                            temperature=c["temperature"], scale=c["scale"])
        s["calls"] = [a]
        s["outputs"] = {k: a.outputs[k] for k in ("loss", "stats", "grad")}


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        for call in state["calls"]:
            call()
        return state["outputs"]
    return PLAIN[state["case"]["op"]](state)


def _plain_embedding(s):
    c = s["case"]
    at = s["ids"].long() - c["first"]
    here = (at >= 0) & (at < c["rows"])
    rows = s["table"][at.clamp(0, c["rows"] - 1)].float() * c["scale"]
    return {"out": torch.where(here[:, None], rows, 0.0).to(TYPE[c["out"]])}


def _plain_embedding_grad(s):
    c = s["case"]
    ids = s["ids"].long()
    at = ids - c["first"]
    here = (at >= 0) & (at < c["rows"]) & (ids != c["padding"])
    rows = torch.where(here[:, None], s["grad_out"].float() * c["scale"], 0.0)
    at = at.clamp(0, c["rows"] - 1)
    table = s["grad_table"]
    if table.dtype == torch.float32:
        if not c["accumulate"]:
            table.zero_()
        table.index_add_(0, at, rows)
    else:
        total = table.float() if c["accumulate"] else torch.zeros(table.shape, device="cuda")
        total.index_add_(0, at, rows)
        table.copy_(total)
    return {"grad_table": table}


def _norm_parts(s):
    c = s["case"]
    y, x = s["y"].float(), s["x"].float()
    post_rstd = torch.rsqrt((y * y).mean(dim=1) + c["eps"])
    n = y * post_rstd[:, None] * s["post_weight"].float()
    gate = s["gate"].float().repeat_interleave(c["tokens"] // c["gates"], dim=0)
    r = c["residual_scale"] * x + gate * n
    pre_rstd = torch.rsqrt((r * r).mean(dim=1) + c["eps"])
    return r, gate, post_rstd, pre_rstd


def _plain_block_norm(s):
    t = TYPE[s["case"]["dtype"]]
    r, _, post_rstd, pre_rstd = _norm_parts(s)
    z = r * pre_rstd[:, None] * s["pre_weight"].float()
    return {"r": r.to(t), "z": z.to(t), "post_rstd": post_rstd, "pre_rstd": pre_rstd}


def _plain_block_norm_grad(s):
    c = s["case"]
    t, w = TYPE[c["dtype"]], TYPE[c["weight"]]
    gz, gr = s["grad_z"].float(), s["grad_r"].float()
    gate = s["gate"].float().repeat_interleave(c["tokens"] // c["gates"], dim=0)
    post = s["post_weight"].float()
    y_hat = s["y"].float() * s["post_rstd"][:, None]
    r_hat = (c["residual_scale"] * s["x"].float() + gate * (y_hat * post)) * s["pre_rstd"][:, None]
    h = gz * s["pre_weight"].float()
    total = gr + s["pre_rstd"][:, None] * (h - r_hat * (h * r_hat).mean(dim=1, keepdim=True))
    a = total * y_hat
    k = total * gate * post
    grad_y = s["post_rstd"][:, None] * (k - y_hat * (k * y_hat).mean(dim=1, keepdim=True))
    grad_gate = (a * post).view(c["gates"], -1, c["dim"]).sum(dim=1)
    return {"grad_y": grad_y.to(t), "grad_x": (c["residual_scale"] * total).to(t),
            "grad_post_weight": (a * gate).sum(dim=0).to(w), "grad_gate": grad_gate.to(w),
            "grad_pre_weight": (gz * r_hat).sum(dim=0).to(w)}


def _plain_distill(s):
    c = s["case"]
    tau = c["temperature"]
    x = s["logits"].float()
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp((x - top) / tau)
    total = e.sum(dim=1, keepdim=True)
    ids = s["teacher_ids"].long()
    valid = (ids >= 0) & (ids < c["vocab"])
    ids = ids.clamp(0, c["vocab"] - 1)
    t = torch.where(valid, s["teacher_logits"].float(), -math.inf)
    t_top = t.amax(dim=1, keepdim=True)
    t = t - torch.where(t_top > -math.inf, t_top, 0.0)
    te = torch.exp(t / tau)
    t_total = te.sum(dim=1, keepdim=True)
    weight = (s["row_weight"] * c["scale"])[:, None]
    active = (weight != 0) & (t_total > 0)
    p = te / torch.where(t_total > 0, t_total, 1.0)
    log_p = t / tau - torch.log(t_total)
    log_q = (x.gather(1, ids) - top) / tau - torch.log(total)
    loss = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(dim=1, keepdim=True) * (tau * tau) * weight
    grad = (e / total).scatter_add_(1, ids, -p) * (tau * weight)
    return {"loss": torch.where(active, loss, 0.0)[:, 0],
            "stats": torch.where(active, torch.cat([top, total], dim=1), 0.0),
            "grad": torch.where(active, grad, 0.0).to(TYPE[c["dtype"]])}


PLAIN = {"embedding": _plain_embedding, "embedding_grad": _plain_embedding_grad, "block_norm": _plain_block_norm,
         "block_norm_grad": _plain_block_norm_grad, "distill": _plain_distill}


# ------------------------------------------------------------------ definitions in 64 bits
def exact(case, seed):
    c = case
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    D = torch.float64
    if c["op"] == "embedding":
        padded = torch.cat([s["table"].to(D) * c["scale"], torch.zeros(1, c["dim"], dtype=D, device="cuda")])
        at = s["ids"].long() - c["first"]
        at[(at < 0) | (at >= c["rows"])] = c["rows"]
        return {"out": padded[at]}
    if c["op"] == "embedding_grad":
        keep = ((s["ids"] >= c["first"]) & (s["ids"] < c["first"] + c["rows"]) & (s["ids"] != c["padding"])).nonzero()[:, 0]
        at, order = torch.sort(s["ids"].long()[keep] - c["first"], stable=True)
        g = s["grad_table"].to(D) if c["accumulate"] else torch.zeros(c["rows"], c["dim"], dtype=D, device="cuda")
        return {"grad_table": g.index_add_(0, at, s["grad_out"][keep[order]].to(D), alpha=c["scale"])}
    if c["op"].startswith("block_norm"):
        leaf = {k: s[k].to(D).requires_grad_() for k in ("y", "x", "post_weight", "gate", "pre_weight")}
        y, x = leaf["y"], leaf["x"]
        n = torch.nn.functional.rms_norm(y, (c["dim"],), leaf["post_weight"], c["eps"])
        T, G, d = c["tokens"], c["gates"], c["dim"]
        r = x * c["residual_scale"] + (n.view(G, T // G, d) * leaf["gate"][:, None, :]).view(T, d)
        z = torch.nn.functional.rms_norm(r, (d,), leaf["pre_weight"], c["eps"])
        if c["op"] == "block_norm":
            with torch.no_grad():
                return {"r": r, "z": z, "post_rstd": (y.pow(2).sum(1) / d + c["eps"]).pow(-0.5),
                        "pre_rstd": (r.pow(2).sum(1) / d + c["eps"]).pow(-0.5)}
        torch.autograd.backward([r, z], [s["grad_r"].to(D), s["grad_z"].to(D)])
        return {"grad_" + k: v.grad for k, v in leaf.items()}
    tau, parts = c["temperature"], []
    step = max(1, (1 << 26) // c["vocab"])
    for a in range(0, c["tokens"], step):
        x = s["logits"][a:a + step].to(D).requires_grad_()
        ids = s["teacher_ids"][a:a + step].long()
        off = (ids < 0) | (ids >= c["vocab"])
        log_p = torch.log_softmax(s["teacher_logits"][a:a + step].to(D).masked_fill(off, -math.inf) / tau, dim=1)
        log_q = torch.log_softmax(x / tau, dim=1).gather(1, ids.masked_fill(off, 0))
        kl = (log_p.exp() * (log_p - log_q)).masked_fill(off, 0.0).sum(dim=1)
        w = s["row_weight"][a:a + step].to(D) * c["scale"]
        loss = kl * w * tau ** 2
        loss.sum().backward()
        with torch.no_grad():
            top = x.max(dim=1).values
            total = torch.exp(torch.logsumexp(x / tau, dim=1) - top / tau)
            stats = torch.stack([top, total], dim=1) * (w != 0)[:, None]
        parts.append((loss.detach(), stats, x.grad))
    loss, stats, grad = (torch.cat(v) for v in zip(*parts))
    return {"loss": loss, "stats": stats, "grad": grad}
