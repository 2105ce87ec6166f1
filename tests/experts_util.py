"""64-bit definitions of the expert layer's operators, with the sums of the
magnitudes of the terms, and groups of rows to run them on."""
import torch

from training_util import D


def groups(kind, experts, rows, seed=0):
    """offsets of `experts` groups among `rows` rows (int32, CUDA), as a list too."""
    r = torch.Generator().manual_seed(seed)
    if kind == "even":
        cuts = [rows * e // experts for e in range(experts + 1)]
    elif kind == "skewed":  # a few experts hold most rows, some none, some rows are in no group
        share = torch.rand(experts, generator=r) ** 6
        share[torch.rand(experts, generator=r) < 0.3] = 0
        share[int(torch.randint(0, experts, (1,), generator=r))] += 0.1
        ends = (share.cumsum(0) / share.sum() * max(0, rows - rows // 10)).long().tolist()
        cuts = [0] + ends
    elif kind == "last":  # all rows in the last group, which begins behind some rows
        cuts = [rows // 7] * experts + [rows]
    elif kind == "none":
        cuts = [0] * (experts + 1)
    else:
        raise ValueError(kind)
    return torch.tensor(cuts, dtype=torch.int32, device="cuda"), cuts


def matmul(x, weight, cuts):
    """(out, magnitude) in 64 bits; NaN where no group is."""
    out = torch.full((x.shape[0], weight.shape[1]), float("nan"), dtype=D, device=x.device)
    mag = torch.zeros_like(out)
    for e in range(weight.shape[0]):
        a, b = cuts[e], cuts[e + 1]
        w = weight[e].to(D).t()
        out[a:b] = x[a:b].to(D) @ w
        mag[a:b] = x[a:b].to(D).abs() @ w.abs()
    return out, mag


def matmul_grad(grad_out, x, weight, cuts, old=None):
    """(grad_x, its magnitude, grad_weight, its magnitude, rows of each expert)"""
    gx, gx_mag = matmul(grad_out, weight.transpose(1, 2), cuts)
    gw = torch.zeros(weight.shape, dtype=D, device=x.device) if old is None else old.to(D).clone()
    mag = gw.abs()
    n = torch.zeros(weight.shape[0], 1, 1, dtype=D, device=x.device)
    for e in range(weight.shape[0]):
        a, b = cuts[e], cuts[e + 1]
        g, v = grad_out[a:b].to(D), x[a:b].to(D)
        gw[e] += g.t() @ v
        mag[e] += g.abs().t() @ v.abs()
        n[e] = b - a
    return gx, gx_mag, gw, mag, n


def plan(ids, experts, first):
    """(offsets, tokens, slots) as lists, by definition."""
    flat = ids.reshape(-1).tolist()
    top = ids.shape[1]
    slots, tokens, offsets = [-1] * len(flat), [-1] * len(flat), [0]
    mine = {}
    for i, e in enumerate(flat):
        mine.setdefault(e - first, []).append(i)
    at = 0
    for e in range(experts):
        for i in mine.get(e, []):
            slots[i], tokens[at] = at, i // top
            at += 1
        offsets.append(at)
    return offsets, tokens, slots
