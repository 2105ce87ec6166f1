"""64-bit definitions of the training operators, with, for every output, the
sum of the magnitudes of the terms that make it (what rounding errors are
relative to), and buffers with guard bands."""
import torch

D = torch.float64
BITS = {torch.float32: 24, torch.bfloat16: 8}  # of the significand, with its leading one
EPS = 2.0 ** -24


def guarded(rows, cols, dtype, stride=None, offset=0):
    """(view, check): a rows x cols view with the given row stride, `offset`
    elements after a 16-byte boundary, and a function that says whether
    everything around the view's elements is as it was."""
    stride = stride or cols
    guard = 64
    flat = torch.full((guard + offset + max(rows, 1) * stride + guard,), -7.25, dtype=dtype, device="cuda")
    view = flat[guard + offset:].as_strided((rows, cols), (stride, 1))
    mask = torch.ones_like(flat, dtype=torch.bool)
    mask[guard + offset:].as_strided((rows, cols), (stride, 1)).fill_(False)

    def intact():
        return bool((flat[mask] == -7.25).all())
    return view, intact


def strided(t, stride=None, offset=0):
    """t's values in a strided, offset view (guards around it)."""
    view, _ = guarded(t.shape[0], t.shape[1], t.dtype, stride, offset)
    view.copy_(t)
    return view


def half_ulp(ref, dtype):
    """Half a unit in the last place of dtype at ref."""
    _, e = torch.frexp(ref)  # |ref| in [2^(e-1), 2^e)
    return torch.ldexp(torch.ones_like(ref), e - 1 - BITS[dtype])


def assert_close(got, ref, mag, ops, name=""):
    """|got - ref| <= (half a unit in got's last place) + ops * 2^-24 * mag, and the
    same infinities and NaNs."""
    ref, mag = ref.to("cuda"), mag.to("cuda")
    g = got.to(D)
    odd = ~torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), name
    assert torch.equal(g[odd & ~torch.isnan(ref)], ref[odd & ~torch.isnan(ref)]), name
    bound = half_ulp(ref.masked_fill(odd, 0.0), got.dtype) + ops * EPS * mag + 1e-37
    bad = ((g - ref).abs() > bound * 1.001) & ~odd
    if bool(bad.any()):
        i = bad.nonzero()[0].tolist()
        raise AssertionError("%s: %d of %d off; at %s: %r, not %r (bound %.3g)"
                             % (name, int(bad.sum()), bad.numel(), i, float(g[tuple(i)]), float(ref[tuple(i)]),
                                float(bound[tuple(i)])))


def embedding(table, ids, scale, first):
    at = ids.reshape(-1).to(torch.int64) - first
    out = torch.zeros(at.numel(), table.shape[1], dtype=D, device=table.device)
    here = (at >= 0) & (at < table.shape[0])
    out[here] = table.to(D)[at[here]] * scale
    return out


def embedding_grad(grad_out, ids, rows, scale, first, padding, old=None):
    """(gradient, magnitude, tokens of every row)"""
    ids = ids.reshape(-1).to(torch.int64)
    at = ids - first
    here = (at >= 0) & (at < rows)
    if padding >= 0:
        here &= ids != padding
    dev, dim = grad_out.device, grad_out.shape[1]
    g = torch.zeros(rows, dim, dtype=D, device=dev) if old is None else old.to(D).clone()
    mag = g.abs()
    n = torch.zeros(rows, dtype=D, device=dev)
    terms = grad_out[here].to(D) * scale
    g.index_add_(0, at[here], terms)
    mag.index_add_(0, at[here], terms.abs())
    n.index_add_(0, at[here], torch.ones_like(at[here], dtype=D))
    return g, mag, n


def block_norm(y, x, post, gate, pre, a, eps):
    """r, z, post_rstd, pre_rstd and the magnitude of r's terms, in 64 bits;
    post, gate (expanded to rows) and pre are 64-bit tensors or 1.0."""
    y, x = y.to(D), x.to(D)
    s = ((y * y).mean(dim=1, keepdim=True) + eps) ** -0.5
    n = gate * (y * s * post)
    r = a * x + n
    q = ((r * r).mean(dim=1, keepdim=True) + eps) ** -0.5
    return r, r * q * pre, s, q, (a * x).abs() + n.abs()


def distill(logits, teacher, ids, weight, tau, scale):
    """loss, grad, stats, active rows, and the log-probabilities' sizes."""
    x, t = logits.to(D), teacher.to(D)
    ids = ids.to(torch.int64)
    valid = (ids >= 0) & (ids < x.shape[1]) & (t != -torch.inf)
    w = (weight.to(D) if weight is not None else torch.ones(x.shape[0], dtype=D, device=x.device)) * scale
    active = (w != 0) & valid.any(dim=1)
    safe = ids.masked_fill(~valid, 0)
    x = torch.where(active[:, None], x, 0.0)
    t = torch.where(active[:, None], t, 0.0)
    log_q = torch.log_softmax(x / tau, dim=1)
    valid_or = valid | ~active[:, None]
    log_p = torch.log_softmax((t / tau).masked_fill(~valid_or, -torch.inf), dim=1)
    p = torch.where(valid, log_p.exp(), 0.0)
    lq = log_q.gather(1, safe)
    terms = torch.where(p != 0, p * (log_p - lq), 0.0)
    sizes = torch.where(p != 0, p * (1 + log_p.abs() + lq.abs()), 0.0).sum(dim=1)
    top = x.max(dim=1).values
    a = (top[:, None] - x) / tau
    e = torch.exp(-a)
    total = e.sum(dim=1)
    total_mag = torch.where(e > 0, e * (4 + a), 0.0).sum(dim=1)
    scat = torch.zeros_like(x).scatter_add_(1, safe, p)
    g = w[:, None] * tau * (log_q.exp() - scat)
    mag = (w[:, None] * tau).abs() * (log_q.exp() * (4 + log_q.abs()) + 4 * scat)
    z = torch.zeros((), dtype=D, device=x.device)
    loss = torch.where(active, w * tau * tau * terms.sum(dim=1), z)
    return {"loss": loss, "loss_mag": torch.where(active, (w * tau * tau).abs() * sizes, z),
            "grad": torch.where(active[:, None], g, z), "grad_mag": torch.where(active[:, None], mag, z),
            "stats": torch.where(active[:, None], torch.stack([top, total], dim=1), z),
            "stats_mag": torch.where(active[:, None], torch.stack([top.abs(), total_mag], dim=1), z)}
