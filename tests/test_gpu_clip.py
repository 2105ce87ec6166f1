"""Gradient clipping against its definition in 64 bits: types, many tensors,
odd sizes and places, values whose squares overflow or vanish, NaN and
infinities, in place and apart, after an AllReduce, in graphs.

Bounds: the norm is a binary64 sum of groups of at most 64 squares summed in
binary32 (64 roundings of 2^-24, half of which a square root leaves), rounded
once; an output is one product by a factor that is off by as much as the norm
and one rounding of its own, and is rounded once.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import collective_communication_algorithms_gb300 as hc  # noqa: E402
from training_util import D, assert_close, half_ulp  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NORM_OPS = 34  # 64 / 2, and the final roundings


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from collective_communication_algorithms_gb300 import build
    build.build()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def place(values, offset, dtype):
    """values at an offset of elements behind a 16-byte boundary, guards around."""
    flat = torch.full((64 + offset + values.numel() + 64,), -7.25, dtype=dtype, device="cuda")
    v = flat[64 + offset:64 + offset + values.numel()]
    v.copy_(values)
    return v, lambda: bool((flat[:64 + offset] == -7.25).all() and (flat[64 + offset + values.numel():] == -7.25).all())


def norm_of(ts):
    return math.sqrt(sum(float((t.to(D) ** 2).sum()) for t in ts))


def check(grads, before, o, max_norm, scale, eps):
    ref = norm_of(before) * abs(scale)
    assert abs(float(o["norm"]) - ref) <= NORM_OPS * 2.0 ** -24 * ref
    factor = min(1.0, max_norm / (ref + eps)) * scale
    assert abs(float(o["factor"]) - factor) <= (NORM_OPS + 2) * 2.0 ** -24 * abs(factor)
    for g, b in zip(grads, before):
        want = b.to(D) * factor
        assert_close(g, want, want.abs(), NORM_OPS + 3, "grad")


SIZES = [1, 2, 3, 7, 8, 9, 31, 1001, 0, 16384, 16385, 70001, 8191, 40000]


@pytest.mark.parametrize("in_dtype,out_dtype", [(F32, None), (BF16, None), (F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("max_norm,scale", [(1.0, 0.25), (1e9, 1.0), (1e9, -0.5), (2.0, 1.0)])
def test_clip(in_dtype, out_dtype, max_norm, scale):
    g = gen(1)
    grads, outs, intacts = [], [], []
    for i, n in enumerate(SIZES):
        v, ok = place(torch.randn(n, generator=g, device="cuda"), i % 9, in_dtype)
        grads.append(v)
        intacts.append(ok)
        if out_dtype is not None:
            v, ok = place(torch.zeros(n, device="cuda"), (i * (1 + i % 2)) % 9, out_dtype)
            outs.append(v)
            intacts.append(ok)
    before = [v.clone() for v in grads]
    o = hc.clip_grads(grads, max_norm, out=outs or None, scale=scale)
    check(outs or grads, before, o, max_norm, scale, 1e-6)
    assert all(ok() for ok in intacts)
    if outs:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    n = hc.grad_norm(before, scale=scale)["norm"]
    assert torch.equal(n, o["norm"])


@pytest.mark.parametrize("num", [1, 31, 32, 33, 255, 257, 1160, 1161, 2500])
def test_many_tensors(num):
    g = gen(num)
    n = torch.randint(1, 400, (num,), generator=torch.Generator().manual_seed(num)).tolist()
    grads = [torch.randn(k, generator=g, device="cuda").to(BF16 if i % 3 == 0 else F32) for i, k in enumerate(n)]
    before = [v.clone() for v in grads]
    o = hc.clip_grads(grads, 1.0)
    check(grads, before, o, 1.0, 1.0, 1e-6)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e-13, 1e13, 1e18, 1e25, 2e36])
def test_squares_that_binary32_does_not_hold(dtype, size):
    g = gen(4)
    grads = [(torch.randn(5000, generator=g, device="cuda") * size).to(dtype),
             (torch.randn(300, generator=g, device="cuda") * size * 1e-3).to(dtype)]
    before = [v.clone() for v in grads]
    o = hc.clip_grads(grads, 0.5 * size, eps=0.0)
    check(grads, before, o, 0.5 * size, 1.0, 0.0)


def test_a_few_huge_values_among_small_ones():
    g = gen(6)
    grads = [torch.randn(50000, generator=g, device="cuda") * 1e-25, torch.zeros(3000, device="cuda")]
    grads[0][17] = 3e25
    grads[1][5] = -4e25
    assert float(hc.grad_norm(grads)["norm"]) == pytest.approx(5e25, rel=1e-6)
    assert float(hc.grad_norm([grads[0][100:200]])["norm"]) == pytest.approx(norm_of([grads[0][100:200]]), rel=1e-6)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nan_and_infinities(dtype):
    a = torch.ones(1000, device="cuda", dtype=dtype)
    a[3] = float("inf")
    b = torch.ones(9, device="cuda", dtype=dtype)
    o = hc.clip_grads([a, b], 1.0)
    assert float(o["norm"]) == math.inf and float(o["factor"]) == 0.0
    assert bool(torch.isnan(a[3])) and bool((a[:3] == 0).all()) and bool((b == 0).all())
    a.fill_(1)
    a[999] = float("nan")
    o = hc.clip_grads([a, b], 1.0)
    assert math.isnan(float(o["norm"])) and bool(torch.isnan(a).all()) and bool(torch.isnan(b).all())
    c = torch.ones(4, device="cuda", dtype=dtype)
    c[0] = float("inf")
    o = hc.clip_grads([c], math.inf)  # no limit: untouched
    assert c.tolist() == [math.inf, 1.0, 1.0, 1.0]


def test_zeros_and_no_limit():
    z = [torch.zeros(77, device="cuda"), torch.zeros(0, device="cuda")]
    o = hc.clip_grads(z, 1.0)
    assert float(o["norm"]) == 0.0 and float(o["factor"]) == 1.0 and bool((z[0] == 0).all())
    o = hc.clip_grads([torch.zeros(0, device="cuda")], 1.0)
    assert float(o["norm"]) == 0.0
    g = torch.randn(1000, device="cuda")
    b = g.clone()
    o = hc.clip_grads([g], math.inf)
    assert torch.equal(g, b) and float(o["factor"]) == 1.0
    o = hc.clip_grads([g], math.inf, scale=0.5)
    assert torch.equal(g, b * 0.5) and float(o["factor"]) == 0.5


def test_below_the_limit_in_place_is_bit_exact():
    g = torch.randn(5000, device="cuda", generator=gen(8))
    b = g.clone()
    hc.clip_grads([g], 1e6)
    assert torch.equal(g, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large(dtype):
    """More chunks than blocks, and the same bits again."""
    g = gen(10)
    grads = [torch.randn(30_000_001, generator=g, device="cuda").to(dtype), torch.randn(7_000_003, generator=g, device="cuda")]
    before = [v.clone() for v in grads]
    outs = [torch.empty_like(v, dtype=F32) for v in grads]
    o = hc.clip_grads(grads, 3.0, out=outs, scale=0.5)
    check(outs, before, o, 3.0, 0.5, 1e-6)
    again = hc.clip_grads(grads, 3.0, out=[torch.empty_like(v, dtype=F32) for v in grads], scale=0.5)
    assert torch.equal(again["norm"], o["norm"]) and all(torch.equal(a, b) for a, b in zip(again["grads"], outs))


def test_after_an_allreduce():
    """The mean of the ranks' gradients, clipped on every rank's buffer alike."""
    P, sizes = 4, [1000, 24, 500]
    flat = [torch.randn(1524, device="cuda", generator=gen(20 + r)) for r in range(P)]
    total = sum(f.to(D) for f in flat)
    hc.allreduce(flat)
    outs = []
    for f in flat:
        views = list(f.split(sizes))
        hc.clip_grads(views, 0.5, scale=1.0 / P)
        outs.append(f)
    mean = total / P
    n = float(mean.norm())
    want = mean * min(1.0, 0.5 / (n + 1e-6))
    mag = sum(torch.randn(1524, device="cuda", generator=gen(20 + r)).abs().to(D) for r in range(P))
    assert bool(((outs[0].to(D) - want).abs() <= (NORM_OPS + 8) * 2.0 ** -24 * mag + half_ulp(want, F32)).all())
    for f in outs[1:]:
        assert torch.equal(f, outs[0])


def test_segments_of_a_reduce_scatter():
    """The norm over the ranks' segments is that of the whole vector."""
    P, n = 4, 4096
    send = [torch.randn(n, device="cuda", generator=gen(40 + r)) for r in range(P)]
    whole = sum(s.to(D) for s in send)
    segs = hc.segments("ring", "reducescatter", P, n, "float32")
    recv = [torch.empty(ln, device="cuda") for _, ln in segs]
    hc.reduce_scatter(send, recv)
    assert float(hc.grad_norm(recv)["norm"]) == pytest.approx(float(whole.norm()), rel=1e-6)


def test_streams_and_graphs():
    grads = [torch.randn(20000, device="cuda", generator=gen(2)), torch.randn(33, device="cuda").to(BF16)]
    outs = [[torch.empty_like(v) for v in grads] for _ in range(3)]
    first = hc.bind_clip_grads(grads, 1.0, out=outs[0])
    first()
    want = [v.clone() for v in outs[0]]
    torch.cuda.synchronize()
    graphs = []
    for k in (1, 2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        c = hc.bind_clip_grads(grads, 1.0, out=outs[k], stream=s)
        c()
        s.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            c()
        graphs.append((gr, c))
        for v in outs[k]:
            v.zero_()
    for gr, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for k in (1, 2):
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want))
    grads[0].mul_(3.0)
    first()
    for gr, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for k in (1, 2):
        assert all(torch.equal(a, b) for a, b in zip(outs[k], outs[0]))
