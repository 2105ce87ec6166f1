"""The expert layer's operators against their definitions in 64 bits: types,
odd sizes, strides and layouts, groups that are empty, huge or behind rows of
no group, infinities and NaN next to a group, streams and CUDA graphs,
gradients against differences.

Bounds: an output is rounded once to its type (half a unit in its last
place).  Products of bf16 values are exact in binary32; a sum of n terms,
in whatever order, adds at most n roundings, each of at most 2^-23 of the sum
of the terms' magnitudes where additions may cut off instead of rounding (2 n
times 2^-24), 2^-24 where they round; binary32 products add one rounding each.
"""
import pytest

torch = pytest.importorskip("torch")

import collective_communication_algorithms_gb300 as hc  # noqa: E402
from experts_util import groups, matmul, matmul_grad, plan  # noqa: E402
from training_util import D, assert_close, guarded, strided  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from collective_communication_algorithms_gb300 import build
    build.build()
    yield
    from collective_communication_algorithms_gb300 import _binding as B
    assert B.hc_device_status() == 0


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("tokens,top,experts", [(1, 1, 1), (1, 2, 8), (7, 3, 5), (64, 2, 8), (1000, 8, 256), (513, 1, 1024),
                                                (8192, 1, 3), (8193, 1, 3), (4099, 6, 40), (70001, 8, 1000), (65536, 8, 256)])
@pytest.mark.parametrize("kind", ["uniform", "one", "none", "part"])
def test_plan(tokens, top, experts, kind):
    g = gen(tokens + experts)
    first = 0
    if kind == "uniform":
        ids = torch.randint(-1, experts + 1, (tokens, top), generator=g, device="cuda")
    elif kind == "one":
        ids = torch.full((tokens, top), experts - 1, device="cuda")
    elif kind == "none":
        ids = torch.full((tokens, top), -1, device="cuda")
    else:
        first = 2 * experts
        ids = torch.randint(0, 5 * experts, (tokens, top), generator=g, device="cuda")
    ids = ids.to(torch.int32 if (tokens + top) % 2 else torch.int64)
    o = hc.expert_plan(ids, experts, first_expert=first)
    offsets, rows, slots = plan(ids.cpu(), experts, first)
    assert o["offsets"].tolist() == offsets
    assert o["tokens"].tolist() == rows
    assert o["slots"].reshape(-1).tolist() == slots


def test_plan_of_no_tokens_and_of_far_ids():
    o = hc.expert_plan(torch.empty(0, 4, dtype=torch.int64, device="cuda"), 5)
    assert o["offsets"].tolist() == [0] * 6
    far = torch.tensor([[2 ** 63 - 1, -2 ** 63], [2 ** 62, 3]], device="cuda")
    o = hc.expert_plan(far, 4, first_expert=2 ** 62)
    assert o["slots"].tolist() == [[-1, -1], [0, -1]] and o["tokens"].tolist() == [1, -1, -1, -1]
    o = hc.expert_plan(far, 4, first_expert=-2 ** 63)
    assert o["slots"].tolist() == [[-1, 0], [-1, -1]]


# ------------------------------------------------------------------ products
SIZES = [  # rows, experts, in, out
    (1, 1, 8, 8), (1, 3, 64, 40), (2, 8, 1024, 512), (5, 2, 1, 1), (16, 4, 72, 264), (33, 3, 17, 9), (130, 2, 128, 256),
    (257, 5, 200, 136), (300, 40, 64, 64), (1000, 7, 129, 383), (1025, 16, 512, 264), (4099, 3, 264, 520), (37, 1024, 24, 16),
    (600, 4, 1032, 2056),
    # tiles that two blocks share, in all three products
    (5006, 16, 193, 2003), (20011, 5, 1040, 776),
    # few rows of weights that no tiled copy takes
    (13, 5, 1003, 37), (16, 40, 515, 129), (3, 2, 8193, 9),
    # sums of few tiles that several blocks share
    (40, 3, 3843, 70), (30, 2, 96, 2500), (3000, 1, 65, 40),
]
KINDS = ["even", "skewed", "last", "none"]


def layout_of(w, layout):
    """The same weights, stored experts x in x out."""
    return w.transpose(1, 2).contiguous().transpose(1, 2) if layout == "in_out" else w


@pytest.mark.parametrize("rows,experts,inner,outer", SIZES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_matmul(rows, experts, inner, outer, kind, dtype, out_dtype, layout):
    g = gen(rows + inner)
    offsets, cuts = groups(kind, experts, rows)
    x = normal(g, rows, inner, dtype=dtype)
    w = normal(g, experts, outer, inner, dtype=dtype, std=inner ** -0.5)
    outside = torch.ones(rows, dtype=torch.bool, device="cuda")
    outside[cuts[0]:cuts[-1]] = False
    x[outside] = float("nan")
    out, intact = guarded(rows, outer, out_dtype)
    hc.expert_matmul(x, layout_of(w, layout), offsets, out=out)
    ref, mag = matmul(x, w, cuts)
    assert_close(out[~outside], ref[~outside], mag[~outside], 2 * inner + 2, "out")
    assert bool((out[outside] == -7.25).all()) and intact()


@pytest.mark.parametrize("rows,experts,inner,outer", SIZES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,grad_dtype,accumulate", [(BF16, BF16, False), (BF16, F32, True), (BF16, BF16, True),
                                                         (BF16, F32, False), (F32, F32, False), (F32, F32, True),
                                                         (F32, BF16, True)])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_matmul_grad(rows, experts, inner, outer, kind, dtype, grad_dtype, accumulate, layout):
    g = gen(rows + outer)
    offsets, cuts = groups(kind, experts, rows, seed=1)
    x = normal(g, rows, inner, dtype=dtype)
    w = normal(g, experts, outer, inner, dtype=dtype, std=inner ** -0.5)
    go = normal(g, rows, outer, dtype=dtype)
    outside = torch.ones(rows, dtype=torch.bool, device="cuda")
    outside[cuts[0]:cuts[-1]] = False
    x[outside] = float("inf")
    go[outside] = float("nan")
    gx, intact = guarded(rows, inner, dtype)
    wide = (experts * outer, inner) if layout == "out_in" else (experts * inner, outer)
    flat, intact_w = guarded(*wide, grad_dtype)
    gw = flat.view(experts, outer, inner) if layout == "out_in" else flat.view(experts, inner, outer).transpose(1, 2)
    old = normal(g, experts, outer, inner, dtype=grad_dtype)
    if accumulate:
        gw.copy_(old)
    hc.expert_matmul_grad(go, offsets, x=x, weight=layout_of(w, layout), grad_x=gx, grad_weight=gw, accumulate=accumulate)
    rx, mx, rw, mw, n = matmul_grad(go, x, w, cuts, old if accumulate else None)
    assert_close(gx[~outside], rx[~outside], mx[~outside], 2 * outer + 2, "grad_x")
    assert bool((gx[outside] == -7.25).all()) and intact()
    assert_close(gw, rw, mw, 2 * n + 3, "grad_weight")
    assert intact_w()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_matmul_grad_parts(dtype):
    """Either gradient alone gives the same bits as both."""
    g = gen(5)
    offsets, _ = groups("skewed", 6, 500)
    x, go = normal(g, 500, 72, dtype=dtype), normal(g, 500, 200, dtype=dtype)
    w = normal(g, 6, 200, 72, dtype=dtype)
    both = hc.expert_matmul_grad(go, offsets, x=x, weight=w)
    assert torch.equal(hc.expert_matmul_grad(go, offsets, weight=w)["grad_x"], both["grad_x"])
    assert torch.equal(hc.expert_matmul_grad(go, offsets, x=x)["grad_weight"], both["grad_weight"])
    assert both["grad_weight"].dtype == dtype
    again = hc.expert_matmul_grad(go, offsets, x=x, weight=w)
    assert torch.equal(again["grad_weight"], both["grad_weight"]) and torch.equal(again["grad_x"], both["grad_x"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("stride,offset", [(80, 0), (81, 0), (88, 3), (73, 8), (72, 1)])
def test_matmul_strided(dtype, stride, offset):
    g = gen(stride + offset)
    rows, experts, inner, outer = 190, 3, 72, 56
    offsets, cuts = groups("even", experts, rows)
    x = strided(normal(g, rows, inner, dtype=dtype), stride, offset)
    go = strided(normal(g, rows, outer, dtype=dtype), stride, offset)
    # experts apart from each other by more than their rows
    step = outer * stride + 24
    store = torch.zeros(offset + experts * step + stride, dtype=dtype, device="cuda")
    w = store[offset:].as_strided((experts, outer, inner), (step, stride, 1))
    w.copy_(normal(g, experts, outer, inner, dtype=dtype))
    out, intact = guarded(rows, outer, dtype, stride + 1, offset)
    hc.expert_matmul(x, w, offsets, out=out)
    ref, mag = matmul(x, w, cuts)
    assert_close(out, ref, mag, 2 * inner + 2, "out")
    assert intact()
    gx, intact = guarded(rows, inner, dtype, stride + 1, offset)
    gstore = torch.full((offset + experts * step + stride,), -7.25, dtype=F32, device="cuda")
    gw = gstore[offset:].as_strided((experts, outer, inner), (step, stride, 1))
    hc.expert_matmul_grad(go, offsets, x=x, weight=w, grad_x=gx, grad_weight=gw)
    rx, mx, rw, mw, n = matmul_grad(go, x, w, cuts)
    assert_close(gx, rx, mx, 2 * outer + 2, "grad_x")
    assert_close(gw, rw, mw, 2 * n + 3, "grad_weight")
    assert intact()
    gw.fill_(-7.25)
    assert bool((gstore == -7.25).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inner,outer", [(72, 136), (65, 131), (200, 24)])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_infinities_and_nan_stay_with_their_expert(dtype, inner, outer, layout):
    g = gen(inner)
    cuts = [0, 37, 37, 90, 101]
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    x, go = normal(g, 101, inner, dtype=dtype), normal(g, 101, outer, dtype=dtype)
    w = normal(g, 4, outer, inner, dtype=dtype)
    x[40, 3] = float("nan")
    go[41, 5] = float("inf")
    w[1] = float("nan")  # the expert without rows
    w[3, 0, 0] = float("inf")
    out = hc.expert_matmul(x, layout_of(w, layout), offsets)["out"]
    bad = ~torch.isfinite(out)
    assert bool(bad[40].all()) and bool(bad[90:, 0].all())
    bad[40] = False
    bad[90:, 0] = False
    assert not bool(bad.any())
    o = hc.expert_matmul_grad(go, offsets, x=x, weight=layout_of(w, layout))
    bad = ~torch.isfinite(o["grad_x"])
    assert bool(bad[41].all()) and bool(bad[90:, 0].all())
    bad[41] = False
    bad[90:, 0] = False
    assert not bool(bad.any())
    bad = ~torch.isfinite(o["grad_weight"])
    assert bool(bad[2, :, 3].all()) and bool(bad[2, 5, :].all())
    bad[2, :, 3] = False
    bad[2, 5, :] = False
    assert not bool(bad.any())
    assert bool((o["grad_weight"][1] == 0).all())


def test_offsets_out_of_range_are_clamped():
    g = gen(9)
    x, w = normal(g, 50, 16, dtype=BF16), normal(g, 4, 24, 16, dtype=BF16)
    given = torch.tensor([-5, 20, 10, 1 << 30, 30], dtype=torch.int32, device="cuda")
    cuts = [0, 20, 20, 50, 50]
    out = hc.expert_matmul(x, w, given)["out"]
    ref, mag = matmul(x, w, cuts)
    assert_close(out, ref, mag, 2 * 16 + 2, "out")
    go = normal(g, 50, 24, dtype=BF16)
    o = hc.expert_matmul_grad(go, given, x=x, weight=w)
    rx, mx, rw, mw, n = matmul_grad(go, x, w, cuts)
    assert_close(o["grad_x"], rx, mx, 2 * 24 + 2, "grad_x")
    assert_close(o["grad_weight"], rw, mw, 2 * n + 3, "grad_weight")


def test_matmul_of_no_rows():
    x, w = torch.empty(0, 16, dtype=BF16, device="cuda"), torch.ones(3, 24, 16, dtype=BF16, device="cuda")
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert hc.expert_matmul(x, w, offsets)["out"].shape == (0, 24)
    go = torch.empty(0, 24, dtype=BF16, device="cuda")
    gw = torch.full((3, 24, 16), 5.0, device="cuda")
    hc.expert_matmul_grad(go, offsets, x=x, grad_weight=gw, accumulate=True)
    assert bool((gw == 5).all())
    hc.expert_matmul_grad(go, offsets, x=x, weight=w, grad_weight=gw)
    assert bool((gw == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_behind_two_gib(dtype):
    """Row offsets in elements pass 2^31."""
    inner, rows = 32768, 70000
    free = torch.cuda.mem_get_info()[0]
    if free < 12 * rows * inner * 2:
        pytest.skip("needs %d GB" % (12 * rows * inner * 2 >> 30))
    offsets = torch.tensor([0, rows - 3, rows], dtype=torch.int32, device="cuda")
    x = torch.empty(rows, inner, dtype=dtype, device="cuda")
    g = gen(2)
    x[-8:] = normal(g, 8, inner, dtype=dtype)
    x[:-8] = 0
    w = normal(g, 2, 8, inner, dtype=dtype)
    out = hc.expert_matmul(x, w, offsets)["out"]
    ref, mag = matmul(x[-8:], w, [0, 5, 8])
    assert_close(out[-8:], ref, mag, 2 * inner + 2, "out")
    go = normal(g, rows, 8, dtype=dtype)
    o = hc.expert_matmul_grad(go, offsets, x=x, weight=w)
    rx, mx, rw, mw, n = matmul_grad(go[-8:], x[-8:], w, [0, 5, 8])
    assert_close(o["grad_x"][-8:], rx, mx, 18, "grad_x")
    assert_close(o["grad_weight"], rw, mw, 2 * 70000 + 3, "grad_weight")


def test_gradients_against_differences():
    """Along a random direction of each input, binary32 and its 64-bit
    definition's central differences."""
    g = gen(77)
    rows, experts, inner, outer = 60, 4, 24, 20
    offsets, cuts = groups("skewed", experts, rows)
    x, w = normal(g, rows, inner), normal(g, experts, outer, inner)
    go = normal(g, rows, outer)
    o = hc.expert_matmul_grad(go, offsets, x=x, weight=w)
    inside = slice(cuts[0], cuts[-1])

    def value(x, w):
        return float((matmul(x, w, cuts)[0][inside] * go[inside].to(D)).sum())
    for name, at in (("x", x), ("weight", w)):
        d = normal(g, *at.shape).to(D)
        h = 1e-3
        args = [x.to(D), w.to(D)]
        k = 0 if name == "x" else 1
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + h * d, args[k] - h * d
        slope = (value(*up) - value(*down)) / (2 * h)  # the value is linear in each input
        got = float((o["grad_" + name].to(D) * d)[inside if name == "x" else slice(None)].sum())
        size = float((o["grad_" + name].to(D).abs() * d.abs())[inside if name == "x" else slice(None)].sum())
        assert abs(got - slope) <= (outer + rows) * 2.0 ** -23 * size + 1e-9 * abs(slope)


@pytest.mark.parametrize("rows,experts,inner,outer", [(5006, 16, 1001, 2003), (5006, 16, 1000, 2000), (2003, 64, 520, 1040),
                                                      (20000, 88, 440, 944)])
def test_many_calls_one_after_the_other(rows, experts, inner, outer):
    """Blocks follow one another on an SM thousands of times, without a wait
    that gives up and with the same bits."""
    from collective_communication_algorithms_gb300 import _binding as B
    g = gen(outer)
    offsets, _ = groups("even", experts, rows)
    x, w = normal(g, rows, inner, dtype=BF16), normal(g, experts, outer, inner, dtype=BF16)
    go = normal(g, rows, outer, dtype=BF16)
    a = hc.bind_expert_matmul(x, w, offsets)
    b = hc.bind_expert_matmul_grad(go, offsets, x=x, weight=w)
    a()
    b()
    first = [v.clone() for c in (a, b) for v in c.outputs.values()]
    for _ in range(20):
        for _ in range(150):
            a()
        for _ in range(50):
            b()
        torch.cuda.synchronize()
        assert B.hc_device_status() == 0
    assert all(torch.equal(u, v) for u, v in zip(first, [v for c in (a, b) for v in c.outputs.values()]))


@pytest.mark.parametrize("rows,experts,inner,outer", [(100, 3, 72, 136), (5006, 16, 264, 2000), (2003, 64, 520, 1040)])
def test_expired_wait_reports_timeout_then_recovers(rows, experts, inner, outer):
    """hc_test_expire_waits: the first wait on the copies gives up after 1 ms,
    although they land; the call ends, writes nowhere else, reports, and the
    next one is right."""
    import time
    from collective_communication_algorithms_gb300 import _binding as B
    g = gen(rows)
    offsets, cuts = groups("even", experts, rows)
    x, w = normal(g, rows, inner, dtype=BF16), normal(g, experts, outer, inner, dtype=BF16)
    go = normal(g, rows, outer, dtype=BF16)
    out, intact = guarded(rows, outer, BF16)
    gx, intact_x = guarded(rows, inner, BF16)
    flat, intact_w = guarded(experts * outer, inner, F32)
    a = hc.bind_expert_matmul(x, w, offsets, out=out)
    b = hc.bind_expert_matmul_grad(go, offsets, x=x, weight=w, grad_x=gx, grad_weight=flat.view(experts, outer, inner))
    for call in (a, b):
        call()
        torch.cuda.synchronize()
        want = [v.clone() for v in call.outputs.values()]
        assert B.hc_device_status() == 0
        B.hc_test_expire_waits(True)
        try:
            t0 = time.perf_counter()
            call()
            torch.cuda.synchronize()
            elapsed = time.perf_counter() - t0
        finally:
            B.hc_test_expire_waits(False)
        assert elapsed < 1.0, elapsed
        assert B.hc_device_status(clear=True) == 6
        assert B.hc_device_status() == 0
        assert intact() and intact_x() and intact_w()
        call()
        torch.cuda.synchronize()
        assert B.hc_device_status() == 0
        assert all(torch.equal(u, v) for u, v in zip(want, call.outputs.values()))


# ------------------------------------------------------------------ combine
def combine(y, slots, w):
    here = (slots >= 0) & (slots < y.shape[0])
    rows = torch.where(here[:, :, None], y.to(D)[slots.long().clamp(0, y.shape[0] - 1)], 0.0)
    ww = torch.ones(slots.shape, dtype=D, device="cuda") if w is None else w.to(D)
    ww = torch.where(here, ww, 0.0)
    terms = rows * ww[:, :, None]
    return terms.sum(dim=1), terms.abs().sum(dim=1), rows, here


def some_slots(g, tokens, top, rows):
    n = max(rows, tokens * top)
    slots = torch.randperm(n, generator=g, device="cuda")[:tokens * top].to(torch.int32).view(tokens, top)
    return torch.where(slots < rows, slots, torch.where(slots % 2 == 0, -1, slots))  # beyond the rows, or -1


@pytest.mark.parametrize("tokens,top,rows,dim", [(1, 1, 1, 1), (1, 8, 9, 4096), (3, 2, 6, 8), (33, 2, 60, 1001), (700, 4, 2800, 264),
                                                 (64, 9, 500, 40), (5000, 8, 40000, 72), (17, 17, 300, 520), (9000, 1, 9000, 33)])
@pytest.mark.parametrize("dtype,weight", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16), (BF16, None), (F32, None)])
def test_combine(tokens, top, rows, dim, dtype, weight):
    g = gen(tokens + dim)
    y = normal(g, rows, dim, dtype=dtype)
    slots = some_slots(g, tokens, top, rows)
    w = normal(g, tokens, top, dtype=weight) if weight is not None else None
    out, intact = guarded(tokens, dim, dtype)
    hc.expert_combine(y, slots, weights=w, out=out)
    ref, mag, y_rows, here = combine(y, slots, w)
    assert_close(out, ref, mag, top, "out")
    assert intact()
    go = normal(g, tokens, dim, dtype=dtype)
    gy, intact = guarded(rows, dim, dtype)
    o = hc.expert_combine_grad(go, slots, y=y, weights=w, grad_y=gy)
    want = torch.full((rows, dim), -7.25, dtype=D, device="cuda")
    ww = torch.ones(slots.shape, dtype=D, device="cuda") if w is None else w.to(D)
    want[slots[here].long()] = (ww[:, :, None] * go.to(D)[:, None, :])[here]
    assert_close(gy, want, want.abs(), 1, "grad_y")
    assert intact()
    if w is not None:
        terms = y_rows * go.to(D)[:, None, :]
        assert_close(o["grad_weights"], terms.sum(dim=2), terms.abs().sum(dim=2), dim + 1, "grad_weights")
        alone = hc.expert_combine_grad(go, slots, y=y, weights=w, want_grad_y=False)
        assert list(alone) == ["grad_weights"] and torch.equal(alone["grad_weights"], o["grad_weights"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("stride,offset", [(80, 0), (81, 0), (88, 3), (73, 8)])
def test_combine_strided_and_in_place(dtype, stride, offset):
    g = gen(stride)
    y = strided(normal(g, 40, 72, dtype=dtype), stride, offset)
    slots = some_slots(g, 19, 2, 40)
    w = normal(g, 19, 2)
    out, intact = guarded(19, 72, dtype, stride + 2, offset)
    hc.expert_combine(y, slots, weights=w, out=out)
    ref, mag, y_rows, here = combine(y, slots, w)
    assert_close(out, ref, mag, 2, "out")
    assert intact()
    go = strided(normal(g, 19, 72, dtype=dtype), stride, offset)
    apart = hc.expert_combine_grad(go, slots, y=y, weights=w, grad_y=y.clone())
    place = hc.expert_combine_grad(go, slots, y=y, weights=w, grad_y=y)
    assert torch.equal(place["grad_y"], apart["grad_y"])
    assert torch.equal(place["grad_weights"], apart["grad_weights"])


def test_rows_without_part_are_not_looked_at():
    y = torch.full((4, 16), float("nan"), device="cuda")
    y[2] = 3.0
    slots = torch.tensor([[2, -1], [-1, 4], [7, -2 ** 31]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 1.0], [1.0, 1.0]], device="cuda")
    out = hc.expert_combine(y, slots, weights=w)["out"]
    assert bool((out[0] == 1.5).all()) and bool((out[1:] == 0).all())
    o = hc.expert_combine_grad(torch.ones(3, 16, device="cuda"), slots, y=y, weights=w)
    assert o["grad_weights"].tolist() == [[48.0, 0.0], [0.0, 0.0], [0.0, 0.0]]
    assert bool((o["grad_y"][2] == 0.5).all()) and bool((o["grad_y"][[0, 1, 3]] == 0).all())


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_plan_gather_products_and_sum(dtype):
    """The layer as a whole: each token's sum over its experts."""
    g = gen(3)
    T, K, E, d, f = 333, 3, 6, 64, 88
    x = normal(g, T, d, dtype=dtype)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1).indices
    ids[5] = -1
    p = torch.rand(T, K, generator=g, device="cuda")
    up, down = normal(g, E, f, d, dtype=dtype, std=d ** -0.5), normal(g, E, d, f, dtype=dtype, std=f ** -0.5)
    pl = hc.expert_plan(ids, E)
    rows = hc.embedding(x, pl["tokens"])["out"]
    h = hc.expert_matmul(rows, up, pl["offsets"], out_dtype=F32)["out"]
    y = hc.expert_matmul(h.to(dtype), down, pl["offsets"], out_dtype=F32)["out"]
    out = hc.expert_combine(y, pl["slots"], weights=p)["out"]
    hh = torch.einsum("td,efd->tef", x.to(D), up.to(D))
    hr = hh.to(dtype).to(D)  # rounded once between the products
    yy = torch.einsum("tef,edf->ted", hr, down.to(D))
    take = ids.clamp(min=0)
    w = torch.where(ids >= 0, p.to(D), 0.0)
    ref = (yy.gather(1, take[:, :, None].expand(T, K, d)) * w[:, :, None]).sum(dim=1)
    size = torch.einsum("tef,edf->ted", hr.abs(), down.to(D).abs())
    size = (size.gather(1, take[:, :, None].expand(T, K, d)) * w[:, :, None]).sum(dim=1)
    # h lies at most one step of its type beside its own rounding
    steps = 2.0 ** (-7 if dtype == BF16 else -22)
    assert bool(((out.to(D) - ref).abs() <= size * (steps + 2.0 ** -20) + 1e-30).all())
    # the gradient of the gather: the same sum without weights
    gr = normal(g, T * K, d, dtype=dtype)
    back = hc.expert_combine(gr, pl["slots"])["out"]
    want = torch.zeros(T, d, dtype=D, device="cuda")
    mag = torch.zeros_like(want)
    n = int(pl["offsets"][-1])
    want.index_add_(0, pl["tokens"][:n].long(), gr[:n].to(D))
    mag.index_add_(0, pl["tokens"][:n].long(), gr[:n].to(D).abs())
    assert_close(back, want, mag, K, "gather gradient")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_streams_and_graphs(dtype):
    """Two captured graphs and an eager call on another stream give what a
    first call gave, after their inputs change in place."""
    g = gen(11)
    T, K, E, d, f = 200, 2, 5, 72, 136
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda")
    x, w = normal(g, T * K, d, dtype=dtype), normal(g, E, f, d, dtype=dtype)
    go, p = normal(g, T * K, f, dtype=dtype), torch.rand(T, K, generator=g, device="cuda")

    def calls(stream=None):
        a = hc.bind_expert_plan(ids, E, stream=stream)
        b = hc.bind_expert_matmul(x, w, a.outputs["offsets"], stream=stream)
        c = hc.bind_expert_matmul_grad(go, a.outputs["offsets"], x=x, weight=w, stream=stream)
        e = hc.bind_expert_combine(b.outputs["out"], a.outputs["slots"], weights=p, stream=stream)
        h = hc.bind_expert_combine_grad(e.outputs["out"], a.outputs["slots"], y=b.outputs["out"], weights=p, stream=stream)
        return [a, b, c, e, h]

    def values(cs):
        return [v.clone() for c in cs for v in c.outputs.values()]

    def run(cs):
        for c in cs:
            c()
    eager = calls()
    run(eager)
    first = values(eager)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = calls(side)
    graphs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        cs = calls(s)
        with torch.cuda.stream(s):
            run(cs)  # once before the capture
        s.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            run(cs)
        graphs.append((gr, cs))
    run(other)
    for gr, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for cs in (other, graphs[0][1], graphs[1][1]):
        assert all(torch.equal(a, b) for a, b in zip(values(cs), first))
    ids.copy_(torch.randint(0, E, (T, K), generator=g, device="cuda"))
    x.copy_(normal(g, T * K, d, dtype=dtype))
    run(eager)
    for gr, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    second = values(eager)
    assert not torch.equal(first[0], second[0])
    for _, cs in graphs:
        assert all(torch.equal(a, b) for a, b in zip(values(cs), second))
