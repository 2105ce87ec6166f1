"""How exact the sums of the expert layer's bf16 products are.

Small integers: every partial sum is a whole number below 2^24, which binary32
holds whatever is cut off and in whatever order, so results are the definition's
to the last bit.  A row that is lost, taken twice or taken from a neighbour shows.

Terms of one sign: published measurements of tensor cores (Fasi, Higham,
Mikaitis and Pranesh, 2021, and later ones) have them bring the 16 products of a
step and the sum so far to the largest one's exponent and cut off what lies two
bits below binary32's last place, and cut the new sum off to binary32.  While n
terms come in, the sum is half of its end on average: the terms lose at most
n 2^-25 / 2 of the end, the sums n / 16 2^-23 / 2 (CUT for each term).  Sums taken
out every s terms and added up, rounded (at most 2^-24 of the sum so far, each),
end short by at most s CUT + n / s 2^-25.
"""
import pytest

torch = pytest.importorskip("torch")

import collective_communication_algorithms_gb300 as hc  # noqa: E402
from training_util import D, half_ulp  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
CUT = 2.0 ** -26 + 2.0 ** -28


def short(n, segment):
    return segment * CUT + n / segment * 2.0 ** -25


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


def whole(g, *shape):
    """Whole numbers from -3 to 3: 16384 products of two make less than 2^18."""
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(BF16)


def upper(g, *shape):
    """bf16 values in [0.5, 1)."""
    return (0.5 + torch.randint(0, 128, shape, generator=g, device="cuda") / 256.0).to(BF16)


def cut_at(counts):
    cuts = [0]
    for n in counts:
        cuts.append(cuts[-1] + n)
    return cuts, torch.tensor(cuts, dtype=torch.int32, device="cuda")


def weight_gradient(go, x, cuts):
    return torch.stack([go[a:b].to(D).t() @ x[a:b].to(D) for a, b in zip(cuts, cuts[1:])])


# groups around the steps of an instruction, a stage and a segment
COUNTS = [1, 15, 16, 17, 63, 64, 65, 127, 511, 512, 513, 0, 575, 576, 1023, 1024, 1025, 2047, 4097, 8191, 8192, 8193]


@pytest.mark.parametrize("inner,outer", [(40, 24), (129, 136), (264, 520)])
@pytest.mark.parametrize("grad_dtype,accumulate", [(F32, False), (F32, True), (BF16, False), (BF16, True)])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_weight_gradients_of_whole_numbers(inner, outer, grad_dtype, accumulate, layout):
    g = gen(inner)
    cuts, offsets = cut_at(COUNTS)
    x, go = whole(g, cuts[-1], inner), whole(g, cuts[-1], outer)
    shape = (len(COUNTS), outer, inner) if layout == "out_in" else (len(COUNTS), inner, outer)
    gw = whole(g, *shape).to(grad_dtype)
    gw = gw if layout == "out_in" else gw.transpose(1, 2)
    want = weight_gradient(go, x, cuts) + (gw.to(D) if accumulate else 0.0)
    hc.expert_matmul_grad(go, offsets, x=x, grad_weight=gw, accumulate=accumulate)
    assert torch.equal(gw, want.to(F32).to(grad_dtype))  # exact in binary32, rounded once


@pytest.mark.parametrize("inner", [1, 15, 16, 17, 63, 64, 65, 511, 512, 513, 1000, 1025, 2048, 4099])
@pytest.mark.parametrize("outer", [40, 131])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_products_of_whole_numbers(inner, outer, out_dtype, layout):
    g = gen(inner)
    cuts, offsets = cut_at([130, 0, 31, 257, 1, 600])
    x, w = whole(g, cuts[-1], inner), whole(g, 6, outer, inner)
    if layout == "in_out":
        w = w.transpose(1, 2).contiguous().transpose(1, 2)
    out = hc.expert_matmul(x, w, offsets, out_dtype=out_dtype)["out"]
    want = torch.cat([x[a:b].to(D) @ w[e].to(D).t() for e, (a, b) in enumerate(zip(cuts, cuts[1:]))])
    assert torch.equal(out, want.to(F32).to(out_dtype))


@pytest.mark.parametrize("rows", [8192, 32768])
@pytest.mark.parametrize("inner,outer", [(40, 24), (1032, 2056)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_long_weight_gradients_in_binary32(rows, inner, outer, accumulate):
    """Segments of 512 rows, any number of them."""
    g = gen(rows)
    cuts, offsets = cut_at([rows + 5, 0, 77])
    x, go = upper(g, cuts[-1], inner), upper(g, cuts[-1], outer)
    gw = torch.zeros(3, outer, inner, device="cuda")
    hc.expert_matmul_grad(go, offsets, x=x, grad_weight=gw, accumulate=accumulate)
    want = weight_gradient(go, x, cuts)
    off = (gw.to(D) - want).abs() / want.clamp(min=1e-9)
    assert float(off.max()) <= short(rows + 5, 512), float(off.max())


@pytest.mark.parametrize("inner", [8192, 65536])
@pytest.mark.parametrize("rows,outer", [(100, 24), (3000, 2000)])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_long_products_in_binary32(inner, rows, outer, layout):
    """The same segments along the inputs."""
    g = gen(inner)
    cuts, offsets = cut_at([rows // 3, 0, rows - rows // 3])
    x = upper(g, rows, inner)
    w = upper(g, 3, outer, inner)
    if layout == "in_out":
        w = w.transpose(1, 2).contiguous().transpose(1, 2)
    out = hc.expert_matmul(x, w, offsets, out_dtype=F32)["out"]
    for e in (0, 2):
        want = torch.cat([x[cuts[e]:cuts[e + 1]].to(D) @ part.to(D).t() for part in w[e].split(256)], dim=1)
        off = (out[cuts[e]:cuts[e + 1]].to(D) - want).abs() / want
        assert float(off.max()) <= short(inner, 512), float(off.max())


@pytest.mark.parametrize("inner,outer", [(24, 40), (33, 17), (264, 520)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradients_in_bf16_of_a_million_rows(inner, outer, accumulate):
    """Segments of 8192 rows, and the rounding to bf16, which is 12 times as much."""
    g = gen(inner)
    cuts, offsets = cut_at([(1 << 20) + 77, 1000])
    x, go = upper(g, cuts[-1], inner), upper(g, cuts[-1], outer)
    gw = upper(g, 2, outer, inner)
    want = weight_gradient(go, x, cuts) + (gw.to(D) if accumulate else 0.0)
    hc.expert_matmul_grad(go, offsets, x=x, grad_weight=gw, accumulate=accumulate)
    off = ((gw.to(D) - want).abs() - half_ulp(want, BF16)) / want
    assert float(off.max()) <= short((1 << 20) + 77, 8192), float(off.max())


@pytest.mark.parametrize("inner", [16384, 16385, 65536])
@pytest.mark.parametrize("rows,outer", [(100, 24), (3000, 2003)])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_long_products_in_bf16(inner, rows, outer, layout):
    """Sums of more than 16384 terms are taken out too."""
    g = gen(inner)
    cuts, offsets = cut_at([rows // 3, 0, rows - rows // 3])
    x = upper(g, rows, inner)
    w = upper(g, 3, outer, inner)
    if layout == "in_out":
        w = w.transpose(1, 2).contiguous().transpose(1, 2)
    out = hc.expert_matmul(x, w, offsets)["out"]
    for e in (0, 2):
        want = torch.cat([x[cuts[e]:cuts[e + 1]].to(D) @ part.to(D).t() for part in w[e].split(256)], dim=1)
        off = ((out[cuts[e]:cuts[e + 1]].to(D) - want).abs() - half_ulp(want, BF16)) / want
        assert float(off.max()) <= short(inner, 16384 if inner <= 16384 else 8192), float(off.max())


@pytest.mark.parametrize("inner,outer", [(40, 24), (129, 136), (264, 520)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_weight_gradients_of_whole_numbers_over_many_rows(inner, outer, accumulate, layout):
    """Groups around a bf16 segment, and a strided, unaligned gradient whose
    surroundings stay as they are."""
    g = gen(outer)
    counts = [8191, 0, 8192, 8193, 16385, 1, 63, 64]
    cuts, offsets = cut_at(counts)
    x, go = whole(g, cuts[-1], inner), whole(g, cuts[-1], outer)
    a, b = (outer, inner) if layout == "out_in" else (inner, outer)
    store = torch.full((len(counts) * (a * (b + 3) + 5) + 7,), -7.0, dtype=BF16, device="cuda")
    gw = store[1:].as_strided((len(counts), a, b), (a * (b + 3) + 5, b + 3, 1))
    gw.copy_(whole(g, len(counts), a, b))
    gw = gw if layout == "out_in" else gw.transpose(1, 2)
    want = weight_gradient(go, x, cuts) + (gw.to(D) if accumulate else 0.0)
    hc.expert_matmul_grad(go, offsets, x=x, grad_weight=gw, accumulate=accumulate)
    assert torch.equal(gw, want.to(F32).to(BF16))
    gw.fill_(-7.0)
    assert bool((store == -7.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_whole_numbers_behind_two_gib(dtype):
    """Every output of rows whose offsets in elements pass 2^31, to the bit."""
    inner, rows = 32768, 70001
    if torch.cuda.mem_get_info()[0] < 12 * rows * inner * 2:
        pytest.skip("needs %d GB" % (12 * rows * inner * 2 >> 30))
    g = gen(12)
    cuts, offsets = cut_at([rows - 35, 0, 33])  # the last two rows are in no group
    x = torch.zeros(rows, inner, dtype=dtype, device="cuda")
    x[-200:] = whole(g, 200, inner).to(dtype)
    x[:100] = whole(g, 100, inner).to(dtype)
    w, go = whole(g, 3, 24, inner).to(dtype), whole(g, rows, 24).to(dtype)
    out = hc.expert_matmul(x, w, offsets)["out"]
    gw = torch.empty(3, 24, inner, device="cuda")
    o = hc.expert_matmul_grad(go, offsets, x=x, weight=w, grad_weight=gw)
    for e in range(3):
        a, b = cuts[e], cuts[e + 1]
        for c in range(a, b, 8192):
            d = min(b, c + 8192)
            assert torch.equal(out[c:d], (x[c:d].to(D) @ w[e].to(D).t()).to(F32).to(dtype))
            assert torch.equal(o["grad_x"][c:d], (go[c:d].to(D) @ w[e].to(D)).to(F32).to(dtype))
        near = torch.tensor([r for r in range(a, b) if r < 100 or r >= rows - 200], dtype=torch.long, device="cuda")  # others are 0
        assert torch.equal(gw[e], (go[near].to(D).t() @ x[near].to(D)).to(F32))
    assert bool((out[-2:] == 0).all()) and bool((o["grad_x"][-2:] == 0).all())
