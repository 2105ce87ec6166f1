"""Layouts of experts' weights: which of the two a tensor has, what a weight and
its gradient have in common where a dimension of one leaves the choice, and
(on a GPU) that the gradients of such weights are right."""
import itertools

import pytest

torch = pytest.importorskip("torch")

from collective_communication_algorithms_gb300 import experts as X  # noqa: E402

E, I = 3, 10


def stored(rows, cols, pad, dtype=torch.float32, device="cpu"):
    """experts x rows x cols whose rows lie cols + pad apart."""
    return torch.zeros(E, rows, cols + pad, dtype=dtype, device=device)[:, :, :cols]


def with_one(which, layout, pad, dtype=torch.float32, device="cpu"):
    """experts x out x in with one output or one input, stored in a layout."""
    out, inner = (1, I) if which == "output" else (I, 1)
    if layout == "out_in":
        return stored(out, inner, pad, dtype, device)
    return stored(inner, out, pad, dtype, device).transpose(1, 2)


@pytest.mark.parametrize("which", ["output", "input"])
@pytest.mark.parametrize("a,b", list(itertools.product([("out_in", 0), ("out_in", 3), ("in_out", 0)], repeat=2)))
def test_one_output_or_input_leaves_the_choice(which, a, b):
    w, g = with_one(which, *a), with_one(which, *b)
    layout = X._layout(weight=w, grad_weight=g)
    for t in (w, g):
        rows, cols, stride, unit = X._rows_of(t, layout)
        assert (cols == 1 or unit == 1) and (rows == 1 or stride >= cols)


@pytest.mark.parametrize("pad", [2, 5])
def test_padded_columns_of_one(pad):
    """One column of a wider store: rows lie apart in the stored layout alone."""
    w, g = with_one("output", "in_out", 0), with_one("output", "in_out", pad)
    assert X._layout(weight=w) == "out_in" and X._layout(weight=w, grad_weight=g) == "in_out"
    w, g = with_one("input", "out_in", 0), with_one("input", "out_in", pad)
    assert X._layout(weight=w, grad_weight=g) == "out_in"


def test_layouts_that_do_not_fit():
    w, t = stored(4, 5, 0), stored(5, 4, 1).transpose(1, 2)
    assert X._layout(weight=w) == "out_in" and X._layout(weight=t) == "in_out"
    with pytest.raises(ValueError, match="laid out as weight is"):
        X._layout(weight=w, grad_weight=t)
    for bad in (stored(4, 10, 0)[:, :, ::2], w.expand(E, 4, 5)[:, :1].expand(E, 4, 5), torch.zeros(4, 5, E).permute(2, 0, 1)):
        with pytest.raises(ValueError, match="unit stride"):
            X._layout(weight=bad)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["output", "input"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("a,b", list(itertools.product([("out_in", 0), ("out_in", 3), ("in_out", 0), ("in_out", 7)], repeat=2)))
def test_gradients_of_one_output_or_input(which, dtype, a, b):
    """Whole numbers, to the bit; a weight and a gradient that have no layout in
    common (padded in different directions) are refused."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import collective_communication_algorithms_gb300 as hc
    from collective_communication_algorithms_gb300 import build
    build.build()
    g = torch.Generator("cuda").manual_seed(1)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)
    out, inner = (1, I) if which == "output" else (I, 1)
    w, gw = with_one(which, *a, dtype, "cuda"), with_one(which, *b, torch.float32, "cuda")
    w.copy_(whole(E, out, inner))
    cuts = [0, 50, 50, 131]
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    x, go = whole(131, inner), whole(131, out)
    try:
        X._layout(weight=w, grad_weight=gw)
    except ValueError:
        with pytest.raises(ValueError, match="laid out"):
            hc.expert_matmul_grad(go, offsets, x=x, weight=w, grad_weight=gw)
        return
    o = hc.expert_matmul_grad(go, offsets, x=x, weight=w, grad_weight=gw)
    for e in range(E):
        r = slice(cuts[e], cuts[e + 1])
        assert torch.equal(gw[e].double(), go[r].double().t() @ x[r].double())
        assert torch.equal(o["grad_x"][r].double(), go[r].double() @ w[e].double())
