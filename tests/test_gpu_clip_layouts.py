"""Gradient clipping of gradients that are dense but not in their own order
(transposed views, as expert_matmul_grad returns them for transposed weights)."""
import math

import pytest

torch = pytest.importorskip("torch")

import collective_communication_algorithms_gb300 as hc  # noqa: E402
from training_util import D, assert_close  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
OPS = 40  # roundings: half of 64 in the norm, and those of the factor and the product


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from collective_communication_algorithms_gb300 import build
    build.build()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def check(got, before, o, max_norm):
    norm = math.sqrt(sum(float((v.to(D) ** 2).sum()) for v in before))
    assert abs(float(o["norm"]) - norm) <= OPS * 2.0 ** -24 * norm
    factor = min(1.0, max_norm / (norm + 1e-6))
    for v, b in zip(got, before):
        assert_close(v, b.to(D) * factor, b.to(D).abs() * factor, OPS)


def dense(dtype):
    g = gen(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)
    return [normal(5, 33, 18).transpose(1, 2), normal(40, 7).t(), normal(3, 4, 5, 6).permute(2, 0, 3, 1), normal(31),
            normal(1, 9, 1).transpose(0, 1), normal(4, 8, 3, 3).to(memory_format=torch.channels_last),
            torch.empty(8, 0, 3, device="cuda", dtype=dtype).transpose(0, 2), normal(16, 1).expand(16, 1)[:, 0]]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dense_gradients_in_place(dtype):
    grads = dense(dtype)
    before = [v.clone() for v in grads]
    o = hc.clip_grads(grads, 0.5)
    assert all(a is b for a, b in zip(o["grads"], grads))
    check(grads, before, o, 0.5)
    assert torch.equal(hc.grad_norm(before)["norm"], o["norm"])


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, F32), (F32, BF16)])
def test_dense_gradients_into_others_of_the_same_layout(dtype, out_dtype):
    grads = dense(dtype)
    before = [v.clone() for v in grads]
    outs = [torch.empty_like(v, dtype=out_dtype) for v in grads]
    assert all(a.stride() == b.stride() for a, b in zip(outs, grads) if a.numel())
    o = hc.clip_grads(grads, 0.5, out=outs)
    check(outs, before, o, 0.5)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


def test_gradients_of_transposed_weights():
    """What expert_matmul_grad returns goes into clip_grads as it is."""
    g = gen(7)
    x, go = torch.randn(50, 24, generator=g, device="cuda"), torch.randn(50, 40, generator=g, device="cuda")
    w = torch.randn(3, 24, 40, generator=g, device="cuda").transpose(1, 2)
    offsets = torch.tensor([0, 20, 20, 50], dtype=torch.int32, device="cuda")
    gw = hc.expert_matmul_grad(go, offsets, x=x, weight=w)["grad_weight"]
    assert not gw.is_contiguous()
    before = gw.clone()
    o = hc.clip_grads([gw, x], 1.0)
    norm = float(o["norm"])
    assert_close(gw, before.to(D) / (norm + 1e-6), before.to(D).abs() / norm, OPS)


def test_gradients_that_are_not_dense_or_not_laid_out_alike():
    a = torch.ones(6, 10, device="cuda")
    for bad in (a[:, ::2], a[:, :9], a[::2], torch.ones(4, 1, device="cuda").expand(4, 3),
                torch.ones(9, device="cuda").as_strided((3, 3), (2, 1))):
        with pytest.raises(ValueError, match="dense"):
            hc.clip_grads([bad], 1.0)
        with pytest.raises(ValueError, match="dense"):
            hc.clip_grads([torch.ones(bad.shape, device="cuda")], 1.0, out=[bad])
    with pytest.raises(ValueError, match="laid out"):
        hc.clip_grads([a], 1.0, out=[torch.empty(10, 6, device="cuda").t()])
    with pytest.raises(ValueError, match="shape"):
        hc.clip_grads([a], 1.0, out=[torch.empty(10, 6, device="cuda")])
    assert bool((a == 1).all())
