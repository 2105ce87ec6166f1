"""examples/expert_layer_step.py: an expert layer between the collectives.  The
step's summed gradients against the whole batch's in 64 bits (with the
experts that the step chose), their clipping, and the ranks bit for bit alike."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from collective_communication_algorithms_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("expert_layer_step", os.path.join(ROOT, "examples", "expert_layer_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(m, ranks, tokens_of_all_ranks):
    """Loss and gradients of the whole batch by automatic differentiation in
    64 bits, and the magnitude of each parameter's gradient by rank."""
    D, rms = torch.float64, torch.nn.functional.rms_norm
    q = {k: v.detach().to(D).requires_grad_() for k, v in ranks[0].params.items()}
    total = 0.0
    for r in ranks:
        row = torch.where((r.ids == m.PADDING)[:, None], q["table"][r.ids].detach(), q["table"][r.ids])
        x = row * m.SCALE
        n = rms(x, (m.DIM,), q["norm"], 1e-6)
        p = torch.softmax((n @ q["router"]).gather(1, r.experts), dim=1)
        up, down = q["up"][r.experts], q["down"][r.experts]  # tokens x choices x ...
        h = torch.einsum("td,tkfd->tkf", n, up).clamp(min=0)
        c = (torch.einsum("tkf,tkdf->tkd", h, down) * p[:, :, None]).sum(dim=1)
        s = x + rms(c, (m.DIM,), q["post"], 1e-6)
        z = rms(s, (m.DIM,), q["pre"], 1e-6)
        log_q = torch.log_softmax(z @ q["out"] / 2.0, dim=1).gather(1, r.teacher_ids)
        log_p = torch.log_softmax(r.teacher_logits.to(D) / 2.0, dim=1)
        kl = (log_p.exp() * (log_p - log_q)).sum(dim=1)
        total = total + (kl * r.row_weight.to(D)).sum() * 4.0 / tokens_of_all_ranks
    total.backward()
    return float(total.detach()), {k: v.grad for k, v in q.items()}


@pytest.mark.parametrize("P", [1, 3])
def test_step_gradients(example, P):
    tokens = 150
    ranks = [example.Rank(r, tokens) for r in range(P)]
    loss = sum(float(r.gradients(P * tokens)) for r in ranks)
    want, ref = reference(example, ranks, P * tokens)
    assert abs(loss - want) <= 1e-4 * abs(want)
    example.hc.allreduce([r.grads_flat for r in ranks])
    # binary32 products of up to 500 terms one after the other, seven of them in
    # a chain: 7 * 500 * 2^-24 of the magnitudes, by norm
    for k in ref:
        err = (ranks[0].grads[k].double() - ref[k]).norm() / ref[k].norm()
        assert float(err) <= 7 * 500 * 2.0 ** -24, k
    # clipped: the same direction, the limit's length
    before = [v.clone() for v in ranks[0].grads.values()]
    whole = float(torch.cat([v.reshape(-1) for v in ref.values()]).norm())
    outs = [example.hc.clip_grads(list(r.grads.values()), 0.5 * whole) for r in ranks]
    assert float(outs[0]["norm"]) == pytest.approx(whole, rel=7 * 500 * 2.0 ** -24)
    factor = float(outs[0]["factor"])
    assert factor == pytest.approx(0.5, rel=1e-3)
    for v, b in zip(ranks[0].grads.values(), before):
        assert torch.equal(v, b * outs[0]["factor"])
    for r in ranks[1:]:
        assert torch.equal(r.grads_flat, ranks[0].grads_flat)


def test_steps_run_and_ranks_stay_alike(example):
    ranks = [example.Rank(r, 200) for r in range(4)]
    for _ in range(4):
        loss, norm = example.step(ranks, 800, max_norm=0.1, rate=0.5)
        assert bool(torch.isfinite(loss)) and bool(torch.isfinite(norm).all())
    for r in ranks[1:]:
        for k in r.params:
            assert torch.equal(r.params[k], ranks[0].params[k]), k
