"""examples/data_parallel_step.py: the training operators and the AllReduce
together.  The step's summed gradients against the whole batch's in 64 bits,
the ranks bit for bit alike after every step, and a loss that falls."""
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
    spec = importlib.util.spec_from_file_location("data_parallel_step",
                                                  os.path.join(ROOT, "examples", "data_parallel_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(example, ranks, tokens_of_all_ranks):
    """Gradients of the whole batch's loss by automatic differentiation of the
    model in 64 bits."""
    D = torch.float64
    q = {k: v.detach().to(D).requires_grad_() for k, v in ranks[0].params.items()}
    total = 0.0
    for r in ranks:
        table = q["table"].clone()
        # the padding id's row gets no gradient
        row = torch.where((r.ids == example.PADDING)[:, None], table[r.ids].detach(), table[r.ids])
        x = row * example.DIM ** 0.5
        y = x @ q["w1"]
        n = torch.nn.functional.rms_norm(y, (example.DIM,), q["post_weight"], 1e-6)
        s = x + q["gate"] * n
        z = torch.nn.functional.rms_norm(s, (example.DIM,), q["pre_weight"], 1e-6)
        log_q = torch.log_softmax(z @ q["w2"] / 2.0, dim=1).gather(1, r.teacher_ids)
        log_p = torch.log_softmax(r.teacher_logits.to(D) / 2.0, dim=1)
        kl = (log_p.exp() * (log_p - log_q)).sum(dim=1)
        total = total + (kl * r.row_weight.to(D)).sum() * 4.0 / tokens_of_all_ranks
    total.backward()
    return float(total.detach()), {k: v.grad for k, v in q.items()}


@pytest.mark.parametrize("P", [1, 3, 4])
def test_step_gradients(example, P):
    tokens = 200
    ranks = [example.Rank(r, tokens) for r in range(P)]
    for r in ranks:
        r.bind(P * tokens)
    loss, ref = reference(example, ranks, P * tokens)
    got = sum(float(r.gradients()) for r in ranks)
    example.hc.allreduce([r.grads_flat for r in ranks])
    # binary32 products of 256 and 1000 terms one after the other, four of
    # them in a chain: 4 * 1000 * 2^-24 of the magnitudes, by norm
    assert abs(got - loss) <= 1e-4 * abs(loss)
    for k in ref:
        err = (ranks[0].grads[k].double() - ref[k]).norm() / ref[k].norm()
        assert float(err) <= 4 * 1000 * 2.0 ** -24, k
    for r in ranks[1:]:
        assert torch.equal(r.grads_flat, ranks[0].grads_flat)


def test_losses_fall_and_ranks_stay_alike(example):
    losses, ranks = example.run(P=4, steps=15)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert losses[-1] < 0.9 * losses[0]
    for r in ranks[1:]:
        for k in r.params:
            assert torch.equal(r.params[k], ranks[0].params[k]), k
    whole = example.hc.embedding(ranks[0].params["table"], ranks[0].ids, scale=example.DIM ** 0.5)["out"]
    for part in example.vocabulary_parallel_lookup(ranks[0].params["table"], ranks[0].ids, 4):
        assert torch.equal(part, whole)
