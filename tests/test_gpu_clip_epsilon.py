"""Gradient clipping with limits and epsilons whose quotient binary32 does not
hold before the scale brings it back."""
import math

import pytest

torch = pytest.importorskip("torch")

import collective_communication_algorithms_gb300 as hc  # noqa: E402

pytestmark = pytest.mark.gpu

F32 = torch.float32
OPS = 40  # roundings: half of 64 in the norm, and those of the factor and the product


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from collective_communication_algorithms_gb300 import build
    build.build()


@pytest.mark.parametrize("max_norm,scale,eps", [(1e-10, 1e10, 1e35), (1e-15, 1e16, 3e38), (1e-17, 1.0, 1e20), (1e17, 1e-15, 1e30),
                                                (1.0, 1.0, 1e18), (1e-12, 1e12, 3e20)])
def test_large_epsilons(max_norm, scale, eps):
    g = torch.ones(1000, device="cuda")
    out = torch.empty_like(g)
    o = hc.clip_grads([g], max_norm, out=[out], scale=scale, eps=eps)
    m, s, e = (float(torch.tensor(v, dtype=F32)) for v in (max_norm, scale, eps))
    factor = min(1.0, m / (math.sqrt(1000) * s + e)) * s
    assert abs(float(o["factor"]) - factor) <= OPS * 2.0 ** -24 * factor + 2.0 ** -149
    assert abs(float(out[0]) - factor) <= OPS * 2.0 ** -24 * factor + 2.0 ** -149
