"""Calls of the expert layer's products that take longer than a wait may last."""
import pytest

torch = pytest.importorskip("torch")

import collective_communication_algorithms_gb300 as hc  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from collective_communication_algorithms_gb300 import build
    build.build()


def test_a_call_of_seconds_reports_no_expired_wait():
    """One expert with nearly 2^30 rows: one block's work, for several times the
    2 s of a wait.  All products are 1, so the gradient is the number of rows."""
    rows = (1 << 30) - 37
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.ones(rows, 8, dtype=BF16, device="cuda")
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    from collective_communication_algorithms_gb300 import _binding as B
    for dtype in (F32, BF16):
        gw = torch.zeros(1, 8, 8, dtype=dtype, device="cuda")
        hc.expert_matmul_grad(x, offsets, x=x, grad_weight=gw)
        torch.cuda.synchronize()
        assert B.hc_device_status(clear=True) == 0
        # whole numbers below 2^30 in multiples of 64 are exact in binary32, the last addition rounds
        assert bool((gw == torch.tensor(rows, device="cuda").to(F32).to(dtype)).all()), gw


@pytest.mark.parametrize("what", ["product in binary32", "long product in bf16", "gradient of many rows in bf16"])
@pytest.mark.parametrize("large", [False, True])
def test_expired_waits_of_sums_in_segments(what, large):
    """hc_test_expire_waits: the first wait on the copies gives up after 1 ms,
    although they land; the call ends and reports, and the next one is right."""
    from collective_communication_algorithms_gb300 import _binding as B
    g = torch.Generator("cuda").manual_seed(5)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(BF16)
    rows = 20011 if "rows" in what else 2500 if large else 90
    inner, outer = (2048, 2500) if large else (200, 136)
    if "long" in what:
        inner = 16392
    offsets = torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32, device="cuda")
    x, w, go = normal(rows, inner), normal(3, outer, inner), normal(rows, outer)
    if "rows" in what:
        call = hc.bind_expert_matmul_grad(go, offsets, x=x)
    else:
        call = hc.bind_expert_matmul(x, w, offsets, out_dtype=F32 if "binary32" in what else None)
    call()
    torch.cuda.synchronize()
    want = [v.clone() for v in call.outputs.values()]
    assert B.hc_device_status() == 0
    B.hc_test_expire_waits(True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        B.hc_test_expire_waits(False)
    assert B.hc_device_status(clear=True) == 6
    call()
    torch.cuda.synchronize()
    assert B.hc_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, call.outputs.values()))
