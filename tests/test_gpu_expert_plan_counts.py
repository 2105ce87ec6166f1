"""The plan at numbers of experts whose tables in shared memory end just below
48 KiB, in processes that have planned for no more experts before (what a kernel
may use of shared memory, once raised, stays raised)."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
sys.path[:0] = [%r, %r]
import torch
import collective_communication_algorithms_gb300 as hc
from experts_util import plan
tokens, top, counts = int(sys.argv[1]), int(sys.argv[2]), [int(v) for v in sys.argv[3:]]
for experts in counts:
    ids = torch.randint(-1, experts + 1, (tokens, top), generator=torch.Generator("cuda").manual_seed(experts), device="cuda")
    o = hc.expert_plan(ids, experts)
    offsets, rows, slots = plan(ids.cpu(), experts, 0)
    assert o["offsets"].tolist() == offsets, experts
    assert o["tokens"].tolist() == rows, experts
    assert o["slots"].reshape(-1).tolist() == slots, experts
""" % (ROOT, os.path.join(ROOT, "tests"))


@pytest.mark.parametrize("tokens,top,counts", [
    (4096, 2, [765, 766, 767, 768, 769]),  # one block: 64 bytes an expert
    (4099, 2, [679, 680, 681, 682, 683]),  # several blocks: 72 bytes
])
def test_tables_that_end_below_48_kib(tokens, top, counts):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from collective_communication_algorithms_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT, str(tokens), str(top)] + [str(c) for c in counts], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
