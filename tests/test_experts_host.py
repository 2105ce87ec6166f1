"""Refusals of the expert layer's operators and of gradient clipping: every
bad argument is answered before anything is launched (no GPU needed; device
pointers are made up and never read)."""
import ctypes

import pytest

from collective_communication_algorithms_gb300 import _binding as B

OK, INVALID, UNSUPPORTED, ALIGN, SCRATCH, CUDA = 0, 1, 2, 3, 4, 5
BASE = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    from collective_communication_algorithms_gb300 import build
    build.build()
    return B.lib()


def _no_gpu():
    try:
        import torch
        return not torch.cuda.is_available()
    except Exception:
        return True


host_only = pytest.mark.skipif(not _no_gpu(), reason="uses fake device pointers")


def at(i):
    return BASE + (i << 32)


VALID = {
    "hc_expert_plan": dict(expert_ids=at(0), offsets=at(1), row_tokens=at(2), slots=at(3), scratch=at(4),
                           scratch_bytes=1 << 30, tokens=1000, top=2, experts=8, id_type="int64", first_expert=0),
    "hc_expert_matmul": dict(x=at(0), weight=at(1), offsets=at(2), out=at(3), scratch=at(4), scratch_bytes=1 << 30,
                             rows=100, experts=4, in_dim=64, out_dim=128, dtype="bfloat16", out_dtype="bfloat16",
                             weight_layout="out_in"),
    "hc_expert_matmul_grad": dict(grad_out=at(0), x=at(1), weight=at(2), offsets=at(3), grad_x=at(4), grad_weight=at(5),
                                  scratch=at(6), scratch_bytes=1 << 30, rows=100, experts=4, in_dim=64, out_dim=128,
                                  dtype="bfloat16", grad_weight_dtype="float32", weight_layout="out_in", accumulate=0),
    "hc_expert_combine": dict(y=at(0), slots=at(1), weights=at(2), out=at(3), tokens=50, top=2, rows=100, dim=64,
                              dtype="bfloat16", weight_dtype="float32"),
    "hc_expert_combine_grad": dict(grad_out=at(0), y=at(1), slots=at(2), weights=at(3), grad_y=at(4),
                                   grad_weights=at(5), tokens=50, top=2, rows=100, dim=64, dtype="bfloat16",
                                   weight_dtype="float32"),
}


def status(name, **change):
    args = B.operator_args(name, **dict(VALID[name], **change))
    try:
        B.hc_operator(name, args)
        return OK
    except B.HcError as e:
        return e.status


@host_only
@pytest.mark.parametrize("name", sorted(VALID))
def test_valid_calls_and_common_refusals(name):
    assert status(name) == CUDA
    args = B.operator_args(name, **VALID[name])
    args.struct_size -= 8
    with pytest.raises(B.HcError) as e:
        B.hc_operator(name, args)
    assert e.value.status == INVALID
    assert getattr(B.lib(), name)(None, None) == INVALID
    for field, _ in B.OPERATORS[name]._fields_:
        if field.endswith("dtype"):
            assert status(name, **{field: 7}) == INVALID, field
            assert status(name, **{field: "int32"}) == UNSUPPORTED, field
        if field == "id_type":
            assert status(name, id_type=2) == INVALID
        if field == "weight_layout":
            assert status(name, weight_layout=2) == INVALID
        if field.endswith("_stride"):
            assert status(name, **{field: 3}) == INVALID, field
            assert status(name, **{field: 2 ** 62}) == INVALID, field


@host_only
@pytest.mark.parametrize("name,fields", [
    ("hc_expert_plan", "expert_ids offsets"), ("hc_expert_matmul", "x weight offsets out"),
    ("hc_expert_matmul_grad", "grad_out x weight offsets"), ("hc_expert_combine", "y slots out"),
    ("hc_expert_combine_grad", "grad_out y slots")])
def test_missing_and_misaligned_pointers(name, fields):
    for f in fields.split():
        assert status(name, **{f: 0}) == INVALID, f
    for f in [n for n, t in B.OPERATORS[name]._fields_ if t is ctypes.c_void_p and n != "scratch"]:
        assert status(name, **{f: VALID[name][f] + 1}) == ALIGN, f


@host_only
def test_sizes():
    for n in ("hc_expert_matmul", "hc_expert_matmul_grad"):
        for f in ("experts", "in_dim", "out_dim"):
            assert status(n, **{f: 0}) == INVALID
        assert status(n, experts=1025) == UNSUPPORTED
        assert status(n, in_dim=65537) == UNSUPPORTED
        assert status(n, out_dim=65537) == UNSUPPORTED
        assert status(n, rows=1 << 31) == UNSUPPORTED
    assert status("hc_expert_matmul_grad", accumulate=2) == INVALID
    assert status("hc_expert_plan", experts=1025) == UNSUPPORTED
    assert status("hc_expert_plan", experts=0) == INVALID
    assert status("hc_expert_plan", top=0) == INVALID
    assert status("hc_expert_plan", tokens=1 << 30, top=2) == UNSUPPORTED
    assert status("hc_expert_plan", tokens=1 << 62, top=1 << 62) == UNSUPPORTED
    for n in ("hc_expert_combine", "hc_expert_combine_grad"):
        assert status(n, top=0) == INVALID
        assert status(n, dim=0) == INVALID
        assert status(n, rows=1 << 31) == UNSUPPORTED
        assert status(n, tokens=1 << 30, top=2) == UNSUPPORTED


@host_only
def test_optional_operands_and_nothing_to_do():
    assert status("hc_expert_plan", row_tokens=0, slots=0) == CUDA
    assert status("hc_expert_plan", tokens=0, expert_ids=0, row_tokens=0, slots=0) == CUDA  # offsets to write
    assert status("hc_expert_matmul", rows=0, x=0, weight=0, out=0, offsets=0) == OK
    g = "hc_expert_matmul_grad"
    assert status(g, grad_x=0, weight=0) == CUDA
    assert status(g, grad_weight=0, x=0) == CUDA
    assert status(g, grad_x=0, grad_weight=0) == INVALID
    assert status(g, rows=0, grad_out=0, x=0, accumulate=1) == OK
    assert status(g, rows=0, grad_out=0, x=0) == CUDA                                        # zeros to write
    assert status("hc_expert_combine", weights=0) == CUDA
    assert status("hc_expert_combine", weights=0, weight_dtype=9) == CUDA
    assert status("hc_expert_combine", tokens=0, y=0, slots=0, out=0) == OK
    g = "hc_expert_combine_grad"
    assert status(g, grad_weights=0, y=0) == CUDA
    assert status(g, grad_y=0) == CUDA
    assert status(g, grad_y=0, grad_weights=0) == INVALID


@host_only
def test_overlaps_and_scratch():
    n = "hc_expert_matmul"
    assert status(n, out=at(0)) == INVALID
    assert status(n, out=at(1) + 64) == INVALID
    assert status(n, out=at(2)) == INVALID
    g = "hc_expert_matmul_grad"
    for f in ("grad_x", "grad_weight"):
        for i in range(4):
            assert status(g, **{f: at(i)}) == INVALID
    assert status(g, grad_x=at(5)) == INVALID
    # weights apart by more than their rows: taken as one piece
    assert status(g, expert_stride=128 * 64 + 8, grad_x=at(2) + 64) == INVALID
    assert status("hc_expert_combine", out=at(0)) == INVALID
    c = "hc_expert_combine_grad"
    assert status(c, grad_y=at(1)) == CUDA          # in place
    assert status(c, grad_y=at(1) + 128) == INVALID
    assert status(c, grad_y=at(0)) == INVALID
    assert status(c, grad_weights=at(3)) == INVALID
    p = "hc_expert_plan"
    assert status(p, slots=at(2)) == INVALID
    assert status(p, offsets=at(0)) == INVALID
    need = B.hc_operator_scratch_bytes(p, B.operator_args(p, **dict(VALID[p], tokens=100000)))
    assert need > 0
    assert status(p, tokens=100000, scratch=0) == SCRATCH
    assert status(p, tokens=100000, scratch_bytes=need - 1) == SCRATCH
    assert status(p, tokens=100000, scratch=at(4) + 8) == ALIGN
    assert status(p, tokens=100000, scratch=at(0)) == INVALID
    assert status(p, tokens=100, scratch=0, scratch_bytes=0) == CUDA


# ------------------------------------------------------------------ clipping
def clip(listed, name="hc_clip_grads", **change):
    table = (B.hc_grad_t * max(1, len(listed)))()
    for t, (i, o, n, a, b) in zip(table, listed):
        t.in_, t.out, t.count, t.in_dtype, t.out_dtype = i, o, n, a, b
    kw = dict(tensors=ctypes.addressof(table), num=len(listed), norm=at(40), factor=at(41), scratch=at(42),
              scratch_bytes=1 << 20, scale=1.0, max_norm=1.0, eps=1e-6)
    args = B.operator_args(name, **dict(kw, **change))
    try:
        B.hc_operator(name, args)
        return OK
    except B.HcError as e:
        return e.status


@host_only
def test_clip_refusals():
    f, b = 1, 2
    one = [(at(0), 0, 100, f, 0)]
    assert clip(one) == CUDA
    assert clip([]) == CUDA
    assert clip([], tensors=0) == CUDA
    assert clip(one, tensors=0) == INVALID
    assert clip(one, norm=0) == INVALID
    assert clip(one, norm=at(40) + 2) == ALIGN
    assert clip(one, factor=0) == CUDA
    for v in (0.0, -1.0, float("nan")):
        assert clip(one, max_norm=v) == INVALID
        assert clip(one, "hc_grad_norm", max_norm=v) == CUDA
    assert clip(one, max_norm=float("inf")) == CUDA
    for v in (-1.0, float("nan"), float("inf")):
        assert clip(one, eps=v) == INVALID
    for v in (float("nan"), float("inf")):
        assert clip(one, scale=v) == INVALID
        assert clip(one, "hc_grad_norm", scale=v) == INVALID
    assert clip([(0, 0, 100, f, 0)]) == INVALID
    assert clip([(0, 0, 0, f, 0)]) == CUDA
    assert clip([(at(0) + 2, 0, 100, f, 0)]) == ALIGN
    assert clip([(at(0) + 2, 0, 100, b, 0)]) == CUDA
    assert clip([(at(0), at(1) + 2, 100, b, f)]) == ALIGN
    assert clip([(at(0), 0, 100, 0, 0)]) == UNSUPPORTED
    assert clip([(at(0), at(1), 100, f, 0)]) == UNSUPPORTED
    assert clip([(at(0), at(1), 100, f, 9)]) == INVALID
    assert clip([(at(0), 0, 1 << 56, f, 0)]) == UNSUPPORTED
    need = B.hc_operator_scratch_bytes("hc_clip_grads", _args([(at(0), 0, 100000, f, 0)]))
    assert need > 0
    assert clip([(at(0), 0, 100000, f, 0)], scratch_bytes=need - 1) == SCRATCH
    assert clip([(at(0), 0, 100000, f, 0)], scratch=0) == SCRATCH
    assert clip([(at(0), 0, 100000, f, 0)], scratch=at(42) + 8) == ALIGN


_kept = []


def _args(tensors):
    table = (B.hc_grad_t * len(tensors))()
    for t, (i, o, n, a, b) in zip(table, tensors):
        t.in_, t.out, t.count, t.in_dtype, t.out_dtype = i, o, n, a, b
    _kept.append(table)
    return B.operator_args("hc_clip_grads", tensors=ctypes.addressof(table), num=len(tensors))


@host_only
def test_clip_overlaps():
    f, b = 1, 2
    a, c = (at(0), 0, 100, f, 0), (at(1), 0, 100, f, 0)
    assert clip([a, c]) == CUDA
    assert clip([a, a]) == INVALID                                   # listed twice
    assert clip([a, a], "hc_grad_norm") == CUDA
    assert clip([a, (at(0) + 396, 0, 1, f, 0)]) == INVALID
    assert clip([a, (at(0) + 400, 0, 1, f, 0)]) == CUDA              # right behind
    assert clip([(at(0), at(0), 100, f, f)]) == CUDA                 # in place, said so
    assert clip([(at(0), at(0), 100, f, b)]) == INVALID              # with another type
    assert clip([(at(0), at(0) + 4, 100, f, f)]) == INVALID
    assert clip([(at(0), at(2), 100, f, f), (at(0), at(3), 100, f, f)]) == CUDA   # one input, two outputs
    assert clip([(at(0), at(2), 100, f, f), (at(1), at(2), 100, f, f)]) == INVALID
    assert clip([(at(0), at(1) + 80, 100, f, f), c]) == INVALID      # over another gradient
    assert clip([a], norm=at(0) + 8) == INVALID
    assert clip([a], "hc_grad_norm", norm=at(0) + 8) == INVALID
    assert clip([a], factor=at(40)) == INVALID
    assert clip([a], scratch=at(0)) == INVALID


def test_tensor_functions_refuse():
    torch = pytest.importorskip("torch")
    import collective_communication_algorithms_gb300 as hc
    cpu = torch.zeros(4, 8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: hc.clip_grads([]), lambda: hc.clip_grads([cpu], 1.0), lambda: hc.grad_norm([cpu]),
                 lambda: hc.expert_plan(ids, 3), lambda: hc.expert_matmul(cpu, torch.zeros(2, 3, 8), ids[0]),
                 lambda: hc.expert_matmul_grad(cpu, ids[0], x=cpu), lambda: hc.expert_combine(cpu, ids),
                 lambda: hc.expert_combine_grad(cpu, ids, rows=3)):
        with pytest.raises((ValueError, TypeError)):
            call()
