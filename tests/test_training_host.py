"""Refusals of the training operators: every bad argument is answered before
anything is launched (no GPU needed; device pointers are made up and never
read)."""
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
    "hc_embedding": dict(table=at(0), ids=at(1), out=at(2), tokens=10, rows=20, dim=64, table_dtype="float32",
                         out_dtype="bfloat16", id_type="int64", scale=1.0),
    "hc_embedding_grad": dict(grad_out=at(0), ids=at(1), grad_table=at(2), tokens=1000, rows=20, dim=64,
                              grad_out_dtype="bfloat16", grad_table_dtype="float32", id_type="int32", scale=1.0,
                              padding_id=-1, scratch=at(3), scratch_bytes=1 << 30),
    "hc_block_norm": dict(y=at(0), x=at(1), post_weight=at(2), gate=at(3), pre_weight=at(4), r=at(5), z=at(6),
                          post_rstd=at(7), pre_rstd=at(8), tokens=12, dim=64, gate_rows=4, dtype="bfloat16",
                          weight_dtype="float32", residual_scale=1.0, eps=1e-6),
    "hc_block_norm_grad": dict(grad_r=at(0), grad_z=at(1), y=at(2), x=at(3), post_weight=at(4), gate=at(5),
                               pre_weight=at(6), post_rstd=at(7), pre_rstd=at(8), grad_y=at(9), grad_x=at(10),
                               grad_post_weight=at(11), grad_gate=at(12), grad_pre_weight=at(13), tokens=12, dim=64,
                               gate_rows=4, dtype="bfloat16", weight_dtype="float32", residual_scale=1.0,
                               scratch=at(14), scratch_bytes=1 << 30),
    "hc_distill": dict(logits=at(0), teacher_logits=at(1), teacher_ids=at(2), row_weight=at(3), loss=at(4),
                       stats=at(5), grad_logits=at(6), tokens=10, vocab=1000, top=8, dtype="bfloat16",
                       teacher_dtype="float32", id_type="int64", temperature=2.0, scale=1.0),
}
VALID["hc_distill_grad"] = dict(VALID["hc_distill"], loss=0)


def status(name, **change):
    args = B.operator_args(name, **dict(VALID[name], **change))
    try:
        B.hc_operator(name, args)
        return OK
    except B.HcError as e:
        return e.status


@host_only
@pytest.mark.parametrize("name", sorted(VALID))
def test_valid_calls_without_gpu_report_the_missing_device(name):
    assert status(name) == CUDA


@host_only
@pytest.mark.parametrize("name", sorted(VALID))
def test_common_refusals(name):
    args = B.operator_args(name, **VALID[name])
    args.struct_size -= 8
    with pytest.raises(B.HcError) as e:
        B.hc_operator(name, args)
    assert e.value.status == INVALID
    lib = B.lib()
    assert getattr(lib, name)(None, None) == INVALID
    for field, ctype in B.OPERATORS[name]._fields_:
        if field.endswith("dtype"):
            assert status(name, **{field: 7}) == INVALID, field
            assert status(name, **{field: "int32"}) == UNSUPPORTED, field
        if field == "id_type":
            assert status(name, id_type=2) == INVALID
        if field.endswith("_stride"):
            assert status(name, **{field: 3}) == INVALID, field
            assert status(name, **{field: 2 ** 62}) == INVALID, field


@host_only
@pytest.mark.parametrize("name,fields", [
    ("hc_embedding", "table ids out"), ("hc_embedding_grad", "grad_out ids grad_table"),
    ("hc_block_norm", "y x r"), ("hc_block_norm_grad", "y x post_rstd pre_rstd grad_y grad_x"),
    ("hc_distill", "logits teacher_logits teacher_ids loss"),
    ("hc_distill_grad", "logits teacher_logits teacher_ids stats grad_logits")])
def test_missing_and_misaligned_pointers(name, fields):
    for f in fields.split():
        assert status(name, **{f: 0}) == INVALID, f
        assert status(name, **{f: VALID[name][f] + 1}) == ALIGN, f


@host_only
def test_sizes():
    for name in ("hc_embedding", "hc_embedding_grad"):
        assert status(name, dim=0) == INVALID
        assert status(name, rows=0) == INVALID
        assert status(name, tokens=1 << 31) == UNSUPPORTED
        assert status(name, rows=1 << 31) == UNSUPPORTED
        assert status(name, dim=(1 << 24) + 1) == UNSUPPORTED
    for name in ("hc_block_norm", "hc_block_norm_grad"):
        assert status(name, dim=0) == INVALID
        assert status(name, dim=32769) == UNSUPPORTED
        assert status(name, gate_rows=5) == INVALID   # does not divide the tokens
        assert status(name, gate_rows=0) == INVALID
        assert status(name, gate=0, grad_gate=0, gate_rows=5) == CUDA if name.endswith("grad") else True
    for name in ("hc_distill", "hc_distill_grad"):
        assert status(name, vocab=0) == INVALID
        assert status(name, top=0) == INVALID
        assert status(name, top=1025) == UNSUPPORTED
        assert status(name, vocab=(3 << 18) + 1) == UNSUPPORTED       # 1.5 MiB of bf16
        assert status(name, vocab=(3 << 17) + 1, dtype="float32") == UNSUPPORTED
        for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
            assert status(name, temperature=tau) == INVALID
        assert status(name, scale=float("inf")) == INVALID
    for eps in (-1.0, float("nan"), float("inf")):
        assert status("hc_block_norm", eps=eps) == INVALID


@host_only
def test_lookup_scale():
    """Zero rows stay zeros: a scale that would make NaN of them is refused."""
    for scale in (float("inf"), float("-inf"), float("nan")):
        assert status("hc_embedding", scale=scale) == INVALID
    assert status("hc_embedding", scale=-2.0) == CUDA
    assert status("hc_embedding", scale=0.0) == CUDA


@host_only
def test_optional_operands():
    assert status("hc_block_norm", z=0, pre_rstd=0) == CUDA
    assert status("hc_block_norm", z=0) == INVALID            # pre_rstd without the norm
    assert status("hc_block_norm", post_weight=0, gate=0, pre_weight=0, post_rstd=0, pre_rstd=0) == CUDA
    g = "hc_block_norm_grad"
    assert status(g, grad_r=0) == CUDA
    assert status(g, grad_z=0, pre_rstd=0) == CUDA
    assert status(g, grad_r=0, grad_z=0) == INVALID
    assert status(g, gate=0) == INVALID                       # grad_gate without a gate
    assert status(g, grad_post_weight=0, grad_gate=0, grad_pre_weight=0) == CUDA
    assert status("hc_distill", row_weight=0, stats=0, grad_logits=0) == CUDA
    assert status("hc_embedding_grad", accumulate=2) == INVALID


@host_only
def test_scratch():
    for name, tokens in (("hc_embedding_grad", 1000), ("hc_block_norm_grad", 1200)):
        need = B.hc_operator_scratch_bytes(name, B.operator_args(name, **dict(VALID[name], tokens=tokens)))
        assert need > 0
        assert status(name, tokens=tokens, scratch=0) == SCRATCH
        assert status(name, tokens=tokens, scratch_bytes=need - 1) == SCRATCH
        assert status(name, tokens=tokens, scratch_bytes=need) == CUDA
        assert status(name, tokens=tokens, scratch=at(14) + 8) == ALIGN
        assert status(name, tokens=tokens, scratch=at(0)) == INVALID         # over an input
    few = dict(VALID["hc_embedding_grad"], tokens=200)
    assert B.hc_operator_scratch_bytes("hc_embedding_grad", B.operator_args("hc_embedding_grad", **few)) == 0
    assert status("hc_embedding_grad", tokens=200, scratch=0, scratch_bytes=0) == CUDA
    # few tokens of the block norm: one block, no partial sums
    few = dict(VALID["hc_block_norm_grad"], tokens=4)
    assert B.hc_operator_scratch_bytes("hc_block_norm_grad", B.operator_args("hc_block_norm_grad", **few)) == 0
    assert status("hc_block_norm_grad", tokens=4, scratch=0, scratch_bytes=0) == CUDA
    bad = B.operator_args("hc_embedding_grad", **dict(VALID["hc_embedding_grad"], rows=0))
    assert B.hc_operator_scratch_bytes("hc_embedding_grad", bad) == 0


@host_only
def test_scratch_of_a_call_without_a_gate_does_not_depend_on_gate_rows():
    name = "hc_block_norm_grad"
    for rows in (0, 1, 5, 7, 1200, 5000):  # 7 and 5000 do not divide the tokens
        call = dict(VALID[name], tokens=1200, gate=0, grad_gate=0, gate_rows=rows)
        need = B.hc_operator_scratch_bytes(name, B.operator_args(name, **call))
        assert need > 0
        assert status(name, **dict(call, scratch_bytes=need)) == CUDA
    refused = dict(VALID[name], tokens=1200, dim=32769, gate_rows=7)
    assert B.hc_operator_scratch_bytes(name, B.operator_args(name, **refused)) == 0


@host_only
def test_overlaps():
    assert status("hc_embedding", out=at(0) + 64) == INVALID
    assert status("hc_embedding", out=at(1)) == INVALID
    n = "hc_block_norm"
    assert status(n, r=at(1), z=at(0)) == CUDA                # in place
    assert status(n, r=at(0), z=at(1)) == CUDA
    assert status(n, r=at(1) + 128) == INVALID                # one row further
    assert status(n, r=at(1), r_stride=128) == INVALID        # in place with another stride
    assert status(n, r=at(6)) == INVALID                      # two outputs in one place
    assert status(n, r=at(2)) == INVALID                      # over a weight
    assert status(n, post_rstd=at(0)) == INVALID
    # the halves of one buffer of 128 columns interleave without overlapping
    halves = dict(r=at(20), z=at(20) + 128, r_stride=128, z_stride=128)
    assert status(n, **halves) == CUDA
    assert status(n, **dict(halves, z=at(20) + 126)) == INVALID
    assert status(n, **dict(halves, z=at(20) + 130)) == INVALID
    g = "hc_block_norm_grad"
    assert status(g, grad_x=at(0), grad_y=at(1)) == CUDA
    assert status(g, grad_x=at(2), grad_y=at(3)) == CUDA
    assert status(g, grad_x=at(0), grad_y=at(0)) == INVALID
    assert status(g, grad_gate=at(5)) == INVALID
    assert status("hc_distill", grad_logits=at(0)) == CUDA
    assert status("hc_distill", grad_logits=at(0) + 2) == INVALID
    assert status("hc_distill", stats=at(4)) == INVALID
    assert status("hc_distill_grad", grad_logits=at(5)) == INVALID


@host_only
def test_no_tokens_launch_nothing():
    assert status("hc_embedding", tokens=0, table=0, ids=0, out=0) == OK
    assert status("hc_embedding_grad", tokens=0, grad_out=0, ids=0, accumulate=1) == OK
    assert status("hc_embedding_grad", tokens=0, grad_out=0, ids=0) == CUDA   # zeros to write
    assert status("hc_block_norm", tokens=0, y=0, x=0, r=0) == OK
    assert status("hc_distill", tokens=0, logits=0, teacher_logits=0, teacher_ids=0, loss=0) == OK


def test_tensor_functions_refuse():
    torch = pytest.importorskip("torch")
    import collective_communication_algorithms_gb300 as hc
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        hc.embedding(cpu, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        hc.block_norm(cpu, cpu)
    with pytest.raises(ValueError):
        hc.distill(cpu, cpu, torch.zeros(4, 8, dtype=torch.int64))
