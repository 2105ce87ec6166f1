"""Which GPU a training operator runs on: its tensors', whatever the current
one is.  Stand-in tensors, streams and entry points; nothing is launched."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import collective_communication_algorithms_gb300 as hc  # noqa: E402
from collective_communication_algorithms_gb300 import _binding as B  # noqa: E402
from collective_communication_algorithms_gb300 import training  # noqa: E402


class Tensor:
    def __init__(self, shape, dtype=torch.float32, index=1):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, torch.device("cuda", index), True
        self.recorded = []

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def stride(self, i):
        return torch.Size(self.shape[i % self.dim() + 1:]).numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 40

    def record_stream(self, stream):
        self.recorded.append((stream.device, stream.cuda_stream))


class Stream:
    def __init__(self, handle, index):
        self.cuda_stream, self.device = handle, torch.device("cuda", index)


@pytest.fixture
def gpus(monkeypatch):
    """Two GPUs, the first one current; the entry points record the current one and their stream."""
    state = type("State", (), {"current": 0, "calls": [], "streams": {0: Stream(0, 0), 1: Stream(0, 1)}})()

    def index(device):
        return state.current if device is None else device if isinstance(device, int) else torch.device(device).index

    @contextlib.contextmanager
    def on_device(device):
        was, state.current = state.current, index(device)
        try:
            yield
        finally:
            state.current = was

    @contextlib.contextmanager
    def on_stream(stream):
        i = stream.device.index
        was, state.streams[i] = state.streams[i], stream
        try:
            with on_device(i):
                yield
        finally:
            state.streams[i] = was

    def entry(args, stream):
        state.calls.append((state.current, stream.value if stream is not None else 0))
        return 0

    class Lib:
        def __getitem__(self, name):
            def call(args, stream):
                return entry(args, stream)
            return call

    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", on_device)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state.streams[index(device)])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0, index(device)))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: Stream(h, index(device)))
    monkeypatch.setattr(B, "lib", lambda: Lib())
    monkeypatch.setattr(B, "hc_operator_scratch_bytes", lambda name, args: 64)
    monkeypatch.setattr(training, "_new", lambda like, shape, dtype: Tensor(shape, dtype, like.device.index))
    return state


def binds(**kw):
    ids = Tensor((5,), torch.int64)
    rows, w = Tensor((5, 8)), Tensor((8,))
    teacher, tid, per_row = Tensor((5, 2)), Tensor((5, 2), torch.int64), Tensor((5,))
    yield hc.bind_embedding(Tensor((9, 8)), ids, **kw)
    yield hc.bind_embedding_grad(rows, ids, Tensor((9, 8)), **kw)
    yield hc.bind_block_norm(rows, rows, w, None, w, **kw)
    yield hc.bind_block_norm_grad(rows, rows, rows, rows, per_row, per_row, w, None, w, **kw)
    yield hc.bind_distill(rows, teacher, tid, **kw)
    yield hc.bind_distill_grad(rows, teacher, tid, Tensor((5, 2)), **kw)


def test_calls_run_on_their_tensors_gpu(gpus):
    gpus.streams[1] = Stream(17, 1)
    for call in binds():
        call()
        assert gpus.calls.pop() == (1, 17) and gpus.current == 0
        gpus.current = 1  # another one current at a later call
        call()
        assert gpus.calls.pop() == (1, 17) and gpus.current == 1
        gpus.current = 0


@pytest.mark.parametrize("stream,handle", [(Stream(23, 1), 23), (23, 23), (0, 0), (Stream(0, 1), 0)])
def test_streams_are_those_of_the_tensors_gpu(gpus, stream, handle):
    gpus.streams[1] = Stream(17, 1)
    for call in binds(stream=stream):
        call()
        assert gpus.calls.pop() == (1, handle) and gpus.current == 0
        for t in call.outputs.values():
            assert all(d.index == 1 for d, _ in t.recorded)


def test_a_stream_of_another_gpu_is_refused(gpus):
    for handle in (0, 5):
        with pytest.raises(ValueError, match="stream"):
            hc.bind_embedding(Tensor((9, 8)), Tensor((5,), torch.int64), stream=Stream(handle, 0))


def test_operands_of_two_gpus_are_refused(gpus):
    with pytest.raises(ValueError, match="cuda:0"):
        hc.bind_embedding(Tensor((9, 8)), Tensor((5,), torch.int64, 0))
