"""Whose memory the operators' and layers' scratch is (no GPU: the stream, the allocator and
the C calls are stand-ins)."""
import contextlib

import pytest
import torch

import onnx_recurrent_layers_amd as rl


class Stream:
    def __init__(self, handle):
        self.device, self.cuda_stream, self.waited = torch.device("cuda", 0), handle, []

    def record_event(self):
        return ("event", self.cuda_stream)

    def wait_event(self, event):
        self.waited.append(event)


class Machine:
    """A current stream, and an allocator that notes which one it counted memory to."""

    def __init__(self, monkeypatch):
        self.now, self.made, self.recorded, self.capturing = Stream(0), [], [], set()
        cuda = torch.cuda

        @contextlib.contextmanager
        def on(stream):
            before, self.now = self.now, self.now if stream is None else stream
            yield
            self.now = before

        machine = self

        class Memory:
            def data_ptr(self):
                return 1 << 20

            def record_stream(self, stream):
                machine.recorded.append(stream.cuda_stream)

        def empty(size, **_):
            self.made.append((size, self.now.cuda_stream))
            return Memory()

        monkeypatch.setattr(cuda, "stream", on)
        monkeypatch.setattr(cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(cuda, "current_device", lambda: 0)
        monkeypatch.setattr(cuda, "is_current_stream_capturing", lambda: self.now.cuda_stream in self.capturing)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: self.now.cuda_stream)
        monkeypatch.setattr(torch, "empty", empty)


@pytest.fixture
def machine(monkeypatch):
    monkeypatch.setenv("RNN_SCAN_CHUNK", "16")
    return Machine(monkeypatch)


def scan():
    op = rl.SelectiveScan(dtype="f32", seq=64, batch=3, channels=6, state=4, device="cuda:0")
    op.calls = []
    op._encode = op._encode_backward = lambda *args: op.calls.append(args[-1] or 0) or rl.RNN_OK
    return op


def test_scratch_counts_to_the_first_calls_stream(machine):
    """Memory that the allocator counts to one stream may still be in use by that stream's queued work when another
    stream's first call writes it."""
    op, other = scan(), Stream(7)
    assert op.forward_bytes and op.backward_bytes and machine.made == []
    op.encode({}, stream=other)
    op.backward({}, stream=other)
    assert machine.made == [(op.forward_bytes, 7), (op.backward_bytes, 7)]
    assert op.calls == [7, 7] and machine.recorded == []
    op.encode({})        # a later call on another stream: kept until that has run
    assert op.calls[-1] == 0 and machine.recorded == [0] and len(machine.made) == 2


def test_scratch_of_a_changed_current_stream(machine):
    op = scan()
    machine.now = Stream(5)
    op.encode({})
    op.backward({})
    assert [s for _, s in machine.made] == [5, 5]


def test_capture_is_the_calls_streams(machine):
    """A stream that is being captured without being the current one."""
    op, other = scan(), Stream(7)
    machine.capturing = {7}
    with pytest.raises(rl.RnnError, match="scratch: call backward once"):
        op.backward({}, stream=other)
    assert op.calls == [] and machine.made == []
    op.backward({})
    op.backward({}, stream=other)
    assert op.calls == [0, 7] and machine.recorded == []


def test_another_devices_stream_takes_no_scratch(machine):
    op, other = scan(), Stream(7)
    other.device = torch.device("cuda", 1)
    for call in (op.encode, op.backward):
        with pytest.raises(rl.RnnError, match="stream: on cuda:1, expected cuda:0"):
            call({}, stream=other)
    assert machine.made == [] and op.calls == []


def test_layer_on_another_stream_waits_for_its_scratch(machine, monkeypatch):
    """A layer's scratch is made with the layer: a call on another stream waits for what was queued before it."""
    from onnx_recurrent_layers_amd.synth import LayerSpec
    calls = []
    monkeypatch.setattr(rl, "rnn_encode", lambda *args: calls.append(args[-1]))
    layer = rl.Layer(LayerSpec("LSTM", seq=5, batch=3, input=4, hidden=6), device="cuda:0")
    other = Stream(7)
    layer.encode({})
    assert other.waited == machine.now.waited == [] and machine.recorded == []
    layer.encode({}, stream=other)
    assert calls == [0, 7] and other.waited == [("event", 0)] and machine.recorded == [7, 7]
    machine.capturing = {9}
    captured = Stream(9)
    layer.encode({}, stream=captured)      # (no wait for uncaptured work may be captured)
    assert captured.waited == [] and machine.recorded == [7, 7]


def test_layer_off_the_device():
    """A layer's plan and scratch sizes can be had where there is no GPU."""
    from onnx_recurrent_layers_amd.synth import LayerSpec
    layer = rl.Layer(LayerSpec("LSTM", seq=5, batch=3, input=4, hidden=6), device="cpu")
    assert layer.plan.steps == 5 and layer.state.numel() >= layer.state_bytes
