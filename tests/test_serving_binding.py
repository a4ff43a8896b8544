"""The binding's side of the serving operators: which workspace a call gets.
CPU only: torch's CUDA state is a fake."""
import contextlib

import pytest

import w4a8_quantized_gemm_quantize_b200 as w4a8
from w4a8_quantized_gemm_quantize_b200 import build as w4a8_build

torch = pytest.importorskip("torch")


class FakeCuda:
    """Two devices, the current one and which of their streams are being captured."""

    def __init__(self, monkeypatch, current=0, capturing=()):
        self.current, self.capturing, self.streams = current, set(capturing), {0: 100, 1: 200}
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.current in self.capturing)
        monkeypatch.setattr(torch.cuda, "device", self.device)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: self.streams[index], raising=False)
        monkeypatch.setattr(w4a8, "_kv8_ws", {})
        w4a8_build.build()
        self.q = torch.zeros(1)  # where its workspace is made: here

    @contextlib.contextmanager
    def device(self, index):
        saved, self.current = self.current, index
        try:
            yield
        finally:
            self.current = saved

    def workspace(self, index, nbytes=4096):
        return w4a8._kv8_workspace_for(self.q, index, nbytes)


def test_a_workspace_is_kept_for_each_stream(monkeypatch):
    f = FakeCuda(monkeypatch)
    a = f.workspace(0)
    assert f.workspace(0) is a and not a[:w4a8.KV8_COUNTER_BYTES].any()
    f.streams[0] = 101
    assert f.workspace(0) is not a


@pytest.mark.parametrize("current,index,capturing,kept", [(0, 0, {0}, False), (0, 1, {1}, False), (1, 0, {0}, False),
                                                          (0, 1, {0}, True), (1, 0, {1}, True), (0, 0, set(), True)])
def test_a_captured_call_is_that_of_the_tensors_device(monkeypatch, current, index, capturing, kept):
    """The stream that counts is the current one of the tensors' device, not of the current device."""
    f = FakeCuda(monkeypatch, current, capturing)
    a = f.workspace(index)
    assert (f.workspace(index) is a) == kept and bool(w4a8._kv8_ws) == kept
    assert f.current == current


@pytest.mark.parametrize("device", [None, 0, "cuda:0", "cuda"])
def test_a_cleared_device_error_begins_with_new_workspaces(monkeypatch, device):
    """A wait that gave up leaves counters that would have later calls join too
    early: clearing the error lets every stream's kept workspace of that device go."""
    f = FakeCuda(monkeypatch)

    class Lib:
        def w4a8_clear_device_error(self, stream):
            return 0

    a, other = f.workspace(0), f.workspace(1)
    f.streams[0] = 101
    b = f.workspace(0)
    for ws in (a, b, other):
        ws[:64] = 1  # arrivals of a call that gave up
    with monkeypatch.context() as m:
        m.setattr(w4a8, "lib", Lib)
        m.setattr(w4a8, "_stream", lambda d: None)
        w4a8.clear_device_error(torch.device(device) if device == "cuda:0" else device)
    again = f.workspace(0)
    f.streams[0] = 100
    assert not again[:64].any() and not f.workspace(0)[:64].any()
    assert f.workspace(1) is other  # another device's is its own


@pytest.mark.parametrize("capturing", [False, True])
def test_no_more_than_the_counters_is_filled(monkeypatch, capturing):
    """A captured call fills its workspace at every replay: 1 KiB of it, not the
    megabytes of partial results behind."""
    f = FakeCuda(monkeypatch, 0, {0} if capturing else ())
    made = []

    def empty(n, **kw):
        made.append(torch.full((n,), 0x7F, **kw))
        return made[-1]

    def zeros(*a, **kw):
        raise AssertionError("the whole workspace is filled")
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", empty)
        m.setattr(torch, "zeros", zeros)
        ws = f.workspace(0, 1 << 16)
    n = w4a8.KV8_COUNTER_BYTES
    assert ws is made[0] and not ws[:n].any() and bool((ws[n:] == 0x7F).all())
