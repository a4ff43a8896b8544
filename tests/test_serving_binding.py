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

    def workspace(self, index, B=2, T=2, Hq=8, Hkv=2):
        return w4a8._kv8_workspace_for(self.q, index, B, T, Hq, Hkv)


def test_a_workspace_is_kept_for_each_stream(monkeypatch):
    f = FakeCuda(monkeypatch)
    a = f.workspace(0)
    assert f.workspace(0) is a and not a.any()
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
