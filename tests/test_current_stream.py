"""The stream and device that a call goes to are those torch names."""
import types

import pytest
import torch

import mixture_experts_fp32_b200 as moe

from test_binding_checks import FakeCuda


class OnDevice(FakeCuda):
    def __init__(self, index):
        super().__init__((4, 256))
        self.index = index
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.index


def test_default_stream_without_torchs_private_call(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=0x5150))
    assert moe._stream(None) == 0x5150
    assert moe._stream(77) == 77
    assert moe._stream(types.SimpleNamespace(cuda_stream=9)) == 9


@pytest.mark.gpu
def test_default_stream_is_torchs_current_one():
    assert moe._stream(None) == torch.cuda.current_stream().cuda_stream
    for st in (torch.cuda.Stream(), torch.cuda.Stream(priority=-1)):
        with torch.cuda.stream(st):
            assert moe._stream(None) == st.cuda_stream == torch.cuda.current_stream().cuda_stream
    assert moe._stream(None) == torch.cuda.default_stream().cuda_stream


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    moe._on_current_device((OnDevice(1), None))
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        moe._on_current_device((OnDevice(1), OnDevice(0)))
