"""Devices of the operators' tensors, as the binding checks them.  CPU only: the
tensors are stand-ins that know their device's number."""
import pytest

from ring_all_reduce_scatter_amd import _operators


class On:
    def __init__(self, index):
        self.index = index
        self.device = f"cuda:{index}" if index >= 0 else "cpu"

    def get_device(self):
        return self.index


def test_tensors_of_one_gpu():
    _operators._on_gpu(On(0), None, On(0))
    _operators._on_gpu(On(3), On(3))
    _operators._on_gpu(None)
    for ts in ((On(-1),), (On(0), On(-1)), (On(-1), On(0)), (None, On(-1))):
        with pytest.raises(ValueError, match="GPU tensor, got one on cpu"):
            _operators._on_gpu(*ts)
    for ts in ((On(0), On(1)), (On(1), None, On(1), On(0))):
        with pytest.raises(ValueError, match="on one device"):
            _operators._on_gpu(*ts)


def test_default_stream_of_another_device(monkeypatch):
    """A default stream is address 0 on every device, and a launch there goes to
    the current device."""
    streams = {0: 0, 1: 0, 2: 0x70}
    monkeypatch.setattr(_operators, "_current_stream", streams.__getitem__)
    monkeypatch.setattr(_operators, "_current_device", lambda: 0)
    assert _operators._stream(None, On(0)) == 0
    assert _operators._stream(None, On(2)) == 0x70  # an address names its device
    assert _operators._stream(0x30, On(1)) == 0x30
    with pytest.raises(ValueError, match="cuda:1 need it as the current device"):
        _operators._stream(None, On(1))
    monkeypatch.setattr(_operators, "_current_device", None)  # a process that sees one GPU
    assert _operators._stream(None, On(0)) == 0
