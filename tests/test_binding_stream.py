"""Which stream the binding passes when the caller names none (no GPU: torch is
a stand-in)."""

import sys
from types import SimpleNamespace

import pytest

from split_backward_gemms_gb300 import build as B


@pytest.fixture(scope="module")
def zb():
    B.build()
    from split_backward_gemms_gb300 import zb as _zb
    return _zb


def stand_in(handle, initialized=True, private=True):
    torch = SimpleNamespace(cuda=SimpleNamespace(
        is_initialized=lambda: initialized,
        current_stream=lambda: SimpleNamespace(cuda_stream=handle)))
    if private:
        torch._C = SimpleNamespace(_cuda_getDevice=lambda: 3, _cuda_getCurrentRawStream=lambda d: handle + d)
    return torch


def test_raw_handle_of_the_current_device(zb, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", stand_in(4096))
    assert zb._stream(None) == 4099


def test_public_call_where_torch_lacks_the_private_ones(zb, monkeypatch):
    torch = stand_in(4096, private=False)
    monkeypatch.setitem(sys.modules, "torch", torch)
    assert zb._stream(None) == 4096
    torch._C = SimpleNamespace()
    assert zb._stream(None) == 4096


@pytest.mark.parametrize("torch", [None, SimpleNamespace(), stand_in(4096, initialized=False)])
def test_default_stream_without_cuda(zb, monkeypatch, torch):
    monkeypatch.setitem(sys.modules, "torch", torch)
    assert zb._stream(None) is None


def test_default_stream_has_no_handle(zb, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", stand_in(0, private=False))
    assert zb._stream(None) is None
