"""The stream that a call without one is given, on the CPU with stand-ins for torch."""
import sys
import types

import pytest

import block_sparse_long_bsa_b200 as bsa


def _torch(initialized, available=True, **internal):
    cuda = types.SimpleNamespace(is_initialized=lambda: initialized, is_available=lambda: available,
                                 current_stream=lambda: types.SimpleNamespace(cuda_stream=71))
    return types.SimpleNamespace(cuda=cuda, _C=types.SimpleNamespace(**internal))


INTERNAL = dict(_cuda_getCurrentRawStream=lambda device: 50 + device, _cuda_getDevice=lambda: 3)


@pytest.mark.parametrize("torch,stream", [
    (_torch(True, **INTERNAL), 53),
    (_torch(True), 71),                                              # a torch without the internal names
    (_torch(True, _cuda_getDevice=INTERNAL["_cuda_getDevice"]), 71),
    (_torch(False, **INTERNAL), 71),
    (_torch(False, available=False), 0),
    (None, 0),                                                       # no torch at all
])
def test_the_current_stream(monkeypatch, torch, stream):
    monkeypatch.setattr(bsa, "_raw_stream", None)
    monkeypatch.setitem(sys.modules, "torch", torch)
    assert bsa._stream(None) == stream
    assert bsa._stream(None) == stream                               # and once it is known how to ask
    assert bsa._stream(9) == 9 and bsa._stream(types.SimpleNamespace(cuda_stream=12)) == 12
