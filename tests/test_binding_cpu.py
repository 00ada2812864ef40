"""The binding on a torch without the private functions that it takes where they are."""
import importlib.util
import types

import torch

import token_dispatch_moe_b200 as moe


def test_device_and_stream_by_public_functions(monkeypatch):
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=100 + device))
    spec = importlib.util.spec_from_file_location("moe_on_another_torch", moe.__file__,
                                                  submodule_search_locations=[])
    other = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(other)
    assert other._current_device() == 3
    assert other._stream(None) == 103
    assert other._stream(17) == 17
