"""The binding loads on torch builds that lack the private names which its short path uses, and then takes the
public ones."""
import importlib.util
import types

import torch

from head_latent_attention_rmsnorm_gb300 import mla

PRIVATE = ("_cuda_getCurrentRawStream", "_cuda_getDevice")


def load():
    spec = importlib.util.spec_from_file_location("mla_again", mla.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_loads_without_private_torch_names(monkeypatch):
    for name in PRIVATE:
        monkeypatch.delattr(torch._C, name, raising=False)
    m = load()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: types.SimpleNamespace(cuda_stream=100 + index))
    assert m._current_device() == 3 and m._raw_stream(2) == 102
