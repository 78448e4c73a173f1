"""The current device and stream without torch's private helpers (not gpu)."""

import importlib

import torch

from zero_sharded_mixed_flatparameter_gb300 import _current


def test_public_functions_stand_in(monkeypatch):
    with monkeypatch.context() as m:
        for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
            m.delattr(torch._C, name, raising=False)
        public = importlib.reload(_current)
        assert public.current_device is torch.cuda.current_device

        class Stream:
            cuda_stream = 77

        m.setattr(torch.cuda, "current_stream", lambda device: Stream if device == 3 else None)
        assert public.current_stream(3) == 77
    importlib.reload(_current)
