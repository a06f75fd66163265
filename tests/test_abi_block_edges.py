"""Binding and entry points of the block operators off the usual paths (no GPU needed)."""
import types

import torch

from timestep_adaptive_bit_amd import _lib as L


def test_stream_handle_without_the_private_call(monkeypatch):
    """Where torch has no call for the handle, or the device names no index, the public one is asked."""
    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d: asked.append(d) or types.SimpleNamespace(cuda_stream=1234))
    monkeypatch.setattr(L, "_raw_stream", None)
    assert L._stream(torch.device("cuda", 1)) == 1234 and asked == [torch.device("cuda", 1)]
    monkeypatch.setattr(L, "_raw_stream", lambda index: 77 + index)
    assert L._stream(torch.device("cuda", 1)) == 78
    assert L._stream(torch.device("cuda")) == 1234
