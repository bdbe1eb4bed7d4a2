"""The binding finds the current device and stream with the public calls where torch lacks the quick ones."""
import types

import torch

from moe_layer_gemm_b200 import abi


def test_public_calls_where_the_quick_ones_are_missing(monkeypatch):
    monkeypatch.setattr(torch, "_C", types.SimpleNamespace())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(cuda_stream=1000 + dev))
    assert abi._stream(None) == 1003
    got = []
    abi._launch(lambda *args: got.append(args) or abi.MOE_OK, "f", 3, None, (1, 2))
    assert got == [(1, 2, 1003)]


def test_given_streams_are_taken_as_they_are():
    assert abi._stream(77) == 77 and abi._stream(types.SimpleNamespace(cuda_stream=78)) == 78
