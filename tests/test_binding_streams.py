"""The binding asks torch for the current stream and device by its faster private calls where they exist and by
the public ones where they do not (a stand-in for torch: no GPU)."""
import types

import pytest
import torch

from bit_quantization_aware_blockwise_b200 import _binding as b

DEV = torch.device("cuda", 1)


def stand_in(private, current=1):
    asked = []

    def note(name, value):
        def call(*args):
            asked.append((name, *args))
            return value
        return call
    cuda = types.SimpleNamespace(current_stream=note("current_stream", types.SimpleNamespace(cuda_stream=77)),
                                 current_device=note("current_device", current),
                                 device=note("device", None), stream=note("stream", None))
    c = types.SimpleNamespace()
    if private:
        c._cuda_getCurrentRawStream = note("raw_stream", 77)
        c._cuda_getDevice = note("get_device", current)
    return types.SimpleNamespace(cuda=cuda, _C=c), asked


@pytest.mark.parametrize("private", [True, False])
def test_current_stream(monkeypatch, private):
    fake, asked = stand_in(private)
    monkeypatch.setattr(b, "_torch_module", fake)
    assert b._stream_handle(None, DEV) == 77
    assert asked == ([("raw_stream", 1)] if private else [("current_stream", DEV)])
    assert b._stream_handle(types.SimpleNamespace(cuda_stream=5), DEV) == 5
    assert len(asked) == 1                           # a stream that is given is not asked for


@pytest.mark.parametrize("private", [True, False])
def test_current_device(monkeypatch, private):
    fake, asked = stand_in(private)
    monkeypatch.setattr(b, "_torch_module", fake)
    assert b._at(DEV, None) is b._HERE_ALREADY
    assert asked == [("get_device",) if private else ("current_device",)]
    fake, asked = stand_in(private, current=0)
    monkeypatch.setattr(b, "_torch_module", fake)
    assert isinstance(b._at(DEV, None), b._on)
    assert asked[-1] == ("device", DEV)
    given = types.SimpleNamespace(device=DEV)
    assert isinstance(b._at(DEV, given), b._on) and asked[-1] == ("stream", given)
