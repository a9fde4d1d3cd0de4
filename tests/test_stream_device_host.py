"""Which stream a call of the cache's and the layer's operators goes to when its operands
are not on the current device (no GPU needed: torch's two queries are replaced)."""
import types

import pytest
import torch

from int4_weight_quantized_amd import kv, layer

ONE = torch.device("cuda:1")


@pytest.fixture
def current(monkeypatch):
    """Device 0 is current; each device's current stream is set by the test."""
    handles = {0: 0, 1: 0}
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: handles[i], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return handles


@pytest.mark.parametrize("stream", [None, 0, types.SimpleNamespace(cuda_stream=0)])
def test_the_default_stream_of_another_device_is_refused(current, stream):
    assert layer._stream is kv._stream
    with pytest.raises(ValueError, match="operands are on cuda:1"):
        kv._stream(stream, ONE)
    assert kv._stream(stream, torch.device("cuda:0")) == 0


def test_streams_with_a_handle_are_taken(current):
    current[1] = 0x1234
    assert kv._stream(None, ONE) == 0x1234
    assert kv._stream(0x55, ONE) == 0x55
    assert kv._stream(types.SimpleNamespace(cuda_stream=0x66), ONE) == 0x66
