"""What the key-value cache's binding hands to the library (no GPU needed: the
library is replaced)."""
import pytest
import torch

import int4_weight_quantized_amd as w4
from int4_weight_quantized_amd import kv


@pytest.fixture
def no_library(monkeypatch):
    def reached():
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(kv, "lib", reached)


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("stream", [None, 0])
def test_host_tensors_are_refused(no_library, stream):
    """Calls without a cache have no other operand that must be on a GPU."""
    table, lens, refs = ints(3, 4), ints(3), ints(10)
    with pytest.raises(ValueError, match="table must be a GPU tensor"):
        w4.kv_free(table, lens, refs, ints(2), stream=stream)
    with pytest.raises(ValueError, match="table must be a GPU tensor"):
        w4.kv_reserve(table, lens, refs, ints(3), 16, ok=ints(3),
                      workspace=torch.zeros(300, dtype=torch.uint8), stream=stream)


@pytest.mark.parametrize("bad", [None, 3, [1, 2]])
def test_what_is_no_tensor_is_named(no_library, bad):
    with pytest.raises((TypeError, ValueError), match="table must be"):
        w4.kv_free(bad, ints(3), ints(10), ints(2))
    with pytest.raises((TypeError, ValueError), match="table must be"):
        w4.kv_reserve(bad, ints(3), ints(10), ints(3), 16)
    c = object.__new__(w4.KVCache)
    c.device = torch.device("cuda:0")
    with pytest.raises(TypeError, match="dst_ids must be a tensor"):
        w4.kv_copy_pages(c, bad, c, bad)
    with pytest.raises(TypeError, match="refs must be a tensor"):
        kv._count(bad, "refs")
    with pytest.raises(TypeError, match="workspace must be a tensor"):
        kv._work(bad if bad is not None else 0, 16, c.device, None)
