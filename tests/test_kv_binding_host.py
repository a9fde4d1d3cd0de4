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


class Calls:
    """Stands in for the library: keeps each call's arguments."""

    def __init__(self):
        self.seen = []

    def __call__(self):
        return self

    def __getattr__(self, name):
        return lambda *a: self.seen.append((name, a)) or 0


@pytest.mark.parametrize("stream", [None, 77])
def test_page_moves_use_workspaces_of_the_call_s_stream(monkeypatch, stream):
    """The lists of a fork or a compaction lie in memory of the stream that runs
    it, not in memory that ends with the cache object or belongs to another stream."""
    made = {}

    def empty(shape, dtype, dev, on):
        t = torch.empty(shape, dtype=dtype)
        made[t.data_ptr()] = on
        keep.append(t)
        return t

    keep, calls = [], Calls()
    monkeypatch.setattr(kv, "_empty", empty)
    monkeypatch.setattr(kv, "lib", calls)
    monkeypatch.setattr(kv, "_stream", lambda s, dev: 0 if s is None else s)
    c = object.__new__(w4.KVCache)
    c.device, c.pages, c._ref = torch.device("cpu"), 10, 0
    c._moves = torch.empty(1000, dtype=torch.uint8)
    w4.kv_fork(c, ints(3, 4), ints(3), ints(10), ints(2), ints(2), stream=stream)
    w4.kv_compact(c, ints(3, 4), ints(10), stream=stream)
    assert [n for n, _ in calls.seen] == ["kv_fork", "kv_compact"]
    for name, a in calls.seen:
        ws, size, on = a[-3:]
        assert on == (stream or 0)
        assert made[ws] == stream and size == 256 + (16 * 2 if name == "kv_fork" else 8 * 10)
