"""The served block's adapters through forks that are and are not granted, and
through retirement (GPU)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def block(adapters):
    import decode_layer

    b = decode_layer.Block(256, 4, 1, 64, slots=5, pages=40, pages_per_slot=8, adapters=adapters)
    if adapters:
        b.adapter.copy_(torch.tensor([2, -1, 0, -1, 1], dtype=torch.int32))
    g = torch.Generator(device="cuda").manual_seed(1)
    b.prompts(torch.randn((50, 256), generator=g, device="cuda"), decode_layer.ints(0, 2), decode_layer.ints(0, 20, 50))
    return decode_layer, b


def test_forks_that_are_not_granted_change_no_adapter():
    """A running child, a child named by an earlier fork, and slots outside the table."""
    ex, b = block(3)
    ok = b.fork(ex.ints(2, 0, 2, 0, 5, 2), ex.ints(1, 1, 0, -1, 3, 5))
    assert ok.tolist() == [1, 0, 0, 0, 0, 0]
    assert b.lens.tolist() == [20, 30, 30, 0, 0]
    assert b.adapter.tolist() == [2, 0, 0, -1, 1]
    b.free(ex.ints(2, 2, -1, 5))
    assert b.lens.tolist() == [20, 30, 0, 0, 0]
    assert b.adapter.tolist() == [2, 0, -1, -1, 1]


def test_a_block_without_adapters_forks_as_the_cache_does():
    ex, b = block(0)
    assert b.fork(ex.ints(2, 0, 7), ex.ints(3, -1, 4)).tolist() == [1, 0, 0]
    assert b.lens.tolist() == [20, 0, 30, 30, 0] and b.adapter.tolist() == [-1] * 5


def test_a_padded_batch_of_prompts():
    """Rows of no sequence in front of the prompts and behind them: the prompts have
    their own adapters, as without the padding."""
    import int4_weight_quantized_amd as w4

    ex, b = block(3)
    _, c = block(3)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((40, 256), generator=g, device="cuda")
    seen = []
    project = b.project

    def looked(x, adapter=None):
        seen.append(adapter.tolist())
        return project(x, adapter)
    b.project = looked
    for one in (b, c):
        one.adapter[1], one.adapter[3] = 2, 1
    _, q, o = b.prompts(x, ex.ints(3, 1), ex.ints(3, 14, 31))
    _, r, p = c.prompts(x[3:31].contiguous(), ex.ints(3, 1), ex.ints(0, 11, 28))
    assert seen == [[-1] * 3 + [1] * 11 + [2] * 17 + [-1] * 9]
    assert torch.equal(q[3:31], r) and torch.equal(o[3:31], p)
    for s, n in ((3, 11), (1, 17)):
        got, want = (w4.kv_gather(t.cache, 0, t.table[s:s + 1].contiguous(), ex.ints(0), ex.ints(0, n), n) for t in (b, c))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
