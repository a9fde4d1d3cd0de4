"""The example runs the cache's operators together; every attention result in it
is checked against a plain 64-bit form of the cached values (GPU)."""
import os
import sys

import pytest
import torch

from kv_cases import attend, close

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_served_block(dtype, window, sinks):
    import decode_layer
    import int4_weight_quantized_amd as w4

    history = {}  # slot -> (K, V) as first cached, float64

    def values(b, slot, n):
        one = b.table[slot:slot + 1].contiguous()
        k, v = w4.kv_gather(b.cache, 0, one, decode_layer.ints(0), decode_layer.ints(0, n), n)
        return k.double().cpu(), v.double().cpu()

    def seen(b, what, q, o):
        lens = b.lens.tolist()
        rows = {5: (0, 37), 2: (37, 237)} if what == "prompts" else {
            s: (s, s + 1) for s in range(8) if lens[s] > 0}
        assert len(rows) in (2, 5, 3)
        for s, (lo, hi) in rows.items():
            n = lens[s]
            K, V = values(b, s, n)
            if s in history:  # what was cached stays, through forks and moves
                assert torch.equal(K[:n - 1], history[s][0]) and torch.equal(V[:n - 1], history[s][1])
            history[s] = (K, V)
            ok, worst = close(o[lo:hi], *attend(q[lo:hi], K, V, range(n - (hi - lo), n), window,
                                                sinks, 128 ** -0.5))
            assert ok, (what, s, worst)
        if what == "prompts":
            for child, parent in ((0, 5), (1, 5), (7, 2)):
                history[child] = history[parent]

    b = decode_layer.serve(20, dtype=dtype, window=window, sinks=sinks, seen=seen)
    assert b.lens.tolist() == [57, 57, 220, 0, 0, 0, 0, 0]
    held = sorted({p for row in b.table.tolist() for p in row if p >= 0})
    assert held == [p for p, r in enumerate(b.refs.tolist()) if r > 0]
    assert sum(b.refs.tolist()) == sum(p >= 0 for row in b.table.tolist() for p in row)


def test_slots_without_pages_left_wait():
    """A pool that runs out: slots that cannot be served keep their length."""
    import decode_layer

    b = decode_layer.Block(256, 4, 1, 64, slots=3, pages=4, pages_per_slot=4)
    x = torch.randn((48, 256), device="cuda")
    b.prompts(x, decode_layer.ints(0, 1, 2), decode_layer.ints(0, 16, 32, 48))
    assert b.lens.tolist() == [16, 16, 16]
    y, q, o = b.step(torch.randn((3, 256), device="cuda"))
    assert b.lens.tolist() == [17, 16, 16]
    assert bool(o[0].any()) and not bool(o[1:].any())
