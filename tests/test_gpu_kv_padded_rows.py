"""Prompt attention of a call with more rows than its sequences have: rows
before the first offset and from the last one on belong to no sequence and are
left as they are, also where the rows' work is split and joined (GPU)."""
import math

import pytest
import torch

from kv_cases import attend, close, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import int4_weight_quantized_amd as pkg
    return pkg


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,heads,D", [(4, 2, 128), (3, 1, 16), (6, 2, 80), (5, 5, 64), (2, 1, 256)])
@pytest.mark.parametrize("cu,T,path", [([0, 6, 6, 11], 20, "kv_prefill_split"),
                                       ([3, 9, 14, 14], 20, "kv_prefill_split"),
                                       ([40, 41, 60, 70], 90, "kv_prefill_split")])
def test_rows_of_no_sequence(w4, cu, T, path, hq, heads, D, dt):
    lens = [200, 64, 37]
    cache, table, tl, K, V = make_cache(w4, lens, heads, 16, D, "bf16", 70)
    g = torch.Generator().manual_seed(71)
    x = torch.randn((T, hq, D), generator=g).to(dt).cuda()
    ws = torch.full((w4.kv_attention_workspace_bytes(T, 3, hq, heads, D) // 4,), math.nan, device="cuda")
    y = torch.full_like(x, 7.0)
    w4.kv_prefill_attention(x, cache, 0, table, tl, torch.tensor(cu, dtype=torch.int32).cuda(), out=y,
                            workspace=ws.view(torch.uint8))
    assert w4.w4_last_path() == path
    assert bool((y[:cu[0]] == 7.0).all()) and bool((y[cu[-1]:] == 7.0).all())
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        ok, worst = close(y[lo:hi], *attend(x[lo:hi], K[b], V[b], range(n - (hi - lo), n), 0, 0, D ** -0.5),
                          p_rounded=dt == torch.bfloat16)
        assert ok, (b, worst)


def test_padded_graph(w4):
    """A captured call of a fixed number of rows whose offsets change between replays."""
    T, hq, heads, D, lens = 24, 4, 2, 64, [150, 90]
    cache, table, tl, K, V = make_cache(w4, lens, heads, 16, D, "int8", 72)
    x = torch.randn((T, hq, D), generator=torch.Generator().manual_seed(73)).cuda()
    y = torch.empty_like(x)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    ws = torch.empty(w4.kv_attention_workspace_bytes(T, 2, hq, heads, D), dtype=torch.uint8, device="cuda")
    w4.kv_prefill_attention(x, cache, 0, table, tl, cu, out=y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.kv_prefill_attention(x, cache, 0, table, tl, cu, out=y, workspace=ws)
    for now in ([0, 24, 24], [0, 7, 19], [2, 3, 9], [0, 0, 1]):
        cu.copy_(torch.tensor(now, dtype=torch.int32))
        y.fill_(-3.0)
        g.replay()
        torch.cuda.synchronize()
        assert bool((y[:now[0]] == -3.0).all()) and bool((y[now[-1]:] == -3.0).all())
        for b, n in enumerate(lens):
            lo, hi = now[b], now[b + 1]
            ok, worst = close(y[lo:hi], *attend(x[lo:hi], K[b], V[b], range(n - (hi - lo), n), 0, 0,
                                                D ** -0.5))
            assert ok, (now, b, worst)
