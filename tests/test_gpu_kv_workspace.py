"""One workspace, sized for the largest call, serves the smaller ones (GPU)."""
import pytest
import torch

from kv_cases import make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,heads,D", [(8, 2, 64), (32, 8, 128)])
def test_one_workspace(hq, heads, D):
    import int4_weight_quantized_amd as w4

    cache, table, tl, K, V = make_cache(w4, [3000, 40], heads, 16, D, "bf16", 110)
    ws = torch.empty(w4.kv_attention_workspace_bytes(4096, 2, hq, heads, D), dtype=torch.uint8, device="cuda")
    q = torch.randn((2048, hq, D), device="cuda")
    for n, m in ((1, 1), (36, 1), (100, 28), (255, 1), (700, 0), (1500, 40)):
        cu = torch.tensor([0, n, n + m], dtype=torch.int32, device="cuda")
        x = q[:n + m]
        a = w4.kv_prefill_attention(x, cache, 0, table, tl, cu, workspace=ws)
        assert torch.equal(a, w4.kv_prefill_attention(x, cache, 0, table, tl, cu))
    x = q[:2]
    a = w4.kv_decode_attention(x, cache, 0, table, tl, workspace=ws)
    assert torch.equal(a, w4.kv_decode_attention(x, cache, 0, table, tl))
