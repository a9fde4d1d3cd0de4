"""The cache's rounding is one rule, whichever call writes a token: bytes and scales of
kv_append and kv_append_rope against the definition, over the range of fp32 (GPU)."""
import pytest
import torch

import int4_weight_quantized_amd as w4

pytestmark = pytest.mark.gpu


def rule(x):
    """(codes, scales) of vectors x [T, h, D] as the definition rounds them (fp32, on the CPU)."""
    s = x.abs().amax(-1) * torch.full((), 1.0, dtype=torch.float32).div(127)
    c = torch.round(x / s[..., None]).clamp(-128, 127)
    return torch.where(s[..., None] > 0, c, 0.0).to(torch.int8), s


@pytest.mark.parametrize("D", [16, 64, 80, 128, 160, 256])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_both_appends_write_the_same(D, dt):
    T, h = 300, 3
    g = torch.Generator().manual_seed(D)
    size = 2.0 ** torch.linspace(-149, 126, T).round()[:, None, None].double()
    x = (torch.rand((T, h, D), generator=g) * 2 - 1).double()
    x[:, :, 0] = 1.0  # the largest of the vector
    k, v = ((t * size).float().to(dt) for t in (x, -x))
    v[5] = 0.0
    k[7, :, 1:] = 0.0
    table = torch.arange((T + 15) // 16, dtype=torch.int32, device="cuda")[None]
    start, cu = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0], [0, T]))
    still = w4.Rope.of(torch.zeros(D // 2, dtype=torch.float64, device="cuda"))  # turns nothing
    for dtype in (torch.int8, torch.bfloat16):
        a, b = (w4.KVCache.empty(1, table.shape[1], h, 16, D, dtype) for _ in range(2))
        w4.kv_append(a, 0, k.cuda(), v.cuda(), table, start, cu)
        w4.kv_append_rope(b, 0, k.cuda(), k.cuda(), v.cuda(), table, start, still, cu)
        for c in (a, b):
            for pool, scales, t in ((c.k, c.k_scale, k), (c.v, c.v_scale, v)):
                got = pool[0].transpose(1, 2).flatten(0, 1)[:T].cpu()
                if dtype == torch.bfloat16:
                    assert torch.equal(got, t.to(torch.bfloat16))
                    continue
                codes, s = rule(t.float())
                assert torch.equal(scales[0].transpose(1, 2).flatten(0, 1)[:T].cpu(), s)
                assert torch.equal(got, codes)
