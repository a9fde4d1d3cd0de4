"""Norms whose factor lies in the middle between two fp32 values: every variant gives
one of the two, and the int8 rows are those of the fp32 norm (GPU)."""
import math
import random

import pytest
import torch

import int4_weight_quantized_amd as w4

pytestmark = pytest.mark.gpu


def border(x):
    """(eps, the two neighbouring factors) of a row: 1 / sqrt(mean + eps) in the middle."""
    mean = math.fsum(float(v) ** 2 for v in x.tolist()) / x.numel()  # (squares are exact)
    low = torch.tensor(1 / math.sqrt(mean * (1 + 1e-6)), dtype=torch.float32)
    high = torch.nextafter(low, torch.tensor(math.inf))
    return 1 / ((float(low) + float(high)) / 2) ** 2 - mean, low, high


@pytest.mark.parametrize("K", [64, 512, 1000, 4096, 8192, 40000])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_factors_between_two_values(K, dt):
    rnd = random.Random(K)
    g = torch.Generator().manual_seed(K)
    w = 1 + 0.2 * torch.randn((K,), generator=g)
    for _ in range(12):
        x = (torch.randn((1, K), generator=g) * rnd.uniform(0.5, 3)).to(dt)
        eps, low, high = border(x[0])
        assert eps > 0
        either = [(x.float() * r) * w for r in (low, high)]
        wide = torch.empty(K + 1, dtype=dt, device="cuda")
        wide[1:] = x[0].cuda()
        for xc in (x.cuda(), wide[1:].view(1, K)):  # aligned to 16 bytes, and to an element
            y, _ = w4.rms_norm(xc, w.cuda(), eps, dtype=torch.float32)
            assert any(torch.equal(y.cpu(), e) for e in either)
            assert torch.equal(w4.rms_norm(xc, w.cuda(), eps, dtype=torch.bfloat16)[0], y.bfloat16())
            q, sx, _ = w4.a8_rms_norm(xc, w.cuda(), eps)
            q2, sx2 = w4.a8_quantize_act(y)
            assert torch.equal(q, q2) and torch.equal(sx, sx2)
