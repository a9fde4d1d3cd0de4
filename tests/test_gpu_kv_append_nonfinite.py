"""Appending values that are not finite: an int8 cache keeps no finite number
in their place (GPU)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
INV127 = torch.tensor(1.0 / 127.0, dtype=torch.float32)


@pytest.fixture(scope="module")
def w4():
    import int4_weight_quantized_amd as pkg
    return pkg


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


BAD = [math.nan, math.inf, -math.inf]


def rows(D, dt):
    """[12, 2, D]: in rows 3 .. 11 head 1 holds one value, a few or only such values."""
    x = torch.randn((12, 2, D), generator=torch.Generator().manual_seed(80)).to(dt)
    for i, v in enumerate(BAD):
        x[3 + i, 1, D - 1 - i] = v
        x[6 + i, 1, i::5] = v
        x[9 + i, 1] = v
    x[7, 1, 2] = -math.inf  # beside +inf
    return x


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [16, 80, 128, 256])
def test_append_int8(w4, D, dt):
    x = rows(D, dt)
    c = w4.KVCache.empty(1, 3, 2, 16, D, torch.int8)
    w4.kv_append(c, 0, x.cuda(), x.flip(0).cuda(), ints([[1]]), ints([2]), ints([0, 12]))
    for codes, scales, src in ((c.k, c.k_scale, x), (c.v, c.v_scale, x.flip(0))):
        f = src.float()
        fine = f.isfinite().all(-1)
        s = scales[0, 1, :, 2:14].T.cpu()
        assert bool(s[~fine].isnan().all()) and int((~fine).sum()) == 9
        assert torch.equal(s[fine], (f.abs().amax(-1) * INV127)[fine])
        got = codes[0, 1, :, 2:14].transpose(0, 1).cpu()
        assert torch.equal(got[fine], torch.round(f[fine] / s[fine][:, None]).to(torch.int8))
    k, v = w4.kv_gather(c, 0, ints([[1]]), ints([2]), ints([0, 12]), 12)
    assert torch.equal(k.isnan().cpu(), (~x.float().isfinite().all(-1))[..., None].expand(12, 2, D))
    o = w4.kv_decode_attention(torch.ones((1, 2, D), device="cuda"), c, 0, ints([[1]]), ints([14]),
                               window=12)
    assert bool(o[0, 1].isnan().all()) and bool(o[0, 0].isfinite().all())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_append_bf16(w4, dt):
    x = rows(128, dt)
    c = w4.KVCache.empty(1, 3, 2, 16, 128)
    w4.kv_append(c, 0, x.cuda(), x.cuda(), ints([[1]]), ints([2]), ints([0, 12]))
    got = c.k[0, 1, :, 2:14].transpose(0, 1).cpu()
    assert torch.equal(got.isnan(), x.isnan())
    assert torch.equal(got[~x.isnan()], x[~x.isnan()].bfloat16())


def test_largest_values(w4):
    """The largest finite values are no infinities."""
    big = torch.finfo(torch.float32).max
    x = torch.full((1, 1, 64), 1.0)
    x[0, 0, 5] = -big
    c = w4.KVCache.empty(1, 1, 1, 16, 64, torch.int8)
    w4.kv_append(c, 0, x.cuda(), x.cuda(), ints([[0]]), ints([0]))
    assert float(c.k_scale[0, 0, 0, 0]) == float(torch.tensor(big) * INV127)
    assert int(c.k[0, 0, 0, 0, 5]) == -127 and int(c.k[0, 0, 0, 0].abs().sum()) == 127
