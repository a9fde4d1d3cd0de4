"""int8 caches whose scales of V are far from one, zero, infinite or NaN: the
prompt attention takes a visible token's value as code * scale, as the decode
attention and the gather do, and lets nothing of a hidden one in (GPU)."""
import math

import pytest
import torch

from kv_cases import attend, close, make_cache

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
# the split path and the unsplit one (many cache heads)
CALLS = [(4, 2, 64, [(150, 9), (70, 70)], "kv_prefill_split"), (6, 2, 128, [(700, 40)], "kv_prefill_split"),
         (130, 130, 32, [(150, 150)], "kv_prefill"), (3, 1, 256, [(90, 90)], "kv_prefill_split")]


@pytest.fixture(scope="module")
def w4():
    import int4_weight_quantized_amd as pkg
    return pkg


def setup(w4, heads, D, pairs, hq, q, seed):
    cache, table, tl, K, V = make_cache(w4, [n for n, _ in pairs], heads, 16, D, "int8", seed)
    cu = [0]
    for _, m in pairs:
        cu.append(cu[-1] + m)
    g = torch.Generator().manual_seed(seed + 1)
    x = torch.randn((cu[-1], hq, D), generator=g).to(DT[q]).cuda()
    return cache, table, tl, K, V, x, cu


def place(table, b, t):
    return int(table[b, t // 16]), t % 16


def check(y, x, K, V, pairs, cu, q, window=0, sinks=0, only=lambda b, p: True):
    for b, (n, m) in enumerate(pairs):
        s = slice(cu[b], cu[b + 1])
        out, rel, mean = attend(x[s], K[b], V[b], range(n - m, n), window, sinks, x.shape[2] ** -0.5)
        rows = [i for i in range(m) if only(b, n - m + i)]
        ok, worst = close(y[s][rows], out[rows], rel[rows], mean[rows], p_rounded=q == "bf16")
        assert ok, (b, worst)


@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,heads,D,pairs,path", CALLS)
@pytest.mark.parametrize("value", [-math.inf, math.inf, math.nan, -3e38, 1e-42])
def test_hidden_scales(w4, value, hq, heads, D, pairs, path, q):
    """Whatever stands in the scales of slots without a token, behind the window
    and after a row."""
    cache, table, tl, K, V, x, cu = setup(w4, heads, D, pairs, hq, q, 90)
    for b, (n, m) in enumerate(pairs):
        for t in range(n, -(-n // 16) * 16):
            page, slot = place(table, b, t)
            cache.k_scale[0, page, :, slot] = cache.v_scale[0, page, :, slot] = value
    n, m = pairs[0]
    hidden = [t for t in (n - m // 2, n - m - 40) if t >= 0]  # later than some rows; behind every window
    for t in hidden:
        page, slot = place(table, 0, t)
        cache.k_scale[0, page, :, slot] = cache.v_scale[0, page, :, slot] = value
        K[0][t] = V[0][t] = 0
    y = w4.kv_prefill_attention(x, cache, 0, table, tl, torch.tensor(cu, dtype=torch.int32).cuda(),
                                window=32, sinks=2)
    assert w4.w4_last_path() == path
    check(y, x, K, V, pairs, cu, q, 32, 2,
          lambda b, p: b > 0 or not any(t <= p < t + 32 for t in hidden))


@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,heads,D,pairs,path", CALLS)
@pytest.mark.parametrize("power", [-105, -79, -40, 60, 100])
def test_far_scales(w4, power, hq, heads, D, pairs, path, q):
    """Values times a power of two: outputs times the power of two."""
    cache, table, tl, K, V, x, cu = setup(w4, heads, D, pairs, hq, q, 92)
    cache.v_scale.mul_(2.0 ** power)
    tcu = torch.tensor(cu, dtype=torch.int32).cuda()
    y = w4.kv_prefill_attention(x, cache, 0, table, tl, tcu)
    assert w4.w4_last_path() == path
    check((y.float() * 2.0 ** -power).to(y.dtype), x, K, V, pairs, cu, q)


@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,heads,D,pairs,path", CALLS)
@pytest.mark.parametrize("power", [-200, -110, 30])
def test_mixed_scales(w4, power, hq, heads, D, pairs, path, q):
    """Some visible tokens with a scale of zero, others times a power of two
    (-200: zero, too), the rest ordinary."""
    cache, table, tl, K, V, x, cu = setup(w4, heads, D, pairs, hq, q, 94)
    f = torch.tensor(2.0 ** power, dtype=torch.float32)
    for b, (n, m) in enumerate(pairs):
        for t in range(0, n, 3):
            page, slot = place(table, b, t)
            cache.v_scale[0, page, :, slot] *= float(f) if t % 2 else 0.0
            V[b][t] *= float(f) if t % 2 else 0.0
    y = w4.kv_prefill_attention(x, cache, 0, table, tl, torch.tensor(cu, dtype=torch.int32).cuda())
    assert w4.w4_last_path() == path
    check(y, x, K, V, pairs, cu, q)


@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,heads,D,pairs,path", CALLS)
def test_all_zero(w4, hq, heads, D, pairs, path, q):
    cache, table, tl, K, V, x, cu = setup(w4, heads, D, pairs, hq, q, 96)
    cache.v_scale.mul_(0.0).nan_to_num_(0.0)
    y = w4.kv_prefill_attention(x, cache, 0, table, tl, torch.tensor(cu, dtype=torch.int32).cuda())
    assert w4.w4_last_path() == path and not bool(y.any())


@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,heads,D,pairs,path", CALLS)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_visible_scales(w4, value, hq, heads, D, pairs, path, q):
    """A row that sees a scale that is not finite has no finite output; the
    other rows hold the bound."""
    cache, table, tl, K, V, x, cu = setup(w4, heads, D, pairs, hq, q, 98)
    n, m = pairs[-1]
    at = n - m // 2
    page, slot = place(table, len(pairs) - 1, at)
    cache.v_scale[0, page, :, slot] = value
    V[-1][at] = 0
    y = w4.kv_prefill_attention(x, cache, 0, table, tl, torch.tensor(cu, dtype=torch.int32).cuda())
    assert w4.w4_last_path() == path
    check(y, x, K, V, pairs, cu, q, only=lambda b, p: b + 1 < len(pairs) or p < at)
    seen = y[cu[-1] - (n - at):]
    assert not bool(seen.isfinite().any())
    one = w4.kv_decode_attention(x[-1:], cache, 0, table[-1:].contiguous(), tl[-1:])
    assert not bool(one.isfinite().any())
