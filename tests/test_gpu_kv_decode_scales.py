"""int8 caches whose scales of V are far from one: the decode attention keeps its
accuracy (GPU)."""
import pytest
import torch

from kv_cases import attend, close
from test_gpu_kv_value_scales import CALLS, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import int4_weight_quantized_amd as pkg
    return pkg


@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,heads,D,pairs,path", CALLS)
@pytest.mark.parametrize("power", [-105, -79, -40, 60, 100])
@pytest.mark.parametrize("W", [0, 400])
def test_far_scales(w4, W, power, hq, heads, D, pairs, path, q):
    """Values times a power of two: outputs times the power of two, in a table of
    each width that chooses a kernel."""
    cache, table, tl, K, V, x, cu = setup(w4, heads, D, pairs, hq, q, 92)
    cache.v_scale.mul_(2.0 ** power)
    if W:
        table = torch.nn.functional.pad(table, (0, W - table.shape[1]), value=-1).contiguous()
    one = torch.stack([x[e - 1] for e in cu[1:]])
    y = w4.kv_decode_attention(one, cache, 0, table, tl)
    assert w4.w4_last_path() == ("kv_decode_split" if W else "kv_decode")
    y = (y.float() * 2.0 ** -power).to(y.dtype)
    for b, (n, m) in enumerate(pairs):
        assert close(y[b:b + 1], *attend(one[b:b + 1], K[b], V[b], [n - 1], 0, 0, D ** -0.5))[0]


@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [0, 400])
def test_one_far_part(w4, W, q):
    """Tiny scales in some of a row's parts, ordinary ones in the others: every part
    counts with its own weight."""
    hq, heads, D, pairs = 8, 2, 128, [(700, 1)]
    cache, table, tl, K, V, x, cu = setup(w4, heads, D, pairs, hq, q, 120)
    for lo, hi in ((0, 64), (256, 512)):
        pages = table[0, lo // 16:hi // 16].long()
        cache.v_scale[0, pages] *= 2.0 ** -90
        V[0][lo:hi] *= 2.0 ** -90
    if W:
        table = torch.nn.functional.pad(table, (0, W - table.shape[1]), value=-1).contiguous()
    y = w4.kv_decode_attention(x, cache, 0, table, tl)
    ok, worst = close(y, *attend(x, K[0], V[0], [699], 0, 0, D ** -0.5))
    assert ok, worst


@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [0, 400])
@pytest.mark.parametrize("power", [-105, -40, 89])
def test_zeros_before_far_scales(w4, power, W, q):
    """Scales of zero, and pages that are gone, in front of the far ones say nothing
    about them."""
    hq, heads, D, pairs = 8, 2, 128, [(700, 1)]
    cache, table, tl, K, V, x, cu = setup(w4, heads, D, pairs, hq, q, 122)
    cache.v_scale.mul_(2.0 ** power)
    hole = torch.zeros(700, dtype=torch.bool)
    for lo in range(0, 512, 128):
        pages = table[0, lo // 16:lo // 16 + 2].long()
        cache.v_scale[0, pages] = 0.0
        V[0][lo:lo + 32] = 0.0
        table[0, lo // 16 + 2:lo // 16 + 4] = -1
        hole[lo + 32:lo + 64] = True
    if W:
        table = torch.nn.functional.pad(table, (0, W - table.shape[1]), value=-1).contiguous()
    y = w4.kv_decode_attention(x, cache, 0, table, tl)
    y = (y.float() * 2.0 ** -power).to(y.dtype)
    ok, worst = close(y, *attend(x, K[0], V[0], [699], 0, 0, D ** -0.5, hole))
    assert ok, worst
