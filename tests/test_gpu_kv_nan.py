"""A NaN that a query row holds or sees comes out as NaN, whatever way its work
was split over waves and workgroups and joined (GPU)."""
import math

import pytest
import torch

from kv_cases import attend, close, make_cache

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SHAPES = [(8, 2, 128, "bf16", "fp32"), (12, 1, 64, "int8", "bf16"), (4, 4, 80, "int8", "fp32"),
          (16, 1, 256, "bf16", "bf16"), (20, 1, 128, "bf16", "fp32")]


@pytest.fixture(scope="module")
def w4():
    import int4_weight_quantized_amd as pkg
    return pkg


def queries(n, hq, D, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.3 * torch.randn((n, hq, D), generator=g)).to(DT[dt]).cuda()


def spoil_keys(cache, table, b, lo, hi):
    """NaN in the keys of sequence b's tokens lo .. hi - 1 (whole pages)."""
    ps = cache.page_size
    pages = table[b, lo // ps:hi // ps].long()
    (cache.k_scale if cache.int8 else cache.k)[0, pages] = math.nan


@pytest.mark.parametrize("hq,heads,D,kv,q", SHAPES)
@pytest.mark.parametrize("path,lens,W", [("kv_decode", [700, 5], 60), ("kv_decode_split", [700, 5], 400),
                                         ("kv_decode_split", [9000, 40], 600)])
def test_decode_nan_query(w4, path, lens, W, hq, heads, D, kv, q):
    cache, table, tl, K, V = make_cache(w4, lens, heads, 16, D, kv, 50, W=W)
    x = queries(2, hq, D, q, 51)
    want = w4.kv_decode_attention(x, cache, 0, table, tl)
    bad = [(0, 1), (1, hq - 1)]
    for i, (b, h) in enumerate(bad):
        x[b, h, i:: 1 + i * (D - 1)] = math.nan  # the whole row, then one value of one
    y = w4.kv_decode_attention(x, cache, 0, table, tl)
    assert w4.w4_last_path() == path
    for b, h in bad:
        assert bool(y[b, h].isnan().all())
        y[b, h] = want[b, h]
    assert torch.equal(y, want)


@pytest.mark.parametrize("hq,heads,D,kv,q", SHAPES)
@pytest.mark.parametrize("path,lens,W", [("kv_decode", [700, 300], 60), ("kv_decode_split", [700, 300], 400),
                                         ("kv_decode_split", [9000, 300], 600)])
def test_decode_nan_keys(w4, path, lens, W, hq, heads, D, kv, q):
    """NaN in every key of a stretch longer than any one wave's or workgroup's
    part, with finite keys in the other parts."""
    cache, table, tl, K, V = make_cache(w4, lens, heads, 16, D, kv, 52, W=W)
    x = queries(2, hq, D, q, 53)
    want = w4.kv_decode_attention(x, cache, 0, table, tl)
    spoil_keys(cache, table, 0, 256, 512)
    y = w4.kv_decode_attention(x, cache, 0, table, tl)
    assert w4.w4_last_path() == path
    assert bool(y[0].isnan().all())
    assert torch.equal(y[1], want[1])


def check_prefill(w4, cache, table, tl, K, V, pairs, x, path, bad):
    """bad: (row, head) pairs whose outputs must be NaN; the others hold the bound."""
    cu = [0]
    for _, m in pairs:
        cu.append(cu[-1] + m)
    y = w4.kv_prefill_attention(x, cache, 0, table, tl, torch.tensor(cu, dtype=torch.int32).cuda())
    assert w4.w4_last_path() == path
    D = x.shape[2]
    for b, (n, m) in enumerate(pairs):
        lo, hi = cu[b], cu[b + 1]
        out, rel, mean = attend(x[lo:hi].nan_to_num(0.0), K[b], V[b], range(n - m, n), 0, 0, D ** -0.5)
        for r, h in bad:
            if lo <= r < hi:
                assert bool(y[r, h].isnan().all()), (r, h)
                y[r, h] = out[r - lo, h].to(y.dtype)
        ok, worst = close(y[lo:hi], out, rel, mean, p_rounded=x.dtype == torch.bfloat16)
        assert ok, (b, worst)


@pytest.mark.parametrize("hq,heads,D,kv,q", SHAPES)
def test_prefill_split_nan_query(w4, hq, heads, D, kv, q):
    pairs = [(700, 3), (90, 5)]
    data = make_cache(w4, [n for n, _ in pairs], heads, 16, D, kv, 54)
    x = queries(8, hq, D, q, 55)
    x[1, hq - 1] = math.nan
    x[6, 0, 3] = math.nan
    check_prefill(w4, *data, pairs, x, "kv_prefill_split", [(1, hq - 1), (6, 0)])


@pytest.mark.parametrize("hq,heads,D,kv,q", SHAPES)
def test_prefill_nan_query(w4, hq, heads, D, kv, q):
    pairs = [(19, 2)] * 300
    data = make_cache(w4, [19] * 300, heads, 16, D, kv, 56)
    x = queries(600, hq, D, q, 57)
    x[1, hq - 1] = math.nan
    x[6, 0, 3] = math.nan
    check_prefill(w4, *data, pairs, x, "kv_prefill", [(1, hq - 1), (6, 0)])


@pytest.mark.parametrize("hq,heads,D,kv,q", SHAPES)
def test_prefill_split_nan_keys(w4, hq, heads, D, kv, q):
    """NaN in every key of two of sixteen parts of one tile each: the rows that see
    them are NaN (all of sequence 0's), the other sequence's are not touched."""
    pairs = [(1024, 3), (90, 5)]
    cache, table, tl, K, V = make_cache(w4, [n for n, _ in pairs], heads, 16, D, kv, 58)
    x = queries(8, hq, D, q, 59)
    spoil_keys(cache, table, 0, 64, 192)
    check_prefill(w4, cache, table, tl, K, V, pairs, x, "kv_prefill_split",
                  [(r, h) for r in range(3) for h in range(hq)])


@pytest.mark.parametrize("hq,heads,D,kv,q", [(130, 130, 32, "bf16", "fp32"), (130, 130, 64, "int8", "bf16")])
def test_prefill_nan_keys(w4, hq, heads, D, kv, q):
    """Keys of tokens 64 .. 191: rows before them do not see them."""
    pairs = [(300, 300)]
    cache, table, tl, K, V = make_cache(w4, [300], heads, 16, D, kv, 60)
    x = queries(300, hq, D, q, 61)
    spoil_keys(cache, table, 0, 64, 192)
    check_prefill(w4, cache, table, tl, K, V, pairs, x, "kv_prefill",
                  [(r, h) for r in range(64, 300) for h in range(hq)])
