"""Attention over the paged cache against a plain 64-bit form (GPU).

Lengths around every tile and page edge, zero and one; heads that share a
cache head; sliding windows, sinks, pages that are gone; NaN in every place
that holds no visible token.
"""
import math

import pytest
import torch

from kv_cases import attend, close, make_cache

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def w4():
    import int4_weight_quantized_amd as pkg
    return pkg


def make_q(shape, dt, seed):
    g = torch.Generator().manual_seed(seed + 1)
    return (1.3 * torch.randn(shape, generator=g)).to(DT[dt]).cuda()


def check_decode(w4, lens, hq, heads, D, ps, kv, q, window=0, sinks=0, scale=None, seed=0, W=None):
    cache, table, tl, K, V = make_cache(w4, lens, heads, ps, D, kv, seed, W=W)
    x = make_q((len(lens), hq, D), q, seed)
    y = w4.kv_decode_attention(x, cache, 0, table, tl, scale=scale, window=window, sinks=sinks)
    again = w4.kv_decode_attention(x, cache, 0, table, tl, scale=scale, window=window, sinks=sinks)
    assert torch.equal(y, again)
    sc = 1 / math.sqrt(D) if scale is None else scale
    for b, n in enumerate(lens):
        ok, worst = close(y[b:b + 1], *attend(x[b:b + 1], K[b], V[b], [n - 1], window, sinks, sc))
        assert ok, (b, n, worst)
        if n == 0:
            assert not y[b].any()


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 511, 777]


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,heads,D,ps", [(8, 2, 128, 16), (4, 1, 256, 32), (6, 6, 64, 64),
                                           (21, 3, 80, 16), (32, 1, 96, 128), (17, 1, 16, 16),
                                           (5, 5, 240, 256), (40, 2, 128, 64)])
def test_decode_edges(w4, hq, heads, D, ps, q, kv):
    check_decode(w4, EDGES, hq, heads, D, ps, kv, q)


@pytest.mark.parametrize("kv,q", [("bf16", "fp32"), ("int8", "bf16")])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 17), (100, 0), (128, 64),
                                          (500, 600), (4096, 4)])
def test_decode_window(w4, window, sinks, q, kv):
    check_decode(w4, EDGES + [1500], 8, 2, 128, 16, kv, q, window=window, sinks=sinks, seed=3)


@pytest.mark.parametrize("lens", [[1], [700], [5000], [1, 20000], [3000] * 3 + [0] + [17] * 40,
                                  [9001, 2, 64, 1024]])
@pytest.mark.parametrize("hq,heads,D,kv,q", [(8, 2, 128, "bf16", "fp32"), (4, 4, 64, "int8", "fp32"),
                                             (16, 1, 256, "bf16", "bf16")])
def test_decode_split(w4, lens, hq, heads, D, kv, q):
    """Long and ragged lengths: work that is split over the length and joined."""
    check_decode(w4, lens, hq, heads, D, 32, kv, q, seed=5)


def test_decode_wide_table(w4):
    """A table much wider than any length (the host knows only its width)."""
    check_decode(w4, [1, 300, 0, 65], 8, 2, 128, 16, "bf16", "fp32", seed=6, W=4000)


def test_decode_scale(w4):
    check_decode(w4, [40, 333], 4, 2, 64, 16, "bf16", "fp32", scale=0.5, seed=7)
    check_decode(w4, [40, 333], 4, 2, 64, 16, "bf16", "fp32", scale=-0.2, seed=7)
    check_decode(w4, [40, 333], 4, 2, 64, 16, "int8", "fp32", scale=0.0, seed=7)


def test_decode_large_scores(w4):
    """Scores of thousands: the running maximum keeps the exponentials finite."""
    check_decode(w4, [70, 600, 2000], 4, 2, 128, 16, "bf16", "fp32", scale=30.0, seed=8)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_decode_pages_gone(w4, kv):
    """Tokens whose table entry is no page (-1, or out of range) are left out;
    pages behind a window may be gone, with whatever their place held."""
    lens, ps = [200, 64, 333], 16
    cache, table, tl, K, V = make_cache(w4, lens, 2, ps, 128, kv, 9)
    t = table.cpu()
    t[0, 3] = -1
    t[0, 5] = cache.pages
    t[1, :4] = -7
    t[2, 0] = 2 ** 31 - 1
    t[2, 10] = -2 ** 31
    hole = [torch.zeros(n, dtype=torch.bool) for n in lens]
    for b, n in enumerate(lens):
        for j in range(-(-n // ps)):
            if not 0 <= int(t[b, j]) < cache.pages:
                hole[b][j * ps:(j + 1) * ps] = True
    x = make_q((3, 8, 128), "fp32", 9)
    y = w4.kv_decode_attention(x, cache, 0, t.cuda(), tl)
    for b in range(3):
        ok, worst = close(y[b:b + 1], *attend(x[b:b + 1], K[b], V[b], [lens[b] - 1], 0, 0,
                                              128 ** -0.5, hole[b]))
        assert ok, (b, worst)
    assert not y[1].any()


def test_decode_lengths_out_of_range(w4):
    """A negative length is 0, one beyond the table's row is the row's."""
    cache, table, tl, K, V = make_cache(w4, [64, 64], 2, 16, 64, "bf16", 10, W=4)
    x = make_q((2, 4, 64), "fp32", 10)
    lens = torch.tensor([-5, 2 ** 31 - 1], dtype=torch.int32).cuda()
    y = w4.kv_decode_attention(x, cache, 0, table, lens)
    assert not y[0].any()
    ok, worst = close(y[1:], *attend(x[1:], K[1], V[1], [63], 0, 0, 0.125))
    assert ok, worst


def test_decode_hidden_infinities(w4):
    """Infinities and NaN outside the window, in K and V, reach nothing."""
    lens, window, sinks = [300], 50, 5
    cache, table, tl, K, V = make_cache(w4, lens, 2, 16, 64, "bf16", 11)
    x = make_q((1, 4, 64), "fp32", 11)
    for t in list(range(sinks, 300 - window)):
        page, slot = int(table[0, t // 16]), t % 16
        cache.k[0, page, :, slot] = math.inf if t % 2 else math.nan
        cache.v[0, page, :, slot] = -math.inf if t % 3 else math.nan
    y = w4.kv_decode_attention(x, cache, 0, table, tl, window=window, sinks=sinks)
    K[0][sinks:300 - window] = 0
    V[0][sinks:300 - window] = 0
    ok, worst = close(y, *attend(x, K[0], V[0], [299], window, sinks, 0.125))
    assert ok, worst


def test_decode_strided_queries(w4):
    """Query rows inside a joint projection's output."""
    lens = [100, 37, 260]
    cache, table, tl, K, V = make_cache(w4, lens, 2, 16, 128, "bf16", 12)
    joint = make_q((3, 12, 128), "fp32", 12)
    y = w4.kv_decode_attention(joint[:, 2:10], cache, 0, table, tl)
    assert torch.equal(y, w4.kv_decode_attention(joint[:, 2:10].contiguous(), cache, 0, table, tl))


def test_decode_layers(w4):
    cache, table, tl, K, V = make_cache(w4, [77, 130], 2, 16, 64, "int8", 13, layers=3)
    x = make_q((2, 6, 64), "fp32", 13)
    y = w4.kv_decode_attention(x, cache, 2, table, tl)
    for b, n in enumerate([77, 130]):
        assert close(y[b:b + 1], *attend(x[b:b + 1], K[b], V[b], [n - 1], 0, 0, 0.125))[0]


def test_large_pool(w4):
    """A pool whose offsets pass 32 bits (in values and in bytes)."""
    lens = [700, 90]
    cache, table, tl, K, V = make_cache(w4, lens, 8, 64, 128, "bf16", 14, pages=40000)
    assert cache.k.numel() > 2 ** 31
    x = make_q((2, 16, 128), "fp32", 14)
    y = w4.kv_decode_attention(x, cache, 0, table, tl)
    cu = torch.tensor([0, 9, 12], dtype=torch.int32).cuda()
    xp = make_q((12, 16, 128), "fp32", 15)
    yp = w4.kv_prefill_attention(xp, cache, 0, table, tl, cu)
    for b, n in enumerate(lens):
        ok, worst = close(y[b:b + 1], *attend(x[b:b + 1], K[b], V[b], [n - 1], 0, 0, 128 ** -0.5))
        assert ok, worst
        lo, hi = int(cu[b]), int(cu[b + 1])
        ok, worst = close(yp[lo:hi], *attend(xp[lo:hi], K[b], V[b], range(n - (hi - lo), n), 0, 0,
                                             128 ** -0.5))
        assert ok, worst


# ------------------------------------------------------------------- prompts
def check_prefill(w4, pairs, hq, heads, D, ps, kv, q, window=0, sinks=0, seed=0, scale=None):
    """pairs: (cached tokens, new ones) of each sequence."""
    lens = [n for n, _ in pairs]
    cache, table, tl, K, V = make_cache(w4, lens, heads, ps, D, kv, seed)
    cu = [0]
    for _, m in pairs:
        cu.append(cu[-1] + m)
    x = make_q((cu[-1], hq, D), q, seed)
    tcu = torch.tensor(cu, dtype=torch.int32).cuda()
    y = w4.kv_prefill_attention(x, cache, 0, table, tl, tcu, window=window, sinks=sinks, scale=scale)
    again = w4.kv_prefill_attention(x, cache, 0, table, tl, tcu, window=window, sinks=sinks,
                                    scale=scale)
    assert torch.equal(y, again)
    sc = 1 / math.sqrt(D) if scale is None else scale
    for b, (n, m) in enumerate(pairs):
        s = slice(cu[b], cu[b + 1])
        ok, worst = close(y[s], *attend(x[s], K[b], V[b], range(n - m, n), window, sinks, sc),
                          p_rounded=q == "bf16")
        assert ok, (b, n, m, worst)


RAGGED = [(1, 1), (17, 17), (64, 64), (65, 1), (130, 129), (200, 3), (0, 0), (96, 33), (31, 31),
          (513, 70)]


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,heads,D,ps", [(8, 2, 128, 16), (4, 1, 256, 32), (6, 6, 64, 64),
                                           (21, 3, 80, 16), (32, 1, 96, 128), (3, 3, 16, 16),
                                           (5, 5, 240, 256)])
def test_prefill_ragged(w4, hq, heads, D, ps, q, kv):
    check_prefill(w4, RAGGED, hq, heads, D, ps, kv, q)


@pytest.mark.parametrize("kv,q", [("bf16", "fp32"), ("int8", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 17), (100, 0), (128, 64),
                                          (500, 600), (4096, 4)])
def test_prefill_window(w4, window, sinks, q, kv):
    check_prefill(w4, RAGGED + [(700, 700)], 4, 2, 128, 16, kv, q, window=window, sinks=sinks, seed=3)


@pytest.mark.parametrize("pairs", [[(1500, 1500)], [(4000, 5)], [(3000, 1), (2, 2), (900, 300)],
                                   [(2500, 8)] * 3])
@pytest.mark.parametrize("hq,heads,D,kv,q", [(8, 2, 128, "bf16", "bf16"), (4, 4, 64, "int8", "fp32"),
                                             (16, 1, 256, "bf16", "bf16")])
def test_prefill_long(w4, pairs, hq, heads, D, kv, q):
    check_prefill(w4, pairs, hq, heads, D, 32, kv, q, seed=5)


def test_prefill_rows_before_the_start(w4):
    """More queries than cached tokens: those at negative positions see
    nothing and give zeros."""
    check_prefill(w4, [(3, 10), (0, 4), (40, 40)], 4, 2, 64, 16, "bf16", "fp32", seed=16)


def test_prefill_one_token_is_decode(w4):
    """One query a sequence: the decode call's result within both bounds."""
    lens = [5, 130, 1000]
    cache, table, tl, K, V = make_cache(w4, lens, 2, 16, 128, "int8", 17)
    x = make_q((3, 8, 128), "fp32", 17)
    cu = torch.arange(4, dtype=torch.int32).cuda()
    a = w4.kv_prefill_attention(x, cache, 0, table, tl, cu)
    for b, n in enumerate(lens):
        assert close(a[b:b + 1], *attend(x[b:b + 1], K[b], V[b], [n - 1], 0, 0, 128 ** -0.5))[0]


def test_prefill_future_infinities(w4):
    """Infinities and NaN in later tokens and behind the window of a row reach
    only the rows that see them."""
    n, window, sinks = 150, 40, 2
    cache, table, tl, K, V = make_cache(w4, [n], 2, 16, 64, "bf16", 18)
    x = make_q((n, 4, 64), "bf16", 18)
    bad = {100: math.inf, 30: math.nan}
    for t, val in bad.items():
        page, slot = int(table[0, t // 16]), t % 16
        cache.k[0, page, :, slot] = val
        cache.v[0, page, :, slot] = val
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    y = w4.kv_prefill_attention(x, cache, 0, table, tl, cu, window=window, sinks=sinks)
    clean = [p for p in range(n) if not any(t <= p < t + window for t in bad)]
    for t in bad:
        K[0][t] = 0
        V[0][t] = 0
    out, rel, mean = attend(x, K[0], V[0], range(n), window, sinks, 0.125)
    ok, worst = close(y[clean], out[clean], rel[clean], mean[clean], p_rounded=True)
    assert ok, worst


def test_attention_in_a_graph_and_on_another_stream(w4):
    lens = [700, 33, 0, 129]
    cache, table, tl, K, V = make_cache(w4, lens, 2, 16, 128, "bf16", 19)
    x = make_q((4, 8, 128), "fp32", 19)
    cu = torch.tensor([0, 3, 5, 5, 9], dtype=torch.int32).cuda()
    xp = make_q((9, 8, 128), "bf16", 20)
    want = w4.kv_decode_attention(x, cache, 0, table, tl)
    wantp = w4.kv_prefill_attention(xp, cache, 0, table, tl, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = w4.kv_decode_attention(x, cache, 0, table, tl, stream=s)
    yp = w4.kv_prefill_attention(xp, cache, 0, table, tl, cu, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(yp, wantp)
    ws = torch.empty(w4.kv_attention_workspace_bytes(9, 4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out, outp = torch.empty_like(x), torch.empty_like(xp)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        w4.kv_decode_attention(x, cache, 0, table, tl, out=out, workspace=ws)
        w4.kv_prefill_attention(xp, cache, 0, table, tl, cu, out=outp, workspace=ws)
    for i in range(3):
        x.copy_(make_q((4, 8, 128), "fp32", 30 + i))
        eager = w4.kv_decode_attention(x, cache, 0, table, tl)
        out.fill_(math.nan)
        outp.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(outp, wantp)


def test_paths(w4):
    """The variants that the sizes select."""
    def decode(lens, W):
        cache, table, tl, K, V = make_cache(w4, lens, 2, 16, 64, "bf16", 40, W=W)
        w4.kv_decode_attention(make_q((len(lens), 4, 64), "fp32", 40), cache, 0, table, tl)
        return w4.w4_last_path(), w4.w4_last_kernel()

    def prefill(B, new):
        cache, table, tl, K, V = make_cache(w4, [new] * B, 2, 16, 64, "bf16", 41)
        cu = torch.arange(0, B * new + 1, new, dtype=torch.int32).cuda()
        w4.kv_prefill_attention(make_q((B * new, 4, 64), "bf16", 41), cache, 0, table, tl, cu)
        return w4.w4_last_path(), w4.w4_last_kernel()

    for (path, kernel), want in ((decode([5, 9], 8), "kv_decode"),
                                 (decode([5, 9], 200), "kv_decode_split"),
                                 (prefill(2, 200), "kv_prefill_split"),
                                 (prefill(300, 3), "kv_prefill")):
        assert path == want and "k_" + want.replace("_split", "") in kernel


def test_many_sequences(w4):
    """More sequences than a wave has lanes, at every place that searches them."""
    lens = [(i * 37) % 90 for i in range(200)]
    lens[150] = 4000
    check_decode(w4, lens, 4, 2, 64, 16, "bf16", "fp32", seed=42)
    pairs = [(n, min(n, i % 4)) for i, n in enumerate(lens)]
    check_prefill(w4, pairs, 4, 2, 64, 16, "int8", "fp32", seed=43)


@pytest.mark.parametrize("q", ["bf16", "fp32"])
@pytest.mark.parametrize("pairs", [[(400, 6)], [(90, 90)] * 12])
def test_prefill_hidden_infinities_split(w4, q, pairs):
    """The same as test_prefill_future_infinities for more layouts of the work,
    infinities in several tiles, a missing page among them."""
    hq, heads, D, ps = 4, 1, 128, 16
    lens = [n for n, _ in pairs]
    cache, table, tl, K, V = make_cache(w4, lens, heads, ps, D, "bf16", 44)
    cu = [0]
    for _, m in pairs:
        cu.append(cu[-1] + m)
    x = make_q((cu[-1], hq, D), q, 44)
    n, m = pairs[-1]
    bad = [n - 1, n - 3]
    for t in bad:
        page, slot = int(table[-1, t // ps]), t % ps
        cache.k[0, page, :, slot] = math.nan
        cache.v[0, page, :, slot, ::3] = -math.inf
    t = table.clone()
    t[-1, 1] = -1
    y = w4.kv_prefill_attention(x, cache, 0, t, tl, torch.tensor(cu, dtype=torch.int32).cuda())
    hole = torch.zeros(n, dtype=torch.bool)
    hole[ps:2 * ps] = True
    for i in bad:
        K[-1][i] = 0
        V[-1][i] = 0
    out, rel, mean = attend(x[cu[-2]:], K[-1], V[-1], range(n - m, n), 0, 0, D ** -0.5, hole)
    rows = m - 3
    ok, worst = close(y[cu[-2]:][:rows], out[:rows], rel[:rows], mean[:rows], p_rounded=q == "bf16")
    assert ok, worst
    assert not torch.isfinite(y[-1]).all()


def test_prefill_unequal_scales(w4):
    """int8: scales of hidden tokens that are infinite or NaN reach nothing."""
    n = 150
    cache, table, tl, K, V = make_cache(w4, [n], 2, 16, 64, "int8", 45)
    x = make_q((n, 4, 64), "bf16", 45)
    for t, val in ((100, math.inf), (30, math.nan)):
        page, slot = int(table[0, t // 16]), t % 16
        cache.k_scale[0, page, :, slot] = val
        cache.v_scale[0, page, :, slot] = val
        K[0][t] = 0
        V[0][t] = 0
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    y = w4.kv_prefill_attention(x, cache, 0, table, tl, cu, window=40, sinks=2)
    clean = [p for p in range(n) if not any(t <= p < t + 40 for t in (100, 30))]
    out, rel, mean = attend(x, K[0], V[0], range(n), 40, 2, 0.125)
    ok, worst = close(y[clean], out[clean], rel[clean], mean[clean], p_rounded=True)
    assert ok, worst


def test_prefill_rows_before_the_first_offset(w4):
    """Rows that belong to no sequence are not computed: 40 of them make a tile
    of 128 (token, head) rows before the first sequence's own."""
    heads, G, T, lo = 160, 4, 60, 40
    cache, table, tl, K, V = make_cache(w4, [90], heads, 16, 16, "bf16", 46)
    x = make_q((T, heads * G, 16), "fp32", 46)
    y = torch.full_like(x, 7.0)
    w4.kv_prefill_attention(x, cache, 0, table, tl, torch.tensor([lo, T], dtype=torch.int32).cuda(),
                            out=y)
    assert w4.w4_last_path() == "kv_prefill"
    assert (y[:lo] == 7.0).all()
    ok, worst = close(y[lo:], *attend(x[lo:], K[0], V[0], list(range(90 - (T - lo), 90)), 0, 0, 0.25))
    assert ok, worst
