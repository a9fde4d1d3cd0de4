"""Argument checks of the key-value cache's calls (no GPU needed, nothing is
launched): every refusal returns its documented status."""
import ctypes

import pytest
import torch

import int4_weight_quantized_amd as w4
from int4_weight_quantized_amd.kv import _Cache

OK, NULL, SHAPE, ALIGN, WS, ARG = 0, -1, -2, -3, -5, -7
FAKE = 1 << 20  # a non-NULL, 256-aligned address; never dereferenced by these calls
BIG = 1 << 40


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, layers=2, pages=10, heads=2,
             page_size=16, head_dim=64, dtype=w4.KV_BF16)
    d.update(kw)
    return _Cache(*(d[n] for n, _ in _Cache._fields_))


def ref(c):
    return None if c is None else ctypes.addressof(c)


def append(c, **kw):
    d = dict(layer=0, k=FAKE, v=FAKE, x=0, ldk=128, ldv=128, T=4, B=2, table=FAKE, W=3, start=FAKE,
             cu=FAKE)
    d.update(kw)
    return w4.lib().kv_append(ref(c), *d.values(), None)


def gather(c, **kw):
    d = dict(layer=0, k=FAKE, v=FAKE, x=1, T=4, B=2, table=FAKE, W=3, start=FAKE, cu=FAKE)
    d.update(kw)
    return w4.lib().kv_gather(ref(c), *d.values(), None)


def decode(c, **kw):
    d = dict(layer=0, q=FAKE, x=1, ldq=256, B=2, hq=4, table=FAKE, W=3, lens=FAKE, scale=0.125,
             window=0, sinks=0, out=FAKE, ws=FAKE, wsb=BIG)
    d.update(kw)
    return w4.lib().kv_decode_attention(ref(c), *d.values(), None)


def prefill(c, **kw):
    d = dict(layer=0, q=FAKE, x=1, ldq=256, T=5, B=2, hq=4, table=FAKE, W=3, lens=FAKE, cu=FAKE,
             scale=0.125, window=0, sinks=0, out=FAKE, ws=FAKE, wsb=BIG)
    d.update(kw)
    return w4.lib().kv_prefill_attention(ref(c), *d.values(), None)


def copy(c, other=None, **kw):
    d = dict(di=FAKE, si=FAKE, n=2)
    d.update(kw)
    src = cache() if other is None else other
    return w4.lib().kv_copy_pages(ref(c), d["di"], ref(src), d["si"], d["n"], None)


def reserve(**kw):
    d = dict(table=FAKE, S=3, W=4, lens=FAKE, refs=FAKE, pages=10, ps=16, add=FAKE, ok=FAKE,
             ws=FAKE, wsb=8 * 3 + 256)
    d.update(kw)
    return w4.lib().kv_reserve(*d.values(), None)


def fork(c, **kw):
    d = dict(table=FAKE, S=3, W=4, lens=FAKE, refs=FAKE, par=FAKE, kid=FAKE, n=2, ok=FAKE, ws=FAKE,
             wsb=16 * 2 + 256)
    d.update(kw)
    return w4.lib().kv_fork(ref(c), *d.values(), None)


def free(**kw):
    d = dict(table=FAKE, S=3, W=4, lens=FAKE, refs=FAKE, pages=10, slots=FAKE, n=2)
    d.update(kw)
    return w4.lib().kv_free(*d.values(), None)


def compact(c, **kw):
    d = dict(table=FAKE, S=3, W=4, refs=FAKE, to=FAKE, ro=FAKE, live=FAKE, ws=FAKE,
             wsb=8 * 10 + 256)
    d.update(kw)
    return w4.lib().kv_compact(ref(c), *d.values(), None)


WITH_CACHE = [append, gather, decode, prefill, copy, fork, compact]


@pytest.mark.parametrize("call", WITH_CACHE)
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(dtype=2), ARG), (dict(dtype=w4.KV_INT8), NULL),
    (dict(k_scale=FAKE), ARG), (dict(layers=0), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages=1 << 31), SHAPE), (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=8192), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(head_dim=72), SHAPE), (dict(head_dim=272), SHAPE),
    (dict(layers=1 << 20, pages=1 << 20, heads=8), SHAPE), (dict(k=FAKE + 8), ALIGN),
    (dict(v=FAKE + 2), ALIGN),
    (dict(dtype=w4.KV_INT8, k_scale=FAKE + 4, v_scale=FAKE), ALIGN),
])
def test_cache_refusals(call, kw, status):
    assert call(cache(**kw)) == status


@pytest.mark.parametrize("call", WITH_CACHE)
def test_no_cache(call):
    assert call(None) == NULL


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(table=None), NULL), (dict(start=None), NULL),
    (dict(layer=2), ARG), (dict(layer=-1), ARG), (dict(x=2), ARG), (dict(T=0), SHAPE),
    (dict(B=0), SHAPE), (dict(W=0), SHAPE), (dict(B=1 << 16, W=1 << 16), SHAPE),
    (dict(T=1 << 26), SHAPE), (dict(cu=None), SHAPE), (dict(ldk=127), SHAPE), (dict(ldv=0), SHAPE),
    (dict(ldk=1 << 45), SHAPE), (dict(k=FAKE + 1), ALIGN), (dict(x=1, v=FAKE + 2), ALIGN),
    (dict(table=FAKE + 2), ALIGN), (dict(start=FAKE + 1), ALIGN), (dict(cu=FAKE + 2), ALIGN)])
def test_append_refusals(kw, status):
    assert append(cache(), **kw) == status
    if not set(kw) & {"ldk", "ldv", "k", "v"}:
        assert gather(cache(), **kw) == status


def test_gather_alignment():
    assert gather(cache(), k=FAKE + 8) == ALIGN
    assert gather(cache(), v=None) == NULL


@pytest.mark.parametrize("call", [decode, prefill])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(x=-1), ARG), (dict(layer=2), ARG), (dict(window=-1), ARG), (dict(sinks=-1), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(B=0), SHAPE),
    (dict(W=0), SHAPE), (dict(hq=0), SHAPE), (dict(hq=3), SHAPE), (dict(hq=65536, ldq=1 << 23), SHAPE),
    (dict(ldq=255), SHAPE), (dict(ldq=1 << 46), SHAPE), (dict(ldq=257), ALIGN), (dict(q=FAKE + 4), ALIGN),
    (dict(out=FAKE + 8), ALIGN), (dict(lens=FAKE + 2), ALIGN), (dict(ws=None), WS), (dict(wsb=0), WS),
    (dict(ws=FAKE + 128), ALIGN)])
def test_attention_refusals(call, kw, status):
    assert call(cache(), **kw) == status


def test_prefill_refusals():
    assert prefill(cache(), cu=None) == NULL
    assert prefill(cache(), cu=FAKE + 2) == ALIGN
    assert prefill(cache(), T=0) == SHAPE
    assert prefill(cache(), T=(1 << 23) + 1) == SHAPE


def test_attention_workspace():
    f = w4.kv_attention_workspace_bytes
    for rows, B, hq, h, d in ((1, 1, 4, 1, 256), (64, 64, 32, 8, 128), (8192, 1, 32, 8, 128)):
        need = f(rows, B, hq, h, d)
        assert need > 0
        c = cache(heads=h, head_dim=d)
        kw = dict(B=B, hq=hq, ldq=hq * d, wsb=need - 1)
        assert prefill(c, T=rows, **kw) == WS
        if rows == B:
            assert decode(c, **kw) == WS
    for bad in ((0, 1, 4, 1, 64), (1, 0, 4, 1, 64), (1, 1, 3, 2, 64), (1, 1, 4, 1, 65),
                (1, 1, 4, 1, 512), (1, 1, 0, 1, 64), ((1 << 23) + 1, 1, 4, 1, 64)):
        assert f(*bad) == 0


@pytest.mark.parametrize("kw,status", [(dict(di=None), NULL), (dict(si=None), NULL), (dict(n=0), SHAPE),
                                       (dict(n=(1 << 23) + 1), SHAPE), (dict(di=FAKE + 2), ALIGN),
                                       (dict(other=cache(layers=3)), SHAPE),
                                       (dict(other=cache(heads=1)), SHAPE),
                                       (dict(other=cache(page_size=32)), SHAPE),
                                       (dict(other=cache(head_dim=32)), SHAPE),
                                       (dict(other=cache(dtype=1, k_scale=FAKE, v_scale=FAKE)), ARG)])
def test_copy_refusals(kw, status):
    assert copy(cache(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), NULL), (dict(lens=None), NULL), (dict(refs=None), NULL), (dict(add=None), NULL),
    (dict(ok=None), NULL), (dict(S=0), SHAPE), (dict(W=0), SHAPE), (dict(pages=0), SHAPE),
    (dict(ps=15), SHAPE), (dict(ps=0), SHAPE), (dict(add=FAKE + 1), ALIGN), (dict(ws=None), WS),
    (dict(wsb=279), WS), (dict(ws=FAKE + 8), ALIGN)])
def test_reserve_refusals(kw, status):
    assert reserve(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), NULL), (dict(lens=None), NULL), (dict(refs=None), NULL), (dict(par=None), NULL),
    (dict(kid=None), NULL), (dict(ok=None), NULL), (dict(S=0), SHAPE), (dict(n=0), SHAPE),
    (dict(n=(1 << 23) + 1), SHAPE), (dict(kid=FAKE + 1), ALIGN), (dict(ws=None), WS), (dict(wsb=287), WS)])
def test_fork_refusals(kw, status):
    assert fork(cache(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), NULL), (dict(lens=None), NULL), (dict(refs=None), NULL), (dict(slots=None), NULL),
    (dict(S=0), SHAPE), (dict(n=0), SHAPE), (dict(pages=0), SHAPE), (dict(slots=FAKE + 2), ALIGN)])
def test_free_refusals(kw, status):
    assert free(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), NULL), (dict(refs=None), NULL), (dict(to=None), NULL), (dict(ro=None), NULL),
    (dict(live=None), NULL), (dict(S=0), SHAPE), (dict(live=FAKE + 2), ALIGN), (dict(ws=None), WS),
    (dict(wsb=335), WS), (dict(ws=FAKE + 4), ALIGN)])
def test_compact_refusals(kw, status):
    assert compact(cache(), **kw) == status


def test_binding_refuses_host_tensors_and_wrong_shapes():
    k = torch.zeros((1, 4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.KVCache(k, k)
    with pytest.raises(ValueError, match="5-D"):
        w4.KVCache(k[0], k[0])
    with pytest.raises(TypeError, match="bfloat16 or int8"):
        w4.KVCache(k.float(), k.float())
    with pytest.raises(ValueError, match="int8 cache"):
        w4.KVCache(k.to(torch.int8), k.to(torch.int8))
    with pytest.raises(TypeError, match="KVCache"):
        w4.kv_append(k, 0, k, k, k, k)
    with pytest.raises(ValueError, match="cu must"):
        w4.kv_prefill_attention(k, None, 0, k, k, None)
