"""Argument checks of the norms', rotary positions' and adapters' calls, and the
frequencies (no GPU needed, nothing is launched)."""
import ctypes
import math

import pytest
import torch

import int4_weight_quantized_amd as w4
from int4_weight_quantized_amd import kv, layer
from int4_weight_quantized_amd.kv import _Cache
from int4_weight_quantized_amd.layer import _Spec

OK, NULL, SHAPE, ALIGN, WS, ARG = 0, -1, -2, -3, -5, -7
FAKE = 1 << 20  # a non-NULL, 256-aligned address; never dereferenced by these calls
BIG = 1 << 40
NAN, INF = math.nan, math.inf


def norm(**kw):
    d = dict(x=FAKE, xt=1, ldx=64, res=FAKE, w=FAKE, offset=0.0, eps=1e-6, M=2, K=64, sum=FAKE,
             out=FAKE, ot=1)
    d.update(kw)
    return w4.lib().rms_norm(*d.values(), None)


def norm8(**kw):
    d = dict(x=FAKE, xt=1, ldx=64, res=FAKE, w=FAKE, offset=0.0, eps=1e-6, M=2, K=64, sum=FAKE,
             xq=FAKE, sx=FAKE)
    d.update(kw)
    return w4.lib().a8_rms_norm(*d.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), NULL), (dict(sum=None), NULL), (dict(res=None), NULL),
    (dict(xt=2), ARG), (dict(xt=-1), ARG), (dict(eps=-1e-9), ARG), (dict(eps=NAN), ARG),
    (dict(eps=INF), ARG), (dict(offset=NAN), ARG), (dict(offset=-INF), ARG),
    (dict(sum=FAKE, ldx=72), ARG),
    (dict(M=0), SHAPE), (dict(K=0), SHAPE), (dict(M=-1), SHAPE), (dict(ldx=63), SHAPE),
    (dict(M=(1 << 23) + 1), SHAPE), (dict(K=w4.W4_MAX_K + 1, ldx=1 << 18), SHAPE),
    (dict(ldx=1 << 46), SHAPE), (dict(ldx=-64), SHAPE), (dict(M=1 << 22, K=16385, ldx=16385), SHAPE),
    (dict(x=FAKE + 2), ALIGN), (dict(res=FAKE + 2), ALIGN), (dict(sum=FAKE + 1), ALIGN),
    (dict(w=FAKE + 2), ALIGN)])
def test_norm_refusals(kw, rc):
    assert norm(**kw) == rc and norm8(**kw) == rc


def test_norm_refusals_of_outputs():
    assert norm(out=None) == NULL and norm8(xq=None) == NULL and norm8(sx=None) == NULL
    assert norm(ot=2) == ARG and norm(ot=-1) == ARG
    assert norm(out=FAKE + 2) == ALIGN and norm(out=FAKE + 1, ot=0) == ALIGN
    assert norm8(sx=FAKE + 2) == ALIGN


def spec(**kw):
    d = dict(turns=FAKE, rot=64, layout=0, mag=1.0)
    d.update(kw)
    return _Spec(*d.values())


def ref(c):
    return None if c is None else ctypes.addressof(c)


def rope(s="spec", **kw):
    s = spec() if isinstance(s, str) else s
    d = dict(x=FAKE, xt=1, ldx=128, T=3, heads=2, D=64, pos=FAKE, out=FAKE, ldo=128)
    d.update(kw)
    return w4.lib().rope_rotate(ref(s), *d.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), NULL), (dict(pos=None), NULL), (dict(out=None), NULL), (dict(xt=2), ARG),
    (dict(T=0), SHAPE), (dict(T=(1 << 23) + 1), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=1 << 25), SHAPE), (dict(heads=65536, T=1, ldx=1 << 23, ldo=1 << 23), SHAPE), (dict(heads=1 << 60), SHAPE), (dict(D=63), SHAPE),
    (dict(D=65), SHAPE), (dict(D=520, ldx=4096, ldo=4096), SHAPE), (dict(D=32), SHAPE),
    (dict(ldx=127, ldo=127), SHAPE), (dict(ldo=127), SHAPE), (dict(ldo=1 << 46), SHAPE),
    (dict(ldo=256), ARG),  # in place with another stride
    (dict(x=FAKE + 2), ALIGN), (dict(out=FAKE + 2), ALIGN), (dict(pos=FAKE + 2), ALIGN),
    (dict(out=FAKE + 1, xt=0), ALIGN)])
def test_rope_refusals(kw, rc):
    assert rope(**kw) == rc


SPECS = [(None, NULL), (spec(turns=None), NULL), (spec(layout=2), ARG), (spec(layout=-1), ARG),
         (spec(mag=NAN), ARG), (spec(mag=INF), ARG), (spec(rot=0), SHAPE), (spec(rot=63), SHAPE),
         (spec(rot=66), SHAPE), (spec(rot=514), SHAPE), (spec(rot=-2), SHAPE),
         (spec(turns=FAKE + 4), ALIGN)]


@pytest.mark.parametrize("s,rc", SPECS)
def test_specs_are_checked(s, rc):
    assert rope(s) == rc and place(s) == rc


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, layers=2, pages=10, heads=2, page_size=16,
             head_dim=64, dtype=w4.KV_BF16)
    d.update(kw)
    return _Cache(*(d[n] for n, _ in _Cache._fields_))


def place(s="spec", c="cache", **kw):
    s = spec() if isinstance(s, str) else s
    c = cache() if isinstance(c, str) else c
    d = dict(layer=0, rope=ref(s), q=FAKE, k=FAKE, v=FAKE, xt=1, ldq=256, ldk=128, ldv=128, hq=4, T=4,
             B=2, table=FAKE, W=3, start=FAKE, cu=FAKE, out=FAKE, ldo=256)
    d.update(kw)
    return w4.lib().kv_append_rope(ref(c), *d.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL),
    (dict(table=None), NULL), (dict(start=None), NULL), (dict(c=None), NULL),
    (dict(xt=2), ARG), (dict(layer=2), ARG), (dict(layer=-1), ARG), (dict(ldo=512), ARG),
    (dict(hq=0), SHAPE), (dict(hq=65536), SHAPE), (dict(hq=1 << 60), SHAPE),
    (dict(T=1 << 23, hq=60000), SHAPE), (dict(T=0), SHAPE), (dict(T=3, cu=None), SHAPE),
    (dict(ldq=255, ldo=255), SHAPE), (dict(ldk=127), SHAPE), (dict(ldv=127), SHAPE),
    (dict(ldo=255), SHAPE), (dict(W=0), SHAPE), (dict(B=0), SHAPE),
    (dict(c=cache(page_size=24)), SHAPE), (dict(c=cache(head_dim=48)), SHAPE),
    (dict(q=FAKE + 2), ALIGN), (dict(out=FAKE + 2), ALIGN), (dict(k=FAKE + 2), ALIGN),
    (dict(start=FAKE + 2), ALIGN), (dict(cu=FAKE + 1), ALIGN)])
def test_append_rope_refusals(kw, rc):
    assert place(**kw) == rc


def lora(**kw):
    d = dict(x=FAKE, xt=1, ldx=64, M=3, K=64, N=32, ids=FAKE, A=FAKE, B=FAKE, L=2, r=8, scales=FAKE,
             ranks=FAKE, y=FAKE, ldy=32, ws=FAKE, wsb=BIG)
    d.update(kw)
    return w4.lib().lora_add(*d.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), NULL), (dict(ids=None), NULL), (dict(A=None), NULL), (dict(B=None), NULL),
    (dict(y=None), NULL), (dict(xt=3), ARG),
    (dict(M=0), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(r=0), SHAPE), (dict(L=0), SHAPE),
    (dict(r=257), SHAPE), (dict(M=(1 << 23) + 1), SHAPE), (dict(K=w4.W4_MAX_K + 1, ldx=1 << 18), SHAPE),
    (dict(N=1 << 31, ldy=1 << 31), SHAPE), (dict(L=(1 << 20) + 1), SHAPE), (dict(L=1 << 62), SHAPE),
    (dict(L=1 << 20, r=256, N=(1 << 18) + 1, ldy=1 << 19), SHAPE),
    (dict(ldx=63), SHAPE), (dict(ldy=31), SHAPE), (dict(ldx=1 << 46), SHAPE),
    (dict(x=FAKE + 2), ALIGN), (dict(ids=FAKE + 2), ALIGN), (dict(A=FAKE + 1), ALIGN),
    (dict(B=FAKE + 1), ALIGN), (dict(scales=FAKE + 2), ALIGN), (dict(ranks=FAKE + 2), ALIGN),
    (dict(y=FAKE + 2), ALIGN), (dict(ws=FAKE + 64), ALIGN), (dict(ws=None), WS), (dict(wsb=0), WS)])
def test_lora_refusals(kw, rc):
    assert lora(**kw) == rc


def test_lora_workspace():
    f = w4.lora_workspace_bytes
    for bad in ((0, 64, 32, 8), (3, 0, 32, 8), (3, 64, 0, 8), (3, 64, 32, 0), (3, 64, 32, 257),
                ((1 << 23) + 1, 64, 32, 8), (3, w4.W4_MAX_K + 1, 32, 8), (3, 64, 1 << 31, 8)):
        assert f(*bad) == 0
    assert lora(wsb=f(3, 64, 32, 8) - 1) == WS
    # a larger call's workspace serves a smaller one
    sizes = [(1, 1, 1, 1), (1, 64, 64, 8), (16, 64, 64, 8), (17, 4096, 64, 8), (64, 4096, 11008, 16),
             (65, 4097, 11008, 17), (257, 8192, 28672, 64), (2000, 8192, 28672, 65), (8192, 8192, 28672, 128),
             (100000, 131071, 1 << 20, 256)]
    got = [f(*s) for s in sizes]
    assert got[0] > 0 and got == sorted(got)
    for M in range(1, 600, 7):
        assert f(M, 4096, 4096, 16) <= f(M + 7, 4096, 4096, 16) <= f(M + 7, 4097, 4096, 17)
    for K in range(1, 9000, 101):
        assert f(40, K, 4096, 16) <= f(40, K + 101, 4096, 16)


def frequencies(rot, base=10000.0, **kw):
    return w4.rope_frequencies(rot, base, **kw)


def test_frequencies_plain_linear_ntk():
    for rot in (2, 18, 64, 128, 512):
        plain = [10000.0 ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)]
        for kw, want in ((dict(), plain), (dict(scaling="linear", factor=4.0), [f / 4 for f in plain])):
            t, m = frequencies(rot, **kw)
            assert m == 1.0 and t.dtype == torch.float64 and t.shape == (rot // 2,)
            assert all(abs(a - b) <= 4 * 2.0 ** -52 * b for a, b in zip(t.tolist(), want))
    t, m = frequencies(64, scaling="ntk", factor=8.0)
    p, _ = frequencies(64)
    assert m == 1.0 and t[0] == p[0]  # the fastest pair stays, the slowest is divided by the factor
    assert float(t[-1] * 8 / p[-1]) == pytest.approx(1.0, rel=1e-13)
    assert frequencies(2, scaling="ntk", factor=8.0)[0].tolist() == frequencies(2)[0].tolist()


@pytest.mark.parametrize("scaling,fast", [("yarn", 32.0), ("bands", 4.0)])
def test_frequencies_by_parts(scaling, fast):
    """Fast pairs stay, slow ones are divided by the factor, a ramp between them."""
    rot, context, factor = 128, 4096, 16.0
    p, _ = frequencies(rot)
    t, m = frequencies(rot, scaling=scaling, factor=factor, context=context, fast=fast, slow=1.0)
    assert m == (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)
    share = (t / p).tolist()
    turns = (p * context).tolist()
    assert all(a >= b for a, b in zip(share, share[1:]))
    inside = 0
    for s, n in zip(share, turns):
        if scaling == "bands":
            keep = min(max((n - 1.0) / (fast - 1.0), 0.0), 1.0)
            assert s == pytest.approx(keep + (1 - keep) / factor, rel=1e-12)
        if n >= 2 * fast:
            assert s == pytest.approx(1.0, rel=1e-15)
        if n <= 0.5:
            assert s == pytest.approx(1 / factor, rel=1e-15)
        inside += 1 / factor * 1.001 < s < 0.999
    assert inside > 3
    if scaling == "yarn":  # the ramp is linear in the index
        ramp = [(1 - s) / (1 - 1 / factor) for s in share if 1 / factor * 1.001 < s < 0.999]
        steps = [b - a for a, b in zip(ramp, ramp[1:])]
        assert max(steps) == pytest.approx(min(steps), rel=1e-9)
    assert frequencies(rot, scaling=scaling, factor=1.0, context=context, fast=fast)[0].tolist() == \
        pytest.approx(p.tolist(), rel=1e-15)


@pytest.mark.parametrize("a,rc", [
    ((1, 1e4, 0, 1.0, 0, 32.0, 1.0), SHAPE), ((0, 1e4, 0, 1.0, 0, 32.0, 1.0), SHAPE),
    ((514, 1e4, 0, 1.0, 0, 32.0, 1.0), SHAPE), ((7, 1e4, 0, 1.0, 0, 32.0, 1.0), SHAPE),
    ((64, 1.0, 0, 1.0, 0, 32.0, 1.0), ARG), ((64, NAN, 0, 1.0, 0, 32.0, 1.0), ARG),
    ((64, INF, 0, 1.0, 0, 32.0, 1.0), ARG), ((64, 1e4, 5, 1.0, 0, 32.0, 1.0), ARG),
    ((64, 1e4, -1, 1.0, 0, 32.0, 1.0), ARG), ((64, 1e4, 1, 0.5, 0, 32.0, 1.0), ARG),
    ((64, 1e4, 2, NAN, 0, 32.0, 1.0), ARG), ((64, 1e4, 1, INF, 0, 32.0, 1.0), ARG),
    ((64, 1e4, 3, 2.0, 0, 32.0, 1.0), ARG), ((64, 1e4, 4, 2.0, 100, 1.0, 1.0), ARG),
    ((64, 1e4, 3, 2.0, 100, 32.0, 0.0), ARG), ((64, 1e4, 4, 2.0, 100, INF, 1.0), ARG),
    ((64, 1e4, 4, 2.0, 100, 4.0, NAN), ARG), ((64, 1e4, 0, 0.0, 0, 0.0, 0.0), OK)])
def test_frequencies_refusals(a, rc):
    buf, mag = (ctypes.c_double * 256)(), ctypes.c_double()
    assert w4.lib().rope_frequencies(*a, ctypes.addressof(buf), ctypes.addressof(mag)) == rc
    assert w4.lib().rope_frequencies(*a, None, ctypes.addressof(mag)) == NULL
    assert w4.lib().rope_frequencies(*a, ctypes.addressof(buf), None) == NULL


# ------------------------------------------------------------------ the binding
@pytest.fixture
def no_library(monkeypatch):
    def reached():
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(layer, "lib", reached)
    monkeypatch.setattr(kv, "lib", reached)


def test_host_tensors_are_refused(no_library):
    x, w = torch.zeros(2, 64), torch.zeros(64)
    for f in (w4.rms_norm, w4.a8_rms_norm):
        with pytest.raises(ValueError, match="x must be a GPU tensor"):
            f(x, w, 1e-6)
        with pytest.raises(ValueError, match="2-D"):
            f(w, w, 1e-6)
        with pytest.raises(ValueError, match="2-D"):
            f(None, w, 1e-6)
    with pytest.raises(ValueError, match="X must be a GPU tensor"):
        w4.lora_add(x, x, None, None, None)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        w4.rope_rotate(torch.zeros(2, 3, 64), None, None)
    with pytest.raises(ValueError, match="3-D"):
        w4.rope_rotate(x, None, None)
    with pytest.raises(TypeError, match="cache must be a KVCache"):
        w4.kv_append_rope(None, 0, x, x, x, None, None, None)
    with pytest.raises(ValueError, match="unknown scaling"):
        w4.rope_frequencies(64, scaling="dynamic")
    with pytest.raises(ValueError, match="turns must be a GPU tensor"):
        w4.Rope.of(torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="unknown layout"):
        w4.Rope.of(torch.zeros(32, dtype=torch.float64), layout="interleaved")
    with pytest.raises(ValueError, match="1-D"):
        w4.Rope.of(torch.zeros(32, 2, dtype=torch.float64))
    with pytest.raises(TypeError, match="rope must be a Rope"):
        layer._rope(3, torch.device("cuda:0"))
