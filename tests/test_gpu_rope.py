"""Rotary positions, alone and on the way into the cache, against the formula in
64 bits (GPU)."""
import math

import pytest
import torch

import int4_weight_quantized_amd as w4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
U16 = 2.0 ** -8


def rotate(x, pos, rope):
    """(result, bound) in 64 bits, from the rope's own frequencies.  c and s are
    rounded once (half a unit of the magnitude at most), each product and the sum
    once more; the angle's own error, 2 pi 2^-53 of a fraction of a turn and the
    64-bit functions', is below 2^-46."""
    x, t = x.double().cpu(), rope.turns.cpu()
    rot, half = rope.rot_dim, rope.rot_dim // 2
    turns = pos.double().cpu()[:, None] * t
    angle = 2 * math.pi * (turns - turns.round())
    c, s = (rope.magnitude * f(angle)[:, None] for f in (torch.cos, torch.sin))
    a, b = (x[..., :half], x[..., half:rot]) if rope.layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    y, e = x.clone(), torch.zeros_like(x)
    lo, hi = a * c - b * s, b * c + a * s
    step = U * 1.01 + 2.0 ** -46
    elo = (a * c).abs() * 2 * step + (b * s).abs() * 2 * step + lo.abs() * step + 2.0 ** -46 * (a.abs() + b.abs())
    ehi = (b * c).abs() * 2 * step + (a * s).abs() * 2 * step + hi.abs() * step + 2.0 ** -46 * (a.abs() + b.abs())
    if rope.layout == "half":
        y[..., :half], y[..., half:rot], e[..., :half], e[..., half:rot] = lo, hi, elo, ehi
    else:
        y[..., 0:rot:2], y[..., 1:rot:2], e[..., 0:rot:2], e[..., 1:rot:2] = lo, hi, elo, ehi
    return y, e


def close(got, want, bound):
    if got.dtype == torch.bfloat16:
        bound = bound + U16 * (want.abs() + bound)
    d = (got.double().cpu() - want).abs()
    assert (d <= bound + 1e-40).all(), float((d / (bound + 1e-40)).max())


def positions(T, far, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, far, (T,), generator=g, dtype=torch.int32)
    p[0] = 0
    p[-1] = far - 1
    return p


CASES = [(1, 1, 64, 64), (1, 5, 256, 256), (3, 40, 128, 128), (7, 4, 80, 32), (130, 12, 96, 24),
         (65, 3, 72, 70), (9, 2, 40, 2), (5, 1, 512, 512), (6, 2, 512, 510), (4, 3, 8, 8), (33, 80, 64, 16),
         (1000, 6, 128, 64), (2, 300, 16, 6), (17, 2, 264, 100)]


@pytest.mark.parametrize("T,heads,D,rot", CASES)
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rotate(T, heads, D, rot, layout, dt):
    g = torch.Generator().manual_seed(T + D + rot)
    x = torch.randn((T, heads, D), generator=g).to(dt)
    pos = positions(T, 131072, T)
    rope = w4.Rope(rot, layout=layout)
    y, e = rotate(x, pos, rope)
    xc, pc = x.cuda(), pos.cuda()
    got = w4.rope_rotate(xc, pc, rope)
    close(got, y, e)
    assert torch.equal(got[..., rot:], xc[..., rot:])
    # rows that lie apart, with rows between them that stay, and in place
    wide = torch.full((T, heads + 2, D), math.nan, dtype=dt, device="cuda")
    wide[:, 1:-1] = xc
    assert torch.equal(w4.rope_rotate(wide[:, 1:-1], pc, rope), got)
    assert w4.rope_rotate(wide[:, 1:-1], pc, rope, out=wide[:, 1:-1]) is not None
    assert torch.equal(wide[:, 1:-1], got) and wide[:, 0].isnan().all() and wide[:, -1].isnan().all()
    # addresses and strides that are aligned to elements only
    odd = torch.zeros(T * (heads * D + 3) + 1, dtype=dt, device="cuda")[1:].view(T, -1)[:, :heads * D]
    odd = odd.unflatten(1, (heads, D))
    odd.copy_(xc)
    assert torch.equal(w4.rope_rotate(odd, pc, rope), got)
    w4.rope_rotate(odd, pc, rope, out=odd)
    assert torch.equal(odd, got)


@pytest.mark.parametrize("scaling,kw", [("linear", {}), ("ntk", {}), ("yarn", dict(context=4096)),
                                        ("bands", dict(context=4096, fast=4.0))])
def test_stretched_far_positions(scaling, kw):
    """Up to the end of 32 bits, both signs."""
    rope = w4.Rope(128, base=500000.0, scaling=scaling, factor=32.0, **kw)
    x = torch.randn((6, 3, 128), generator=torch.Generator().manual_seed(1))
    pos = torch.tensor([0, 1, 10 ** 6, 2 ** 31 - 1, -1, -2 ** 31], dtype=torch.int32)
    y, e = rotate(x, pos, rope)
    close(w4.rope_rotate(x.cuda(), pos.cuda(), rope), y, e)


def test_a_turn_back_and_differences_of_positions():
    """The rotation by -p undoes that by p, and the product of two rotated heads
    goes by the difference of their positions alone."""
    rope = w4.Rope(64)
    g = torch.Generator().manual_seed(2)
    q, k = (torch.randn((5, 1, 64), generator=g).cuda() for _ in range(2))
    p = positions(5, 4000, 1).cuda()
    back = w4.rope_rotate(w4.rope_rotate(q, p, rope), -p, rope)
    size = q.unflatten(-1, (2, 32)).norm(dim=-2, keepdim=True).expand(-1, -1, 2, -1).flatten(-2)
    assert ((back - q).abs() <= 12 * U * size).all()  # five roundings of the pair each way, and of c and s
    for shift in (0, 777):
        d = (w4.rope_rotate(q, p + 3 + shift, rope) * w4.rope_rotate(k, p + shift, rope)).double().sum(-1)
        if shift == 0:
            first = d
    # each rotated value is off by 3 units of its pair at most: 6 of the product of the norms, twice
    assert ((d - first).abs() <= 16 * U * q.double().norm(dim=-1) * k.double().norm(dim=-1)).all()


def test_values_that_are_not_finite_stay_in_their_pair():
    rope = w4.Rope(64)
    x = torch.ones((2, 2, 96), device="cuda")
    x[0, 1, 5] = math.nan
    x[1, 0, 40] = math.inf
    x[1, 1, 80] = math.inf
    y = w4.rope_rotate(x, torch.tensor([3, 4], dtype=torch.int32, device="cuda"), rope)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[0, 1, 5] = bad[0, 1, 37] = bad[1, 0, 8] = bad[1, 0, 40] = bad[1, 1, 80] = True
    assert torch.equal(~y.isfinite(), bad)


# ------------------------------------------------------------------ into the cache
def setting(lens, new, hq, heads, D, ps, kv, dt, seed, joint=True):
    """A cache with everything that a call of kv_append_rope needs; pages in random order."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    W = max(need) + 1
    order = torch.randperm(sum(need) + 3, generator=g)
    table = torch.full((len(lens), W), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    T = cu[-1]
    rows = torch.randn((T, hq + 2 * heads, D), generator=g).to(dt).cuda()
    q, k, v = rows[:, :hq], rows[:, hq:hq + heads], rows[:, hq + heads:]
    if not joint:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    start = torch.tensor([n - m for n, m in zip(lens, new)], dtype=torch.int32)
    pos = torch.cat([torch.arange(n - m, n, dtype=torch.int32) for n, m in zip(lens, new)])

    def cache():
        c = w4.KVCache.empty(2, len(order), heads, ps, D, torch.int8 if kv == "int8" else torch.bfloat16)
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                t.zero_()
        return c
    return cache, table.cuda(), start.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), q, k, v, pos.cuda()


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y)
               for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)))


PLACES = [([1], [1], 1, 1, 64, 64, 16), ([5, 1, 700], [1, 1, 1], 4, 1, 256, 256, 32),
          ([64, 17, 300], [40, 17, 1], 12, 4, 80, 32, 16), ([130] * 70, [1] * 70, 32, 8, 128, 128, 64),
          ([900, 33], [513, 0], 6, 2, 96, 46, 64), ([20, 3, 9], [0, 3, 0], 2, 2, 16, 16, 16),
          ([2000], [2000], 5, 5, 64, 10, 128)]


@pytest.mark.parametrize("lens,new,hq,heads,D,rot,ps", PLACES)
@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_append_rope(lens, new, hq, heads, D, rot, ps, kv, dt, layout):
    """The same bits as the rotation in fp32 followed by kv_append, and within the
    rotation's bound of the formula."""
    cache, table, start, cu, q, k, v, pos = setting(lens, new, hq, heads, D, ps, kv, dt, len(lens) + D)
    rope = w4.Rope(rot, layout=layout, scaling="linear", factor=2.0)
    a, b = cache(), cache()
    out = w4.kv_append_rope(a, 1, q, k, v, table, start, rope, cu)
    assert torch.equal(out, w4.rope_rotate(q, pos, rope))
    close(out, *rotate(q, pos, rope))
    w4.kv_append(b, 1, w4.rope_rotate(k.float(), pos, rope), v.float(), table, start, cu)
    assert same(a, b)
    assert not a.k[0].any() and not a.v[0].any()
    if kv == "bf16":
        got, values = w4.kv_gather(a, 1, table, start, cu, k.shape[0], dtype=torch.bfloat16)
        close(got, *rotate(k, pos, rope))
        assert torch.equal(values, v.bfloat16())
    # in place, within the joint rows: keys and values stay
    keys = k.clone()
    c = cache()
    w4.kv_append_rope(c, 1, q, k, v, table, start, rope, cu, out=q)
    assert torch.equal(q, out) and torch.equal(k, keys) and same(a, c)
    if all(n == 1 for n in new):  # one token a sequence, without offsets
        d = cache()
        again = setting(lens, new, hq, heads, D, ps, kv, dt, len(lens) + D, joint=False)
        assert torch.equal(w4.kv_append_rope(d, 1, again[4], again[5], again[6], table, start, rope), out)
        assert same(a, d)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_rows_of_no_sequence_and_tokens_without_pages(kv):
    cache, table, start, cu, q, k, v, pos = setting([40, 33, 20], [30, 5, 20], 4, 2, 64, 16, kv,
                                                    torch.float32, 9)
    rope = w4.Rope(64)
    start[1] = -7                 # skipped
    table[0, 2] = -1              # tokens 32 ... 39 of sequence 0 have no page
    table[2, 1] = 10 ** 6         # nor have 16 ... 19 of sequence 2
    more = torch.cat([torch.full((3, 8, 64), math.nan).cuda(), torch.cat([q, k, v], 1),
                      torch.full((2, 8, 64), math.nan).cuda()])
    cu = cu + 3
    a, b = cache(), cache()
    out = torch.full((60, 4, 64), 5.0, device="cuda")
    w4.kv_append_rope(a, 0, more[:, :4], more[:, 4:6], more[:, 6:], table, start, rope, cu, out=out)
    want = w4.rope_rotate(q, pos, rope)
    keep = list(range(3)) + list(range(33, 38)) + [58, 59]
    assert (out[keep] == 5.0).all()
    assert torch.equal(out[3:33], want[:30]) and torch.equal(out[38:58], want[35:])
    w4.kv_append(b, 0, torch.cat([more[:3, 4:6], w4.rope_rotate(k, pos, rope), more[-2:, 4:6]]), more[:, 6:].contiguous(),
                 table, start, cu)
    assert same(a, b)


def test_int8_keys_that_are_not_finite():
    cache, table, start, cu, q, k, v, pos = setting([8], [8], 2, 2, 64, 16, "int8", torch.float32, 3)
    k[3, 1, 7] = math.inf
    v[5, 0, 1] = math.nan
    a = cache()
    w4.kv_append_rope(a, 0, q, k, v, table, start, w4.Rope(64), cu)
    page = int(table[0, 0])
    bad = torch.zeros(2, 16, dtype=torch.bool, device="cuda")
    bad[1, 3] = True
    assert torch.equal(a.k_scale[0, page].isnan(), bad)
    assert a.v_scale[0, page].isnan().sum() == 1 and a.v_scale[0, page, 0, 5].isnan()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 80, 256])
def test_int8_scales_of_every_size(D, dt):
    """Codes and scales of tiny, huge and zero vectors are kv_append's."""
    sizes = [0.0, 1e-44, 1e-38, 1e-30, 2e-18, 1e-10, 1.0, 1e10, 1e30, 1e38]
    n = len(sizes)
    cache, table, start, cu, q, k, v, pos = setting([n], [n], 2, 2, D, 16, "int8", torch.float32, 5)
    by = torch.tensor(sizes, device="cuda")[:, None, None] / 4
    q, k, v = ((t * by).to(dt) for t in (q, k, v))
    v[3, 0] = 0.0
    rope = w4.Rope(32)
    a, b = cache(), cache()
    w4.kv_append_rope(a, 0, q, k, v, table, start, rope, cu)
    w4.kv_append(b, 0, w4.rope_rotate(k.float(), pos, rope), v.float(), table, start, cu)
    assert same(a, b)


def test_the_far_end_of_a_large_pool():
    """Pages at offsets beyond 32 bits."""
    heads, D, ps = 8, 256, 64
    pages = (1 << 31) // (heads * D * ps) + 3
    c = w4.KVCache.empty(1, pages, heads, ps, D)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    x = torch.randn((70, 3 * heads, D), device="cuda")
    cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    start = torch.tensor([5], dtype=torch.int32, device="cuda")
    rope = w4.Rope(D)
    pos = torch.arange(5, 75, dtype=torch.int32, device="cuda")
    out = w4.kv_append_rope(c, 0, x[:, :heads], x[:, heads:2 * heads], x[:, 2 * heads:], table, start, rope, cu)
    k, v = w4.kv_gather(c, 0, table, start, cu, 70)
    assert torch.equal(out, w4.rope_rotate(x[:, :heads], pos, rope))
    assert torch.equal(k, w4.rope_rotate(x[:, heads:2 * heads], pos, rope).bfloat16().float())
    assert torch.equal(v, x[:, 2 * heads:].bfloat16().float())


def test_refusals():
    rope = w4.Rope(64)
    x = torch.zeros((3, 2, 64), device="cuda")
    p = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="positions must have shape"):
        w4.rope_rotate(x, p[:2], rope)
    with pytest.raises(TypeError, match="positions must be"):
        w4.rope_rotate(x, p.long(), rope)
    with pytest.raises(TypeError, match="x must be"):
        w4.rope_rotate(x.half(), p, rope)
    with pytest.raises(ValueError, match="contiguous"):
        w4.rope_rotate(x.transpose(0, 2), p, rope)
    with pytest.raises(ValueError, match="out"):
        w4.rope_rotate(x, p, rope, out=x[:2])
    with pytest.raises(TypeError, match="out must be"):
        w4.rope_rotate(x, p, rope, out=x.bfloat16())
    with pytest.raises(w4.W4Error):
        w4.rope_rotate(x[..., :32].contiguous(), p, rope)  # a head smaller than what rotates
    with pytest.raises(w4.W4Error):
        w4.rope_rotate(x[:0], p[:0], rope)
    cache, table, start, cu, q, k, v, pos = setting([8], [8], 2, 2, 64, 16, "bf16", torch.float32, 3)
    c = cache()
    with pytest.raises(TypeError, match="k must be"):
        w4.kv_append_rope(c, 0, q, k.bfloat16(), v, table, start, rope, cu)
    with pytest.raises(ValueError, match="tokens"):
        w4.kv_append_rope(c, 0, q[:4], k, v, table, start, rope, cu)
    with pytest.raises(ValueError, match="k must have shape"):
        w4.kv_append_rope(c, 0, q, q[:, :1], v, table, start, rope, cu)
    with pytest.raises(ValueError, match="cu must have shape"):
        w4.kv_append_rope(c, 0, q, k, v, table, start, rope, cu[:1])
    with pytest.raises(w4.W4Error):
        w4.kv_append_rope(c, 2, q, k, v, table, start, rope, cu)
    with pytest.raises(w4.W4Error):
        w4.kv_append_rope(c, 0, q, k, v, table, start, w4.Rope(128), cu)


def test_captured_and_on_another_stream():
    cache, table, start, cu, q, k, v, pos = setting([50, 300], [1, 1], 4, 2, 128, 16, "int8", torch.float32, 4)
    rope = w4.Rope(128)
    a, b, out = cache(), cache(), torch.empty((2, 4, 128), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.kv_append_rope(a, 0, q, k, v, table, start, rope, stream=side)
    turned = w4.rope_rotate(q, pos, rope, stream=side)
    side.synchronize()
    assert torch.equal(got, w4.rope_rotate(q, pos, rope)) and torch.equal(turned, got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.kv_append_rope(a, 0, q, k, v, table, start, rope, out=out)
        w4.rope_rotate(q, pos, rope, out=turned)
    for i in range(3):
        start -= 7
        pos -= 7
        g.replay()
        torch.cuda.synchronize()
        want = w4.kv_append_rope(b, 0, q, k, v, table, start, rope)
        assert torch.equal(out, want) and torch.equal(turned, want)
        for x, y in zip(w4.kv_gather(a, 0, table, start, None, 2), w4.kv_gather(b, 0, table, start, None, 2)):
            assert torch.equal(x, y)
