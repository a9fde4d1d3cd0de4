"""A block served with a norm, adapters and rotary positions around its quantized
projection and its cache: every stage of every call is checked against its own
formula (GPU)."""
import os
import sys

import pytest
import torch

from kv_cases import attend, close

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
U = 2.0 ** -24


def norm(x, w):
    """The norm as its definition rounds it (fp32, on the CPU)."""
    x = x.cpu()
    r = (1.0 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6)).float()
    return (x * r) * w.cpu()


def turn(x, pos, rope):
    """Rotated heads and the bound of their error, in 64 bits (half layout)."""
    x, half = x.double().cpu(), rope.rot_dim // 2
    a = 2 * torch.pi * ((pos.double()[:, None] * rope.turns.cpu()) % 1.0)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    lo, hi = x[..., :half], x[..., half:rope.rot_dim]
    y = torch.cat([lo * c - hi * s, hi * c + lo * s, x[..., rope.rot_dim:]], -1)
    e = torch.cat([lo.abs() + hi.abs()] * 2 + [x[..., rope.rot_dim:].abs() * 0], -1)
    return y, 4 * U * e  # c or s, the product, the sum: three roundings of the pair at most


@pytest.mark.parametrize("adapters", [0, 3])
@pytest.mark.parametrize("rotary", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
def test_served_block(orc, adapters, rotary, dtype):
    import decode_layer
    import int4_weight_quantized_amd as w4

    rope = w4.Rope(96, scaling="linear", factor=2.0) if rotary else None
    b = decode_layer.Block(512, 8, 2, 128, slots=4, pages=40, pages_per_slot=10, dtype=dtype, norm=True,
                           rope=rope, adapters=adapters)
    if adapters:
        b.adapter.copy_(torch.tensor([2, -1, 0, 1], dtype=torch.int32))
    packed, sw = b.wqkv.cpu().numpy(), b.sqkv.cpu().numpy()
    inputs = []
    project = b.project

    def looked(x, adapter=None):
        out = project(x, adapter)
        inputs.append((x, adapter, [t.clone() for t in out]))
        return out
    b.project = looked
    history = {}

    def check(slots, rows, lens, q, o):
        """slots[i] has rows[i] = (first, last) of the call and lens[i] cached tokens."""
        x, adapter, (q0, k0, v0) = inputs.pop()
        h = norm(x, b.norm)
        y = torch.from_numpy(orc.w4a8_linear(h.numpy(), packed, sw))
        got = torch.cat([t.flatten(1) for t in (q0, k0, v0)], 1).cpu()
        if not adapters:
            assert torch.equal(got, y)  # the int8 rows, and so the product, bit for bit
        else:
            want, bound = y.double(), 2 * U * y.double().abs()
            for m, a in enumerate(adapter.tolist()):
                if a >= 0:
                    A, B = b.A[a].double().cpu(), b.B[a].double().cpu()
                    d = (h[m].double() @ A.T) @ B.T
                    e = (h[m].double().abs() @ A.abs().T) @ B.abs().T
                    want[m] += d
                    bound[m] += (512 + 16 + 64) * U * e + 2 * U * d.abs()
            assert ((got.double() - want).abs() <= bound).all()
        for s, (lo, hi), n in zip(slots, rows, lens):
            pos = torch.arange(n - (hi - lo), n)
            one = b.table[s:s + 1].contiguous()
            k, v = (t.double().cpu() for t in w4.kv_gather(b.cache, 0, one, decode_layer.ints(0),
                                                           decode_layer.ints(0, n), n))
            kt, ke = turn(k0[lo:hi], pos, rope) if rotary else (k0[lo:hi].double().cpu(), 0.0)
            vt = v0[lo:hi].double().cpu()
            for cached, t, e in ((k[n - (hi - lo):], kt, ke), (v[n - (hi - lo):], vt, 0.0)):
                # bf16: half a unit; int8: half a step of absmax / 127, whose scale and value are rounded
                step = 2.0 ** -8 * t.abs() if dtype == torch.bfloat16 else \
                    t.abs().amax(-1, keepdim=True) * (0.5 / 127 + 8 * U)
                assert ((cached - t).abs() <= step + 1.01 * e).all()
            if s in history:  # what was cached stays
                assert torch.equal(k[:len(history[s])], history[s])
            history[s] = k
            qt, qe = turn(q0[lo:hi], pos, rope) if rotary else (q0[lo:hi].double().cpu(), 0.0)
            assert ((q[lo:hi].double().cpu() - qt).abs() <= qe).all()
            ok, worst = close(o[lo:hi], *attend(q[lo:hi], k, v, pos.tolist(), 0, 0, 128 ** -0.5))
            assert ok, worst

    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((70, 512), generator=g, device="cuda")
    _, q, o = b.prompts(x, decode_layer.ints(2, 0, 1), decode_layer.ints(0, 33, 34, 70))
    check([2, 0, 1], [(0, 33), (33, 34), (34, 70)], [33, 1, 36], q, o)
    b.fork(decode_layer.ints(2), decode_layer.ints(3))
    history[3] = history[2]
    assert b.adapter.tolist() == ([2, -1, 0, 0] if adapters else [-1] * 4)
    for i in range(4):
        x = torch.randn((4, 512), generator=g, device="cuda")
        _, q, o = b.step(x)
        check([0, 1, 2, 3], [(s, s + 1) for s in range(4)], [2 + i, 37 + i, 34 + i, 34 + i], q, o)


def test_example_runs():
    import decode_layer
    import int4_weight_quantized_amd as w4

    b = decode_layer.serve(6, norm=True, rope=w4.Rope(128), adapters=3)
    assert b.lens.tolist() == [43, 43, 206, 0, 0, 0, 0, 0]
    assert b.adapter.tolist()[:2] == [2, 2]


@pytest.mark.parametrize("adapters", [0, 3])
def test_a_captured_step(adapters):
    """A whole step captured once and replayed, against the same steps one by one."""
    import decode_layer
    import int4_weight_quantized_amd as w4

    def block():
        b = decode_layer.Block(512, 8, 2, 128, slots=4, pages=40, pages_per_slot=10, norm=True,
                               rope=w4.Rope(128), adapters=adapters)
        if adapters:
            b.adapter.copy_(torch.tensor([2, -1, 0, 1], dtype=torch.int32))
        g = torch.Generator(device="cuda").manual_seed(3)
        b.prompts(torch.randn((50, 512), generator=g, device="cuda"), decode_layer.ints(3, 0),
                  decode_layer.ints(0, 30, 50))
        return b

    one, two = block(), block()
    x = torch.zeros((4, 512), device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = two.step(x)
    assert two.lens.tolist() == [20, 0, 0, 30]  # (captured, not run)
    gen = torch.Generator(device="cuda").manual_seed(9)
    for i in range(5):
        fresh = torch.randn((4, 512), generator=gen, device="cuda")
        x.copy_(fresh)
        g.replay()
        torch.cuda.synchronize()
        want = one.step(fresh)
        run = one.lens > 0
        for a, b in zip(out, want):
            assert torch.equal(a[run], b[run])
        assert torch.equal(one.lens, two.lens) and torch.equal(one.table, two.table)
        cu = decode_layer.ints(0, 20 + i + 1)
        a, b = (w4.kv_gather(c.cache, 0, c.table[:1].contiguous(), decode_layer.ints(0), cu, 20 + i + 1)
                for c in (one, two))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert one.lens.tolist() == [25, 0, 0, 35]
