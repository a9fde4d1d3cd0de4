"""Root-mean-square norms against the formula in 64 bits (GPU)."""
import math

import pytest
import torch

import int4_weight_quantized_amd as w4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24   # half a unit of fp32
U16 = 2.0 ** -8  # of bf16


def make(M, K, dt, res, seed, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    x[:, seed % K] *= 50
    r = (3 * torch.randn((M, K), generator=g)).to(dt) if res else None
    w = 0.2 * torch.randn((K,), generator=g) + (1 - offset)
    return x.to(dt), r, w


def formula(x, r, w, offset, eps):
    """(fp32 norm as the definition rounds it, h): the mean is taken in 64 bits."""
    h = x.float() if r is None else x.float() + r.float()
    rs = (1.0 / torch.sqrt((h.double() ** 2).mean(-1, keepdim=True) + eps)).float()
    return (h * rs) * (offset + (torch.ones(x.shape[1]) if w is None else w)), h


def exact(x, r, w, offset, eps):
    h = x.double() if r is None else x.double() + r.double()
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * (offset + w.double())


def cuda(*t):
    return [None if x is None else x.cuda() for x in t]


SHAPES = [(1, 1), (3, 7), (1, 64), (2, 100), (5, 512), (1, 1152), (64, 1000), (7, 1024), (33, 2048),
          (130, 2056), (2, 4096), (300, 4096), (9, 5120), (4, 8192), (257, 8192), (3, 11008), (2, 16384),
          (3, 16392), (1, 28672), (2, 131071), (1100, 520), (2, 131064)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("res,offset", [(False, 0.0), (True, 1.0)])
def test_norm(M, K, dt, res, offset):
    """Bit for bit what the definition says, in every output type; the error
    against 64 bits is that of its six roundings (r's mean holds two half units of
    h, so that r is off by one of them and its own), and one more for bf16."""
    x, r, w = make(M, K, dt, res, M + K, offset)
    y, h = formula(x, r, w, offset, 1e-6)
    xc, rc, wc = cuda(x, r, w)
    for ot in (torch.float32, torch.bfloat16):
        o, s = w4.rms_norm(xc, wc, 1e-6, residual=rc, offset=offset, dtype=ot)
        assert torch.equal(o.cpu(), y.to(ot))
        assert (s is None) if r is None else torch.equal(s.cpu(), h.to(dt))
    e = exact(x, r, w, offset, 1e-6)
    assert ((y.double() - e).abs() <= 7 * U * e.abs()).all()
    assert ((o.double().cpu() - e).abs() <= (7 * U + 1.01 * U16) * e.abs()).all()
    q, sx, s = w4.a8_rms_norm(xc, wc, 1e-6, residual=rc, offset=offset)
    q2, sx2 = w4.a8_quantize_act(w4.rms_norm(xc, wc, 1e-6, residual=rc, offset=offset,
                                             dtype=torch.float32)[0])
    assert torch.equal(q, q2) and torch.equal(sx, sx2)
    assert (s is None) if r is None else torch.equal(s.cpu(), h.to(dt))


def test_codes_against_the_oracle(orc):
    x, r, w = make(21, 1152, torch.float32, True, 5)
    y, _ = formula(x, r, w, 0.0, 1e-5)
    q, sx, _ = w4.a8_rms_norm(*cuda(x, w), 1e-5, residual=r.cuda())
    qo, so = orc.quantize_act(y.numpy())
    assert (q.cpu().numpy() == qo).all() and (sx.cpu().numpy() == so).all()


@pytest.mark.parametrize("K", [64, 72, 4096, 4100, 20000, 32767, 40001])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_in_place_strided_and_shifted(K, dt):
    """The sum over the residual or over x; rows of x that lie apart; operands at
    addresses that are aligned to their elements only."""
    x, r, w = make(6, K, dt, True, K)
    y, h = formula(x, r, w, 0.0, 1e-6)
    xc, rc, wc = cuda(x, r, w)
    rr = rc.clone()
    o, s = w4.rms_norm(xc, wc, 1e-6, residual=rr, sum=rr, dtype=torch.float32)
    assert s is rr and torch.equal(rr.cpu(), h.to(dt)) and torch.equal(o.cpu(), y)
    xx = xc.clone()
    q, sx, s = w4.a8_rms_norm(xx, wc, 1e-6, residual=rc, sum=xx)
    q0, sx0, _ = w4.a8_rms_norm(xc, wc, 1e-6, residual=rc)
    assert torch.equal(xx.cpu(), h.to(dt)) and torch.equal(q, q0) and torch.equal(sx, sx0)
    for pad, first in ((8, 0), (8, 8), (5, 3), (1, 1)):
        wide = torch.full((6, K + pad), math.nan, dtype=dt, device="cuda")
        wide[:, first:first + K] = xc
        o, s = w4.rms_norm(wide[:, first:first + K], wc, 1e-6, residual=rc, dtype=torch.float32)
        assert torch.equal(o.cpu(), y) and torch.equal(s.cpu(), h.to(dt))
    def shift(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.flatten()
        return b[1:].view(t.shape)
    outs = [shift(torch.zeros(6, K, dtype=t, device="cuda")) for t in (torch.int8, torch.bfloat16)]
    q, sx, s = w4.a8_rms_norm(shift(xc), shift(wc), 1e-6, residual=shift(rc), Xq=outs[0],
                              sx=shift(torch.zeros(6, device="cuda")), sum=shift(torch.zeros_like(xc)))
    assert q is outs[0] and torch.equal(q, q0) and torch.equal(sx, sx0) and torch.equal(s.cpu(), h.to(dt))
    for one in ("x", "residual", "weight", "sum", "out"):  # each by itself
        t = dict(x=xc, residual=rc, weight=wc, sum=torch.empty_like(xc), out=torch.empty_like(outs[1]))
        t[one] = shift(t[one])
        o, s = w4.rms_norm(t["x"], t["weight"], 1e-6, residual=t["residual"], sum=t["sum"], out=t["out"])
        assert torch.equal(o.cpu(), y.bfloat16()) and torch.equal(s.cpu(), h.to(dt)), one


def test_without_weight():
    x, _, _ = make(5, 1152, torch.float32, False, 1)
    for off in (0.0, 1.0):
        y, _ = formula(x, None, None, off, 1e-6)
        assert torch.equal(w4.rms_norm(x.cuda(), None, 1e-6, offset=off)[0].cpu(), y)


@pytest.mark.parametrize("K", [512, 1001])
def test_rows_at_the_ends_of_the_range(K):
    """Zeros, tiny and huge rows, and rows with values that are not finite; every
    row is the formula's, and no row touches another."""
    x = torch.randn((9, K), generator=torch.Generator().manual_seed(3))
    w = torch.ones(K)
    x[1] = 0.0
    x[2] *= 1e-30
    x[3] *= 1e37   # squares beyond fp32
    x[4] = 1e-42   # subnormal
    x[5, 7] = math.inf
    x[6, 9] = math.nan
    x[7, 3] = -math.inf
    y, _ = formula(x, None, w, 0.0, 1e-6)
    o, _ = w4.rms_norm(*cuda(x, w), 1e-6)
    fine = [0, 1, 2, 3, 4, 8]
    assert torch.equal(o.cpu()[fine], y[fine])
    assert torch.equal(o.cpu()[5:8].isnan(), y[5:8].isnan())
    q, sx, _ = w4.a8_rms_norm(*cuda(x, w), 1e-6)
    q2, sx2 = w4.a8_quantize_act(o[fine].contiguous())
    assert torch.equal(q[fine], q2) and torch.equal(sx[fine], sx2)
    assert sx[5:8].isnan().all() and sx[1] == 0 and not q[1].any()
    # eps as it is given, not rounded: rows far below it are scaled by it alone
    for eps in (1e-6, 1e-5, 3e-7, 1e-12):
        assert torch.equal(w4.rms_norm(*cuda(x[2:3], w), eps)[0].cpu(), formula(x[2:3], None, w, 0.0, eps)[0])
    # eps 0: a row of zeros is NaN, the others are not touched
    o, _ = w4.rms_norm(*cuda(x[:3], w), 0.0)
    assert o[1].isnan().all() and torch.equal(o.cpu()[::2], formula(x[:3:2], None, w, 0.0, 0.0)[0])
    _, sx, _ = w4.a8_rms_norm(*cuda(x[:3], w), 0.0)
    assert sx.isnan().tolist() == [False, True, False]
    # weights that make tiny outputs: scales below the division-free range
    ws = torch.full((K,), 1e-25)
    y, _ = formula(x[:1], None, ws, 0.0, 1e-6)
    q, sx, _ = w4.a8_rms_norm(*cuda(x[:1], ws), 1e-6)
    q2, sx2 = w4.a8_quantize_act(y.cuda())
    assert torch.equal(q, q2) and torch.equal(sx, sx2) and float(sx) < 2.0 ** -64


def test_refusals():
    x = torch.zeros(2, 64, device="cuda")
    w = torch.zeros(64, device="cuda")
    for f in (w4.rms_norm, w4.a8_rms_norm):
        with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
            f(x.half(), w, 1e-6)
        with pytest.raises(ValueError, match="contiguous"):
            f(torch.zeros(64, 2, device="cuda").t(), w, 1e-6)
        with pytest.raises(ValueError, match="weight must have shape"):
            f(x, w[:32], 1e-6)
        with pytest.raises(TypeError, match="residual must be"):
            f(x, w, 1e-6, residual=x.bfloat16())
        with pytest.raises(ValueError, match="residual must have shape"):
            f(x, w, 1e-6, residual=x[:1])
        with pytest.raises(ValueError, match="sum belongs"):
            f(x, w, 1e-6, sum=x)
        with pytest.raises(w4.W4Error):
            f(x, w, -1.0)
        with pytest.raises(w4.W4Error):
            f(x[:0], w, 1e-6)
        with pytest.raises(w4.W4Error):
            f(x[:1].expand(2, 64), w, 1e-6)  # rows on top of each other
    with pytest.raises(TypeError, match="a8_rms_norm"):
        w4.rms_norm(x, w, 1e-6, dtype=torch.int8)
    with pytest.raises(TypeError, match="out must be"):
        w4.rms_norm(x, w, 1e-6, dtype=torch.float32, out=x.bfloat16())


def test_captured_and_on_another_stream():
    x, r, w = make(17, 4096, torch.float32, True, 2)
    xc, rc, wc = cuda(x, r, w)
    q, sx, s = torch.empty(17, 4096, dtype=torch.int8, device="cuda"), torch.empty(17, device="cuda"), xc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.a8_rms_norm(xc, wc, 1e-5, residual=rc, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        w4.a8_rms_norm(xc, wc, 1e-5, residual=rc, Xq=q, sx=sx, sum=s)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, (q, sx, s)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.a8_rms_norm(xc, wc, 1e-5, residual=rc, Xq=q, sx=sx, sum=s)
    for i in range(3):
        xc.copy_(x * (i + 1))
        g.replay()
        torch.cuda.synchronize()
        want = w4.a8_rms_norm(xc, wc, 1e-5, residual=rc)
        assert all(torch.equal(a, b) for a, b in zip(want, (q, sx, s)))


@pytest.mark.parametrize("M,K", [(4097, 90), (1001, 128), (513, 512), (6, 3), (10, 513), (2049, 16)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_many_short_rows(M, K, dt):
    x, r, w = make(M, K, dt, True, M)
    y, h = formula(x, r, w, 0.0, 1e-6)
    xc, rc, wc = cuda(x, r, w)
    o, s = w4.rms_norm(xc, wc, 1e-6, residual=rc, dtype=torch.float32)
    assert torch.equal(o.cpu(), y) and torch.equal(s.cpu(), h.to(dt))
    q, sx, _ = w4.a8_rms_norm(xc, wc, 1e-6, residual=rc)
    q2, sx2 = w4.a8_quantize_act(o)
    assert torch.equal(q, q2) and torch.equal(sx, sx2)
