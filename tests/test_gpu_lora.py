"""Low-rank adapters against the formula in 64 bits (GPU)."""
import math

import pytest
import torch

import int4_weight_quantized_amd as w4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(M, K, N, r, L, dt, seed, ragged=False, order="mixed"):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn((M, K), generator=g).to(dt)
    A = (torch.randn((L, r, K), generator=g) * K ** -0.5).bfloat16()
    B = (torch.randn((L, N, r), generator=g) * 0.3).bfloat16()
    scales = 0.5 + 2 * torch.rand((L,), generator=g)
    ids = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    if order == "runs":
        ids = ids.sort().values
    elif order == "one":
        ids[:] = L - 1
    ranks = torch.randint(0, r + 1, (L,), generator=g, dtype=torch.int32) if ragged else None
    return X, A, B, scales, ids, ranks, torch.randn((M, N), generator=g)


def formula(X, A, B, scales, ids, ranks, Y):
    """(Y, bound) in 64 bits.  K products and sums of X A^T in fp32, rank of them in
    the second product, in any order (partial sums and the splitting of a value
    into terms add at most 64), the scale and the addition to Y."""
    Y, K, r = Y.double().clone(), X.shape[1], A.shape[1]
    E = torch.zeros_like(Y)
    for a in set(ids.tolist()):
        if not 0 <= a < A.shape[0]:
            continue
        rows = (ids == a).nonzero()[:, 0]
        n = r if ranks is None else min(max(int(ranks[a]), 0), r)
        s = 1.0 if scales is None else float(scales[a])
        x, ad, bd = X[rows].double(), A[a, :n].double(), B[a, :, :n].double()
        d = s * ((x @ ad.T) @ bd.T)
        mag = abs(s) * ((x.abs() @ ad.abs().T) @ bd.abs().T)
        E[rows] = (K + n + 64) * U * mag + 2 * U * (Y[rows].abs() + d.abs())
        Y[rows] += d
    return Y, E


def cuda(*t):
    return [None if x is None else x.cuda() for x in t]


def close(got, want, bound):
    d = (got.double().cpu() - want).abs()
    assert (d <= bound).all(), float((d / bound.clamp(min=1e-300)).max())


SIZES = [(1, 64, 64, 8, 1), (1, 1152, 6912, 8, 4), (2, 1, 1, 1, 1), (3, 7, 5, 3, 2), (5, 100, 33, 17, 3),
         (16, 512, 256, 16, 5), (17, 1000, 130, 32, 40), (64, 4096, 1000, 16, 32), (16, 2048, 512, 64, 16),
         (9, 520, 264, 100, 3), (33, 256, 1024, 128, 4), (4, 8192, 96, 256, 2), (70, 1001, 77, 5, 6),
         (200, 640, 320, 24, 8), (300, 1024, 512, 16, 3), (1000, 264, 200, 40, 5), (2, 131071, 16, 4, 2),
         (700, 131, 1025, 9, 2), (5, 4096, 4096, 1, 2), (129, 136, 72, 250, 3)]


@pytest.mark.parametrize("M,K,N,r,L", SIZES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ragged,order", [(False, "mixed"), (True, "runs"), (True, "one")])
def test_adapters(M, K, N, r, L, dt, ragged, order):
    X, A, B, scales, ids, ranks, Y = make(M, K, N, r, L, dt, M + K + r, ragged, order)
    want, bound = formula(X, A, B, scales, ids, ranks, Y)
    c = cuda(X, A, B, scales, ids, ranks)
    y = Y.cuda()
    got = w4.lora_add(y, c[0], c[4], c[1], c[2], scales=c[3], ranks=c[5])
    assert got is y
    close(y, want, bound)
    none = (ids < 0).nonzero()[:, 0]
    assert torch.equal(y.cpu()[none], Y[none])
    # again: the same bits
    z = w4.lora_add(Y.cuda(), c[0], c[4], c[1], c[2], scales=c[3], ranks=c[5])
    assert torch.equal(y, z)


@pytest.mark.parametrize("M", [1, 5, 40, 150, 520])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_do_not_depend_on_each_other(M, dt):
    """A row alone, and rows in another order, in the same call size."""
    X, A, B, scales, ids, ranks, Y = cuda(*make(M, 512, 200, 24, 4, dt, M))
    y = w4.lora_add(Y.clone(), X, ids, A, B, scales=scales)
    p = torch.randperm(M, generator=torch.Generator().manual_seed(M)).cuda()
    z = w4.lora_add(Y[p].contiguous(), X[p].contiguous(), ids[p].contiguous(), A, B, scales=scales)
    assert torch.equal(y[p], z)
    for m in range(0, M, max(1, M // 5)):
        other = torch.full_like(ids, -1)
        other[m] = ids[m]
        z = w4.lora_add(Y.clone(), X, other, A, B, scales=scales)
        assert torch.equal(z[m], y[m])
        rest = torch.arange(M).cuda() != m
        assert torch.equal(z[rest], Y[rest])


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_what_takes_no_part_may_hold_anything(M, dt):
    """Padding of ranks, adapters that no row names, rows without an adapter, ids
    outside the pool, and rows whose own values are not finite."""
    K, N, r, L = 264, 136, 40, 6
    X, A, B, scales, ids, ranks, Y = make(M, K, N, r, L, dt, M)
    ranks = torch.tensor([40, 7, 0, 32, 33, 8], dtype=torch.int32)
    ids = (torch.arange(M) % 5).int()
    ids[1] = -5
    ids[2 % M] = 2
    if M > 3:
        ids[3], ids[4] = L, 2 ** 31 - 1
    want, bound = formula(X, A, B, scales, ids, ranks, Y)
    for a in range(L):
        A[a, ranks[a]:] = math.nan
        B[a, :, ranks[a]:] = math.nan
    A[5], B[5], scales[5] = math.nan, math.inf, math.nan
    X[1] = math.nan
    c = cuda(X, A, B, scales, ids, ranks)
    y = w4.lora_add(Y.cuda(), c[0], c[4], c[1], c[2], scales=c[3], ranks=c[5])
    close(y, want, bound)
    assert torch.equal(y[1].cpu(), Y[1])
    bad = 0
    c[0][bad, 3] = math.inf
    z = w4.lora_add(Y.cuda(), c[0], c[4], c[1], c[2], scales=c[3], ranks=c[5])
    assert not z[bad].isfinite().any() and torch.equal(z[1:], y[1:])
    # ranks beyond the pool's are the pool's
    X, A, B, scales, ids, _, Y = cuda(*make(M, K, N, r, L, dt, M))
    big = torch.full((L,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    assert torch.equal(w4.lora_add(Y.clone(), X, ids, A, B, ranks=big), w4.lora_add(Y.clone(), X, ids, A, B))
    assert torch.equal(w4.lora_add(Y.clone(), X, ids, A, B, ranks=-big), Y)


@pytest.mark.parametrize("r", [3, 7, 8, 9, 15, 31, 33, 61, 100, 127, 201, 255])
@pytest.mark.parametrize("M,K", [(4, 97), (60, 131), (260, 300)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_pieces_that_share_ranks(r, M, K, dt):
    """Ranks and lengths that end inside a piece of 8, with NaN behind each adapter's
    own rank, in a row without an adapter, and in the first row of a tile."""
    N, own = 139, [r, r - 1, 1, max(r - 8, 1), max(r - 9, 2), 0]
    X, A, B, scales, ids, _, Y = make(M, K, N, r, 6, dt, M + r)
    ids = (torch.arange(M) % 7 - 1).int()  # (row 0 has none)
    ranks = torch.tensor(own, dtype=torch.int32)
    want, bound = formula(X, A, B, scales, ids, ranks, Y)
    for a, n in enumerate(own):
        A[a, n:], B[a, :, n:] = math.nan, math.nan
    X[ids < 0] = math.nan
    c = cuda(X, A, B, scales, ids, ranks)
    y = w4.lora_add(Y.cuda(), c[0], c[4], c[1], c[2], scales=c[3], ranks=c[5])
    close(y, want, bound)
    assert torch.equal(y.cpu()[ids < 0], Y[ids < 0])


@pytest.mark.parametrize("M,r", [(2, 8), (50, 16), (300, 20)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_strided_and_shifted(M, r, dt):
    """Slices of wider rows (columns beside them stay) and operands at addresses
    that are aligned to their elements only."""
    K, N, L = 320, 192, 3
    X, A, B, scales, ids, ranks, Y = make(M, K, N, r, L, dt, M + r)
    want, bound = formula(X, A, B, scales, ids, None, Y)
    X, A, B, scales, ids, Y = cuda(X, A, B, scales, ids, Y)

    def wide(t, left, right):
        w = torch.full((M, left + t.shape[1] + right), math.nan, dtype=t.dtype, device="cuda")
        w[:, left:left + t.shape[1]] = t
        return w, w[:, left:left + t.shape[1]]

    def shift(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.flatten()
        return b[1:].view(t.shape)

    base = w4.lora_add(Y.clone(), X, ids, A, B, scales=scales)
    close(base, want, bound)
    for left, right in ((8, 8), (4, 0), (1, 2)):
        (wx, x), (wy, y) = wide(X, left, right), wide(Y, left, right)
        w4.lora_add(y, x, ids, A, B, scales=scales)
        close(y, want, bound)
        assert wy[:, :left].isnan().all() and wy[:, left + N:].isnan().all()
    for one in ("Y", "X", "A", "B", "scales", "ids"):
        t = dict(Y=Y.clone(), X=X, A=A, B=B, scales=scales, ids=ids)
        t[one] = shift(t[one])
        close(w4.lora_add(t["Y"], t["X"], t["ids"], t["A"], t["B"], scales=t["scales"]), want, bound)


def test_large_values_and_small_ones():
    """The splitting of fp32 values into terms holds from the smallest normal
    values to the largest."""
    X = torch.zeros((6, 64))
    X[0, :2] = torch.tensor([3.4e38, -3.3999e38])
    X[1, 0] = 1.1754944e-38
    X[2, :3] = torch.tensor([1 + 2.0 ** -23, 2.0 ** -12 + 2.0 ** -30, 1 / 3])
    X[3, 5] = -1e30
    X[4, 63] = 16777215.0
    A = torch.zeros((1, 8, 64))
    A[0, 0] = 1.0
    B = torch.zeros((1, 16, 8))
    B[0, :, 0] = 1.0
    y = torch.zeros((6, 16), device="cuda")
    w4.lora_add(y, X.cuda(), torch.zeros(6, dtype=torch.int32, device="cuda"), A.bfloat16().cuda(),
                B.bfloat16().cuda())
    want = X.double().sum(1)
    assert ((y.double().cpu() - want[:, None]).abs() <= 6 * U * X.double().abs().sum(1)[:, None]).all()


def test_a_pool_beyond_32_bits():
    L, r, K, N = 70, 256, 131071, 64
    A = torch.zeros((L, r, K), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    A[-1] = (torch.randn((r, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    B = torch.randn((L, N, r), generator=g, device="cuda").bfloat16()
    X = torch.randn((2, K), generator=g, device="cuda")
    ids = torch.tensor([L - 1, 3], dtype=torch.int32, device="cuda")
    y = w4.lora_add(torch.zeros((2, N), device="cuda"), X, ids, A, B)
    x, ad, bd = X[0].double(), A[-1].double(), B[-1].double()
    d, mag = (x @ ad.T) @ bd.T, (x.abs() @ ad.abs().T) @ bd.abs().T
    assert ((y[0].double() - d).abs() <= (K + r + 64) * U * mag).all() and not y[1].any()


def test_refusals():
    X, A, B, scales, ids, ranks, Y = cuda(*make(3, 64, 32, 8, 2, torch.float32, 1, True))
    for kw, what in ((dict(Y=Y[:2]), "rows"), (dict(ids=ids[:2]), "ids must have shape"),
                     (dict(A=A[0]), "A must be a 3-D"), (dict(B=B[:1]), "B must have shape"),
                     (dict(A=A[..., :32].contiguous()), "A must have shape"),
                     (dict(scales=scales[:1]), "scales must have shape"), (dict(ranks=ranks[:1]), "ranks must have shape"),
                     (dict(X=X.t()), "contiguous"), (dict(Y=Y.bfloat16()), "Y must be"), (dict(X=X.half()), "X must be"),
                     (dict(A=A.float()), "A must be"), (dict(ids=ids.long()), "ids must be"),
                     (dict(workspace=torch.empty(8, device="cuda")), "workspace must be")):
        t = dict(Y=Y, X=X, ids=ids, A=A, B=B, scales=scales, ranks=ranks)
        t.update(kw)
        with pytest.raises((ValueError, TypeError), match=what):
            w4.lora_add(**t)
    with pytest.raises(w4.W4Error):
        w4.lora_add(Y, X, ids, A, B, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(w4.W4Error):
        w4.lora_add(Y[:0], X[:0], ids[:0], A, B)
    with pytest.raises(w4.W4Error):
        w4.lora_add(Y[:1].expand(3, 32), X, ids, A, B)


@pytest.mark.parametrize("M", [5, 200])
def test_captured_and_on_another_stream(M):
    """Two captured calls share one workspace, replayed between eager calls."""
    X, A, B, scales, ids, ranks, Y = cuda(*make(M, 512, 256, 16, 4, torch.float32, M))
    work = torch.empty(w4.lora_workspace_bytes(M, 512, 256, 16), dtype=torch.uint8, device="cuda")
    want = w4.lora_add(Y.clone(), X, ids, A, B, scales=scales)
    side = torch.cuda.Stream()
    y = Y.clone()
    side.wait_stream(torch.cuda.current_stream())
    w4.lora_add(y, X, ids, A, B, scales=scales, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    out = [Y.clone(), Y.clone()]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w4.lora_add(out[i], X, ids, A, B, scales=scales, workspace=work)
        graphs.append(g)
    for k in range(3):
        ids.copy_((ids + 1) % 4)
        base = torch.full_like(Y, float(k))
        want = w4.lora_add(base.clone(), X, ids, A, B, scales=scales)
        for i in range(2):
            out[i].copy_(base)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(out[i], want)
            w4.lora_add(base[:1].clone(), X[:1], ids[:1], A, B, workspace=work)


@pytest.mark.parametrize("M,N,L", [(1200007, 8, 3), (2100001, 4, 1), (2, 1200000, 2)])
def test_many_rows_or_channels(M, N, L):
    """More tiles than a grid dimension holds, and a long row."""
    K, r = 8, 8
    g = torch.Generator(device="cuda").manual_seed(M)
    X = torch.randn((M, K), generator=g, device="cuda")
    A = torch.randn((L, r, K), generator=g, device="cuda").bfloat16()
    B = torch.randn((L, N, r), generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    Y = torch.randn((M, N), generator=g, device="cuda")
    y = w4.lora_add(Y.clone(), X, ids, A, B)
    low = (X.double() @ A.double().view(L * r, K).T).view(M, L, r)
    mag = (X.double().abs() @ A.double().abs().view(L * r, K).T).view(M, L, r)
    take = (ids[:, None] == torch.arange(L, device="cuda"))[..., None]
    Bd = B.double().transpose(1, 2).reshape(L * r, N)
    d = torch.where(take, low, 0.0).view(M, -1) @ Bd
    e = torch.where(take, mag, 0.0).view(M, -1) @ Bd.abs()
    assert ((y.double() - Y.double() - d).abs() <= (K + r + 64) * U * e + 2 * U * (Y.double().abs() + d.abs())).all()
