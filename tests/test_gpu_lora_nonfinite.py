"""Adapters with infinities and NaN in what takes part, with sums beyond fp32, and with
values at the lower end of the range (GPU).  The contract: outputs that one of the
former reaches are infinite or NaN, never a number; all others are the formula's."""
import math

import pytest
import torch

import int4_weight_quantized_amd as w4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
INF, NAN = math.inf, math.nan


def make(M, K, N, r, dt, seed):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn((M, K), generator=g).to(dt)
    A = (torch.randn((3, r, K), generator=g) * K ** -0.5).bfloat16()
    B = torch.randn((3, N, r), generator=g).bfloat16()
    return X, A, B, (torch.arange(M) % 4 - 1).int(), torch.randn((M, N), generator=g)


def check(X, A, B, ids, Y):
    """Against the formula in 64 bits, where sums beyond fp32 are infinite."""
    y = w4.lora_add(Y.cuda(), X.cuda(), ids.cuda(), A.cuda(), B.cuda()).double().cpu()
    want, bound = Y.double().clone(), torch.zeros(Y.shape, dtype=torch.float64)
    for a in range(A.shape[0]):
        rows = (ids == a).nonzero()[:, 0]
        x, ad, bd = X[rows].double(), A[a].double(), B[a].double()
        low = x @ ad.T
        low = torch.where(low.abs() > 3.5e38, low * INF, low)
        d = low @ bd.T
        e = (x.abs() @ ad.abs().T) @ bd.abs().T
        want[rows] += d
        bound[rows] = (X.shape[1] + A.shape[1] + 64) * U * e + 2 * U * (Y[rows].double().abs() + d.abs())
    fine = want.isfinite()
    assert not y[~fine].isfinite().any()
    assert ((y - want).abs()[fine] <= bound[fine]).all()
    return fine


@pytest.mark.parametrize("M,K,N,r", [(5, 64, 48, 8), (5, 65, 47, 7), (40, 1040, 260, 40), (300, 264, 136, 20), (300, 263, 131, 33)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_what_is_not_finite_stays_where_it_belongs(M, K, N, r, dt):
    base = make(M, K, N, r, dt, M + K)
    assert check(*base).all()
    for bad in (INF, -INF, NAN):
        X, A, B, ids, Y = (t.clone() for t in base)
        X[1, K - 1] = X[4, 0] = bad  # (row 4 has no adapter)
        fine = check(X, A, B, ids, Y)
        assert not fine[1].any() and fine[torch.arange(M) != 1].all()
        X, A, B, ids, Y = (t.clone() for t in base)
        A[1, r - 1, K // 2] = bad
        fine = check(X, A, B, ids, Y)
        assert not fine[ids == 1].any() and fine[ids != 1].all()
        X, A, B, ids, Y = (t.clone() for t in base)
        B[2, N - 2, 0] = bad
        fine = check(X, A, B, ids, Y)
        assert not fine[ids == 2, N - 2].any() and int((~fine).sum()) == int((ids == 2).sum())


@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_sums_beyond_fp32(M, dt):
    K, N, r = 64, 32, 8
    X, A, B, ids, Y = make(M, K, N, r, dt, 1)
    ids[2] = 1
    X[2] = 3e38
    A[1] = 1.0
    B[1] = 1.0
    fine = check(X, A, B, ids, Y)
    assert not fine[2].any() and fine[torch.arange(M) != 2].all()


@pytest.mark.parametrize("M", [20, 300])
def test_the_lower_end_of_the_range(M):
    """Values of X, and of X A^T, from 2^-100 to the smallest: each is off by its bits
    below 2^-133, times the other factors, and by rounding."""
    e = [-100, -110, -112, -120, -126, -127, -130, -133, -140, -149]
    v = torch.tensor([2.0 ** k * (1 + 2.0 ** -23) for k in e], dtype=torch.float64).float()
    X = torch.zeros((M, 64))
    X[:len(e), 3] = v
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    for first, second in ((2.0 ** 100, 1.0), (1.0, 2.0 ** 100)):
        A, B = torch.zeros((1, 8, 64)), torch.zeros((1, 16, 8))
        A[0, 0], B[0, :, 0] = first, second
        y = w4.lora_add(torch.zeros((M, 16), device="cuda"), X.cuda(), ids, A.bfloat16().cuda(), B.bfloat16().cuda())
        want = X[:, 3].double()[:, None] * 2.0 ** 100
        assert ((y.double().cpu() - want).abs() <= 2.0 ** (100 - 133) + 4 * U * want).all()
