"""What an adapted row depends on: in calls of one M, K and rank on itself alone, also
where K is summed in several parts; between sizes within the bound of the sums (GPU)."""
import pytest
import torch

import int4_weight_quantized_amd as w4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(M, K, N, r, L, dt):
    g = torch.Generator(device="cuda").manual_seed(K + r)
    X = torch.randn((M, K), generator=g, device="cuda").to(dt)
    A = (torch.randn((L, r, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    B = torch.randn((L, N, r), generator=g, device="cuda").bfloat16()
    Y = torch.randn((M, N), generator=g, device="cuda")
    return X, A, B, torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32), Y


@pytest.mark.parametrize("M,K,r", [(40, 4096, 16), (300, 4095, 20), (4672, 4096, 8), (4673, 4096, 8), (2177, 8192, 16)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_of_one_call_size(M, K, r, dt):
    X, A, B, ids, Y = make(M, K, 24, r, 4, dt)
    y = w4.lora_add(Y.clone(), X, ids, A, B)
    p = torch.randperm(M, generator=torch.Generator().manual_seed(M)).cuda()
    z = w4.lora_add(Y[p].contiguous(), X[p].contiguous(), ids[p].contiguous(), A, B)
    assert torch.equal(y[p], z)
    for m in (0, M // 3, M - 1):
        other, x = torch.full_like(ids, -1), torch.full_like(X, float("nan"))
        other[m], x[m] = ids[m], X[m]
        z = w4.lora_add(Y.clone(), x, other, A, B)
        assert torch.equal(z[m], y[m])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_a_row_in_calls_of_many_sizes(dt):
    """The same first rows in calls on either side of a change of the parts of K."""
    K, r, N, top = 4096, 16, 24, 8161
    X, A, B, ids, Y = make(top, K, N, r, 4, dt)
    n = 17
    x, a, b = X[:n].double(), A[ids[:n].long()].double(), B[ids[:n].long()].double()
    low, mag = (torch.bmm(t(x)[:, None], t(a).transpose(1, 2).contiguous()) for t in (lambda v: v, torch.abs))
    d, e = (torch.bmm(v, t(b).transpose(1, 2).contiguous())[:, 0] for v, t in ((low, lambda v: v), (mag, torch.abs)))
    want, bound = Y[:n].double() + d, (K + r + 64) * U * e + 2 * U * (Y[:n].double().abs() + d.abs())
    seen = []
    for M in (n, 257, 4672, 4673, 8160, 8161):
        y = w4.lora_add(Y[:M].clone(), X[:M], ids[:M], A, B)[:n]
        assert ((y.double() - want).abs() <= bound).all()
        seen.append(y)
    for i, j in ((0, 1), (1, 2)):  # eight parts in each of these
        assert torch.equal(seen[i], seen[j])
