"""The usage that the README shows, run as it stands (GPU)."""
import os
import re

import pytest
import torch

import int4_weight_quantized_amd as w4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def test_usage():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        code, = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    K, N, r, slots, heads, D = 256, 192, 16, 3, 2, 64
    names = dict(W=normal(K, N), X=normal(slots, K), b=normal(N), layers=1, pages=12, kv_heads=heads, head_dim=D,
                 table=torch.full((slots, 4), -1, dtype=torch.int32, device="cuda"), lens=ints(0, 0, 0),
                 refs=torch.zeros(12, dtype=torch.int32, device="cuda"), add=ints(2, 1, 1), q=normal(slots, 4, D),
                 k=normal(slots, heads, D), v=normal(slots, heads, D), x=normal(slots, K), h=3 * normal(slots, K),
                 weight=1 + 0.1 * normal(K), ids=ints(1, -1, 0), A=(normal(2, r, K) / 16).bfloat16(),
                 B=normal(2, N, r).bfloat16())
    exec(code, names)
    assert names["granted"].tolist() == [1, 1, 1] and names["o"].isfinite().all()
    # the adapters' rows are the product's: the norm of the sum
    h = names["h"].cpu()
    n = h * (1.0 / torch.sqrt((h.double() ** 2).mean(-1, keepdim=True) + 1e-6)).float() * names["weight"].cpu()
    want = w4.w4a8_linear(n.cuda(), names["packed"], names["sw"]).double().cpu()
    bound = 2 * U * want.abs()
    for m, a in ((0, 1), (2, 0)):
        A, B = names["A"][a].double().cpu(), names["B"][a].double().cpu()
        d = (n[m].double() @ A.T) @ B.T
        want[m] += d
        bound[m] += (K + r + 64) * U * ((n[m].double().abs() @ A.abs().T) @ B.abs().T) + 2 * U * d.abs()
    assert ((names["y"].double().cpu() - want).abs() <= bound).all()
