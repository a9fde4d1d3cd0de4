"""Each variant of the norms', rotations' and adapters' kernels, chosen by the sizes and
addresses that it is for, is the one that runs, and gives the formula's values (GPU)."""
import pytest
import torch

import int4_weight_quantized_amd as w4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def shift(t):
    """The same values at an address that is aligned to elements only."""
    b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    b[1:] = t.flatten()
    return b[1:].view(t.shape)


def normal(*shape, seed=1):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("K,off,path", [(4096, False, "rms_norm"), (4096, True, "rms_norm_odd"), (4098, False, "rms_norm_odd"),
                                        (32768, False, "rms_norm"), (32776, False, "rms_norm_long"),
                                        (40000, True, "rms_norm_long")])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_norm(K, off, path, dt):
    x = normal(3, K).to(dt)
    x = shift(x) if off else x
    want = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6)
    y, _ = w4.rms_norm(x, None, 1e-6, dtype=torch.float32)
    assert w4.w4_last_path() == path
    assert ((y.double() - want).abs() <= 4 * U * want.abs()).all()  # r, its mean's share, the product
    w4.a8_rms_norm(x, None, 1e-6)
    assert w4.w4_last_path() == path


@pytest.mark.parametrize("D,off,suffix", [(64, False, ""), (80, False, "_cached"), (64, True, "_odd"), (80, True, "_odd")])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rotation(D, off, suffix, dt):
    T = 20
    rope = w4.Rope(D)
    q, k = normal(T, 4, D).to(dt), normal(T, 2, D, seed=2).to(dt)
    if off:
        q, k = shift(q), shift(k)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    a = 2 * torch.pi * ((pos.double()[:, None] * rope.turns) % 1.0)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    lo, hi = q[..., :D // 2].double(), q[..., D // 2:].double()
    want = torch.cat([lo * c - hi * s, hi * c + lo * s], -1)
    bound = (4 * U + (0 if dt == torch.float32 else 2.0 ** -8 * (1 + 4 * U))) * torch.cat([lo.abs() + hi.abs()] * 2, -1)
    y = w4.rope_rotate(q, pos, rope)
    assert w4.w4_last_path() == "rope_rotate" + suffix
    assert ((y.double() - want).abs() <= bound).all()
    cache = w4.KVCache.empty(1, 2, 2, 16, D, torch.int8)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    start, cu = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0], [0, T]))
    z = w4.kv_append_rope(cache, 0, q, k, k, table, start, rope, cu)
    assert w4.w4_last_path() == "kv_append_rope" + suffix
    assert torch.equal(z, y)


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("odd", ["", "x", "b", "xb", "y", "xy", "by", "xby"])
@pytest.mark.parametrize("how", ["sizes", "addresses"])
def test_adapters(M, dt, odd, how):
    sizes = how == "sizes"
    K, r, N = (259 if sizes and "x" in odd else 264), (13 if sizes and "b" in odd else 16), (131 if sizes and "y" in odd else 132)
    X, A, B, Y = normal(M, K).to(dt), normal(2, r, K, seed=2).bfloat16() / 16, normal(2, N, r, seed=3).bfloat16(), normal(M, N, seed=4)
    ids = (torch.arange(M, device="cuda") % 3 - 1).int()
    if not sizes:
        X, B, Y = (shift(t) if c in odd else t for c, t in (("x", X), ("b", B), ("y", Y)))
    want, bound = Y.double(), 2 * U * Y.double().abs()
    for a in range(2):
        m = ids == a
        low, mag = X[m].double() @ A[a].double().T, X[m].double().abs() @ A[a].double().abs().T
        d, e = low @ B[a].double().T, mag @ B[a].double().abs().T
        want[m] += d
        bound[m] += (K + r + 64) * U * e + 2 * U * d.abs()
    y = w4.lora_add(Y, X, ids, A, B)
    assert w4.w4_last_path() == ("lora_odd_" + odd if odd else "lora")
    assert ((y.double() - want).abs() <= bound).all()
