"""The attention's workspace for a call covers every smaller call (no GPU needed)."""
import random

import pytest

import int4_weight_quantized_amd as w4

SHAPES = [(32, 8, 128), (64, 8, 128), (4, 1, 256), (12, 4, 64), (8, 8, 80), (1, 1, 16), (40, 2, 128), (300, 300, 64)]


@pytest.mark.parametrize("hq,heads,D", SHAPES)
def test_covers_smaller_calls(hq, heads, D):
    f = w4.kv_attention_workspace_bytes
    r = random.Random(hq * D)
    for T, B in [(8192, 1), (8192, 64), (256, 1), (37, 3), (1 << 18, 16), (64, 64), (5000, 200)]:
        most = f(T, B, hq, heads, D)
        assert most > 0
        small = [(1, 1), (37, 1), (128, 1), (256, 1), (T, 1), (1, B), (max(T // 2, 1), B)]
        small += [(r.randint(1, T), r.randint(1, B)) for _ in range(200)]
        small += [(r.randint(1, min(T, 600)), r.randint(1, B)) for _ in range(200)]
        for t, b in small:
            if t <= T:
                assert f(t, b, hq, heads, D) <= most, (t, b, T, B)


@pytest.mark.parametrize("hq,heads,D", SHAPES)
def test_is_not_wasteful(hq, heads, D):
    """No more than the parts of one call that fills the chip: at most 512
    workgroups of 128 rows, or one part of decode for each of them."""
    rows = 512 * 128
    bound = max(rows * (D + 4) * 4, 768 * (16 + 2 * 16 * (256 + 4) * 4))
    for T in (1, 100, 1000, 10000, 1 << 18):
        assert w4.kv_attention_workspace_bytes(T, 1, hq, heads, D) <= bound
