"""Defaults of the stretched frequencies' ramps (no GPU needed)."""
import pytest

import int4_weight_quantized_amd as w4


@pytest.mark.parametrize("scaling,fast", [("yarn", 32.0), ("bands", 4.0)])
def test_the_ramp_without_bounds(scaling, fast):
    """Each rule's own: by the pair's index from 32 turns to 1, by its turns from 4 to 1."""
    kw = dict(scaling=scaling, factor=8.0, context=8192)
    t, m = w4.rope_frequencies(128, 500000.0, **kw)
    u, n = w4.rope_frequencies(128, 500000.0, fast=fast, slow=1.0, **kw)
    other, _ = w4.rope_frequencies(128, 500000.0, fast=36.0 - fast, slow=1.0, **kw)
    assert t.tolist() == u.tolist() and m == n and t.tolist() != other.tolist()


def test_bands_share_of_each_pair():
    """A pair of more than 4 turns within the context stays, one of less than one is
    divided by the factor."""
    p = w4.rope_frequencies(64)[0]
    t = w4.rope_frequencies(64, scaling="bands", factor=8.0, context=2048)[0]
    for a, b in zip(p.tolist(), t.tolist()):
        turns = 2048 * a
        keep = min(max((turns - 1) / 3, 0.0), 1.0)
        assert b == pytest.approx(a * (keep + (1 - keep) / 8), rel=1e-12)


@pytest.mark.parametrize("rot", [-2, 0, 7, 514, 1 << 45])
def test_sizes_are_refused_before_memory_is_taken(rot):
    with pytest.raises(w4.W4Error):
        w4.rope_frequencies(rot)
    assert w4.rope_frequencies(512)[0].shape == (256,)
