"""Why angles are taken in 64 bits: what 32 bits lose of them (no GPU needed)."""
import math

import numpy as np

import int4_weight_quantized_amd as w4


def test_what_fp32_loses_of_an_angle():
    """At position 10^6 about a hundredth of a turn, nearly a tenth of a radian; fp64
    keeps 10^-10 of a turn."""
    p = 10 ** 6
    turns = w4.rope_frequencies(128)[0].tolist()
    lost = max(abs(float(np.float32(p) * np.float32(t)) - p * t) for t in turns)
    assert 0.01 < lost < 0.017 and 0.06 < 2 * math.pi * lost < 0.11
    assert max(math.ulp(p * t) for t in turns) < 1e-10
