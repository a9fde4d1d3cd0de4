"""CPU model of the direct-to-LDS loads of the adapters' first kernel
(k_lora_down_lds): every lane's address lies inside its row of X or A, every place
inside its stage, no place is written twice, and the operands that a wave reads back
are the 8 values of its row and k-step.  16 lanes that read one piece hit all 64
banks.  (The formulas are those of the kernel, written again.)"""
import itertools

import numpy as np
import pytest

OOB = 0x7FFF0000
STAGE = 128


def loads(fp32, MT, RC, K, k, k1, ranks, ldx, match):
    """{(operand, place in its stage): byte offset in its array or None} of one stage."""
    xrow, arow = STAGE * (4 if fp32 else 2), STAGE * 2
    xloads, aloads = 16 * MT * xrow // 4096, RC
    out = {}
    for wave, lane in itertools.product(range(4), range(64)):
        for i in range(xloads):
            n = (wave * xloads + i) * 64 + lane
            m = n // (xrow // 16)
            xk = ((n % (xrow // 16)) ^ (m % 16)) * (4 if fp32 else 8)
            off = (m * ldx + xk + k) * (4 if fp32 else 2) if match >> m & 1 and k + xk < k1 else None
            at = (wave * xloads + i) * 1024 + 16 * lane
            assert ("x", at) not in out and at + 16 <= 16 * MT * xrow
            out["x", at] = off
        for i in range(aloads):
            n = (wave * aloads + i) * 64 + lane
            j = n // (arow // 16)
            ak = ((n % (arow // 16)) ^ (j % 16)) * 8
            off = (j * K + ak + k) * 2 if j < ranks and k + ak < k1 else None
            at = (wave * aloads + i) * 1024 + 16 * lane
            assert ("a", at) not in out and at + 16 <= 16 * RC * arow
            out["a", at] = off
    return out


def reads(fp32, MT, RC, wave, lane):
    """[(operand, place, row, first k of the stage)] of a wave's lane in one stage."""
    c16, q = lane % 16, lane // 16
    xrow, arow = STAGE * (4 if fp32 else 2), STAGE * 2
    out = [("a", (16 * c + c16) * arow + ((4 * wave + q) ^ c16) * 16, 16 * c + c16, 32 * wave + 8 * q) for c in range(RC)]
    for t in range(MT):
        row = (16 * t + c16) * xrow
        if fp32:
            out += [("x", row + ((8 * wave + 2 * q + h) ^ c16) * 16, 16 * t + c16, 32 * wave + 8 * q + 4 * h) for h in (0, 1)]
        else:
            out.append(("x", row + ((4 * wave + q) ^ c16) * 16, 16 * t + c16, 32 * wave + 8 * q))
    return out


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("MT", [1, 2])
@pytest.mark.parametrize("RC", [1, 2, 4])
@pytest.mark.parametrize("K,k,k1", [(256, 0, 256), (256, 128, 256), (1152, 1024, 1152), (264, 256, 264),
                                    (8, 0, 8), (136, 0, 128), (136, 128, 136)])
def test_stage(fp32, MT, RC, K, k, k1):
    ranks, ldx, match = 16 * RC - 3, K + 8, (1 << 16 * MT) - 1 ^ 0b1010
    got = loads(fp32, MT, RC, K, k, k1, ranks, ldx, match)
    size = 4 if fp32 else 2
    for (what, _), off in got.items():
        if off is None:
            continue
        assert off % 16 == 0 and off < OOB
        if what == "x":  # within its row's K values, of a row that belongs to the adapter
            m, at = divmod(off // size, ldx)
            assert match >> m & 1 and at + 16 // size <= K
        else:
            assert off + 16 <= ranks * K * 2
    for wave, lane in itertools.product(range(4), range(64)):
        for what, at, row, kk in reads(fp32, MT, RC, wave, lane):
            off = got[what, at]
            valid = k + kk < k1 and (match >> row & 1 if what == "x" else row < ranks)
            assert (off is not None) == bool(valid)
            if valid:
                assert off == ((row * ldx if what == "x" else row * K) + k + kk) * (size if what == "x" else 2)
    for wave, q in itertools.product(range(4), range(4)):
        rows = [reads(fp32, MT, RC, wave, 16 * q + c) for c in range(16)]
        for i in range(len(rows[0])):
            assert len({r[i][1] // 16 % 16 for r in rows}) == 16


@pytest.mark.parametrize("fp32", [True, False])
def test_largest_offsets(fp32):
    """A tile's last row at the widest stride, and the longest row of A."""
    size = 4 if fp32 else 2
    assert 31 * (1 << 23) * size + 131071 * size < 0x7F000000
    assert 64 * 131071 * 2 < 0x7F000000
    for n in np.arange(0, 256 * 4 + 1, 64):  # channels of a workgroup at the largest rank
        assert int(n) * 256 * 2 + OOB < 1 << 32
