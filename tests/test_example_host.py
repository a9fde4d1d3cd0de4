"""What the served block keeps beside the cache: each slot's adapter through forks
and retirement, in plain tensors (no GPU needed)."""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_layer  # noqa: E402


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_forks_hand_on_adapters():
    """Granted forks alone, as the call reports them: slots outside the table, running
    children and children named again are not granted and change nothing."""
    a = ints(4, -1, 7, 2)
    decode_layer.hand_on(a, ints(0, 2), ints(1, 3), ints(1, 1))
    assert a.tolist() == [4, 4, 7, 7]
    a = ints(4, -1, 7, 2)
    decode_layer.hand_on(a, ints(2, 0, 0, 99, 0, -1), ints(1, 1, 3, 0, -1, 4), ints(1, 0, 0, 0, 0, 0))
    assert a.tolist() == [4, 7, 7, 2]
    a = ints(5)
    decode_layer.hand_on(a, ints(0, 1), ints(1, 0), ints(0, 0))
    assert a.tolist() == [5]
    a = ints(4, 9, -1)  # parents are as they were before the call
    decode_layer.hand_on(a, ints(0, 1), ints(1, 2), ints(1, 1))
    assert a.tolist() == [4, 4, 9]


def test_retired_slots_name_no_adapter():
    a = ints(4, 1, 7, 2)
    decode_layer.drop(a, ints(2, 0, 2, -1, 4, 2 ** 31 - 1, -2 ** 31))
    assert a.tolist() == [-1, 1, -1, 2]


def test_rows_of_a_padded_batch():
    """Rows before the first sequence and behind the last have no adapter, and
    sequences of no rows take none."""
    f = decode_layer.of_rows
    assert f(ints(7, 3), ints(0, 2, 5), 5).tolist() == [7, 7, 3, 3, 3]
    assert f(ints(7, 3), ints(1, 2, 4), 6).tolist() == [-1, 7, 3, 3, -1, -1]
    assert f(ints(7, 3, -1, 5), ints(0, 0, 2, 3, 3), 4).tolist() == [3, 3, -1, -1]
    assert f(ints(7), ints(2, 2), 3).tolist() == [-1, -1, -1]
    assert f(ints(7), ints(0, 1), 1).dtype == torch.int32
