"""Sequence extension over tables that hold entries outside the pool where blocks are to be given
back: recorded, left as they are, and the blocks around them come back."""
import pytest
import torch

from paged_kv_attention_18_gb300 import binding

pytestmark = pytest.mark.gpu

NB = 40


def extend(tables, lens, news, window=0, sinks=0, held=None):
    """Returns (tables, stack, error code)."""
    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    T = sum(max(n, 0) for n in news)
    bt, free, count = i32(tables), i32([-9] * NB), i32([0])
    qsl, slots, pos = i32([0] * (len(lens) + 1)), i32([0] * T), i32([0] * T)
    binding.extend_sequences(bt, i32(lens), i32(news), free, count, NB, qsl, slots, pos, window,
                             sinks, held_pages=None if held is None else i32(held))
    torch.cuda.synchronize()
    return bt.tolist(), free[:int(count)].tolist(), binding.device_error()


@pytest.mark.parametrize("bad", [NB, NB + 5, 2 ** 31 - 1])
@pytest.mark.parametrize("held", [False, True])
def test_behind_a_window(bad, held):
    """Pages 0 to 4 lie behind the window of 100 tokens; the sinks keep page 0."""
    row = [1, 2, bad, 4, 5, 6, 7]
    for sinks, back, left in ((0, [5, 4, 2, 1], [-1, -1, bad, -1, -1, 6, 7]),
                              (3, [5, 4, 2], [1, -1, bad, -1, -1, 6, 7])):
        got = extend([row], [100], [1], 20, sinks, [7] if held else None)
        assert got == ([left], back, 1)
    # up to the first that is gone
    got = extend([[1, -1, bad, 4, 5, 6, 7]], [100], [1], 20, 0, [7] if held else None)
    assert got == ([[1, -1, bad, -1, -1, 6, 7]], [5, 4], 1)


@pytest.mark.parametrize("bad", [NB, 2 ** 31 - 1])
@pytest.mark.parametrize("at", [0, 3, 33, 39])
def test_of_a_sequence_that_ends(bad, at):
    row = [NB - 1 - q for q in range(40)]
    row[at], row[20] = bad, -1
    got = extend([[0] * 40, row], [1, 640], [0, -1])
    left = [-1] * 40
    left[at] = bad
    back = [e for e in reversed(row) if 0 <= e < NB]
    assert got == ([[0] * 40, left], back, 1)


def test_entries_that_are_not_given_back_do_not_count():
    """Past the length, ahead of the window and among the sinks' nothing is looked at."""
    row = [NB + 1, 2, 3, 4, NB + 2, 6, NB + 3, NB + 4]
    got = extend([row], [80], [0], 20, 5)
    assert got == ([[NB + 1, -1, -1, 4, NB + 2, 6, NB + 3, NB + 4]], [3, 2], 0)
