"""Sequence extension (ps_extend_sequences) against a plain implementation."""
import pytest
import torch

from paged_kv_attention_18_gb300 import binding
from tests import loop_ref as R

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Cache:
    """Tables over a pool, its free blocks on a stack; NaN-like marks in what is not to change."""

    def __init__(self, lens, width, spare, seed, capacity=None):
        g = torch.Generator().manual_seed(seed)
        held = [max(0, -(-L // 16)) for L in lens]
        self.nb = max(sum(held) + spare, 1)
        ids = torch.randperm(self.nb, generator=g).tolist()
        self.bt = [[-9] * width for _ in lens]
        for row, n in zip(self.bt, held):
            for q in range(min(n, width)):
                row[q] = ids.pop()
        self.free = ids[:spare] + [-9] * ((capacity or self.nb) - spare)
        self.count, self.lens = spare, list(lens)

    def step(self, news, T=None, window=0, sinks=0, separate=False, error=None, **kw):
        T = sum(max(n, 0) for n in news) if T is None else T
        B = len(self.lens)
        want = R.extend(self.bt, self.lens, news, self.free, self.count, T, self.nb, window, sinks)
        bt, lens, free, count = i32(self.bt), i32(self.lens), i32(self.free), i32([self.count])
        qsl, slots, pos = (torch.full((n,), -7, dtype=torch.int32, device="cuda")
                           for n in (B + 1, T, T))
        outs = {}
        if separate:
            outs = dict(out_seq_lens=torch.full_like(lens, -7),
                        out_free_count=torch.full_like(count, -7))
        binding.extend_sequences(bt, lens, i32(news), free, count, self.nb, qsl, slots, pos, window,
                                 sinks, **outs, **kw)
        torch.cuda.synchronize()
        code = binding.device_error()
        assert code in want[7] if want[7] else code == 0, (code, want[7])
        if error is not None:
            assert code == error
        if separate:
            assert lens.tolist() == self.lens and count.tolist() == [self.count]
            lens, count = outs["out_seq_lens"], outs["out_free_count"]
        assert bt.tolist() == want[0]
        assert lens.tolist() == want[1]
        assert count.tolist() == [want[3]]
        assert free.tolist() == want[2]
        assert qsl.tolist() == want[4]
        assert slots.tolist() == want[5]
        assert pos.tolist() == want[6]
        self.bt, self.lens, self.free, self.count = want[0], want[1], want[2], want[3]


@pytest.mark.parametrize("separate", [False, True])
@pytest.mark.parametrize("lens,news", [
    ([0], [1]), ([15], [1]), ([16], [1]), ([17], [0]), ([0, 0, 0], [0, 0, 0]),
    ([1, 16, 31, 32, 0], [1, 1, 1, 1, 40]), ([100, 7], [5, 200]),
    ([i % 50 for i in range(600)], [1] * 600),
    ([3 * i for i in range(70)], [i for i in range(70)])])
def test_steps(lens, news, separate):
    need = sum(-(-(a + b) // 16) for a, b in zip(lens, news))
    c = Cache(lens, max(max(a + 3 * b for a, b in zip(lens, news)) // 16 + 1, 1), 3 * need + 2, 1)
    for extra in (0, 5, 0):
        c.step(news, T=sum(news) + extra, separate=separate)


def test_prompts_of_any_length():
    lens, news = [0, 5, 300, 0], [9000, 1, 2049, 12345]
    c = Cache(lens, 800, 1600, 2)
    c.step(news, T=24000)


def test_largest_batch():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 70, (8192,), generator=g).tolist()
    news = torch.randint(0, 5, (8192,), generator=g).tolist()
    c = Cache(lens, 6, 9000, 3)
    c.step(news)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (16, 4), (33, 17), (64, 16), (100, 0)])
def test_a_window_gives_blocks_back(window, sinks):
    """Streams under a window: what falls behind it comes back, step after step, and a pool of the
    window's size is never short."""
    lens = [0, 200, 37, 16 * 40, 5]
    c = Cache(lens, 60, 24, 4)
    for news in ([3, 1, 1, 1, 1], [1, 1, 1, 1, 1], [20, 0, 17, 1, 30], [1, 2, 3, 4, 5], [1] * 5):
        c.step(news, window=window, sinks=sinks)
    for _ in range(40):
        c.step([1, 2, 0, 3, 1], window=window, sinks=sinks)


def test_sequences_end_and_begin():
    c = Cache([40, 16, 0, 100, 33], 10, 3, 5)
    c.step([1, -1, 20, -1, 1])
    c.step([-5, 30, 1, 64, -1])
    c.step([50, -1, -1, -1, -1], window=20, sinks=2)
    assert c.lens == [50, 0, 0, 0, 0]


def test_blocks_that_run_out():
    """Those that need none, or whose blocks are there, are served; the others wait."""
    c = Cache([16, 3, 32, 15, 48], 8, 2, 6)
    c.step([1, 1, 17, 1, 1], error=7)
    assert c.lens == [17, 4, 32, 16, 48]
    # one comes back beside the one left: the two that 32 + 17 tokens need
    c.step([0, -1, 17, 0, 0], error=0)
    assert c.lens == [17, 0, 49, 16, 48] and c.count == 0
    c.step([0, 0, 16, 0, 0], error=7)
    c = Cache([0, 0], 40, 0, 7)
    c.step([1, 0], error=7)


def test_packed_tokens_that_do_not_fit():
    c = Cache([0, 5, 9], 8, 20, 8)
    c.step([4, 6, 3], T=10, error=3)
    assert c.lens == [4, 11, 9]


@pytest.mark.parametrize("at", [0, 2, 700])
def test_bad_sequences(at):
    """A length below 0, a table outgrown, numbers at the end of 32 bits: left out, the rest
    served."""
    for L, n in ((-1, 1), (-5, -1), (100, 29), (129, 0), (2 ** 31 - 1, 1), (5, 2 ** 31 - 1),
                 (2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, 3), (140, -1), (3, -2 ** 31)):
        lens, news = [20] * 701, [1] * 701
        c = Cache(lens, 8, 50, 9)
        c.lens[at], news[at] = L, n
        c.step(news, T=800, window=9, sinks=1, error=None if n == -2 ** 31 else 3)


def test_bad_blocks():
    c = Cache([20, 20, 16], 4, 6, 10)
    c.free[5] = c.nb  # the top of the stack
    c.step([13, 1, 1], error=1)
    c = Cache([20, 20], 4, 6, 11)
    c.bt[1][1] = c.nb + 3
    c.step([1, 1], error=1)
    c = Cache([20, 16], 4, 6, 12)
    c.count = 100
    c.step([1, 1], error=1)
    c = Cache([20, 16], 4, 6, 13)
    c.count = -1
    c.step([1, 0], error=1)
    c = Cache([64, 64], 6, 2, 14, capacity=4)  # more comes back than the stack holds
    c.step([-1, 1], error=1)


def test_everything_at_once():
    """Sequences that end, grow under a window, are bad, go without and do not fit, together."""
    g = torch.Generator().manual_seed(21)

    def ints(lo, hi, n):
        return torch.randint(lo, hi, (n,), generator=g).tolist()

    for B in (7, 130, 900):
        c = Cache(ints(0, 400, B), 30, B // 2 + 3, B)
        for step in range(12):
            news = ints(-1, 6, B)
            for b in ints(0, B, 3):
                news[b] = (-1, 100, 600)[b % 3]
            T = max(sum(max(n, 0) for n in news) - (step % 4) * 5, 0)
            c.step(news, T=T, window=(0, 33, 100)[step % 3], sinks=step % 20)


def test_an_empty_batch():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    qsl, slots, pos = i32([5]), i32([5, 5]), i32([5, 5])
    count = i32([1])
    binding.extend_sequences(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), z, z, i32([3]),
                             count, 8, qsl, slots, pos)
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    assert qsl.tolist() == [0] and slots.tolist() == [-1, -1] and pos.tolist() == [0, 0]
    assert count.tolist() == [1]


def test_slots_are_those_of_slot_mapping():
    c = Cache([100, 3, 47], 30, 60, 15)
    news = [50, 7, 1]
    bt, lens, free, count = i32(c.bt), i32(c.lens), i32(c.free), i32([c.count])
    qsl, slots, pos = i32([0] * 4), i32([0] * 60), i32([0] * 60)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    binding.extend_sequences(bt, lens, i32(news), free, count, c.nb, qsl, slots, pos, stream=stream)
    stream.synchronize()
    again = binding.slot_mapping(bt, lens, qsl, 58, c.nb)
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    assert torch.equal(again, slots[:58]) and slots[58:].tolist() == [-1, -1]
    assert lens.tolist() == [150, 10, 48]


def test_replayed_from_a_graph():
    """A captured decode step advances its sequences in place with every replay."""
    B, width = 40, 12
    c = Cache([3 * b for b in range(B)], width, 130, 16)
    bt, lens, free, count = i32(c.bt), i32(c.lens), i32(c.free), i32([c.count])
    news, qsl = i32([1] * B), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots, pos = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        binding.extend_sequences(bt, lens, news, free, count, c.nb, qsl, slots, pos, 40, 5)
    for _ in range(50):
        want = R.extend(c.bt, c.lens, [1] * B, c.free, c.count, B, c.nb, 40, 5)
        graph.replay()
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        assert bt.tolist() == want[0] and lens.tolist() == want[1] and count.tolist() == [want[3]]
        assert slots.tolist() == want[5] and pos.tolist() == want[6]
        c.bt, c.lens, c.free, c.count = want[0], want[1], want[2], want[3]


def test_shapes():
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    bt, one, four = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), i32([0]), i32([0] * 4)
    good = [bt, z, z, z, one, 8, four, z, z]
    for at, bad in ((1, four), (2, four), (4, z), (6, z), (8, four), (0, z), (1, z.long()),
                    (7, four[::2])):
        args = list(good)
        args[at] = bad
        with pytest.raises(binding.PagedServeError):
            binding.extend_sequences(*args)
    with pytest.raises(binding.PagedServeError):
        binding.extend_sequences(*good, window=-1)
