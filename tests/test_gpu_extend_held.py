"""Sequence extension with held pages (ps_extend_held_sequences): sequences that take tokens back,
against a plain implementation, and in a loop that verifies drafts."""
import random

import pytest
import torch

from paged_kv_attention_18_gb300 import binding
from tests.held_ref import Held, pages_of

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Both:
    """The plain form and the call, side by side."""

    def __init__(self, *args, **kw):
        self.ref = Held(*args, **kw)
        c = self.ref
        self.bt, self.lens, self.held = i32(c.tables), i32(c.lens), i32(c.held)
        self.free = i32(c.stack + [-9] * (c.nb - len(c.stack)))
        self.count = i32([len(c.stack)])

    def step(self, news, T, window=0, sinks=0, error=None):
        c, B = self.ref, len(news)
        want = c.step(news, T, window, sinks)
        qsl, slots, pos = (torch.full((n,), -7, dtype=torch.int32, device="cuda")
                           for n in (B + 1, T, T))
        binding.extend_sequences(self.bt, self.lens, i32(news), self.free, self.count, c.nb, qsl,
                                 slots, pos, window, sinks, held_pages=self.held)
        torch.cuda.synchronize()
        code = binding.device_error()
        assert code in want[3] if want[3] else code == 0, (code, want[3])
        assert error is None or code == error
        assert [qsl.tolist(), slots.tolist(), pos.tolist()] == list(want[:3])
        self.check()

    def shorten(self, by):
        self.ref.shorten(by)
        self.lens -= i32(by)

    def check(self):
        c, n = self.ref, int(self.count)
        assert self.bt.tolist() == c.tables
        assert self.lens.tolist() == c.lens and self.held.tolist() == c.held
        assert self.free[:n].tolist() == c.stack
        c.check_blocks()


@pytest.mark.parametrize("B", [1, 9, 600, 2100])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5), (48, 33)])
def test_steps_with_tokens_taken_back(B, window, sinks):
    """Steps of up to 40 tokens of which any number goes again (no more than a window allows for),
    sequences that end and begin, more asked for than there are blocks or room."""
    r = random.Random(B + window)
    lens = [r.randint(0, 90) for _ in range(B)]
    nb = sum(pages_of(L) for L in lens) + 2 * B + 3
    c = Both(lens, 14, 2 * B + 3, nb)
    for step in range(14):
        room = [14 * 16 - L for L in c.ref.lens]
        news = [min(r.choice([0, 1, 1, 5, 17, 40]), n) for n in room]
        for b in range(B):
            if r.random() < (0.05 if B > 1 else 0.2):
                news[b] = -1
        T = max(sum(max(n, 0) for n in news) - (7 if step % 5 == 4 else 0), 0)
        before = list(c.ref.lens)
        c.step(news, T, window and window + 40, sinks)
        c.shorten([r.randint(0, max(a - b, 0)) for a, b in zip(c.ref.lens, before)])
    c.step([-1] * B, 0)
    assert len(c.ref.stack) == nb and c.ref.held == [0] * B


def test_pages_reserved_ahead():
    """Pages beyond the length's are the caller's to give: the next tokens take no others."""
    c = Both([0, 5, 32], 8, 4, 20, extra=(3, 0, 2))
    tables = [list(t) for t in c.ref.tables]
    c.step([48, 11, 32], 100)
    assert c.ref.tables == tables and len(c.ref.stack) == 4
    c.step([1, 1, 1], 3)
    assert len(c.ref.stack) == 1


def test_bad_counts_of_pages():
    """Fewer pages than the length's, more than the table's: left out, the others served."""
    for held in (1, 0, -1, -2 ** 31, 9, 2 ** 31 - 1):
        for n in (1, 0, -1):
            c = Both([20, 20, 20], 8, 10, 16)
            c.ref.held[1], c.held[1] = held, held
            want = c.ref.step([1, n, 1], 5)
            qsl, slots, pos = i32([0] * 4), i32([0] * 5), i32([0] * 5)
            binding.extend_sequences(c.bt, c.lens, i32([1, n, 1]), c.free, c.count, 16, qsl, slots,
                                     pos, held_pages=c.held)
            torch.cuda.synchronize()
            assert binding.device_error() == 3 and want[3] == {3}
            assert [qsl.tolist(), slots.tolist(), pos.tolist()] == list(want[:3])
            assert c.bt.tolist() == c.ref.tables and c.lens.tolist() == [21, 20, 21]
            assert c.held.tolist() == [2, held, 2]


def test_largest_batch():
    r = random.Random(3)
    lens = [r.randint(0, 70) for _ in range(8192)]
    nb = sum(pages_of(L) for L in lens) + 9000
    c = Both(lens, 7, 9000, nb)
    for _ in range(2):
        news = [r.randint(0, 5) for _ in lens]
        c.step(news, sum(news))
        c.shorten([r.randint(0, n) for n in news])


def test_the_argument():
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    bt, one, four = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), i32([0]), i32([0] * 4)
    for bad in (four, z.long(), z[:2], torch.zeros(6, dtype=torch.int32, device="cuda")[::2],
                z.cpu(), z):  # (the last: the lengths themselves)
        with pytest.raises(binding.PagedServeError):
            binding.extend_sequences(bt, z, torch.zeros_like(z), one, one.clone(), 8, four, z, z,
                                     held_pages=bad)


def verify_loop(captured, window, B=7, k=5, V=11, steps=70):
    """Sequences that verify k drafts a step: a token and its drafts are added, the accepted ones
    stay, the rest is taken back. Returns what happened, step by step, and whether the window gave
    blocks back."""
    g = torch.Generator().manual_seed(5)
    nb, width = 40, 24
    bt = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens, held = i32([0] * B), i32([0] * B)
    free, count = torch.randperm(nb, generator=g).int().cuda(), i32([nb])
    news = i32([k + 1] * B)
    qsl, slots, pos = i32([0] * (B + 1)), i32([0] * (B * (k + 1))), i32([0] * (B * (k + 1)))
    probs = torch.zeros(B, k + 1, V, device="cuda")
    drafts, bits = i32([[0] * k] * B), i32([[0] * (k + 1)] * B)
    ws = torch.empty(max(binding.lib().ps_spec_accept_workspace_size(B, k, V), 256),
                     dtype=torch.uint8, device="cuda")

    def step():
        binding.extend_sequences(bt, lens, news, free, count, nb, qsl, slots, pos, window=window,
                                 sinks=4, held_pages=held)
        _, accepted = binding.spec_accept(probs, drafts, bits, workspace=ws)
        added = qsl[1:] - qsl[:-1]
        lens.sub_((added - 1 - accepted).clamp(min=0).int())

    graph, history, gaps = None, [], False
    for i in range(steps):
        probs.copy_(torch.softmax(torch.randn(B, k + 1, V, generator=g) * 2, -1))
        drafts.copy_(torch.randint(0, V, (B, k), generator=g))
        bits.copy_(torch.randint(-(1 << 31), 1 << 31, (B, k + 1), generator=g))
        n = torch.full((B,), k + 1)
        n[torch.rand(B, generator=g) < 0.04] = -1  # some end, their places begin anew
        news.copy_(n)
        if captured and i >= 2:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        stack = free[:int(count)].tolist()
        table = [e for e in bt.flatten().tolist() if e >= 0]
        assert sorted(table + stack) == list(range(nb)), i  # every block in one place
        for b in range(B):
            assert pages_of(int(lens[b])) <= int(held[b]) <= pages_of(int(lens[b]) + k)
            assert all(e < 0 for e in bt[b, int(held[b]):].tolist())
            gaps = gaps or -1 in bt[b, :int(held[b])].tolist()
            assert int(lens[b]) == 0 or int(bt[b, (int(lens[b]) - 1) // 16]) >= 0
        history.append((bt.clone(), lens.clone(), slots.clone(), stack))
    news.fill_(-1)
    step()
    torch.cuda.synchronize()
    assert sorted(free[:int(count)].tolist()) == list(range(nb))
    assert lens.tolist() == held.tolist() == [0] * B
    return history, gaps


@pytest.mark.parametrize("window", [48, 20])
def test_drafts_verified_until_all_end(window):
    """A pool that would drain with every rejected page does not; captured, it goes the same way."""
    (eager, gaps), (captured, _) = verify_loop(False, window), verify_loop(True, window)
    assert gaps or window > 20
    for a, b in zip(eager, captured):
        assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3])) and a[3] == b[3]
