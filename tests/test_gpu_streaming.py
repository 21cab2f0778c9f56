"""Attention with a window and sinks (ps_paged_attention_streaming) against a plain 64-bit
implementation."""
import pytest
import torch

from paged_kv_attention_18_gb300 import binding
from tests import loop_ref as S
from tests import operator_ref as R

pytestmark = pytest.mark.gpu

DTS = [torch.float16, torch.bfloat16]


class Streams:
    """Sequences [(context, new tokens)] over a random pool. Whatever no row may read holds NaN:
    free blocks, rows past a context, rows between the sinks and the first row's window, whose
    pages have been given back (-1)."""

    def __init__(self, seqs, hq, hkv, d, dt, window, sinks, softcap=0.0, std=1.0, seed=1,
                 spare_columns=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.seqs, self.window, self.sinks, self.softcap = seqs, window, sinks, softcap
        self.d, self.dt, self.scale = d, dt, d ** -0.5
        B, T = len(seqs), sum(n for _, n in seqs)
        pages = [(L + 15) // 16 for L, _ in seqs]
        nb = sum(pages) + 5
        ids = torch.randperm(nb, generator=g, device="cuda").int()
        self.q = (torch.randn(T, hq, d, generator=g, device="cuda") * std).to(dt)
        self.k = torch.randn(nb, 16, hkv, d, generator=g, device="cuda").to(dt)
        self.v = torch.randn(nb, 16, hkv, d, generator=g, device="cuda").to(dt)
        self.bt = torch.full((B, max(max(pages), 1) + spare_columns), -1, dtype=torch.int32,
                             device="cuda")
        at, free = 0, [ids[sum(pages):].long()]
        for b, (L, n) in enumerate(seqs):
            blk = ids[at:at + pages[b]]
            at += pages[b]
            self.bt[b, :pages[b]] = blk
            seen = torch.zeros(16 * pages[b], dtype=torch.bool, device="cuda")
            if n:
                j = torch.arange(16 * pages[b], device="cuda")
                seen = (j < L) & ((j < sinks) | (j > L - n - window) | (window == 0))
            rows = seen.view(-1, 16)
            dead = ~rows
            for pool in (self.k, self.v):
                part = pool[blk.long()]
                part[dead] = float("nan")
                pool[blk.long()] = part
            gone = ~rows.any(1)
            self.bt[b, :pages[b]][gone] = -1
        for f in free:
            self.k[f] = self.v[f] = float("nan")
        self.sl = torch.tensor([L for L, _ in seqs], dtype=torch.int32, device="cuda")
        self.off = [0]
        for _, n in seqs:
            self.off.append(self.off[-1] + n)
        self.qs = torch.tensor(self.off, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        out = torch.full_like(self.q, float("nan"))
        binding.streaming_paged_attention(self.q, self.k, self.v, self.bt, self.sl, self.qs,
                                          self.scale, self.window, self.sinks,
                                          softcap=self.softcap, out=out, **kw)
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        return out

    def check(self, out):
        for b, (L, n) in enumerate(self.seqs):
            if n == 0:
                continue
            a, e = self.off[b], self.off[b + 1]
            pos = torch.arange(L - n, L, device="cuda")
            ref, absv, size, tail = S.attend_stream(
                self.q[a:e], R.gather(self.k, self.bt[b], L), R.gather(self.v, self.bt[b], L), pos,
                self.scale, self.window, self.sinks, self.softcap)
            tol = R.attention_tolerance(ref, absv, size, tail, self.d, self.dt)
            err = (out[a:e].double() - ref).abs()
            assert not (err > tol).any() and torch.isfinite(out[a:e]).all(), \
                (b, L, n, float((err - tol).max()), int((~(err <= tol)).sum()))


DECODES = [(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (300, 1), (2049, 1), (129, 1)]
LONG = [(9000, 1), (5, 1), (700, 1), (33, 4), (12000, 2)]
CHUNKS = [(300, 300), (1, 1), (513, 200), (64, 64), (900, 129), (40, 1)]
BATCHES = {"decodes": DECODES, "long": LONG, "chunks": CHUNKS,
           "small_chunks": [(200, 100), (90, 33)],
           "one": [(1, 1)], "one_long": [(3000, 1)], "one_chunk": [(1500, 1400)],
           "verify": [(500, 5), (61, 5), (5, 5), (2000, 5)],
           "gaps": [(50, 0), (20, 3), (0, 0), (400, 1), (16, 0)],
           "long_chunks": [(5000, 700), (2500, 2500), (800, 30)]}
HEADS = [(12, 2, 128), (8, 8, 64), (7, 1, 128), (14, 2, 64), (40, 2, 64)]
MASKS = [(1, 1), (24, 4), (100, 17), (130, 130), (1000, 16), (20000, 4), (16, 32)]


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_masks(name, hq, hkv, d):
    for i, (window, sinks) in enumerate(MASKS):
        b = Streams(BATCHES[name], hq, hkv, d, DTS[i % 2], window, sinks, seed=i)
        b.check(b.run())


@pytest.mark.parametrize("name", ["decodes", "long", "chunks", "one_chunk", "verify"])
@pytest.mark.parametrize("cap", [15.0, 50.0, 1e3])
@pytest.mark.parametrize("hq,hkv,d", [(12, 2, 128), (14, 2, 64)])
def test_capped_scores(name, cap, hq, hkv, d):
    for dt in DTS:
        b = Streams(BATCHES[name], hq, hkv, d, dt, 70, 20, softcap=cap, std=6.0)
        b.check(b.run())


@pytest.mark.parametrize("sinks", list(range(1, 36)) + [127, 128, 129, 300])
def test_every_place_of_the_sinks(sinks):
    """Sinks that end anywhere in a page, a window that begins anywhere behind or inside them."""
    seqs = [(60 + i, 1) for i in range(34)]
    b = Streams(seqs, 4, 2, 64, torch.bfloat16, 37, sinks)
    b.check(b.run())
    b = Streams([(150, 150), (333, 40)], 4, 2, 64, torch.float16, 37, sinks)
    b.check(b.run())


@pytest.mark.parametrize("count,n,ctx", [(400, 1, 90), (300, 1, 2000), (90, 4, 900), (40, 33, 700)])
def test_large_batches(count, n, ctx):
    """Planned batches: splits of a context among them, whose first lies in the sinks."""
    g = torch.Generator().manual_seed(ctx)
    seqs = [(int(torch.randint(n, ctx + 1, (1,), generator=g)), n) for _ in range(count)]
    for window, sinks in ((3000, 6), (200, 150), (40, 4)):
        b = Streams(seqs, 12, 2, 128, torch.bfloat16, window, sinks, spare_columns=200)
        b.check(b.run())


@pytest.mark.parametrize("window,sinks", [(9000, 4), (4096, 260), (20000, 1000)])
def test_split_contexts(window, sinks):
    """Few sequences, long windows: a row's keys are shared out to many CTAs and joined."""
    for seqs in ([(16000, 1)], [(16000, 4), (30, 1)], [(12000, 300)], [(9999, 1)] * 3):
        b = Streams(seqs, 8, 2, 128, torch.float16, window, sinks)
        b.check(b.run())


SHARED = [([(3000, 1)], 2500, 4), ([(700, 1)], 600, 20), ([(60, 1), (2100, 1), (0, 0)], 2000, 33),
          ([(4100, 5)], 4000, 100), ([(1200, 3), (900, 5), (5, 2), (17, 1)], 1000, 4),
          ([(20000, 1)], 30000, 4), ([(9000, 2), (40, 2)], 8000, 1), ([(1500, 40)], 1400, 17),
          ([(800 + 37 * i, 1) for i in range(17)], 900, 4),
          ([(600 + 70 * i, 1 + i % 5) for i in range(9)], 1100, 50)]


@pytest.mark.parametrize("case", range(len(SHARED)))
@pytest.mark.parametrize("hq,hkv,d", HEADS + [(16, 1, 128), (2, 2, 64), (32, 8, 128)])
def test_an_item_on_several_ctas(case, hq, hkv, d):
    """Small batches: clusters of CTAs share an item's pages, many with none of a short sequence."""
    seqs, window, sinks = SHARED[case]
    for dt in DTS:
        for cap in (0.0, 30.0):
            b = Streams(seqs, hq, hkv, d, dt, window, sinks, seed=case, softcap=cap)
            out = b.run()
            b.check(out)
            assert torch.equal(out, b.run())


def test_clusters_captured_and_on_two_streams():
    """Calls by clusters replayed from one graph, with other queries, while another stream makes
    its own."""
    a = Streams([(3000, 1), (40, 1)], 12, 2, 128, torch.bfloat16, 2500, 20, seed=3)
    b = Streams([(2600, 4)], 14, 2, 64, torch.float16, 2500, 20, seed=4)
    want_b = b.run()
    other, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    out = torch.full_like(a.q, float("nan"))
    call = lambda: binding.streaming_paged_attention(
        a.q, a.k, a.v, a.bt, a.sl, a.qs, a.scale, a.window, a.sinks, out=out)
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(3):
            call()
    outs = [torch.empty_like(b.q) for _ in range(8)]
    for i in range(4):
        a.q.copy_(torch.randn(a.q.shape, device="cuda").to(a.dt))
        torch.cuda.synchronize()
        out.fill_(float("nan"))
        graph.replay()
        for o in outs:
            binding.streaming_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, b.window,
                                              b.sinks, out=o, stream=other)
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        a.check(out)
        assert all(torch.equal(o, want_b) for o in outs)


def test_more_items_than_clusters():
    """Offsets that go back: the sequence is recorded as bad, those around it are served, though
    together they have more tokens than the batch."""
    b = Streams([(700, 40), (900, 40), (800, 40)], 4, 1, 128, torch.bfloat16, 600, 9)
    T = 48  # sequence 0: tokens 0 .. 39, 1: bad, 2: 8 .. 47
    b.qs[:] = torch.tensor([0, 40, 8, 48], dtype=torch.int32)
    q = b.q[:T].contiguous()
    out = torch.full_like(q, 7.0)
    binding.streaming_paged_attention(q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, 600, 9, out=out)
    torch.cuda.synchronize()
    assert binding.device_error() == 3
    for s, a, e in ((0, 0, 8), (2, 40, 48)):  # (tokens of one sequence alone)
        L, first = b.seqs[s][0], 0 if s == 0 else 8
        pos = torch.arange(L - 40 + a - first, L - 40 + e - first, device="cuda")
        ref, absv, size, tail = S.attend_stream(
            q[a:e], R.gather(b.k, b.bt[s], L), R.gather(b.v, b.bt[s], L), pos, b.scale, 600, 9)
        tol = R.attention_tolerance(ref, absv, size, tail, b.d, b.dt)
        assert not ((out[a:e].double() - ref).abs() > tol).any()


def test_without_a_window_or_sinks_it_is_the_masked_attention():
    for window, sinks in ((0, 0), (0, 7), (40, 0)):
        b = Streams(CHUNKS, 12, 2, 128, torch.bfloat16, window, sinks)
        want = binding.masked_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale,
                                              window=window)
        assert torch.equal(b.run(), want)


def test_more_sinks_than_the_context():
    for sinks in (2000, 1 << 20, 2 ** 31 - 1):
        for window in (1, 2 ** 31 - 1):
            for seqs in (DECODES, CHUNKS):
                b = Streams(seqs, 12, 2, 128, torch.bfloat16, window, 4000)
                b.sinks = sinks
                if sinks == 2000:
                    b = Streams(seqs, 12, 2, 128, torch.bfloat16, window, sinks)
                out = b.run()
                b.sinks = min(sinks, 4000)
                b.check(out)


@pytest.mark.parametrize("name", ["decodes", "chunks", "long", "verify"])
def test_padded_batches(name):
    """Rows behind the last sequence are left as they were."""
    for hq, hkv, d in ((12, 2, 128), (14, 2, 64)):
        b = Streams(BATCHES[name], hq, hkv, d, torch.bfloat16, 50, 5)
        T = b.q.shape[0]
        q = torch.cat([b.q, torch.full((37, hq, d), float("nan"), device="cuda").bfloat16()])
        out = torch.full_like(q, 3.0)
        binding.streaming_paged_attention(q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, 50, 5, out=out)
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        assert (out[T:] == 3.0).all()
        b.check(out[:T])


@pytest.mark.parametrize("name", ["decodes", "chunks", "long"])
@pytest.mark.parametrize("length", [-1, 2 ** 31 - 1, 2 ** 31 - 16, 40000])
def test_bad_lengths(name, length):
    """A length beyond the table: recorded, the sequence left out, the others served."""
    seqs = list(BATCHES[name]) + [(30, 2)]
    b = Streams(seqs, 12, 2, 128, torch.bfloat16, 60, 9)
    b.sl[-1] = length
    out = torch.full_like(b.q, 7.0)
    binding.streaming_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, 60, 9, out=out)
    torch.cuda.synchronize()
    assert binding.device_error() == 3
    assert (out[b.off[-2]:] == 7.0).all()
    b.seqs[-1] = (30, 0)
    b.check(out)


@pytest.mark.parametrize("name", ["decodes", "chunks", "long"])
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_blocks(name, bad):
    """A block of the sinks outside the pool is recorded; the other sequences are served."""
    b = Streams(BATCHES[name], 12, 2, 128, torch.bfloat16, 60, 9)
    at = max(range(len(b.seqs)), key=lambda i: b.seqs[i][0])
    b.bt[at, 0] = bad
    out = torch.zeros_like(b.q)
    binding.streaming_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, 60, 9, out=out)
    torch.cuda.synchronize()
    assert binding.device_error() == 1
    b.seqs = [(L, 0 if i == at else n) for i, (L, n) in enumerate(b.seqs)]
    b.check(out)


def test_streams_and_graphs():
    for seqs in (DECODES, CHUNKS, LONG):
        b = Streams(seqs, 12, 2, 128, torch.bfloat16, 90, 6)
        want = b.run()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        got = binding.streaming_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, 90, 6,
                                                stream=other)
        other.synchronize()
        assert torch.equal(got, want)
        ws = binding.alloc_workspace(b.q.shape[0], len(seqs), 12, 2, 128, 12000)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = binding.streaming_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, 90, 6,
                                                    workspace=ws)
        b.q.copy_(torch.randn_like(b.q))
        graph.replay()
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        b.check(out)


def test_the_smallest_workspace():
    for seqs in ([(16000, 1)], LONG, [(9000, 800)]):
        b = Streams(seqs, 12, 2, 128, torch.bfloat16, 8000, 100)
        n = binding.workspace_size(b.q.shape[0], len(seqs), 12, 2, 128, 0)
        b.check(b.run(workspace=torch.empty(n, dtype=torch.uint8, device="cuda")))


def test_scores_of_any_order():
    """Scores that rise and fall along the keys by many powers of two: the running maximum moves
    from the sinks to the window and back."""
    for seqs in ([(2000, 1), (700, 1)], [(1000, 400)]):
        for first in (40.0, 0.01):
            b = Streams(seqs, 8, 2, 64, torch.float16, 300, 20, std=4.0)
            for i, (L, n) in enumerate(seqs):
                b.k[b.bt[i, 0].long()] *= first
                b.k[b.bt[i, 1].long()] *= first
            b.check(b.run())
