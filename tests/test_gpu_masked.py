"""Masked paged attention (ps_paged_attention_masked) against a plain 64-bit implementation."""
import math

import pytest
import torch

from paged_kv_attention_18_gb300 import binding
from tests import operator_ref as R

pytestmark = pytest.mark.gpu

DTS = [torch.float16, torch.bfloat16]


class Batch:
    """Sequences [(context, new tokens)] over a random pool; with `holes`, whatever no row
    may read holds NaN: free blocks, rows past a context, blocks before a window (-1)."""

    def __init__(self, seqs, hq, hkv, d, dt, seed, window=0, prefix=None, starts=None,
                 softcap=0.0, slopes=None, std=1.0, holes=True):
        g = torch.Generator("cuda").manual_seed(seed)
        self.seqs, self.window, self.softcap = seqs, window, softcap
        self.hq, self.hkv, self.d, self.dt = hq, hkv, d, dt
        B, T = len(seqs), sum(n for _, n in seqs)
        pages = [(L + 15) // 16 for L, _ in seqs]
        width = max(max(pages), 1)
        nb = sum(pages) + 5
        ids = torch.randperm(nb, generator=g, device="cuda").int()
        self.q = (torch.randn(T, hq, d, generator=g, device="cuda") * std).to(dt)
        self.k = torch.randn(nb, 16, hkv, d, generator=g, device="cuda").to(dt)
        self.v = torch.randn(nb, 16, hkv, d, generator=g, device="cuda").to(dt)
        self.bt = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.low = []
        at = 0
        nan = float("nan")
        if holes:
            free = ids[sum(pages):].long()
            self.k[free] = nan
            self.v[free] = nan
        for b, (L, n) in enumerate(seqs):
            blk = ids[at:at + pages[b]]
            at += pages[b]
            self.bt[b, :pages[b]] = blk
            lo = max(0, L - n - window + 1) if window else 0
            if starts is not None and n:
                lo = max(lo, min(starts[b]))
            self.low.append(lo)
            if holes and pages[b]:
                last = blk[-1].long()
                self.k[last, L - 16 * (pages[b] - 1):] = nan
                self.v[last, L - 16 * (pages[b] - 1):] = nan
                if window and n:
                    first = min(max(0, L - n - window + 1) // 16, pages[b] - 1)
                    self.bt[b, :first] = -1
                if n and lo < L and lo % 16:  # the first page's rows before the first key
                    self.k[blk[lo // 16].long(), :lo % 16] = nan
                    self.v[blk[lo // 16].long(), :lo % 16] = nan
        self.sl = torch.tensor([L for L, _ in seqs], dtype=torch.int32, device="cuda")
        off = [0]
        for _, n in seqs:
            off.append(off[-1] + n)
        self.off = off
        self.qs = torch.tensor(off, dtype=torch.int32, device="cuda")
        self.prefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32,
                                                               device="cuda")
        self.starts = None
        if starts is not None:
            flat = [s for row in starts for s in row]
            self.starts = torch.tensor(flat, dtype=torch.int32, device="cuda")
        self.slopes = slopes
        self.scale = d ** -0.5

    def kwargs(self):
        return dict(softcap=self.softcap, distance_slopes=self.slopes, window=self.window,
                    prefix_lens=self.prefix, key_starts=self.starts)

    def run(self, **kw):
        out = torch.full_like(self.q, float("nan"))
        binding.masked_paged_attention(self.q, self.k, self.v, self.bt, self.sl, self.qs,
                                       self.scale, out=out, **self.kwargs(), **kw)
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        return out

    def check(self, out):
        for b, (L, n) in enumerate(self.seqs):
            if n == 0:
                continue
            a, e = self.off[b], self.off[b + 1]
            pos = torch.arange(L - n, L, device="cuda")
            ref, absv, size, tail = R.attend_dense(
                self.q[a:e], R.gather(self.k, self.bt[b], L), R.gather(self.v, self.bt[b], L), pos,
                self.scale, self.softcap, self.slopes, self.window,
                0 if self.prefix is None else int(self.prefix[b]),
                None if self.starts is None else self.starts[a:e])
            tol = R.attention_tolerance(ref, absv, size, tail, self.d, self.dt)
            err = (out[a:e].double() - ref).abs()
            assert not (err > tol).any() and torch.isfinite(out[a:e]).all(), \
                (b, L, n, float((err - tol).max()), int((~(err <= tol)).sum()))


def slopes_of(hq, top=1.0):
    return (top * 2.0 ** (-8.0 * torch.arange(1, hq + 1) / hq)).float().cuda()


DECODES = [(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (300, 1), (2049, 1), (129, 1)]
LONG = [(9000, 1), (5, 1), (700, 1), (33, 4), (12000, 2)]
CHUNKS = [(300, 300), (1, 1), (513, 200), (64, 64), (900, 129), (40, 1)]
SMALL_CHUNKS = [(200, 100), (90, 33)]
BATCHES = {"decodes": DECODES, "long": LONG, "chunks": CHUNKS, "small_chunks": SMALL_CHUNKS,
           "one": [(1, 1)], "one_long": [(3000, 1)], "one_chunk": [(1500, 1400)],
           "gaps": [(50, 0), (20, 3), (0, 0), (400, 1), (16, 0)]}
HEADS = [(12, 2, 128), (8, 8, 64), (7, 1, 128), (14, 2, 64), (40, 2, 64)]


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_capped_scores(name, hq, hkv, d):
    for dt in DTS:
        b = Batch(BATCHES[name], hq, hkv, d, dt, 1, softcap=15.0, std=6.0)
        b.check(b.run())


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_distance_bias(name, hq, hkv, d):
    for dt in DTS:
        b = Batch(BATCHES[name], hq, hkv, d, dt, 2, slopes=slopes_of(hq))
        b.check(b.run())


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 1024, 2 ** 31 - 1])
def test_sliding_window(name, window):
    b = Batch(BATCHES[name], 12, 2, 128, torch.bfloat16, 3, window=window)
    b.check(b.run())
    b = Batch(BATCHES[name], 14, 2, 64, torch.float16, 3, window=window, softcap=30.0, std=4.0,
              slopes=slopes_of(14))
    b.check(b.run())


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("prefix", [0, 1, 16, 130, 100000])
def test_bidirectional_prefix(name, prefix):
    for dt, heads, kw in ((torch.bfloat16, (12, 2, 128), {}),
                          (torch.float16, (14, 2, 64), dict(slopes=slopes_of(14))),
                          (torch.float16, (8, 8, 64), dict(window=200))):
        b = Batch(BATCHES[name], *heads, dt, 4, prefix=[prefix - i for i in
                                                        range(len(BATCHES[name]))],
                  holes="window" not in kw, **kw)
        b.check(b.run())


def doc_starts(seqs, step):
    """Documents of `step` positions each."""
    return [[(p // step) * step for p in range(L - n, L)] for L, n in seqs]


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("step", [1, 7, 16, 100, 700])
def test_packed_documents(name, step):
    seqs = BATCHES[name]
    for dt, heads, kw in ((torch.bfloat16, (12, 2, 128), {}),
                          (torch.float16, (14, 2, 64), dict(window=50, softcap=20.0))):
        b = Batch(seqs, *heads, dt, 5, starts=doc_starts(seqs, step), **kw)
        b.check(b.run())


@pytest.mark.parametrize("name", list(BATCHES))
def test_rows_without_keys_are_zeros(name):
    # every third row onwards starts past its own position: it sees nothing
    seqs = BATCHES[name]
    starts = [[0 if i < n // 2 else L + 5 for i in range(n)] for L, n in seqs]
    for dt, heads in ((torch.bfloat16, (12, 2, 128)), (torch.float16, (14, 2, 64))):
        b = Batch(seqs, *heads, dt, 6, starts=starts)
        out = b.run()
        b.check(out)
        for i, (L, n) in enumerate(seqs):
            for r in range(n // 2, n):
                assert (out[b.off[i] + r] == 0).all()


def test_every_row_without_keys():
    b = Batch([(5000, 1), (300, 200), (20, 2)], 12, 2, 128, torch.bfloat16, 6,
              starts=[[2 ** 31 - 1], [2 ** 31 - 1] * 200, [2 ** 31 - 1] * 2])
    assert (b.run() == 0).all()


@pytest.mark.parametrize("name", ["decodes", "long", "chunks", "one_chunk"])
def test_without_any_of_it_as_the_causal_attention(name):
    b = Batch(BATCHES[name], 12, 2, 128, torch.bfloat16, 7, holes=False)
    out = b.run()
    b.check(out)
    ref = binding.paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale)
    # the two round the same P; scores differ by fp32 roundings
    assert (out.double() - ref.double()).abs().max() <= 2.0 ** -6


def test_steep_slopes_and_large_caps():
    # the bias climbs by hundreds of log2 units from tile to tile; a cap no score reaches
    for dt in DTS:
        b = Batch([(4000, 1), (1000, 900), (2500, 70)], 12, 2, 128, dt, 8,
                  slopes=slopes_of(12, 40.0), softcap=1e4)
        b.check(b.run())
        b = Batch([(4000, 1), (1000, 900)], 12, 2, 128, dt, 8, slopes=-slopes_of(12, 0.5))
        b.check(b.run())


def test_saturated_caps():
    # scores far past the cap: tanh is 1 and -1 to the last bit
    b = Batch([(700, 1), (500, 300)], 8, 2, 64, torch.float16, 9, softcap=2.0, std=200.0)
    b.check(b.run())


@pytest.mark.parametrize("name", ["one", "small_chunks", "chunks", "one_chunk", "long", "decodes"])
def test_rows_behind_the_last_sequence_stay(name):
    # a batch padded to a fixed number of tokens, in every mode: direct, tiles alone, planned
    b = Batch(BATCHES[name], 12, 2, 128, torch.bfloat16, 10, window=300)
    T = b.q.shape[0]
    q = torch.cat([b.q, b.q[:1].expand(9, -1, -1)]).contiguous()
    out = torch.full_like(q, 7.0)
    binding.masked_paged_attention(q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, window=300, out=out)
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    b.check(out[:T])
    assert (out[T:] == 7.0).all()


def test_bad_blocks_and_sequences_are_recorded():
    b = Batch([(300, 1), (500, 300)], 12, 2, 128, torch.bfloat16, 11, holes=False)
    b.bt[0, 3] = 10 ** 6
    out = torch.empty_like(b.q)
    binding.masked_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, out=out)
    assert binding.device_error() == 1
    b = Batch([(300, 1), (500, 300)], 12, 2, 128, torch.bfloat16, 11, holes=False)
    b.sl[0] = 0  # one token of a context of none
    out = torch.full_like(b.q, 7.0)
    binding.masked_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, out=out)
    assert binding.device_error() == 3
    assert (out[0] == 7.0).all()
    b.seqs = [(1, 0), (500, 300)]
    b.off = [0, 1, 301]
    b.check(out)


@pytest.mark.parametrize("name", ["one", "small_chunks", "chunks", "long"])
@pytest.mark.parametrize("what", ["length", "offsets"])
def test_lengths_and_offsets_at_the_end_of_32_bits(name, what):
    # recorded and left unwritten in every mode, the other sequences served
    b = Batch(BATCHES[name] + [(30, 3)], 12, 2, 128, torch.float16, 25, window=50, holes=False)
    b.bt[b.bt < 0] = 0
    T, last = b.q.shape[0], len(b.seqs) - 1
    if what == "length":
        b.sl[last] = 2 ** 31 - 1  # a few more, and the count of its pages would be negative
        bad, b.seqs = slice(T - 3, T), b.seqs[:last]
    else:
        b.qs[last] = 2 ** 31 - 1  # the last two sequences' tokens; the others may be left too
        b.qs[last + 1] = -2 ** 31
        bad, b.seqs = slice(b.off[last - 1], T), []
    out = torch.full_like(b.q, 7.0)
    binding.masked_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, window=50, out=out)
    torch.cuda.synchronize()
    assert binding.device_error() == 3
    assert (out[bad] == 7.0).all()
    b.check(out)


def test_one_workspace_two_calls_and_other_stream():
    b = Batch(LONG, 12, 2, 128, torch.bfloat16, 12, window=300, softcap=20.0, std=3.0)
    c = Batch(CHUNKS, 12, 2, 128, torch.bfloat16, 13, prefix=[40] * len(CHUNKS))
    n = max(binding.workspace_size(x.q.shape[0], len(x.seqs), 12, 2, 128, 16 * x.bt.shape[1])
            for x in (b, c))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    first = b.run(workspace=ws)
    c.check(c.run(workspace=ws))
    assert torch.equal(b.run(workspace=ws), first)  # the same bits again
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = binding.masked_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, stream=s,
                                         **b.kwargs())
    s.synchronize()
    b.check(out)


def test_two_streams_at_once_with_a_workspace_each():
    batches = [Batch(LONG, 12, 2, 128, torch.bfloat16, 22, window=3000, softcap=20.0, std=3.0),
               Batch(CHUNKS, 12, 2, 128, torch.bfloat16, 23, slopes=slopes_of(12))]
    want = [b.run() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    outs = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for i, b in enumerate(batches):
            outs[i].append(binding.masked_paged_attention(
                b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, stream=streams[i], **b.kwargs()))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])


def test_a_small_workspace_splits_less():
    b = Batch([(20000, 1), (7000, 1)], 12, 2, 128, torch.bfloat16, 14, softcap=20.0, std=3.0)
    ws = binding.alloc_workspace(2, 2, 12, 2, 128, 0)
    b.check(b.run(workspace=ws))


def test_captured_with_lengths_that_grow():
    b = Batch([(400, 1), (900, 1), (77, 1)], 12, 2, 128, torch.bfloat16, 15, window=128,
              holes=False)
    b.bt[b.bt < 0] = 0
    ws = binding.alloc_workspace(3, 3, 12, 2, 128, 1024)
    out = torch.empty_like(b.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.masked_paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, out=out,
                                       workspace=ws, **b.kwargs())
    for step in (0, 1, 3):
        b.sl.add_(step if step < 3 else -200)
        if step == 3:
            b.sl.clamp_(min=1)
        graph.replay()
        torch.cuda.synchronize()
        b.seqs = [(int(x), 1) for x in b.sl]
        b.check(out)
    assert binding.device_error() == 0


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (6, 2, 64), (5, 5, 128), (14, 2, 128)])
@pytest.mark.parametrize("kw", [{}, dict(window=700, softcap=12.0, std=5.0), dict(bias=1)])
def test_decode_items_of_eight_rows(hq, hkv, d, kw):
    # no more tokens than sequences: 8-row items, some of a sequence with several tokens
    kw = dict(kw)
    if kw.pop("bias", None):
        kw["slopes"] = slopes_of(hq)
    seqs = [(5000, 1), (2300, 5), (9, 0), (7000, 0), (2049, 1), (15, 2), (3000, 0), (77, 1),
            (1, 1), (0, 0), (4000, 1), (600, 0)]
    for dt in DTS:
        b = Batch(seqs, hq, hkv, d, dt, 18, **kw)
        b.check(b.run())


@pytest.mark.parametrize("hq,hkv,d", [(12, 4, 128), (14, 2, 64), (40, 4, 64), (36, 3, 128)])
@pytest.mark.parametrize("count", [1, 12, 60, 90])
@pytest.mark.parametrize("kw", [{}, dict(window=40, softcap=12.0, std=5.0), dict(prefix=30)])
def test_small_batches_in_one_launch(hq, hkv, d, count, kw):
    # as many tokens as sequences, contexts of at most 2048: a sequence's row groups are taken
    # by several CTAs, by one CTA after the other, and with 90 sequences planned
    kw = dict(kw)
    some = [(2048, 1), (900, 9), (5, 0), (0, 0), (31, 4), (17, 1), (600, 0), (1, 1), (1300, 1),
            (16, 0), (33, 1), (700, 0)]
    seqs = [(700, 1)] if count == 1 else \
        [(max(L - 3 * (i // 12), n), n) for i in range(0, count, 12) for L, n in some][:count]
    while sum(n for _, n in seqs) < len(seqs):
        i = [n for _, n in seqs].index(0)
        seqs[i] = (max(seqs[i][0], 1), 1)
    while sum(n for _, n in seqs) > len(seqs):
        seqs.append((40, 0))
    if kw.get("prefix"):
        kw["prefix"] = [kw["prefix"]] * len(seqs)
    for dt in DTS:
        b = Batch(seqs, hq, hkv, d, dt, 24, **kw)
        b.check(b.run())


@pytest.mark.parametrize("hq,hkv,d", [(12, 2, 128), (14, 2, 64), (8, 8, 64), (32, 2, 128)])
@pytest.mark.parametrize("seqs", [
    [(700 + i, 4) for i in range(16)],                           # tokens to verify
    [(50 * i + 1, 1) for i in range(40)] + [(1900, 48)],         # decodes and a short chunk
    [(300, 7), (0, 0), (2000, 2), (1, 1), (64, 64), (5, 0)] * 6 + [(9, 0)] * 29,  # over 64
    [(200, 12)],
    [(i % 50 + 1, (1, 1, 2, 0, 1)[i % 5]) for i in range(150)],  # found by several counts
])
def test_several_tokens_in_one_launch(hq, hkv, d, seqs):
    for dt, kw in ((torch.float16, dict(slopes=slopes_of(hq), window=333)),
                   (torch.bfloat16, dict(softcap=20.0, std=4.0))):
        b = Batch(seqs, hq, hkv, d, dt, 26, **kw)
        b.check(b.run())


def test_many_sequences():
    # more sequences than the planner stages in shared memory
    seqs = [(1 + (7 * i) % 90, 1) for i in range(4200)]
    b = Batch(seqs, 4, 2, 64, torch.bfloat16, 16, window=20)
    out = b.run()
    b.seqs = seqs[:40] + [(L, 0) for L, _ in seqs[40:-40]] + seqs[-40:]
    b.check(out)


def test_math_of_the_cap_at_zero_length_scores():
    # q = 0: every score is 0 whatever the cap, so the output is the mean of the values
    b = Batch([(40, 1), (200, 150)], 8, 2, 64, torch.float16, 17, softcap=10.0, std=0.0)
    out = b.run()
    b.check(out)
    assert math.isfinite(float(out.float().sum()))


@pytest.mark.parametrize("seqs", [
    [(300, 200)], [(700 + i, 4) for i in range(16)], [(200, 100), (90, 33)], [(33, 1), (47, 20)],
    [(1500, 1400)], [(513, 200), (1, 1), (64, 64), (900, 129), (40, 1), (5000, 2)],
    [(9000, 4), (700, 1), (12000, 2)]])
@pytest.mark.parametrize("step,live", [(40, 30), (4, 3), (7, 2), (160, 16)])
def test_rows_without_keys_between_documents(seqs, step, live):
    # documents padded to a multiple of `step`: a padding row starts at the next document, so it
    # sees nothing, and nothing sees its key, which was never written
    starts = [[p // step * step + (step if p % step >= live else 0) for p in range(L - n, L)]
              for L, n in seqs]
    for dt, heads, kw in ((torch.bfloat16, (12, 2, 128), {}),
                          (torch.float16, (14, 2, 64), dict(window=50, softcap=20.0)),
                          (torch.bfloat16, (4, 4, 64), dict(slopes=slopes_of(4)))):
        b = Batch(seqs, *heads, dt, 27, starts=starts, holes=False, **kw)
        for i, (L, _) in enumerate(seqs):
            p = torch.arange(L, device="cuda")
            p = p[p % step >= live]
            blk = b.bt[i].long()[p // 16]
            b.k[blk, p % 16] = float("nan")
            b.v[blk, p % 16] = float("nan")
        out = b.run()
        b.check(out)
        empty = torch.tensor([s > p for (L, n), row in zip(seqs, starts)
                              for p, s in zip(range(L - n, L), row)], device="cuda")
        assert (out[empty] == 0).all()


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("cap", [1e3, 1e4, 1e5, 1e6, 1e8, 1e30, 2e38])
def test_caps_far_above_the_scores(name, cap):
    # cap * tanh(x / cap) tends to x: the error has the size of the score, not of the cap. The
    # cap takes a score's value off by 2^-20 of it at most (the polynomial 2^-20.7, or one
    # reciprocal's 2^-22 of the cap where the score is half of it at least), in numerator and
    # denominator; without the cap's own share `size` is the scores' (tanh only shrinks them).
    for dt, heads, kw in ((torch.bfloat16, (12, 2, 128), {}), (torch.float16, (7, 1, 64), {}),
                          (torch.bfloat16, (14, 2, 64), dict(slopes=slopes_of(14)))):
        b = Batch(BATCHES[name], *heads, dt, 28, softcap=cap, **kw)
        out = b.run()
        for i, (L, n) in enumerate(b.seqs):
            if n == 0:
                continue
            a, e = b.off[i], b.off[i + 1]
            args = (b.q[a:e], R.gather(b.k, b.bt[i], L), R.gather(b.v, b.bt[i], L),
                    torch.arange(L - n, L, device="cuda"), b.scale)
            _, _, size, _ = R.attend_dense(*args, 0.0, b.slopes)
            ref, absv, _, tail = R.attend_dense(*args, cap, b.slopes)
            tol = R.attention_tolerance(ref, absv, size, tail, b.d, dt) + \
                math.log(2) * 2.0 ** -20 * size[..., None] * (absv + ref.abs())
            err = (out[a:e].double() - ref).abs()
            assert not (err > tol).any() and torch.isfinite(out[a:e]).all(), \
                (i, L, n, float((err - tol).max()))


@pytest.mark.parametrize("name", ["small_chunks", "chunks", "one_chunk", "decodes"])
@pytest.mark.parametrize("cap", [15.0, 29.0, 31.0, 45.0, 50.0, 51.0, 62.0, 63.0, 200.0])
def test_rows_near_either_end_of_the_cap(name, cap):
    # every score of a row within a few hundredths of -cap, or of +cap: whatever the softmax is
    # taken against, products with small and with large values keep their bits
    for dt, std in ((torch.bfloat16, 2.0 ** -36), (torch.bfloat16, 1.0), (torch.bfloat16, 2.0 ** 36),
                    (torch.float16, 1.0)):
        b = Batch(BATCHES[name], 12, 2, 128, dt, 29, softcap=cap, holes=False)
        g = torch.Generator("cuda").manual_seed(30)
        u = 0.7 + 0.6 * torch.rand(b.k.shape[:3], generator=g, device="cuda")
        b.k = u[..., None].expand(b.k.shape).to(dt).contiguous()
        sign = torch.randint(0, 2, b.q.shape[:2], generator=g, device="cuda") * 2.0 - 1.0
        b.q = (sign * (2.0 * cap / b.scale / b.d))[..., None].expand(b.q.shape).to(dt).contiguous()
        b.v = (b.v.float() * std).to(dt)
        b.check(b.run())
