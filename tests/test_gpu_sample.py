"""Sampling (ps_sample) against a plain 64-bit implementation."""
import math

import pytest
import torch

from paged_kv_attention_18_gb300 import binding
from tests import loop_ref as R

pytestmark = pytest.mark.gpu

DTS = [torch.float16, torch.bfloat16, torch.float32]


def words(B, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(-(1 << 31), 1 << 31, (B,), generator=g, dtype=torch.int64)
    w[: min(B, 2)] = torch.tensor([0, -1])[: min(B, 2)]  # both ends
    return w.to(torch.int32).cuda()


def logits(B, V, dt, seed, std=2.5, peak=6.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(B, V, generator=g, device="cuda") * std
    at = torch.randint(0, V, (B, 8), generator=g, device="cuda")
    x.scatter_(1, at, torch.rand(B, 8, generator=g, device="cuda") * peak + 2.0)
    return x.to(dt)


def f32(*v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(x, bits, **kw):
    tok, lp = binding.sample(x, bits, **kw)
    torch.cuda.synchronize()
    R.check_draws(x, tok, lp, bits, kw.get("temperature"), kw.get("top_k"), kw.get("top_p"),
                  kw.get("min_p"))
    return tok, lp


SIZES = [(1, 1), (5, 2), (3, 31), (40, 50), (9, 1003), (7, 4096), (4, 50257), (6, 151936)]


@pytest.mark.parametrize("B,V", SIZES)
@pytest.mark.parametrize("dt", DTS)
def test_filters(B, V, dt):
    x, bits = logits(B, V, dt, B + V), words(B, V)
    g = torch.Generator().manual_seed(V)

    def pick(values, t):
        return torch.tensor(values, dtype=t)[torch.randint(len(values), (B,), generator=g)].cuda()

    T = pick([0.3, 0.7, 1.0, 1.7], torch.float32)
    k = pick([0, 1, 7, 50, 1000, V, V + 3, -2], torch.int32)
    p = pick([0.1, 0.5, 0.9, 0.95, 0.999, 1.0], torch.float32)
    m = pick([0.0, 0.01, 0.2, 1.0], torch.float32)
    run(x, bits)
    run(x, bits, temperature=T)
    run(x, bits, top_k=k)
    run(x, bits, top_p=p)
    run(x, bits, min_p=m)
    run(x, bits, temperature=T, top_k=k, top_p=p)
    run(x, bits, temperature=T, top_p=p, min_p=m)
    run(x, bits, temperature=T, top_k=k, top_p=p, min_p=m)


@pytest.mark.parametrize("dt", DTS)
def test_every_draw_of_a_small_distribution(dt):
    """One row many times, the random words spread evenly: every token as often as its weight."""
    B, V = 4096, 6
    x = torch.tensor([0.0, 1.0, -2.0, 1.0, -math.inf, 0.5]).to(dt).cuda().expand(B, V).contiguous()
    bits = (torch.arange(B, dtype=torch.int64) << 20).to(torch.int32).cuda()
    tok, _ = run(x, bits)
    w = torch.softmax(x[0].double(), 0).cpu()
    n = torch.bincount(tok.long().cpu(), minlength=V).double()
    assert ((n - B * w).abs() <= 1).all()  # (each interval's ends are off by less than one word)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("V", [37, 5000, 70000])
def test_ties(dt, V):
    """Equal logits everywhere and in groups: the lowest tokens are kept."""
    x = torch.zeros(6, V, device="cuda")
    x[1] = torch.arange(V, device="cuda") % 3
    x[2, ::2] = -0.0
    x[3] = 5.0 - (torch.arange(V, device="cuda") // 10).clamp(max=40)
    x[4, V // 2:] = -math.inf
    x[5] = torch.finfo(dt).min
    x = x.to(dt)
    bits = words(6, 3)
    for k in (1, 2, 10, 15, V // 2, V - 1):
        run(x, bits, top_k=i32(*[k] * 6))
        run(x, bits, top_k=i32(*[k] * 6), top_p=f32(*[0.6] * 6))
    for p in (0.0, 1e-6, 0.25, 0.5, 0.9):
        run(x, bits, top_p=f32(*[p] * 6))
    run(x, bits, min_p=f32(*[1.0] * 6))
    run(x, bits, temperature=f32(*[0.0] * 6))


@pytest.mark.parametrize("dt", DTS)
def test_values_at_the_ends(dt):
    """-inf, NaN, +inf, masks of the type's least value, finite logits of any size."""
    V, big = 3001, torch.finfo(dt).max
    x = logits(12, V, dt, 5)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 7] = math.inf
    x[3, ::2] = math.nan
    x[4, 1:] = -math.inf
    x[5, 5:] = torch.finfo(dt).min
    x[6] = -big
    x[6, 100] = big
    x[7] = torch.where(torch.arange(V, device="cuda") % 2 == 0, big, -big)
    x[8, 20:] = -math.inf
    x[8, 3] = math.nan
    x[9] = -big
    x[10] *= 1e-4
    x[11] = torch.finfo(dt).smallest_normal / 4
    bits = words(12, 6)
    n = x.shape[0]
    run(x, bits)
    for T in (0.0, 1e-35, 1e-6, 0.5, 40.0, 1e30, math.inf):
        run(x, bits, temperature=f32(*[T] * n))
        run(x, bits, temperature=f32(*[T] * n), top_k=i32(*[30] * n), top_p=f32(*[0.7] * n))
    run(x, bits, temperature=f32(*[math.nan] * n))
    run(x, bits, top_k=i32(*[50] * n), min_p=f32(*[0.3] * n))
    run(x, bits, min_p=f32(*[7.0] * n))
    tok, lp = binding.sample(x, bits, top_p=f32(*[math.nan] * n), min_p=f32(*[math.nan] * n))
    plain = binding.sample(x, bits)
    assert torch.equal(tok, plain[0]) and torch.equal(lp, plain[1])
    assert tok[:3].tolist() == [-1, -1, -1]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("V,pad,at", [(1003, 5, 1), (50257, 15, 3), (4097, 7, 0)])
def test_views(dt, V, pad, at):
    """Rows inside a padded vocabulary at any alignment; what lies around them is not read."""
    B = 5
    big = torch.full((B, V + pad), math.inf, dtype=dt, device="cuda")
    x = big[:, at:at + V]
    x.copy_(logits(B, V, dt, 8))
    bits = words(B, 9)
    run(x, bits, top_k=i32(0, 40, 3, 0, 500), top_p=f32(0.9, 1.0, 0.8, 1.0, 0.95))


def shapes_of_rows(B, V, dt, seed):
    """Rows of very different distributions: flat, steep, in steps, one token, two levels a hair
    apart, geometric, a heavy tail."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(B, V, generator=g, device="cuda")
    i = torch.arange(V, device="cuda").float()
    x[0::8] *= 1e-3
    x[1::8] *= 12.0
    x[2::8] = torch.floor(x[2::8] * 3.0)
    x[3::8, 5] = 40.0
    x[4::8] = (i % 2) * 0.004
    x[5::8] = -i * 0.01
    x[6::8] = -torch.log(i + 1.0) * 1.01
    return x.to(dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("B,V", [(64, 20011), (16, 151936), (150, 2000)])
def test_borders(dt, B, V):
    """Shares, counts and temperatures all over their ranges: the border's bin is not always the one
    that the counts point at."""
    x, bits = shapes_of_rows(B, V, dt, B), words(B, V)
    g = torch.Generator().manual_seed(B)
    for _ in range(3):
        p = torch.rand(B, generator=g)
        p[::3] = 1.0 - 10.0 ** (-5.0 * p[::3])
        k = (V * torch.rand(B, generator=g) ** 3).int() + 2
        T = 0.05 + 3.0 * torch.rand(B, generator=g) ** 2
        m = torch.rand(B, generator=g) ** 8
        p, k, T, m = p.cuda(), k.cuda(), T.cuda(), m.cuda()
        run(x, bits, top_p=p)
        run(x, bits, top_p=p, temperature=T)
        run(x, bits, top_k=k)
        run(x, bits, top_k=k, top_p=p, temperature=T)
        run(x, bits, top_p=p, min_p=m, temperature=T)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("k", [40, 63, 64, 65, 127, 128, 129, 200])
def test_small_and_large_k(dt, k):
    """Around the counts at which a list gives way to bins; rows masked by the least finite value to
    fewer tokens than k."""
    x = logits(12, 30000, dt, k)
    x[1, 50:] = torch.finfo(dt).min
    x[2, 100:] = -math.inf
    x[3] = x[3].round()
    x[4] = 1.0
    ks = torch.full((12,), k, dtype=torch.int32, device="cuda")
    bits = words(12, k)
    run(x, bits, top_k=ks)
    run(x, bits, top_k=ks, top_p=torch.full((12,), 0.7, device="cuda"))


def test_calls_at_once():
    """Calls that overlap on two streams share nothing."""
    xs = [logits(40, 151936, torch.bfloat16, 30 + i) for i in range(2)]
    bits, p = words(40, 31), torch.full((40,), 0.93, device="cuda")
    want = [binding.sample(x, bits, top_p=p) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            got[i].append(binding.sample(xs[i], bits, top_p=p, stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        for tok, lp in got[i]:
            assert torch.equal(tok, want[i][0]) and torch.equal(lp, want[i][1])


def test_large_vocabularies():
    for dt, V in ((torch.float32, 393216), (torch.bfloat16, 393211), (torch.float16, 262208)):
        x, bits = logits(3, V, dt, 11), words(3, 12)
        run(x, bits, top_p=f32(0.95, 0.5, 1.0), top_k=i32(0, 2000, 0))
    with pytest.raises(binding.PagedServeError):
        binding.sample(torch.zeros(1, 393217, device="cuda"), words(1, 0))


def test_many_rows():
    """More rows than clusters fit the GPU at once; the same row gives the same token anywhere."""
    x = logits(2000, 600, torch.bfloat16, 13)
    bits = words(2000, 14)
    T, k = torch.full((2000,), 0.9, device="cuda"), torch.full((2000,), 40, device="cuda").int()
    tok, lp = run(x, bits, temperature=T, top_k=k)
    order = torch.randperm(2000, device="cuda")
    again = binding.sample(x[order], bits[order], temperature=T, top_k=k)
    assert torch.equal(again[0], tok[order]) and torch.equal(again[1], lp[order])


def test_slices_do_not_change_the_draw():
    """One row alone is cut into more slices than in a batch: the sums are exact either way."""
    x, bits = logits(80, 151936, torch.bfloat16, 15), words(80, 16)
    p = torch.full((80,), 0.97, device="cuda")
    tok, lp = binding.sample(x, bits, top_p=p)
    for b in (0, 1, 7, 79):
        one = binding.sample(x[b:b + 1], bits[b:b + 1], top_p=p[b:b + 1])
        assert torch.equal(one[0], tok[b:b + 1]) and torch.equal(one[1], lp[b:b + 1])


def test_streams_and_graphs():
    x, bits = logits(33, 5003, torch.float16, 17), words(33, 18)
    k = torch.full((33,), 25, device="cuda").int()
    want = run(x, bits, top_k=k)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = binding.sample(x, bits, top_k=k, stream=other)
    other.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.sample(x, bits, top_k=k)
    for seed in (19, 20):
        x.copy_(logits(33, 5003, torch.float16, seed))
        bits.copy_(words(33, seed))
        graph.replay()
        torch.cuda.synchronize()
        R.check_draws(x, *out, bits, k=k)


def test_empty_and_shapes():
    tok, lp = binding.sample(torch.zeros(0, 7, device="cuda"), words(0, 0))
    assert tok.shape == (0,) and lp.shape == (0,)
    x = torch.zeros(2, 7, device="cuda")
    for bad in (dict(top_k=f32(1, 1)), dict(top_p=f32(1)), dict(temperature=i32(1, 1))):
        with pytest.raises(binding.PagedServeError):
            binding.sample(x, words(2, 0), **bad)
    with pytest.raises(binding.PagedServeError):
        binding.sample(x.t(), words(7, 0))
    with pytest.raises(binding.PagedServeError):
        binding.sample(x.double(), words(2, 0))
    with pytest.raises(binding.PagedServeError):
        binding.sample(x, None)
