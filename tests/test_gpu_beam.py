"""Beam selection (ps_beam_select) and forks of the cache (ps_fork_sequences) against 64 bits."""
import math

import pytest
import torch

from paged_kv_attention_18_gb300 import binding
from tests import operator_ref as R

pytestmark = pytest.mark.gpu

# lse: ex2 is off by 2^-22 and the exponent's argument, a fused multiply-add, by half a step of
# at most 2^6 for terms that weigh; each of a thread's at most 40 adds in turn (chunks of up
# to 40960 logits at these sizes, four sums), of the 13 joins across the threads and of the log
# by 2^-24: (4 + 4 + 40 + 13 + 1) 2^-24 < 2^-18
LSE_TOL = 2.0 ** -18


def check(logits, scores, n, got, finished=None, pad=0):
    par, tok, val = (x.cpu() for x in got)
    B, W, V = logits.shape
    for b, cand in enumerate(R.beam(logits, scores, n, finished, pad)):
        near = [(cand[i][0] - cand[i + 1][0]) for i in range(min(n, len(cand) - 1))
                if cand[i][1] // V != cand[i + 1][1] // V and cand[i][0] != cand[i + 1][0]]
        assert not near or min(near) > 2 * LSE_TOL, "the oracle's order is not decided"
        for i in range(n):
            if i < len(cand):
                s, flat = cand[i]
                assert (int(par[b, i]), int(tok[b, i])) == (flat // V, flat % V), (b, i)
                assert abs(float(val[b, i]) - s) <= LSE_TOL + 2.0 ** -24 * abs(s)
            else:
                assert int(par[b, i]) == int(tok[b, i]) == -1
                assert float(val[b, i]) == -math.inf


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,W,V,n", [
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 4, 1003, 4), (3, 3, 8191, 6), (2, 2, 8192, 2),
    (1, 5, 8193, 32), (4, 4, 50001, 8), (2, 32, 700, 32), (1, 2, 151936, 4), (70, 1, 333, 1), (64, 4, 50001, 8),
    (700, 1, 333, 2), (160, 4, 70001, 8)])
def test_selection(B, W, V, n, dt):
    g = torch.Generator("cuda").manual_seed(B * 7 + V)
    logits = (torch.randn(B, W, V, generator=g, device="cuda") * 3).to(dt)
    scores = -torch.rand(B, W, generator=g, device="cuda") * 10
    check(logits, scores, n, binding.beam_select(logits, scores, n))


@pytest.mark.parametrize("skew", [0, 1, 3, 7])
def test_padded_rows_at_odd_offsets(skew):
    # rows of a wider tensor, starting off 16-byte boundaries, NaN around them
    B, W, V, ld = 2, 3, 9001, 9013
    for dt in (torch.float16, torch.float32):
        g = torch.Generator("cuda").manual_seed(skew)
        buf = torch.full((skew + B * W * ld,), float("nan"), device="cuda", dtype=dt)
        logits = buf[skew:].view(B, W, ld)[:, :, :V]
        logits.copy_((torch.randn(B, W, V, generator=g, device="cuda") * 3).to(dt))
        scores = -torch.rand(B, W, generator=g, device="cuda")
        check(logits, scores, 5, binding.beam_select(logits, scores, 5))


def test_finished_masked_and_broken_beams():
    g = torch.Generator("cuda").manual_seed(3)
    B, W, V, n = 6, 4, 20011, 8
    logits = torch.randn(B, W, V, generator=g, device="cuda") * 2
    scores = -torch.rand(B, W, generator=g, device="cuda") * 4
    fin = torch.zeros(B, W, dtype=torch.uint8, device="cuda")
    fin[0, 1] = fin[1, 0] = 1
    fin[2] = 1                                  # every beam finished: four candidates in all
    logits[0, 1] = float("nan")                 # a finished beam's logits are not read
    scores[3, 1:] = -math.inf                   # the first step: one live beam
    logits[4, :, 3:] = -math.inf                # constrained to three tokens
    logits[4, 0] = -math.inf                    # a beam with no continuation
    logits[4, 1, 1] = float("nan")              # NaN is no continuation
    logits[5, 2, 77] = math.inf                 # nor has a beam with an infinite logit any
    scores[5, 3] = float("nan")
    ref = logits.clone()
    ref[5, 2] = -math.inf
    check(ref, scores, n, binding.beam_select(logits, scores, n, finished=fin, pad_token=V - 1),
          fin, V - 1)
    check(ref, scores, n, binding.beam_select(logits, scores, n, finished=fin.bool(),
                                              pad_token=17), fin, 17)


@pytest.mark.parametrize("V", [40, 8200, 30000])
def test_ties_go_to_the_lowest_index(V):
    # all logits equal: more ties than any list holds; then two values, and signed zeros
    B, W, n = 2, 4, 16
    scores = torch.zeros(B, W, device="cuda")
    for fill in (0.0, -3.0):
        logits = torch.full((B, W, V), fill, device="cuda", dtype=torch.bfloat16)
        par, tok, _ = binding.beam_select(logits, scores, n)
        assert (par == 0).all() and torch.equal(tok.cpu(), torch.arange(n).int().expand(B, n))
    logits = torch.zeros(B, W, V, device="cuda")
    logits[:, :, ::2] = -0.0
    par, tok, _ = binding.beam_select(logits, scores, n)
    assert (par == 0).all() and torch.equal(tok.cpu(), torch.arange(n).int().expand(B, n))
    logits[:, :, 5::7] = 1.0
    par, tok, _ = binding.beam_select(logits, scores, n)
    want = [(w, t) for w in range(W) for t in range(5, V, 7)][:n]
    assert [(int(a), int(b)) for a, b in zip(par[1], tok[1])] == want


@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
def test_logits_in_order(dt):
    # rising and falling along the vocabulary, in steps that the type can tell apart or not
    V, n = 40000, 8
    for x in (torch.arange(V) / 500.0, -torch.arange(V) / 500.0, torch.arange(V) // 1000 * 1.0):
        logits = x.to(dt).cuda().expand(2, 2, V).contiguous()
        scores = torch.tensor([[-1.0, -0.5], [0.0, 0.0]], device="cuda")
        check(logits, scores, n, binding.beam_select(logits, scores, n))


def test_identical_beams_and_one_workspace_twice():
    g = torch.Generator("cuda").manual_seed(8)
    row = torch.randn(151936, generator=g, device="cuda").bfloat16()
    logits = row.expand(1, 4, -1).contiguous()
    scores = torch.full((1, 4), -1.5, device="cuda")
    ws = binding.alloc_beam_workspace(1, 4, 151936, 8)
    first = binding.beam_select(logits, scores, 8, workspace=ws)
    again = binding.beam_select(logits, scores, 8, workspace=ws)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    check(logits, scores, 8, first)
    assert first[0][0, :4].tolist() == [0, 1, 2, 3]  # the same continuation of each beam


def test_selection_in_a_graph_and_on_another_stream():
    g = torch.Generator("cuda").manual_seed(21)
    logits = torch.randn(3, 4, 5003, generator=g, device="cuda")
    scores = -torch.rand(3, 4, generator=g, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = binding.beam_select(logits, scores, 4, stream=s)
    s.synchronize()
    check(logits, scores, 4, got)
    ws = binding.alloc_beam_workspace(3, 4, 5003, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = binding.beam_select(logits, scores, 4, workspace=ws)
    logits.copy_(torch.randn(3, 4, 5003, generator=g, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    check(logits, scores, 4, got)


# ------------------------------------------------------------------------------------
# forks
# ------------------------------------------------------------------------------------
def fork_case(groups, n_in, n_out, lens, layers, hkv, d, dt, seed, width=None):
    g = torch.Generator().manual_seed(seed)
    N, M = groups * n_in, groups * n_out
    pages = [(L + 15) // 16 for L in lens]
    width = width or max(pages) + 1
    nb = sum(pages) + M + 3
    ids = torch.randperm(nb, generator=g).int()
    bt = torch.full((N, width), -1, dtype=torch.int32)
    at = 0
    for i, p in enumerate(pages):
        bt[i, :p] = ids[at:at + p]
        at += p
    tails = ids[at:at + M].view(groups, n_out).clone()
    parents = torch.randint(0, n_in, (groups, n_out), generator=g).int()
    pools = torch.randn(2, layers, nb, 16, hkv, d, generator=g).to(dt)
    return bt, torch.tensor(lens).int(), parents, tails, pools


def fork_ref(bt, lens, parents, tails, pools, out_bt, out_lens):
    groups, n_out = parents.shape
    n_in = bt.shape[0] // groups
    bt2, len2, p2 = out_bt.clone(), out_lens.clone(), pools.clone()
    for c in range(groups * n_out):
        g, i = divmod(c, n_out)
        par = int(parents[g, i])
        if par < 0 or par >= n_in:
            len2[c] = 0
            continue
        r = g * n_in + par
        L = int(lens[r])
        if L < 0 or (L + 15) // 16 > bt.shape[1]:
            len2[c] = 0
            continue
        full, rest = divmod(L, 16)
        len2[c] = L
        bt2[c, :full] = bt[r, :full]
        if rest:
            bt2[c, full] = tails[g, i]
            p2[:, :, int(tails[g, i]), :rest] = pools[:, :, int(bt[r, full]), :rest]
    return bt2, len2, p2


def run_fork(bt, lens, parents, tails, pools, err=0):
    out_bt = torch.full((parents.numel(), bt.shape[1]), -7, dtype=torch.int32)
    out_lens = torch.full((parents.numel(),), -7, dtype=torch.int32)
    want = fork_ref(bt, lens, parents, tails, pools, out_bt, out_lens)
    dp, ob, ol = pools.cuda(), out_bt.cuda(), out_lens.cuda()
    binding.fork_sequences(bt.cuda(), lens.cuda(), parents.cuda(), tails.cuda(), dp[0], dp[1], ob,
                           ol)
    assert binding.device_error() == err
    assert torch.equal(ob.cpu(), want[0]) and torch.equal(ol.cpu(), want[1])
    assert torch.equal(dp.cpu().view(torch.int16), want[2].view(torch.int16))


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("groups,n_in,n_out,lens,layers,hkv,d", [
    (1, 1, 4, [300], 1, 2, 128), (1, 1, 1, [0], 1, 1, 64), (2, 2, 2, [16, 32, 1, 15], 3, 2, 64),
    (3, 4, 4, [17, 17, 17, 17, 31, 31, 31, 31, 640, 640, 640, 640], 5, 8, 128),
    (1, 3, 8, [1000, 5, 16], 28, 1, 64)])
def test_forks(groups, n_in, n_out, lens, layers, hkv, d, dt):
    run_fork(*fork_case(groups, n_in, n_out, lens, layers, hkv, d, dt, len(lens)))


def test_fork_leaves_out_dead_and_bad_parents():
    bt, lens, parents, tails, pools = fork_case(2, 3, 3, [20, 33, 47, 9, 16, 100], 2, 2, 64,
                                                torch.bfloat16, 4)
    parents[0] = torch.tensor([-1, 2, 2])
    parents[1] = torch.tensor([1, -5, 0])
    run_fork(bt, lens, parents, tails, pools)
    parents[0, 0] = 3
    run_fork(bt, lens, parents, tails, pools, err=3)
    parents[0, 0] = 0
    lens[0] = 16 * bt.shape[1] + 1  # beyond the table
    run_fork(bt, lens, parents, tails, pools, err=3)


def test_fork_skips_blocks_outside_the_pool():
    bt, lens, parents, tails, pools = fork_case(1, 1, 2, [25], 1, 2, 64, torch.float16, 6)
    tails[0, 1] = pools.shape[2]
    dp = pools.cuda()
    ob, ol = torch.zeros(2, bt.shape[1], dtype=torch.int32).cuda(), torch.zeros(2).int().cuda()
    binding.fork_sequences(bt.cuda(), lens.cuda(), parents.cuda(), tails.cuda(), dp[0], dp[1], ob,
                           ol)
    assert binding.device_error() == 1
    want = pools.clone()
    want[:, :, int(tails[0, 0]), :9] = pools[:, :, int(bt[0, 1]), :9]
    assert torch.equal(dp.cpu(), want)


def test_fork_of_one_layer_without_its_dimension():
    bt, lens, parents, tails, pools = fork_case(1, 2, 2, [25, 40], 1, 2, 64, torch.float16, 7)
    ob = torch.full((2, bt.shape[1]), -7, dtype=torch.int32)
    ol = torch.zeros(2, dtype=torch.int32)
    want = fork_ref(bt, lens, parents, tails, pools, ob, ol)
    dp, ob, ol = pools[:, 0].contiguous().cuda(), ob.cuda(), ol.cuda()
    binding.fork_sequences(bt.cuda(), lens.cuda(), parents.cuda(), tails.cuda(), dp[0], dp[1], ob,
                           ol)
    assert torch.equal(ob.cpu(), want[0]) and torch.equal(dp.cpu(), want[2][:, 0])


# ------------------------------------------------------------------------------------
# masks that are finite numbers
# ------------------------------------------------------------------------------------
MIN32, MIN16 = torch.finfo(torch.float32).min, torch.finfo(torch.bfloat16).min


def best_of(logits, scores, n):
    """(score, flat index), best first, in 64 bits with the largest logit taken off first (a log
    of the sum added to a logit of 1e30 is lost in 64 bits too); below fp32's range -inf."""
    B, W, V = logits.shape
    res = []
    for b in range(B):
        cand = []
        for w in range(W):
            x = logits[b, w].double().cpu()
            d = x - x.max()
            s = float(scores[b, w]) + (d - math.log(float(torch.exp(d).sum())))
            s = torch.where(s < MIN32 * (1 + 2.0 ** -25), -math.inf, s)
            for t in torch.sort(-x, stable=True).indices[:n].tolist():
                cand.append((float(s[t]), w * V + t))
        res.append(sorted(cand, key=lambda c: (-c[0], c[1]))[:n])
    return res


def check_best(logits, scores, n, got, live=None):
    """Parents, tokens and scores; with `live` only the first `live` of each prompt by index. A
    score is the sum of numbers up to its size, 48 bits of them (2^-46), and the fp32 rounding."""
    par, tok, val = (x.cpu() for x in got)
    V = logits.shape[2]
    for b, want in enumerate(best_of(logits, scores, n)):
        for i, (s, flat) in enumerate(want):
            got_s = float(val[b, i])
            assert got_s == s or abs(got_s - s) <= LSE_TOL + 2.0 ** -23 * abs(s), (b, i, got_s, s)
            if live is None or i < live:
                assert (int(par[b, i]), int(tok[b, i])) == (flat // V, flat % V), (b, i)


@pytest.mark.parametrize("dt,mask", [
    (torch.float32, MIN32), (torch.float32, -1e30), (torch.float32, -1e12), (torch.float32, -1e10),
    (torch.float32, -1e9), (torch.float32, -1e4), (torch.bfloat16, MIN16), (torch.bfloat16, -1e10),
    (torch.float16, -65504.0)])
@pytest.mark.parametrize("V", [700, 50001, 151936])
def test_finite_masks(dt, mask, V):
    # constrained to a few tokens (whole threads and chunks masked); a vocabulary's tail masked;
    # every other run of 8 masked, ahead of live ones in a thread's rounds; the first half masked
    g = torch.Generator("cuda").manual_seed(V)
    scores = torch.tensor([[-1.0, -4.0, -9.0, -13.0]] * 4, device="cuda")
    logits = (torch.randn(4, 4, V, generator=g, device="cuda") * 3).to(dt)
    keep = logits.clone()
    logits[0] = mask
    for w, t in enumerate((1, V // 2, V - 1, 17)):
        logits[0, w, t] = keep[0, w, t]
        logits[0, w, (t + 300) % V] = keep[0, w, 0]
    logits[1, :, V - 200:] = mask
    logits[2] = torch.where(torch.arange(V, device="cuda") // 8 % 2 == 0, mask, keep[2])
    logits[3, :, :V // 2] = mask
    got = binding.beam_select(logits, scores, 8)
    check_best(logits, scores, 8, got)
    # more than the live tokens: the masked ones, whose order is decided where fp32 pairs tell
    # the beams' scores apart; their scores are those of the masks
    check_best(logits, scores, 12, binding.beam_select(logits, scores, 12), live=8)


@pytest.mark.parametrize("dt,fill", [
    (torch.float32, MIN32), (torch.float32, -1e30), (torch.float32, -1e10), (torch.float32, 1e10),
    (torch.float32, 3.4e38), (torch.bfloat16, MIN16), (torch.bfloat16, -1e10),
    (torch.bfloat16, 3.3e38), (torch.float16, 65504.0)])
@pytest.mark.parametrize("V", [9, 8200, 151936])
def test_every_logit_the_same_far_from_zero(dt, fill, V):
    logits = torch.full((2, 3, V), fill, device="cuda", dtype=dt)
    scores = torch.tensor([[-1.0, -2.0, -4.0], [-7.0, -1.0, -2.0]], device="cuda")
    check_best(logits, scores, 6, binding.beam_select(logits, scores, 6))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_large_logits_among_small_ones(dt):
    # one logit far above (alone it has all the weight), one thread's share, a whole chunk
    V = 151936
    g = torch.Generator("cuda").manual_seed(5)
    logits = torch.randn(3, 2, V, generator=g, device="cuda").to(dt)
    logits[0, :, 77] = 1e10
    logits[1, :, 800:808] = 1e10
    logits[2, 0, 4096:8192] = 3e38
    logits[2, 1] = -3e38
    logits[2, 1, 5] = 3e38
    scores = torch.tensor([[-1.0, -3.0]] * 3, device="cuda")
    check_best(logits, scores, 8, binding.beam_select(logits, scores, 8), live=1)


def test_scores_and_logits_both_masked():
    # the first step with the other beams at finfo.min, and logits at finfo.min: their sums leave
    # fp32 and come last, at -inf
    V, n = 20011, 8
    scores = torch.tensor([[-1.0, MIN32, MIN32]], device="cuda")
    logits = torch.full((1, 3, V), MIN32, device="cuda")
    logits[0, 0, 4:7] = torch.tensor([1.0, 3.0, 2.0])
    logits[0, 1, 9] = logits[0, 2, 3] = 0.0
    got = binding.beam_select(logits, scores, n)
    check_best(logits, scores, n, got, live=3)
    fin = torch.tensor([[0, 1, 0]], dtype=torch.uint8, device="cuda")
    par, tok, val = binding.beam_select(logits, scores, n, finished=fin, pad_token=2)
    assert par[0, :3].tolist() == [0, 0, 0] and tok[0, :3].tolist() == [5, 6, 4]
    assert (val[0, 3:] == MIN32).all()
    logits[0, 0] = torch.where(logits[0, 0] == MIN32, -math.inf, logits[0, 0])
    par, tok, val = binding.beam_select(logits, scores, n)
    assert par[0].tolist() == [0, 0, 0, 1, 2, 1, 1, 1]
    assert tok[0].tolist() == [5, 6, 4, 9, 3, 0, 1, 2]
    assert (val[0, 3:5] == MIN32).all() and (val[0, 5:] == -math.inf).all()
