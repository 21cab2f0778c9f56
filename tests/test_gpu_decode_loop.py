"""The operators together, as a decode loop of beam search calls them: rotary positions into
the cache, masked attention over it, a toy head, selection, forks of the cache."""
import pytest
import torch

from paged_kv_attention_18_gb300 import binding, rotary
from tests import operator_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,hq,hkv,d,window", [(torch.bfloat16, 12, 2, 128, 24),
                                                (torch.float16, 8, 8, 64, 0)])
def test_beam_search_steps(dt, hq, hkv, d, window):
    P, W, V, width = 2, 3, 501, 6
    g = torch.Generator("cuda").manual_seed(4)
    emb = torch.randn(V, (hq + 2 * hkv) * d, generator=g, device="cuda").to(dt)
    head = torch.randn(hq * d, V, generator=g, device="cuda") * 0.3
    nb = 80
    k_pool = torch.full((nb, 16, hkv, d), float("nan"), dtype=dt, device="cuda")
    v_pool = k_pool.clone()
    freq = rotary.frequencies(d // 2, 1e4, factor=2.0, device="cuda")
    slopes = (2.0 ** -torch.arange(1.0, hq + 1)).cuda()
    free = list(range(nb))
    # prompts of 21 and 30 tokens, prefilled as chunks
    lens = [21, 30]
    tables = torch.full((P, width), -1, dtype=torch.int32)
    for p, L in enumerate(lens):
        for i in range((L + 15) // 16):
            tables[p, i] = free.pop()
    tables = tables.cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    tokens = torch.randint(0, V, (sum(lens),), generator=g, device="cuda")
    history = None

    def layer(tokens, tables, sl, counts):
        """One layer's attention of the new tokens; history of each sequence updated."""
        nonlocal history
        B, T = len(counts), tokens.numel()
        qs = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
        qkv = emb[tokens].view(T, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        pos = torch.cat([torch.arange(int(sl[b]) - n, int(sl[b])) for b, n in enumerate(counts)])
        pos = pos.int().cuda()
        slots = binding.slot_mapping(tables, sl, qs, T, nb)
        qr = torch.empty(T, hq, d, dtype=dt, device="cuda")
        binding.rotary_reshape_and_cache(q, k, v, pos, slots, k_pool, v_pool, freq,
                                         interleaved=True, q_out=qr)
        out = binding.masked_paged_attention(qr, k_pool, v_pool, tables, sl, qs, d ** -0.5,
                                             softcap=20.0, distance_slopes=slopes, window=window)
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        # the cached rows: turned keys, values as they are
        flat_k, flat_v = k_pool.view(-1, hkv, d)[slots.long()], v_pool.view(-1, hkv, d)[slots.long()]
        ref, pair = R.rotary(k, pos, freq, True, 1.0)
        u = torch.finfo(dt).eps / 2
        assert ((flat_k.double() - ref).abs() <= u * ref.abs() + 2.0 ** -20 * pair
                + torch.finfo(dt).smallest_normal * u).all()
        assert torch.equal(flat_v, v)
        at = 0
        for b, n in enumerate(counts):
            hk = flat_k[at:at + n] if history[b] is None else torch.cat([history[b][0], flat_k[at:at + n]])
            hv = flat_v[at:at + n] if history[b] is None else torch.cat([history[b][1], flat_v[at:at + n]])
            history[b] = (hk, hv)
            ref, absv, size, tail = R.attend_dense(qr[at:at + n], hk, hv, pos[at:at + n],
                                                   d ** -0.5, 20.0, slopes, window)
            tol = R.attention_tolerance(ref, absv, size, tail, d, dt)
            assert ((out[at:at + n].double() - ref).abs() <= tol).all(), b
            at += n
        return out

    history = [None] * P
    out = layer(tokens, tables, sl, lens)
    last = out[(sl.cumsum(0) - 1).long()]
    n_in, scores = 1, torch.zeros(P, 1, device="cuda")
    for step in range(14):
        logits = (last.float().view(P, n_in, -1) @ head)
        par, tok, scores = binding.beam_select(logits, scores, W)
        for b, cand in enumerate(R.beam(logits, torch.zeros_like(scores) if n_in == 1 else prev, W)):
            assert [(int(a), int(t)) for a, t in zip(par[b], tok[b])] == \
                [(c[1] // V, c[1] % V) for c in cand[:W]]
        prev = scores
        # fork: tails of the children's own; the parents' tails go back afterwards
        tails = torch.tensor([free.pop() for _ in range(P * W)], dtype=torch.int32).view(P, W)
        new_t = torch.full((P * W, width), -1, dtype=torch.int32, device="cuda")
        new_l = torch.empty(P * W, dtype=torch.int32, device="cuda")
        binding.fork_sequences(tables, sl, par, tails.cuda(), k_pool, v_pool, new_t, new_l)
        assert binding.device_error() == 0
        src = [p * n_in + int(par[p, w]) for p in range(P) for w in range(W)]
        assert new_l.tolist() == [int(sl[s]) for s in src]
        held = set(new_t[new_t >= 0].tolist())
        free = [i for i in range(nb) if i not in held]
        tables, sl, n_in = new_t, new_l + 1, W
        for c in range(P * W):  # a block for the next token where the last one is full
            if int(new_l[c]) % 16 == 0:
                tables[c, int(new_l[c]) // 16] = free.pop()
        history = [history[s] for s in src]
        last = layer(tok.view(-1), tables, sl, [1] * (P * W))
