"""The measured cases of four operators of the paged-cache step.

rotary   rotary positions (interleaved or half layout, whole head or part of it, a table
         of frequencies) of a step's queries and keys, with the cache write.
attend   attention over the paged cache with capped scores, a bias that falls with the
         distance, a sliding window, a bidirectional prefix or documents packed into one
         sequence; decode rows and chunks of new tokens.
select   beam search's choice over beams and vocabulary.
fork     the cache after that choice: block tables by parent, the partly filled last
         block of every child in a block of its own.

``own`` chooses between the plain form (elementary torch operations) and the calls of
this repository's binding.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PAGE = 16


def _binding():
    from paged_kv_attention_18_gb300 import binding
    return binding


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------
def _rotary(T, hq, hkv, d, rot, inter, dtype, factor):
    return {"op": "rotary", "T": T, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "inter": inter,
            "dtype": dtype, "factor": factor}


def _attend(B, n, ctx, hq, hkv, d, dtype, cap=0.0, slopes=False, window=0, prefix=0, docs=0):
    """n: new tokens of a sequence, at most; ctx: context after them, at most (both ragged);
    prefix: bidirectional keys at a sequence's start; docs: documents a chunk is packed of."""
    return {"op": "attend", "B": B, "n": n, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "cap": cap, "slopes": slopes, "window": window, "prefix": prefix,
            "docs": docs}


def _select(B, W, V, n, dtype, finished):
    return {"op": "select", "B": B, "W": W, "V": V, "n": n, "dtype": dtype,
            "finished": finished}


def _fork(B, win, wout, ctx, layers, hkv, d, dtype):
    return {"op": "fork", "B": B, "win": win, "wout": wout, "ctx": ctx, "layers": layers,
            "hkv": hkv, "d": d, "dtype": dtype}


def listed():
    return [
        # one token of a small model: the latency of a call
        {"name": "rotary_one_token", **_rotary(1, 14, 2, 64, 32, True, "f16", 1.0)},
        # a decode step of many sequences, interleaved, whole head, scaled positions
        {"name": "rotary_decode_batch", **_rotary(257, 12, 2, 128, 128, True, "bf16", 4.0)},
        # prompts: half of each head rotated, half layout
        {"name": "rotary_prompt", **_rotary(8192, 32, 8, 128, 64, False, "bf16", 8.0)},
        # a few short sequences with capped scores: the latency of a call
        {"name": "attend_tiny_capped", **_attend(4, 1, 128, 12, 2, 128, "bf16", cap=30.0)},
        # decode far past a sliding window, capped scores: only the window is read
        {"name": "attend_decode_window",
         **_attend(128, 1, 32768, 16, 4, 128, "bf16", cap=50.0, window=4096)},
        # decode with a distance bias, every query head its own KV head
        {"name": "attend_decode_bias", **_attend(64, 1, 8191, 16, 16, 64, "f16", slopes=True)},
        # chunks of prompts with capped scores
        {"name": "attend_chunk_capped", **_attend(4, 2048, 8192, 32, 8, 128, "bf16", cap=30.0)},
        # ragged chunks of packed documents behind a bidirectional prefix
        {"name": "attend_chunk_prefix_docs",
         **_attend(6, 1000, 1500, 14, 2, 64, "f16", prefix=130, docs=5)},
        # one prompt's beams over a small odd vocabulary
        {"name": "select_one_prompt", **_select(1, 4, 1003, 4, "f32", False)},
        # many prompts over a large vocabulary, twice the beams kept, some beams finished
        {"name": "select_batch", **_select(48, 4, 151936, 8, "bf16", True)},
        # a prompt's cache forked into its beams
        {"name": "fork_prompt", **_fork(1, 1, 4, 300, 1, 2, 128, "bf16")},
        # the beams of many prompts through every layer's cache
        {"name": "fork_batch", **_fork(32, 4, 4, 1021, 28, 2, 128, "bf16")},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "attend", "attend", "select", "fork"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "rotary":
        hq, hkv = rng.choice([(14, 2), (12, 2), (32, 8), (16, 16), (7, 1)])
        d = rng.choice([64, 128])
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d])
        return _rotary(_log(rng, 1, 8192), hq, hkv, d, rot, rng.random() < 0.5, dtype,
                       rng.choice([1.0, 4.0, 8.0]))
    if op == "attend":
        hq, hkv = rng.choice([(14, 2), (12, 2), (16, 4), (32, 8), (8, 8), (7, 1)])
        d = rng.choice([64, 128])
        kind = rng.choice(["cap", "bias", "window", "prefix", "docs", "all"])
        cap = rng.choice([20.0, 30.0, 50.0]) if kind in ("cap", "all") else 0.0
        slopes = kind in ("bias", "all")
        if rng.random() < 0.5:  # decode rows, or a few tokens to verify
            n, B = rng.choice([1, 1, 1, 4]), _log(rng, 1, 96)
            ctx = _log(rng, 1, min(16384, 500_000_000 // (B * hkv * d)))
        else:
            n, B = _log(rng, 17, 1500), rng.randint(1, 4)
            ctx = n + rng.choice([0, _log(rng, 1, 4000)])
        n = min(n, ctx)
        window = _log(rng, 1, 4096) if kind in ("window", "all") else 0
        prefix = _log(rng, 1, max(1, ctx)) if kind == "prefix" else 0
        docs = rng.randint(2, 6) if kind == "docs" else 0
        return _attend(B, n, ctx, hq, hkv, d, dtype, cap, slopes, window, prefix, docs)
    if op == "select":
        W = rng.choice([1, 2, 3, 4, 8])
        V = _log(rng, 50, 151936)
        n = min(rng.choice([W, 2 * W]), W * V)
        return _select(_log(rng, 1, 192 // W), W, V, n, rng.choice(["bf16", "f16", "f32"])
                       if V < 60000 else dtype, rng.random() < 0.5)
    win, wout = rng.choice([(1, 4), (4, 4), (1, 5), (3, 3), (8, 8)])
    hkv, d = rng.choice([(2, 128), (2, 64), (8, 128), (1, 64)])
    layers = _log(rng, 1, max(1, 28 * 2 * 128 // (hkv * d) // 2))
    return _fork(_log(rng, 1, 16), win, wout, _log(rng, 1, 1021), layers, hkv, d, dtype)


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------
def _ragged(g, count, most, least):
    """`count` lengths in [least, most], the first of them `most`."""
    x = torch.randint(least, most + 1, (count,), generator=g)
    x[0] = most
    return x


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=gg, device="cuda") * std).to(dtype)

    return {"rotary": _prepare_rotary, "attend": _prepare_attend, "select": _prepare_select,
            "fork": _prepare_fork}[case["op"]](case, g, gg, dt, normal)


def _prepare_rotary(c, g, gg, dt, normal):
    T, hq, hkv, d, R = c["T"], c["hq"], c["hkv"], c["d"], c["rot"]
    # the three are views of one projection's output, as a layer has them
    qkv = normal(T, hq + 2 * hkv, d)
    nb = (T + PAGE - 1) // PAGE + 4
    slots = torch.randperm(nb * PAGE, generator=g)[:T].to(torch.int32)
    # long contexts: positions up to 128 Ki tokens; wavelengths stretched by `factor`
    pos = torch.randint(0, 1 << 17, (T,), generator=g, dtype=torch.int32)
    freq = 10000.0 ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R) / c["factor"]
    return {"case": c, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
            "pos": pos.cuda(), "slots": slots.cuda(), "freq": freq.cuda(),
            "mag": 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0,
            "q_out": torch.empty(T, hq, d, dtype=dt, device="cuda"),
            "k_pool": normal(nb, PAGE, hkv, d), "v_pool": normal(nb, PAGE, hkv, d)}


def _attend_shape(c):
    """Host lengths of a batch: contexts, new tokens, prefixes. They are the case's own, so
    that inputs of every seed have the same number of packed tokens."""
    B, n, ctx = c["B"], c["n"], c["ctx"]
    g = torch.Generator().manual_seed(B * 1_000_003 + n * 1009 + ctx)
    news = _ragged(g, B, n, max(1, n // 2))
    lens = torch.maximum(_ragged(g, B, ctx, max(1, ctx // 2)), news)
    pre = torch.randint(c["prefix"] // 2, c["prefix"] + 1, (B,), generator=g)
    return lens, news, pre


def _starts(c, g, lens, news):
    """First key of each new token's document, per packed token (0 without documents)."""
    T = int(news.sum())
    seq = torch.repeat_interleave(torch.arange(c["B"]), news)
    first = torch.cat([torch.zeros(1, dtype=torch.long), news.cumsum(0)[:-1]])
    pos = (lens - news)[seq] + torch.arange(T) - first[seq]
    if not c["docs"]:
        return seq, pos, torch.zeros(T, dtype=torch.long)
    # document borders of a sequence, in order; a token's document starts at the last
    # border at or before it
    cuts = (torch.rand(c["B"], c["docs"], generator=g) * lens[:, None]).long()
    below = cuts[seq] <= pos[:, None]
    return seq, pos, torch.where(below, cuts[seq], 0).max(1).values


def _prepare_attend(c, g, gg, dt, normal):
    B, hq, hkv, d = c["B"], c["hq"], c["hkv"], c["d"]
    lens, news, pre = _attend_shape(c)
    seq, pos, start = _starts(c, g, lens, news)
    T = int(news.sum())
    qsl = torch.cat([torch.zeros(1, dtype=torch.long), news.cumsum(0)])
    pages = (lens + PAGE - 1) // PAGE
    most = int(pages.max())
    # blocks of a pool in random order; what lies before a sliding window has been given
    # back, and its entries are -1
    col = torch.arange(most)[None, :]
    low = torch.zeros(B, dtype=torch.long)
    if c["window"]:
        low = (lens - news - c["window"] + 1).clamp(min=0)
    held = (col < pages[:, None]) & (col >= (low // PAGE)[:, None])
    count = int(held.sum())
    nb = count + count // 16 + 1
    bt = torch.full((B, most), -1, dtype=torch.int32)
    bt[held] = torch.randperm(nb, generator=g)[:count].to(torch.int32)
    # queries wide enough that a cap bends the scores
    st = {"case": c, "q": normal(T, hq, d, std=3.0 if c["cap"] else 1.0),
          "k_pool": normal(nb, PAGE, hkv, d), "v_pool": normal(nb, PAGE, hkv, d),
          "bt": bt.cuda(), "lens": lens.to(torch.int32).cuda(),
          "qsl": qsl.to(torch.int32).cuda(), "scale": d ** -0.5,
          "slopes": (2.0 ** (-8.0 * torch.arange(1, hq + 1) / hq)).float().cuda()
          if c["slopes"] else None,
          "pre": pre.to(torch.int32).cuda() if c["prefix"] else None,
          "start": start.to(torch.int32).cuda() if c["docs"] else None,
          "out": torch.empty(T, hq, d, dtype=dt, device="cuda"),
          # what the program knows of its batch on the host
          "T": T, "most_new": int(news.max()), "most_len": int(lens.max()),
          "span": int((lens - low).max()), "low": low.cuda()}
    st["ws"] = None
    return st


def _prepare_select(c, g, gg, dt, normal):
    B, W, V = c["B"], c["W"], c["V"]
    scores = -torch.rand(B, W, generator=gg, device="cuda") * 8.0
    fin = torch.zeros(B, W, dtype=torch.uint8)
    if c["finished"]:
        fin = (torch.rand(B, W, generator=g) < 0.25).to(torch.uint8)
    return {"case": c, "logits": normal(B, W, V, std=3.0), "scores": scores,
            "fin": fin.cuda() if c["finished"] else None, "pad": V - 1, "ws": None}


def _prepare_fork(c, g, gg, dt, normal):
    B, win, wout, ctx, hkv, d = c["B"], c["win"], c["wout"], c["ctx"], c["hkv"], c["d"]
    lens = torch.repeat_interleave(_ragged(g, B, ctx, max(1, ctx // 2)), win)
    pages = (lens + PAGE - 1) // PAGE
    most = int(pages.max()) + 1
    # a prompt's beams share its blocks but for their last ones
    own_pages = 3
    group = torch.arange(B * win) // win
    nb_shared = B * most
    nb = nb_shared + B * win * own_pages + B * wout
    ids = torch.randperm(nb, generator=g).to(torch.int32)
    col = torch.arange(most)[None, :]
    shared = ids[group[:, None] * most + col]
    private = ids[nb_shared + torch.arange(B * win)[:, None] * own_pages
                  + (pages[:, None] - 1 - col).clamp(0, own_pages - 1)]
    bt = torch.where(pages[:, None] - 1 - col < own_pages, private, shared)
    bt = torch.where(col < pages[:, None], bt, -1).to(torch.int32)
    tails = ids[nb - B * wout:].view(B, wout).clone()
    parents = torch.randint(0, win, (B, wout), generator=g, dtype=torch.int32)
    L = c["layers"]
    return {"case": c, "bt": bt.cuda(), "lens": lens.to(torch.int32).cuda(),
            "parents": parents.cuda(), "tails": tails.cuda(),
            "k_pool": normal(L, nb, PAGE, hkv, d), "v_pool": normal(L, nb, PAGE, hkv, d),
            "out_bt": torch.full((B * wout, most), -1, dtype=torch.int32, device="cuda"),
            "out_lens": torch.zeros(B * wout, dtype=torch.int32, device="cuda")}


# ------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "attend": _own_attend, "select": _own_select,
                "fork": _own_fork}[op](state)
    return {"rotary": _plain_rotary, "attend": _plain_attend, "select": _plain_select,
            "fork": _plain_fork}[op](state)


def _own_rotary(s):
    _binding().rotary_reshape_and_cache(s["q"], s["k"], s["v"], s["pos"], s["slots"],
                                        s["k_pool"], s["v_pool"], s["freq"],
                                        interleaved=s["case"]["inter"], magnitude=s["mag"],
                                        q_out=s["q_out"])
    return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}


def _own_attend(s):
    b, c = _binding(), s["case"]
    if s["ws"] is None:  # a program's workspace, kept from step to step
        s["ws"] = b.alloc_workspace(s["T"], c["B"], c["hq"], c["hkv"], c["d"], s["most_len"])
    return b.masked_paged_attention(s["q"], s["k_pool"], s["v_pool"], s["bt"], s["lens"],
                                    s["qsl"], s["scale"], softcap=c["cap"],
                                    distance_slopes=s["slopes"], window=c["window"],
                                    prefix_lens=s["pre"], key_starts=s["start"], out=s["out"],
                                    workspace=s["ws"])


def _own_select(s):
    b, c = _binding(), s["case"]
    if s["ws"] is None:
        s["ws"] = b.alloc_beam_workspace(c["B"], c["W"], c["V"], c["n"])
    return b.beam_select(s["logits"], s["scores"], c["n"], finished=s["fin"],
                         pad_token=s["pad"], workspace=s["ws"])


def _own_fork(s):
    _binding().fork_sequences(s["bt"], s["lens"], s["parents"], s["tails"], s["k_pool"],
                              s["v_pool"], s["out_bt"], s["out_lens"])
    return {"bt": s["out_bt"], "lens": s["out_lens"], "k": s["k_pool"], "v": s["v_pool"]}


def _turn(x, cos, sin, R, inter, dt):
    """x [T, H, d] turned by cos, sin [T, 1, R/2] over its first R elements."""
    x = x.float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([y, x[..., R:]], -1).to(dt)


def _plain_rotary(s):
    c = s["case"]
    R, dt = c["rot"], s["q"].dtype
    ang = s["pos"].double()[:, None, None] * s["freq"]  # far positions: 64 bits
    cos, sin = (s["mag"] * ang.cos()).float(), (s["mag"] * ang.sin()).float()
    s["q_out"].copy_(_turn(s["q"], cos, sin, R, c["inter"], dt))
    at = s["slots"].long()
    s["k_pool"].view(-1, c["hkv"], c["d"])[at] = _turn(s["k"], cos, sin, R, c["inter"], dt)
    s["v_pool"].view(-1, c["hkv"], c["d"])[at] = s["v"]
    return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}


def _plain_attend(s):
    c = s["case"]
    B, hq, hkv, d, n, span = c["B"], c["hq"], c["hkv"], c["d"], s["most_new"], s["span"]
    lens, qsl, dev = s["lens"].long(), s["qsl"].long(), s["q"].device
    news = qsl[1:] - qsl[:-1]
    key = s["low"][:, None] + torch.arange(span, device=dev)                # [B, span]
    page = (key // PAGE).clamp(max=s["bt"].shape[1] - 1)
    at = s["bt"].gather(1, page).long().clamp(min=0) * PAGE + key % PAGE
    k = s["k_pool"].view(-1, hkv, d)[at].float().permute(0, 2, 3, 1)       # [B, hkv, d, span]
    v = s["v_pool"].view(-1, hkv, d)[at].float().permute(0, 2, 1, 3)       # [B, hkv, span, d]
    i = torch.arange(n, device=dev)
    row = (qsl[:-1, None] + i).clamp(max=s["T"] - 1)                        # [B, n]
    q = s["q"][row].float().view(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    x = (q.reshape(B, hkv, -1, d) @ k).view(B, hq, n, span) * s["scale"]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    pos = (lens - news)[:, None] + i                                        # [B, n]
    away = pos[:, :, None] - key[:, None, :]                                # [B, n, span]
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * away[:, None].abs()
    see = away >= 0
    if s["pre"] is not None:
        see = see | (key < s["pre"][:, None])[:, None, :]
    see = see & (key < lens[:, None])[:, None, :]
    if c["window"]:
        see = see & (away < c["window"])
    if s["start"] is not None:
        see = see & (key[:, None, :] >= s["start"][row][:, :, None])
    x = x.masked_fill(~see[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    y = (x.view(B, hkv, -1, span) @ v).view(B, hq, n, d).transpose(1, 2)    # [B, n, hq, d]
    seq = torch.arange(B, device=dev).repeat_interleave(news, output_size=s["T"])
    s["out"].copy_(y[seq, torch.arange(s["T"], device=dev) - qsl[seq]])
    return s["out"]


def _plain_select(s):
    c = s["case"]
    B, W, V, n = c["B"], c["W"], c["V"], c["n"]
    x = s["logits"].double()  # candidates next to one another: 64 bits
    top = x.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    cand = s["scores"].double()[:, :, None] + (x - lse)
    if s["fin"] is not None:  # a finished beam has one candidate: the pad token, unchanged
        only = torch.full((V,), -math.inf, dtype=torch.float64, device=x.device)
        only[s["pad"]] = 0.0
        cand = torch.where(s["fin"][:, :, None] != 0, s["scores"].double()[:, :, None] + only,
                           cand)
    best, at = torch.sort(cand.view(B, W * V), dim=-1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    none = best == -math.inf
    return (torch.where(none, -1, at // V).int(), torch.where(none, -1, at % V).int(),
            best.float())


def _plain_fork(s):
    c = s["case"]
    B, win, wout = c["B"], c["win"], c["wout"]
    dev = s["bt"].device
    src = (torch.arange(B, device=dev)[:, None] * win + s["parents"]).view(-1)
    lens = s["lens"][src].long()
    tails = s["tails"].view(-1)
    full, rest = lens // PAGE, lens % PAGE
    col = torch.arange(s["bt"].shape[1], device=dev)[None, :]
    last = (col == full[:, None]) & (rest[:, None] > 0)
    table = s["bt"][src]
    s["out_bt"].copy_(torch.where(col < full[:, None], table,
                                  torch.where(last, tails[:, None], s["out_bt"])))
    s["out_lens"].copy_(lens)
    page = table.gather(1, full[:, None]).view(-1).long().clamp(min=0)
    keep = (torch.arange(PAGE, device=dev) < rest[:, None])[None, :, :, None, None]
    to = tails.long()
    for pool in (s["k_pool"], s["v_pool"]):
        pool[:, to] = torch.where(keep, pool[:, page], pool[:, to])
    return {"bt": s["out_bt"], "lens": s["out_lens"], "k": s["k_pool"], "v": s["v_pool"]}


# ------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------
def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rotary":
        T, hq, hkv, d = c["T"], c["hq"], c["hkv"], c["d"]
        return {"bytes": 2 * T * (hq + 2 * hkv) * d * size + 8 * T + 4 * c["rot"],
                "flops": 3 * T * (hq + hkv) * c["rot"]}
    if c["op"] == "attend":
        lens, news, pre = _attend_shape(c)
        # (the documents' borders are drawn by the seed; of a batch like it)
        seq, pos, start = _starts(c, torch.Generator().manual_seed(1), lens, news)
        hi = torch.minimum(torch.maximum(pos + 1, pre[seq]), lens[seq])
        lo = torch.maximum(start, pos - c["window"] + 1) if c["window"] else start
        seen = (hi - lo.clamp(min=0)).clamp(min=0)
        first = torch.full((c["B"],), 1 << 40).scatter_reduce(0, seq, lo.clamp(min=0), "amin")
        end = torch.zeros(c["B"], dtype=torch.long).scatter_reduce(0, seq, hi, "amax")
        keys = int((end - first).clamp(min=0).sum())
        return {"bytes": 2 * 2 * keys * c["hkv"] * c["d"]
                + 2 * 2 * int(news.sum()) * c["hq"] * c["d"] + 4 * ((keys + PAGE) // PAGE),
                "flops": 4 * c["d"] * c["hq"] * int(seen.sum())}
    if c["op"] == "select":
        n = c["B"] * c["W"] * c["V"]
        return {"bytes": n * size + 12 * c["B"] * c["n"], "flops": 3 * n}
    rows = c["B"] * c["wout"]
    per = c["layers"] * 2 * c["hkv"] * c["d"] * size
    return {"bytes": int(rows * (2 * 7.5 * per + 2 * 4 * (0.75 * c["ctx"] / PAGE) + 16)),
            "flops": 0}


# ------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "attend": _exact_attend, "select": _exact_select,
            "fork": _exact_fork}[case["op"]](case, s)


def _exact_rotary(c, s):
    R = c["rot"]
    z = torch.polar(torch.full((c["T"], R // 2), float(s["mag"]), dtype=torch.float64,
                               device="cuda"),
                    s["pos"].double()[:, None] * s["freq"][None, :])[:, None, :]

    def turned(x):
        y = x.double().clone()
        i = torch.arange(R // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if c["inter"] else (i, i + R // 2)
        w = torch.complex(y[..., first], y[..., second]) * z
        y[..., first], y[..., second] = w.real, w.imag
        return y

    k, v = s["k_pool"].double(), s["v_pool"].double()
    block, line = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    k[block, line] = turned(s["k"])
    v[block, line] = s["v"].double()
    return {"q": turned(s["q"]), "k": k, "v": v}


def _exact_attend(c, s):
    out = torch.zeros(s["T"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lens, qsl = s["lens"].tolist(), s["qsl"].tolist()
    pre = s["pre"].tolist() if s["pre"] is not None else [0] * c["B"]
    group = c["hq"] // c["hkv"]
    for b in range(c["B"]):
        L, lo, hi = lens[b], qsl[b], qsl[b + 1]
        j = torch.arange(L, device="cuda")
        p = torch.arange(L - (hi - lo), L, device="cuda")[:, None]
        see = (j <= p) | (j < pre[b])
        if c["window"]:
            see &= j > p - c["window"]
        if s["start"] is not None:
            see &= j >= s["start"][lo:hi, None]
        used = see.any(0).nonzero().view(-1)
        if not len(used):
            continue
        j = torch.arange(int(used[0]), int(used[-1]) + 1, device="cuda")
        see = see[:, j]
        blocks = s["bt"][b, j // PAGE].long()
        for h in range(c["hq"]):
            kk = s["k_pool"][blocks, j % PAGE, h // group].double()
            vv = s["v_pool"][blocks, j % PAGE, h // group].double()
            x = s["q"][lo:hi, h].double() @ kk.T * s["scale"]
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if s["slopes"] is not None:
                x = x - (p - j).abs() * s["slopes"][h].double()
            x = torch.where(see, x, -math.inf)
            w = torch.softmax(x, -1)
            out[lo:hi, h] = torch.where(see.any(1)[:, None], w, 0.0) @ vv
    return out


def _exact_select(c, s):
    B, W, V, n = c["B"], c["W"], c["V"], c["n"]
    par, tok, val = [], [], []
    for b in range(B):
        rows = []
        for w in range(W):
            if s["fin"] is not None and int(s["fin"][b, w]):
                row = torch.full((V,), -math.inf, dtype=torch.float64, device="cuda")
                row[s["pad"]] = s["scores"][b, w].double()
            else:
                row = torch.log_softmax(s["logits"][b, w].double(), 0) + s["scores"][b, w]
            rows.append(row)
        flat = torch.cat(rows)
        # the n-th value, what lies above it, and of those equal to it the first ones
        order = torch.argsort(-flat, stable=True)[:n]
        got = flat[order]
        none = got == -math.inf
        par.append(torch.where(none, -1, order // V).int())
        tok.append(torch.where(none, -1, order % V).int())
        val.append(got)
    return torch.stack(par), torch.stack(tok), torch.stack(val)


def _exact_fork(c, s):
    bt, lens = s["out_bt"].cpu(), s["out_lens"].cpu()
    k, v = s["k_pool"].clone(), s["v_pool"].clone()
    for i in range(c["B"] * c["wout"]):
        b, w = divmod(i, c["wout"])
        src = b * c["win"] + int(s["parents"][b, w])
        L = int(s["lens"][src])
        lens[i] = L
        bt[i, :L // PAGE] = s["bt"][src, :L // PAGE].cpu()
        if L % PAGE:
            old, new = int(s["bt"][src, L // PAGE]), int(s["tails"][b, w])
            bt[i, L // PAGE] = new
            k[:, new, :L % PAGE] = s["k_pool"][:, old, :L % PAGE]
            v[:, new, :L % PAGE] = s["v_pool"][:, old, :L % PAGE]
    return {"bt": bt.cuda(), "lens": lens.cuda(), "k": k, "v": v}
