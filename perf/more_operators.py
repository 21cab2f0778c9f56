"""The measured cases of four operators of a decode loop that stays on the GPU.

sample   a token of every row of logits: temperature, top-k, top-p, min-p, one given random
         word a row.
extend   the step's blocks, slots, positions and packed offsets from each sequence's length
         and number of new tokens, blocks taken from a stack of free ones.
rotary   rotary positions with several axes (time, height, width) of a step's queries and
         keys, with the cache write.
attend   attention over the paged cache where a row sees the last keys before it (a window)
         and the first ones of its sequence (sinks).

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
def _sample(B, V, dtype, temp, k, p, m, mixed):
    """temp, k, p, m: temperature, top-k (0: all), top-p, min-p. mixed: every row has its own
    of each, some are greedy, and some have most of the vocabulary masked."""
    return {"op": "sample", "B": B, "V": V, "dtype": dtype, "temp": temp, "k": k, "p": p,
            "m": m, "mixed": mixed}


def _extend(B, n, ctx):
    """n: new tokens of a sequence, ctx: its context before them, both at most (ragged)."""
    return {"op": "extend", "B": B, "n": n, "ctx": ctx}


def _rotary(T, hq, hkv, d, sections, inter, woven, dtype):
    """sections: frequencies of each axis, as text; woven: the axes take turns along them."""
    return {"op": "rotary", "T": T, "hq": hq, "hkv": hkv, "d": d, "sections": sections,
            "inter": inter, "woven": woven, "dtype": dtype}


def _attend(B, n, ctx, hq, hkv, d, dtype, window, sinks, cap=0.0):
    """n: new tokens of a sequence, at most; ctx: context after them, at most (both ragged)."""
    return {"op": "attend", "B": B, "n": n, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "window": window, "sinks": sinks, "cap": cap}


def listed():
    return [
        # one request over a small odd vocabulary, every filter on: the latency of a call
        {"name": "sample_one", **_sample(1, 1003, "f32", 0.8, 20, 0.9, 0.02, False)},
        # a large decode batch, every request with parameters of its own
        {"name": "sample_mixed_batch", **_sample(256, 151936, "bf16", 0.7, 50, 0.9, 0.0, True)},
        # a batch by nucleus alone, logits in 32 bits
        {"name": "sample_nucleus", **_sample(48, 151936, "f32", 1.0, 0, 0.95, 0.0, False)},
        # the model's own distribution (rollouts), an odd vocabulary
        {"name": "sample_unfiltered", **_sample(100, 50257, "f16", 1.0, 0, 1.0, 0.0, False)},
        # a decode step of many sequences
        {"name": "extend_decode_batch", **_extend(256, 1, 4096)},
        # prompts of a large batch packed into one step
        {"name": "extend_prompts", **_extend(1000, 65, 2000)},
        # one token of a small model: the latency of a call
        {"name": "rotary_one_token", **_rotary(1, 14, 2, 64, "8,12,12", False, False, "f16")},
        # a prompt with images: three axes in sections, half layout
        {"name": "rotary_image_prompt",
         **_rotary(8192, 32, 8, 128, "16,24,24", False, False, "bf16")},
        # a few short streams: the latency of a call
        {"name": "attend_tiny", **_attend(4, 1, 300, 14, 2, 64, "f16", 128, 4)},
        # decode of long streams: only the sinks and the window are read
        {"name": "attend_decode_streams",
         **_attend(128, 1, 32768, 16, 4, 128, "bf16", 4096, 4)},
        # drafts verified, capped scores, sinks that end inside a page
        {"name": "attend_verify_capped",
         **_attend(36, 5, 4000, 12, 2, 128, "f16", 1000, 20, 30.0)},
        # chunks of long prompts
        {"name": "attend_chunk", **_attend(4, 2048, 8192, 32, 8, 128, "bf16", 2000, 4)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "extend", "rotary", "attend", "attend"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "sample":
        V = _log(rng, 50, 151936)
        B = _log(rng, 1, min(512, 256 * 151936 // V))
        return _sample(B, V, rng.choice(["bf16", "f16", "f32"]) if B * V < 2e7 else dtype,
                       rng.choice([0.3, 0.7, 1.0, 1.5]), rng.choice([0, 0, 1, 8, 50, 1000, V]),
                       rng.choice([1.0, 0.5, 0.8, 0.95, 0.99]), rng.choice([0.0, 0.0, 0.01, 0.1]),
                       rng.random() < 0.5)
    if op == "extend":
        if rng.random() < 0.5:
            return _extend(_log(rng, 1, 2000), rng.choice([1, 1, 5]), _log(rng, 1, 8192))
        n = _log(rng, 2, 2000)
        return _extend(_log(rng, 1, max(1, min(1000, 65000 // n))), n, _log(rng, 1, 8192))
    if op == "rotary":
        hq, hkv = rng.choice([(14, 2), (12, 2), (32, 8), (16, 16), (7, 1)])
        d = rng.choice([64, 128])
        sections = rng.choice(["8,12,12", "16,16", "11,11,10", "2,7,7", "5,5,5,1"] if d == 64
                              else ["16,24,24", "32,32", "8,12,12", "24,20,20", "16,16,16,16"])
        return _rotary(_log(rng, 1, 8192), hq, hkv, d, sections, rng.random() < 0.5,
                       rng.random() < 0.5, dtype)
    hq, hkv = rng.choice([(14, 2), (12, 2), (16, 4), (32, 8), (8, 8), (7, 1)])
    d = rng.choice([64, 128])
    window, sinks = _log(rng, 1, 4096), _log(rng, 1, 200)
    cap = rng.choice([0.0, 0.0, 20.0, 50.0])
    if rng.random() < 0.6:  # decode rows, or a few tokens to verify
        n, B = rng.choice([1, 1, 1, 4]), _log(rng, 1, 96)
        ctx = _log(rng, 1, min(16384, 500_000_000 // (B * hkv * d)))
    else:
        n, B = _log(rng, 17, 1500), rng.randint(1, 4)
        ctx = n + rng.choice([0, _log(rng, 1, 6000)])
    return _attend(B, min(n, ctx), ctx, hq, hkv, d, dtype, window, sinks, cap)


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------
def _ragged(g, count, most, least):
    """`count` numbers in [least, most], the first of them `most`."""
    x = torch.randint(least, most + 1, (count,), generator=g)
    x[0] = most
    return x


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator("cuda").manual_seed(seed)
    return {"sample": _prepare_sample, "extend": _prepare_extend, "rotary": _prepare_rotary,
            "attend": _prepare_attend}[case["op"]](case, g, gg)


def _normal(gg, dtype, *shape, std=1.0):
    return (torch.randn(*shape, generator=gg, device="cuda") * std).to(dtype)


def _prepare_sample(c, g, gg):
    B, V = c["B"], c["V"]
    x = torch.randn(B, V, generator=gg, device="cuda") * 2.5
    # a few likely tokens stand out of every row, by a different amount in each
    at = torch.randint(0, V, (B, 12), generator=gg, device="cuda")
    up = torch.rand(B, 12, generator=gg, device="cuda") * 6.0
    up = up + 10.0 * torch.rand(B, 1, generator=gg, device="cuda")
    x.scatter_(1, at, up)
    temp = torch.full((B,), c["temp"])
    k = torch.full((B,), c["k"], dtype=torch.int32)
    p, m = torch.full((B,), c["p"]), torch.full((B,), c["m"])
    if c["mixed"]:
        # rows whose vocabulary is mostly masked (a grammar's), but for its likely tokens
        bare = (torch.rand(B, generator=gg, device="cuda") < 0.2)[:, None]
        cut = torch.rand(B, V, generator=gg, device="cuda") < 0.95
        cut.scatter_(1, at, False)
        x.masked_fill_(bare & cut, -math.inf)
        temp = temp * (0.5 + torch.rand(B, generator=g))
        temp[torch.rand(B, generator=g) < 0.1] = 0.0
        k = (k * (0.2 + 2.0 * torch.rand(B, generator=g))).int()
        k[torch.rand(B, generator=g) < 0.3] = 0
        p = torch.where(torch.rand(B, generator=g) < 0.2, 1.0, p - 0.2 * torch.rand(B, generator=g))
        m = torch.where(torch.rand(B, generator=g) < 0.8, m, 0.05)
    bits = torch.randint(-(1 << 31), 1 << 31, (B,), generator=g, dtype=torch.int64)
    some = c["mixed"]
    return {"case": c, "x": x.to(DTYPES[c["dtype"]]), "bits": bits.to(torch.int32).cuda(),
            "temp": temp.cuda() if some or c["temp"] != 1.0 else None,
            "k": k.cuda() if some or c["k"] else None,
            "p": p.cuda() if some or c["p"] < 1.0 else None,
            "m": m.cuda() if some or c["m"] else None}


def _extend_shape(c):
    """Host lengths of a batch: contexts and new tokens, the case's own (see _attend_shape)."""
    g = torch.Generator().manual_seed(c["B"] * 1_000_003 + c["n"] * 1009 + c["ctx"])
    return (_ragged(g, c["B"], c["ctx"], c["ctx"] // 2),
            _ragged(g, c["B"], c["n"], 1 if c["n"] < 8 else c["n"] // 8))


def _prepare_extend(c, g, gg):
    B = c["B"]
    lens, news = _extend_shape(c)
    held = (lens + PAGE - 1) // PAGE
    after = (lens + news + PAGE - 1) // PAGE
    width = int(after.max())
    count, spare = int(held.sum()), int((after - held).sum()) + 7
    ids = torch.randperm(count + spare, generator=g).to(torch.int32)
    bt = torch.full((B, width), -1, dtype=torch.int32)
    bt[torch.arange(width)[None, :] < held[:, None]] = ids[:count]
    free = torch.full((count + spare,), -1, dtype=torch.int32)
    free[:spare] = ids[count:]
    T = int(news.sum())
    # a step of a fixed number of packed tokens, a few of them padding
    T = T + T % 3

    def buf(n):
        return torch.empty(n, dtype=torch.int32, device="cuda")

    return {"case": c, "T": T, "nb": count + spare, "bt": bt.cuda(),
            "lens": lens.to(torch.int32).cuda(), "news": news.to(torch.int32).cuda(),
            "free": free.cuda(), "count": torch.tensor([spare], dtype=torch.int32).cuda(),
            "out_lens": buf(B), "out_count": buf(1), "qsl": buf(B + 1), "slots": buf(T),
            "pos": buf(T)}


def _sections(c):
    """The axis of every frequency."""
    n = [int(x) for x in c["sections"].split(",")]
    if not c["woven"]:
        return sum(([a] * k for a, k in enumerate(n)), [])
    left, axes = list(n), []
    while sum(left):
        for a in range(len(n)):
            if left[a]:
                left[a] -= 1
                axes.append(a)
    return axes


def _prepare_rotary(c, g, gg):
    T, hq, hkv, d = c["T"], c["hq"], c["hkv"], c["d"]
    dt = DTYPES[c["dtype"]]
    axes = _sections(c)
    A, half = max(axes) + 1, len(axes)
    qkv = _normal(gg, dt, T, hq + 2 * hkv, d)
    nb = (T + PAGE - 1) // PAGE + 4
    slots = torch.randperm(nb * PAGE, generator=g)[:T].to(torch.int32)
    # text and images in turns, far into a conversation: the first axis moves with the
    # tokens, the others with a place in the image
    pos = torch.randint(0, 1 << 15, (1, 1), generator=g) + torch.arange(T)[None, :]
    pos = pos + torch.randint(0, 64, (A, T), generator=g) * (torch.arange(A) > 0)[:, None]
    freq = 1e6 ** (-torch.arange(half, dtype=torch.float64) / half)
    return {"case": c, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
            "pos": pos.to(torch.int32).cuda(), "slots": slots.cuda(), "freq": freq.cuda(),
            "axes": torch.tensor(axes, dtype=torch.int32).cuda(),
            "q_out": torch.empty(T, hq, d, dtype=dt, device="cuda"),
            "k_pool": _normal(gg, dt, nb, PAGE, hkv, d),
            "v_pool": _normal(gg, dt, nb, PAGE, hkv, d)}


def _attend_shape(c):
    """Host lengths of a batch: contexts and new tokens. They are the case's own, so that
    inputs of every seed have the same number of packed tokens."""
    B, n, ctx = c["B"], c["n"], c["ctx"]
    g = torch.Generator().manual_seed(B * 1_000_003 + n * 1009 + ctx)
    news = _ragged(g, B, n, max(1, n // 2))
    return torch.maximum(_ragged(g, B, ctx, max(1, ctx // 2)), news), news


def _prepare_attend(c, g, gg):
    B, hq, hkv, d = c["B"], c["hq"], c["hkv"], c["d"]
    dt = DTYPES[c["dtype"]]
    lens, news = _attend_shape(c)
    T = int(news.sum())
    qsl = torch.cat([torch.zeros(1, dtype=torch.long), news.cumsum(0)])
    pages = (lens + PAGE - 1) // PAGE
    most = int(pages.max())
    # blocks of a pool in random order; those behind the sinks and before the window have
    # been given back, and their entries are -1
    low = (lens - news - c["window"] + 1).clamp(min=0)
    col = torch.arange(most)[None, :]
    held = (col < pages[:, None]) & ((col >= (low // PAGE)[:, None]) | (col * PAGE < c["sinks"]))
    count = int(held.sum())
    nb = count + count // 16 + 1
    bt = torch.full((B, most), -1, dtype=torch.int32)
    bt[held] = torch.randperm(nb, generator=g)[:count].to(torch.int32)
    return {"case": c, "q": _normal(gg, dt, T, hq, d, std=3.0 if c["cap"] else 1.0),
            "k_pool": _normal(gg, dt, nb, PAGE, hkv, d),
            "v_pool": _normal(gg, dt, nb, PAGE, hkv, d), "bt": bt.cuda(),
            "lens": lens.to(torch.int32).cuda(), "qsl": qsl.to(torch.int32).cuda(),
            "scale": d ** -0.5, "out": torch.empty(T, hq, d, dtype=dt, device="cuda"),
            # what the program knows of its batch on the host
            "T": T, "most_new": int(news.max()), "most_len": int(lens.max()),
            "span": int((lens - low).max()), "low": low.cuda(), "ws": None}


# ------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"sample": _own_sample, "extend": _own_extend, "rotary": _own_rotary,
                "attend": _own_attend}[op](state)
    return {"sample": _plain_sample, "extend": _plain_extend, "rotary": _plain_rotary,
            "attend": _plain_attend}[op](state)


def _own_sample(s):
    return _binding().sample(s["x"], s["bits"], temperature=s["temp"], top_k=s["k"],
                             top_p=s["p"], min_p=s["m"])


def _own_extend(s):
    _binding().extend_sequences(s["bt"], s["lens"], s["news"], s["free"], s["count"], s["nb"],
                                s["qsl"], s["slots"], s["pos"], out_seq_lens=s["out_lens"],
                                out_free_count=s["out_count"])
    return {"bt": s["bt"], "lens": s["out_lens"], "count": s["out_count"], "qsl": s["qsl"],
            "slots": s["slots"], "pos": s["pos"]}


def _own_rotary(s):
    _binding().rotary_axes_reshape_and_cache(s["q"], s["k"], s["v"], s["pos"], s["slots"],
                                             s["k_pool"], s["v_pool"], s["freq"], s["axes"],
                                             interleaved=s["case"]["inter"], q_out=s["q_out"])
    return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}


def _own_attend(s):
    b, c = _binding(), s["case"]
    if s["ws"] is None:  # a program's workspace, kept from step to step
        s["ws"] = b.alloc_workspace(s["T"], c["B"], c["hq"], c["hkv"], c["d"], s["most_len"])
    return b.streaming_paged_attention(s["q"], s["k_pool"], s["v_pool"], s["bt"], s["lens"],
                                       s["qsl"], s["scale"], c["window"], c["sinks"],
                                       softcap=c["cap"], out=s["out"], workspace=s["ws"])


def _plain_sample(s):
    # borders between tokens lie close together: 64 bits
    x = s["x"].double()
    B, V = x.shape

    def col(t, least):
        return torch.full((B, 1), least, dtype=torch.float64, device=x.device) if t is None \
            else t.double()[:, None]

    temp, k = col(s["temp"], 1.0), col(s["k"], 0.0)
    k = torch.where(k <= 0, float(V), k)
    xs, at = torch.sort(x, dim=-1, descending=True, stable=True)
    rank = torch.arange(V, device=x.device)[None, :]
    greedy = temp == 0
    w = torch.exp((xs - xs[:, :1]) / torch.where(greedy, 1.0, temp))
    w = torch.where(rank < k, w, 0.0)
    before = w.cumsum(-1) - w
    keep = (before < col(s["p"], 1.0) * w.sum(-1, keepdim=True)) | (col(s["p"], 1.0) >= 1)
    keep = keep & (w >= col(s["m"], 0.0)) & (w > 0) & (~greedy | (rank < 1))
    w = torch.zeros_like(w).scatter_(1, at, torch.where(keep, w, 0.0))
    run_ = w.cumsum(-1)
    z = run_[:, -1:]
    word = (s["bits"].long() & 0xffffffff).double()[:, None]
    token = (run_ <= word * 2.0 ** -32 * z).sum(-1, keepdim=True)
    return token.view(-1).int(), torch.log(w.gather(1, token) / z).view(-1).float()


def _plain_extend(s):
    c, T = s["case"], s["T"]
    dev = s["bt"].device
    lens, news = s["lens"].long(), s["news"].long()
    had = (lens + PAGE - 1) // PAGE
    need = (lens + news + PAGE - 1) // PAGE - had
    ends, upto = need.cumsum(0), news.cumsum(0)
    ok = ((need == 0) | (ends <= s["count"])) & (upto <= T)
    news, need = torch.where(ok, news, 0), torch.where(ok, need, 0)
    first, ends = need.cumsum(0) - need, news.cumsum(0)
    # the blocks, in order of sequences and pages, from the top of the stack
    page = torch.arange(s["bt"].shape[1], device=dev)[None, :]
    nth = first[:, None] + page - had[:, None]
    new = (page >= had[:, None]) & (page < (had + need)[:, None])
    from_top = (s["count"].long() - 1 - nth).clamp(min=0)
    s["bt"].copy_(torch.where(new, s["free"][from_top.clamp(max=s["free"].shape[0] - 1)], s["bt"]))
    s["out_lens"].copy_(lens + news)
    s["out_count"].copy_(s["count"] - need.sum())
    s["qsl"].copy_(torch.cat([torch.zeros_like(ends[:1]), ends]))
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(ends, t, right=True).clamp(max=c["B"] - 1)
    pos = lens[seq] + t - (ends - news)[seq]
    used = t < ends[-1]
    pos = torch.where(used, pos, 0)
    slot = s["bt"][seq, pos // PAGE] * PAGE + pos % PAGE
    s["slots"].copy_(torch.where(used, slot, -1))
    s["pos"].copy_(pos)
    return {"bt": s["bt"], "lens": s["out_lens"], "count": s["out_count"], "qsl": s["qsl"],
            "slots": s["slots"], "pos": s["pos"]}


def _turn(x, cos, sin, R, inter, dt):
    """x [T, H, d] turned by cos, sin [T, 1, R/2] over its first R elements."""
    x = x.float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([y, x[..., R:]], -1).to(dt)


def _plain_rotary(s):
    c = s["case"]
    dt, R = s["q"].dtype, 2 * s["freq"].shape[0]
    # far positions: 64 bits
    ang = (s["pos"].double()[s["axes"].long()].T * s["freq"])[:, None, :]
    cos, sin = ang.cos().float(), ang.sin().float()
    s["q_out"].copy_(_turn(s["q"], cos, sin, R, c["inter"], dt))
    at = s["slots"].long()
    s["k_pool"].view(-1, c["hkv"], c["d"])[at] = _turn(s["k"], cos, sin, R, c["inter"], dt)
    s["v_pool"].view(-1, c["hkv"], c["d"])[at] = s["v"]
    return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}


def _plain_attend(s):
    c = s["case"]
    B, hq, hkv, d, n, S = c["B"], c["hq"], c["hkv"], c["d"], s["most_new"], c["sinks"]
    lens, qsl, dev = s["lens"].long(), s["qsl"].long(), s["q"].device
    news = qsl[1:] - qsl[:-1]
    # the first keys, then those from the first row's window on
    key = torch.cat([torch.arange(S, device=dev)[None, :].expand(B, S),
                     s["low"][:, None] + torch.arange(s["span"], device=dev)], 1)
    first = torch.arange(key.shape[1], device=dev)[None, :] < S
    page = (key // PAGE).clamp(max=s["bt"].shape[1] - 1)
    at = s["bt"].gather(1, page).long().clamp(min=0) * PAGE + key % PAGE
    k = s["k_pool"].view(-1, hkv, d)[at].float().permute(0, 2, 3, 1)       # [B, hkv, d, keys]
    v = s["v_pool"].view(-1, hkv, d)[at].float().permute(0, 2, 1, 3)       # [B, hkv, keys, d]
    i = torch.arange(n, device=dev)
    row = (qsl[:-1, None] + i).clamp(max=s["T"] - 1)                        # [B, n]
    q = s["q"][row].float().view(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    x = (q.reshape(B, hkv, -1, d) @ k).view(B, hq, n, -1) * s["scale"]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    pos = (lens - news)[:, None] + i                                        # [B, n]
    away = pos[:, :, None] - key[:, None, :]                                # [B, n, keys]
    see = (away >= 0) & torch.where(first[:, None, :], True, away < c["window"])
    see = see & (first | (key >= S))[:, None, :] & (key < lens[:, None])[:, None, :]
    x = x.masked_fill(~see[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    y = (x.view(B, hkv, n * (hq // hkv), -1) @ v).view(B, hq, n, d).transpose(1, 2)
    seq = torch.arange(B, device=dev).repeat_interleave(news, output_size=s["T"])
    s["out"].copy_(y[seq, torch.arange(s["T"], device=dev) - qsl[seq]])
    return s["out"]


# ------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------
def work(case):
    c = case
    size = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "sample":
        return {"bytes": c["B"] * c["V"] * size + 24 * c["B"], "flops": 3 * c["B"] * c["V"]}
    if c["op"] == "extend":
        lens, news = _extend_shape(c)
        blocks = int(((lens + news + PAGE - 1) // PAGE - (lens + PAGE - 1) // PAGE).sum())
        return {"bytes": 16 * c["B"] + 8 * int(news.sum()) + 8 * blocks, "flops": 0}
    if c["op"] == "rotary":
        T, hq, hkv, d = c["T"], c["hq"], c["hkv"], c["d"]
        axes = _sections(c)
        return {"bytes": 2 * T * (hq + 2 * hkv) * d * size + 4 * T * (max(axes) + 2)
                + 12 * len(axes), "flops": 6 * T * (hq + hkv) * len(axes)}
    lens, news = _attend_shape(c)
    first = lens - news                                       # position of the first row
    low = (first - c["window"] + 1).clamp(min=0)
    keys = int((lens - torch.maximum(low, torch.minimum(lens, torch.tensor(c["sinks"])))).sum()
               + lens.clamp(max=c["sinks"]).sum())
    seq = torch.repeat_interleave(torch.arange(c["B"]), news)
    pos = first[seq] + torch.arange(len(seq)) - (news.cumsum(0) - news)[seq]
    lo = (pos - c["window"] + 1).clamp(min=0)
    seen = pos + 1 - lo + torch.minimum(lo, torch.tensor(c["sinks"]))
    return {"bytes": 2 * 2 * keys * c["hkv"] * c["d"] + 2 * 2 * len(seq) * c["hq"] * c["d"]
            + 4 * ((keys + PAGE) // PAGE), "flops": 4 * c["d"] * c["hq"] * int(seen.sum())}


# ------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "extend": _exact_extend, "rotary": _exact_rotary,
            "attend": _exact_attend}[case["op"]](case, s)


def _exact_sample(c, s):
    tok, lp = [], []
    for b in range(c["B"]):
        x = s["x"][b].double()
        T = 1.0 if s["temp"] is None else float(s["temp"][b])
        if T == 0:
            tok.append((x == x.max()).nonzero()[:1, 0])
            lp.append(torch.zeros(1, dtype=torch.float64, device="cuda"))
            continue
        prob = torch.softmax(x / T, 0)
        order = torch.argsort(-x, stable=True)
        k = c["V"] if s["k"] is None else int(s["k"][b])
        order = order[:k if k > 0 else c["V"]]
        got = prob[order]
        share = torch.cumsum(got / got.sum(), 0)
        m = len(order)
        if s["p"] is not None and float(s["p"][b]) < 1:  # the fewest that reach the share
            m = min(m, int((share < float(s["p"][b])).sum()) + 1)
        if s["m"] is not None:
            m = min(m, int((got >= float(s["m"][b]) * got[0]).sum()))
        kept = order[:m].sort().values  # in the vocabulary's order
        kept = kept[prob[kept] > 0]
        edge = torch.cumsum(prob[kept], 0)
        u = (int(s["bits"][b]) & 0xffffffff) / 2.0 ** 32
        i = int(torch.searchsorted(edge, u * edge[-1], right=True))
        tok.append(kept[i:i + 1])
        lp.append(torch.log(prob[kept[i:i + 1]] / prob[kept].sum()))
    return torch.cat(tok).int(), torch.cat(lp)


def _exact_extend(c, s):
    bt, lens, news = s["bt"].tolist(), s["lens"].tolist(), s["news"].tolist()
    free, left = s["free"].tolist(), int(s["count"][0])
    qsl, slots, pos, full = [0], [], [], False
    for b in range(c["B"]):
        L, n = lens[b], news[b]
        pages = range(-(-L // PAGE), -(-(L + n) // PAGE))
        if len(pages) > left or qsl[-1] + n > s["T"]:
            n, pages = 0, ()
        for page in pages:
            left -= 1
            bt[b][page] = free[left]
        for p in range(L, L + n):
            pos.append(p)
            slots.append(bt[b][p // PAGE] * PAGE + p % PAGE)
        lens[b] = L + n
        qsl.append(len(pos))
    pad = s["T"] - len(pos)

    def t(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    return {"bt": t(bt), "lens": t(lens), "count": t([left]), "qsl": t(qsl),
            "slots": t(slots + [-1] * pad), "pos": t(pos + [0] * pad)}


def _exact_rotary(c, s):
    axes, R = _sections(c), 2 * s["freq"].shape[0]
    ang = torch.stack([s["pos"][a].double() * s["freq"][i] for i, a in enumerate(axes)], 1)
    z = torch.polar(torch.ones_like(ang), ang)[:, None, :]

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
    group = c["hq"] // c["hkv"]
    for b in range(c["B"]):
        L, lo, hi = lens[b], qsl[b], qsl[b + 1]
        p = torch.arange(L - (hi - lo), L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        j = j[(j < c["sinks"]) | (j > L - (hi - lo) - c["window"])]
        see = (j <= p) & ((j < c["sinks"]) | (j > p - c["window"]))
        blocks = s["bt"][b, j // PAGE].long()
        kk = s["k_pool"][blocks, j % PAGE].double()
        vv = s["v_pool"][blocks, j % PAGE].double()
        for h in range(c["hq"]):
            x = s["q"][lo:hi, h].double() @ kk[:, h // group].T * s["scale"]
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            out[lo:hi, h] = torch.softmax(torch.where(see, x, -math.inf), -1) @ vv[:, h // group]
    return out
