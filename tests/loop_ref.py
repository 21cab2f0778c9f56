"""Plain implementations of sampling, sequence extension and attention with sinks, for the tests:
64 bits, loops over rows, no code shared with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE = 16


# ------------------------------------------------------------------------------------
# sampling
# ------------------------------------------------------------------------------------
def draw(x, T, k, p, m, word, shift=0.0, p_shift=0.0):
    """(token, log probability) of one row x (float64 numpy), None for a filter that is not
    given; -1, -inf where there is no token. shift moves the random point and p_shift the share
    of top-p, relative to the sums."""
    x = np.where(np.isnan(x), -np.inf, x)
    V = len(x)
    top = x.max()
    if not np.isfinite(top):
        return -1, -math.inf
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if T is not None and not T >= 2.0 ** -100:
        return int(order[0]), 0.0
    T = 1.0 if T is None else T
    with np.errstate(over="ignore"):
        w = np.exp((x - top) / T) if not math.isinf(T) else (x > -np.inf).astype(np.float64)
    if k is not None and 0 < k < V:
        order = order[:k]
    n = len(order)
    if p is not None and p < 1.0:
        share = np.cumsum(w[order]) - w[order]  # before each
        n = max(1, int((share < (p + p_shift) * w[order].sum()).sum()))
    if m is not None and m > 0:
        edge = top + T * math.log(m) if m < 1 else top
        n = min(n, int((x[order] >= edge).sum()))
    kept = np.sort(order[:n])
    run = np.cumsum(w[kept])
    u = word / 2.0 ** 32 + shift
    i = min(int(np.searchsorted(run, u * run[-1], side="right")), len(kept) - 1)
    while w[kept[i]] == 0.0:
        i -= 1
    return int(kept[i]), math.log(w[kept[i]] / run[-1])


def check_draws(x, tokens, logprobs, bits, T=None, k=None, p=None, m=None):
    """Every row's token and log probability. Weights are off by 2^-29 of themselves and rounded to
    multiples of 2^-42 of the largest, so V of them add up to within 2^-29 + V 2^-43 of the sum
    (which is no less than the largest), and a border between tokens, a ratio of two such sums, lies
    within twice that of where it is in 64 bits: there either neighbour is right, elsewhere one.
    The log probability is a double rounded once (2^-24 of it), off by the sum's error and by its
    own weight's: 2^-29, and 2^-43 of the largest, which is 2^-43 / w of it."""
    x64 = x.double().cpu().numpy()
    tokens, logprobs = tokens.tolist(), logprobs.double().tolist()
    bits = [b & 0xffffffff for b in bits.tolist()]

    def at(t, b):
        return None if t is None else t[b].item()

    V = x.shape[1]
    eps = 2.0 ** -28 + V * 2.0 ** -42
    for b in range(x.shape[0]):
        args = (at(T, b), at(k, b), at(p, b), at(m, b), bits[b])
        want = draw(x64[b], *args)
        if tokens[b] != want[0]:
            near = [draw(x64[b], *args, shift=s, p_shift=q) for s in (-eps, 0, eps)
                    for q in (-eps, 0, eps)]
            want = next((w for w in near if w[0] == tokens[b]), want)
        assert tokens[b] == want[0], (b, args, tokens[b], want)
        if want[1] == -math.inf:
            assert logprobs[b] == -math.inf
        else:
            # (the weight is at least its share of the sum, of the largest)
            tol = 2.0 ** -24 * abs(want[1]) + eps + 2.0 ** -43 * math.exp(-want[1])
            assert abs(logprobs[b] - want[1]) <= tol, (b, args, logprobs[b], want)


# ------------------------------------------------------------------------------------
# sequence extension
# ------------------------------------------------------------------------------------
def extend(bt, lens, news, free, count, T, num_blocks, window=0, sinks=0):
    """Lists in; returns (tables, lengths, stack, count, offsets, slots, positions, errors):
    errors the set of codes that may be recorded."""
    bt, lens = [list(r) for r in bt], list(lens)
    free, errors, capacity = list(free), set(), len(free)
    width = len(bt[0]) if bt else 0
    if count < 0 or count > capacity:
        errors.add(1)
        count = 0
    bad = []
    for b, (L, n) in enumerate(zip(lens, news)):
        bad.append(L < 0 or L > width * PAGE or (n >= 0 and L + n > width * PAGE))
        if bad[b]:
            errors.add(3)
    for b, (L, n) in enumerate(zip(lens, news)):
        if bad[b]:
            continue
        pages = []
        if n < 0:
            pages = [q for q in reversed(range(-(-L // PAGE))) if 0 <= bt[b][q] < num_blocks]
        elif window > 0:
            for q in reversed(range(-(-sinks // PAGE), max(0, L - window + 1) // PAGE)):
                if not 0 <= bt[b][q] < num_blocks:
                    break
                pages.append(q)
        for q in pages:
            if count < capacity:
                free[count] = bt[b][q]
                count += 1
            else:
                errors.add(1)
            bt[b][q] = -1
    offsets, slots, positions = [0], [], []
    asked, taken, wanted = 0, 0, 0
    for b, (L, n) in enumerate(zip(lens, news)):
        if bad[b] or n < 0:
            if n < 0 and not bad[b]:
                lens[b] = 0
            offsets.append(len(slots))
            continue
        need = -(-(L + n) // PAGE) + (-L // PAGE)
        asked += n
        wanted += need
        if asked > T:
            errors.add(3)
            n = 0
        elif need and wanted > count:
            errors.add(7)
            n = 0
        else:
            for q in range(-(-L // PAGE), -(-(L + n) // PAGE)):
                bt[b][q] = free[count - 1 - taken]
                if not 0 <= bt[b][q] < num_blocks:
                    errors.add(1)
                    bt[b][q] = -1
                taken += 1
        for at in range(L, L + n):
            block = bt[b][at // PAGE]
            if not 0 <= block < num_blocks:
                errors.add(1)
                slots.append(-1)
            else:
                slots.append(block * PAGE + at % PAGE)
            positions.append(at)
        lens[b] = L + n
        offsets.append(len(slots))
    pad = T - len(slots)
    return (bt, lens, free, count - taken, offsets, slots + [-1] * pad, positions + [0] * pad,
            errors)


# ------------------------------------------------------------------------------------
# attention with a window and sinks
# ------------------------------------------------------------------------------------
def attend_stream(q, K, V, pos, scale, window, sinks, softcap=0.0):
    """q [n, H_q, D] at positions pos over K, V [L, H_kv, D]: what operator_ref.attend_dense
    returns, for keys j <= p with j > p - window (window 0: all) or j < sinks."""
    n, H_q, D = q.shape
    L, H_kv, _ = K.shape
    j = torch.arange(L, device=q.device)
    p = pos.long()[:, None]
    see = j <= p
    if window > 0:
        see &= (j > p - window) | (j < sinks)
    out = torch.zeros(n, H_q, D, dtype=torch.float64, device=q.device)
    absv, tail = torch.zeros_like(out), torch.zeros_like(out)
    size = torch.zeros(n, H_q, dtype=torch.float64, device=q.device)
    used = see.any(0)
    K = torch.where(used[:, None, None], K.double(), 0.0)
    V = torch.where(used[:, None, None], V.double(), 0.0)
    for h in range(H_q):
        g = h // (H_q // H_kv)
        x = q[:, h].double() @ K[:, g].T * scale
        m = q[:, h].double().abs() @ K[:, g].abs().T * scale
        if softcap > 0:
            x, m = softcap * torch.tanh(x / softcap), m + softcap
        w = torch.softmax(torch.where(see, x, -math.inf), -1)
        out[:, h], absv[:, h] = w @ V[:, g], w @ V[:, g].abs()
        e = (w.clamp(max=2.0 ** -24) - 2.0 ** -11 * w).clamp(min=0.0)
        tail[:, h] = e @ V[:, g].abs() + e.sum(-1, keepdim=True) * out[:, h].abs()
        size[:, h] = torch.where(w > 1e-12, m, 0.0).max(-1).values * math.log2(math.e)
    return out, absv, size, tail
