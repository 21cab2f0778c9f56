"""Plain 64-bit implementations of the rotary, masked attention, beam selection and fork
operators, for the tests: loops over rows, no code shared with the library."""
from __future__ import annotations

import math

import torch

PAGE = 16


def rotary(x, pos, freq, interleaved, magnitude):
    """x [T, H, D] in 64 bits; returns (turned x, |x| + |y| of each element's pair)."""
    y = x.double().clone()
    mag = torch.zeros_like(y)
    R = 2 * freq.numel()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        ang = pos.double() * freq[i]
        c, s = magnitude * torch.cos(ang)[:, None], magnitude * torch.sin(ang)[:, None]
        u, v = x[:, :, a].double(), x[:, :, b].double()
        y[:, :, a], y[:, :, b] = u * c - v * s, v * c + u * s
        mag[:, :, a] = mag[:, :, b] = abs(magnitude) * (u.abs() + v.abs())
    return y, mag


def gather(pool, table, L):
    """Rows of a sequence's first L positions [L, H_kv, D] (entries below 0 read zeros)."""
    j = torch.arange(L, device=pool.device)
    blk = table.long()[j // PAGE]
    rows = pool[blk.clamp(min=0), j % PAGE].double()
    return torch.where((blk >= 0)[:, None, None], rows, 0.0)


def attend_dense(q, K, V, pos, scale, softcap=0.0, slopes=None, window=0, prefix=0, starts=None):
    """q [n, H_q, D] at positions pos over K, V [L, H_kv, D]. Returns (out, tol_terms): the
    output in 64 bits, sum_j w_j |V_j|, the largest magnitude met in a row's scores (sum |q k|
    scale, in log2 units, with the bias), and sum_j e_j (|V_j| + |out|), e_j what the rounding
    of a weight too small for a normal fp16 can add (attention_tolerance), all [n, H_q, (D)]."""
    n, H_q, D = q.shape
    L, H_kv, _ = K.shape
    j = torch.arange(L, device=q.device)
    p = pos.long()[:, None]
    see = (j <= p) | (j < prefix)
    if window > 0:
        see &= j > p - window
    if starts is not None:
        see &= j >= starts.long()[:, None]
    out = torch.zeros(n, H_q, D, dtype=torch.float64, device=q.device)
    absv, tail = torch.zeros_like(out), torch.zeros_like(out)
    size = torch.zeros(n, H_q, dtype=torch.float64, device=q.device)
    used = see.any(0)
    Kz = torch.where(used[:, None, None], K.double(), 0.0)
    Vz = torch.where(used[:, None, None], V.double(), 0.0)
    for h in range(H_q):
        g = h // (H_q // H_kv)
        x = q[:, h].double() @ Kz[:, g].T * scale
        m = q[:, h].double().abs() @ Kz[:, g].abs().T * scale
        if softcap > 0:
            x = softcap * torch.tanh(x / softcap)
            m = m + softcap
        if slopes is not None:
            b = slopes[h].double() * (p - j).abs()
            x, m = x - b, m + b
        x = torch.where(see, x, -math.inf)
        top = x.max(-1, keepdim=True).values
        w = torch.where(see, torch.exp(x - torch.where(top.isinf(), 0.0, top)), 0.0)
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
        out[:, h], absv[:, h] = w @ Vz[:, g], w @ Vz[:, g].abs()
        e = (w.clamp(max=2.0 ** -24) - 2.0 ** -11 * w).clamp(min=0.0)
        tail[:, h] = e @ Vz[:, g].abs() + e.sum(-1, keepdim=True) * out[:, h].abs()
        # (keys far below the row's maximum carry no weight, so neither do their errors)
        size[:, h] = torch.where(w > 1e-12, m, 0.0).max(-1).values * math.log2(math.e)
    return out, absv, size, tail


def attention_tolerance(out, absv, size, tail, D, dtype):
    """Largest error of an element of the output. u is half a step of the 16-bit type.
      - every weight is rounded to it, in the products and in the sum alike: weights are off
        by at most 2 u relative, the normalised sum by u (sum w |V| + |out|);
      - fp16 weights below the type's least normal, 2^-14, are off by half its least step,
        2^-25, whatever they are. They are taken relative to a sum of at least 1/2 (the
        reference is at most the sum so far, rounded to a power of two), so a weight is off by
        2^-24, or by all of itself if that is less: e = min(w, 2^-24) - u w more than the
        line above counts (bf16 has fp32's exponents: none);
      - the fp32 score is a sum of D products (each add off by at most 2^-23, the tensor
        core truncating) and a few roundings of values of its size: (D + 16) 2^-23 size in
        log2 units; a weight is off by ln 2 of that, and by 2^-22 from ex2; in numerator and
        denominator again;
      - fp32 sums of the products over the keys and over the splits, normalised: 2^-16 of
        sum w |V|;
      - the output is rounded once."""
    u = torch.finfo(dtype).eps / 2
    rel = u + math.log(2) * (D + 16) * 2.0 ** -23 * size[..., None] + 2.0 ** -22
    tiny = torch.finfo(dtype).smallest_normal * u * 4
    tail = tail if dtype == torch.float16 else 0.0
    return rel * (absv + out.abs()) + 2.0 ** -16 * absv + u * out.abs() + tail + tiny


def beam(logits, scores, n, finished=None, pad=0):
    """Lists of (score, flat index) of each prompt, best first, in 64 bits."""
    B, W, V = logits.shape
    res = []
    for b in range(B):
        cand = []
        for w in range(W):
            cum = float(scores[b, w])
            if not math.isfinite(cum):
                continue
            if finished is not None and int(finished[b, w]):
                cand.append((cum, w * V + pad))
                continue
            x = logits[b, w].double()
            x = torch.where(x.isnan(), -math.inf, x)
            top = float(x.max())
            if not math.isfinite(top):
                continue
            lse = top + math.log(float(torch.exp(x - top).sum()))
            k = min(V, n + 1)
            # (a stable sort: ties to the lowest token)
            order = torch.sort(-x, stable=True).indices[:k].tolist()
            for t in order:
                if float(x[t]) > -math.inf:
                    cand.append((cum + (float(x[t]) - lse), w * V + t))
        cand.sort(key=lambda c: (-c[0], c[1]))
        res.append(cand)
    return res
