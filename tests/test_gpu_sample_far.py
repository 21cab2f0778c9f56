"""Sampling at temperatures of 2^100 and more, up to the largest float: weights as exact as at
others, so that draws are decided by the same bound."""
import math
import random

import numpy as np
import pytest
import torch

from paged_kv_attention_18_gb300 import binding
from tests import loop_ref as R

pytestmark = pytest.mark.gpu

MOST = float(np.finfo(np.float32).max)
FIXED = [2.0 ** 100, 2.0 ** 101, 1e36, 1e37, 1e38, 2.1e38, 3e38, MOST]


def rows(dt, count, seed, V=3000):
    """A row for each temperature: the first token above n others by d temperatures, n about e^d, so
    that the border behind it lies in the middle, where an error of the others' weights counts
    most; the rest is no token. Logits as far apart as the type holds, where that is less."""
    r = random.Random(seed)
    T = FIXED + [2.0 ** r.uniform(100, 127.99) for _ in range(count - len(FIXED))]
    T = torch.tensor(T, dtype=torch.float32)
    x = torch.full((count, V), -math.inf, dtype=torch.float64)
    for b in range(count):
        half = min(float(T[b]) * r.uniform(0.5, 3.9), float(torch.finfo(dt).max))
        x[b, 0] = half
        n = min(int(math.exp(2 * half / float(T[b]))) + 1, V - 1)
        x[b, 1:n + 1] = -half
    x = x.to(dt)
    # random points on either side of the border, twice the bound of a decision away from it
    eps = 2.0 ** -28 + V * 2.0 ** -42
    w = np.exp((x.double() - x[:, :1].double()).numpy() / T.double().numpy()[:, None])
    border = w[:, 0] / w.sum(1)
    bits = [[int((c + side * 2 * eps) * 2.0 ** 32) for c in border] for side in (-1, 1)]
    words = torch.tensor(bits, dtype=torch.int64)
    words = (words + 2 ** 31) % 2 ** 32 - 2 ** 31
    return x.cuda(), T.cuda(), words.to(torch.int32).cuda()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_borders_at_far_temperatures(dt):
    x, T, words = rows(dt, 200, 1)
    for side in (0, 1):
        tok, lp = binding.sample(x, words[side], temperature=T)
        torch.cuda.synchronize()
        assert ((tok == 0) == (side == 0)).all(), (T[(tok == 0) != (side == 0)], side)
        R.check_draws(x, tok, lp, words[side], T)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_filters_at_far_temperatures(dt):
    g = torch.Generator("cuda").manual_seed(2)
    B, V = 48, 2500
    T = torch.tensor(FIXED, dtype=torch.float32, device="cuda").repeat(6)
    x = torch.randn(B, V, generator=g, device="cuda", dtype=torch.float64) * 2.0
    most = torch.finfo(dt).max
    x = (x * T.double()[:, None]).clamp(-most, most).to(dt)
    x[::5, ::7] = -math.inf
    words = torch.randint(-(1 << 31), 1 << 31, (B,), dtype=torch.int64,
                          generator=torch.Generator().manual_seed(3)).int().cuda()

    def run(**kw):
        tok, lp = binding.sample(x, words, temperature=T, **kw)
        torch.cuda.synchronize()
        R.check_draws(x, tok, lp, words, T, kw.get("top_k"), kw.get("top_p"), kw.get("min_p"))

    k = torch.tensor([3, 100, 1000, 0, 2400, 1], dtype=torch.int32, device="cuda").repeat(8)
    p = torch.tensor([0.3, 0.9, 1.0, 0.99], device="cuda").repeat(12)
    m = torch.tensor([0.0, 0.2, 0.01], device="cuda").repeat(16)
    run()
    run(top_k=k)
    run(top_p=p)
    run(min_p=m)
    run(top_k=k, top_p=p, min_p=m)
