"""The decode loop's operators over streams that come and go: a sequence ends and gives its blocks
back, another begins in its place with a prompt, while the others keep growing under a window."""
import random

import pytest
import torch

from paged_kv_attention_18_gb300 import binding
from tests import loop_ref as S
from tests import operator_ref as R
from tests.test_gpu_stream_loop import Loop, words

pytestmark = pytest.mark.gpu

WINDOW, SINKS = 45, 5


@pytest.mark.parametrize("dt,hq,hkv,d", [(torch.bfloat16, 12, 2, 128), (torch.float16, 8, 8, 64)])
def test_streams_that_end_and_begin(dt, hq, hkv, d):
    loop = Loop(dt, hq, hkv, d, window=WINDOW, sinks=SINKS)
    B, r = loop.B, random.Random(hq)
    nothing = (torch.zeros(0, hkv, d, dtype=dt, device="cuda"),) * 2
    kept, drawn, ended, begun = [nothing] * B, [0] * B, 0, 0
    for step in range(80):
        news, tokens = [], []
        for b in range(B):
            if len(kept[b][0]) == 0:  # an empty place: a prompt, or nothing yet
                n = r.choice([0, 1, r.randint(2, 60)])
                tokens += [r.randrange(loop.V) for _ in range(n)]
                begun += n > 0
            elif r.random() < 0.04 or len(kept[b][0]) >= 24 * 16 - 1:
                n, ended = -1, ended + 1
            else:
                n = 1
                tokens.append(drawn[b])
            news.append(n)
        T = len(tokens) + 3  # some rows behind the last sequence
        tok = torch.tensor(tokens + [0] * 3, dtype=torch.int32, device="cuda")
        slots, pos = loop.buffers(T)
        q, out = loop.layer(tok, torch.tensor(news, dtype=torch.int32, device="cuda"), slots, pos)
        loop.bits.copy_(words(B, step))
        logits, (draws, lp) = loop.draw(out[(loop.qsl[1:] - 1).clamp(min=0).long()])
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        off = loop.qsl.tolist()
        assert off[-1] == len(tokens) and slots.tolist()[off[-1]:] == [-1] * 3
        for b in range(B):
            a, e = off[b], off[b + 1]
            assert e - a == max(news[b], 0)
            if news[b] < 0:
                kept[b] = nothing
                assert int(loop.lens[b]) == 0 and (loop.bt[b] < 0).all()
            if e == a:
                continue
            rows = slots[a:e].long()
            kept[b] = tuple(torch.cat([old, pool.view(-1, hkv, d)[rows]])
                            for old, pool in zip(kept[b], (loop.k, loop.v)))
            assert pos[a:e].tolist() == list(range(len(kept[b][0]) - (e - a), len(kept[b][0])))
            ref, absv, size, tail = S.attend_stream(q[a:e], *kept[b], pos[a:e], d ** -0.5, WINDOW,
                                                    SINKS)
            tol = R.attention_tolerance(ref, absv, size, tail, d, dt)
            assert ((out[a:e].double() - ref).abs() <= tol).all(), (step, b)
        live = torch.tensor([b for b in range(B) if news[b] > 0], device="cuda")
        if len(live):
            S.check_draws(logits[live], draws[live], lp[live], loop.bits[live], loop.temp[live],
                          loop.top_k[live], loop.top_p[live])
        drawn = draws.tolist()
        held = loop.bt[loop.bt >= 0].tolist()
        assert sorted(held + loop.free[:int(loop.count)].tolist()) == list(range(loop.nb)), step
    assert ended >= 5 and begun >= 5
    # all end
    slots, pos = loop.buffers(1)
    binding.extend_sequences(loop.bt, loop.lens, torch.full_like(loop.lens, -1), loop.free,
                             loop.count, loop.nb, loop.qsl, slots, pos, WINDOW, SINKS)
    torch.cuda.synchronize()
    assert binding.device_error() == 0 and loop.lens.tolist() == [0] * B
    assert sorted(loop.free.tolist()) == list(range(loop.nb)) and int(loop.count) == loop.nb
