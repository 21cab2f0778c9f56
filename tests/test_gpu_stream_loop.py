"""The operators of a decode loop together, as a server of endless streams calls them: a token
drawn, blocks and slots of the step, rotary positions with three axes into the cache, attention
over a window and the first keys, a toy head; eagerly, and as one captured graph."""
import pytest
import torch

from paged_kv_attention_18_gb300 import binding, rotary
from tests import loop_ref as S
from tests import operator_ref as R

pytestmark = pytest.mark.gpu


class Loop:
    """One layer: emb [V, q | k | v], a head of V logits; B streams of at most `width` pages held
    in a pool of far fewer blocks than their contexts fill."""

    def __init__(self, dt, hq, hkv, d, window, sinks, B=5, V=307, T=None):
        g = torch.Generator("cuda").manual_seed(6)
        self.dt, self.hq, self.hkv, self.d, self.B, self.V = dt, hq, hkv, d, B, V
        self.window, self.sinks, self.T = window, sinks, T or B
        self.emb = torch.randn(V, (hq + 2 * hkv) * d, generator=g, device="cuda").to(dt)
        self.head = torch.randn(hq * d, V, generator=g, device="cuda") * 0.1
        self.nb = B * ((window + sinks) // 16 + 6)
        self.k, self.v = (torch.full((self.nb, 16, hkv, d), float("nan"), dtype=dt, device="cuda")
                          for _ in range(2))
        i = dict(dtype=torch.int32, device="cuda")
        self.bt = torch.full((B, 24), -1, **i)
        self.lens, self.count = torch.zeros(B, **i), torch.tensor([self.nb], **i)
        self.free = torch.randperm(self.nb, generator=g, device="cuda").int()
        self.freq = rotary.frequencies(d, 1e4, device="cuda")
        self.axes = rotary.axes([d // 8, 3 * d // 16, 3 * d // 16], device="cuda")
        self.qsl = torch.zeros(B + 1, **i)
        self.bits = torch.zeros(B, **i)
        self.temp = torch.full((B,), 0.8, device="cuda")
        self.top_k, self.top_p = torch.full((B,), 40, **i), torch.full((B,), 0.9, device="cuda")

    def buffers(self, T):
        return (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))

    def layer(self, tokens, news, slots, pos, ws=None):
        """Attention of the packed tokens; returns (rotated q, output)."""
        T, hq, hkv, d = tokens.shape[0], self.hq, self.hkv, self.d
        binding.extend_sequences(self.bt, self.lens, news, self.free, self.count, self.nb, self.qsl,
                                 slots, pos, self.window, self.sinks)
        qkv = self.emb[tokens.long()].view(T, hq + 2 * hkv, d)
        q = torch.empty(T, hq, d, dtype=self.dt, device="cuda")
        at = torch.stack([pos, pos // 5, pos % 5])  # a picture of rows of five, say
        binding.rotary_axes_reshape_and_cache(qkv[:, :hq], qkv[:, hq:hq + hkv],
                                              qkv[:, hq + hkv:], at, slots, self.k, self.v,
                                              self.freq, self.axes, q_out=q)
        return q, binding.streaming_paged_attention(q, self.k, self.v, self.bt, self.lens, self.qsl,
                                                    d ** -0.5, self.window, self.sinks,
                                                    workspace=ws)

    def draw(self, out):
        logits = out.float().view(self.B, -1) @ self.head
        return logits, binding.sample(logits, self.bits, temperature=self.temp, top_k=self.top_k,
                                      top_p=self.top_p)


def words(B, step):
    g = torch.Generator().manual_seed(step)
    return torch.randint(-(1 << 31), 1 << 31, (B,), generator=g, dtype=torch.int64).int().cuda()


@pytest.mark.parametrize("dt,hq,hkv,d", [(torch.bfloat16, 12, 2, 128), (torch.float16, 8, 8, 64)])
def test_streams_past_their_cache(dt, hq, hkv, d):
    loop = Loop(dt, hq, hkv, d, window=45, sinks=5)
    B = loop.B
    prompts = [30, 1, 64, 17, 50]
    kept = [(torch.zeros(0, hkv, d, dtype=dt, device="cuda"),) * 2 for _ in range(B)]
    tokens = torch.randint(0, loop.V, (sum(prompts),), device="cuda").int()
    news = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    for step in range(110):
        slots, pos = loop.buffers(tokens.shape[0])
        q, out = loop.layer(tokens, news, slots, pos)
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        off = loop.qsl.tolist()
        assert off[-1] == tokens.shape[0] and (slots >= 0).all()
        for b in range(B):
            a, e = off[b], off[b + 1]
            rows = slots[a:e].long()
            kept[b] = tuple(torch.cat([old, pool.view(-1, hkv, d)[rows]])
                            for old, pool in zip(kept[b], (loop.k, loop.v)))
            assert pos[a:e].tolist() == list(range(len(kept[b][0]) - (e - a), len(kept[b][0])))
            if step % 10 == 0 or step < 3:
                ref, absv, size, tail = S.attend_stream(q[a:e], *kept[b], pos[a:e], d ** -0.5, 45,
                                                        5)
                tol = R.attention_tolerance(ref, absv, size, tail, d, dt)
                assert ((out[a:e].double() - ref).abs() <= tol).all(), (step, b)
        loop.bits.copy_(words(B, step))
        logits, (tokens, lp) = loop.draw(out[(loop.qsl[1:] - 1).long()])
        S.check_draws(logits, tokens, lp, loop.bits, loop.temp, loop.top_k, loop.top_p)
        news = torch.ones(B, dtype=torch.int32, device="cuda")
    # every block is in one table or free
    held = loop.bt[loop.bt >= 0].tolist()
    stack = loop.free[:int(loop.count)].tolist()
    assert sorted(held + stack) == list(range(loop.nb))
    assert all(int(n) <= 45 // 16 + 4 for n in (loop.bt >= 0).sum(1))


def test_the_loop_as_one_graph():
    """Two loops of the same seeds, one eager and one captured: the same tokens and caches."""
    runs = []
    for captured in (False, True):
        loop = Loop(torch.bfloat16, 12, 2, 128, window=40, sinks=4)
        B = loop.B
        tokens = torch.arange(B, dtype=torch.int32, device="cuda")
        news = torch.ones(B, dtype=torch.int32, device="cuda")
        slots, pos = loop.buffers(B)
        ws = binding.alloc_workspace(B, B, 12, 2, 128, 24 * 16)

        def step():
            _, out = loop.layer(tokens, news, slots, pos, ws)
            _, (tok, lp) = loop.draw(out)
            tokens.copy_(tok)
            return lp

        graph = None
        history = []
        for i in range(60):
            loop.bits.copy_(words(B, i))
            if not captured or i == 0:
                lp = step()
            else:
                if graph is None:
                    torch.cuda.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        lp = step()
                graph.replay()
            history.append((tokens.clone(), lp.clone(), slots.clone()))
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        runs.append((history, loop))
    for a, b in zip(runs[0][0], runs[1][0]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(runs[0][1].bt, runs[1][1].bt)
    assert torch.equal(runs[0][1].lens, runs[1][1].lens)
