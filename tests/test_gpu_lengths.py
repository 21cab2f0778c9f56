"""Context lengths at the end of 32 bits in the causal attention: recorded, the sequence left out
and the others served, in every mode."""
import pytest
import torch

from paged_kv_attention_18_gb300 import binding
from tests.test_gpu_masked import CHUNKS, LONG, SMALL_CHUNKS, Batch

pytestmark = pytest.mark.gpu

BATCHES = {"direct": [(300, 1), (17, 1)], "tiles": SMALL_CHUNKS, "chunks": CHUNKS, "long": LONG,
           "many": [(100 + i, 1) for i in range(400)]}


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 15, 2 ** 31 - 16, 2 ** 31 - 1024])
@pytest.mark.parametrize("at", [0, -1])
def test_lengths_at_the_end_of_32_bits(name, length, at):
    seqs = list(BATCHES[name])
    seqs.insert(0 if at == 0 else len(seqs), (30, 2))
    bad = 0 if at == 0 else len(seqs) - 1
    b = Batch(seqs, 12, 2, 128, torch.bfloat16, 31, holes=False)
    b.sl[bad] = length
    rows = slice(b.off[bad], b.off[bad + 1])
    out = torch.full_like(b.q, 7.0)
    binding.paged_attention(b.q, b.k, b.v, b.bt, b.sl, b.qs, b.scale, out=out)
    torch.cuda.synchronize()
    assert binding.device_error() == 3
    assert (out[rows] == 7.0).all()
    b.seqs[bad] = (30, 0)
    b.check(out)

    # the step: the sequence's new rows get no slot, the others are written where they go
    T = b.q.shape[0]
    k, v = (torch.randn(T, 2, 128, device="cuda").bfloat16() for _ in range(2))
    slots = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    out = torch.full_like(b.q, 7.0)
    kp, vp = b.k.clone(), b.v.clone()
    binding.attention_step(b.q, k, v, b.k, b.v, b.bt, b.sl, b.qs, b.scale, out=out,
                           slot_buf=slots)
    torch.cuda.synchronize()
    assert binding.device_error() == 3
    assert (slots[rows] == -1).all() and (out[rows] == 7.0).all()
    keep = slots >= 0
    for pool, old, new in ((b.k, kp, k), (b.v, vp, v)):
        old.view(-1, 2, 128)[slots[keep].long()] = new[keep]
        assert torch.equal(pool, old)
    b.check(out)
