"""Rotary positions by a table of frequencies (ps_rotary_reshape_and_cache) against 64 bits."""
import math

import pytest
import torch

from paged_kv_attention_18_gb300 import binding, rotary
from tests import operator_ref as R

pytestmark = pytest.mark.gpu


def make(T, hq, hkv, d, dt, seed, slot_holes=False):
    g = torch.Generator("cuda").manual_seed(seed)
    qkv = torch.randn(T, hq + 2 * hkv, d, generator=g, device="cuda").to(dt)
    nb = T // 16 + 3
    slots = torch.randperm(nb * 16, generator=g, device="cuda")[:T].int()
    if slot_holes:
        slots[::3] = -1
    pool = torch.randn(2, nb, 16, hkv, d, generator=g, device="cuda").to(dt)
    return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], slots, pool[0], pool[1]


def check(q, k, v, pos, slots, kp, vp, freq, inter, mag, out_q, kp0, vp0):
    """One rounding (half a step) plus 2^-20 of the pair's magnitudes: the fp32 angle is off
    by 3 pi 2^-24 at most (conversion, constant, product), sincosf by 2^-23, magnitude,
    product and sum by 2^-24 each, 2^-20.1 together; and the table's 2^-53 over |pos|."""
    dt = q.dtype
    u = torch.finfo(dt).eps / 2
    far = (pos.double().abs() * float(freq.abs().max()) * 2.0 ** -51)[:, None, None]

    def near(got, ref, off):
        tol = u * ref.abs() + off + torch.finfo(dt).smallest_normal * u * 2
        bad = (got.double() - ref).abs() > tol
        assert not bad.any(), (int(bad.sum()), float(((got.double() - ref).abs() - tol).max()))

    rq, pair = R.rotary(q, pos, freq, inter, mag)
    near(out_q, rq, (2.0 ** -20 + far) * pair)
    rk, pair = R.rotary(k, pos, freq, inter, mag)
    off = (2.0 ** -20 + far) * pair
    want_v = vp0.clone().view(-1, *vp0.shape[2:])
    flat, touched = kp.view(-1, *kp.shape[2:]), torch.zeros(kp.shape[0] * 16, dtype=torch.bool)
    for t, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        touched[s] = True
        want_v[s] = v[t]
    at = slots[slots >= 0].long()
    near(flat[at], rk[slots >= 0], off[slots >= 0])
    rest = ~touched.to(flat.device)
    assert torch.equal(flat[rest].view(torch.int16), kp0.view(-1, *kp0.shape[2:])[rest].view(torch.int16))
    assert torch.equal(vp.view(torch.int16).view(-1), want_v.view(torch.int16).view(-1))


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,rot", [
    (1, 14, 2, 64, 64), (1, 1, 1, 64, 16), (7, 12, 2, 128, 128), (13, 7, 1, 128, 96),
    (129, 32, 8, 128, 64), (300, 16, 16, 64, 32), (5000, 12, 2, 64, 48)])
def test_layouts_and_parts(T, hq, hkv, d, rot, inter, dt):
    q, k, v, slots, kp, vp = make(T, hq, hkv, d, dt, T + rot)
    pos = torch.randint(0, 1 << 17, (T,), device="cuda", dtype=torch.int32)
    freq = rotary.frequencies(rot, 1e4, factor=4.0, device="cuda")
    kp0, vp0 = kp.clone(), vp.clone()
    out = torch.full_like(q, float("nan")).contiguous()
    got = binding.rotary_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, interleaved=inter,
                                           magnitude=1.25, q_out=out)
    torch.cuda.synchronize()
    assert got is out and binding.device_error() == 0
    check(q, k, v, pos, slots, kp, vp, freq, inter, 1.25, out, kp0, vp0)


@pytest.mark.parametrize("inter", [False, True])
def test_in_place_on_strided_views_with_holes_and_odd_positions(inter):
    # q rotated in place inside one projection's output; skipped slots; negative and the
    # largest positions
    q, k, v, slots, kp, vp = make(37, 6, 3, 128, torch.bfloat16, 5, slot_holes=True)
    pos = torch.randint(-(1 << 20), 1 << 20, (37,), device="cuda", dtype=torch.int32)
    pos[0], pos[1], pos[2] = 2 ** 31 - 1, -2 ** 31, 0
    freq = rotary.frequencies(64, 1e6, original_len=8192, factor=8.0, device="cuda")
    q0, k0, v0, kp0, vp0 = q.clone(), k.clone(), v.clone(), kp.clone(), vp.clone()
    binding.rotary_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, interleaved=inter)
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    assert torch.equal(k, k0) and torch.equal(v, v0)
    check(q0, k0, v0, pos, slots, kp, vp, freq, inter, 1.0, q, kp0, vp0)
    assert torch.equal(q[:, :, 64:], q0[:, :, 64:])  # passed through


def test_whole_head_halves_agree_with_the_one_base_form():
    # the same rotation as ps_rope_reshape_and_cache, whose angles are reduced the same way
    q, k, v, slots, kp, vp = make(200, 12, 2, 128, torch.bfloat16, 9)
    pos = torch.randint(0, 1 << 17, (200,), device="cuda", dtype=torch.int32)
    q1, kp1, vp1 = q.contiguous(), kp.clone(), vp.clone()
    binding.rope_reshape_and_cache(q1, k.contiguous(), v.contiguous(), pos, slots, kp1, vp1, 1e6)
    out = torch.empty_like(q1)
    binding.rotary_reshape_and_cache(q, k, v, pos, slots, kp, vp,
                                     rotary.frequencies(128, 1e6, device="cuda"), q_out=out)
    torch.cuda.synchronize()
    u = torch.finfo(torch.bfloat16).eps
    for a, b in ((out, q1), (kp, kp1), (vp, vp1)):
        # two correct roundings of values 2^-19 of a pair apart: at most a step
        assert ((a.double() - b.double()).abs() <= u * b.double().abs() + 2.0 ** -17).all()


def test_slot_past_the_pool_is_recorded_and_skipped():
    q, k, v, slots, kp, vp = make(20, 4, 2, 64, torch.float16, 3)
    slots[4] = kp.shape[0] * 16
    kp0, vp0 = kp.clone(), vp.clone()
    out = torch.empty(20, 4, 64, dtype=torch.float16, device="cuda")
    pos = torch.arange(20, device="cuda", dtype=torch.int32)
    freq = rotary.frequencies(64, device="cuda")
    binding.rotary_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, q_out=out)
    assert binding.device_error() == 2
    slots[4] = -1
    check(q, k, v, pos, slots, kp, vp, freq, False, 1.0, out, kp0, vp0)


def test_no_tokens():
    q, k, v, slots, kp, vp = make(0, 4, 2, 64, torch.float16, 3)
    kp0 = kp.clone()
    binding.rotary_reshape_and_cache(q.contiguous(), k.contiguous(), v.contiguous(),
                                     torch.empty(0, dtype=torch.int32, device="cuda"), slots, kp,
                                     vp, rotary.frequencies(64, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(kp, kp0)


def test_other_stream_and_graph():
    q, k, v, slots, kp, vp = make(64, 12, 2, 128, torch.bfloat16, 11)
    pos = torch.arange(64, device="cuda", dtype=torch.int32)
    freq = rotary.frequencies(128, 1e4, device="cuda")
    kp0, vp0 = kp.clone(), vp.clone()
    out = torch.empty(64, 12, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    binding.rotary_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, q_out=out, stream=s)
    s.synchronize()
    check(q, k, v, pos, slots, kp, vp, freq, False, 1.0, out, kp0, vp0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.rotary_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, q_out=out)
    pos.add_(1000)  # the next step's positions, read by the replay
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(q, k, v, pos, slots, kp, vp, freq, False, 1.0, out, kp0, vp0)
    assert math.isfinite(float(out.float().sum()))
