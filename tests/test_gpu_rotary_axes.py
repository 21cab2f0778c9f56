"""Rotary positions with several axes (ps_rotary_axes_reshape_and_cache) against the formula in
64 bits."""
import pytest
import torch

from paged_kv_attention_18_gb300 import binding, rotary

pytestmark = pytest.mark.gpu


def turned(x, pos, axes, freq, interleaved, magnitude):
    """x [T, H, D] in 64 bits, and |x| + |y| of each element's pair."""
    y, pair = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    half = freq.numel()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = pos[int(axes[i])].double() * freq[i]
        c, s = magnitude * torch.cos(ang)[:, None], magnitude * torch.sin(ang)[:, None]
        u, v = x[:, :, a].double(), x[:, :, b].double()
        y[:, :, a], y[:, :, b] = u * c - v * s, v * c + u * s
        pair[:, :, a] = pair[:, :, b] = abs(magnitude) * (u.abs() + v.abs())
    return y, pair


def close(got, ref, pair, dt):
    """One rounding to the type, and 2^-20 of the pair for the fp32 cosine and sine."""
    u = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * u
    assert ((got.double() - ref).abs() <= u * ref.abs() + 2.0 ** -20 * pair + tiny).all()


@pytest.mark.parametrize("T", [1, 7, 300, 5000])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,d,sections,inter,woven", [
    (14, 2, 64, [8, 12, 12], False, False), (12, 2, 128, [16, 24, 24], False, True),
    (8, 8, 128, [32, 32], True, False), (7, 1, 64, [5, 5, 5, 1], True, True),
    (4, 2, 128, [8], False, False), (12, 2, 128, [0, 3, 21], False, False)])
def test_axes(T, dt, hq, hkv, d, sections, inter, woven):
    g = torch.Generator("cuda").manual_seed(T)
    qkv = torch.randn(T, hq + 2 * hkv + 1, d, generator=g, device="cuda").to(dt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:hq + 2 * hkv]
    axes = rotary.axes(sections, woven, device="cuda")
    half, A = axes.numel(), len(sections)
    pos = torch.randint(-50, 1 << 20, (A, T), generator=g, device="cuda").int()
    freq = rotary.frequencies(2 * half, 1e6, device="cuda")
    nb = T // 16 + 3
    slots = torch.randperm(nb * 16, generator=g, device="cuda")[:T].int()
    slots[T // 2] = -1
    kp, vp = (torch.randn(nb, 16, hkv, d, generator=g, device="cuda").to(dt) for _ in range(2))
    k0, v0, q0 = kp.clone(), vp.clone(), qkv.clone()
    out = torch.empty(T, hq, d, dtype=dt, device="cuda")
    binding.rotary_axes_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, axes,
                                          interleaved=inter, magnitude=1.25, q_out=out)
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    assert torch.equal(qkv, q0)
    close(out, *turned(q, pos, axes, freq, inter, 1.25), dt)
    keep = slots >= 0
    at = slots[keep].long()
    ref, pair = turned(k, pos, axes, freq, inter, 1.25)
    close(kp.view(-1, hkv, d)[at], ref[keep], pair[keep], dt)
    assert torch.equal(vp.view(-1, hkv, d)[at], v[keep])
    other = torch.ones(nb * 16, dtype=torch.bool, device="cuda")
    other[at] = False
    assert torch.equal(kp.view(-1, hkv, d)[other], k0.view(-1, hkv, d)[other])
    assert torch.equal(vp.view(-1, hkv, d)[other], v0.view(-1, hkv, d)[other])
    # in place
    binding.rotary_axes_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, axes,
                                          interleaved=inter, magnitude=1.25)
    assert torch.equal(q, out)


def test_text_turns_as_with_one_axis():
    T, hq, hkv, d, dt = 130, 12, 2, 128, torch.bfloat16
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").to(dt) for h in (hq, hkv, hkv))
    pos = torch.randint(0, 1 << 17, (T,), generator=g, device="cuda").int()
    slots = torch.randperm(160, generator=g, device="cuda")[:T].int()
    freq = rotary.frequencies(d, 1e6, device="cuda")
    res = []
    for axes in (None, rotary.axes([16, 24, 24], device="cuda")):
        kp, vp = (torch.zeros(10, 16, hkv, d, dtype=dt, device="cuda") for _ in range(2))
        out = torch.empty_like(q)
        if axes is None:
            binding.rotary_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, q_out=out)
        else:
            binding.rotary_axes_reshape_and_cache(q, k, v, pos.expand(3, T).contiguous(), slots,
                                                  kp, vp, freq, axes, q_out=out)
        res.append((out, kp, vp))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_bad_axes_and_slots_are_recorded():
    T, dt = 40, torch.float16
    q, k, v = (torch.randn(T, h, 64, device="cuda").to(dt) for h in (4, 2, 2))
    pos = torch.randint(0, 900, (2, T), device="cuda").int()
    freq = rotary.frequencies(32, device="cuda")
    axes = rotary.axes([8, 8], device="cuda")
    kp, vp = (torch.zeros(3, 16, 2, 64, dtype=dt, device="cuda") for _ in range(2))
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    for bad in (2, -1, 2 ** 31 - 1):
        wrong = axes.clone()
        wrong[5] = bad
        out = torch.empty_like(q)
        binding.rotary_axes_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, wrong, q_out=out)
        torch.cuda.synchronize()
        assert binding.device_error() == 8
        still = freq.clone()
        still[5] = 0.0
        close(out, *turned(q, pos, axes, still, False, 1.0), dt)
    slots[7] = 48
    binding.rotary_axes_reshape_and_cache(q, k, v, pos, slots, kp, vp, freq, axes)
    torch.cuda.synchronize()
    assert binding.device_error() == 2


def test_shapes():
    T = 4
    q, k, v = (torch.randn(T, h, 64, device="cuda").half() for h in (4, 2, 2))
    pos, slots = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((3, T), (T,)))
    pool = torch.zeros(1, 16, 2, 64, device="cuda").half()
    freq, axes = rotary.frequencies(32, device="cuda"), rotary.axes([6, 5, 5], device="cuda")
    f = binding.rotary_axes_reshape_and_cache
    for args in ((pos[0], axes), (pos[:, :3].contiguous(), axes), (pos, axes[:15]),
                 (pos, axes.long()), (pos[:0], axes)):
        with pytest.raises(binding.PagedServeError):
            f(q, k, v, args[0], slots, pool, pool.clone(), freq, args[1])
