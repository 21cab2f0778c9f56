"""Refusals of the rotary, masked attention, beam selection and fork entry points (no GPU),
and the tables of rotary frequencies."""
import ctypes
import math

import pytest
import torch

from paged_kv_attention_18_gb300 import binding, rotary

FAKE = 0x10000
F = ctypes.c_float


def caller(f, names):
    return lambda **kw: f(*[kw.get(n, d) for n, d in names])


def test_rotary_refuses(lib):
    f = caller(lib.ps_rotary_reshape_and_cache, (
        ("q", FAKE), ("qs", 12 * 128), ("k", FAKE), ("ks", 256), ("v", FAKE), ("vs", 256),
        ("pos", FAKE), ("slots", FAKE), ("kp", FAKE), ("vp", FAKE), ("freq", FAKE), ("rot", 64),
        ("inter", 0), ("mag", F(1.0)), ("out", FAKE + 16), ("os", 12 * 128), ("T", 4), ("hq", 12),
        ("hkv", 2), ("d", 128), ("nb", 8), ("dt", 1), ("s", None)))
    assert f(d=96) == -2 and f(hq=5) == -2 and f(dt=2) == -2
    assert f(rot=0) == -1 and f(rot=144) == -1 and f(rot=-16) == -1
    assert f(rot=24) == -2 and f(rot=2) == -2
    assert f(T=-1) == -1 and f(nb=0) == -1 and f(nb=1 << 28) == -1
    assert f(mag=F(math.nan)) == -1 and f(mag=F(math.inf)) == -1
    assert f(qs=12 * 128 - 8) == -1 and f(ks=248) == -1 and f(vs=0) == -1 and f(os=8) == -1
    assert f(qs=12 * 128 + 4) == -3 and f(vs=257) == -3
    assert f(q=FAKE + 2) == -3 and f(out=FAKE + 8) == -3 and f(freq=FAKE + 4) == -3
    for name in ("q", "k", "v", "pos", "slots", "kp", "vp", "freq", "out"):
        assert f(**{name: None}) == -1
    assert f(out=FAKE, os=12 * 128 + 8) == -1  # in place with another stride
    assert f(T=0, q=None, k=None, v=None, out=None) == 0


def test_masked_attention_refuses(lib):
    need = lib.ps_paged_attention_workspace_size(3, 2, 12, 2, 128, 64)
    f = caller(lib.ps_paged_attention_masked, (
        ("q", FAKE), ("kp", FAKE), ("vp", FAKE), ("bt", FAKE), ("mb", 4), ("sl", FAKE),
        ("qsl", FAKE), ("B", 2), ("T", 3), ("hq", 12), ("hkv", 2), ("d", 128), ("nb", 64),
        ("scale", F(0.1)), ("cap", F(0.0)), ("slopes", None), ("window", 0), ("prefix", None),
        ("starts", None), ("out", FAKE), ("ws", FAKE), ("wsb", need), ("dt", 1), ("s", None)))
    for bad in (0.0, -1.0, math.nan, math.inf, 3e38):
        assert f(scale=F(bad)) == -1
    for bad in (-1.0, math.nan, math.inf, 1e-42, 3e38):
        assert f(cap=F(bad)) == -1
    assert f(window=-1) == -1
    assert f(d=96) == -2 and f(hq=5) == -2 and f(dt=2) == -2
    assert f(T=-1) == -1 and f(B=-1) == -1 and f(B=0) == -1 and f(nb=0) == -1 and f(mb=0) == -1
    for name in ("q", "kp", "vp", "bt", "sl", "qsl", "out"):
        assert f(**{name: None}) == -1
    assert f(q=FAKE + 8) == -3 and f(out=FAKE + 2) == -3
    assert f(ws=None) == -4 and f(ws=FAKE + 16) == -4 and f(wsb=256) == -4
    assert f(T=0, B=0) == 0


def test_beam_select_refuses(lib):
    size = lib.ps_beam_select_workspace_size
    need = size(2, 4, 1000, 4)
    assert need > 0
    for bad in ((-1, 4, 10, 4), (2, 0, 10, 4), (2, 33, 10, 4), (2, 4, 0, 4), (2, 4, 10, 0),
                (2, 4, 10, 33), (1, 32, 1 << 27, 4)):
        assert size(*bad) == 0
    f = caller(lib.ps_beam_select, (
        ("x", FAKE), ("ld", 1000), ("sc", FAKE), ("fin", None), ("pad", 0), ("B", 2), ("W", 4),
        ("V", 1000), ("n", 4), ("dt", 2), ("par", FAKE), ("tok", FAKE), ("out", FAKE),
        ("ws", FAKE), ("wsb", need), ("s", None)))
    assert f(B=-1) == -1 and f(W=0) == -1 and f(V=0) == -1 and f(n=0) == -1
    assert f(W=33) == -2 and f(n=33) == -2 and f(V=1 << 30) == -2
    assert f(dt=3) == -2 and f(dt=-1) == -2
    assert f(ld=999) == -1
    assert f(fin=FAKE, pad=1000) == -1 and f(fin=FAKE, pad=-1) == -1
    for name in ("x", "sc", "par", "tok", "out"):
        assert f(**{name: None}) == -1
    assert f(x=FAKE + 2) == -3 and f(x=FAKE + 1, dt=0) == -3
    assert f(ws=None) == -4 and f(ws=FAKE + 8) == -4 and f(wsb=need - 1) == -4
    assert f(B=0, x=None, sc=None, ws=None) == 0


def test_fork_refuses(lib):
    f = caller(lib.ps_fork_sequences, (
        ("bt", FAKE), ("mb", 8), ("sl", FAKE), ("par", FAKE), ("tails", FAKE), ("g", 2),
        ("nin", 4), ("nout", 4), ("kp", FAKE), ("vp", FAKE), ("layers", 3), ("nb", 64),
        ("hkv", 2), ("d", 128), ("dt", 1), ("obt", 2 * FAKE), ("ol", 2 * FAKE), ("s", None)))
    assert f(d=96) == -2 and f(dt=2) == -2 and f(hkv=0) == -1
    assert f(g=-1) == -1 and f(nin=0) == -1 and f(nout=0) == -1 and f(layers=0) == -1
    assert f(mb=0) == -1 and f(nb=0) == -1 and f(nb=1 << 28) == -1
    assert f(g=1 << 30) == -1 and f(layers=1 << 21) == -1
    for name in ("bt", "sl", "par", "tails", "kp", "vp", "obt", "ol"):
        assert f(**{name: None}) == -1
    assert f(obt=FAKE) == -1 and f(ol=FAKE) == -1  # the children's own arrays
    assert f(kp=FAKE + 8) == -3
    assert f(g=0, bt=None) == 0


def test_the_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(binding.PagedServeError):
        binding.rotary_reshape_and_cache(x, x, x, i, i, x, x, torch.zeros(32).double())
    with pytest.raises(binding.PagedServeError):
        binding.rotary_reshape_and_cache(x.float(), x, x, i, i, x, x, torch.zeros(32).double())
    with pytest.raises(binding.PagedServeError):
        binding.masked_paged_attention(x, x, x, i, i, i, 1.0)
    with pytest.raises(binding.PagedServeError):
        binding.beam_select(torch.zeros(1, 2, 5), torch.zeros(1, 2), 2)
    with pytest.raises(binding.PagedServeError):
        binding.fork_sequences(i, i, i, i, x, x, i, i)


def test_frequencies():
    R = 64
    plain = rotary.frequencies(R, 1e4)
    assert plain.dtype == torch.float64 and plain.shape == (R // 2,)
    for i in (0, 1, 17, 31):
        assert abs(float(plain[i]) - 1e4 ** (-2 * i / R)) <= 1e-15
    assert torch.equal(rotary.frequencies(R, 1e4, factor=4.0), plain / 4)
    base = rotary.frequencies(R, 1e4, theta_factor=8.0)
    assert float(base[0]) == 1.0
    assert abs(float(base[-1] * 8 / plain[-1]) - 1) < 1e-12  # the lowest falls by the factor
    by = rotary.frequencies(R, 1e4, factor=8.0, original_len=4096, low=1.0, high=4.0)
    for i in range(R // 2):
        turns = 4096 * float(plain[i]) / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / 3.0))
        assert abs(float(by[i]) - float(plain[i]) * (keep + (1 - keep) / 8)) < 1e-15
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, factor=0.0),
                dict(rotary_dim=2, theta_factor=2.0),
                dict(rotary_dim=8, original_len=100, low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            rotary.frequencies(**bad)
