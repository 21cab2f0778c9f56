"""Refusals of sampling, sequence extension, rotary positions with several axes and attention
with sinks (no GPU), and the tables of axes."""
import ctypes
import math

import pytest
import torch

from paged_kv_attention_18_gb300 import binding, rotary
from tests import loop_ref as R

FAKE = 0x10000
F = ctypes.c_float


def caller(f, names):
    return lambda **kw: f(*[kw.get(n, d) for n, d in names])


def test_sample_refuses(lib):
    f = caller(lib.ps_sample, (
        ("x", FAKE), ("ld", 1000), ("temp", None), ("k", None), ("p", None), ("m", None),
        ("bits", FAKE), ("B", 2), ("V", 1000), ("dt", 2), ("tok", FAKE), ("lp", FAKE), ("s", None)))
    assert f(B=-1) == -1 and f(V=0) == -1 and f(ld=999) == -1
    assert f(dt=3) == -2 and f(dt=-1) == -2
    assert f(V=393217, ld=1 << 30) == -2 and f(B=(1 << 24) + 1) == -2
    for name in ("x", "bits", "tok", "lp"):
        assert f(**{name: None}) == -1
    assert f(x=FAKE + 2) == -3 and f(x=FAKE + 1, dt=0) == -3
    assert f(B=0, x=None, bits=None, tok=None, lp=None) == 0


def test_extend_refuses(lib):
    f = caller(lib.ps_extend_sequences, (
        ("bt", FAKE), ("mb", 8), ("sl", FAKE), ("nl", FAKE + 64), ("free", FAKE), ("cap", 64),
        ("count", FAKE), ("B", 2), ("T", 5), ("nb", 64), ("window", 0), ("sinks", 0),
        ("qsl", FAKE), ("slots", FAKE), ("pos", FAKE), ("ol", FAKE), ("oc", FAKE), ("s", None)))
    assert f(ol=2 * FAKE, nl=2 * FAKE) == -1  # the numbers are read while lengths are written
    assert f(B=-1) == -1 and f(T=-1) == -1 and f(mb=0) == -1 and f(cap=-1) == -1
    assert f(nb=0) == -1 and f(nb=1 << 28) == -1 and f(window=-1) == -1 and f(sinks=-1) == -1
    assert f(B=8193) == -2 and f(B=8192, mb=1 << 18) == -2 and f(T=2 ** 31 - 1) == -2
    for name in ("bt", "sl", "nl", "free", "count", "qsl", "slots", "pos", "ol", "oc"):
        assert f(**{name: None}) == -1


def test_rotary_axes_refuses(lib):
    f = caller(lib.ps_rotary_axes_reshape_and_cache, (
        ("q", FAKE), ("qs", 12 * 128), ("k", FAKE), ("ks", 256), ("v", FAKE), ("vs", 256),
        ("pos", FAKE), ("axes", FAKE), ("na", 3), ("slots", FAKE), ("kp", FAKE), ("vp", FAKE),
        ("freq", FAKE), ("rot", 64), ("inter", 0), ("mag", F(1.0)), ("out", FAKE + 16),
        ("os", 12 * 128), ("T", 4), ("hq", 12), ("hkv", 2), ("d", 128), ("nb", 8), ("dt", 1),
        ("s", None)))
    assert f(na=0) == -1 and f(na=-1) == -1 and f(axes=None) == -1
    assert f(d=96) == -2 and f(hq=5) == -2 and f(dt=2) == -2 and f(rot=24) == -2
    assert f(rot=0) == -1 and f(rot=144) == -1 and f(mag=F(math.nan)) == -1
    assert f(qs=12 * 128 + 4) == -3 and f(q=FAKE + 2) == -3 and f(freq=FAKE + 4) == -3
    for name in ("q", "k", "v", "pos", "slots", "kp", "vp", "freq", "out"):
        assert f(**{name: None}) == -1
    assert f(T=0, axes=None, q=None) == 0


def test_streaming_attention_refuses(lib):
    need = lib.ps_paged_attention_workspace_size(3, 2, 12, 2, 128, 64)
    f = caller(lib.ps_paged_attention_streaming, (
        ("q", FAKE), ("kp", FAKE), ("vp", FAKE), ("bt", FAKE), ("mb", 4), ("sl", FAKE),
        ("qsl", FAKE), ("B", 2), ("T", 3), ("hq", 12), ("hkv", 2), ("d", 128), ("nb", 64),
        ("scale", F(0.1)), ("cap", F(0.0)), ("window", 100), ("sinks", 4), ("out", FAKE),
        ("ws", FAKE), ("wsb", need), ("dt", 1), ("s", None)))
    for bad in (0.0, -1.0, math.nan, math.inf, 3e38):
        assert f(scale=F(bad)) == -1
    for bad in (-1.0, math.nan, math.inf, 1e-42, 3e38):
        assert f(cap=F(bad)) == -1
    assert f(window=-1) == -1 and f(sinks=-1) == -1
    assert f(d=96) == -2 and f(hq=5) == -2 and f(dt=2) == -2
    assert f(T=-1) == -1 and f(B=0) == -1 and f(nb=0) == -1 and f(mb=0) == -1
    for name in ("q", "kp", "vp", "bt", "sl", "qsl", "out"):
        assert f(**{name: None}) == -1
    assert f(q=FAKE + 8) == -3 and f(out=FAKE + 2) == -3
    assert f(ws=None) == -4 and f(ws=FAKE + 16) == -4 and f(wsb=256) == -4
    assert f(T=0, B=0) == 0


def test_the_binding_refuses_host_tensors():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(binding.PagedServeError):
        binding.sample(torch.zeros(2, 5), i)
    with pytest.raises(binding.PagedServeError):
        binding.extend_sequences(i, i, i, i, i, 4, i, i, i)
    with pytest.raises(binding.PagedServeError):
        binding.rotary_axes_reshape_and_cache(x, x, x, i, i, x, x, torch.zeros(32).double(), i)
    with pytest.raises(binding.PagedServeError):
        binding.streaming_paged_attention(x, x, x, i, i, i, 1.0, 8, 4)


def test_axes():
    assert rotary.axes([2, 3, 1]).tolist() == [0, 0, 1, 1, 1, 2]
    assert rotary.axes([2, 3, 1], interleaved=True).tolist() == [0, 1, 2, 0, 1, 1]
    assert rotary.axes([0, 2]).tolist() == [1, 1]
    assert rotary.axes([4]).dtype == torch.int32
    for bad in ([], [0], [3, -1]):
        with pytest.raises(ValueError):
            rotary.axes(bad)


def test_the_references():
    """The plain forms at cases worked by hand."""
    import numpy as np
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    word = int(0.45 * 2 ** 32)
    assert R.draw(x, None, None, None, None, word)[0] == 1
    assert R.draw(x, None, 2, None, None, word)[0] == 1       # of 0.4, 0.3: 0.45 * 0.7 < 0.4
    assert R.draw(x, None, 2, None, None, int(0.6 * 2 ** 32))[0] == 3
    assert R.draw(x, None, None, 0.65, None, int(0.99 * 2 ** 32))[0] == 3  # 0.4, 0.3
    assert R.draw(x, None, None, None, 0.6, 0)[0] == 1        # 0.4 and 0.3 of 0.4
    assert R.draw(x, 0.0, None, None, None, word) == (1, 0.0)
    assert R.draw(np.array([-np.inf, np.nan]), None, None, None, None, 5)[0] == -1
    got = R.extend([[3, -1, -1], [5, 6, -1]], [16, 20], [2, 1], [9, 8, 7], 3, 4, 10)
    assert got[0] == [[3, 7, -1], [5, 6, -1]] and got[1] == [18, 21] and got[3] == 2
    assert got[4] == [0, 2, 3] and got[5] == [112, 113, 100, -1] and got[6] == [16, 17, 20, 0]
    got = R.extend([[3, 4, 5, 6]], [50], [1], [0, 0, 0, 0], 0, 1, 10, window=3, sinks=10)
    assert got[0] == [[3, -1, -1, 6]] and got[2][:2] == [5, 4] and got[3] == 2
