"""Rotary positions without a GPU: the frequencies against their formulas, and the
arguments that the calls refuse on the host."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_99_gb300 as pa
from paged_kv_cache_99_gb300 import build_ext

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: every case below fails host checks first
INVALID, UNSUPPORTED = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return pa._lib()


@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("base", [100.0, 10000.0, 1e6])
def test_unscaled_and_linear_frequencies(lib, rot, base):
    i = np.arange(rot // 2)
    want = base ** (-2.0 * i / rot)
    np.testing.assert_allclose(pa.pa_rope_frequencies(rot, base), want, rtol=1e-14)
    np.testing.assert_allclose(pa.pa_rope_frequencies(rot, base, pa.PA_ROPE_LINEAR, 8.0), want / 8, rtol=1e-14)


def test_by_parts_frequencies(lib):
    # fast components keep their frequency, slow ones are divided, the ones between are blended
    f = pa.pa_rope_frequencies(128, 10000.0)
    g = pa.pa_rope_frequencies(128, 10000.0, pa.PA_ROPE_BY_PARTS, 16.0, 8192, 1.0, 32.0)
    turns = 8192 * f / (2 * math.pi)
    assert np.all(g[turns >= 32] == f[turns >= 32])
    np.testing.assert_allclose(g[turns <= 1], f[turns <= 1] / 16, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert mid.sum() > 3
    keep = (turns[mid] - 1) / 31
    np.testing.assert_allclose(g[mid], keep * f[mid] + (1 - keep) * f[mid] / 16, rtol=1e-13)


def test_frequencies_refusals(lib):
    out = np.zeros(64)

    def call(rot=128, base=1e4, kind=0, factor=1.0, trained=8192.0, low=1.0, high=32.0, ptr=out.ctypes.data):
        return lib.pa_rope_frequencies(ptr, rot, base, kind, factor, trained, low, high)

    assert call() == 0
    for rot in (0, 8, 24, 144, -16):
        assert call(rot=rot) == UNSUPPORTED
    assert call(kind=3) == UNSUPPORTED
    assert call(ptr=None) == INVALID
    for base in (0.0, -1.0, math.inf, math.nan):
        assert call(base=base) == INVALID
    for factor in (0.0, -2.0, math.inf, math.nan):
        assert call(kind=1, factor=factor) == INVALID
        assert call(factor=factor) == 0                       # not read
    assert call(kind=2, trained=0.0) == INVALID
    assert call(kind=2, low=32.0, high=32.0) == INVALID
    assert call(kind=2, low=-1.0) == INVALID
    assert call(kind=2, high=math.inf) == INVALID


def test_frequencies_that_are_not_finite_are_refused(lib):
    # finite arguments whose formula leaves the range of doubles
    out = np.full(64, 7.0)
    for base, kind, factor, trained in ((5e-324, 0, 1.0, 0.0), (1e4, 1, 1e-310, 0.0), (1e4, 2, 5e-324, 8192.0)):
        assert lib.pa_rope_frequencies(out.ctypes.data, 128, base, kind, factor, trained, 1.0, 32.0) == INVALID
        assert np.all(out == 7.0)                # nothing is written
    assert lib.pa_rope_frequencies(out.ctypes.data, 128, 1e-300, 0, 1.0, 0.0, 1.0, 32.0) == 0 and np.isfinite(out).all()
    # the largest blended frequency is 0.0063 / 1e-310: still a double
    assert lib.pa_rope_frequencies(out.ctypes.data, 128, 1e4, 2, 1e-310, 8192.0, 1.0, 32.0) == 0
    assert np.isfinite(out).all() and 6e307 < out.max() < 7e307
    # every component turns more than 32 times over 8192 positions: all are kept, factor does not enter
    assert lib.pa_rope_frequencies(out.ctypes.data, 128, 1e-310, 2, 1e-310, 8192.0, 1.0, 32.0) == 0
    np.testing.assert_allclose(out, 1e-310 ** (-2.0 * np.arange(64) / 128), rtol=1e-14)


def test_table_refusals(lib):
    f = np.ones(64)

    def call(out=FAKE, n=10, rot=128, freqs=f.ctypes.data, attention=1.0):
        return lib.pa_rope_table(out, n, rot, freqs, attention, None)

    assert call(n=0, out=None) == 0
    assert call(n=-1) == INVALID
    assert call(rot=20) == UNSUPPORTED
    assert call(freqs=None) == INVALID
    assert call(out=None) == INVALID
    assert call(out=ctypes.c_void_p(0x10008)) == INVALID
    assert call(attention=math.nan) == INVALID
    bad = np.ones(64)
    bad[63] = math.inf
    assert call(freqs=bad.ctypes.data) == INVALID


def _rope(lib, **kw):
    a = dict(qo=FAKE, qos=1024, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, kc=FAKE, vc=FAKE, slots=FAKE, pos=FAKE,
             table=FAKE, maxp=100, rot=128, layout=0, T=4, Hq=8, Hkv=2, d=128, bs=16, nb=10, src=0, cache=0,
             kscale=None, vscale=None, ws=None, stream=None)
    a.update(kw)
    return lib.pa_rope_and_cache(*a.values())


def test_rope_and_cache_refusals(lib):
    assert _rope(lib, T=0, q=None, qo=None, k=None, v=None, slots=None, pos=None) == 0     # nothing to do
    for bad in (dict(d=64), dict(bs=64), dict(rot=8), dict(rot=136), dict(rot=40), dict(layout=2), dict(src=2),
                dict(src=0, cache=1)):
        assert _rope(lib, **bad) == UNSUPPORTED, bad
    for name in ("qo", "q", "k", "v", "kc", "vc", "slots", "pos", "table"):
        assert _rope(lib, **{name: None}) == INVALID, name
    for name in ("qo", "q", "k", "v", "kc", "vc", "table"):
        assert _rope(lib, **{name: ctypes.c_void_p(0x10008)}) == INVALID, name
    for bad in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(nb=0), dict(maxp=0), dict(qs=1028), dict(ks=-8), dict(qos=1016),
                dict(qs=4096), dict(cache=2), dict(ws=ctypes.c_void_p(0x10010))):
        assert _rope(lib, **bad) == INVALID, bad
    assert _rope(lib, T=1 << 30) == UNSUPPORTED              # more rows than 32 bits number


def test_binding_wants_cuda_tensors():
    import torch
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        pa.pa_rope_and_cache(x, x, x, x, x, x, x, x, x)
