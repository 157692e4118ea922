"""pa_evict without a GPU: the arguments it refuses on the host."""
import ctypes

import pytest

import paged_kv_cache_99_gb300 as pa
from paged_kv_cache_99_gb300 import build_ext

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: every case below fails host checks first
OTHER = ctypes.c_void_p(0x20000)
INVALID, UNSUPPORTED = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return pa._lib()


def _evict(lib, **kw):
    a = dict(kept=FAKE, lens_out=FAKE, wout=FAKE, w=FAKE, stride=64, kc=FAKE, vc=FAKE, bt=OTHER, maxb=4, lens=OTHER, nt=FAKE,
             maxn=2, B=2, budget=20, sinks=2, recent=4, Hkv=2, d=128, bs=16, nb=10, cache=0, ws=None, stream=None)
    a.update(kw)
    return lib.pa_evict(*a.values())


def test_refusals(lib):
    assert _evict(lib, B=0, kept=None, lens_out=None, wout=None, w=None, bt=None, lens=None, nt=None) == 0
    for bad in (dict(d=64), dict(bs=64), dict(cache=4), dict(cache=-1)):
        assert _evict(lib, **bad) == UNSUPPORTED, bad
    for name in ("kept", "lens_out", "wout", "w", "kc", "vc", "bt", "lens", "nt"):
        assert _evict(lib, **{name: None}) == INVALID, name
    for name in ("wout", "w", "kc", "vc"):
        assert _evict(lib, **{name: ctypes.c_void_p(0x10008)}) == INVALID, name
    for name in ("kept", "lens_out", "lens", "bt", "nt"):
        assert _evict(lib, **{name: ctypes.c_void_p(0x10002)}) == INVALID, name
    for bad in (dict(B=-1), dict(Hkv=0), dict(nb=0), dict(maxb=0), dict(maxn=0), dict(budget=0), dict(sinks=-1),
                dict(recent=-1), dict(sinks=10, recent=11), dict(sinks=2**31 - 1, recent=2**31 - 1), dict(stride=60),
                dict(stride=66), dict(maxn=1), dict(lens=FAKE), dict(bt=FAKE), dict(ws=ctypes.c_void_p(0x10010))):
        assert _evict(lib, **bad) == INVALID, bad
    for bad in (dict(nb=1 << 27), dict(B=1 << 27), dict(maxb=1 << 26, stride=1 << 30), dict(budget=1 << 30, maxn=4),
                dict(budget=2**31 - 1, maxn=4)):
        assert _evict(lib, **bad) == UNSUPPORTED, bad
