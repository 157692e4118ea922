"""pa_decode_weights without a GPU: the arguments it refuses on the host."""
import ctypes

import pytest

import paged_kv_cache_99_gb300 as pa
from paged_kv_cache_99_gb300 import build_ext

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: every case below fails host checks first
INVALID, UNSUPPORTED = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return pa._lib()


def _weights(lib, **kw):
    a = dict(out=FAKE, wout=FAKE, win=FAKE, stride=64, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, maxb=4, sl=FAKE, B=2, Hq=8, Hkv=2,
             d=128, bs=16, nb=10, scale=0.088, qd=0, cd=0, ks=None, vs=None, ws=FAKE, wsb=1 << 20, stream=None)
    a.update(kw)
    return lib.pa_decode_weights(*a.values())


def test_refusals(lib):
    assert _weights(lib, B=0, out=None, q=None, bt=None, sl=None, wout=None, win=None) == 0
    for bad in (dict(d=64), dict(bs=64), dict(qd=2), dict(cd=1)):
        assert _weights(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(stride=63), dict(stride=-64), dict(wout=None), dict(wout=ctypes.c_void_p(0x10002)), dict(q=None),
                dict(win=ctypes.c_void_p(0x10002)), dict(Hq=7), dict(cd=2), dict(ws=None), dict(scale=float("nan"))):
        assert _weights(lib, **bad) == INVALID, bad


def test_workspace_size_refusals(lib):
    f = lib.pa_workspace_size_weights
    assert f(2, 8, 2, 64, 100) == 0
    assert f(2, 7, 2, 128, 100) == 0
    assert f(2, 8, 2, 128, -1) == 0


def test_tables_of_more_tokens_than_32_bits_number(lib):
    # one KV head: few enough 16-key units, but the kernels number a sequence's tokens in 32 bits
    one = dict(B=1, Hq=1, Hkv=1)
    for bs, maxb in ((8, 1 << 28), (16, 1 << 27), (32, 1 << 26), (16, (1 << 27) - 1)):
        assert _weights(lib, **one, bs=bs, maxb=maxb, stride=bs * maxb) == UNSUPPORTED, (bs, maxb)
        a = [FAKE, FAKE, FAKE, FAKE, FAKE, maxb, FAKE, 1, 1, 1, 128, bs, 10, 0.088, 0, 0, None, None, FAKE, 1 << 20, None]
        assert lib.pa_decode(*a) == UNSUPPORTED, (bs, maxb)
