"""Host checks of the calls with normed heads, axes, trees and scores that are not plain: what
the library and the Python calls refuse, shown without a GPU."""
import ctypes

import pytest
import torch

import paged_kv_cache_99_gb300 as pa
from paged_kv_cache_99_gb300 import build_ext
from tests.test_binding_host import _Reached, _t

FAKE = ctypes.c_void_p(0x10000)     # never dereferenced: every case below fails host checks first
F = ctypes.c_float
LL = ctypes.c_longlong


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(build_ext.build())


@pytest.fixture(autouse=True)
def nothing_is_launched(monkeypatch):
    def reached(*a):
        raise _Reached
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", reached, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", reached)


def _norm(lib, **kw):
    a = dict(qo=FAKE, qos=LL(1024), q=FAKE, qs=LL(1536), k=FAKE, ks=LL(1536), v=FAKE, vs=LL(1536), qw=FAKE, kw=FAKE,
             eps=F(1e-6), off=F(0), kc=FAKE, vc=FAKE, slots=FAKE, pos=FAKE, axes=1, map=None, table=FAKE, maxp=100,
             rot=128, layout=0, T=3, hq=8, hkv=2, d=128, bs=16, nb=10, sd=0, cd=0, kscale=None, vscale=None, ws=None,
             stream=None)
    a.update(kw)
    return lib.pa_norm_rope_and_cache(*a.values())


def test_norm_rope_refusals(lib):
    for kw in (dict(d=64), dict(bs=64), dict(sd=2), dict(cd=1), dict(rot=24), dict(rot=144), dict(layout=3), dict(axes=0),
               dict(axes=5)):
        assert _norm(lib, **kw) == 2, kw
    three = (ctypes.c_uint8 * 64)(*([0] * 63 + [3]))
    for kw in (dict(q=None), dict(pos=None), dict(table=None), dict(cd=2), dict(eps=F(-1)), dict(eps=F(float("nan"))),
               dict(off=F(float("inf"))), dict(qw=ctypes.c_void_p(0x10008)), dict(qs=LL(1537)), dict(qos=LL(1000)),
               dict(T=-1), dict(maxp=0), dict(axes=3, map=three), dict(ws=ctypes.c_void_p(0x10010))):
        assert _norm(lib, **kw) == 1, kw
    assert _norm(lib, T=0, q=None, pos=None) == 0


def _scored(lib, **kw):
    a = dict(out=FAKE, q=FAKE, qsl=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, maxb=4, sl=FAKE, prefix=None, slopes=None, cap=F(0),
             window=0, B=2, T=3, hq=8, hkv=2, d=128, bs=16, nb=10, scale=F(0.088), qd=0, cd=0, ks=None, vs=None, ws=FAKE,
             wsb=ctypes.c_size_t(1 << 40), stream=None)
    a.update(kw)
    return lib.pa_mixed_scored(*a.values())


def _tree(lib, **kw):
    a = dict(out=FAKE, q=FAKE, qsl=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, maxb=4, sl=FAKE, masks=FAKE, words=1, cap=F(0),
             window=0, B=2, T=3, hq=8, hkv=2, d=128, bs=16, nb=10, scale=F(0.088), qd=0, cd=0, ks=None, vs=None, ws=FAKE,
             wsb=ctypes.c_size_t(1 << 40), stream=None)
    a.update(kw)
    return lib.pa_tree(*a.values())


@pytest.mark.parametrize("call", [_scored, _tree])
def test_scored_and_tree_refusals(lib, call):
    odd = ctypes.c_void_p(0x10002)
    for kw in (dict(d=64), dict(bs=64), dict(qd=2), dict(cd=1), dict(hq=258, hkv=2), dict(T=1 << 29),
               dict(maxb=1 << 28, B=64), dict(nb=1 << 28), dict(cap=F(9e-7)), dict(cap=F(1.1e6)),
               dict(cap=F(1e-6), scale=F(1e34))):
        assert call(lib, **kw) == 2, kw
    for kw in (dict(q=None), dict(out=None), dict(qsl=None), dict(kc=None), dict(sl=None), dict(bt=None), dict(ws=None),
               dict(hq=7), dict(B=-1), dict(B=9000), dict(T=-1), dict(cap=F(-1)), dict(cap=F(float("nan"))),
               dict(cap=F(float("inf"))), dict(window=-1), dict(cd=2), dict(scale=F(float("inf"))), dict(qsl=odd),
               dict(ws=ctypes.c_void_p(0x10010)), dict(q=ctypes.c_void_p(0x10008))):
        assert call(lib, **kw) == 1, kw


def test_what_only_one_of_them_takes(lib):
    odd = ctypes.c_void_p(0x10002)
    assert _scored(lib, prefix=odd) == 1 and _scored(lib, slopes=odd) == 1
    assert _tree(lib, masks=None) == 1 and _tree(lib, words=0) == 1 and _tree(lib, masks=ctypes.c_void_p(0x10004)) == 1


def _commit(lib, **kw):
    ptrs = ctypes.c_void_p * 2
    a = dict(out=ctypes.c_void_p(0x20000), ks=ptrs(0x100000, 0x200000), vs=ptrs(0x300000, 0x400000), layers=2, paths=FAKE,
             pl=FAKE, maxp=4, qsl=FAKE, bt=FAKE, maxb=4, sl=FAKE, B=2, hkv=2, d=128, bs=16, nb=10, cd=0, ws=None,
             stream=None)
    a.update(kw)
    return lib.pa_tree_commit(*a.values())


def test_commit_refusals(lib):
    ptrs = ctypes.c_void_p * 2
    for kw in (dict(d=64), dict(bs=4), dict(cd=9), dict(maxb=1 << 28), dict(B=8000, hkv=1 << 18)):
        assert _commit(lib, **kw) == 2, kw
    for kw in (dict(out=None), dict(paths=None), dict(pl=None), dict(qsl=None), dict(bt=None), dict(sl=None),
               dict(out=FAKE), dict(B=-1), dict(layers=-1), dict(maxp=-1), dict(hkv=0), dict(ks=None),
               dict(ks=ptrs(0x100000, None)), dict(vs=ptrs(0x300008, 0x400000)), dict(vs=ptrs(0x100000, 0x400000)),
               dict(ks=ptrs(0x100000, 0x100000)), dict(ks=ptrs(0x100000, 0x300000)), dict(ws=ctypes.c_void_p(0x10010))):
        assert _commit(lib, **kw) == 1, kw
    assert _commit(lib, B=0, out=None, paths=None) == 0
    assert _commit(lib, layers=0, ks=None, vs=None) == 0


# ---- the Python calls ------------------------------------------------------------

def _i(*shape, dtype=torch.int32):
    return _t(*shape, dtype=dtype)


def _py_scored(**kw):
    a = dict(out=_t(3, 8, 128), q=_t(3, 8, 128), query_start_loc=_i(3), k_cache=_t(10, 2, 16, 128), v_cache=_t(10, 2, 16, 128),
             block_tables=_i(2, 4), seq_lens=_i(2), scale=0.088, workspace=_t(1 << 10, dtype=torch.uint8))
    a.update(kw)
    pa.pa_mixed_scored(**a)


def _py_tree(**kw):
    a = dict(out=_t(3, 8, 128), q=_t(3, 8, 128), query_start_loc=_i(3), k_cache=_t(10, 2, 16, 128), v_cache=_t(10, 2, 16, 128),
             block_tables=_i(2, 4), seq_lens=_i(2), masks=_i(3, 1, dtype=torch.int64), scale=0.088,
             workspace=_t(1 << 10, dtype=torch.uint8))
    a.update(kw)
    pa.pa_tree(**a)


@pytest.mark.parametrize("call", [_py_scored, _py_tree])
def test_python_scored_shapes(call):
    with pytest.raises(_Reached):
        call()
    for kw in (dict(out=_t(3, 8, 64)), dict(out=_t(2, 8, 128)), dict(query_start_loc=_i(2)), dict(seq_lens=_i(3)),
               dict(block_tables=_i(3, 4)), dict(v_cache=_t(10, 2, 8, 128)), dict(k_cache=_t(10, 2, 16, 64)),
               dict(q=_t(3, 16, 128)[:, ::2])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=torch.zeros(3, 8, 128)), dict(seq_lens=_i(2, dtype=torch.int64)), dict(workspace=None), dict(cap="x"),
               dict(k_cache=_t(10, 2, 16, 128, dtype=torch.uint8), v_cache=_t(10, 2, 16, 128, dtype=torch.uint8)),
               dict(window=1.5)):
        with pytest.raises(TypeError):
            call(**kw)


def test_python_options():
    with pytest.raises(ValueError):
        _py_scored(slopes=_t(2, dtype=torch.float32))
    with pytest.raises(ValueError):
        _py_scored(prefix_lens=_i(3))
    with pytest.raises(_Reached):
        _py_scored(slopes=_t(8, dtype=torch.float32), prefix_lens=_i(2), window=1 << 40)
    with pytest.raises(ValueError):
        _py_tree(masks=_i(2, 1, dtype=torch.int64))


def _py_norm(**kw):
    a = dict(q_out=_t(3, 8, 128), q=_t(3, 8, 128), k=_t(3, 2, 128), v=_t(3, 2, 128), k_cache=_t(10, 2, 16, 128),
             v_cache=_t(10, 2, 16, 128), slot_mapping=_i(3, dtype=torch.int64), positions=_i(3, dtype=torch.int64),
             cos_sin=_t(50, 128, dtype=torch.float32), q_weight=_t(128), k_weight=_t(128))
    a.update(kw)
    pa.pa_norm_rope_and_cache(**a)


def test_python_norm_rope():
    for kw in (dict(), dict(positions=_i(3, 3, dtype=torch.int64), axes=pa.rope_axes((16, 24, 24))), dict(q_weight=None)):
        with pytest.raises(_Reached):
            _py_norm(**kw)
    for kw in (dict(q_weight=_t(64)), dict(positions=_i(3, 2, dtype=torch.int64)), dict(positions=_i(1, 1, 3, dtype=torch.int64)),
               dict(axes=bytes(32)), dict(v=_t(3, 4, 128)), dict(k_weight=_t(2, 128))):
        with pytest.raises(ValueError):
            _py_norm(**kw)
    for kw in (dict(q_weight=_t(128, dtype=torch.float32)), dict(axes=[0] * 64), dict(eps=None)):
        with pytest.raises(TypeError):
            _py_norm(**kw)


def _py_commit(**kw):
    a = dict(seq_lens_out=_i(2), k_caches=[_t(10, 2, 16, 128)] * 3, v_caches=[_t(10, 2, 16, 128)] * 3, paths=_i(2, 4),
             path_lens=_i(2), query_start_loc=_i(3), block_tables=_i(2, 4), seq_lens=_i(2))
    a.update(kw)
    pa.pa_tree_commit(**a)


def test_python_commit():
    with pytest.raises(_Reached):
        _py_commit()
    for kw in (dict(k_caches=[]), dict(v_caches=[_t(10, 2, 16, 128)] * 2), dict(paths=_i(3, 4)), dict(path_lens=_i(3)),
               dict(query_start_loc=_i(2)), dict(k_caches=[_t(10, 2, 16, 128)] * 2 + [_t(11, 2, 16, 128)])):
        with pytest.raises(ValueError):
            _py_commit(**kw)
    for kw in (dict(k_caches=3), dict(k_caches=[None] * 3), dict(v_caches=[_t(10, 2, 16, 128, dtype=torch.uint8)] * 3)):
        with pytest.raises(TypeError):
            _py_commit(**kw)


def test_rope_axes():
    assert pa.rope_axes((2, 1)) == bytes([0, 0, 1])
    assert pa.rope_axes((3, 1, 2), in_turns=True) == bytes([0, 1, 2, 0, 2, 0])
    for bad in ((), (1, 1, 1, 1, 1), (2, -1)):
        with pytest.raises(ValueError):
            pa.rope_axes(bad)
