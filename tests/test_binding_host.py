"""What the Python calls refuse before anything reaches the library, shown without a GPU:
CPU tensors that say they are on cuda:0 pass every check of the device, so that what is
refused is refused for its shape."""
import pytest
import torch

import paged_kv_cache_99_gb300 as pa
from paged_kv_cache_99_gb300 import build_ext


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on cuda:0.  No call may get past its checks with one."""

    is_cuda = True

    def get_device(self):
        return 0


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture(scope="module", autouse=True)
def built():
    build_ext.build()


class _Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def nothing_is_launched(monkeypatch):
    """The stream is asked for once every check is passed: the call ends there."""
    def reached(*a):
        raise _Reached
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", reached, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", reached)


def _weights(**kw):
    a = dict(out=_t(2, 8, 128), weights_out=_t(2, 2, 64, dtype=torch.float32), q=_t(2, 8, 128), k_cache=_t(10, 2, 16, 128),
             v_cache=_t(10, 2, 16, 128), block_tables=_t(2, 4, dtype=torch.int32), seq_lens=_t(2, dtype=torch.int32),
             scale=0.088, workspace=_t(1 << 10, dtype=torch.uint8))
    a.update(kw)
    pa.pa_decode_weights(**a)


def test_decode_weights_wants_a_cache_of_the_querys_head_dimension():
    with pytest.raises(_Reached):
        _weights()
    # half the rows the query's head dimension would read
    with pytest.raises(ValueError):
        _weights(k_cache=_t(10, 2, 16, 64), v_cache=_t(10, 2, 16, 64))
    with pytest.raises(ValueError):
        _weights(v_cache=_t(10, 2, 16, 64))
    with pytest.raises(ValueError):
        _weights(k_cache=_t(10, 2, 16, 256), v_cache=_t(10, 2, 16, 256))


def _q(B=2):
    return dict(out=_t(B, 8, 128), q=_t(B, 8, 128), scale=0.088)


def _batch(B=2):
    return dict(block_tables=_t(B, 4, dtype=torch.int32), seq_lens=_t(B, dtype=torch.int32))


def _calls():
    ws = dict(workspace=_t(1 << 10, dtype=torch.uint8))
    new = dict(k_new=_t(2, 2, 128), v_new=_t(2, 2, 128), slot_mapping=_t(2, dtype=torch.int64))
    return {
        "pa_decode": dict(**_q(), **_batch(), **ws),
        "pa_decode_append": dict(**_q(), **_batch(), **ws, **new),
        "pa_decode_shared_prefix": dict(**_q(), **_batch(), **ws, prefix_blocks=1),
        "pa_mixed": dict(**_q(), **_batch(), **ws, query_start_loc=_t(3, dtype=torch.int32), max_q_len=1),
        "pa_decode_noalloc": dict(**_q(), **_batch()),
        "pa_copy_blocks": dict(src=_t(1, dtype=torch.int32), dst=_t(1, dtype=torch.int32)),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_both_caches_have_one_shape_and_the_querys_head_dimension(name):
    def call(k, v):
        getattr(pa, name)(k_cache=k, v_cache=v, **_calls()[name])

    good = _t(10, 2, 16, 128)
    with pytest.raises(_Reached):
        call(good, good)
    for other in (_t(5, 2, 16, 128), _t(10, 1, 16, 128), _t(10, 2, 8, 128), _t(10, 2, 16, 64)):
        with pytest.raises(ValueError):
            call(good, other)
        with pytest.raises(ValueError):
            call(other, good)
    if name != "pa_copy_blocks":          # no query: the library checks its head dimension
        with pytest.raises(ValueError):
            call(_t(10, 2, 16, 64), _t(10, 2, 16, 64))
