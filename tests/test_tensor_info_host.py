"""What is read from a tensor directly (csrc/tensor_info.cpp) is what its Python methods say,
shown on CPU tensors."""
import ctypes

import pytest
import torch

from paged_kv_cache_99_gb300 import build_ext

TYPES = [torch.bfloat16, torch.float16, torch.uint8, torch.float8_e4m3fn, torch.float32, torch.int32, torch.int64]


class Info(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("shape", ctypes.POINTER(ctypes.c_int64)), ("stride", ctypes.POINTER(ctypes.c_int64)),
                ("ndim", ctypes.c_int), ("type", ctypes.c_int), ("device", ctypes.c_int), ("contiguous", ctypes.c_int)]


@pytest.fixture(scope="module")
def read():
    build_ext.build()
    lib = ctypes.PyDLL(build_ext.BINDING_PATH)
    try:
        fn = lib.pa_tensor_info
    except AttributeError:
        pytest.skip("torch's headers are not there")
    fn.argtypes = [ctypes.py_object, ctypes.POINTER(Info)]

    def read(t):
        info = Info()
        return info if fn(t, ctypes.byref(info)) == 0 else None
    return read


def _strided():
    x = torch.arange(4 * 6 * 8).view(4, 6, 8)
    return [x, x[1:], x[:, 2:4], x.transpose(0, 1), x[:, :, ::2], x[:0], x[0, 0, 0], x.expand(2, 4, 6, 8), torch.empty(0, 3),
            torch.nn.Parameter(torch.zeros(3, 5)), torch.zeros(3, requires_grad=True)]


def test_direct_reading_agrees_with_the_methods(read):
    for t in _strided() + [torch.ones(3, 4, dtype=t)[:, 1:] for t in TYPES]:
        info = read(t)
        assert (info.ptr or 0) == t.data_ptr()
        assert info.ndim == t.dim() and [info.shape[d] for d in range(t.dim())] == list(t.shape)
        assert [info.stride[d] for d in range(t.dim())] == list(t.stride())
        assert bool(info.contiguous) == t.is_contiguous() and info.device == t.get_device() == -1
        assert TYPES[info.type] == t.dtype


def test_other_types_and_what_is_no_plain_tensor(read):
    assert read(torch.zeros(2, dtype=torch.float64)).type == -1
    assert read(torch.zeros(2, dtype=torch.bool)).type == -1

    class Sub(torch.Tensor):
        pass
    for t in (torch.zeros(2).as_subclass(Sub), torch.zeros(2, 2).to_sparse(), None, 3, "x"):
        assert read(t) is None


def test_a_lazy_clone_is_written_to_itself_alone(read):
    """An output whose storage is shared until it is written: the pointer that is written through
    is its own, as data_ptr() gives it."""
    if not hasattr(torch, "_lazy_clone"):
        pytest.skip("no lazy clones in this torch")
    x = torch.full((3, 16), 5.0)
    for view in (lambda t: t, lambda t: t[1:]):
        y = torch._lazy_clone(x)
        v = view(y)
        ctypes.memset(read(v).ptr, 0, v.numel() * 4)
        assert bool((x == 5).all()) and bool((view(y) == 0).all())
        assert read(v).ptr == v.data_ptr()
