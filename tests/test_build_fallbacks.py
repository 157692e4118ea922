"""The Python calls' extension module is built without the direct reading of tensors where torch
cannot be found or linked, and no intermediate file stays behind."""
import glob
import importlib.util
import os
import types

import pytest

from paged_kv_cache_99_gb300 import build_ext


@pytest.fixture
def path(monkeypatch):
    """A place beside libpa.so, which the module looks for there."""
    build_ext.build()
    path = os.path.join(build_ext.BUILD_DIR, f"_binding-fallback-{os.getpid()}.so")
    monkeypatch.setattr(build_ext, "BINDING_PATH", path)
    yield path
    left = glob.glob(path + "*") + glob.glob(os.path.join(build_ext.BUILD_DIR, f"*.{os.getpid()}.o"))
    for f in left:
        os.remove(f)
    assert set(left) <= {path}


def calls_of(path):
    spec = importlib.util.spec_from_file_location("_binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def has_direct_reading(path):
    with open(path, "rb") as f:
        return b"THPVariable" in f.read()


def test_without_torch(path, monkeypatch):
    monkeypatch.setattr(build_ext.importlib.util, "find_spec", lambda name: None)
    with pytest.warns(RuntimeWarning, match="tensor_info.cpp"):
        build_ext.build()
    assert not has_direct_reading(path)
    with pytest.raises(TypeError):
        calls_of(path).rope_table(None, [1.0] * 8, 1.0, None)


def test_where_torch_does_not_link(path, monkeypatch, tmp_path):
    # its headers are there, its libraries are not
    real = os.path.dirname(importlib.util.find_spec("torch").origin)
    os.symlink(os.path.join(real, "include"), tmp_path / "include")
    (tmp_path / "lib").mkdir()
    spec = types.SimpleNamespace(origin=str(tmp_path / "__init__.py"))
    monkeypatch.setattr(build_ext.importlib.util, "find_spec", lambda name: spec)
    with pytest.warns(RuntimeWarning, match="tensor_info.cpp"):
        build_ext.build()
    assert not has_direct_reading(path)
    with pytest.raises(TypeError):
        calls_of(path).rope_table(None, [1.0] * 8, 1.0, None)


def test_headers_that_do_not_compile_leave_nothing(path, monkeypatch, tmp_path):
    paths = dict(build_ext.sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(build_ext.sysconfig, "get_paths", lambda: paths)
    with pytest.warns(RuntimeWarning, match="binding.c was not built"):
        build_ext.build()
    assert not os.path.exists(path)
