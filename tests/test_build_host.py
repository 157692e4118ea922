"""The library builds without what only the extension module of the Python calls needs."""
import os
import subprocess
import sys
import sysconfig

import pytest

import paged_kv_cache_99_gb300 as pa
from paged_kv_cache_99_gb300 import build_ext


@pytest.fixture
def no_python_headers(monkeypatch, tmp_path):
    lib = build_ext.build()
    paths = dict(sysconfig.get_paths(), include=str(tmp_path / "none"))
    monkeypatch.setattr(build_ext.sysconfig, "get_paths", lambda: paths)
    monkeypatch.setattr(build_ext, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(pa, "_BINDING", None)
    return lib


def test_the_library_stands_without_the_extension_module(no_python_headers):
    before = os.stat(no_python_headers).st_mtime_ns
    for _ in range(2):
        with pytest.warns(RuntimeWarning, match="Python.h"):
            assert build_ext.build() == no_python_headers
    assert os.stat(no_python_headers).st_mtime_ns == before          # nothing is compiled again
    assert pa.pa_version() >= 102
    with pytest.raises(ImportError):
        pa.pa_rope_table(None, [1.0] * 8)


def test_a_module_that_cannot_be_rebuilt_does_not_stay(no_python_headers):
    # it would pass arguments as an older header has them
    with open(build_ext.BINDING_PATH, "w") as f:
        f.write("an older build")
    os.utime(build_ext.BINDING_PATH, (1, 1))
    with pytest.warns(RuntimeWarning):
        build_ext.build()
    assert not os.path.exists(build_ext.BINDING_PATH)


def test_the_package_imports_without_numpy():
    # only the calls that take or give host arrays need it
    code = ("import sys; sys.modules['numpy'] = None; import paged_kv_cache_99_gb300 as pa; "
            "assert pa.pa_version() >= 102; print('imported')")
    res = subprocess.run([sys.executable, "-W", "ignore", "-c", code], cwd=build_ext.ROOT, capture_output=True, text=True)
    assert res.stdout.strip().endswith("imported"), res.stderr
