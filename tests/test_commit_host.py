"""pa_tree_commit refuses new lengths that share memory with what it reads: other warps, and the
launches of later layers, would read them as path lengths, places or blocks.  Shown without a GPU."""
import ctypes

import pytest
import torch

from paged_kv_cache_99_gb300 import build_ext
from tests.test_scored_host import _commit

P = ctypes.c_void_p
# arrays of 3 sequences, paths of 4 nodes, tables of 5 blocks, each at a place of its own
SIZES = dict(paths=4 * 12, pl=4 * 3, qsl=4 * 4, bt=4 * 15, sl=4 * 3)
PLACES = dict(paths=0x10000, pl=0x11000, qsl=0x12000, bt=0x13000, sl=0x14000)


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(build_ext.build())


def call(lib, out):
    return _commit(lib, out=P(out), B=3, maxp=4, maxb=5, **{k: P(v) for k, v in PLACES.items()})


@pytest.mark.parametrize("name", list(SIZES))
def test_new_lengths_within_an_input(lib, name):
    at, size = PLACES[name], SIZES[name]
    for out in (at, at + 4, at - 8, at + size - 4, at + size // 8 * 4):
        assert call(lib, out) == 1, (name, out - at)


def test_new_lengths_beside_an_input(lib):
    if torch.cuda.is_available():
        pytest.skip("would launch")
    for name, at in PLACES.items():
        for out in (at - 12, at + SIZES[name]):
            assert call(lib, out) == 3, name            # reaches the launch, which fails without a GPU
