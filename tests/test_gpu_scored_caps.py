"""Caps of any size beside scores of any size, with and without a bias, against float64 attention
(the tolerance: tests/_scored.py).  A cap far above the scores leaves them as they are, so its
rounding has to follow the score's size and not the cap's."""
import pytest
import torch

from tests._scored import DEV, Batch
from tests.test_gpu_scored import one, slopes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,kind", [("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16")])
@pytest.mark.parametrize("cap", [1e-6, 0.5, 3.0, 1000.0, 3e4, 1e5, 1e6])
def test_caps_from_tight_to_wide_with_a_bias(cap, cache, kind):
    for size in (0.05, 2.0, 40.0):
        b = Batch(5, [300, 140], [1, 40], 8, 2, cache, kind, q_size=size)
        one(b, cap, slopes_of(8), what=f"q {size}")


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("cap", [30.0, 1e4, 1e5, 1e6])
def test_rows_whose_scores_differ_widely(cap, bias):
    # the heads of a query share a warp: one's scores pass the cap, the others' lie far below it
    b = Batch(6, [300, 140, 700], [1, 40, 9], 8, 2)
    b.q[:, 1] *= 1e6
    b.q[:, 6] *= 1e4
    b.q[:, 3] *= 0.01
    one(b, cap, slopes_of(8) if bias else None)

