"""What is small in the attention with scores that are not plain: scales and caps near the ends
of their ranges, and weights far below a row's largest."""
import pytest

from tests._scored import Batch
from tests.test_gpu_scored import one

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,kind", [("bf16", "bf16"), ("fp8", "fp16")])
@pytest.mark.parametrize("cap,scale", [(1e-6, 1.2e-14), (1e-6, 5e-14), (1e-5, 1.1e-13), (1e-4, 1e-11), (1e-6, -1.2e-14),
                                       (40.0, 5e-7), (1e-6, 1e-40)])
def test_scores_that_vanish_beside_a_cap(cap, scale, cache, kind):
    # all weights are alike, and keys that a row does not see weigh nothing
    b = Batch(7, [300, 140, 33], [1, 40, 20], 8, 2, cache, kind)
    b.scale = scale
    one(b, cap)
    one(b, cap, None, 37)
