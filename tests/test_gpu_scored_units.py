"""Units that begin and end all the time: what the two threads of a row tell each other at a
unit's last step (maximum, then sum, in the same place) is not mixed up."""
import pytest
import torch

from tests._scored import Batch, causal, check, random_trees, reference, tree_sight
from tests.test_gpu_scored import call
from tests.test_gpu_tree import call as call_tree

pytestmark = pytest.mark.gpu


def batch(seed, cache, kind, q_size):
    g = torch.Generator().manual_seed(seed)
    rows = [int(x) for x in torch.randint(1, 80, (160,), generator=g)] + [1] * 160
    lens = [r + int(torch.randint(0, 200, (1,), generator=g)) for r in rows]
    return Batch(seed, lens, rows, 16, 2, cache, kind, q_size=q_size)


# scores near zero: the sums (up to 64 to a thread and step) lie far above the maxima
@pytest.mark.parametrize("q_size", [0.02, 2.0])
@pytest.mark.parametrize("cache,kind", [("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16"), ("fp8", "fp16")])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_maxima_and_sums_of_many_short_units(q_size, cache, kind, cap):
    b = batch(71, cache, kind, q_size)
    first = call(b, cap=cap)
    check(first, *reference(b, causal(b), cap))
    for _ in range(30):
        assert torch.equal(call(b, cap=cap), first)


def test_maxima_and_sums_of_many_short_trees():
    b = batch(72, "bf16", "bf16", 0.02)
    sight, masks = tree_sight(b, random_trees(b, 1))
    first = call_tree(b, masks)
    check(first, *reference(b, sight))
    for _ in range(30):
        assert torch.equal(call_tree(b, masks), first)
