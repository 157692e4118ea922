"""pa_norm_rope_and_cache with q_out in the place of q, a slice of the fused projection, at sizes
where tokens are copied ahead and worked rows go back in bulk: bit for bit what another q_out gets."""
import pytest
import torch

import paged_kv_cache_99_gb300 as pa
from tests.test_gpu_norm_rope import DEV, Case

pytestmark = pytest.mark.gpu


# a group of threads per row; four CTAs of four warps to an SM; three of six (16-bit caches)
@pytest.mark.parametrize("T", [200, 3000, 8000])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(T, cache, interleaved):
    def case():
        c = Case(T, T, 32, 8, 128, "bf16", cache, axes=list(pa.rope_axes((24, 20, 20))))
        g = torch.Generator(device=DEV).manual_seed(2)
        pad = torch.rand(T, generator=g, device=DEV) < 0.1
        c.pos[1, pad] = -1
        c.slots[torch.rand(T, generator=g, device=DEV) < 0.1] = -1
        return c, pad

    c, pad = case()
    keep = c.qkv.clone()
    want = c.run(interleaved=interleaved)
    assert torch.equal(c.qkv, keep)
    d, _ = case()
    q = d.qkv[:, :32]
    for _ in range(2):                      # the second time on fresh values in the same memory
        d.qkv.copy_(keep)
        d.run(q_out=q, interleaved=interleaved)
        assert torch.equal(q[~pad], want[~pad])
        assert torch.equal(q[pad], keep[pad, :32]) and torch.equal(d.qkv[:, 32:], keep[:, 32:])
        assert torch.equal(c.kc, d.kc) and torch.equal(c.vc, d.vc)
