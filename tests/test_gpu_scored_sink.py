"""A row whose weight lies nearly all on one token that carries nothing (an attention sink), over
a long context: what the others add up to is the output, however little each weighs."""
import pytest
import torch

from tests._scored import DEV, Batch
from tests.test_gpu_scored import call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,kind", [("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16"), ("fp8", "fp16")])
@pytest.mark.parametrize("cap", [0.0, 50.0])
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("bits", [20, 26])
@pytest.mark.parametrize("seqs", [1, 160])
def test_many_small_weights_beside_a_sink(cache, kind, cap, rows, bits, seqs):
    """seqs: sequences over the same blocks; with many of them a CTA goes through a whole context."""
    n = 60000
    b = Batch(8, [n], [rows], 4, 1, cache, kind)
    # every query is a constant, the fifth key the same constant: a score of `bits` in log2 units
    # above most, with a V of zeros; the other Vs are positive
    at = (int(b.tables[0, 5 // b.bs]), slice(None), 5 % b.bs)
    kc, vc = b.caches
    if cache == "fp8":
        kc[at] = 0x7E
        vc &= 0x7F
        vc[at] = 0
        value = 448 * float(b.ks[0])
        vs = float(b.vs[0])
        held = vc.view(torch.float8_e4m3fn)
    else:
        value, vs = 4.5, 1.0
        kc[at] = value
        vc.abs_()
        vc[at] = 0
        held = vc
    high = bits * 0.6931471805599453
    x = high / cap if cap else 0.0
    score = cap * 0.5 * torch.log(torch.tensor((1 + x) / (1 - x), dtype=torch.float64)).item() if cap else high
    b.q[:] = score / (128 * value * b.scale)
    p = torch.arange(n, device=DEV)
    place = b.tables[0].long()[p // b.bs]
    b.v[0] = held[place, :, p % b.bs].double() * vs
    b.k[0][5] = value if cache != "fp8" else b.k[0].new_tensor(448.0) * b.ks.double()
    b.tables, b.lens, b.lens_h = b.tables.repeat(seqs, 1), b.lens.repeat(seqs), [n] * seqs
    b.start = torch.arange(seqs + 1, dtype=torch.int32, device=DEV) * rows
    one = b.q
    b.q = one.repeat(seqs, 1, 1)
    got = call(b, cap=cap).double().view(seqs, rows, 4, 128)
    b.q = one
    s = torch.einsum("mhd,nd->mhn", b.q.double(), b.k[0][:, 0]) * b.scale
    e = 128 * 2.0 ** -23 * torch.einsum("mhd,nd->mhn", b.q.double().abs(), b.k[0][:, 0].abs()) * b.scale + 2.0 ** -18 * s.abs()
    if cap:
        s = cap * torch.tanh(s / cap)
    see = p <= (n - rows + torch.arange(rows, device=DEV))[:, None]
    w = torch.softmax(s.masked_fill(~see[:, None], float("-inf")), -1)
    want = torch.einsum("mhn,nd->mhd", w, b.v[0][:, 0])
    # a weight is off by its score's error e, with the largest's, and by its rounding to 16 bits: half a
    # step, or below fp16's normal range 2^-25 of a unit that stands 2^6 below the row's largest; the
    # exponential and the sum 2^-19; the output by half a step of its type
    u_p, u_o = 2.0 ** -8 if cache == "bf16" else 2.0 ** -11, 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    rel = u_p + 2.0 ** -19 + torch.expm1(e + e.amax(-1, keepdim=True))
    tol = torch.einsum("mhn,nd->mhd", w * rel, b.v[0][:, 0])
    if cache != "bf16":
        tol += 2.0 ** -31 * torch.einsum("mn,nd->md", see.double(), b.v[0][:, 0])[:, None]
    tol += u_o * (want + tol) + (2.0 ** -25 if kind == "fp16" else 0.0)
    off = (got - want).abs()
    assert bool((off <= tol).all()), (float((off / want).max()), float((tol / want).max()))
