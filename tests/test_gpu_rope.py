"""Rotary positions on the GPU: the table against float64 angles, and the rotation
fused with the slot write against float64 rotations of the same table.

Tolerances.  The table: the angle keeps 32 bits of a quarter turn (2^-24 of it after
the conversion), the polynomial and the attention factor round a handful of times to
2^-24 of values up to 1: 2^-22 covers them.  The rotation: two products and a sum, each
off by 2^-24 of at most |a| + |b| (cosine and sine are at most the attention factor, 1
here), then half a step of the type stored (finfo.eps / 2, and half the smallest
subnormal below the normal range)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_99_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25}
NAN_BITS = 0x7FC1


@pytest.mark.parametrize("rot", [16, 48, 96, 128])
@pytest.mark.parametrize("positions", [1, 2, 41, 5000, 300001])
def test_table(rot, positions):
    f = pa.pa_rope_frequencies(rot, 500000.0, pa.PA_ROPE_BY_PARTS, 16.0, 8192)
    f[0] = 7.5                                   # over a turn per position: whole turns fall off
    t = torch.full((positions + 1, rot), 9.0, device=DEV)
    pa.pa_rope_table(t[:positions], f, 1.25)
    angle = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * torch.from_numpy(f).to(DEV)
    want = torch.cat((angle.cos(), angle.sin()), 1) * 1.25
    assert float((t[:positions].double() - want).abs().max()) <= 1.25 * 2.0 ** -22
    assert bool((t[positions] == 9.0).all())     # the row behind the table is left as it was


def test_table_of_negative_and_zero_frequencies():
    f = np.array([0.0, -0.0, -1e-300, -0.25, -3.0, 1e-30, 6.0, 2.0])
    t = torch.zeros(1000, 16, device=DEV)
    pa.pa_rope_table(t, f)
    angle = torch.arange(1000, dtype=torch.float64, device=DEV)[:, None] * torch.from_numpy(f).to(DEV)
    assert float((t.double() - torch.cat((angle.cos(), angle.sin()), 1)).abs().max()) <= 2.0 ** -22


@pytest.mark.parametrize("base,factor", [(1e4, 1.0), (5e5, 1.0), (1e6, 16.0), (1e6, -64.0)])
@pytest.mark.parametrize("rot,positions,attention", [(128, 200, 1.0), (128, 70000, 1.25), (16, 3001, 0.75)])
def test_table_entries_near_zero(base, factor, rot, positions, attention):
    """Every entry relative to itself, a slow component's sine at the first positions and
    a cosine beside a quarter turn included.  Tolerance: the sine and cosine are within
    2.2 x 2^-24 of themselves (what the polynomials' roundings add up to), the attention
    factor's product rounds once more; the angle is cut to 2^-55 quarter turns and the
    component to 2^-64 turns per position (2 pi 2^-64 < 2^-61); its quotient by 2 pi here,
    and the product with the position in the reference, round to 2^-53 of the angle, the
    constant 2 pi as well."""
    f = pa.pa_rope_frequencies(rot, base) / factor
    t = torch.empty(positions, rot, device=DEV)
    pa.pa_rope_table(t, f, attention)
    p = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None]
    angle = p * torch.from_numpy(f).to(DEV)
    want = torch.cat((angle.cos(), angle.sin()), 1) * attention
    off = (2.0 ** -54 + p * 2.0 ** -61 + 3 * 2.0 ** -53 * angle.abs()).repeat(1, 2)
    assert bool(((t.double() - want).abs() <= 3.5 * 2.0 ** -24 * want.abs() + attention * off).all())


def test_table_of_a_callers_own_frequencies():
    # a blend over the component's index between two whole components, which by-parts scaling is not
    base, factor, lo, hi = 1e6, 4.0, 23, 39
    i = np.arange(64)
    f = base ** (-2.0 * i / 128)
    keep = 1 - np.clip((i - lo) / (hi - lo), 0, 1)
    f = keep * f + (1 - keep) * f / factor
    by_parts = pa.pa_rope_frequencies(128, base, pa.PA_ROPE_BY_PARTS, factor, 32768)
    assert int((np.maximum(f / by_parts, by_parts / f) > 1.01).sum()) >= 8
    t = torch.empty(5000, 128, device=DEV)
    pa.pa_rope_table(t, f)
    angle = torch.arange(5000, dtype=torch.float64, device=DEV)[:, None] * torch.from_numpy(f).to(DEV)
    assert float((t.double() - torch.cat((angle.cos(), angle.sin()), 1)).abs().max()) <= 2.0 ** -22


class Case:
    def __init__(self, seed, T, Hq, Hkv, rot, src, cache, bs, context=4096):
        g = torch.Generator().manual_seed(seed)
        self.T, self.Hq, self.Hkv, self.rot, self.src, self.cache, self.bs = T, Hq, Hkv, rot, src, cache, bs
        self.qkv = torch.randn(T, Hq + 2 * Hkv, 128, generator=g).to(TYPES[src]).to(DEV)
        nb = -(-T // bs) + 3
        self.slots = torch.randperm(nb * bs, generator=g)[:T].to(DEV)
        self.positions = torch.randint(0, context, (T,), generator=g).to(DEV)
        angle = torch.arange(context, dtype=torch.float64)[:, None] * torch.from_numpy(pa.pa_rope_frequencies(rot))
        self.cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float().to(DEV)
        shape = (nb, Hkv, bs, 128)
        self.ks = self.vs = None
        if cache.startswith("fp8"):
            self.kc = torch.randint(0, 127, shape, generator=g, dtype=torch.uint8).to(DEV)
            n = Hkv if cache == "fp8 heads" else 1
            self.ks = (torch.rand(n, generator=g) * 0.02 + 0.005).to(DEV)
            self.vs = (torch.rand(n, generator=g) * 0.02 + 0.005).to(DEV)
        else:
            self.kc = torch.randn(shape, generator=g).to(TYPES[cache]).to(DEV)
        self.vc = self.kc.flip(0).contiguous()
        self.q_out = torch.full((T, Hq, 128), 3.0, dtype=TYPES[src], device=DEV)

    def parts(self):
        return self.qkv[:, :self.Hq], self.qkv[:, self.Hq:self.Hq + self.Hkv], self.qkv[:, self.Hq + self.Hkv:]

    def call(self, interleaved, **kw):
        q, k, v = self.parts()
        pa.pa_rope_and_cache(self.q_out, q, k, v, self.kc, self.vc, self.slots, self.positions, self.cos_sin,
                             interleaved=interleaved, k_scale=self.ks, v_scale=self.vs, **kw)

    def check(self, interleaved, k0, v0, wrote=None, turned=None):
        """Against float64; k0, v0: the caches before.  wrote / turned: masks of the tokens."""
        x = self.qkv.double()
        T, Hq, Hkv, half = self.T, self.Hq, self.Hkv, self.rot // 2
        every = torch.ones(T, dtype=torch.bool, device=DEV)
        wrote, turned = every if wrote is None else wrote, every if turned is None else turned
        c = self.cos_sin.double()[self.positions.clamp(0, self.cos_sin.shape[0] - 1)][:, None]
        want, size = x.clone(), torch.zeros_like(x)
        i = torch.arange(half, device=DEV)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        n = Hq + Hkv
        xa, xb = x[:, :n, a], x[:, :n, b]
        want[:, :n, a] = xa * c[..., :half] - xb * c[..., half:]
        want[:, :n, b] = xb * c[..., :half] + xa * c[..., half:]
        size[:, :n, a] = size[:, :n, b] = 3 * 2.0 ** -24 * (xa.abs() + xb.abs())
        eps = torch.finfo(TYPES[self.src]).eps / 2

        got = self.q_out.double()
        tol = eps * want[:, :Hq].abs() + size[:, :Hq] * (1 + eps) + TINY[self.src]
        assert bool(((got - want[:, :Hq]).abs() <= tol)[turned].all())
        assert bool((got[:, :, self.rot:] == x[:, :Hq, self.rot:])[turned].all())       # bits past the rotated part
        assert bool((got[~turned] == 3.0).all())

        for cache, before, scale, w, z in ((self.kc, k0, self.ks, want[:, Hq:n], size[:, Hq:n]),
                                           (self.vc, v0, self.vs, want[:, n:], size[:, n:])):
            flat, was = (t.transpose(1, 2).reshape(-1, Hkv, 128) for t in (cache, before))
            at = self.slots[wrote]
            rows = flat[at]
            w, z = w[wrote], z[wrote]
            if scale is None:
                assert bool(((rows.double() - w).abs() <= eps * w.abs() + z * (1 + eps) + TINY[self.src]).all())
            else:
                s = scale.double().view(1, -1, 1)
                w, z = (w / s).clamp(-448, 448), z / s + 2.0 ** -24 * (w / s).abs()
                code = rows.view(torch.float8_e4m3fn).double()
                assert bool(((code - w).abs() <= 2.0 ** -4 * (w.abs() + z) + z + 2.0 ** -10).all())
            rest = torch.ones(flat.shape[0], dtype=torch.bool, device=DEV)
            rest[at] = False
            assert torch.equal(flat[rest], was[rest])                # nothing else is touched


@pytest.mark.parametrize("src,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8"), ("fp16", "fp8 heads")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,rot,bs", [(1, 8, 2, 128, 16), (1, 1, 1, 16, 8), (3, 12, 2, 64, 32), (33, 5, 5, 48, 8),
                                             (130, 64, 8, 128, 16), (1000, 32, 8, 112, 16), (4097, 12, 2, 96, 32)])
def test_rotation_and_slot_write(src, cache, interleaved, T, Hq, Hkv, rot, bs):
    c = Case(T + rot, T, Hq, Hkv, rot, src, cache, bs)
    k0, v0 = c.kc.clone(), c.vc.clone()
    c.call(interleaved)
    c.check(interleaved, k0, v0)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_values_and_unrotated_rows_equal_the_plain_slot_write(cache):
    # v, and at position 0 (cosine 1, sine 0) k too, are what pa_reshape_and_cache stores, bit
    # for bit, infinities and NaN included
    c = Case(5, 300, 8, 2, 64, "bf16", cache, 16)
    c.positions.zero_()
    bits = c.qkv.view(torch.int16)
    bits[3, 10:, 7] = NAN_BITS
    bits[4, 10:, 70] = 0x7F80
    bits[5, 8:10, 100] = -0x80                   # -inf, past the rotated part of k
    bits[6, 10:, 0] = -0x8000                    # -0
    k0, v0 = c.kc.clone(), c.vc.clone()
    c.call(False)
    q, k, v = c.parts()
    pa.pa_reshape_and_cache(k.contiguous(), v.contiguous(), k0, v0, c.slots, c.ks, c.vs)
    as_bits = (lambda t: t) if cache == "fp8" else (lambda t: t.view(torch.int16))
    assert torch.equal(as_bits(c.vc), as_bits(v0))
    assert torch.equal(as_bits(c.kc), as_bits(k0))


def test_padding_and_places_out_of_range():
    c = Case(6, 200, 8, 2, 128, "bf16", "bf16", 16)
    free = c.slots.clone()
    wrote = torch.ones(200, dtype=torch.bool, device=DEV)
    turned = wrote.clone()
    c.positions[7] = -1                          # padding: nothing
    c.positions[8] = c.cos_sin.shape[0]          # beyond the table: recorded, nothing
    c.slots[9] = -5                              # no slot: q alone
    c.slots[10] = c.kc.shape[0] * 16             # beyond the pool: recorded, q alone
    c.slots[11] = 1 << 40
    turned[7] = turned[8] = False
    wrote[7:12] = False
    k0, v0 = c.kc.clone(), c.vc.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    c.call(False, workspace=ws)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_OUT_OF_RANGE
    c.check(False, k0, v0, wrote, turned)
    c.slots.copy_(free)
    c.positions[7:9] = 0
    c.call(False, workspace=ws)
    assert pa.pa_read_device_status(ws) == pa.PA_OK


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(interleaved):
    c = Case(7, 70, 12, 2, 80, "bf16", "bf16", 16)
    q, k, v = c.parts()
    kc, vc = c.kc.clone(), c.vc.clone()
    c.call(interleaved)
    pa.pa_rope_and_cache(q, q, k, v, kc, vc, c.slots, c.positions, c.cos_sin, interleaved=interleaved)
    assert torch.equal(q, c.q_out) and torch.equal(kc, c.kc)


def test_graph_replay_and_another_stream():
    c = Case(8, 40, 8, 2, 128, "bf16", "fp8", 16)
    c.call(True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.call(True)
    new = Case(9, 40, 8, 2, 128, "bf16", "fp8", 16)
    for name in ("qkv", "positions"):
        getattr(c, name).copy_(getattr(new, name))
    k0, v0 = c.kc.clone(), c.vc.clone()
    c.q_out.fill_(3.0)
    g.replay()
    torch.cuda.synchronize()
    c.check(True, k0, v0)
    k0, v0 = c.kc.clone(), c.vc.clone()
    torch.cuda.synchronize()
    c.q_out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        c.call(False)
    torch.cuda.synchronize()
    c.check(False, k0, v0)


def test_no_tokens_and_one_token_of_any_stride():
    c = Case(11, 5, 8, 2, 64, "bf16", "bf16", 16)
    q, k, v = c.parts()
    k0, v0 = c.kc.clone(), c.vc.clone()
    args = (c.kc, c.vc, c.slots[:0], c.positions[:0], c.cos_sin)
    pa.pa_rope_and_cache(c.q_out[:0], q[:0], k[:0], v[:0], *args)
    assert torch.equal(c.kc, k0) and torch.equal(c.vc, v0) and bool((c.q_out == 3.0).all())
    # a single token: its stride means nothing, an odd one included
    one = torch.empty(4096, dtype=torch.bfloat16, device=DEV)
    views = [one[i:i + h * 128].as_strided((1, h, 128), (7, 128, 1)) for i, h in ((0, 8), (1024, 2), (1280, 2))]
    for view, part in zip(views, (q, k, v)):
        view.copy_(part[3:4])
    pa.pa_rope_and_cache(c.q_out[:1], *views, c.kc, c.vc, c.slots[3:4], c.positions[3:4], c.cos_sin)
    got = c.q_out[0].clone()
    pa.pa_rope_and_cache(c.q_out, q, k, v, k0, v0, c.slots, c.positions, c.cos_sin)
    assert torch.equal(got, c.q_out[3])
    at = int(c.slots[3])
    assert torch.equal(c.kc[at // 16, :, at % 16], k0[at // 16, :, at % 16])


def test_the_tensors_device_is_made_current(monkeypatch):
    # as if device 1 were the current one: device 0 is set for the call, and 1 again behind it
    c = Case(12, 40, 8, 2, 128, "bf16", "bf16", 16)
    k0, v0 = c.kc.clone(), c.vc.clone()
    torch.cuda.synchronize()
    seen = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_setDevice", seen.append)
    c.call(True)
    monkeypatch.undo()
    assert seen == [0, 1]
    c.check(True, k0, v0)


def test_refusals():
    c = Case(10, 6, 8, 2, 64, "bf16", "fp8", 16)
    q, k, v = c.parts()
    args = lambda **kw: {**dict(q_out=c.q_out, q=q, k=k, v=v, k_cache=c.kc, v_cache=c.vc, slot_mapping=c.slots,  # noqa: E731
                                positions=c.positions, cos_sin=c.cos_sin, k_scale=c.ks, v_scale=c.vs), **kw}
    for bad in (dict(positions=c.positions[:-1]), dict(slot_mapping=c.slots[1:]), dict(k=k[:, :1]), dict(q_out=c.q_out[:-1]),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(k_scale=c.ks.repeat(3)),
                dict(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)), dict(positions=c.positions.cpu()),
                dict(positions=None), dict(v_cache=None)):
        with pytest.raises((ValueError, TypeError)):
            pa.pa_rope_and_cache(**args(**bad))
    for bad in (dict(positions=c.positions.int()), dict(q_out=c.q_out.half()), dict(k_scale=None, v_scale=None),
                dict(cos_sin=c.cos_sin.double())):
        with pytest.raises((TypeError, pa.PagedAttentionError)):
            pa.pa_rope_and_cache(**args(**bad))
    f = pa.pa_rope_frequencies(64)
    for table, freqs in ((c.cos_sin, f[:-1]), (c.cos_sin, f.reshape(2, -1)), (c.cos_sin[:, ::2], f[:16]), (c.cos_sin[0], f)):
        with pytest.raises(ValueError):
            pa.pa_rope_table(table, freqs)
    for table in (c.cos_sin.half(), c.cos_sin.cpu(), None):
        with pytest.raises(TypeError):
            pa.pa_rope_table(table, f)
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_rope_table(c.cos_sin, f * float("inf"))
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_rope_and_cache(**args(cos_sin=c.cos_sin[:, :40].contiguous()))      # 40 components: not a multiple of 16
