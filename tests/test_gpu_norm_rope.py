"""pa_norm_rope_and_cache on the GPU against float64 norms and rotations of the same table.

Tolerance.  A normed component: the sum of 128 squares in float32 is off by at most 128 x
2^-24 of itself, half of that in its root; mean, eps, root (2^-22) and the products by it and
by the weight a few times 2^-24: 2^-16 of the component covers them (s below).  The rotation
adds the pair's two products and their sum, 2^-23 each of |a| + |b|.  Then half a step of the
type stored (finfo.eps / 2 of the value, half the smallest subnormal below the normal range)."""
import pytest
import torch

import paged_kv_cache_99_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Case:
    def __init__(self, seed, T, hq, hkv, rot, kind="bf16", cache="bf16", bs=16, axes=None, context=600, per_head=False):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.T, self.hq, self.hkv, self.rot, self.kind, self.cache, self.bs = T, hq, hkv, rot, kind, cache, bs
        self.qkv = torch.randn(T, hq + 2 * hkv, 128, generator=g, device=DEV)
        self.qkv[:, :hq + hkv] *= torch.exp(2 * torch.randn(T, hq + hkv, 1, generator=g, device=DEV))
        self.qkv = self.qkv.to(TYPES[kind])
        self.wq, self.wk = ((1 + 0.5 * torch.randn(128, generator=g, device=DEV)).to(TYPES[kind]) for _ in range(2))
        n = 1 if axes is None else max(axes) + 1
        self.axes = axes
        self.pos = torch.randint(0, context, (n, T), generator=g, device=DEV)
        f = 10000.0 ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)
        angle = torch.arange(context, device=DEV, dtype=torch.float64)[:, None] * f
        self.table = torch.cat((angle.cos(), angle.sin()), 1).float()
        pool = -(-T // bs) + 3
        self.slots = torch.randperm(pool * bs, generator=g, device=DEV)[:T]
        dt = torch.uint8 if cache == "fp8" else TYPES[cache]
        self.kc, self.vc = (torch.randint(0, 100, (pool, hkv, bs, 128), generator=g, device=DEV).to(dt) for _ in range(2))
        self.ks = self.vs = None
        if cache == "fp8":
            k = hkv if per_head else 1
            self.ks, self.vs = (0.02 + 0.02 * torch.rand(k, generator=g, device=DEV) for _ in range(2))

    def parts(self):
        return self.qkv[:, :self.hq], self.qkv[:, self.hq:self.hq + self.hkv], self.qkv[:, self.hq + self.hkv:]

    def run(self, q_out=None, wq=True, wk=True, **kw):
        q_out = torch.full((self.T, self.hq, 128), 5.0, device=DEV, dtype=self.qkv.dtype) if q_out is None else q_out
        q, k, v = self.parts()
        pa.pa_norm_rope_and_cache(q_out, q, k, v, self.kc, self.vc, self.slots, kw.pop("positions", self.pos), self.table,
                                  self.wq if wq else None, self.wk if wk else None,
                                  axes=bytes(self.axes) if self.axes is not None else None, k_scale=self.ks,
                                  v_scale=self.vs, **kw)
        return q_out

    def turned(self, x, weight, eps, offset, interleaved):
        """(values, error before the last rounding), float64."""
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * (weight.double() + offset)
            e = 2.0 ** -16 * x.abs()
        else:
            e = torch.zeros_like(x)
        half = self.rot // 2
        axes = self.axes or [0] * half
        out, err = x.clone(), e.clone()
        for i in range(half):
            row = self.table[self.pos[axes[i]]].double()
            c, s = row[:, None, i], row[:, None, half + i]
            one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            a, b = x[..., one], x[..., two]
            out[..., one], out[..., two] = a * c - b * s, b * c + a * s
            r = (e[..., one] + e[..., two]) + 3 * 2.0 ** -23 * (a.abs() + b.abs())
            err[..., one] = err[..., two] = r
        return out, err

    def check(self, q_out, before, eps=1e-6, offset=0.0, interleaved=False, wq=True, wk=True):
        u, tiny = torch.finfo(self.qkv.dtype).eps / 2, 2.0 ** -25 if self.kind == "fp16" else 0.0
        q, k, v = self.parts()
        want, err = self.turned(q, self.wq if wq else None, eps, offset, interleaved)
        off = (q_out.double() - want).abs()
        assert bool((off <= err + u * (want.abs() + err) + tiny).all()), float((off - err - u * want.abs()).max())
        want, err = self.turned(k, self.wk if wk else None, eps, offset, interleaved)
        for cache, old, scale, (val, er) in ((self.kc, before[0], self.ks, (want, err)),
                                             (self.vc, before[1], self.vs, (v.double(), torch.zeros_like(v.double())))):
            rows = cache[self.slots // self.bs, :, self.slots % self.bs]
            if scale is None:
                assert bool(((rows.double() - val).abs() <= er + u * (val.abs() + er) + tiny).all())
            else:
                z = scale.double().view(1, -1, 1)
                y, ye = (val / z), er / z + 2.0 ** -23 * (val / z).abs()
                lim = y.clamp(-448, 448)
                got = rows.view(torch.float8_e4m3fn).double()
                assert bool(((got - lim).abs() <= ye + 2.0 ** -4 * (lim.abs() + ye) + 2.0 ** -10).all())
            # nothing else is written
            keep = torch.ones(cache.shape[0] * self.bs, dtype=torch.bool, device=DEV)
            keep[self.slots[self.slots >= 0]] = False
            flat, was = (c.transpose(1, 2).reshape(-1, self.hkv, 128) for c in (cache, old))
            assert torch.equal(flat[keep], was[keep])


def go(c, **kw):
    before = c.kc.clone(), c.vc.clone()
    names = {k: kw[k] for k in ("eps", "interleaved", "wq", "wk") if k in kw}
    if "weight_offset" in kw:
        names["offset"] = kw["weight_offset"]
    q = c.run(**kw)
    c.check(q, before, **names)


@pytest.mark.parametrize("kind,cache,per_head", [("bf16", "bf16", False), ("fp16", "fp16", False), ("bf16", "fp8", False),
                                                 ("fp16", "fp8", True)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 48, 64, 112, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_norm_and_rotation(kind, cache, per_head, interleaved, rot, bs):
    go(Case(rot + bs, 37, 6, 2, rot, kind, cache, bs, per_head=per_head), interleaved=interleaved)


@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 2), (2, 1, 1), (300, 40, 5), (1100, 64, 8), (5000, 32, 8)])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_sizes(T, hq, hkv, cache):
    go(Case(T, T, hq, hkv, 128, "bf16", cache, axes=pa.rope_axes((24, 20, 20), in_turns=True)), weight_offset=1.0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections,rot", [((16, 24, 24), 128), ((5, 3, 0, 24), 64), ((0, 8), 16), ((1, 2, 3, 2), 16),
                                          ((40, 16), 112)])
@pytest.mark.parametrize("in_turns", [False, True])
def test_axes(interleaved, sections, rot, in_turns):
    axes = pa.rope_axes(sections, in_turns)
    assert len(axes) == rot // 2 and [axes.count(a) for a in range(len(sections))] == list(sections)
    go(Case(7, 65, 8, 2, rot, axes=list(axes)), interleaved=interleaved)


def test_without_weights():
    axes = list(pa.rope_axes((16, 24, 24)))
    go(Case(1, 50, 4, 2, 128, axes=axes), wq=False)
    go(Case(2, 50, 4, 2, 128, axes=axes), wk=False)
    c = Case(3, 50, 4, 2, 96)
    before = c.kc.clone(), c.vc.clone()
    q = c.run(wq=False, wk=False)
    c.check(q, before, wq=False, wk=False)
    # one axis and no norm: pa_rope_and_cache, bit for bit
    d = Case(3, 50, 4, 2, 96)
    q2 = torch.empty_like(q)
    qq, k, v = d.parts()
    pa.pa_rope_and_cache(q2, qq, k, v, d.kc, d.vc, d.slots, d.pos[0].contiguous(), d.table)
    assert torch.equal(q, q2) and torch.equal(c.kc, d.kc) and torch.equal(c.vc, d.vc)


def test_in_place_and_eps():
    c = Case(4, 40, 8, 2, 128)
    ref = c.run(eps=0.5)
    d = Case(4, 40, 8, 2, 128)
    keep = d.qkv.clone()
    d.run(q_out=d.qkv[:, :8], eps=0.5)
    assert torch.equal(d.qkv[:, :8], ref) and torch.equal(d.qkv[:, 8:], keep[:, 8:])
    assert torch.equal(c.kc, d.kc)
    c.qkv[3] = 0                                    # an all-zero head stays zero
    assert bool((c.run()[3] == 0).all())


def test_padding_and_positions_out_of_range():
    c = Case(5, 20, 8, 2, 128, axes=list(pa.rope_axes((16, 24, 24))))
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    before = c.kc.clone(), c.vc.clone()
    c.pos[1, 4] = -1                                # one axis negative: padding
    c.pos[2, 7] = 600                               # beyond the table
    c.slots[9] = -1                                 # no slot: q alone
    c.slots[11] = c.kc.shape[0] * c.bs              # beyond the pool
    q = c.run(workspace=ws)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_OUT_OF_RANGE
    assert bool((q[[4, 7]] == 5.0).all())
    ok = [i for i in range(20) if i not in (4, 7)]
    c.pos[:, [4, 7]] = 0
    want, err = c.turned(c.parts()[0], c.wq, 1e-6, 0.0, False)
    assert bool(((q.double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err))[ok].all())
    written = [i for i in ok if i not in (9, 11)]
    keep = torch.ones(c.kc.shape[0] * c.bs, dtype=torch.bool, device=DEV)
    keep[c.slots[written]] = False
    for cache, old in zip((c.kc, c.vc), before):
        flat, was = (x.transpose(1, 2).reshape(-1, 2, 128) for x in (cache, old))
        assert torch.equal(flat[keep], was[keep]) and not torch.equal(flat, was)


def test_captured():
    c = Case(6, 9, 8, 2, 128, axes=list(pa.rope_axes((16, 24, 24))))
    ref = c.run()
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(q_out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


@pytest.mark.parametrize("kind,cache,per_head", [("bf16", "bf16", False), ("fp16", "fp16", False), ("bf16", "fp8", False),
                                                 ("fp16", "fp8", True)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_tokens(kind, cache, per_head, interleaved):
    """More tokens than every SM has a few of: rotations of part of a head and several axes."""
    for T, hq, hkv, rot, sections in ((3001, 28, 4, 128, (24, 20, 20)), (9000, 8, 2, 64, (5, 3, 0, 24)), (2500, 40, 8, 112, None)):
        axes = pa.rope_axes(sections, in_turns=True) if sections else None
        go(Case(T, T, hq, hkv, rot, kind, cache, axes=axes, per_head=per_head), interleaved=interleaved)


def test_many_tokens_with_padding():
    c = Case(8, 4000, 28, 4, 128, axes=list(pa.rope_axes((16, 24, 24))))
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    pad = torch.rand(4000, generator=g, device=DEV) < 0.1
    far = torch.rand(4000, generator=g, device=DEV) < 0.05
    none = torch.rand(4000, generator=g, device=DEV) < 0.1
    c.pos[1, pad] = -1
    c.pos[2, far & ~pad] = 600
    c.slots[none] = -1
    q = c.run(workspace=ws)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_OUT_OF_RANGE
    skipped = pad | far
    assert bool((q[skipped] == 5.0).all())
    c.pos[:, skipped] = 0
    want, err = c.turned(c.parts()[0], c.wq, 1e-6, 0.0, False)
    assert bool(((q.double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err))[~skipped].all())
    want, err = c.turned(c.parts()[1], c.wk, 1e-6, 0.0, False)
    live = ~skipped & ~none
    rows = c.kc[c.slots[live] // c.bs, :, c.slots[live] % c.bs].double()
    assert bool(((rows - want[live]).abs() <= err[live] + 2.0 ** -8 * (want[live].abs() + err[live])).all())


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_stored_values_are_those_of_the_slot_write(kind):
    """V in an FP8 cache: the codes that pa_reshape_and_cache writes, bit for bit, NaNs and
    infinities, zeros of both signs and scales of any size among them."""
    T, hq, hkv = 5000, 12, 2
    g = torch.Generator(device=DEV).manual_seed(9)
    bits = torch.randint(-32768, 32768, (T, hq + 2 * hkv, 128), generator=g, device=DEV, dtype=torch.int16)
    qkv = bits.view(TYPES[kind])
    slots = torch.randperm(5008, generator=g, device=DEV)[:T]
    table = torch.ones(16, 128, device=DEV)
    for scale in (1.0, 0.013, 3e-3, 2.0 ** -70, 1e-38, 2.0 ** 66):
        ks = torch.full((1,), scale, device=DEV)
        kc, vc, k2, v2 = (torch.zeros(313, hkv, 16, 128, dtype=torch.uint8, device=DEV) for _ in range(4))
        q = torch.empty(T, hq, 128, dtype=qkv.dtype, device=DEV)
        for t in (T, 40):
            pa.pa_norm_rope_and_cache(q[:t], qkv[:t, :hq], qkv[:t, hq:hq + hkv], qkv[:t, hq + hkv:], kc, vc, slots[:t],
                                      torch.zeros(t, dtype=torch.int64, device=DEV), table, k_scale=ks, v_scale=ks)
            v = qkv[:t, hq + hkv:].contiguous()
            pa.pa_reshape_and_cache(v, v, k2, v2, slots[:t].contiguous(), ks, ks)
            assert torch.equal(vc, v2), scale


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8")])
def test_more_tokens_than_l2_holds(kind, cache):
    # 8,000 x 48 rows of 512 bytes in and out; every thirteenth token has no slot, some of them another
    # negative number than -1: q is written all the same
    c = Case(21, 8000, 32, 8, 128, kind, cache, axes=pa.rope_axes((24, 20, 20)))
    keep = torch.ones(8000, dtype=torch.bool, device=DEV)
    keep[::13] = False
    before = c.kc.clone(), c.vc.clone()
    slots = c.slots.clone()
    c.slots[::13] = -torch.arange(1, len(c.slots[::13]) + 1, device=DEV)
    q = c.run()
    for cache_, old in zip((c.kc, c.vc), before):
        lost = slots[~keep]
        assert torch.equal(cache_[lost // c.bs, :, lost % c.bs], old[lost // c.bs, :, lost % c.bs])
    want, err = c.turned(c.parts()[0], c.wq, 1e-6, 0.0, False)
    u = torch.finfo(c.qkv.dtype).eps / 2
    assert bool(((q.double() - want).abs() <= err + u * (want.abs() + err) + (2.0 ** -25 if kind == "fp16" else 0.0)).all())
    c.slots, c.qkv, c.pos, c.T = c.slots[keep], c.qkv[keep], c.pos[:, keep], int(keep.sum())
    c.check(q[keep], before)
