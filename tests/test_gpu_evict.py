"""pa_evict on the GPU against a plain selection and copy on the host.  Everything it
returns is whole numbers or copied bits, so everything has to be equal."""
import numpy as np
import pytest
import torch

import paged_kv_cache_99_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.uint8}


class Case:
    def __init__(self, seed, lens, Hkv, cache, bs, budget, sinks=0, recent=0, weights=None, extra=0, shared=0):
        g = np.random.default_rng(seed)
        self.lens, self.Hkv, self.bs, self.budget, self.sinks, self.recent = lens, Hkv, bs, budget, sinks, recent
        blocks = [-(-n // bs) for n in lens]
        new = [-(-min(n, budget) // bs) for n in lens]
        self.nb = sum(blocks) + sum(new) + 3
        perm = g.permutation(self.nb)
        self.tables = np.full((len(lens), max(blocks) + 1), -1, np.int32)
        self.new = np.full((len(lens), max(new) + 1), -1, np.int32)
        at = 0
        for s, b in enumerate(blocks):
            self.tables[s, :b] = perm[at:at + b]
            at += b
        if shared:                                   # every sequence starts with the first one's blocks
            for s, b in enumerate(blocks):
                self.tables[s, :min(b, shared)] = self.tables[0, :min(b, shared)]
        for s, b in enumerate(new):
            self.new[s, :b] = perm[at:at + b]
            at += b
        shape = (self.nb, Hkv, bs, 128)
        bits = g.integers(0, 256 if cache == "fp8" else 65536, shape)        # NaN patterns among them
        self.k, self.v = (bits.astype(np.uint8 if cache == "fp8" else np.uint16),
                          (bits[::-1] ^ 0x55).astype(np.uint8 if cache == "fp8" else np.uint16))
        self.cache = cache
        self.stride = self.tables.shape[1] * bs + 4 * extra
        w = np.exp(2 * g.standard_normal((len(lens), Hkv, self.stride)) - 6).astype(np.float32)
        w[g.random(w.shape) < 0.15] = 0
        if weights is not None:
            w = weights(g, w)
        self.w = w.astype(np.float32)

    def device(self):
        as_cache = lambda x: torch.from_numpy(x.view(np.int16) if x.dtype == np.uint16 else x).to(DEV).view(TYPES[self.cache])  # noqa: E731
        self.kc, self.vc = as_cache(self.k), as_cache(self.v)
        self.dw = torch.from_numpy(self.w).to(DEV)
        self.wout = torch.full_like(self.dw, 7.0)
        self.kept = torch.full((len(self.lens), self.Hkv, self.budget), -9, dtype=torch.int32, device=DEV)
        self.lens_out = torch.full((len(self.lens),), -9, dtype=torch.int32, device=DEV)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.dt, self.dn = torch.from_numpy(self.tables).to(DEV), torch.from_numpy(self.new).to(DEV)
        return self

    def call(self, wout=None, **kw):
        pa.pa_evict(self.kept, self.lens_out, self.wout if wout is None else wout, self.dw, self.kc, self.vc, self.dt,
                    self.dlens, self.dn, self.budget, self.sinks, self.recent, **kw)

    def expect(self):
        k, v = self.k.copy(), self.v.copy()
        kept = np.full((len(self.lens), self.Hkv, self.budget), -1, np.int32)
        wout = np.full_like(self.w, 7.0)
        for s, n in enumerate(self.lens):
            m = min(n, self.budget)
            for h in range(self.Hkv):
                t = np.arange(n)
                x = self.w[s, h, :n].astype(np.float64)
                nan = np.isnan(x)
                x = np.where(nan, 0.0, x)
                sure = (t < self.sinks) | (t >= n - self.recent)
                pick = np.sort(np.lexsort((t, -x, nan, ~sure))[:m])
                kept[s, h, :m] = pick
                wout[s, h, :n] = 0
                wout[s, h, :m] = self.w[s, h, pick]
                src, dst = self.tables[s][pick // self.bs], self.new[s][np.arange(m) // self.bs]
                k[dst, h, np.arange(m) % self.bs] = self.k[src, h, pick % self.bs]
                v[dst, h, np.arange(m) % self.bs] = self.v[src, h, pick % self.bs]
        return kept, wout, k, v

    def check(self, wout=None, in_place=False):
        kept, want, k, v = self.expect()
        assert np.array_equal(self.kept.cpu().numpy(), kept)
        assert self.lens_out.tolist() == [min(n, self.budget) for n in self.lens]
        got = (self.wout if wout is None else wout).cpu().numpy()
        if in_place:
            for s, n in enumerate(self.lens):
                want[s, :, n:] = self.w[s, :, n:]
        np.testing.assert_array_equal(got, want)             # NaN where NaN, -0 as 0
        as_bits = lambda x: x.cpu().numpy() if self.cache == "fp8" else x.cpu().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
        assert np.array_equal(as_bits(self.kc), k) and np.array_equal(as_bits(self.vc), v)


LENS = [0, 1, 7, 16, 63, 64, 65, 66, 200, 777, 2500]


@pytest.mark.parametrize("cache", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("budget,sinks,recent", [(64, 4, 16), (65, 0, 0), (1, 0, 0), (1, 0, 1), (33, 33, 0), (40, 10, 30),
                                                 (777, 3, 700), (5000, 4, 4)])
def test_selection_and_copy(cache, bs, budget, sinks, recent):
    c = Case(budget + bs, LENS, 3, cache, bs, budget, sinks, recent, extra=bs % 3).device()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    c.call(workspace=ws)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    c.check()


def _all_equal(g, w):
    return np.full_like(w, 0.25)


def _few_values(g, w):
    return g.integers(0, 3, w.shape) * 0.5


def _odd_values(g, w):
    vals = np.array([np.inf, -np.inf, np.nan, -np.nan, 0.0, -0.0, 1.0, -1.0, 1e-45, -1e-45, 3.4e38, -3.4e38], np.float32)
    return vals[g.integers(0, len(vals), w.shape)]


def _close_values(g, w):
    # neighbours in the last bits: the last pass decides
    return (np.float32(1.0).view(np.int32) + g.integers(0, 5000, w.shape)).astype(np.int32).view(np.float32)


@pytest.mark.parametrize("weights", [_all_equal, _few_values, _odd_values, _close_values])
@pytest.mark.parametrize("budget,sinks,recent", [(64, 4, 16), (500, 0, 0), (1000, 0, 999)])
def test_ties_and_odd_weights(weights, budget, sinks, recent):
    c = Case(3, LENS + [5000], 2, "fp8", 16, budget, sinks, recent, weights=weights).device()
    c.call()
    c.check()


@pytest.mark.parametrize("lens,budget", [([20000], 3000), ([20000, 9], 4096), ([60000, 30000], 777), ([130000], 16384), ([390000], 5000)])
@pytest.mark.parametrize("weights", [None, _few_values])
def test_long_rows_over_several_ctas(lens, budget, weights):
    c = Case(11, lens, 2, "fp8", 16, budget, 4, 256, weights=weights).device()
    c.call()
    c.check()
    c.call(wout=c.dw)              # the source blocks are as they were: the same again, compacted in place
    c.check(wout=c.dw, in_place=True)


@pytest.mark.parametrize("weights", [None, _odd_values])
def test_in_place(weights):
    c = Case(12, LENS, 2, "bf16", 16, 50, 4, 10, weights=weights, extra=2).device()
    c.call(wout=c.dw)
    c.check(wout=c.dw, in_place=True)


def test_many_long_rows():
    # more CTAs than SMs, each with more keys than shared memory holds without asking
    c = Case(19, [100000] * 20, 1, "fp8", 32, 300, 4, 64).device()
    c.call(wout=c.dw)
    c.check(wout=c.dw, in_place=True)


def test_a_row_too_long_to_stage():
    c = Case(13, [400000], 1, "fp8", 32, 1000, 4, 64, weights=_few_values).device()
    with pytest.raises(pa.PagedAttentionError):
        c.call(wout=c.dw)
    c.call()
    c.check()


def test_shared_source_blocks():
    c = Case(14, [300, 280, 310, 64], 2, "bf16", 16, 90, 4, 16, shared=12).device()
    c.call()
    c.check()


def test_blocks_out_of_range_and_lengths_beyond_the_table():
    c = Case(15, [100, 100, 100], 2, "fp16", 16, 40, 0, 0).device()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    c.call(workspace=ws)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    base_k = c.kc.clone()
    c.dn[1, 1] = c.nb                            # the second new block of sequence 1: not copied
    c.kc.copy_(torch.from_numpy(c.k.view(np.int16)).to(DEV).view(torch.float16))
    c.call(workspace=ws)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_OUT_OF_RANGE
    skipped = int(c.new[1, 1])
    want = base_k.view(torch.int16).clone()
    want[skipped] = torch.from_numpy(c.k[skipped].view(np.int16)).to(DEV)
    assert torch.equal(c.kc.view(torch.int16), want)
    c.dn.copy_(torch.from_numpy(c.new).to(DEV))
    c.dt[2, 0] = -7                              # a source block: read from block 0 instead
    c.call(workspace=ws)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_OUT_OF_RANGE
    c.dt.copy_(torch.from_numpy(c.tables).to(DEV))
    c.dlens[0] = c.tables.shape[1] * 16 + 1      # beyond the table (whose last entry is -1): cut to it
    c.call(workspace=ws)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_OUT_OF_RANGE
    assert c.lens_out.tolist() == [40, 40, 40] and int(c.kept.max()) < c.tables.shape[1] * 16


def test_graph_replay_and_another_stream():
    c = Case(16, LENS, 2, "bf16", 16, 60, 4, 16).device()
    c.call()
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c.call()
    d = Case(17, LENS, 2, "bf16", 16, 60, 4, 16).device()
    # other weights and values in the captured buffers, the first case's tables
    d.tables, d.new = c.tables, c.new
    for name in ("dw", "kc", "vc"):
        getattr(c, name).copy_(getattr(d, name))
    c.wout.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    c.w, c.k, c.v = d.w, d.k, d.v
    c.check()
    c.kc.copy_(d.kc)
    c.vc.copy_(d.vc)
    c.wout.fill_(7.0)
    c.kept.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        c.call()
    torch.cuda.synchronize()
    c.check()


def test_no_sequences_and_refusals():
    c = Case(18, [30, 40], 2, "bf16", 16, 16).device()
    e = lambda t: t[:0]  # noqa: E731
    pa.pa_evict(e(c.kept), e(c.lens_out), e(c.wout), e(c.dw), c.kc, c.vc, e(c.dt), e(c.dlens), e(c.dn), 16)
    args = lambda **kw: {**dict(kept=c.kept, seq_lens_out=c.lens_out, weights_out=c.wout, weights=c.dw, k_cache=c.kc,  # noqa: E731
                                v_cache=c.vc, block_tables=c.dt, seq_lens=c.dlens, new_tables=c.dn, budget=16), **kw}
    for bad in (dict(budget=17), dict(kept=c.kept[:1]), dict(weights_out=c.wout[..., :-4].contiguous()),
                dict(weights=c.dw.transpose(0, 1)), dict(seq_lens=c.dlens.long()), dict(v_cache=c.vc.half()),
                dict(new_tables=c.dn.cpu())):
        with pytest.raises((ValueError, TypeError)):
            pa.pa_evict(**args(**bad))
    for bad in (dict(seq_lens_out=c.dlens), dict(sinks=10, recent=7), dict(new_tables=c.dn[:, :0].contiguous())):
        with pytest.raises(pa.PagedAttentionError):
            pa.pa_evict(**args(**bad))
