"""pa_decode_weights on the GPU against float64 softmax weights.

Tolerance.  A score is a float32 sum of 128 exact products in some order: off by at
most 128 x 2^-23 x the sum of their magnitudes (2^-23 for sums that truncate), times the
softmax scale; the scale's and the FP8 scale's products add 2^-21 of the score, an FP8
cache's query, rounded to fp16, 2^-25 per component below fp16's normal range.  With
every score of a row within e of the exact one a weight is within a factor exp(2 e);
the exponential, the sum and the reciprocal add 2^-20.  The sum over the group and the
running weight round to 2^-24 of what they add up to, a few times."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_99_gb300 as pa
from paged_kv_cache_99_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
LENS = [0, 1, 2, 15, 16, 17, 33, 100, 128, 513, 1200, 4000]


def _case(seed, G, cache="bf16", qd="bf16", bs=16, Hkv=2, fp8_scale="tensor", lens=LENS):
    w = W.build_workload(name="weights", seed=seed, device=DEV, num_layers=1, seq_lens=lens, q_lens=[1] * len(lens),
                         num_q_heads=G * Hkv, num_kv_heads=Hkv, q_dtype=qd, cache_dtype=cache, block_size=bs,
                         fp8_scale=fp8_scale, write_new=False)
    return w


def _args(w):
    return dict(k_scale=w.k_scale[0].reshape(-1) if w.k_scale is not None else None,
                v_scale=w.v_scale[0].reshape(-1) if w.v_scale is not None else None)


def _tokens(w):
    return int((((w.seq_lens + 15) // 16) * 16).sum())


def _workspace(w, spare=0):
    return pa.new_workspace_weights(w.num_seqs, w.num_q_heads, w.num_kv_heads, _tokens(w) + spare)


def _stride(w):
    return w.max_blocks_per_seq * w.block_size


def _call(w, ws, wout, win=None, out=None, q=None):
    out = torch.empty_like(w.q[0]) if out is None else out
    pa.pa_decode_weights(out, wout, w.q[0] if q is None else q, w.k_cache[0], w.v_cache[0], w.block_tables, w.seq_lens,
                         w.scale, ws, weights_in=win, **_args(w))
    return out


def _reference(w, seqs):
    """{sequence: (weights [H_kv, n], tolerance [H_kv, n])} in float64."""
    ref = {}
    G, bs = w.num_q_heads // w.num_kv_heads, w.block_size
    fp8 = w.cache_dtype == "fp8"
    for s in seqs:
        n = int(w.seq_lens[s])
        t = torch.arange(n, device=DEV)
        block = w.block_tables[s].long()[t // bs]
        k = w.k_cache[0][block, :, t % bs]
        k = k.view(torch.float8_e4m3fn).double() * w.k_scale[0].double().reshape(1, -1, 1) if fp8 else k.double()
        q = w.q[0][s].double().view(w.num_kv_heads, G, 128)
        x = torch.einsum("hgd,nhd->hgn", q, k) * w.scale
        size = torch.einsum("hgd,nhd->hgn", q.abs(), k.abs()) * w.scale
        e = 128 * 2.0 ** -23 * size + 2.0 ** -21 * x.abs()
        if fp8:
            e = e + 2.0 ** -25 * k.abs().sum(-1).T[:, None] * w.scale
        p = torch.softmax(x, -1)
        off = 2 * e.amax(-1, keepdim=True) + 2.0 ** -20 if n else e
        assert not n or float(off.max()) < 0.01
        ref[s] = (p.sum(1), (p * off * 1.01).sum(1))
    return ref


def _check(w, got, before, ref, base=None, steps=1):
    """got: weights_out; before: its content before the call; base: what was added to."""
    for s, (p, tol) in ref.items():
        n = int(w.seq_lens[s])
        want = steps * p + (base[s, :, :n].double() if base is not None else 0.0)
        t = steps * tol + 2.0 ** -24 * (8 + steps) * want.abs()
        assert bool(((got[s, :, :n].double() - want).abs() <= t).all()), s
        assert torch.equal(got[s, :, n:].view(torch.int32), before[s, :, n:].view(torch.int32)), s


@pytest.mark.parametrize("cache,qd,fp8_scale", [("bf16", "bf16", "tensor"), ("fp16", "fp16", "tensor"),
                                                ("fp8", "bf16", "tensor"), ("fp8", "fp16", "head")])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_weights_and_output(cache, qd, fp8_scale, G, bs):
    w = _case(900 + G + bs, G, cache, qd, bs, Hkv=3 if fp8_scale == "head" else 2, fp8_scale=fp8_scale)
    ws = _workspace(w)
    base = torch.rand(w.num_seqs, w.num_kv_heads, _stride(w) + bs % 5, device=DEV)
    wout = torch.full_like(base, float("nan"))
    before = wout.clone()
    out = _call(w, ws, wout, base)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    plain = torch.empty_like(out)
    pa.pa_decode(plain, w.q[0], w.k_cache[0], w.v_cache[0], w.block_tables, w.seq_lens, w.scale,
                 pa.new_workspace(w.num_seqs, w.num_q_heads, w.num_kv_heads), **_args(w))
    assert torch.equal(out, plain)
    _check(w, wout, before, _reference(w, range(w.num_seqs)), base)


def test_in_place_over_steps_and_without_a_base():
    w = _case(31, 4)
    ws = _workspace(w, spare=64)
    ref = _reference(w, range(w.num_seqs))
    acc = torch.full((w.num_seqs, w.num_kv_heads, _stride(w)), 5.0, device=DEV)
    before = acc.clone()
    _call(w, ws, acc)                                # no base: this step alone
    _check(w, acc, before, ref)
    for _ in range(3):
        _call(w, ws, acc, acc)
    _check(w, acc, before, ref, steps=4)


def test_long_rows_with_claimed_pieces():
    # 16 x 8192 tokens and 8 KV heads: every warp's range is long enough for run-time pieces
    w = _case(32, 4, "fp16", "fp16", Hkv=8, lens=[8192] * 12 + [8191, 8000, 3, 8177])
    ws = _workspace(w)
    ref = _reference(w, [0, 7, 12, 13, 14, 15])
    for _ in range(3):                               # the work counter is carried from call to call
        wout = torch.zeros(w.num_seqs, w.num_kv_heads, _stride(w), device=DEV)
        _call(w, ws, wout)
        _check(w, wout, torch.zeros_like(wout), ref)


def test_one_long_row():
    w = _case(33, 8, "fp8", Hkv=1, lens=[70000])
    wout = torch.zeros(1, 1, _stride(w), device=DEV)
    _call(w, _workspace(w), wout)
    _check(w, wout, torch.zeros_like(wout), _reference(w, [0]))
    assert abs(float(wout.double().sum()) - 8) < 1e-4


def test_many_sequences():
    # over 1024 sequences: the block prefix comes from the workspace
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 40, 1500)]
    w = _case(34, 2, Hkv=2, lens=lens)
    wout = torch.zeros(w.num_seqs, 2, _stride(w), device=DEV)
    ws = _workspace(w)
    _call(w, ws, wout)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    _check(w, wout, torch.zeros_like(wout), _reference(w, range(0, 1500, 7)))


def test_rows_of_one_value_and_infinite_scores():
    # equal keys: equal weights; a NaN query makes its own sequence's weights NaN and no other's
    w = _case(35, 4, lens=[16, 50, 50, 1])
    w.k_cache[0][w.block_tables[0, 0].long()] = 1.0
    w.q[0][1, 2] = float("nan")
    wout = torch.zeros(4, 2, _stride(w), device=DEV)
    _call(w, _workspace(w), wout)
    assert bool((wout[0, :, :16] - 0.25).abs().max() <= 2.0 ** -20)
    assert bool(wout[1, 0, :50].isnan().all()) and bool((wout[1, :, 50:] == 0).all())
    assert bool(wout[1, 1].isfinite().all()) and bool(wout[2:].isfinite().all())
    assert bool(((wout[3, :, 0] - 4).abs() <= 4 * 2.0 ** -20).all())


def test_workspace_with_too_few_scores_is_recorded():
    w = _case(36, 4, lens=[100, 200])
    ws = pa.new_workspace_weights(2, w.num_q_heads, w.num_kv_heads, _tokens(w) - 16)
    wout = torch.full((2, 2, _stride(w)), 3.0, device=DEV)
    out = _call(w, ws, wout)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_WORKSPACE
    assert bool((wout == 3.0).all())
    plain = torch.empty_like(out)
    pa.pa_decode(plain, w.q[0], w.k_cache[0], w.v_cache[0], w.block_tables, w.seq_lens, w.scale,
                 pa.new_workspace(2, w.num_q_heads, w.num_kv_heads))
    assert torch.equal(out, plain)
    with pytest.raises(pa.PagedAttentionError):
        _call(w, pa.new_workspace(2, w.num_q_heads, w.num_kv_heads), wout)


def test_graph_replay_and_another_stream():
    w = _case(37, 4)
    ws, base = _workspace(w), torch.rand(w.num_seqs, 2, _stride(w), device=DEV)
    wout, out = torch.zeros_like(base), torch.empty_like(w.q[0])
    _call(w, ws, wout, base, out)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        _call(w, ws, wout, base, out)
    w.q[0].copy_(torch.randn_like(w.q[0].float()))
    base.uniform_()
    wout.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    ref = _reference(w, range(w.num_seqs))
    _check(w, wout, torch.zeros_like(wout), ref, base)
    wout.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        _call(w, ws, wout, base, out)
    torch.cuda.synchronize()
    _check(w, wout, torch.zeros_like(wout), ref, base)


def test_observing_the_last_queries_of_a_prompt():
    # one row per query over the same table, each up to its own position; the sums added up
    w = _case(40, 4, lens=[300] + [7] * 5)
    n = torch.arange(295, 301, device=DEV, dtype=torch.int32)
    w.block_tables = w.block_tables[:1].repeat(6, 1).contiguous()
    w.seq_lens = n
    wout = torch.zeros(6, 2, _stride(w), device=DEV)
    _call(w, _workspace(w), wout)
    _check(w, wout, torch.zeros_like(wout), _reference(w, range(6)))
    assert float((wout.double().sum((0, 2)) - 24).abs().max()) < 1e-4        # 6 rows of 4 heads per KV head


def test_no_sequences_and_only_empty_ones():
    w = _case(39, 4, lens=[0, 0, 0])
    wout = torch.full((3, 2, _stride(w)), 2.0, device=DEV)
    out = _call(w, _workspace(w), wout)
    assert bool((out == 0).all()) and bool((wout == 2.0).all())
    e = lambda t: t[:0]  # noqa: E731
    pa.pa_decode_weights(e(out), e(wout), e(w.q[0]), w.k_cache[0], w.v_cache[0], e(w.block_tables), e(w.seq_lens),
                         w.scale, pa.new_workspace_weights(0, 8, 2, 0))


def test_refusals():
    w = _case(38, 4, "fp8", lens=[20, 30])
    ws = _workspace(w)
    good = torch.zeros(2, 2, _stride(w), device=DEV)
    for bad in (good[:1], good[:, :1], good.half(), good.cpu(), good.transpose(0, 1)):
        with pytest.raises((ValueError, TypeError)):
            _call(w, ws, bad)
    with pytest.raises(ValueError):
        _call(w, ws, good, torch.zeros(2, 2, _stride(w) + 16, device=DEV))
    with pytest.raises(pa.PagedAttentionError):
        _call(w, ws, good[..., :-1].contiguous())
    assert math.isfinite(float(good.sum()))


def test_a_workspace_beyond_64_bits_has_no_size():
    assert pa.pa_workspace_size_weights(1, 1 << 24, 1 << 24, (1 << 40) - 1) == 0
    a, b = (pa.pa_workspace_size_weights(1, 1 << 24, 1 << 24, n) for n in (16, 1 << 20))
    assert b - a == ((1 << 16) - 1) * (1 << 24) * 16 * 2 * 4
