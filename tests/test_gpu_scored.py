"""pa_mixed_scored on the GPU against float64 attention (the tolerance: tests/_scored.py)."""
import pytest
import torch

import paged_kv_cache_99_gb300 as pa
from tests._scored import DEV, Batch, causal, check, reference

pytestmark = pytest.mark.gpu


def call(b, out=None, q=None, ws=None, **kw):
    out = torch.full_like(b.q, 7.0) if out is None else out
    ws = pa.new_workspace_scored(len(b.lens_h), b.hq, b.hkv) if ws is None else ws
    pa.pa_mixed_scored(out, b.q if q is None else q, b.start, *b.caches, b.tables, b.lens, b.scale, ws, **b.args(), **kw)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    return out


def slopes_of(hq):
    return 2.0 ** (-8.0 * (torch.arange(hq, device=DEV) + 1) / hq)


def one(b, cap=0.0, slopes=None, window=0, prefix=None, what=""):
    p = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV)
    got = call(b, cap=cap, slopes=slopes, window=window, prefix_lens=p)
    check(got, *reference(b, causal(b, window, prefix), cap, slopes), what)
    return got


LENS = [1, 2, 15, 16, 17, 127, 128, 129, 300, 1025, 0, 64]
ROWS = [1, 2, 1, 16, 3, 127, 1, 129, 1, 40, 0, 5]
FORMATS = [("bf16", "bf16", False), ("fp16", "fp16", False), ("fp8", "bf16", False), ("fp8", "fp16", True)]


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("cache,kind,per_head", FORMATS)
@pytest.mark.parametrize("cap,bias,window,prefix", [(0.0, False, 0, False), (30.0, False, 0, False), (0.0, True, 0, False),
                                                    (0.0, False, 37, False), (0.0, False, 0, True),
                                                    (5.0, True, 130, True), (50.0, False, 1, False)])
def test_against_float64(bs, cache, kind, per_head, cap, bias, window, prefix):
    b = Batch(11 + bs, LENS, ROWS, 8, 2, cache, kind, bs, per_head)
    pre = [min(n, (7 * i) % 90) for i, n in enumerate(LENS)] if prefix else None
    one(b, cap, slopes_of(8) if bias else None, window, pre)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 12, 16, 48, 128])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_groups(G, cache):
    b = Batch(70 + G, [40, 700, 131], [1, 33, 9], G * (1 if G > 16 else 3), 1 if G > 16 else 3, cache, "bf16")
    one(b, 20.0, slopes_of(b.hq), 0, [0, 690, 131])


@pytest.mark.parametrize("cap", [1e-6, 0.5, 3.0, 1000.0, 3e4, 1e6])
def test_caps_from_tight_to_wide(cap):
    # scores far beyond the cap, near it and far below
    for size in (0.05, 2.0, 40.0):
        b = Batch(5, [300, 140], [1, 40], 8, 2, q_size=size)
        one(b, cap, what=f"q {size}")


def test_decode_batches():
    lens = [1 + 97 * i for i in range(70)]
    b = Batch(3, lens, [1] * 70, 16, 4)
    one(b, 50.0, None, 1000)
    b = Batch(4, lens, [1] * 70, 16, 2, "fp8")
    one(b, 0.0, slopes_of(16))


@pytest.mark.parametrize("cache", ["bf16", "fp16", "fp8"])
def test_one_long_sequence(cache):
    for m in (1, 2, 40):
        b = Batch(9, [20011], [m], 4, 1, cache, "fp16" if cache == "fp16" else "bf16")
        one(b, 30.0)
        one(b, 0.0, None, 5000)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_prompts(cache):
    b = Batch(21, [1500, 700, 33], [1500, 651, 33], 8, 2, cache)
    one(b, 50.0)
    one(b, 0.0, slopes_of(8), 200)
    one(b, 20.0, None, 0, [900, 700, 5])
    b = Batch(22, [900], [900], 15, 3, cache)       # 5 heads to a KV head: tiles with spare rows
    one(b, 0.0, None, 300, [450])


def test_masked_blocks_are_not_read():
    """Blocks that no row sees through the window may be anything, and need not be in the table."""
    b = Batch(31, [1000, 400, 2000], [1, 3, 40], 8, 2)
    want = reference(b, causal(b, 100))
    for s, (n, m) in enumerate(zip(b.lens_h, b.rows_h)):
        first = max(0, n - m - 100 + 1)             # the first token any row sees
        b.tables[s, :first // b.bs] = -1 if s != 1 else 1 << 30
        for t in range(first // b.bs * b.bs, first):
            for c in b.caches:
                c[int(b.tables[s, t // b.bs]), :, t % b.bs] = float("nan")
    check(call(b, window=100), *want)


def test_rows_behind_the_last_sequence_stay():
    b = Batch(32, [40, 60], [3, 5], 8, 2)
    q = torch.cat((b.q, torch.full((4, 8, 128), float("nan"), device=DEV, dtype=b.q.dtype)))
    out = torch.full_like(q, 3.0)
    call(b, out, q, cap=20.0)
    assert bool((out[8:] == 3.0).all())
    check(out[:8], *reference(b, causal(b), 20.0))


def test_plain_scores_agree_with_pa_mixed():
    b = Batch(33, LENS, ROWS, 8, 2)
    out = torch.empty_like(b.q)
    ws = pa.new_workspace(len(LENS), 8, 2)
    pa.pa_mixed(out, b.q, b.start, *b.caches, b.tables, b.lens, max(ROWS), b.scale, ws)
    want, tol = reference(b, causal(b))
    got = call(b)
    assert bool(((got.double() - out.double()).abs() <= 2 * tol).all())


def test_bad_lengths_and_blocks_are_recorded():
    def status(b, **kw):
        ws = pa.new_workspace_scored(len(b.lens_h), b.hq, b.hkv)
        out = torch.full_like(b.q, 7.0)
        pa.pa_mixed_scored(out, b.q, b.start, *b.caches, b.tables, b.lens, b.scale, ws, cap=10.0, **kw)
        return pa.pa_read_device_status(ws), out

    b = Batch(34, [40, 60, 30], [3, 5, 1], 8, 2)
    good = call(b, cap=10.0)
    b.lens[1] = 4                                   # fewer tokens than rows
    st, out = status(b)
    assert st == pa.PA_ERR_OUT_OF_RANGE
    assert bool((out[3:8] == 7.0).all()) and torch.equal(out[:3], good[:3]) and torch.equal(out[8:], good[8:])
    b.lens[1] = b.tables.shape[1] * b.bs + 1        # more than the table
    st, out = status(b)
    assert st == pa.PA_ERR_OUT_OF_RANGE and bool((out[3:8] == 7.0).all()) and torch.equal(out[8:], good[8:])
    b.lens[1] = 60
    b.start[3] = 12                                 # a row outside q
    st, out = status(b)
    assert st == pa.PA_ERR_OUT_OF_RANGE and bool((out[8:] == 7.0).all()) and torch.equal(out[:8], good[:8])
    b.start[3] = 9
    b.tables[0, 1] = 1 << 20                        # a block outside the pool
    st, out = status(b)
    assert st == pa.PA_ERR_OUT_OF_RANGE and torch.equal(out[3:], good[3:])


def test_captured_and_replayed():
    b = Batch(35, [300, 129, 1000], [1, 40, 1], 8, 2)
    c = Batch(36, [50, 900, 64], [1, 40, 1], 8, 2)
    ws = pa.new_workspace_scored(3, 8, 2)
    # both graphs share the workspace and follow one another
    graphs, outs = [], []
    for x in (b, c):
        out = torch.zeros_like(x.q)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pa.pa_mixed_scored(out, x.q, x.start, *x.caches, x.tables, x.lens, x.scale, ws, cap=30.0)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    for x, out in zip((b, c), outs):
        check(out, *reference(x, causal(x), 30.0))
    # lengths may change between replays
    c.lens_h = [50, 200, 64]
    c.lens.copy_(torch.tensor(c.lens_h))
    c.k[1], c.v[1] = c.k[1][:200], c.v[1][:200]
    graphs[1].replay()
    torch.cuda.synchronize()
    check(outs[1], *reference(c, causal(c), 30.0))


def test_repeatable_and_on_a_side_stream():
    b = Batch(37, [5000, 129, 2000], [1, 100, 7], 8, 2)
    first = call(b, cap=30.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = pa.new_workspace_scored(3, 8, 2)
    out = torch.empty_like(b.q)
    torch.cuda.synchronize()
    pa.pa_mixed_scored(out, b.q, b.start, *b.caches, b.tables, b.lens, b.scale, ws, cap=30.0, stream=side)
    side.synchronize()
    assert torch.equal(out, first)


def test_empty_calls():
    b = Batch(38, [40], [0], 8, 2)
    call(b)
    e = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=DEV)
    i0, i1 = torch.zeros(0, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = pa.new_workspace_scored(0, 8, 2)
    pa.pa_mixed_scored(e, e, i1, *b.caches, torch.zeros(0, 4, dtype=torch.int32, device=DEV), i0, 0.1, ws)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("scale", [-0.1, 0.0])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, False), (0.0, True), (4.0, True)])
def test_scales_that_turn_or_flatten_the_scores(cache, scale, cap, bias):
    b = Batch(60, [300, 129, 700, 1], [1, 100, 7, 1], 8, 2, cache)
    b.scale = scale
    one(b, cap, slopes_of(8) if bias else None, 64 if bias else 0)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_outputs_on_any_16_bytes(cache):
    b = Batch(61, [5000, 129, 700], [1, 100, 7], 8, 2, cache)
    flat = torch.full((b.q.numel() + 64,), 7.0, dtype=b.q.dtype, device=DEV)
    for at in (0, 8, 16):
        out = flat[at:at + b.q.numel()].view_as(b.q)
        assert out.data_ptr() % 32 == 2 * at % 32
        call(b, out, cap=30.0)
        check(out, *reference(b, causal(b), 30.0), f"at {at}")
    assert bool((flat[b.q.numel() + 16:] == 7).all())


def test_query_rows_that_the_output_replaces():
    b = Batch(62, [5000, 129, 700, 2600], [1, 100, 7, 30], 8, 2)
    want = call(b, cap=30.0)
    q = b.q.clone()
    call(b, q, q, cap=30.0)
    assert torch.equal(q, want)


def test_starts_that_go_back_and_forth():
    # rows that several sequences name, or none: recorded, or their last writer's
    b = Batch(63, [300] * 6, [10] * 6, 8, 2)
    good = call(b)
    ws = pa.new_workspace_scored(6, 8, 2)
    b.start = torch.tensor([0, 60, 10, 60, 20, 25, 60], dtype=torch.int32, device=DEV)
    out = torch.full_like(b.q, 7.0)
    pa.pa_mixed_scored(out, b.q, b.start, *b.caches, b.tables, b.lens, b.scale, ws)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_OUT_OF_RANGE
    assert bool(torch.isfinite(out).all()) and torch.equal(call(Batch(63, [300] * 6, [10] * 6, 8, 2)), good)


def test_a_cache_past_four_gib():
    bs, hkv, blocks = 16, 8, 200000                  # 6.5 GB each
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    b = Batch(64, [300, 129], [1, 100], 16, hkv, bs=bs)
    first = blocks - b.caches[0].shape[0]
    big = [torch.empty(blocks, hkv, bs, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for x, c in zip(big, b.caches):
        x[first:] = c
    b.caches = big
    b.tables = torch.where(b.tables >= 0, b.tables + first, b.tables)
    got = one(b, 30.0)
    # and rows written and moved there
    c = torch.randn(3, 32, 128, device=DEV).bfloat16()
    slots = torch.tensor([(blocks - 1) * bs + 3, blocks * bs - 1, (blocks - 2) * bs], device=DEV)
    table = torch.tensor([[1.0] * 8 + [0.0] * 8], device=DEV)
    q = torch.empty(3, 16, 128, dtype=torch.bfloat16, device=DEV)
    pa.pa_norm_rope_and_cache(q, c[:, :16], c[:, 16:24], c[:, 24:], *big, slots, torch.zeros(3, dtype=torch.int64, device=DEV),
                              table)
    for i, x in enumerate(slots.tolist()):
        assert torch.equal(big[0][x // bs, :, x % bs], c[i, 16:24]) and torch.equal(big[1][x // bs, :, x % bs], c[i, 24:])
    lens = torch.tensor([2 * bs], dtype=torch.int32, device=DEV)
    tables = torch.tensor([[blocks - 2, blocks - 1]], dtype=torch.int32, device=DEV)
    new = torch.zeros_like(lens)
    pa.pa_tree_commit(new, big[:1], big[1:], torch.tensor([[3, 15]], dtype=torch.int32, device=DEV),
                      torch.tensor([2], dtype=torch.int32, device=DEV), torch.tensor([0, bs], dtype=torch.int32, device=DEV),
                      tables, lens)
    assert new.tolist() == [bs + 2]
    for i in range(2):
        assert torch.equal(big[0][blocks - 1, :, i], c[i, 16:24]) and torch.equal(big[1][blocks - 1, :, i], c[i, 24:])
    assert got.shape == b.q.shape


@pytest.mark.parametrize("cache,kind,per_head", FORMATS)
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, False), (0.0, True)])
def test_many_short_units_of_all_sizes(cache, kind, per_head, cap, bias):
    # every SM goes through solos and pairs of one step and of a few, in any order
    g = torch.Generator().manual_seed(65)
    rows = [int(x) for x in torch.randint(0, 4, (400,), generator=g)]
    rows = [r if r < 3 else int(torch.randint(1, 90, (1,), generator=g)) for r in rows]
    lens = [r + int(torch.randint(0, 300, (1,), generator=g)) * int(torch.rand(1, generator=g) < 0.6) for r in rows]
    b = Batch(66, lens, rows, 24, 3, cache, kind, 16, per_head)
    one(b, cap, slopes_of(24) if bias else None)


def test_two_streams_at_once():
    batches = [Batch(67, [5000, 129, 2000], [1, 100, 7], 8, 2), Batch(68, [40] * 200, [1] * 200, 16, 2, "fp8")]
    want = [call(b, cap=30.0) for b in batches]
    spaces = [pa.new_workspace_scored(len(b.lens_h), b.hq, b.hkv) for b in batches]
    outs = [torch.zeros_like(b.q) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(50):
        for b, out, ws, st in zip(batches, outs, spaces, streams):
            pa.pa_mixed_scored(out, b.q, b.start, *b.caches, b.tables, b.lens, b.scale, ws, cap=30.0, stream=st, **b.args())
    torch.cuda.synchronize()
    for out, ws, w in zip(outs, spaces, want):
        assert pa.pa_read_device_status(ws) == pa.PA_OK and torch.equal(out, w)
