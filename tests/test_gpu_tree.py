"""pa_tree and pa_tree_commit on the GPU: attention of drafted trees against float64 (the
tolerance: tests/_scored.py), the commit bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_99_gb300 as pa
from tests._scored import DEV, Batch, check, random_trees, reference, tree_sight

pytestmark = pytest.mark.gpu
FORMATS = [("bf16", "bf16", False), ("fp16", "fp16", False), ("fp8", "bf16", False), ("fp8", "fp16", True)]


def call(b, masks, **kw):
    out = torch.full_like(b.q, 7.0)
    ws = pa.new_workspace_scored(len(b.lens_h), b.hq, b.hkv)
    pa.pa_tree(out, b.q, b.start, *b.caches, b.tables, b.lens, masks, b.scale, ws, **b.args(), **kw)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    return out


def one(b, seed=1, cap=0.0, window=0):
    sight, masks = tree_sight(b, random_trees(b, seed), window)
    check(call(b, masks, cap=cap, window=window), *reference(b, sight, cap))


CTX = [0, 1, 17, 100, 127, 128, 129, 600, 1500]
NODES = [5, 1, 2, 28, 64, 65, 9, 16, 33]


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("cache,kind,per_head", FORMATS)
@pytest.mark.parametrize("cap,window", [(0.0, 0), (30.0, 0), (0.0, 50)])
def test_against_float64(bs, cache, kind, per_head, cap, window):
    b = Batch(40 + bs, [c + m for c, m in zip(CTX, NODES)], NODES, 8, 2, cache, kind, bs, per_head)
    one(b, bs, cap, window)


@pytest.mark.parametrize("nodes", [63, 64, 100, 127, 128, 129, 200, 300])
@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_large_trees(nodes, cache):
    b = Batch(50, [nodes + 70, nodes + 3, nodes], [nodes, nodes, nodes], 4, 1, cache)
    one(b, nodes, 20.0)


@pytest.mark.parametrize("G", [1, 3, 7, 8, 16, 128])
def test_groups(G):
    b = Batch(60 + G, [300 + 20, 33 + 7], [20, 7], G * 2 if G < 16 else G, 2 if G < 16 else 1)
    one(b, G)


def test_few_long_sequences():
    for cache in ("bf16", "fp8"):
        b = Batch(61, [16000 + 24, 9000 + 24], [24, 24], 8, 2, cache)
        one(b)
        one(b, 2, 50.0, 4096)


def test_many_sequences():
    nodes = [1 + (5 * i) % 23 for i in range(80)]
    b = Batch(62, [m + 31 * i for i, m in enumerate(nodes)], nodes, 8, 2)
    one(b)


def test_rows_that_see_no_node_and_nodes_no_row_sees():
    """Padding nodes: their rows see only the context (or nothing), and their K and V, which no
    row sees, may be NaN."""
    for cache in ("bf16", "fp8"):
        b = Batch(63, [90 + 12, 8], [12, 8], 8, 2, cache)
        blind = {8, 9, 10, 11, 12 + 6, 12 + 7}
        trees = [[-1, 0, 0, 1, 1, 2, 4, 5, -1, -1, -1, -1], [-1, 0, 1, 0, 3, 1, -1, -1]]
        sight, masks = tree_sight(b, trees, 0, blind)
        for s, first, n in ((0, 98, 102), (1, 6, 8)):
            for t in range(first, n):
                for c in b.caches:
                    c[int(b.tables[s, t // 16]), :, t % 16] = 0x7F if cache == "fp8" else float("nan")
        masks |= 0                                   # bits from the tree's size on are ignored
        masks[:12] |= -(1 << 40)
        want, tol = reference(b, sight)
        got = call(b, masks)
        check(got, want, tol)
        assert bool((got[18:20] == 0).all())         # no context and no node: zeros


def test_a_chain_is_a_chunk():
    b = Batch(64, [300, 77], [20, 20], 8, 2)
    sight, masks = tree_sight(b, [list(range(-1, 19))] * 2)
    out = torch.empty_like(b.q)
    ws = pa.new_workspace(2, 8, 2)
    pa.pa_mixed(out, b.q, b.start, *b.caches, b.tables, b.lens, 20, b.scale, ws)
    want, tol = reference(b, sight)
    assert bool(((call(b, masks).double() - out.double()).abs() <= 2 * tol).all())


def test_a_tree_wider_than_its_masks_is_recorded():
    b = Batch(65, [100, 90], [70, 20], 8, 2)
    sight, masks = tree_sight(b, random_trees(b, 1))
    good = call(b, masks)
    ws = pa.new_workspace_scored(2, 8, 2)
    out = torch.full_like(b.q, 7.0)
    pa.pa_tree(out, b.q, b.start, *b.caches, b.tables, b.lens, masks[:, :1].contiguous(), b.scale, ws)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_OUT_OF_RANGE
    assert bool((out[:70] == 7.0).all()) and torch.equal(out[70:], good[70:])


# ---- the commit ------------------------------------------------------------------

def commit(b, caches, paths, lens, ws=None, width=None):
    width = max(1, max(lens)) if width is None else width
    p = torch.full((len(paths), width), -5, dtype=torch.int32)
    for i, x in enumerate(paths):
        p[i, :len(x)] = torch.tensor(x, dtype=torch.int32)
    out = torch.full((len(paths),), -9, dtype=torch.int32, device=DEV)
    pa.pa_tree_commit(out, caches[0::2], caches[1::2], p.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                      b.start, b.tables, b.lens, workspace=ws)
    return out


def moved(b, cache, paths, lens):
    """The cache afterwards, row by row on the host's copy."""
    c = cache.clone()
    t = b.tables.tolist()
    for s, path in enumerate(paths):
        base = b.lens_h[s] - b.rows_h[s]
        for i in range(lens[s]):
            x, y = base + path[i], base + i
            c[t[s][y // b.bs], :, y % b.bs] = cache[t[s][x // b.bs], :, x % b.bs].clone()
    return c


def same(a, b):
    return torch.equal(a.view(torch.int8), b.view(torch.int8))


@pytest.mark.parametrize("cache", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("layers", [1, 3, 65])
def test_commit(cache, bs, layers):
    nodes = [1, 5, 16, 40, 64, 130, 7, 0]
    ctx = [0, 3, 15, 16, 33, 100, 64, 20]
    r = np.random.RandomState(bs)
    b = Batch(80 + bs, [c + m for c, m in zip(ctx, nodes)], nodes, 6, 3, cache, bs=bs)
    lens = [1, 3, 0, 17, 33, 100, 7, 0]
    paths = [sorted(r.choice(m, n, replace=False).tolist()) for m, n in zip(nodes, lens)]
    caches = [b.caches[i % 2].roll(i, 0).contiguous() for i in range(2 * layers)]
    before = [c.clone() for c in caches]
    ws = pa.new_workspace_scored(8, 6, 3)
    out = commit(b, caches, paths, lens, ws)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    assert out.tolist() == [c + n for c, n in zip(ctx, lens)]
    for x, y in zip(caches, before):
        assert same(x, moved(b, y, paths, lens))


def test_commit_of_paths_that_are_none_moves_nothing():
    nodes = [8] * 7
    b = Batch(90, [30 + 8] * 7, nodes, 4, 2)
    paths = [[0, 2, 5], [2, 1], [0, 8], [-1, 3], [1, 1], [1, 3], [2, 4, 6]]
    caches = [c.clone() for c in b.caches]
    lens = [3, 2, 2, 2, 2, 9, 3]                    # the sixth is longer than its tree
    b.tables[6, 2] = 1 << 20                        # the last one's nodes lie outside the pool
    ws = pa.new_workspace_scored(7, 4, 2)
    out = commit(b, caches, paths, lens, ws, width=12)
    assert pa.pa_read_device_status(ws) == pa.PA_ERR_OUT_OF_RANGE
    assert out.tolist() == [33] + [-9] * 6
    for x, y in zip(caches, b.caches):
        assert same(x, moved(b, y, paths[:1], lens))


def test_commit_of_the_same_batch_twice_in_a_graph():
    b = Batch(91, [50 + 20, 9 + 20], [20, 20], 4, 2)
    caches = [c.clone() for c in b.caches]
    start = [c.clone() for c in caches]
    p = torch.tensor([[0, 3, 4, 19], [1, 2, 17, -1]], dtype=torch.int32, device=DEV)
    n = torch.tensor([4, 3], dtype=torch.int32, device=DEV)
    out = torch.zeros(2, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_tree_commit(out, caches[:1], caches[1:], p, n, b.start, b.tables, b.lens)
    for _ in range(2):
        for c, s in zip(caches, start):
            c.copy_(s)
        g.replay()
    torch.cuda.synchronize()
    assert out.tolist() == [54, 12]
    for x, y in zip(caches, start):
        assert same(x, moved(b, y, p.tolist(), [4, 3]))


def test_draft_verify_commit_and_on():
    """Tokens written normed and rotated, a tree verified over them, its path committed, and the
    next token decoded over what the cache holds then: as if only the path had ever been written."""
    T, ctx, Hq, H, bs = 12, 45, 8, 2, 16
    parents = [-1, 0, 0, 1, 1, 2, 4, 4, 5, 8, 9, 9]
    path = [0, 2, 5, 8, 9]
    depth = [0] * T
    for i in range(1, T):
        depth[i] = depth[parents[i]] + 1
    g = torch.Generator(device=DEV).manual_seed(3)
    n = ctx + T
    qkv = torch.randn(n + 1, Hq + 2 * H, 128, generator=g, device=DEV).bfloat16()
    wq, wk = (1 + 0.1 * torch.randn(128, generator=g, device=DEV) for _ in range(2))
    wq, wk = wq.bfloat16(), wk.bfloat16()
    table = torch.empty(256, 128, device=DEV)
    pa.pa_rope_table(table, pa.pa_rope_frequencies(128))
    pos = torch.tensor(list(range(ctx)) + [ctx + d for d in depth] + [ctx + len(path)], device=DEV)
    slots = torch.arange(n, device=DEV) + bs

    def write(rows, at, kc, vc):
        x = qkv[rows]
        q = torch.empty(len(x), Hq, 128, dtype=torch.bfloat16, device=DEV)
        pa.pa_norm_rope_and_cache(q, x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], kc, vc, at, pos[rows].contiguous(), table,
                                  wq, wk)
        return q

    kc, vc = (torch.zeros(8, H, bs, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = write(torch.arange(n, device=DEV), slots, kc, vc)
    tables = torch.tensor([[1, 2, 3, 4, 5]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    mask = [0] * T
    for i in range(T):
        mask[i] = (mask[parents[i]] if i else 0) | 1 << i
    masks = torch.tensor(mask, device=DEV).view(T, 1)
    ws = pa.new_workspace_scored(1, Hq, H)
    out = torch.empty(T, Hq, 128, dtype=torch.bfloat16, device=DEV)
    pa.pa_tree(out, q[ctx:].contiguous(), start, kc, vc, tables, lens, masks, 0.088, ws, cap=30.0)
    new = torch.zeros_like(lens)
    pa.pa_tree_commit(new, [kc], [vc], torch.tensor([path], dtype=torch.int32, device=DEV),
                      torch.tensor([len(path)], dtype=torch.int32, device=DEV), start, tables, lens, workspace=ws)
    assert int(new) == ctx + len(path)
    # the next token behind the path
    last = torch.tensor([n], device=DEV)
    q1 = write(last, slots[:1] + int(new), kc, vc)
    step = torch.empty_like(q1)
    pa.pa_mixed_scored(step, q1, torch.tensor([0, 1], dtype=torch.int32, device=DEV), kc, vc, tables, new + 1, 0.088, ws,
                       cap=30.0)
    # only the path and the next token written, as a chunk
    kd, vd = torch.zeros_like(kc), torch.zeros_like(vc)
    rows = torch.tensor(list(range(ctx)) + [ctx + i for i in path] + [n], device=DEV)
    qd = write(rows, slots[:len(rows)], kd, vd)
    m = len(path) + 1
    chunk = torch.empty(m, Hq, 128, dtype=torch.bfloat16, device=DEV)
    pa.pa_mixed_scored(chunk, qd[ctx:].contiguous(), torch.tensor([0, m], dtype=torch.int32, device=DEV), kd, vd, tables,
                       new + 1, 0.088, ws, cap=30.0)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
    live = int(new) + 1
    t = torch.arange(live, device=DEV)
    for a, b in ((kc, kd), (vc, vd)):
        assert torch.equal(a[1 + t // bs, :, t % bs], b[1 + t // bs, :, t % bs])
    both = torch.cat((out[path], step))
    # two orders of the same sums: each off by at most 2 x 2^-8 of Σ p |V| (probabilities and output)
    assert float((both.float() - chunk.float()).abs().max()) <= 4 * 2.0 ** -8 * float(vc.float().abs().max())
