"""The operators of a step over a paged cache with drafted trees and models whose queries,
keys or scores are not plain, as cases that can be measured: queries and keys normed per
head and turned by positions of several axes with the slot write, attention for a tree of
drafted tokens over a cache, the move of the accepted path's rows, and attention whose
scores are capped, biased by distance, windowed or open over a prefix.

``own`` says which side runs: the plain forms below (elementary torch in 32 bits) or the
library's entry points on the same inputs.
"""
import math

import numpy as np
import torch

own = False

D = 128                     # head dimension of the library
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
PAIRS = 1.08e9              # (query row, key, query head) triples of the largest attention case
BYTES = 4.2e8               # bytes of the largest case


def listed():
    return [
        # the smallest decode step (four sequences, one new token each): latency
        {"name": "norm 4 tokens", "op": "norm", "tokens": 4, "hq": 8, "hkv": 2, "rot": 128, "sections": "",
         "interleaved": False, "type": "bf16", "cache": "bf16", "bs": 16, "context": 32768},
        # 16 decode rows and two chunks of 512 of a vision model, its axes dealt out in turns, FP8 cache
        {"name": "norm mixed fp8 3 axes", "op": "norm", "tokens": 1040, "hq": 64, "hkv": 8, "rot": 128,
         "sections": "24,20,20 in turns", "interleaved": False, "type": "bf16", "cache": "fp8", "bs": 16,
         "context": 32768},
        # a prefill step of a long document with pictures (time, height, width one after the other)
        {"name": "norm prefill 16k 3 axes", "op": "norm", "tokens": 16384, "hq": 32, "hkv": 8, "rot": 128,
         "sections": "16,24,24", "interleaved": False, "type": "bf16", "cache": "bf16", "bs": 16, "context": 131072},
        # two short sequences with a handful of drafted tokens: latency
        {"name": "tree tiny", "op": "tree", "batch": 2, "lo": 8, "hi": 46, "nodes": 6, "hq": 8, "hkv": 2, "cap": 0.0,
         "window": 0, "type": "bf16", "cache": "bf16", "bs": 16},
        # one layer of a verification step of 16 sequences, 24 drafted tokens each
        {"name": "tree 16 x 8k", "op": "tree", "batch": 16, "lo": 1024, "hi": 8192, "nodes": 24, "hq": 32, "hkv": 8,
         "cap": 0.0, "window": 0, "type": "bf16", "cache": "bf16", "bs": 16},
        # a wide group and a large tree over an FP8 cache, capped scores
        {"name": "tree 32 x 4k fp8 capped", "op": "tree", "batch": 32, "lo": 512, "hi": 4096, "nodes": 61, "hq": 64,
         "hkv": 8, "cap": 50.0, "window": 0, "type": "bf16", "cache": "fp8", "bs": 16},
        # one layer, four sequences: latency
        {"name": "commit 4, one layer", "op": "commit", "batch": 4, "lo": 8, "hi": 46, "nodes": 16, "depth": 4, "hkv": 2,
         "layers": 1, "cache": "bf16", "bs": 16},
        # the accepted paths of a whole model's step: 28 layers, 64 sequences
        {"name": "commit 64, 28 layers", "op": "commit", "batch": 64, "lo": 16, "hi": 250, "nodes": 64, "depth": 8,
         "hkv": 2, "layers": 28, "cache": "bf16", "bs": 16},
        # the smallest decode step with capped scores: latency
        {"name": "scored decode tiny", "op": "scored", "batch": 4, "lo": 8, "hi": 46, "rows": 0, "chunks": 0, "hq": 8,
         "hkv": 2, "cap": 50.0, "bias": False, "window": 0, "prefix": False, "type": "bf16", "cache": "bf16", "bs": 16},
        # one layer of a 64-sequence decode step, capped scores, a window on the longest
        {"name": "scored decode 64 x 8k capped", "op": "scored", "batch": 64, "lo": 512, "hi": 8192, "rows": 0,
         "chunks": 0, "hq": 16, "hkv": 4, "cap": 50.0, "bias": False, "window": 4096, "prefix": False, "type": "bf16",
         "cache": "bf16", "bs": 16},
        # 16 decode rows and two chunks of 512 over an FP8 cache, a bias that falls with distance
        {"name": "scored mixed fp8 bias", "op": "scored", "batch": 18, "lo": 1024, "hi": 8192, "rows": 512, "chunks": 2,
         "hq": 64, "hkv": 8, "cap": 0.0, "bias": True, "window": 0, "prefix": False, "type": "bf16", "cache": "fp8",
         "bs": 16},
        # one layer of a prompt of 8192 tokens, capped scores, its first part open in both directions
        {"name": "scored prompt 8k capped prefix", "op": "scored", "batch": 1, "lo": 8192, "hi": 8192, "rows": 8192,
         "chunks": 1, "hq": 32, "hkv": 8, "cap": 50.0, "bias": False, "window": 0, "prefix": True, "type": "bf16",
         "cache": "bf16", "bs": 16},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "tree", "tree", "tree", "commit", "scored", "scored", "scored"))
    hkv = rng.choice((1, 2, 4, 5, 8))
    cache, kind = rng.choice((("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16"), ("fp8", "fp16"), ("fp8 heads", "bf16")))
    bs = rng.choice((8, 16, 32))
    hq = hkv * rng.choice((1, 2, 3, 4, 6, 8))
    if op == "norm":
        tokens = _spread(rng, 1, max(1, 16384 * 40 // max(40, hq + hkv)))
        rot = 16 * rng.randint(1, 8)
        cuts = sorted(rng.randint(0, rot // 2) for _ in range(rng.randint(0, 3)))
        ends = [0] + cuts + [rot // 2]
        sections = ",".join(str(b - a) for a, b in zip(ends, ends[1:])) if cuts else ""
        if sections and rng.random() < 0.5:
            sections += " in turns"
        return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "rot": rot, "sections": sections,
                "interleaved": rng.random() < 0.5, "type": kind, "cache": cache, "bs": bs,
                "context": _spread(rng, max(tokens, 2048), 131072)}
    if op == "commit":
        nodes = _spread(rng, 1, 128)
        layers = _spread(rng, 1, 40)
        return {"op": op, "batch": _spread(rng, 1, max(1, min(128, 14336 // (layers * hkv)))), "lo": 0,
                "hi": _spread(rng, 1, 250), "nodes": nodes, "depth": rng.randint(1, min(nodes, 12)), "hkv": hkv,
                "layers": layers, "cache": cache, "bs": bs}
    hi = _spread(rng, 1, 32768)
    lo = rng.choice((0, 1, hi // 4, hi))
    cap = rng.choice((0.0, 0.0, 20.0, 50.0))
    window = rng.choice((0, 0, _spread(rng, 1, 8192)))
    e = 1 if cache.startswith("fp8") else 2
    if op == "tree":
        nodes = _spread(rng, 1, 200)
        most = min(BYTES / (2 * D * e * hkv * (hi + nodes)), PAIRS / (hq * nodes * (hi + nodes)), 128)
        return {"op": op, "batch": _spread(rng, 1, max(1, int(most))), "lo": lo, "hi": hi, "nodes": nodes, "hq": hq,
                "hkv": hkv, "cap": cap, "window": window, "type": kind, "cache": cache, "bs": bs}
    chunks = rng.choice((0, 0, 1, 2, 3))
    rows = _spread(rng, 1, max(1, min(hi, int(PAIRS / (hq * hi * 3))))) if chunks else 0
    batch = _spread(rng, 1, max(1, min(128, int(BYTES / (2 * D * e * hkv * hi)))))
    return {"op": op, "batch": max(batch, chunks), "lo": lo, "hi": hi, "rows": rows, "chunks": chunks, "hq": hq, "hkv": hkv,
            "cap": cap, "bias": rng.random() < 0.4, "window": window, "prefix": chunks > 0 and rng.random() < 0.4,
            "type": kind, "cache": cache, "bs": bs}


def _lengths(case, seed):
    """Tokens of each sequence: uniform in [lo, hi], the first one hi."""
    n = np.random.RandomState(seed % (1 << 31)).randint(case["lo"], case["hi"] + 1, case["batch"])
    n[0] = case["hi"]
    return [int(x) for x in n]


def _work_lengths(case):
    """The lengths work() counts: the first sequence at hi, the others at the mean."""
    return [case["hi"]] + [(case["lo"] + case["hi"]) / 2] * (case["batch"] - 1)


def _cache(shape, cache, g):
    """A cache of N(0, 1) values, and its scale (amax / 448 per tensor or head) if it is FP8."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if not cache.startswith("fp8"):
        return x.to(TYPES[cache]), None
    scale = x.abs().amax(dim=(0, 2, 3)) / 448 if cache == "fp8 heads" else (x.abs().max() / 448).reshape(1)
    return (x / scale.view(1, -1, 1, 1)).to(torch.float8_e4m3fn).view(torch.uint8), scale.contiguous()


def _tables(blocks, pool, g):
    """Block tables (-1 past a sequence's blocks) over a random permutation of the pool."""
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    t = torch.full((len(blocks), max(1, max(blocks))), -1, dtype=torch.int32)
    at = 0
    for s, nb in enumerate(blocks):
        t[s, :nb] = perm[at:at + nb]
        at += nb
    return t


def _axes(sections):
    """Axis of each pair: the sections one after the other, or dealt out in turns until each is used up."""
    counts = [int(x) for x in sections.removesuffix(" in turns").split(",")]
    if not sections.endswith("in turns"):
        return [a for a, c in enumerate(counts) for _ in range(c)]
    out, left = [], list(counts)
    while sum(left):
        for a, c in enumerate(left):
            if c:
                out.append(a)
                left[a] -= 1
    return out


def _prepare_norm(case, seed, g, host):
    t, hq, hkv, rot, bs = case["tokens"], case["hq"], case["hkv"], case["rot"], case["bs"]
    pool = -(-t // bs) + 64
    slots = (torch.randperm(pool, generator=host)[:-(-t // bs)].repeat_interleave(bs) * bs +
             torch.arange(bs).repeat(-(-t // bs)))[:t]
    # queries and keys differ in size from head to head; the learned weights lie around one
    qkv = torch.randn(t, hq + 2 * hkv, D, generator=g, device=DEV)
    qkv[:, :hq + hkv] *= torch.exp(torch.randn(hq + hkv, 1, generator=g, device=DEV))
    qkv = qkv.to(TYPES[case["type"]])
    weights = [(1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(qkv.dtype) for _ in range(2)]
    kc, ks = _cache((pool, hkv, bs, D), case["cache"], g)
    vc, vs = _cache((pool, hkv, bs, D), case["cache"], g)
    if ks is not None:                      # scales that leave room for what comes
        ks, vs = 2 * ks, 2 * vs
    angle = torch.arange(case["context"], device=DEV, dtype=torch.float64)[:, None] * \
        10000.0 ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)
    start = int(torch.randint(0, case["context"] - t + 1, (), generator=host))
    positions = start + torch.arange(t)
    axes = None
    if case["sections"]:
        axes = _axes(case["sections"])
        # a picture's tokens share their time and count rows and columns from its place on
        side = 32
        n = len(case["sections"].split(","))
        rows = [positions, torch.minimum(start + torch.arange(t) // side, positions),
                torch.minimum(start + torch.arange(t) % side, positions), positions // 2][:n]
        positions = torch.stack(rows)
    s = {"op": "norm", "qkv": qkv, "hq": hq, "hkv": hkv, "bs": bs, "rot": rot, "slots": slots.to(DEV),
         "positions": positions.contiguous().to(DEV), "axes": axes, "interleaved": case["interleaved"],
         "cos_sin": torch.cat((angle.cos(), angle.sin()), 1).float(), "wq": weights[0], "wk": weights[1], "kc": kc,
         "vc": vc, "ks": ks, "vs": vs, "q_out": torch.zeros(t, hq, D, device=DEV, dtype=qkv.dtype)}
    if axes:
        s["axes_dev"] = torch.tensor(axes, device=DEV)
        s["axes_bytes"] = bytes(axes)
    return s


def _tree(batch, nodes, seed):
    """Parents of every sequence's nodes (-1: the root, node 0) and the ancestor masks with the nodes
    themselves, int64 words.  A node hangs under one of the few before it or under an early one."""
    r = np.random.RandomState(seed % (1 << 31))
    parents = np.full((batch, nodes), -1, np.int64)
    words = -(-nodes // 64)
    masks = np.zeros((batch, nodes, words), np.uint64)
    rows = np.arange(batch)
    for i in range(nodes):
        if i:
            near = r.randint(max(0, i - 8), i, batch)
            parents[:, i] = np.where(r.rand(batch) < 0.5, near, r.randint(0, i, batch) // 4)
            masks[:, i] = masks[rows, parents[:, i]]
        masks[:, i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return parents, masks.view(np.int64)


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    if op == "norm":
        return _prepare_norm(case, seed, g, host)
    bs, hkv = case["bs"], case["hkv"]
    n = _lengths(case, seed)
    room = case["hi"]
    if op in ("tree", "commit"):        # the drafted tokens come behind the cached ones
        rows = [case["nodes"]] * len(n)
        n = [x + case["nodes"] for x in n]
        room += case["nodes"]
    elif op == "scored":                # the chunks are the last sequences of the batch
        first = len(n) - case["chunks"]
        n = [max(1, x) if i < first else max(x, case["rows"]) for i, x in enumerate(n)]
        rows = [1] * first + [case["rows"]] * case["chunks"]
    # room for every sequence at its longest: the pool's size does not go by the lengths drawn
    pool = len(n) * -(-room // bs) + 16
    tables = _tables([-(-x // bs) for x in n], pool, host)
    start = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
    s = {"op": op, "bs": bs, "hkv": hkv, "n": n, "rows": rows, "tables": tables.to(DEV),
         "lens": torch.tensor(n, dtype=torch.int32, device=DEV), "start": torch.from_numpy(start).to(DEV)}
    if op == "commit":
        caches = [_cache((pool, hkv, bs, D), case["cache"], g)[0] for _ in range(2 * case["layers"])]
        s.update(kcs=caches[0::2], vcs=caches[1::2], new_lens=torch.zeros(len(n), dtype=torch.int32, device=DEV))
        # accepted paths: the first nodes in place, then nodes behind the path's length (so that the
        # same path moved twice is the same as moved once)
        r = np.random.RandomState(seed % (1 << 31))
        paths = np.full((len(n), case["depth"]), -1, np.int32)
        lens = r.randint(0, case["depth"] + 1, len(n)).astype(np.int32)
        lens[0] = case["depth"]
        for i, m in enumerate(lens):
            far = min(r.randint(0, m + 1), case["nodes"] - m)
            paths[i, :m - far] = np.arange(m - far)
            paths[i, m - far:m] = np.sort(r.choice(np.arange(m, case["nodes"]), far, replace=False)) if far else 0
        s.update(paths=torch.from_numpy(paths).to(DEV), path_lens=torch.from_numpy(lens).to(DEV))
        return s
    kc, ks = _cache((pool, hkv, bs, D), case["cache"], g)
    vc, vs = _cache((pool, hkv, bs, D), case["cache"], g)
    q = torch.randn(int(start[-1]), case["hq"], D, generator=g, device=DEV) * 2      # scores of a few units
    q = q.to(TYPES[case["type"]])
    s.update(kc=kc, vc=vc, ks=ks, vs=vs, q=q, out=torch.zeros_like(q), cap=case["cap"], window=case["window"])
    if op == "tree":
        s["parents"], masks = _tree(len(n), case["nodes"], seed)
        s["masks"] = torch.from_numpy(masks.reshape(len(n) * case["nodes"], -1)).to(DEV)
    else:
        s["slopes"] = 2.0 ** (-8.0 * (torch.arange(case["hq"], device=DEV) + 1) / case["hq"]) if case["bias"] else None
        s["prefix"] = None
        if case["prefix"]:
            # a prefix of a prompt: some ends before the chunk, some inside it
            p = [int(x) for x in torch.randint(0, room + 1, (len(n),), generator=host)]
            s["prefix"] = torch.tensor([min(a, b) for a, b in zip(p, n)], dtype=torch.int32, device=DEV)
    if own:
        import paged_kv_cache_99_gb300 as pa
        s["workspace"] = pa.new_workspace_scored(len(n), case["hq"], hkv)
    return s


def _held(cache):
    """The cache's values: FP8 codes as the numbers they stand for (a view)."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def _store(cache, slots, bs, x, scale):
    block, off = slots // bs, slots % bs
    if scale is None:
        cache[block, :, off] = x.to(cache.dtype)
    else:
        y = (x / scale.view(1, -1, 1)).clamp(-448, 448)
        cache[block, :, off] = y.to(torch.float8_e4m3fn).view(torch.uint8)


def _norm_plain(s):
    hq, hkv, half = s["hq"], s["hkv"], s["rot"] // 2
    x = s["qkv"].float()
    w = torch.cat((s["wq"].float().expand(hq, D), s["wk"].float().expand(hkv, D)))
    y = x[:, :hq + hkv]
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    if s["axes"] is None:
        c = s["cos_sin"][s["positions"]]
        cos, sin = c[:, None, :half], c[:, None, half:]
    else:
        at = s["positions"][s["axes_dev"]].t()                     # [tokens, pairs]
        pair = torch.arange(half, device=DEV)
        cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, half + pair][:, None]
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if s["interleaved"] else (y[..., :half], y[..., half:2 * half])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, v), -1).flatten(-2) if s["interleaved"] else torch.cat((u, v), -1)
    y = torch.cat((turned, y[..., 2 * half:]), -1)
    s["q_out"].copy_(y[:, :hq].to(s["q_out"].dtype))
    _store(s["kc"], s["slots"], s["bs"], y[:, hq:], s["ks"])
    _store(s["vc"], s["slots"], s["bs"], x[:, hq + hkv:], s["vs"])
    return s["q_out"], _held(s["kc"]), _held(s["vc"])


def _rows32(s, cache, scale, i, n):
    """[H_kv, n, 128] in 32 bits: sequence i's rows in order."""
    t = torch.arange(n, device=DEV)
    x = _held(cache)[s["tables"][i].long()[t // s["bs"]], :, t % s["bs"]].float()
    if scale is not None:
        x = x * scale.view(1, -1, 1)
    return x.transpose(0, 1)


def _attention_plain(s):
    """Per sequence and KV head: scores, cap, bias, what is visible, softmax, product with V."""
    hkv, hq = s["hkv"], s["q"].shape[1]
    grp = hq // hkv
    first = 0
    for i, (n, m) in enumerate(zip(s["n"], s["rows"])):
        k, v = _rows32(s, s["kc"], s["ks"], i, n), _rows32(s, s["vc"], s["vs"], i, n)
        t = torch.arange(n, device=DEV)
        if s["op"] == "tree":
            bit = torch.arange(m, device=DEV)
            tree = (s["masks"][first:first + m][:, bit // 64] >> (bit % 64)) & 1
            pos = n - m + tree.sum(1) - 1                               # the context and the path above
            seen = torch.cat((torch.ones(m, n - m, dtype=torch.bool, device=DEV), tree.bool()), 1)
            if s["window"]:
                seen = seen & ((t >= n - m) | (pos[:, None] - t < s["window"]))
        else:
            pos = n - m + torch.arange(m, device=DEV)
            seen = t <= pos[:, None]
            if s["prefix"] is not None:
                seen = seen | (t < s["prefix"][i])
            if s["window"]:
                seen = seen & (pos[:, None] - t < s["window"])
        heads = 1 if m * n * grp > 1 << 24 else hkv                     # KV heads at a time
        for h in range(0, hkv, heads):
            q = s["q"][first:first + m, h * grp:(h + heads) * grp].float()
            q = q.view(m, heads, grp, D).permute(1, 2, 0, 3)            # [heads, group, rows, 128]
            x = torch.matmul(q, k[h:h + heads, None].transpose(2, 3)) * (1.0 / math.sqrt(D))
            if s["cap"]:
                x = s["cap"] * torch.tanh(x / s["cap"])
            if s["op"] == "scored" and s["slopes"] is not None:
                far = (pos[:, None] - t).abs().float()
                x = x - s["slopes"][h * grp:(h + heads) * grp].view(heads, grp, 1, 1) * far
            x = x.masked_fill(~seen, float("-inf"))
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - torch.where(top == float("-inf"), torch.zeros_like(top), top))
            p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
            y = torch.matmul(p, v[h:h + heads, None]).permute(2, 0, 1, 3).reshape(m, heads * grp, D)
            s["out"][first:first + m, h * grp:(h + heads) * grp] = y.to(s["out"].dtype)
        first += m
    return s["out"]


def _commit_plain(s):
    bs = s["bs"]
    depth = s["paths"].shape[1]
    base = s["lens"].long() - (s["start"][1:] - s["start"][:-1])        # cached tokens before the tree
    j = torch.arange(depth, device=DEV)
    live = j < s["path_lens"][:, None]
    rows = torch.arange(len(s["n"]), device=DEV)[:, None].expand(-1, depth)[live]
    src = (base[:, None] + s["paths"])[live]
    dst = (base[:, None] + j)[live]
    tables = s["tables"].long()
    src_b, dst_b = tables[rows, src // bs], tables[rows, dst // bs]
    for cache in s["kcs"] + s["vcs"]:
        cache[dst_b, :, dst % bs] = cache[src_b, :, src % bs]
    s["new_lens"].copy_(base + s["path_lens"])
    return [s["new_lens"]] + [_held(c) for c in s["kcs"] + s["vcs"]]


def _run_own(s):
    import paged_kv_cache_99_gb300 as pa
    if s["op"] == "norm":
        hq, hkv, qkv = s["hq"], s["hkv"], s["qkv"]
        pa.pa_norm_rope_and_cache(s["q_out"], qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], s["kc"], s["vc"],
                                  s["slots"], s["positions"], s["cos_sin"], s["wq"], s["wk"], eps=EPS,
                                  axes=s["axes_bytes"] if s["axes"] else None, interleaved=s["interleaved"],
                                  k_scale=s["ks"], v_scale=s["vs"])
        return s["q_out"], _held(s["kc"]), _held(s["vc"])
    if s["op"] == "tree":
        pa.pa_tree(s["out"], s["q"], s["start"], s["kc"], s["vc"], s["tables"], s["lens"], s["masks"], 1.0 / math.sqrt(D),
                   s["workspace"], cap=s["cap"], window=s["window"], k_scale=s["ks"], v_scale=s["vs"])
        return s["out"]
    if s["op"] == "commit":
        pa.pa_tree_commit(s["new_lens"], s["kcs"], s["vcs"], s["paths"], s["path_lens"], s["start"], s["tables"],
                          s["lens"])
        return [s["new_lens"]] + [_held(c) for c in s["kcs"] + s["vcs"]]
    pa.pa_mixed_scored(s["out"], s["q"], s["start"], s["kc"], s["vc"], s["tables"], s["lens"], 1.0 / math.sqrt(D),
                       s["workspace"], cap=s["cap"], slopes=s["slopes"], window=s["window"], prefix_lens=s["prefix"],
                       k_scale=s["ks"], v_scale=s["vs"])
    return s["out"]


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _norm_plain, "commit": _commit_plain}.get(s["op"], _attention_plain)(s)


def _seen(case, n, rows):
    """Keys that a sequence's rows see in all, and the keys that any of them sees."""
    w = case["window"] or n + 1
    if case["op"] == "tree":                    # a node sees its path: the tree's depth is left out
        return rows * min(n - rows, w), min(n, w + rows)
    if case["prefix"]:                          # on the average half of the prompt is open
        return rows * min(0.75 * n if rows > 1 else n, w), n
    return rows * min(n - (rows - 1) / 2, w), min(n, w + rows - 1)


def work(case):
    hkv = case["hkv"]
    e = 1 if case["cache"].startswith("fp8") else 2
    if case["op"] == "norm":
        t, hq, rot = case["tokens"], case["hq"], case["rot"]
        axes = len(case["sections"].split(","))
        # q in and out, k and v in, k and v into the cache, the table's rows, positions and slots
        return {"bytes": t * (4 * D * hq + 4 * D * hkv + 2 * D * e * hkv + 4 * rot + 8 * axes + 8),
                "flops": t * (hq + hkv) * (4 * D + 3 * rot)}
    if case["op"] == "commit":
        # on the average half the depth is accepted and half of that has moved, in and out
        moved = (case["depth"] + (case["batch"] - 1) * case["depth"] / 2) / 2
        return {"bytes": moved * case["layers"] * hkv * 4 * D * e, "flops": 0}
    hq = case["hq"]
    total = {"bytes": 0.0, "flops": 0.0}
    lens = _work_lengths(case)
    for i, n in enumerate(lens):
        if case["op"] == "tree":
            rows = case["nodes"]
            n += rows
        else:
            chunk = i >= len(lens) - case["chunks"]
            rows = case["rows"] if chunk else 1
            n = max(1, n, case["rows"] if chunk else 1)
        pairs, keys = _seen(case, n, rows)
        # K and V once, q and the outputs
        total["bytes"] += 2 * D * e * hkv * keys + 4 * D * hq * rows
        total["flops"] += 4 * D * hq * pairs
    return total


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    return _exact_commit(s) if case["op"] == "commit" else _exact_attention(s)


def _exact_norm(s):
    x = s["qkv"].double()
    hq, hkv, bs, half = s["hq"], s["hkv"], s["bs"], s["rot"] // 2
    for part, w in ((x[:, :hq], s["wq"]), (x[:, hq:hq + hkv], s["wk"])):
        part *= (part.pow(2).sum(-1, keepdim=True) / D + EPS).pow(-0.5)
        part *= w.double()
    axes = s["axes"] or [0] * half
    positions = s["positions"].reshape(-1, x.shape[0])
    table = s["cos_sin"].double()
    for i in range(half):
        c = table[positions[axes[i]]]
        one, two = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        z = torch.complex(x[:, :hq + hkv, one], x[:, :hq + hkv, two]) * torch.complex(c[:, i], c[:, half + i])[:, None]
        x[:, :hq + hkv, one], x[:, :hq + hkv, two] = z.real, z.imag
    caches = []
    for cache, scale, rows in ((s["kc"], s["ks"], x[:, hq:hq + hkv]), (s["vc"], s["vs"], x[:, hq + hkv:])):
        flat = _held(cache).double().transpose(1, 2).reshape(-1, hkv, D)          # [slot, head, 128]
        flat[s["slots"]] = rows if scale is None else (rows / scale.double().view(1, -1, 1)).clamp(-448, 448)
        caches.append(flat.view(-1, bs, hkv, D).transpose(1, 2).contiguous())
    return (x[:, :hq].contiguous(), *caches)


def _places(s, i, n):
    """Slots (of [pool * bs]) of sequence i's tokens, in order."""
    bs = s["bs"]
    blocks = s["tables"][i].tolist()
    return torch.tensor([blocks[t // bs] * bs + t % bs for t in range(n)], dtype=torch.long, device=DEV)


def _exact_visible(s, i, n, m):
    """bool [m, n] on the host, row by row from the definition; the position of each row."""
    t = np.arange(n)
    see = np.zeros((m, n), bool)
    pos = np.zeros(m, np.int64)
    for j in range(m):
        if s["op"] == "tree":
            depth, at = -1, j
            while at >= 0:                      # up the tree
                see[j, n - m + at] = True
                at = int(s["parents"][i, at])
                depth += 1
            pos[j] = n - m + depth
            low = max(0, int(pos[j]) - s["window"] + 1) if s["window"] else 0
            see[j, min(low, n - m):n - m] = True
        else:
            pos[j] = n - m + j
            high = pos[j] + 1 if s["prefix_host"] is None else max(pos[j] + 1, s["prefix_host"][i])
            see[j, (max(0, pos[j] - s["window"] + 1) if s["window"] else 0):high] = True
    return see, pos, t


def _exact_attention(s):
    hkv, hq = s["hkv"], s["q"].shape[1]
    grp = hq // hkv
    s["prefix_host"] = s["prefix"].tolist() if s.get("prefix") is not None else None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    row = 0
    for i, (n, m) in enumerate(zip(s["n"], s["rows"])):
        at = _places(s, i, n)
        see, pos, t = _exact_visible(s, i, n, m)
        some = torch.from_numpy(see.any(1)).to(DEV)
        block = torch.zeros(m, n, dtype=torch.float64, device=DEV)
        block[~torch.from_numpy(see).to(DEV)] = float("-inf")
        block[~some] = 0.0
        away = torch.from_numpy(np.abs(pos[:, None] - t)).to(DEV).double() if s.get("slopes") is not None else None
        k, v = ((_held(c)[at // s["bs"], :, at % s["bs"]].double() * (1.0 if z is None else z.double().view(1, -1, 1)))
                for c, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))               # [n, H_kv, 128]
        for h in range(hq):
            x = s["q"][row:row + m, h].double() @ k[:, h // grp].T / math.sqrt(D)
            if s["cap"]:
                x = torch.tanh(x / s["cap"]) * s["cap"]
            if away is not None:
                x = x - float(s["slopes"][h]) * away
            out[row:row + m, h] = torch.softmax(x + block, -1) @ v[:, h // grp] * some[:, None]
        row += m
    return out


def _exact_commit(s):
    bs, lens, paths = s["bs"], s["path_lens"].tolist(), s["paths"].tolist()
    caches = [_held(c).double() for c in s["kcs"] + s["vcs"]]
    src, dst, new = [], [], []
    for i, (n, m) in enumerate(zip(s["n"], s["rows"])):
        at = _places(s, i, n).tolist()
        for j in range(lens[i]):
            src.append(at[n - m + paths[i][j]])
            dst.append(at[n - m + j])
        new.append(n - m + lens[i])
    src, dst = (torch.tensor(x, dtype=torch.long, device=DEV) for x in (src, dst))
    for c in caches:
        c[dst // bs, :, dst % bs] = c[src // bs, :, src % bs]
    return [torch.tensor(new, dtype=torch.int32, device=DEV)] + caches
