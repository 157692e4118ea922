"""The operators of a bounded paged cache, as cases that can be measured: rotary
positions (their table, and the rotation fused with the slot write), a decode step
that also adds every cached token's attention weight to a running sum, and the
eviction of the tokens with the least of it.

``own`` says which side runs: the plain forms below (elementary torch in 32 bits, in
64 where 32 lose what matters) or the library's entry points on the same inputs.
"""
import math

import numpy as np
import torch

own = False

D = 128                     # head dimension of the library
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the table a server builds at start-up for a 32k context
        {"name": "table 32k", "op": "table", "positions": 32768, "rot": 128, "factor": 1.0},
        # the same for a context stretched 16 times past the trained length
        {"name": "table 512k stretched", "op": "table", "positions": 524288, "rot": 128, "factor": 16.0},
        # the smallest decode step (four sequences, one new token each): latency
        {"name": "rope 4 tokens", "op": "rope", "tokens": 4, "hq": 8, "hkv": 2, "rot": 128, "interleaved": False,
         "type": "bf16", "cache": "bf16", "bs": 16, "context": 32768},
        # a mixed step: 16 decode rows and two chunks of 512, half of each head rotated, FP8 cache
        {"name": "rope mixed fp8", "op": "rope", "tokens": 1040, "hq": 64, "hkv": 8, "rot": 64, "interleaved": True,
         "type": "bf16", "cache": "fp8", "bs": 16, "context": 32768},
        # a prefill step of a long prompt
        {"name": "rope prefill 16k", "op": "rope", "tokens": 16384, "hq": 32, "hkv": 8, "rot": 128,
         "interleaved": False, "type": "bf16", "cache": "bf16", "bs": 16, "context": 131072},
        # the smallest decode step: 4 sequences of 8 to 46 tokens
        {"name": "weights tiny", "op": "weights", "batch": 4, "lo": 8, "hi": 46, "hq": 8, "hkv": 2, "type": "bf16",
         "cache": "bf16", "bs": 16},
        # one layer of a 64-sequence decode step, 6 query heads to a KV head
        {"name": "weights 64 x 4k", "op": "weights", "batch": 64, "lo": 512, "hi": 4096, "hq": 12, "hkv": 2,
         "type": "bf16", "cache": "bf16", "bs": 16},
        # a few long rows over an FP8 cache, 8 query heads to a KV head
        {"name": "weights 16 x 32k fp8", "op": "weights", "batch": 16, "lo": 1024, "hi": 32768, "hq": 64, "hkv": 8,
         "type": "bf16", "cache": "fp8", "bs": 16},
        # one layer of a 40-sequence decode step at 8192 tokens each
        {"name": "weights 40 x 8k", "op": "weights", "batch": 40, "lo": 8192, "hi": 8192, "hq": 32, "hkv": 8,
         "type": "fp16", "cache": "fp16", "bs": 16},
        # one long request brought back to an eighth
        {"name": "evict 32k fp8", "op": "evict", "batch": 1, "lo": 32768, "hi": 32768, "hkv": 8, "budget": 4096,
         "sinks": 4, "recent": 512, "cache": "fp8", "bs": 16},
        # a batch of mixed lengths brought to 512 tokens each
        {"name": "evict 64 x 4k", "op": "evict", "batch": 64, "lo": 512, "hi": 4096, "hkv": 2, "budget": 512,
         "sinks": 4, "recent": 128, "cache": "bf16", "bs": 16},
        # one layer of 40 sequences at 8192 tokens brought to a quarter
        {"name": "evict 40 x 8k", "op": "evict", "batch": 40, "lo": 8192, "hi": 8192, "hkv": 8, "budget": 2048,
         "sinks": 4, "recent": 256, "cache": "fp16", "bs": 16},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("table", "rope", "rope", "weights", "weights", "evict", "evict"))
    if op == "table":
        rot = 16 * rng.randint(1, 8)
        return {"op": op, "positions": _spread(rng, 1000, 524288), "rot": rot,
                "factor": rng.choice((1.0, 2.0, 8.0, 40.0))}
    hkv = rng.choice((1, 2, 4, 5, 8))
    cache, kind = rng.choice((("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16"), ("fp8", "fp16"), ("fp8 heads", "bf16")))
    bs = rng.choice((8, 16, 32))
    if op == "rope":
        hq = hkv * rng.choice((1, 2, 3, 4, 6, 8))
        tokens = _spread(rng, 1, max(1, 16384 * 40 // max(40, hq + hkv)))
        return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "rot": 16 * rng.randint(1, 8),
                "interleaved": rng.random() < 0.5, "type": kind, "cache": cache, "bs": bs,
                "context": _spread(rng, max(tokens, 2048), 131072)}
    hi = _spread(rng, 1, 32768)
    lo = rng.choice((0, 1, hi // 4, hi))
    batch = _spread(rng, 1, min(128, max(1, 40 * 8192 * 8 // (hi * hkv))))
    if op == "weights":
        hq = hkv * rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12))
        return {"op": op, "batch": batch, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "type": kind, "cache": cache, "bs": bs}
    budget = _spread(rng, 1, max(1, hi // 2))
    sinks = rng.randint(0, min(budget, 8))
    return {"op": op, "batch": batch, "lo": lo, "hi": hi, "hkv": hkv, "budget": budget, "sinks": sinks,
            "recent": rng.randint(0, budget - sinks), "cache": cache, "bs": bs}


def _lengths(case, seed):
    """Cached tokens of each sequence: uniform in [lo, hi], the first one hi."""
    n = np.random.RandomState(seed % (1 << 31)).randint(case["lo"], case["hi"] + 1, case["batch"])
    n[0] = case["hi"]
    return [int(x) for x in n]


def _work_lengths(case):
    """The lengths work() counts: the first sequence at hi, the others at the mean."""
    return [case["hi"]] + [(case["lo"] + case["hi"]) / 2] * (case["batch"] - 1)


def _frequencies(rot, base, factor, trained=8192, low=1.0, high=32.0):
    """Rotary frequencies: unscaled for factor 1, else by parts (YaRN): a frequency that
    turns more than `high` times over the trained length stays, one that turns less than
    `low` times is divided by factor, the ones between are blended."""
    f = np.float64(base) ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)
    if factor == 1.0:
        return f
    keep = np.clip((trained * f / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
    return keep * f + (1.0 - keep) * f / factor


def _cache(shape, cache, g):
    """A cache of N(0, 1) values, and its scale (amax / 448 per tensor or head) if it is FP8."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if not cache.startswith("fp8"):
        return x.to(TYPES[cache]), None
    scale = x.abs().amax(dim=(0, 2, 3)) / 448 if cache == "fp8 heads" else (x.abs().max() / 448).reshape(1)
    return (x / scale.view(1, -1, 1, 1)).to(torch.float8_e4m3fn).view(torch.uint8), scale.contiguous()


def _tables(blocks, pool, g, first=0):
    """Block tables (-1 past a sequence's blocks) over a random permutation of the pool."""
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    t = torch.full((len(blocks), max(1, max(blocks))), -1, dtype=torch.int32)
    at = first
    for s, nb in enumerate(blocks):
        t[s, :nb] = perm[at:at + nb]
        at += nb
    return t, perm, at


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    if op == "table":
        base = 10000.0 * (1.0 + 99.0 * float(torch.rand((), generator=host, dtype=torch.float64)))
        return {"op": op, "freqs": _frequencies(case["rot"], base, case["factor"]),
                "attention": 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0,
                "cos_sin": torch.zeros(case["positions"], case["rot"], device=DEV)}
    bs, hkv = case["bs"], case["hkv"]
    if op == "rope":
        t, hq, rot = case["tokens"], case["hq"], case["rot"]
        pool = -(-t // bs) + 64
        slots = (torch.randperm(pool, generator=host)[:-(-t // bs)].repeat_interleave(bs) * bs +
                 torch.arange(bs).repeat(-(-t // bs)))[:t]
        qkv = torch.randn(t, hq + 2 * hkv, D, generator=g, device=DEV).to(TYPES[case["type"]])
        kc, ks = _cache((pool, hkv, bs, D), case["cache"], g)
        vc, vs = _cache((pool, hkv, bs, D), case["cache"], g)
        start = int(torch.randint(0, case["context"] - t + 1, (), generator=host))
        angle = torch.arange(case["context"], device=DEV, dtype=torch.float64)[:, None] * \
            torch.from_numpy(_frequencies(rot, 10000.0, 1.0)).to(DEV)
        return {"op": op, "qkv": qkv, "hq": hq, "hkv": hkv, "bs": bs, "slots": slots.to(DEV),
                "positions": (start + torch.arange(t)).to(DEV), "interleaved": case["interleaved"],
                "cos_sin": torch.cat((angle.cos(), angle.sin()), 1).float(), "kc": kc, "vc": vc, "ks": ks, "vs": vs,
                "q_out": torch.zeros(t, hq, D, device=DEV, dtype=qkv.dtype)}
    n = _lengths(case, seed)
    blocks = [-(-x // bs) for x in n]
    more = [-(-min(x, case["budget"]) // bs) for x in n] if op == "evict" else []
    # room for every sequence at its longest: the pool's size does not go by the lengths drawn
    pool = len(n) * (-(-case["hi"] // bs) + (-(-min(case["hi"], case["budget"]) // bs) if op == "evict" else 0)) + 16
    tables, perm, at = _tables(blocks, pool, host)
    kc, ks = _cache((pool, hkv, bs, D), case["cache"], g)
    vc, vs = _cache((pool, hkv, bs, D), case["cache"], g)
    width = tables.shape[1] * bs
    s = {"op": op, "bs": bs, "hkv": hkv, "kc": kc, "vc": vc, "ks": ks, "vs": vs, "tables": tables.to(DEV),
         "lens": torch.tensor(n, dtype=torch.int32, device=DEV), "n": n}
    # sums of many softmax weights are heavy-tailed; a tenth of the tokens were never looked at
    w = torch.exp(2 * torch.randn(len(n), hkv, width, generator=g, device=DEV) - 6)
    s["weights"] = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.1, torch.zeros_like(w), w)
    s["weights_out"] = torch.zeros_like(w)
    if op == "weights":
        s["q"] = torch.randn(len(n), case["hq"], D, generator=g, device=DEV).to(TYPES[case["type"]])
        s["out"] = torch.zeros_like(s["q"])
        if own:
            import paged_kv_cache_99_gb300 as pa
            s["workspace"] = pa.new_workspace_weights(len(n), case["hq"], hkv, sum(-(-x // 16) * 16 for x in n))
        return s
    t = torch.full((len(n), max(1, max(more))), -1, dtype=torch.int32)
    for i, nb in enumerate(more):
        t[i, :nb] = perm[at:at + nb]
        at += nb
    s.update(new_tables=t.to(DEV), budget=case["budget"], sinks=case["sinks"], recent=case["recent"],
             kept=torch.zeros(len(n), hkv, case["budget"], dtype=torch.int32, device=DEV),
             new_lens=torch.zeros(len(n), dtype=torch.int32, device=DEV))
    return s


def _held(cache):
    """The cache's values: FP8 codes as the numbers they stand for (a view)."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def _table_plain(s):
    p = torch.arange(s["cos_sin"].shape[0], device=DEV, dtype=torch.float64)
    angle = p[:, None] * torch.from_numpy(s["freqs"]).to(DEV)
    s["cos_sin"].copy_((torch.cat((angle.cos(), angle.sin()), 1) * s["attention"]).float())
    return s["cos_sin"]


def _rotate(x, c, interleaved):
    """x [T, H, 128] in 32 bits, rotated in its first rot components by c = (cos, sin) [T, 1, rot]."""
    half = c.shape[-1] // 2
    cos, sin = c[..., :half], c[..., half:]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _store(cache, slots, bs, x, scale):
    block, off = slots // bs, slots % bs
    if scale is None:
        cache[block, :, off] = x.to(cache.dtype)
    else:
        y = (x / scale.view(1, -1, 1)).clamp(-448, 448)
        cache[block, :, off] = y.to(torch.float8_e4m3fn).view(torch.uint8)


def _rope_plain(s):
    hq, hkv = s["hq"], s["hkv"]
    x = s["qkv"].float()
    turned = _rotate(x[:, :hq + hkv], s["cos_sin"][s["positions"]][:, None], s["interleaved"])
    s["q_out"].copy_(turned[:, :hq].to(s["q_out"].dtype))
    _store(s["kc"], s["slots"], s["bs"], turned[:, hq:], s["ks"])
    _store(s["vc"], s["slots"], s["bs"], x[:, hq + hkv:], s["vs"])
    return s["q_out"], _held(s["kc"]), _held(s["vc"])


def _gathered(cache, scale, tables, bs):
    """[B, H_kv, N, 128] in 32 bits: every sequence's rows in order (rows past its length are anything)."""
    t = torch.arange(tables.shape[1] * bs, device=DEV)
    x = _held(cache)[tables.clamp(min=0).long()[:, t // bs], :, t % bs].float()
    if scale is not None:
        x = x * scale.view(1, 1, -1, 1)
    return x.transpose(1, 2)


def _weights_plain(s):
    b, hq, _ = s["q"].shape
    hkv = s["hkv"]
    k = _gathered(s["kc"], s["ks"], s["tables"], s["bs"])
    live = (torch.arange(k.shape[2], device=DEV) < s["lens"][:, None])[:, None]
    x = torch.matmul(s["q"].float().view(b, hkv, hq // hkv, D), k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~live[:, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    v = _gathered(s["vc"], s["vs"], s["tables"], s["bs"]).masked_fill(~live[..., None], 0.0)
    s["out"].copy_(torch.matmul(p, v).view(b, hq, D).to(s["out"].dtype))
    s["weights_out"].copy_(torch.where(live, s["weights"] + p.sum(2), s["weights_out"]))
    return s["out"], s["weights_out"]


def _evict_plain(s):
    w, lens, budget, bs = s["weights"], s["lens"].long(), s["budget"], s["bs"]
    b, hkv, width = w.shape
    t = torch.arange(width, device=DEV)
    n = lens[:, None, None]
    sure = (t < s["sinks"]) | (t >= n - s["recent"])
    # the tokens that stay whatever their weight first, then by weight, then by place; none past the end
    key = torch.where(sure, torch.full_like(w, float("inf")), w).masked_fill(t >= n, float("-inf"))
    order = torch.argsort(key, dim=-1, descending=True, stable=True)[..., :budget]
    if order.shape[-1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]))
    left = torch.minimum(lens, torch.full_like(lens, budget))
    j = torch.arange(budget, device=DEV)
    there = (j < left[:, None, None]).expand(b, hkv, budget)
    kept = torch.where(there, order, torch.full_like(order, width)).sort(-1).values
    at = kept.clamp(max=width - 1)
    rows, heads = torch.arange(b, device=DEV)[:, None, None], torch.arange(hkv, device=DEV)[None, :, None]
    src = s["tables"].long()[rows, at // bs][there]
    off = (at % bs)[there]
    to = s["new_tables"].long()[rows, (j // bs)[None, None]].expand(b, hkv, budget)[there]
    to_off = (j % bs).expand(b, hkv, budget)[there]
    h = heads.expand(b, hkv, budget)[there]
    s["kc"][to, h, to_off] = s["kc"][src, h, off]
    s["vc"][to, h, to_off] = s["vc"][src, h, off]
    new = torch.zeros_like(w)
    new[..., :min(width, budget)] = torch.where(there, w.gather(-1, at), torch.zeros_like(w[..., :1]))[..., :width]
    s["weights_out"].copy_(torch.where(t < n, new, s["weights_out"]))
    s["kept"].copy_(torch.where(there, kept, torch.full_like(kept, -1)))
    s["new_lens"].copy_(left)
    return s["kept"], s["new_lens"], s["weights_out"], _held(s["kc"]), _held(s["vc"])


def _run_own(s):
    import paged_kv_cache_99_gb300 as pa
    if s["op"] == "table":
        pa.pa_rope_table(s["cos_sin"], s["freqs"], s["attention"])
        return s["cos_sin"]
    if s["op"] == "rope":
        hq, hkv = s["hq"], s["hkv"]
        qkv = s["qkv"]
        pa.pa_rope_and_cache(s["q_out"], qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], s["kc"], s["vc"],
                             s["slots"], s["positions"], s["cos_sin"], interleaved=s["interleaved"],
                             k_scale=s["ks"], v_scale=s["vs"])
        return s["q_out"], _held(s["kc"]), _held(s["vc"])
    if s["op"] == "weights":
        pa.pa_decode_weights(s["out"], s["weights_out"], s["q"], s["kc"], s["vc"], s["tables"], s["lens"],
                             1.0 / math.sqrt(D), s["workspace"], weights_in=s["weights"], k_scale=s["ks"],
                             v_scale=s["vs"])
        return s["out"], s["weights_out"]
    pa.pa_evict(s["kept"], s["new_lens"], s["weights_out"], s["weights"], s["kc"], s["vc"], s["tables"], s["lens"],
                s["new_tables"], budget=s["budget"], sinks=s["sinks"], recent=s["recent"])
    return s["kept"], s["new_lens"], s["weights_out"], _held(s["kc"]), _held(s["vc"])


def run(s):
    if own:
        return _run_own(s)
    return {"table": _table_plain, "rope": _rope_plain, "weights": _weights_plain, "evict": _evict_plain}[s["op"]](s)


def work(case):
    if case["op"] == "table":
        return {"bytes": 4 * case["positions"] * case["rot"], "flops": 0}
    e = 1 if case["cache"].startswith("fp8") else 2
    hkv = case["hkv"]
    if case["op"] == "rope":
        t, hq, rot = case["tokens"], case["hq"], case["rot"]
        # q in and out, k and v in, k and v into the cache, the table's rows, positions and slots
        return {"bytes": t * (4 * D * hq + 4 * D * hkv + 2 * D * e * hkv + 4 * rot + 16), "flops": 3 * t * rot * (hq + hkv)}
    n = _work_lengths(case)
    if case["op"] == "weights":
        rows = hkv * sum(n)
        # K and V once, the running weights in and out, q and the outputs
        return {"bytes": rows * (2 * D * e + 8) + 4 * D * case["hq"] * len(n), "flops": 4 * D * case["hq"] * sum(n)}
    kept = hkv * sum(min(x, case["budget"]) for x in n)
    # the weights in and out, the kept rows of K and V in and out, their places
    return {"bytes": hkv * sum(n) * 8 + kept * (4 * D * e + 4), "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "table":
        p = torch.arange(case["positions"], dtype=torch.float64, device=DEV)
        turns = torch.outer(p, torch.as_tensor(s["freqs"], device=DEV))
        return torch.hstack((torch.cos(turns), torch.sin(turns))) * s["attention"]
    if op == "rope":
        return _exact_rope(s)
    return _exact_weights(s) if op == "weights" else _exact_evict(s)


def _exact_rope(s):
    x = s["qkv"].double()
    hq, hkv, bs = s["hq"], s["hkv"], s["bs"]
    c = s["cos_sin"].double()[s["positions"]]
    half = c.shape[1] // 2
    i = torch.arange(half, device=DEV)
    one, two = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    z = torch.complex(x[:, :hq + hkv, one], x[:, :hq + hkv, two]) * torch.complex(c[:, :half], c[:, half:])[:, None]
    x[:, :hq + hkv, one], x[:, :hq + hkv, two] = z.real, z.imag
    caches = []
    for cache, scale, rows in ((s["kc"], s["ks"], x[:, hq:hq + hkv]), (s["vc"], s["vs"], x[:, hq + hkv:])):
        flat = _held(cache).double().transpose(1, 2).reshape(-1, hkv, D)          # [slot, head, 128]
        flat[s["slots"]] = rows if scale is None else rows / scale.double().view(1, -1, 1)
        caches.append(flat.view(-1, bs, hkv, D).transpose(1, 2).contiguous())
    return (x[:, :hq].contiguous(), *caches)


def _rows_of(s, i):
    """Slots (of [pool * bs]) of sequence i's cached tokens, in order."""
    bs, n = s["bs"], s["n"][i]
    blocks = s["tables"][i].tolist()
    return torch.tensor([blocks[t // bs] * bs + t % bs for t in range(n)], dtype=torch.long, device=DEV)


def _exact_weights(s):
    b, hq, _ = s["q"].shape
    hkv, bs = s["hkv"], s["bs"]
    out = torch.zeros(b, hq, D, dtype=torch.float64, device=DEV)
    new = s["weights_out"].double()
    for i in range(b):
        n = s["n"][i]
        if n == 0:
            continue
        at = _rows_of(s, i)
        k, v = ((_held(c)[at // bs, :, at % bs].double() * (1.0 if z is None else z.double().view(1, -1, 1)))
                for c, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))                    # [n, H_kv, 128]
        for h in range(hkv):
            q = s["q"][i, h * (hq // hkv):(h + 1) * (hq // hkv)].double()
            p = torch.softmax(q @ k[:, h].T / math.sqrt(D), -1)
            out[i, h * (hq // hkv):(h + 1) * (hq // hkv)] = p @ v[:, h]
            new[i, h, :n] = s["weights"][i, h, :n].double() + p.sum(0)
    return out, new


def _exact_evict(s):
    budget, hkv, bs = s["budget"], s["hkv"], s["bs"]
    caches = [_held(s["kc"]).double(), _held(s["vc"]).double()]
    kept = np.full((len(s["n"]), hkv, budget), -1, np.int32)
    new = s["weights_out"].double()
    w = s["weights"].cpu().numpy().astype(np.float64)
    for i, n in enumerate(s["n"]):
        m = min(n, budget)
        at = _rows_of(s, i)
        to = s["new_tables"][i].tolist()
        to = torch.tensor([to[j // bs] * bs + j % bs for j in range(m)], dtype=torch.long, device=DEV)
        for h in range(hkv if n else 0):
            place = np.arange(n)
            sure = (place < s["sinks"]) | (place >= n - s["recent"])
            order = np.lexsort((place, -w[i, h, :n], ~sure))
            pick = np.sort(order[:m])
            kept[i, h, :m] = pick
            pick = torch.from_numpy(pick).to(DEV)
            for c in caches:
                c[to // bs, h, to % bs] = c[at[pick] // bs, h, at[pick] % bs]
            new[i, h, :n] = 0
            new[i, h, :m] = s["weights"][i, h][pick].double()
    return (torch.from_numpy(kept).to(DEV), torch.tensor([min(x, budget) for x in s["n"]], dtype=torch.int32, device=DEV),
            new, *caches)
