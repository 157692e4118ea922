"""Batches over a paged cache for the operators with scores or masks that are not plain, and
their attention in float64 from the definition, row by row what it sees."""
import numpy as np
import torch

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Batch:
    """lens: cached tokens of each sequence, the rows' own among them; rows: query rows of each.
    Slots that hold no token are NaN, table entries behind a sequence are -1."""

    def __init__(self, seed, lens, rows, hq, hkv, cache="bf16", kind="bf16", bs=16, per_head=False, spare=3, q_size=2.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        host = torch.Generator().manual_seed(seed)
        self.lens_h, self.rows_h, self.hq, self.hkv, self.bs, self.cache, self.kind = lens, rows, hq, hkv, bs, cache, kind
        blocks = [-(-n // bs) for n in lens]
        pool = sum(blocks) + spare
        perm = torch.randperm(pool, generator=host).to(torch.int32)
        width = max(1, max(blocks, default=1)) + 1
        t = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for s, nb in enumerate(blocks):
            t[s, :nb] = perm[at:at + nb]
            at += nb
        self.tables = t.to(DEV)
        self.ks = self.vs = None
        self.k, self.v = [], []             # float64 rows of each sequence
        self.caches = []
        for which in range(2):
            x = torch.randn(pool, hkv, bs, 128, generator=g, device=DEV)
            if cache == "fp8":
                scale = x.abs().amax(dim=(0, 2, 3)) / 448 if per_head else (x.abs().max() / 448).reshape(1)
                c = (x / scale.view(1, -1, 1, 1)).to(torch.float8_e4m3fn)
                held = c.double() * scale.double().view(1, -1, 1, 1)
                c = c.view(torch.uint8)
                if which:
                    self.vs = scale.contiguous()
                else:
                    self.ks = scale.contiguous()
            else:
                c = x.to(TYPES[cache])
                held = c.double()
            live = torch.zeros(pool, bs, dtype=torch.bool, device=DEV)
            for s, n in enumerate(lens):
                p = torch.arange(n, device=DEV)
                live[self.tables[s].long()[p // bs], p % bs] = True
                (self.v if which else self.k).append(held[self.tables[s].long()[p // bs], :, p % bs])
            dead = ~live[:, None, :, None].expand_as(c)
            c[dead] = 0x7F if cache == "fp8" else float("nan")
            self.caches.append(c.contiguous())
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        start = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
        self.start_h = start
        self.start = torch.from_numpy(start).to(DEV)
        self.q = (torch.randn(int(start[-1]), hq, 128, generator=g, device=DEV) * q_size).to(TYPES[kind])
        self.scale = 128 ** -0.5

    def args(self):
        return dict(k_scale=self.ks, v_scale=self.vs)


def causal(b, window=0, prefix=None):
    """What each row of pa_mixed_scored sees: per sequence (bool [rows, n], positions [rows])."""
    out = []
    for s, (n, m) in enumerate(zip(b.lens_h, b.rows_h)):
        t = torch.arange(n, device=DEV)
        pos = n - m + torch.arange(m, device=DEV)
        see = t <= pos[:, None]
        if prefix is not None:
            see = see | (t < prefix[s])
        if window:
            see = see & (pos[:, None] - t < window)
        out.append((see, pos))
    return out


def tree_sight(b, parents, window=0, blind=()):
    """The same for pa_tree, up every node's path; rows in `blind` see no node.  Also the masks."""
    words = max(1, max(-(-m // 64) for m in b.rows_h))
    masks = np.zeros((sum(b.rows_h), words), np.uint64)
    out = []
    for s, (n, m) in enumerate(zip(b.lens_h, b.rows_h)):
        see = np.zeros((m, n), bool)
        pos = np.zeros(m, np.int64)
        for j in range(m):
            row = int(b.start_h[s]) + j
            depth, at = -1, j
            while at >= 0 and row not in blind:
                see[j, n - m + at] = True
                masks[row, at // 64] |= np.uint64(1) << np.uint64(at % 64)
                at = int(parents[s][at])
                depth += 1
            pos[j] = n - m + max(depth, 0)      # a row that sees no node: the first one's place
            low = max(0, pos[j] - window + 1) if window else 0
            see[j, min(low, n - m):n - m] = True
        out.append((torch.from_numpy(see).to(DEV), torch.from_numpy(pos).to(DEV)))
    return out, torch.from_numpy(masks.view(np.int64)).to(DEV)


def random_trees(b, seed):
    r = np.random.RandomState(seed)
    return [[-1] + [int(r.randint(max(0, i - 5), i)) if r.rand() < 0.6 else int(r.randint(0, i)) for i in range(1, m)]
            for m in b.rows_h]


def reference(b, sight, cap=0.0, slopes=None):
    """(want, tolerance), float64 [rows, H_q, 128].

    Tolerance.  A score is a float32 sum of 128 exact products in some order: off by at most
    128 x 2^-23 of the sum of their magnitudes times the scale; the products by scales, the cap
    and the bias by 2^-18 of the score's and the bias's size (the cap: an exponential, a
    reciprocal or a polynomial of relative error 2^-20 on values up to the score).  With scores
    within e a weight is within a factor exp(2 e).  The probabilities are rounded to 16 bits
    (u = 2^-8 bf16, 2^-11 fp16, FP8 caches' type too, and 2^-25 absolutely where fp16 has no
    normal numbers), exponential and sum add 2^-19; the output is rounded once."""
    u_p = 2.0 ** -8 if b.cache == "bf16" else 2.0 ** -11
    u_o = 2.0 ** -8 if b.kind == "bf16" else 2.0 ** -11
    want = torch.zeros(b.q.shape, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(want)
    grp = b.hq // b.hkv
    for s, (see, pos) in enumerate(sight):
        n, m, r0 = b.lens_h[s], b.rows_h[s], int(b.start_h[s])
        if m == 0 or n == 0:
            continue
        q = b.q[r0:r0 + m].double().view(m, b.hkv, grp, 128)
        x = torch.einsum("mhgd,nhd->mhgn", q, b.k[s]) * b.scale
        size = torch.einsum("mhgd,nhd->mhgn", q.abs(), b.k[s].abs()) * abs(b.scale)
        e = 128 * 2.0 ** -23 * size + 2.0 ** -18 * x.abs()
        if b.cache == "fp8":                # the query as fp16: below its normal range 2^-25 off
            e = e + 2.0 ** -25 * b.k[s].abs().sum(-1).T[None, :, None] * abs(b.scale)
        if cap:
            x = cap * torch.tanh(x / cap)
        if slopes is not None:
            far = (pos[:, None] - torch.arange(n, device=DEV)).abs().double()
            bias = slopes.double().view(1, b.hkv, grp, 1) * far[:, None, None]
            x = x - bias
            # the bias of a row's nearest key is taken off as well: sizes that matter stay near it
            e = e + 2.0 ** -21 * bias
        hide = ~see[:, None, None]
        x = x.masked_fill(hide, float("-inf"))
        top = x.amax(-1, keepdim=True)
        w = torch.exp(x - torch.where(top.isinf(), torch.zeros_like(top), top))
        some = see.any(1)[:, None, None, None]
        p = torch.where(some, w / w.sum(-1, keepdim=True).clamp(min=1e-300), torch.zeros_like(w))
        # errors of keys far below the top do not matter: what their weight is off by at most
        off = torch.expm1(2 * e.masked_fill(hide, 0.0)) * p
        pv = torch.einsum("mhgn,nhd->mhgd", p, b.v[s])
        pa_ = torch.einsum("mhgn,nhd->mhgd", p * (u_p + 2.0 ** -19) + off + (off.sum(-1, keepdim=True)) * p, b.v[s].abs())
        if u_p < 2.0 ** -10:
            pa_ = pa_ + 2.0 ** -25 * torch.einsum("mn,nhd->mhd", see.double(), b.v[s].abs())[:, :, None]
        want[r0:r0 + m] = pv.reshape(m, b.hq, 128)
        t = pa_ + u_o * (pv.abs() + pa_) + (2.0 ** -25 if b.kind == "fp16" else 0.0)
        tol[r0:r0 + m] = t.reshape(m, b.hq, 128)
    return want, tol


def check(got, want, tol, what=""):
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    off = (got.double() - want).abs()
    bad = off > tol
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((off - tol).max()):.3e}, "
                                 f"first {bad.nonzero()[0].tolist()}")
