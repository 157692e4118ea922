"""A bounded cache from end to end, as a server runs it: prompts written with rotary
positions, decode steps that add up attention weights, evictions into fresh blocks of
the pool, and further steps whose positions go on counting past the cache's length.
Checked against a float64 simulation that holds every sequence's kept tokens per KV
head as plain lists."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_99_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, BS, ROT, BASE = 8, 2, 16, 64, 10000.0
BUDGET, SINKS, RECENT = 48, 2, 8
TOL = 1e-2                      # |gpu - ref| <= 1e-2 + 1e-2 |ref|, the attention tolerance of every parity test


def _turn(x, p, f, interleaved):
    y = x.copy()
    half = len(f)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    c, s = np.cos(p * f), np.sin(p * f)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_prompt_decode_evict_decode(cache, interleaved, graph):
    g = torch.Generator().manual_seed(77)
    prompts, steps = [40, 75, 11], 12
    B, T = len(prompts), sum(prompts)
    pool = pa.BlockPool(96, BS)
    tables = [pool.allocate(-(-(n + steps) // BS)) for n in prompts]
    width = max(map(len, tables))
    bt = torch.full((B, width), -1, dtype=torch.int32)
    for s, row in enumerate(tables):
        bt[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
    bt = bt.to(DEV)
    dt = torch.uint8 if cache == "fp8" else torch.bfloat16
    kc = torch.zeros(96, HKV, BS, 128, dtype=dt, device=DEV)
    vc = torch.zeros_like(kc)
    scales = dict(k_scale=torch.tensor([0.02], device=DEV), v_scale=torch.tensor([0.015], device=DEV)) if cache == "fp8" else {}
    f = pa.pa_rope_frequencies(ROT, BASE)
    cos_sin = torch.empty(256, ROT, device=DEV)
    pa.pa_rope_table(cos_sin, f)
    ws = pa.new_workspace_weights(B, HQ, HKV, B * width * BS)
    acc = torch.zeros(B, HKV, width * BS, device=DEV)

    # the simulation: per sequence and head the stored keys and values (what the cache's bits
    # stand for) and the running weights
    keys, vals, sums = ([[[] for _ in range(HKV)] for _ in range(B)] for _ in range(3))

    def held(c, slot, h, scale):
        x = c[slot // BS, h, slot % BS]
        return x.view(torch.float8_e4m3fn).double().cpu().numpy() * float(scale) if cache == "fp8" else x.double().cpu().numpy()

    def note(s, slot, k_want, v_want):
        for h in range(HKV):
            for store, c, want, name in ((keys, kc, k_want, "k_scale"), (vals, vc, v_want, "v_scale")):
                scale = scales.get(name, 1.0)
                got = held(c, slot, h, scale)
                off = 2.0 ** -4 * np.abs(want[h]) + 2.0 ** -10 * float(scale) if cache == "fp8" else 2.0 ** -8 * np.abs(want[h])
                assert np.all(np.abs(got - want[h]) <= off + 1e-5)
                store[s][h].append(got)
            sums[s][h].append(0.0)

    # prompts
    qkv = torch.randn(T, HQ + 2 * HKV, 128, generator=g).bfloat16().to(DEV)
    pos = np.concatenate([np.arange(n) for n in prompts])
    slots = np.concatenate([[tables[s][t // BS] * BS + t % BS for t in range(n)] for s, n in enumerate(prompts)])
    q_out = torch.empty(T, HQ, 128, dtype=torch.bfloat16, device=DEV)
    pa.pa_rope_and_cache(q_out, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], kc, vc,
                         torch.from_numpy(slots).to(DEV), torch.from_numpy(pos).to(DEV), cos_sin, interleaved=interleaved,
                         workspace=ws, **scales)
    x = qkv.double().cpu().numpy()
    i = 0
    for s, n in enumerate(prompts):
        for t in range(n):
            note(s, int(slots[i]), _turn(x[i, HQ:HQ + HKV], t, f, interleaved), x[i, HQ + HKV:])
            i += 1

    # decode steps over fixed buffers, as a captured step would hold them
    lens = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    step_qkv = torch.zeros(B, HQ + 2 * HKV, 128, dtype=torch.bfloat16, device=DEV)
    step_slots, step_pos = (torch.zeros(B, dtype=torch.int64, device=DEV) for _ in range(2))
    q_rot, out = (torch.zeros(B, HQ, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def step():
        pa.pa_rope_and_cache(q_rot, step_qkv[:, :HQ], step_qkv[:, HQ:HQ + HKV], step_qkv[:, HQ + HKV:], kc, vc, step_slots,
                             step_pos, cos_sin, interleaved=interleaved, workspace=ws, **scales)
        pa.pa_decode_weights(out, acc, q_rot, kc, vc, bt, lens, 1 / math.sqrt(128), ws, weights_in=acc, **scales)

    captured = None
    if graph:
        # padding while the step is warmed up and captured: nothing is written or attended
        keep = lens.clone()
        lens.zero_()
        step_slots.fill_(-1)
        step_pos.fill_(-1)
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        lens.copy_(keep)
    host_lens, seen = list(prompts), list(prompts)
    for it in range(steps):
        if it in (4, 9):
            # eviction into fresh blocks; the old ones go back to the pool
            new = [pool.allocate(-(-(min(n, BUDGET) + steps) // BS)) for n in host_lens]
            nt = torch.full((B, max(map(len, new))), -1, dtype=torch.int32)
            for s, row in enumerate(new):
                nt[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
            kept = torch.empty(B, HKV, BUDGET, dtype=torch.int32, device=DEV)
            new_lens = torch.empty_like(lens)
            before = acc.double().cpu().numpy()
            pa.pa_evict(kept, new_lens, acc, acc, kc, vc, bt, lens, nt.to(DEV), BUDGET, SINKS, RECENT, workspace=ws)
            got = kept.cpu().numpy()
            for s, n in enumerate(host_lens):
                m = min(n, BUDGET)
                for h in range(HKV):
                    t = np.arange(n)
                    sure = (t < SINKS) | (t >= n - RECENT)
                    # the choice goes by the running sums as the cache holds them (float32)
                    pick = np.sort(np.lexsort((t, -before[s, h, :n], ~sure))[:m]) if n > BUDGET else t
                    assert np.array_equal(got[s, h, :m], pick)
                    for store in (keys, vals, sums):
                        store[s][h] = [store[s][h][j] for j in pick]
                host_lens[s] = m
            lens.copy_(new_lens)
            assert lens.tolist() == host_lens
            for row in tables:
                pool.free(row)
            tables = new
            bt.fill_(-1)
            bt[:, :nt.shape[1]] = nt[:, :width].to(DEV) if nt.shape[1] > width else nt.to(DEV)
        new_qkv = torch.randn(B, HQ + 2 * HKV, 128, generator=g).bfloat16()
        step_qkv.copy_(new_qkv)
        at = [tables[s][n // BS] * BS + n % BS for s, n in enumerate(host_lens)]
        step_slots.copy_(torch.tensor(at))
        step_pos.copy_(torch.tensor(seen))
        lens += 1
        (captured.replay if graph else step)()
        torch.cuda.synchronize()
        assert pa.pa_read_device_status(ws) == pa.PA_OK
        x = new_qkv.double().numpy()
        got, running = out.double().cpu().numpy(), acc.double().cpu().numpy()
        for s in range(B):
            note(s, at[s], _turn(x[s, HQ:HQ + HKV], seen[s], f, interleaved), x[s, HQ + HKV:])
            host_lens[s] += 1
            q = q_rot[s].double().cpu().numpy()
            want = _turn(x[s, :HQ], seen[s], f, interleaved)
            assert np.all(np.abs(q - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)
            seen[s] += 1
            for h in range(HKV):
                k, v = np.stack(keys[s][h]), np.stack(vals[s][h])
                for e in range(HQ // HKV):
                    z = k @ q[h * HQ // HKV + e] / math.sqrt(128)
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    ref = p @ v
                    assert np.all(np.abs(got[s, h * HQ // HKV + e] - ref) <= TOL + TOL * np.abs(ref))
                    sums[s][h] = [a + b for a, b in zip(sums[s][h], p)]
                # a step's weights are off by under 1e-4 of themselves, each sum by 2^-24 of it
                np.testing.assert_allclose(running[s, h, :host_lens[s]], sums[s][h], rtol=2e-4, atol=1e-9)
                assert np.all(running[s, h, host_lens[s]:] == 0)
    assert max(seen) > max(host_lens)                # positions ran on past the cache


def test_blocks_beyond_four_gigabytes():
    # every row the calls touch lies past 2^32 bytes into the caches
    nb, bs = 1_200_000, 16                       # 4096 bytes a block and head: 4.9 GB per cache
    far = 1_100_000
    kc = torch.empty(nb, 1, bs, 128, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    kc[far:], vc[far:] = float("nan"), float("nan")
    T = 100
    blocks = torch.randperm(nb - far, generator=torch.Generator().manual_seed(3))[:14] + far
    qkv = torch.randn(T, 6, 128, generator=torch.Generator().manual_seed(4)).bfloat16().to(DEV)
    slots = (blocks[torch.arange(T) // bs] * bs + torch.arange(T) % bs).to(DEV)
    cos_sin = torch.empty(T, 64, device=DEV)
    pa.pa_rope_table(cos_sin, pa.pa_rope_frequencies(64))
    q = torch.empty(T, 4, 128, dtype=torch.bfloat16, device=DEV)
    pa.pa_rope_and_cache(q, qkv[:, :4], qkv[:, 4:5], qkv[:, 5:], kc, vc, slots, torch.arange(T, device=DEV), cos_sin)
    # the same into a small cache
    kn, vn = (torch.empty(7, 1, bs, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    qn = torch.empty_like(q)
    pa.pa_rope_and_cache(qn, qkv[:, :4], qkv[:, 4:5], qkv[:, 5:], kn, vn, torch.arange(T, device=DEV),
                         torch.arange(T, device=DEV), cos_sin)
    assert torch.equal(q, qn)
    at = blocks[:7].to(DEV)
    rows = lambda c: c.reshape(-1, 128)[:T]  # noqa: E731
    assert torch.equal(rows(kc[at]), rows(kn)) and torch.equal(rows(vc[at]), rows(vn))
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    ws = pa.new_workspace_weights(1, 4, 1, 112)
    tables = [blocks[None, :7].int().to(DEV), torch.arange(7, dtype=torch.int32, device=DEV)[None]]
    out, w = [], []
    for (k, v), t in zip(((kc, vc), (kn, vn)), tables):
        out.append(torch.empty(1, 4, 128, dtype=torch.bfloat16, device=DEV))
        w.append(torch.zeros(1, 1, 112, device=DEV))
        pa.pa_decode_weights(out[-1], w[-1], q[-1:], k, v, t, lens, 0.088, ws)
    assert torch.equal(out[0], out[1]) and torch.equal(w[0], w[1])
    kept = torch.empty(1, 1, 40, dtype=torch.int32, device=DEV)
    new_lens = torch.empty_like(lens)
    new = blocks[7:10]
    pa.pa_evict(kept, new_lens, w[1], w[0], kc, vc, tables[0], lens, new[None].int().to(DEV), 40, 2, 8, workspace=ws)
    pick = torch.topk(w[0][0, 0, 2:92], 30).indices.sort().values.cpu() + 2
    pick = torch.cat((torch.arange(2), pick, torch.arange(92, 100)))
    assert torch.equal(kept[0, 0].cpu(), pick.int())
    assert torch.equal(kc[new.to(DEV)].reshape(-1, 128)[:40], rows(kn)[pick.to(DEV)])
    assert torch.equal(vc[new.to(DEV)].reshape(-1, 128)[:40], rows(vn)[pick.to(DEV)])
    assert pa.pa_read_device_status(ws) == pa.PA_OK


def test_two_graphs_share_a_workspace():
    # two captured decode steps over one workspace, replayed in turns beside eager calls
    g = torch.Generator(device=DEV).manual_seed(9)
    lens = [[300, 17, 2000, 1], [64, 900]]
    ws = pa.new_workspace_weights(4, 8, 2, 4 * 2000)
    calls = []
    for n in lens:
        nb = [-(-x // BS) for x in n]
        t = torch.full((len(n), max(nb)), -1, dtype=torch.int32)
        perm = torch.randperm(sum(nb), generator=torch.Generator().manual_seed(len(n))).int()
        for s, b in enumerate(nb):
            t[s, :b] = perm[sum(nb[:s]):sum(nb[:s]) + b]
        kc, vc = (torch.randn(sum(nb), 2, BS, 128, generator=g, device=DEV).bfloat16() for _ in range(2))
        q = torch.randn(len(n), 8, 128, generator=g, device=DEV).bfloat16()
        calls.append(dict(q=q, k_cache=kc, v_cache=vc, block_tables=t.to(DEV), scale=0.088, workspace=ws,
                          seq_lens=torch.tensor(n, dtype=torch.int32, device=DEV),
                          out=torch.empty_like(q), weights_out=torch.zeros(len(n), 2, max(nb) * BS, device=DEV)))
    want, graphs = [], []
    for c in calls:
        pa.pa_decode_weights(**c)
        want.append((c["out"].clone(), c["weights_out"].clone()))
    torch.cuda.synchronize()
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pa.pa_decode_weights(**c)
    for i in (0, 1, 1, 0, 0, 1):
        for c in calls:
            c["out"].zero_()
            c["weights_out"].zero_()
        graphs[i].replay()
        pa.pa_decode_weights(**calls[1 - i])
        for c, (o, w) in zip(calls, want):
            assert torch.equal(c["out"], o) and torch.equal(c["weights_out"], w)
    assert pa.pa_read_device_status(ws) == pa.PA_OK
