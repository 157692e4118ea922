// Eviction of the cached tokens with the least accumulated attention weight, sm_103a.
//
// For every sequence and KV head the first `sinks` and the last `recent` tokens stay,
// and of the tokens between them those of the largest weights, `budget` in all (ties go
// to the lower index).  Every KV head keeps tokens of its own but all heads the same
// number of them, so the block table still serves all heads.  The kept rows of K and V
// go, in order, to the blocks of a new table; the source blocks are only read, so they
// may be shared with other sequences.
//
// One launch.  A cluster of CTAs (one CTA for tables of up to 8192 tokens, 4096 where there
// are few rows) takes a row, that is, a sequence and KV head: it finds the k-th largest
// weight by radix select, writes the kept places in order, and copies their rows.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 2048;                  // 11 bits of a key at a time: 11 + 11 + 10
constexpr int kMaxCluster = 8;
constexpr int kMaxStaged = 48 * 1024;        // keys of a CTA's part of a row in shared memory

// Weights in an order of unsigned integers: larger weight, larger key; -0 counts as 0,
// NaN (1) lies below everything (-inf is 0x007fffff), +inf is 0xff800000.
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
    if ((bits & 0x7fffffffu) > 0x7f800000u) return 1u;
    if (bits == 0x80000000u) bits = 0u;
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

// The weight of a key (of -0: 0, of a NaN: a NaN).
__device__ __forceinline__ uint32_t bits_of(uint32_t key) { return key & 0x80000000u ? key ^ 0x80000000u : ~key; }

// The copy of a row's kept places to the new blocks, by all warps of its cluster, each
// taking kTile consecutive places at a time: its lanes look up a place's source and
// destination rows at once (three dependent loads for all of them together), then 16 lanes
// (8 for FP8) move a row of K and one of V, 16 bytes each, kBatch such pairs in flight per
// lane.  HBM-bound: 40 sequences of 8192 tokens to 2048 in fp16, 0.67 GB in and out, about
// 105 us (6.4 TB/s).  The warps of a row work side by side on short tiles, which keeps the
// rows in flight close together in the blocks they come from: tiles of 16 and 32 places
// took 117, eight pairs in flight 130.
constexpr int kTile = 8;

template <bool Fp8, int kBatch>
__device__ __forceinline__ void copy_kept(const EvictParams& p, int s, int h, const int32_t* kept, int left, int warp,
                                          int warps) {
    constexpr int kLanes = Fp8 ? 8 : 16;                   // lanes per row
    constexpr int kPer = 32 / kLanes;                      // rows a warp moves at a time
    constexpr int kRowBytes = kLanes * 16;
    const int lane = threadIdx.x & 31;
    const int bs = 1 << p.block_shift;
    const int sub = lane / kLanes, off = (lane % kLanes) * 16;
    uint8_t* kc = static_cast<uint8_t*>(p.k_cache) + off;
    uint8_t* vc = static_cast<uint8_t*>(p.v_cache) + off;
#pragma unroll 1
    for (int j0 = kTile * warp; j0 < left; j0 += kTile * warps) {
        int src = -1, dst = -1;                            // rows of the cache; -1: nothing to move
        const int j = j0 + lane;
        if (lane < kTile && j < left) {
            const int t = __ldcg(kept + j);
            int from = __ldg(p.block_tables + static_cast<size_t>(s) * p.max_blocks + (t >> p.block_shift));
            const int to = __ldg(p.new_tables + static_cast<size_t>(s) * p.max_new_blocks + (j >> p.block_shift));
            const bool bad_from = static_cast<unsigned>(from) >= static_cast<unsigned>(p.num_blocks);
            const bool bad_to = static_cast<unsigned>(to) >= static_cast<unsigned>(p.num_blocks);
            if ((bad_from || bad_to) && p.status) atomicOr(p.status, kDevErrRange);
            if (bad_from) from = 0;
            if (!bad_to) {
                src = ((from * p.num_kv_heads + h) << p.block_shift) + (t & (bs - 1));
                dst = ((to * p.num_kv_heads + h) << p.block_shift) + (j & (bs - 1));
            }
        }
#pragma unroll 1
        for (int r0 = 0; r0 < kTile; r0 += kPer * kBatch) {
            uint4 kx[kBatch], vx[kBatch];
            int to[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int from = __shfl_sync(0xffffffffu, src, r0 + u * kPer + sub);
                to[u] = __shfl_sync(0xffffffffu, dst, r0 + u * kPer + sub);
                if (to[u] >= 0) {
                    kx[u] = __ldcg(reinterpret_cast<const uint4*>(kc + static_cast<size_t>(from) * kRowBytes));
                    vx[u] = __ldcg(reinterpret_cast<const uint4*>(vc + static_cast<size_t>(from) * kRowBytes));
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (to[u] >= 0) {
                    *reinterpret_cast<uint4*>(kc + static_cast<size_t>(to[u]) * kRowBytes) = kx[u];
                    *reinterpret_cast<uint4*>(vc + static_cast<size_t>(to[u]) * kRowBytes) = vx[u];
                }
            }
        }
    }
}

// One cluster per (sequence, KV head), its CTAs taking equal parts of the row and their
// warps contiguous segments.  Staged: a CTA keeps the keys of its part in shared memory, so
// that the row is read once and may be compacted in place (the weights are read back from
// the keys).  Otherwise (rows too long for a cluster's shared memory) it is read again, from
// L2, in each pass.
//
// Radix select: a histogram of the top 11 bits of the keys (shared-memory atomics; the
// CTAs' histograms are added up in the first one through distributed shared memory, which
// hands the result to all) gives the bin that holds the k-th largest; two more passes over
// the keys of that bin give the key itself and how many of the keys equal to it stay.  A
// bin that stays as a whole ends the search early: 22 bits tell most weights apart.
// Bound by the latency of loads, barriers and scans and by instruction issue (stamps in a
// row of 4096 on one CTA: load 1.5 us, a pass 0.5 and its scan 0.4, counts and writes 1.0; a
// cluster adds 1 us per exchange): keys are computed once, a pass costs three or four
// instructions per key, and the keys live in shared memory rather than in registers so
// that all rows of a batch of 320 are resident at once (registers: 22 us of selection, now
// about 15).  With the copy a launch of its own, 64 sequences of up to 4096 tokens took
// 20.5 us, now 18.4; the largest batches take the same.
template <int Threads, bool Staged, bool Fp8>
__global__ void __launch_bounds__(Threads, Threads == 1024 ? 1 : Threads == 512 ? 3 : 4) evict_kernel(const EvictParams p) {
    constexpr int kWarps = Threads / 32;
    constexpr int kOwn = kBins / Threads;        // bins a thread owns
    extern __shared__ uint4 staged[];            // keys of the CTA's part, from t0 on
    __shared__ alignas(16) unsigned hist[kBins];
    __shared__ alignas(16) unsigned total[kBins];
    __shared__ int warp_sum[kWarps];
    __shared__ int warp_sure[kWarps], warp_eq[kWarps];
    __shared__ int part_sure[kMaxCluster], part_eq[kMaxCluster];
    __shared__ int found[3];                     // digit, tokens still to take, tokens of that bin

    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / parts;
    const int s = row / p.num_kv_heads, h = row % p.num_kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kBins / 4; i += Threads) {
        reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4*>(total)[i] = make_uint4(0, 0, 0, 0);
    }
    grid_dependency_wait();
    grid_launch_dependents();

    const int cap = p.max_blocks << p.block_shift;
    const int len = p.seq_lens[s];
    const int n = min(max(len, 0), cap);
    const int left = min(n, p.budget);           // tokens that stay
    if (h == 0 && rank == 0 && tid == 0) {
        p.seq_lens_out[s] = left;
        if (len > cap && p.status) atomicOr(p.status, kDevErrRange);
    }
    // the tokens to choose from: [lo, hi)
    const int lo = min(n, p.sinks), hi = max(lo, n - p.recent);
    const int per = ((n + parts - 1) / parts + 3) & ~3;
    const int t0 = min(n, rank * per), t1 = min(n, t0 + per);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p.weights) + static_cast<size_t>(row) * p.weight_stride;
    uint32_t* keys = reinterpret_cast<uint32_t*>(staged);
    if constexpr (Staged) {
        // whole quads: a row holds a multiple of four weights
        const uint4* from = reinterpret_cast<const uint4*>(w + t0);
#pragma unroll 2
        for (int q = tid; 4 * q < t1 - t0; q += Threads) {
            const uint4 x = from[q];
            staged[q] = make_uint4(key_of(x.x), key_of(x.y), key_of(x.z), key_of(x.w));
        }
    }
    auto key_at = [&](int t) -> uint32_t { return Staged ? keys[t - t0] : key_of(w[t]); };
    // f(key) for every token of the part to choose from, in any order
    const int a = max(t0, lo), b = min(t1, hi);
    auto each = [&](auto&& f) {
        if constexpr (Staged) {
#pragma unroll 2
            for (int q = (a - t0) / 4 + tid; 4 * q < b - t0; q += Threads) {
                const uint4 x = staged[q];
                const int t = t0 + 4 * q;
                if (t >= a && t + 4 <= b) {
                    f(x.x);
                    f(x.y);
                    f(x.z);
                    f(x.w);
                } else {
                    if (t >= a) f(x.x);
                    if (t + 1 >= a && t + 1 < b) f(x.y);
                    if (t + 2 >= a && t + 2 < b) f(x.z);
                    if (t + 3 < b) f(x.w);
                }
            }
        } else {
            for (int t = a + tid; t < b; t += Threads) f(key_of(w[t]));
        }
    };
    // every CTA runs, its histograms cleared, before another adds to them
    if (parts > 1) cluster.sync();
    else __syncthreads();

    int k = left - lo - (n - hi);                // tokens of [lo, hi) that stay
    uint32_t threshold = 0u;                     // keys above it stay (all, so far) ...
    int take_eq = 0;                             // ... and this many of those equal to it
    if (n > p.budget) {
        threshold = 0xffffffffu;
        if (k > 0) {
            uint32_t prefix = 0u;
#pragma unroll 1
            for (int pass = 0; pass < 3; ++pass) {
                if (pass == 0) {
                    each([&](uint32_t x) { atomicAdd(&hist[x >> 21], 1u); });
                } else if (pass == 1) {
                    each([&](uint32_t x) {
                        if ((x >> 21) == prefix) atomicAdd(&hist[(x >> 10) & 2047u], 1u);
                    });
                } else {
                    each([&](uint32_t x) {
                        if ((x >> 10) == prefix) atomicAdd(&hist[x & 1023u], 1u);
                    });
                }
                __syncthreads();
                // a thread owns kOwn bins, the first thread the highest: it adds them to the
                // cluster's (or takes them as they are) and clears them for the next pass
                const int bin = kBins - kOwn * (tid + 1);
                int c[kOwn];
                auto take = [&](unsigned* from) {
#pragma unroll
                    for (int e = 0; e < kOwn; e += 2) {
                        const uint2 x = *reinterpret_cast<uint2*>(from + bin + e);
                        *reinterpret_cast<uint2*>(from + bin + e) = make_uint2(0, 0);
                        c[e] = static_cast<int>(x.x);
                        c[e + 1] = static_cast<int>(x.y);
                    }
                };
                take(hist);
                if (parts > 1) {
                    unsigned* to = cluster.map_shared_rank(total, 0) + bin;
#pragma unroll
                    for (int e = 0; e < kOwn; ++e)
                        if (c[e]) atomicAdd(to + e, static_cast<unsigned>(c[e]));
                    cluster.sync();
                    if (rank == 0) take(total);
                }
                if (rank == 0) {
                    // the bin in which the k-th largest lies: a scan over the threads
                    int own = 0;
#pragma unroll
                    for (int e = 0; e < kOwn; ++e) own += c[e];
                    int incl = own;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += y;
                    }
                    if (lane == 31) warp_sum[warp] = incl;
                    __syncthreads();
                    const int other = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane & (kWarps - 1)] : 0);
                    int before = incl - own + other;
                    if (before < k && k <= before + own) {
                        int d = kOwn - 1, in = 0;
#pragma unroll
                        for (int e = kOwn - 1; e >= 0; --e) {
                            if (e == d) {
                                in = c[e];
                                if (before + in < k) {
                                    before += in;
                                    --d;
                                }
                            }
                        }
                        for (int r = 0; r < parts; ++r) {
                            int* to = parts > 1 ? cluster.map_shared_rank(found, r) : found;
                            to[0] = bin + d;
                            to[1] = k - before;
                            to[2] = in;
                        }
                    }
                }
                if (parts > 1) cluster.sync();
                else __syncthreads();
                const int bits = pass == 2 ? 10 : 11;
                prefix = (prefix << bits) | static_cast<uint32_t>(found[0]);
                k = found[1];
                if (pass == 2) {
                    threshold = prefix;
                    take_eq = k;
                } else if (k == found[2]) {
                    // the whole bin stays: everything above the key before its first
                    threshold = prefix == 0u ? 0u : (prefix << (pass == 0 ? 21 : 10)) - 1u;
                    break;
                }
            }
        }
    }

    // counts of the tokens that surely stay and of those equal to the threshold: per warp,
    // per CTA, per cluster
    const int seg = ((per + kWarps - 1) / kWarps + 31) & ~31;
    const int w0 = min(t1, t0 + warp * seg), w1 = min(t1, w0 + seg);
    const int m0 = max(w0, lo), m1 = min(w1, hi);          // to choose from
    int n_sure = lane == 0 ? w1 - w0 - max(m1 - m0, 0) : 0, n_eq = 0;
#pragma unroll 4
    for (int t = m0 + lane; t < m1; t += 32) {
        const uint32_t x = key_at(t);
        n_sure += x > threshold;
        n_eq += x == threshold;
    }
    if (take_eq == 0) n_eq = 0;
    n_sure = __reduce_add_sync(0xffffffffu, n_sure);
    n_eq = __reduce_add_sync(0xffffffffu, n_eq);
    if (lane == 0) {
        warp_sure[warp] = n_sure;
        warp_eq[warp] = n_eq;
    }
    __syncthreads();
    int sure_before = 0, eq_before = 0;
    if (parts > 1) {
        if (tid < parts) {
            int g = 0, e = 0;
            for (int v = 0; v < kWarps; ++v) {
                g += warp_sure[v];
                e += warp_eq[v];
            }
            *cluster.map_shared_rank(&part_sure[rank], tid) = g;
            *cluster.map_shared_rank(&part_eq[rank], tid) = e;
        }
        // after this no CTA touches another's shared memory, and (Staged) every weight of the
        // row has been read: places and weights can be written
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            sure_before += part_sure[r];
            eq_before += part_eq[r];
        }
    }
    for (int v = 0; v < warp; ++v) {
        sure_before += warp_sure[v];
        eq_before += warp_eq[v];
    }
    int32_t* kept = p.kept + static_cast<size_t>(row) * p.budget;
    uint32_t* wo = reinterpret_cast<uint32_t*>(p.weights_out) + static_cast<size_t>(row) * p.weight_stride;
    const unsigned below = (1u << lane) - 1u;
#pragma unroll 2
    for (int t = w0 + lane; t - lane < w1; t += 32) {
        const uint32_t x = t < w1 ? key_at(t) : 0u;
        const bool choose = t >= lo && t < hi;
        const bool sure = t < w1 && (!choose || x > threshold);
        const unsigned ms = __ballot_sync(0xffffffffu, sure);
        int at = sure_before + __popc(ms & below);
        bool stays = sure;
        if (take_eq > 0) {
            const bool eq = t < w1 && choose && x == threshold;
            const unsigned me = __ballot_sync(0xffffffffu, eq);
            const int eq_rank = eq_before + __popc(me & below);
            stays = sure || (eq && eq_rank < take_eq);
            at += min(eq_rank, take_eq);
            eq_before += __popc(me);
        }
        if (stays) {
            kept[at] = t;
            wo[at] = bits_of(x);
        }
        sure_before += __popc(ms);
    }
    // what the row no longer holds: weights of 0, places of -1
    for (int t = left + rank * Threads + tid; t < n; t += parts * Threads) wo[t] = 0u;
    for (int j = left + rank * Threads + tid; j < p.budget; j += parts * Threads) kept[j] = -1;
    // every place is written, and visible to the cluster: the rows can move
    if (parts > 1) cluster.sync();
    else __syncthreads();
    copy_kept<Fp8, Fp8 ? 2 : (Threads == 512 ? 2 : 4)>(p, s, h, kept, left, rank * kWarps + warp, parts * kWarps);
}

}  // namespace

// CTAs per row and threads per CTA: one CTA up to 8192 tokens, a cluster beyond, or for
// long rows while they leave most of the device idle; 1024 threads where there is an SM for
// every CTA, else 512, and 256 for short rows.  "Tokens" are the block table's (cap): the
// host does not know the lengths, and a CTA's shared memory must hold its part of the
// longest row they allow.  A table wider than its sequences costs: 512 rows of 400 to 800
// tokens take 33 us with a table of 800, 42 with 8192, 55 with 8208, 69 with 32768 and 156
// with 131072; 320 rows of 8192 tokens 121 with a table of 8192, 128 with 8208 and 16384,
// 193 with 131072.  Tables cut to the longest sequence avoid it.
EvictPlan evict_plan(long long rows, long long cap, int sms) {
    EvictPlan e;
    e.parts = 1;
    while (e.parts < kMaxCluster && (cap > 8192ll * e.parts || (rows * e.parts <= sms / 2 && cap > 4096ll * e.parts)))
        e.parts *= 2;
    const long long per = ((cap + e.parts - 1) / e.parts + 3) & ~3ll;
    e.staged = per <= kMaxStaged;
    e.smem = e.staged ? static_cast<size_t>(per) * 4 : 0;
    e.threads = per <= 1024 ? 256 : rows * e.parts <= sms ? 1024 : 512;
    return e;
}

namespace {
template <bool Fp8>
const void* evict_fn(const EvictPlan& plan) {
    if (!plan.staged) return reinterpret_cast<const void*>(&evict_kernel<1024, false, Fp8>);
    return plan.threads == 256   ? reinterpret_cast<const void*>(&evict_kernel<256, true, Fp8>)
           : plan.threads == 512 ? reinterpret_cast<const void*>(&evict_kernel<512, true, Fp8>)
                                 : reinterpret_cast<const void*>(&evict_kernel<1024, true, Fp8>);
}
}  // namespace

cudaError_t evict_prepare() {
    for (int threads : {512, 1024}) {            // 256 threads: at most 1024 tokens
        EvictPlan plan = {1, threads, true, 0};
        cudaError_t e = cudaFuncSetAttribute(evict_fn<true>(plan), cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxStaged * 4);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_fn<false>(plan), cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxStaged * 4);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_evict(const EvictParams& p, const EvictPlan& plan, bool fp8, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.num_seqs) * p.num_kv_heads * plan.parts));
    cfg.blockDim = dim3(static_cast<unsigned>(plan.staged ? plan.threads : 1024));
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(plan.parts);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void* args[] = {const_cast<EvictParams*>(&p)};
    return cudaLaunchKernelExC(&cfg, fp8 ? evict_fn<true>(plan) : evict_fn<false>(plan), args);
}

}  // namespace pa
