// Eviction of the cached tokens with the least accumulated attention weight, sm_103a.
//
// For every sequence and KV head the first `sinks` and the last `recent` tokens stay,
// and of the tokens between them those of the largest weights, `budget` in all (ties go
// to the lower index).  Every KV head keeps tokens of its own but all heads the same
// number of them, so the block table still serves all heads.  The kept rows of K and V
// go, in order, to the blocks of a new table; the source blocks are only read, so they
// may be shared with other sequences.
//
// Two launches.  The selection finds the k-th largest weight of each row by radix
// select and writes the kept places in order; the copy is pure data movement
// (HBM-bound) over those places.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;                  // 11 bits of a key at a time: 11 + 11 + 10
constexpr int kMaxCluster = 8;
// tokens of one CTA's part of a row that fit its shared memory beside the histograms
constexpr int kMaxStaged = 48 * 1024;

// Weights in an order of unsigned integers: larger weight, larger key; -0 counts as 0,
// NaN lies below everything (even -inf).
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
    if ((bits & 0x7fffffffu) > 0x7f800000u) return 0u;
    if (bits == 0x80000000u) bits = 0u;
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

// One cluster per (sequence, KV head), its CTAs taking equal parts of the row.  Staged:
// each CTA reads its part once into shared memory (the weights may then be compacted in
// place); rows too long for that are read from L2 in every pass.
//
// Radix select: a histogram of the top 11 bits of the keys (shared-memory atomics, the
// CTAs' histograms added up through distributed shared memory) gives the bin that holds
// the k-th largest; two more passes over the keys in that bin give the key itself and
// how many of the keys equal to it are kept.  Latency-bound: three passes over a few
// thousand keys per CTA, so a row is spread over more CTAs while the device has room.
template <bool Staged>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
    extern __shared__ uint32_t staged[];
    __shared__ unsigned hist[kBins];
    __shared__ unsigned total[kBins];
    __shared__ int warp_sum[kSelWarps];
    __shared__ int warp_gt[kSelWarps], warp_eq[kSelWarps];
    __shared__ int part_gt[kMaxCluster], part_eq[kMaxCluster];
    __shared__ unsigned found_digit;
    __shared__ int found_left;

    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    grid_dependency_wait();
    grid_launch_dependents();
    if (parts > 1) cluster.sync();               // every CTA runs before its shared memory is written
    const int row = blockIdx.x / parts;
    const int s = row / p.num_kv_heads, h = row % p.num_kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int cap = p.max_blocks << p.block_shift;
    const int len = p.seq_lens[s];
    const int n = min(max(len, 0), cap);
    const int left = min(n, p.budget);           // tokens that stay
    if (h == 0 && rank == 0 && tid == 0) {
        p.seq_lens_out[s] = left;
        if (len > cap && p.status) atomicOr(p.status, kDevErrRange);
    }
    const int per = ((n + parts - 1) / parts + 3) & ~3;
    const int t0 = min(n, rank * per), t1 = min(n, t0 + per);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p.weights) + static_cast<size_t>(row) * p.weight_stride;
    if (Staged) {
        const uint4* src = reinterpret_cast<const uint4*>(w + t0);
        for (int i = tid; i < (t1 - t0) / 4; i += kSelThreads) reinterpret_cast<uint4*>(staged)[i] = src[i];
        for (int i = ((t1 - t0) & ~3) + tid; i < t1 - t0; i += kSelThreads) staged[i] = w[t0 + i];
    }
    auto bits_at = [&](int t) -> uint32_t { return Staged ? staged[t - t0] : w[t]; };

    // the tokens to choose from, and how many of them stay
    const int lo = min(n, p.sinks), hi = max(lo, n - p.recent);
    int k = left - lo - (n - hi);
    uint32_t threshold = 0u;                     // keys above it stay ...
    int take_eq = 0x7fffffff;                    // ... and this many of those equal to it
    if (n > p.budget) {
        threshold = 0xffffffffu;
        take_eq = 0;
        if (k > 0) {
            uint32_t prefix = 0u;
            const int a = max(t0, lo), b = min(t1, hi);
#pragma unroll 1
            for (int pass = 0; pass < 3; ++pass) {
                const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
                const int above = pass == 0 ? 32 : (pass == 1 ? 21 : 10);    // bits fixed so far end here
                for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0u;
                __syncthreads();
                for (int t = a + tid; t < b; t += kSelThreads) {
                    const uint32_t key = key_of(bits_at(t));
                    if (pass == 0 || (key >> above) == prefix)
                        atomicAdd(&hist[(key >> shift) & (pass == 2 ? 1023u : 2047u)], 1u);
                }
                if (parts > 1) {
                    // the cluster's histogram: each CTA adds up its share of the bins for all
                    cluster.sync();
                    const int share = kBins / parts;
                    for (int i = tid; i < share; i += kSelThreads) {
                        const int bin = rank * share + i;
                        unsigned sum = 0u;
                        for (int r = 0; r < parts; ++r) sum += *cluster.map_shared_rank(&hist[bin], r);
                        for (int r = 0; r < parts; ++r) *cluster.map_shared_rank(&total[bin], r) = sum;
                    }
                    cluster.sync();
                } else {
                    __syncthreads();
                }
                // the bin in which the k-th largest lies: a scan from the top, four bins a thread
                const unsigned* from = parts > 1 ? total : hist;
                const int top = kBins - 1 - 4 * tid;
                const int c0 = from[top], c1 = from[top - 1], c2 = from[top - 2], c3 = from[top - 3];
                int incl = c0 + c1 + c2 + c3;
                const int own = incl;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                if (lane == 31) warp_sum[warp] = incl;
                __syncthreads();
                for (int v = 0; v < warp; ++v) incl += warp_sum[v];
                int before = incl - own;
                if (before < k && k <= incl) {
                    int d = top;
                    if (before + c0 < k) {
                        before += c0;
                        --d;
                        if (before + c1 < k) {
                            before += c1;
                            --d;
                            if (before + c2 < k) {
                                before += c2;
                                --d;
                            }
                        }
                    }
                    found_digit = static_cast<unsigned>(d);
                    found_left = k - before;
                }
                __syncthreads();
                prefix = (prefix << (pass == 2 ? 10 : 11)) | found_digit;
                k = found_left;
            }
            threshold = prefix;
            take_eq = k;
        }
    }
    __syncthreads();

    // counts of the tokens that surely stay and of those equal to the threshold: per warp
    // (each a contiguous segment), per CTA, per cluster
    const int seg = ((t1 - t0 + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int w0 = min(t1, t0 + warp * seg), w1 = min(t1, w0 + seg);
    auto classify = [&](int t, bool& sure, bool& eq) {
        const bool in = t < w1;
        const bool fixed = in && (t < lo || t >= hi);
        const uint32_t key = in && !fixed ? key_of(bits_at(t)) : 0u;
        sure = fixed || (in && key > threshold);
        eq = in && !fixed && key == threshold;
    };
    int n_sure = 0, n_eq = 0;
    for (int b = w0; b < w1; b += 32) {
        bool sure, eq;
        classify(b + lane, sure, eq);
        n_sure += __popc(__ballot_sync(0xffffffffu, sure));
        n_eq += __popc(__ballot_sync(0xffffffffu, eq));
    }
    if (lane == 0) {
        warp_gt[warp] = n_sure;
        warp_eq[warp] = n_eq;
    }
    __syncthreads();
    if (tid < parts) {
        int g = 0, e = 0;
        for (int v = 0; v < kSelWarps; ++v) {
            g += warp_gt[v];
            e += warp_eq[v];
        }
        *cluster.map_shared_rank(&part_gt[rank], tid) = g;
        *cluster.map_shared_rank(&part_eq[rank], tid) = e;
    }
    // after this no CTA touches another's shared memory, and every weight of the row has
    // been read (staged rows): places and weights can be written
    cluster.sync();
    int sure_before = 0, eq_before = 0;
    for (int r = 0; r < rank; ++r) {
        sure_before += part_gt[r];
        eq_before += part_eq[r];
    }
    for (int v = 0; v < warp; ++v) {
        sure_before += warp_gt[v];
        eq_before += warp_eq[v];
    }
    int32_t* kept = p.kept + static_cast<size_t>(row) * p.budget;
    uint32_t* wo = reinterpret_cast<uint32_t*>(p.weights_out) + static_cast<size_t>(row) * p.weight_stride;
    const unsigned below = (1u << lane) - 1u;
    for (int b = w0; b < w1; b += 32) {
        bool sure, eq;
        const int t = b + lane;
        classify(t, sure, eq);
        const unsigned ms = __ballot_sync(0xffffffffu, sure), me = __ballot_sync(0xffffffffu, eq);
        const int eq_rank = eq_before + __popc(me & below);
        if (sure || (eq && eq_rank < take_eq)) {
            const int at = sure_before + __popc(ms & below) + min(eq_rank, take_eq);
            kept[at] = t;
            wo[at] = bits_at(t);
        }
        sure_before += __popc(ms);
        eq_before += __popc(me);
    }
    // what the row no longer holds: weights of 0, places of -1
    for (int t = left + rank * kSelThreads + tid; t < n; t += parts * kSelThreads) wo[t] = 0u;
    for (int j = left + rank * kSelThreads + tid; j < p.budget; j += parts * kSelThreads) kept[j] = -1;
}

// Copy of the kept rows to the new blocks.  A warp takes kRows consecutive places of one
// (sequence, KV head): its lanes look up a place's source and destination rows at once
// (three dependent loads for all of them together), then 16 lanes (8 for FP8) move a row
// of K and one of V, 16 bytes each, with kBatch such pairs in flight per lane.
template <bool Fp8, int kRows>
__global__ void __launch_bounds__(256) evict_copy_kernel(const EvictParams p, int tiles) {
    constexpr int kLanes = Fp8 ? 8 : 16;                   // lanes per row
    constexpr int kPer = 32 / kLanes;                      // rows a warp moves at a time
    constexpr int kBatch = kRows / kPer < 4 ? kRows / kPer : 4;
    constexpr int kRowBytes = kLanes * 16;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const long long row = unit / tiles;
    if (row >= static_cast<long long>(p.num_seqs) * p.num_kv_heads) return;
    const int s = static_cast<int>(row / p.num_kv_heads), h = static_cast<int>(row % p.num_kv_heads);
    const int j0 = static_cast<int>(unit % tiles) * kRows;
    const int left = __ldcg(p.seq_lens_out + s);
    if (j0 >= left) return;
    const int bs = 1 << p.block_shift;
    int src = -1, dst = -1;                                // rows of the cache; -1: nothing to move
    const int j = j0 + lane;
    if (lane < kRows && j < left) {
        const int t = __ldcg(p.kept + static_cast<size_t>(row) * p.budget + j);
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
    const int sub = lane / kLanes, off = (lane % kLanes) * 16;
    uint8_t* kc = static_cast<uint8_t*>(p.k_cache) + off;
    uint8_t* vc = static_cast<uint8_t*>(p.v_cache) + off;
    const int rows = min(kRows, left - j0);
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kPer * kBatch) {
        uint4 kx[kBatch], vx[kBatch];
        int to[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int r = (r0 + u * kPer + sub) & 31;
            const int from = __shfl_sync(0xffffffffu, src, r);
            to[u] = __shfl_sync(0xffffffffu, dst, r);
            if (to[u] >= 0) {
                kx[u] = __ldcs(reinterpret_cast<const uint4*>(kc + static_cast<size_t>(from) * kRowBytes));
                vx[u] = __ldcs(reinterpret_cast<const uint4*>(vc + static_cast<size_t>(from) * kRowBytes));
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

}  // namespace

// CTAs per row: as few as hold its weights in shared memory (Staged), then more while
// the device has room and each has over 1024 tokens to look at.
EvictPlan evict_plan(int num_seqs, int num_kv_heads, long long cap, int sms) {
    const long long rows = static_cast<long long>(num_seqs) * num_kv_heads;
    EvictPlan e;
    e.parts = 1;
    while (e.parts < kMaxCluster && (cap > static_cast<long long>(e.parts) * kMaxStaged ||
                                     (rows * e.parts * 2 <= 2ll * sms && cap > 2048ll * e.parts)))
        e.parts *= 2;
    e.staged = cap <= static_cast<long long>(e.parts) * kMaxStaged;
    e.smem = e.staged ? static_cast<size_t>(((cap + e.parts - 1) / e.parts + 3) & ~3ll) * 4 : 0;
    return e;
}

cudaError_t evict_prepare() {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(&evict_select_kernel<true>),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxStaged * 4);
}

cudaError_t launch_evict_select(const EvictParams& p, const EvictPlan& plan, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.num_seqs) * p.num_kv_heads * plan.parts));
    cfg.blockDim = dim3(kSelThreads);
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
    return plan.staged ? cudaLaunchKernelEx(&cfg, evict_select_kernel<true>, p)
                       : cudaLaunchKernelEx(&cfg, evict_select_kernel<false>, p);
}

cudaError_t launch_evict_copy(const EvictParams& p, bool fp8, int max_left, int sms, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.num_seqs) * p.num_kv_heads;
    // tiles of 32 places where that fills the device's warp slots, else of 8
    const bool wide = rows * ((max_left + 31) / 32) >= 64ll * sms;
    const int tile = wide ? 32 : 8;
    int tiles = (max_left + tile - 1) / tile;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows * tiles + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (fp8)
        return wide ? cudaLaunchKernelEx(&cfg, evict_copy_kernel<true, 32>, p, tiles)
                    : cudaLaunchKernelEx(&cfg, evict_copy_kernel<true, 8>, p, tiles);
    return wide ? cudaLaunchKernelEx(&cfg, evict_copy_kernel<false, 32>, p, tiles)
                : cudaLaunchKernelEx(&cfg, evict_copy_kernel<false, 8>, p, tiles);
}

}  // namespace pa
