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
constexpr uint32_t kNone = 0u;               // key of a place past the end: never kept
constexpr uint32_t kSure = 0xffffffffu;      // key of a token that stays whatever its weight

// Weights in an order of unsigned integers: larger weight, larger key; -0 counts as 0,
// NaN (1) lies below everything (-inf is 0x007fffff), +inf is 0xff800000.
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
    if ((bits & 0x7fffffffu) > 0x7f800000u) return 1u;
    if (bits == 0x80000000u) bits = 0u;
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

// One cluster per (sequence, KV head), its CTAs taking equal parts of the row and their
// warps contiguous segments.  With Keys > 0 a thread holds the (at most Keys) weights of
// its places and their keys in registers: the row is read once, and may be compacted in
// place.  Keys = 0 takes rows of any length and reads them again (from L2) in each pass.
//
// Radix select: a histogram of the top 11 bits of the keys (shared-memory atomics; the
// CTAs' histograms are added up in the first one through distributed shared memory, which
// hands the result to all) gives the bin that holds the k-th largest; two more passes over
// the keys of that bin give the key itself and how many of the keys equal to it stay.  A
// bin that stays as a whole ends the search early: 22 bits tell most weights apart.
// Bound by instruction issue and barrier latency (the row itself is small): keys are
// computed once, a pass costs about four instructions per key.
template <int Keys>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
    __shared__ alignas(16) unsigned hist[kBins];
    __shared__ alignas(16) unsigned total[kBins];
    __shared__ int warp_sum[kSelWarps];
    __shared__ int warp_sure[kSelWarps], warp_eq[kSelWarps];
    __shared__ int part_sure[kMaxCluster], part_eq[kMaxCluster];
    __shared__ int found[3];                     // digit, tokens still to take, tokens of that bin

    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / parts;
    const int s = row / p.num_kv_heads, h = row % p.num_kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    *reinterpret_cast<uint4*>(hist + 4 * tid) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(total + 4 * tid) = make_uint4(0, 0, 0, 0);
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
    const int per = (n + parts - 1) / parts;
    const int t0 = min(n, rank * per), t1 = min(n, t0 + per);
    const int seg = ((per + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int w0 = min(t1, t0 + warp * seg), w1 = min(t1, w0 + seg);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p.weights) + static_cast<size_t>(row) * p.weight_stride;
    auto classify = [&](int t, uint32_t bits) -> uint32_t {
        return t >= w1 ? kNone : t < lo || t >= hi ? kSure : key_of(bits);
    };
    uint32_t raw[Keys > 0 ? Keys : 1], key[Keys > 0 ? Keys : 1];
    if constexpr (Keys > 0) {
#pragma unroll
        for (int i = 0; i < Keys; ++i) raw[i] = w0 + 32 * i + lane < w1 ? w[w0 + 32 * i + lane] : 0u;
#pragma unroll
        for (int i = 0; i < Keys; ++i) key[i] = classify(w0 + 32 * i + lane, raw[i]);
    }
    // f(key, weight's bits, place) for the warp's places, 32 at a time
    auto each = [&](auto&& f) {
        if constexpr (Keys > 0) {
#pragma unroll
            for (int i = 0; i < Keys; ++i)
                if (32 * i < seg) f(key[i], raw[i], w0 + 32 * i + lane);
        } else {
#pragma unroll 1
            for (int b = w0; b < w1; b += 32) {
                const uint32_t x = b + lane < w1 ? w[b + lane] : 0u;
                f(classify(b + lane, x), x, b + lane);
            }
        }
    };
    // every CTA runs, its histograms cleared, before another adds to them
    if (parts > 1) cluster.sync();
    else __syncthreads();

    int k = left - lo - (n - hi);                // tokens of [lo, hi) that stay
    uint32_t threshold = kNone;                  // keys above it stay ...
    int take_eq = 0;                             // ... and this many of those equal to it
    if (n > p.budget) {
        threshold = kSure - 1u;
        if (k > 0) {
            uint32_t prefix = 0u;
#pragma unroll 1
            for (int pass = 0; pass < 3; ++pass) {
                if (pass == 0) {
                    each([&](uint32_t x, uint32_t, int) {
                        if (x - 1u < kSure - 1u) atomicAdd(&hist[x >> 21], 1u);
                    });
                } else if (pass == 1) {
                    each([&](uint32_t x, uint32_t, int) {
                        if ((x >> 21) == prefix && x != kNone) atomicAdd(&hist[(x >> 10) & 2047u], 1u);
                    });
                } else {
                    each([&](uint32_t x, uint32_t, int) {
                        if ((x >> 10) == prefix && x != kNone) atomicAdd(&hist[x & 1023u], 1u);
                    });
                }
                __syncthreads();
                // a thread owns four bins, from the top down: it adds them to the cluster's
                // (or takes them as they are) and clears them for the next pass
                const int bin = kBins - 4 - 4 * tid;
                uint4 c = *reinterpret_cast<uint4*>(hist + bin);
                *reinterpret_cast<uint4*>(hist + bin) = make_uint4(0, 0, 0, 0);
                if (parts > 1) {
                    unsigned* to = cluster.map_shared_rank(total, 0) + bin;
                    if (c.x) atomicAdd(to, c.x);
                    if (c.y) atomicAdd(to + 1, c.y);
                    if (c.z) atomicAdd(to + 2, c.z);
                    if (c.w) atomicAdd(to + 3, c.w);
                    cluster.sync();
                    if (rank == 0) {
                        c = *reinterpret_cast<uint4*>(total + bin);
                        *reinterpret_cast<uint4*>(total + bin) = make_uint4(0, 0, 0, 0);
                    }
                }
                if (rank == 0) {
                    // the bin in which the k-th largest lies: a scan over the threads
                    const int own = static_cast<int>(c.x + c.y + c.z + c.w);
                    int incl = own;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += y;
                    }
                    if (lane == 31) warp_sum[warp] = incl;
                    __syncthreads();
                    int other = lane < warp ? warp_sum[lane & (kSelWarps - 1)] : 0;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) other += __shfl_xor_sync(0xffffffffu, other, o);
                    int before = incl - own + other;
                    if (before < k && k <= before + own) {
                        int d = bin + 3, in = static_cast<int>(c.w);
                        if (before + in < k) {
                            before += in;
                            --d;
                            in = static_cast<int>(c.z);
                            if (before + in < k) {
                                before += in;
                                --d;
                                in = static_cast<int>(c.y);
                                if (before + in < k) {
                                    before += in;
                                    --d;
                                    in = static_cast<int>(c.x);
                                }
                            }
                        }
                        for (int r = 0; r < parts; ++r) {
                            int* to = parts > 1 ? cluster.map_shared_rank(found, r) : found;
                            to[0] = d;
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
                    threshold = prefix == 0u ? kNone : (prefix << (pass == 0 ? 21 : 10)) - 1u;
                    break;
                }
            }
        }
    }

    // counts of the tokens that surely stay and of those equal to the threshold: per warp,
    // per CTA, per cluster
    int n_sure = 0, n_eq = 0;
    each([&](uint32_t x, uint32_t, int) {
        n_sure += x > threshold;
        n_eq += x == threshold;
    });
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
            for (int v = 0; v < kSelWarps; ++v) {
                g += warp_sure[v];
                e += warp_eq[v];
            }
            *cluster.map_shared_rank(&part_sure[rank], tid) = g;
            *cluster.map_shared_rank(&part_eq[rank], tid) = e;
        }
        // after this no CTA touches another's shared memory, and (Keys > 0) every weight of
        // the row has been read: places and weights can be written
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
    if (take_eq == 0) {
        each([&](uint32_t x, uint32_t bits, int t) {
            const unsigned ms = __ballot_sync(0xffffffffu, x > threshold);
            if (x > threshold) {
                const int at = sure_before + __popc(ms & below);
                kept[at] = t;
                wo[at] = bits;
            }
            sure_before += __popc(ms);
        });
    } else {
        each([&](uint32_t x, uint32_t bits, int t) {
            const bool sure = x > threshold, eq = x == threshold;
            const unsigned ms = __ballot_sync(0xffffffffu, sure), me = __ballot_sync(0xffffffffu, eq);
            const int eq_rank = eq_before + __popc(me & below);
            if (sure || (eq && eq_rank < take_eq)) {
                const int at = sure_before + __popc(ms & below) + min(eq_rank, take_eq);
                kept[at] = t;
                wo[at] = bits;
            }
            sure_before += __popc(ms);
            eq_before += __popc(me);
        });
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

// CTAs per row and weights per thread: parts of at most 4096 tokens (8 per thread)
// while a cluster reaches, then 8192 and 16384; longer rows are read again in each pass.
EvictPlan evict_plan(long long cap) {
    EvictPlan e;
    e.parts = 1;
    while (e.parts < kMaxCluster && cap > 4096ll * e.parts) e.parts *= 2;
    const long long per = (cap + e.parts - 1) / e.parts;
    e.keys = per <= 2048 ? 4 : per <= 4096 ? 8 : per <= 8192 ? 16 : per <= 16384 ? 32 : 0;
    return e;
}

cudaError_t launch_evict_select(const EvictParams& p, const EvictPlan& plan, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.num_seqs) * p.num_kv_heads * plan.parts));
    cfg.blockDim = dim3(kSelThreads);
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
    switch (plan.keys) {
        case 4: return cudaLaunchKernelEx(&cfg, evict_select_kernel<4>, p);
        case 8: return cudaLaunchKernelEx(&cfg, evict_select_kernel<8>, p);
        case 16: return cudaLaunchKernelEx(&cfg, evict_select_kernel<16>, p);
        case 32: return cudaLaunchKernelEx(&cfg, evict_select_kernel<32>, p);
    }
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<0>, p);
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
