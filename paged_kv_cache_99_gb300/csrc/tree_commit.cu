// Commit of accepted paths (sm_103a): after a tree of drafted tokens was verified, the K and V
// rows of the nodes on the accepted path move to the places right behind the tokens before the
// tree, in all layers' caches.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kCommitWarps = 4;
constexpr int kCommitRows = 16;         // rows a warp has in flight

// Node path[i] (ascending, path[i] >= i) moves to place i.  A store to place i can only
// overwrite the row of a path[k] with k <= i, so a warp that takes the rows in order and loads
// a batch of them before it stores the batch needs no copy beside the cache.
//
// Few bytes move (a row is 128 elements of one KV head; a path is a handful of nodes), so a
// call is as long as its chain of loads: lengths, then the path and the table's entries, then
// rows.  One warp takes one (sequence, KV head, cache); lane i checks node i of the path and
// finds both its places, and the rows' addresses go round by shuffles: 4 sequences of one
// layer take 3.1 us, 64 sequences of 28 layers (2 heads, 7.5 MB in and out) 6.2.  A path of more than 32
// nodes is checked first and then taken 32 nodes at a time.
template <int RowBytes>
__global__ void __launch_bounds__(kCommitWarps * 32) tree_commit_kernel(const __grid_constant__ CommitParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int kLanes = RowBytes / 16;           // lanes of a row: 16 (16-bit) or 8 (FP8)
    constexpr int kAtOnce = 32 / kLanes;            // rows of one load instruction
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kCommitWarps + (threadIdx.x >> 5);
    const int per_seq = p.num_kv_heads * 2 * p.num_layers;
    if (item >= static_cast<long long>(p.num_seqs) * per_seq) return;
    const int s = static_cast<int>(item / per_seq);
    const int rest = static_cast<int>(item % per_seq);
    const int h = rest % p.num_kv_heads;
    const int which = rest / p.num_kv_heads;        // 2 layer, + 1 for V
    uint8_t* cache = static_cast<uint8_t*>(p.caches[which]);

    const int len = p.path_lens[s];
    const int n = p.seq_lens[s];
    const int nodes = p.query_start_loc[s + 1] - p.query_start_loc[s];
    bool ok = nodes >= 0 && n >= nodes && n <= static_cast<long long>(p.max_blocks) << p.block_shift && len >= 0 &&
              len <= nodes && len <= p.max_path;
    const int base = n - nodes;
    const int32_t* path = p.paths + static_cast<size_t>(s) * p.max_path;
    const int32_t* table = p.block_tables + static_cast<size_t>(s) * p.max_blocks;
    // row of the cache (in tokens of a head) at a place of the sequence, or -1 outside the pool
    auto row_of = [&](int place) -> long long {
        const int block = __ldg(table + (place >> p.block_shift));
        if (static_cast<unsigned>(block) >= static_cast<unsigned>(p.num_blocks)) return -1;
        return (((static_cast<long long>(block) * p.num_kv_heads + h) << p.block_shift)) + (place & ((1 << p.block_shift) - 1));
    };
    // lane's node i: where it is and where it goes
    long long from = 0, to = 0;
    int node = 0;
    auto look = [&](int i) {
        bool good = true;
        from = to = 0;
        node = i;
        if (i < len) {
            node = path[i];
            good = node >= i && node < nodes && (i == 0 || path[i - 1] < node);
            if (good && node != i) {
                from = row_of(base + node);
                to = row_of(base + i);
                good = from >= 0 && to >= 0;
            }
        }
        return good;
    };
    if (ok) {
        for (int i = lane; i - lane < len; i += 32) ok = ok && look(i);
        ok = __all_sync(0xffffffffu, ok);
    }
    if (rest == 0 && lane == 0) {
        if (!ok && p.status) atomicOr(p.status, kDevErrRange);
        if (ok && p.seq_lens_out) p.seq_lens_out[s] = base + len;
    }
    if (!ok) return;                                // nothing of the sequence moves
    const int sub = lane / kLanes, part = lane % kLanes;
    for (int i0 = 0; i0 < len; i0 += 32) {
        if (len > 32) look(i0 + lane);
        const int m = min(32, len - i0);
        // nodes that stay where they are, at the front of every path that starts at the root
        const unsigned moves = __ballot_sync(0xffffffffu, node != i0 + lane && lane < m);
        if (moves == 0) continue;
        for (int r0 = __ffs(moves) - 1; r0 < m; r0 += kCommitRows) {
            uint4 x[kCommitRows / kAtOnce];
            long long dst[kCommitRows / kAtOnce];
#pragma unroll
            for (int e = 0; e < kCommitRows / kAtOnce; ++e) {
                const int r = r0 + e * kAtOnce + sub;
                const long long src = __shfl_sync(0xffffffffu, from, r & 31);
                dst[e] = __shfl_sync(0xffffffffu, to, r & 31);
                const bool live = r < m && (moves >> (r & 31) & 1);
                if (live) x[e] = __ldcg(reinterpret_cast<const uint4*>(cache + src * RowBytes) + part);
                else dst[e] = -1;
            }
            __syncwarp();                           // every load of the batch before its first store
#pragma unroll
            for (int e = 0; e < kCommitRows / kAtOnce; ++e)
                if (dst[e] >= 0) __stcg(reinterpret_cast<uint4*>(cache + dst[e] * RowBytes) + part, x[e]);
            __syncwarp();
        }
    }
}

}  // namespace

cudaError_t launch_tree_commit(const CommitParams& p, bool fp8, cudaStream_t stream) {
    const long long items = static_cast<long long>(p.num_seqs) * p.num_kv_heads * 2 * p.num_layers;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((items + kCommitWarps - 1) / kCommitWarps));
    cfg.blockDim = dim3(kCommitWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return fp8 ? cudaLaunchKernelEx(&cfg, tree_commit_kernel<kHeadDim>, p)
               : cudaLaunchKernelEx(&cfg, tree_commit_kernel<2 * kHeadDim>, p);
}

}  // namespace pa
