// Attention over the paged cache whose scores or masks are not plain (sm_103a): scores capped by
// a tanh, biased by distance, windowed, open over a prefix, or masked by a tree of drafted tokens.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

// The cached tokens [lo, hi) that a row sees and its position; a tree's row also sees the nodes
// of its mask, which lie behind hi.
struct RowView {
    int pos, lo, hi;
};

// Lengths of a sequence that fit q, the table and the masks.
__device__ __forceinline__ bool scored_lengths_ok(const ScoredParams& p, int q0, int q_len, int n) {
    return q0 >= 0 && q_len >= 0 && q0 <= p.total_rows && q_len <= p.total_rows - q0 && n >= q_len &&
           n <= (p.max_blocks << p.block_shift) && (!p.masks || q_len <= 64ll * p.mask_words);
}

// Row j of a sequence of n tokens whose last q_len are the rows'.
__device__ __forceinline__ RowView row_view(const ScoredParams& p, int s, int q0, int q_len, int n, int j) {
    RowView v;
    v.pos = n - q_len + j;
    v.hi = v.pos + 1;
    if (p.masks) {
        // a node's position: behind the context, as deep as its path is long
        int bits = 0;
        const unsigned long long* words = p.masks + static_cast<size_t>(q0 + j) * p.mask_words;
        for (int i = 0; 64 * i < q_len; ++i) {
            unsigned long long w = words[i];
            if (q_len - 64 * i < 64) w &= (1ull << (q_len - 64 * i)) - 1;
            bits += __popcll(w);
        }
        v.pos = n - q_len + bits - 1;
        v.hi = n - q_len;
    } else if (p.prefix_lens) {
        v.hi = max(v.hi, min(p.prefix_lens[s], n));
    }
    v.lo = p.window > 0 ? max(0, v.pos - p.window + 1) : 0;
    return v;
}

// One warp per (query row, query head): a lane holds four of the head's 128 components, every
// visible key costs one shuffled sum.  Online softmax in 32 bits.
template <int Kind, bool QBf16>
__global__ void __launch_bounds__(256) scored_kernel(const ScoredParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr bool kFp8 = Kind == kKindFp8;
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int row = static_cast<int>(item / p.num_q_heads), head = static_cast<int>(item % p.num_q_heads);
    if (row >= p.total_rows) return;
    // the sequence whose rows hold `row`
    int lo = 0, hi = p.num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.query_start_loc[mid] <= row) lo = mid; else hi = mid;
    }
    const int s = lo;
    const int q0 = p.query_start_loc[s], q_len = p.query_start_loc[s + 1] - q0, n = p.seq_lens[s];
    const int j = row - q0;
    if (j < 0 || j >= q_len) return;                        // a row behind the last sequence
    if (!scored_lengths_ok(p, q0, q_len, n)) {
        if (lane == 0) atomicOr(p.status, kDevErrRange);
        return;
    }
    const RowView v = row_view(p, s, q0, q_len, n, j);
    const int h = head / p.group;
    float ks = 1.f, vs = 1.f;
    if constexpr (kFp8) {
        ks = __ldg(p.k_scale + h * p.scale_stride);
        vs = __ldg(p.v_scale + h * p.scale_stride);
    }
    const uint2 qw = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) +
                                                     (static_cast<size_t>(row) * p.num_q_heads + head) * kHeadDim + 4 * lane);
    const float q[4] = {to_float<QBf16>(qw.x & 0xffffu), to_float<QBf16>(qw.x >> 16), to_float<QBf16>(qw.y & 0xffffu),
                        to_float<QBf16>(qw.y >> 16)};
    const float slope = p.slopes ? __ldg(p.slopes + head) : 0.f;
    const int32_t* bt = p.block_tables + static_cast<size_t>(s) * p.max_blocks;
    auto load4 = [&](const void* cache, size_t at, float (&x)[4]) {
        if constexpr (kFp8) {
            const uint32_t w = __ldg(reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(cache) + at));
            const uint32_t a = e4m3x2_to_f16x2(w & 0xffffu), b = e4m3x2_to_f16x2(w >> 16);
            x[0] = to_float<false>(a & 0xffffu); x[1] = to_float<false>(a >> 16);
            x[2] = to_float<false>(b & 0xffffu); x[3] = to_float<false>(b >> 16);
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(cache) + at));
            x[0] = to_float<Kind == kKindBf16>(w.x & 0xffffu); x[1] = to_float<Kind == kKindBf16>(w.x >> 16);
            x[2] = to_float<Kind == kKindBf16>(w.y & 0xffffu); x[3] = to_float<Kind == kKindBf16>(w.y >> 16);
        }
    };
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    auto take = [&](int t) {
        int phys = __ldg(bt + (t >> p.block_shift));
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
            if (lane == 0) atomicOr(p.status, kDevErrRange);
            phys = 0;
        }
        const size_t at = ((((static_cast<size_t>(phys) * p.num_kv_heads + h) << p.block_shift) +
                            (t & (p.block_size - 1))) * kHeadDim) + 4 * lane;
        float k[4], x[4];
        load4(p.k_cache, at, k);
        load4(p.v_cache, at, x);
        float dot = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
        for (int e = 16; e; e >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, e);
        float sc = dot * (p.scale * ks);
        if (p.cap > 0.f) sc = p.cap * tanhf(sc / p.cap);
        sc -= slope * fabsf(static_cast<float>(v.pos - t));
        const float mn = fmaxf(m, sc), a = expf(m - mn), w = expf(sc - mn);
        m = mn;
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = o[e] * a + w * x[e];
    };
    for (int t = v.lo; t < v.hi; ++t) take(t);
    if (p.masks) {
        const unsigned long long* words = p.masks + static_cast<size_t>(row) * p.mask_words;
        for (int i = 0; i < q_len; ++i)
            if (words[i >> 6] >> (i & 63) & 1) take(n - q_len + i);
    }
    const float inv = l > 0.f ? vs / l : 0.f;
    uint16_t* dst = static_cast<uint16_t*>(p.out) + (static_cast<size_t>(row) * p.num_q_heads + head) * kHeadDim + 4 * lane;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<QBf16>(o[0] * inv, o[1] * inv), pack2<QBf16>(o[2] * inv, o[3] * inv));
}

}  // namespace

cudaError_t launch_scored(CacheKind kind, bool q_bf16, const ScoredParams& p, cudaStream_t stream) {
    const long long items = static_cast<long long>(p.total_rows) * p.num_q_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((items + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (kind) {
        case kKindBf16: return cudaLaunchKernelEx(&cfg, scored_kernel<kKindBf16, true>, p);
        case kKindFp16: return cudaLaunchKernelEx(&cfg, scored_kernel<kKindFp16, false>, p);
        case kKindFp8:
            return q_bf16 ? cudaLaunchKernelEx(&cfg, scored_kernel<kKindFp8, true>, p)
                          : cudaLaunchKernelEx(&cfg, scored_kernel<kKindFp8, false>, p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
