// Attention over the paged cache whose scores or masks are not plain, on the 5th-generation
// tensor cores (sm_103a): scores capped by a tanh, biased by distance, windowed, open over a
// prefix, or masked by a tree of drafted tokens; decode rows, drafts and prompts in one launch.
//
// A row (query, head) at position pos sees the cached tokens [lo, hi) of its sequence, a tree's
// row also the nodes of its mask behind them; with x = scale q.k its score is cap tanh(x / cap)
// - slope |pos - t|, and its output the softmax of the scores times V, by a running maximum and
// sum over steps of 128 keys.
//
// Work.  A unit is one KV head and up to 256 rows (queries x the head's group) of one sequence;
// it takes the steps of 128 keys that any of its rows sees.  All units' steps are laid end to
// end and cut into one equal range per SM, whatever the lengths: a decode step over a few long
// sequences, a verification of small trees and a long prompt all fill the GPU.  A CTA takes
// its range as segments, one per unit it touches; a unit that several CTAs share leaves
// unnormalised partials (output, maximum, sum) that a second small kernel adds up.
//
// A unit of more than 128 rows is a pair: tiles A and B are its first and second 128 rows and
// share every K and V tile.  A unit of up to 128 rows (decode rows, most trees) is a solo: A
// takes the even steps and B the odd ones, with a softmax of their own, and the two are added
// up at the end through tensor memory, where both hold a row in the same lane.  Either way one
// tile's softmax runs beside the other's products, and K and V stream through a ring that runs
// ahead across segments.  Rows past the unit's are not computed: a warp whose 32 rows are all
// past them only passes the barriers.
//
// Warps: 0 walks the range, describes its segments to the others and issues every copy (TMA,
// 128-byte swizzle: a lane per 8 or 16 rows of a block of K and V, one box of queries); 1 issues
// tcgen05.mma; with a 16-bit cache 3 zeroes V rows that no row sees (0 x NaN is NaN), with an FP8
// cache 2 and 3 widen the copied e4m3 rows exactly to fp16, which costs them about as long as a
// step's products take; 4-11 and 12-19 are the softmax of tiles A and B, two threads to a row,
// each with 64 of a step's keys.  The two tiles go from segment to segment on their own (a pair's
// A ends half a step before B), and read the next segment's masks and scales, and with FP8 caches
// turn its bf16 queries to fp16, while the last products run: 8192 tokens of one prompt, 32/8
// heads, plain scores 493 -> 439 us.
// Every wait is bounded.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kRows = 128;                   // MMA M of one tile
constexpr int kKeys = 128;                   // keys per step (MMA N of S, K of P.V)
constexpr uint32_t kHalfBytes = 16384;       // [128 rows][64 elements], 128-byte swizzle
constexpr uint32_t kTileBytes = 2 * kHalfBytes;
constexpr int kSegs = 4;                     // segments described ahead
constexpr int kSegInts = 16;
constexpr int kSoftmaxWarps = 16;            // 4 ..: two threads to a row of a tile
constexpr int kWarps = 4 + kSoftmaxWarps;
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = kKeys / 2;             // a softmax thread's keys of a step
// registers per thread at launch, and the shares of warps 0-3 and the softmax after setmaxnreg
constexpr int kRegsLaunch = 96, kRegsFront = 64, kRegsSoftmax = 104;
constexpr float kRescale = 8.0f;             // lazy rescale threshold (factor 256)
// fp16 weights stand this far above the row's reference, in log2 units: the largest is then 2^14 at most,
// and what falls below fp16's range is 2^-31 of the row's largest rather than 2^-25, which would add up
// over a long context whose largest weight is a sink's
constexpr float kLift = 6.0f;

template <int Kind>
struct Cfg {
    static constexpr bool kFp8 = Kind == kKindFp8;
    static constexpr bool kMmaBf16 = Kind == kKindBf16;
    static constexpr int kStages = kFp8 ? 3 : 4;         // K and V tiles of 16-bit elements
    static constexpr int kRaw = kFp8 ? 4 : 1;            // FP8: e4m3 tiles as copied
    static constexpr uint32_t kOffStage = 2 * kTileBytes;                    // behind Q_A, Q_B
    static constexpr uint32_t kOffRaw = kOffStage + kStages * kTileBytes;
    static constexpr uint32_t kOffBars = kOffRaw + (kFp8 ? kRaw * kHalfBytes : 0);
    static constexpr uint32_t kOffSegs = kOffBars + 480;
    static constexpr uint32_t kOffRow = kOffSegs + kSegs * kSegInts * 4;     // [tile][2][128] values of rows
    static constexpr uint32_t kOffScan = kOffRow + 4 * kRows * 4;            // [kWarps]
    static constexpr uint32_t kSmem = kOffScan + 96;
};
static_assert(kSegs * kSegInts * 4 % 16 == 0 && 480 % 16 == 0, "alignment");
static_assert(32 * (4 * kRegsFront + kSoftmaxWarps * kRegsSoftmax) <= 32 * kWarps * kRegsLaunch &&
                  32 * kWarps * kRegsLaunch <= 65536, "register split above the launch total");
static_assert(Cfg<kKindBf16>::kSmem <= 232448 && Cfg<kKindFp8>::kSmem <= 232448, "shared memory");

enum {                                       // barriers, 8 bytes each
    kFull = 0,                               // [stage] a 16-bit tile has landed
    kEmpty = kFull + 5,                      // [stage]
    kRawFull = kEmpty + 5,                   // [raw stage]
    kRawEmpty = kRawFull + 4,                // [raw stage]
    kSegFull = kRawEmpty + 4,                // [segment slot]
    kSegEmpty = kSegFull + kSegs,            // [segment slot]
    kQFull = kSegEmpty + kSegs,              // [Q buffer]
    kQEmpty = kQFull + 2,                    // [Q buffer]
    kSFull = kQEmpty + 2,                    // [tile]
    kPFull = kSFull + 2,                     // [tile] P is stored, O rescaled where it had to be
    kSegDone = kPFull + 2,                   // [tile] every product of the segment is done
    kMlReady = kSegDone + 2,                             // solo: both tiles' (maximum, sum) are in shared memory
    kOFree,                                  // solo: the segment's outputs are read
    kFixed,                                  // [stage] V rows that no row sees are zeroed (edge steps)
    kIssued = kFixed + 5,                    // [stage] the copy of an edge step's V is under way
    kQLand = kIssued + 5,                    // [Q buffer] an FP8 cache's bf16 queries have landed
    kPair = kQLand + 2,                      // [tile][warp's rows] the two threads of a row have met
    kNumBars = kPair + 8
};
static_assert(kNumBars * 8 + 4 <= 480, "barriers");

// The cached tokens [lo, hi) that a row sees and its position; a tree's row also sees the nodes
// of its mask, which lie behind hi.
struct RowView {
    int pos, lo, hi;
};

// A sequence's rows and lengths; q_len is 0 where there is nothing to do.
struct SeqView {
    int q0, q_len, n, prefix;
};

__device__ __forceinline__ SeqView seq_view(const ScoredParams& p, int s, bool report) {
    SeqView v;
    v.q0 = p.query_start_loc[s];
    const int q1 = p.query_start_loc[s + 1];
    v.n = p.seq_lens[s];
    v.prefix = p.prefix_lens ? min(p.prefix_lens[s], v.n) : 0;
    v.q_len = q1 - v.q0;
    if (v.q_len == 0) return v;
    // lengths that fit q, the table and the masks
    if (v.q0 < 0 || q1 < v.q0 || q1 > p.total_rows || v.n < v.q_len || v.n > (p.max_blocks << p.block_shift) ||
        (p.masks && v.q_len > 64ll * p.mask_words)) {
        if (report) atomicOr(p.status, kDevErrRange);
        v.q_len = 0;
    }
    return v;
}

// 32 bits of a row's mask from node `at` on (negative: the nodes start inside the word).
__device__ __forceinline__ uint32_t tree_bits(const unsigned long long* words, int q_len, int at) {
    if (at >= q_len || at <= -32) return 0;
    uint32_t w;
    if (at < 0) {
        w = static_cast<uint32_t>(__ldg(words)) << -at;
        const int left = q_len - at;             // bits of the word before the tree's end
        return left < 32 ? w & ((1u << left) - 1) : w;
    }
    const int i = at >> 6, sh = at & 63;
    w = static_cast<uint32_t>(__ldg(words + i) >> sh);
    if (sh > 32 && 64 * (i + 1) < q_len) w |= static_cast<uint32_t>(__ldg(words + i + 1) << (64 - sh));
    const int left = q_len - at;
    return left < 32 ? w & ((1u << left) - 1) : w;
}

// Row j of a sequence.
__device__ __forceinline__ RowView row_view(const ScoredParams& p, const SeqView& s, int j) {
    RowView v;
    v.pos = s.n - s.q_len + j;
    v.hi = v.pos + 1;
    if (p.masks) {
        // a node's position: behind the context, as deep as its path is long
        int bits = 0;
        const unsigned long long* words = p.masks + static_cast<size_t>(s.q0 + j) * p.mask_words;
        for (int i = 0; i < s.q_len; i += 32) bits += __popc(tree_bits(words, s.q_len, i));
        v.hi = s.n - s.q_len;
        v.pos = v.hi + max(bits - 1, 0);
    } else {
        v.hi = max(v.hi, s.prefix);
    }
    v.lo = p.window > 0 ? max(0, v.pos - p.window + 1) : 0;
    return v;
}

// Unit t of a sequence: its queries [ja, ja + nq), the keys [klo, khi) that they see in all,
// and the steps of 128 keys that hold these.
struct Unit {
    int ja, nq, klo, khi, step0, steps;
};

__device__ __forceinline__ Unit unit_of(const ScoredParams& p, const SeqView& s, int t) {
    Unit u;
    u.ja = t * 2 * p.queries_per_tile;
    u.nq = min(s.q_len - u.ja, 2 * p.queries_per_tile);
    const int ctx = s.n - s.q_len;
    // position of the first row (of any node: not before the first)
    const int first = p.masks ? ctx : ctx + u.ja;
    u.khi = p.masks ? s.n : max(ctx + u.ja + u.nq, s.prefix);
    u.klo = p.window > 0 ? max(0, first - p.window + 1) : 0;
    u.step0 = u.klo / kKeys;
    u.steps = (u.khi + kKeys - 1) / kKeys - u.step0;
    return u;
}

// A unit's share of the ranges: its steps, and what beginning a unit costs in steps (the
// queries, the first scores and the last products run alone): two steps of a pair, one of a solo.
// With 1, 2, 3, 4 steps a pair, 8192 tokens of one prompt (32/8 heads) took 513, 439, 441, 447 us;
// with 1, 2 a solo, 64 decode rows of up to 8192 tokens 99.7, 101.2.
__device__ __forceinline__ int unit_lead(const ScoredParams& p, const Unit& u) { return u.nq <= p.queries_per_tile ? 1 : 2; }
__device__ __forceinline__ int unit_cost(const ScoredParams& p, const Unit& u) { return u.steps + unit_lead(p, u); }

__device__ __forceinline__ int units_per_head(const ScoredParams& p, const SeqView& s) {
    return (s.q_len + 2 * p.queries_per_tile - 1) / (2 * p.queries_per_tile);
}

// Cost of a sequence, all heads.
__device__ __forceinline__ int seq_cost(const ScoredParams& p, int s, bool report) {
    const SeqView v = seq_view(p, s, report);
    const int np = units_per_head(p, v);
    int sum = 0;
    for (int t = 0; t < np; ++t) sum += unit_cost(p, unit_of(p, v, t));
    return sum * p.num_kv_heads;             // (one sequence's: the host has checked that it fits)
}

// A segment as its CTA's warps see it: steps [step, step + steps) of a unit.
enum {
    kSegHead, kSegRow0, kSegNq, kSegStep, kSegSteps, kSegKlo, kSegKhi,
    kSegCtx,                                 // tree: tokens before it, else INT_MAX
    kSegJ0, kSegTail, kSegQLen, kSegN, kSegPrefix,   // the unit's first query, see edge_step, the sequence
    kSegFlags,                               // 1: solo, 2: the whole unit, 4: the first step is an edge
    kSegSlot                                 // where its partial goes
};

struct Seg {
    int h, row0, nq, step, steps, klo, khi, ctx, q_len, tail, flags;
};

__device__ __forceinline__ Seg read_seg(const int* d) {
    Seg g;
    g.h = d[kSegHead]; g.row0 = d[kSegRow0]; g.nq = d[kSegNq]; g.step = d[kSegStep]; g.steps = d[kSegSteps];
    g.klo = d[kSegKlo]; g.khi = d[kSegKhi]; g.ctx = d[kSegCtx]; g.q_len = d[kSegQLen];
    g.tail = d[kSegTail]; g.flags = d[kSegFlags];
    return g;
}

// Whether some of a segment's i-th step's V rows may be seen by no row: keys before the
// unit's first, from step `tail` on keys behind its last or nodes of a tree.
__device__ __forceinline__ bool edge_step(int flags, int tail, int i) { return (i == 0 && (flags & 4)) || i >= tail; }

// The keys `at` .. at + 31 that some row of the segment's unit may see (by a whole warp).
__device__ __forceinline__ uint32_t seen_keys(const ScoredParams& p, const Seg& g, int at, int lane) {
    const int a = max(g.klo - at, 0), b = min(g.khi - at, 32);
    uint32_t seen = b <= a ? 0u : (0xffffffffu << a) & (0xffffffffu >> (32 - b));
    if (at + 32 > g.ctx) {
        // nodes: those in some row's mask
        uint32_t any = 0;
        for (int j = lane; j < g.nq; j += 32)
            any |= tree_bits(p.masks + static_cast<size_t>(g.row0 + j) * p.mask_words, g.q_len, at - g.ctx);
        any = __reduce_or_sync(0xffffffffu, any);
        seen &= any | (at < g.ctx ? (1u << (g.ctx - at)) - 1 : 0u);
    }
    return seen;
}

// tcgen05.mma by descriptors' low words (address and leading offset, in 16 bytes); the high
// word is the same for every tile: 8-row groups 1024 bytes apart, version 1, 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// the same with A from tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

// Four e4m3 codes to fp16, exactly (free to be scheduled: the two warps that widen live by it).
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

// Tile order in the ring: K0, K1, V0, K2, V1, K3, ...: each K two steps ahead of its V.  Place of
// V(i) among a segment's tiles.
__device__ __forceinline__ int item_v(int steps, int i) { return min(2, steps) + i + min(i, max(steps - 2, 0)); }

// tanh(x) / x as polynomials in x^2 (interpolated at Chebyshev nodes): on |x| <= kCapTiny within
// 2^-19.7 of it, on |x| <= kCapSmall within 2^-23.7.
constexpr float kCapTiny = 0.3f, kCapSmall = 0.6f;
constexpr float kTiny0 = 0.999998835f, kTiny1 = -0.333099888f, kTiny2 = 0.126335824f;
constexpr float kTanh0 = 0.999999926f, kTanh1 = -0.33332302f, kTanh2 = 0.133100644f, kTanh3 = -0.0520966534f,
                kTanh4 = 0.0154687513f;

// c2 tanh(y) = c2 - 2 c2 / (1 + e^2y), by the exponential unit: within 2^-21 of c2.
__device__ __forceinline__ float capped_far(float y, float c2) {
    return fmaf(-2.f * c2, rcp_approx(1.f + ex2_approx(y * 2.8853900817779268f)), c2);
}

// c2 tanh(y) + add for |y| <= kCapSmall.
__device__ __forceinline__ float capped_near(float y, float c2, float add) {
    const float u = y * y;
    return fmaf(y * c2, fmaf(u, fmaf(u, fmaf(u, fmaf(u, kTanh4, kTanh3), kTanh2), kTanh1), kTanh0), add);
}

// c2 tanh(y) by the exponential unit.  Far above a score a cap rounds it to what fits the cap (at 1e6
// a tenth of a score): up to kWideCap that is 2^-13 of a score at most, half of what fp16 weights
// are rounded by; wider caps take the polynomial for scores that are small beside them, in forms of
// the kernel that only they pay for (8192 tokens of one prompt, 32/8 heads, a cap of 300: 527 -> 531 us
// where no score passes 0.6 of it, 921 -> 1829 where some do everywhere, 799 -> 1207 with a bias; at run
// time the choice cost the FP8 trees with a cap of 50 8%).
template <bool Wide>
__device__ __forceinline__ float capped(float y, float c2) {
    return Wide && fabsf(y) <= kCapSmall ? capped_near(y, c2, 0.f) : capped_far(y, c2);
}

}  // namespace

template <int Kind, bool QBf16, int Form>
__global__ void __launch_bounds__(kThreads, 1)
    scored_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap qmap, const ScoredParams p) {
    using C = Cfg<Kind>;
    constexpr bool kFp8 = C::kFp8;
    constexpr bool kMmaBf16 = C::kMmaBf16;
    constexpr bool kCapped = Form == kCappedScores || Form == kWideCappedScores;
    constexpr bool kBiased = Form == kBiasedScores || Form == kWideBiasedScores;
    constexpr bool kWide = Form == kWideCappedScores || Form == kWideBiasedScores;
    constexpr int NS = C::kStages;
    constexpr int kSegReaders = kSoftmaxWarps + (kFp8 ? 3 : 2);      // and warps 1, 3, with FP8 caches 2

    extern __shared__ __align__(1024) uint8_t sm[];             // as the 128-byte swizzle wants it
    const uint32_t sbase = smem_addr(sm);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffBars + kNumBars * 8);
    int* segs = reinterpret_cast<int*>(sm + C::kOffSegs);
    float* row_smem = reinterpret_cast<float*>(sm + C::kOffRow);
    int* scan = reinterpret_cast<int*>(sm + C::kOffScan);
    int* cum = reinterpret_cast<int*>(sm + C::kOffStage);        // only before the first copy
    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBars + 8u * i; };
    auto stage = [&](int r) -> uint32_t { return sbase + C::kOffStage + static_cast<uint32_t>(r % NS) * kTileBytes; };

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar(kFull + i), kFp8 ? 2 : 1);
            mbar_init(bar(kEmpty + i), 1);
            mbar_init(bar(kFixed + i), 1);
            mbar_init(bar(kIssued + i), 1);
        }
        for (int i = 0; i < C::kRaw; ++i) {
            mbar_init(bar(kRawFull + i), 1);
            mbar_init(bar(kRawEmpty + i), 2);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(bar(kSegFull + i), 1);
            mbar_init(bar(kSegEmpty + i), kSegReaders);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kQFull + i), kFp8 && QBf16 ? kSoftmaxWarps : 1);
            mbar_init(bar(kQEmpty + i), 1);
            mbar_init(bar(kQLand + i), 1);
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kPFull + i), 8);
            mbar_init(bar(kSegDone + i), 1);
        }
        mbar_init(bar(kMlReady), kSoftmaxWarps);
        mbar_init(bar(kOFree), kSoftmaxWarps);
        for (int i = 0; i < 8; ++i) mbar_init(bar(kPair + i), 2);
        fence_barrier_init();
        tmap_prefetch(&kmap);
        tmap_prefetch(&vmap);
        tmap_prefetch(&qmap);
    }

    grid_dependency_wait();
    grid_launch_dependents();

    // ---- cost per sequence: exclusive scan into cum ----
    // (Sums stop at 2^31 - 1, which no batch reaches whose rows are q's, each in one sequence.)
    const int B = p.num_seqs;
    {
        auto add = [](int a, int b) { return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 0x7fffffffu)); };
        const int per = (B + kThreads - 1) / kThreads;
        const int beg = min(B, static_cast<int>(threadIdx.x) * per), end = min(B, beg + per);
        int local = 0;
        for (int s = beg; s < end; ++s) {
            const int w = seq_cost(p, s, blockIdx.x == 0);
            cum[s] = w;
            local = add(local, w);
        }
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl = add(incl, y);
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        const int behind = __shfl_up_sync(0xffffffffu, incl, 1);
        int run = lane ? behind : 0;
        for (int w = 0; w < warp; ++w) run = add(run, scan[w]);
        for (int s = beg; s < end; ++s) {
            const int w = cum[s];
            cum[s] = run;
            run = add(run, w);
        }
        if (threadIdx.x == kThreads - 1) cum[B] = run;
        __syncthreads();
    }
    const int sum = cum[B];
    if (sum == INT_MAX && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, kDevErrRange);
    const int T = sum == INT_MAX ? 0 : sum;
    const int W = min(static_cast<int>(gridDim.x), T);
    const int cta = blockIdx.x;
    if (cta >= W) {
        if (threadIdx.x == 0) p.records[cta].rows = 0;
        return;
    }
    // ---- this CTA's range, found by warp 0 ----
    int f = static_cast<int>(static_cast<long long>(T) * cta / W);
    int left = static_cast<int>(static_cast<long long>(T) * (cta + 1) / W) - f;
    int cs = 0, ct = 0, ch = 0, coff = 0;    // sequence, unit, head, place within the unit's cost
    SeqView sv_cur = {};
    if (warp == 0) {
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cum[mid] <= f) lo = mid; else hi = mid;
        }
        cs = lo;
        int rem = f - cum[lo];
        sv_cur = seq_view(p, cs, false);
        const int np = units_per_head(p, sv_cur);
        // a lane per unit: the unit whose cost (all heads) holds the rest
        for (int t0 = 0; t0 < np; t0 += 32) {
            const int w = t0 + lane < np ? unit_cost(p, unit_of(p, sv_cur, t0 + lane)) * p.num_kv_heads : 0;
            int incl = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, incl > rem);
            if (past) {
                const int k = __ffs(past) - 1;
                ct = t0 + k;
                rem -= __shfl_sync(0xffffffffu, incl - w, k);
                break;
            }
            rem -= __shfl_sync(0xffffffffu, incl, 31);
        }
        const int cost = unit_cost(p, unit_of(p, sv_cur, ct));
        ch = rem / cost;
        coff = rem % cost;
    }
    fence_proxy_async_smem();                // cum was written where the first copies go
    if (warp == 1) tmem_alloc(smem_addr(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    auto tS = [&](int x) -> uint32_t { return tmem + 128u * x; };          // S, then P over its first 64 columns
    auto tO = [&](int x) -> uint32_t { return tmem + 256u + 128u * x; };
    const int G = p.group;
    const int QT = p.queries_per_tile;
    bool ok = true;

    // every role follows the segments in order
    int k = 0;                               // segments taken so far
    auto next_seg = [&](Seg& g) -> bool {
        if (!warp_wait_all(bar(kSegFull + k % kSegs), (k / kSegs) & 1, p.timeout_ns)) {
            ok = false;
            return false;
        }
        g = read_seg(segs + (k % kSegs) * kSegInts);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSegEmpty + k % kSegs));
        ++k;
        return g.steps > 0;
    };

    if (warp < 4) {
        setmaxnreg_dec<kRegsFront>();
        if (warp == 0) {
            // ================= the walk over the range, and its copies =================
            const int bsh = p.block_shift;
            const int rsh = min(bsh, 4);                          // log2 of a piece's rows
            const int per_step = kKeys >> rsh;                    // pieces per step: 8 or 16
            if (lane == 0) p.records[cta].rows = 0;
            SeqView at = sv_cur;
            int r = 0;                                            // tiles copied so far
            // bit b: the Q buffer was filled, parity of its fills, of its releases
            unsigned q_used = 0, q_sent = 0, q_par = 0;
            while (ok) {
                // the range's part of the next unit, places [coff, coff + take) of its cost, of which
                // the first `lead` stand for its start: steps [a, b)
                Unit u = {};
                SeqView sv = at;
                int a = 0, steps = 0, seq = cs, head = ch, cost = 0, unit_f = f;
                while (left > 0 && steps == 0) {
                    u = unit_of(p, at, ct);
                    const int lead = unit_lead(p, u);
                    cost = u.steps + lead;
                    const int take = min(left, cost - coff);
                    a = max(coff - lead, 0);
                    steps = max(coff + take - lead, 0) - a;       // 0: nothing but the start, the next CTA has the steps
                    sv = at;
                    seq = cs;
                    head = ch;
                    unit_f = f - coff;
                    f += take;
                    left -= take;
                    coff = 0;
                    if (left > 0 && ++ch == p.num_kv_heads) {
                        ch = 0;
                        if (++ct == units_per_head(p, at)) {
                            ct = 0;
                            do {
                                at = seq_view(p, ++cs, false);
                            } while (at.q_len == 0);
                        }
                    }
                }
                const bool solo = u.nq <= QT;
                const int row0 = sv.q0 + u.ja, step0 = u.step0 + a;
                int flags = solo ? 1 : 0, tail = 0;
                // ---- its description ----
                {
                    const int sl = k % kSegs;
                    if (k >= kSegs && !warp_wait_all(bar(kSegEmpty + sl), ((k / kSegs) - 1) & 1, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    ++k;
                    const bool starts = a == 0, ends = a + steps == u.steps;
                    const int ctx = p.masks ? sv.n - sv.q_len : INT_MAX;
                    flags |= (starts && ends ? 2 : 0) | (step0 * kKeys < u.klo ? 4 : 0);
                    // the first step that reaches behind the last key, or the first node
                    tail = max(min(u.khi, ctx) / kKeys - step0, 0);
                    if (lane == 0) {
                        int* d = segs + sl * kSegInts;
                        d[kSegHead] = head;
                        d[kSegRow0] = row0;
                        d[kSegNq] = u.nq;
                        d[kSegStep] = step0;
                        d[kSegSteps] = steps;
                        d[kSegKlo] = u.klo;
                        d[kSegKhi] = u.khi;
                        d[kSegCtx] = ctx;
                        d[kSegJ0] = u.ja;
                        d[kSegTail] = tail;
                        d[kSegQLen] = sv.q_len;
                        d[kSegN] = sv.n;
                        d[kSegPrefix] = sv.prefix;
                        d[kSegFlags] = flags;
                        // a partial that continues another CTA's unit goes to the CTA's first slot, one
                        // that starts a unit to its second: the range has one of each at most
                        d[kSegSlot] = 2 * cta + (starts ? 1 : 0);
                        mbar_arrive(bar(kSegFull + sl));
                    }
                    if (steps == 0) break;                        // the range's end
                    if (starts && !ends && lane == 0) {
                        // the CTA whose range holds the unit's last step
                        const int last = static_cast<int>(((static_cast<long long>(unit_f) + cost) * W - 1) / T);
                        p.records[cta] = CombineRecord{u.nq * G, row0, head * G, solo ? 1 : 0, last, {0, 0, 0}};
                    }
                }
                // ---- its copies ----
                // a solo's keys are read once, beside partials and tables that are read again: they leave
                // L2 first (16 x 8192 tokens, trees of 24: 70.6 -> 66.6 us)
                const uint64_t policy = solo ? l2_policy_evict_first() : l2_policy_evict_normal();
                const int32_t* bt = p.block_tables + static_cast<size_t>(seq) * p.max_blocks;
                const int c_lo = u.klo >> rsh, c_hi = (u.khi - 1) >> rsh;     // pieces that hold keys
                // the lane's piece of a step: its row in the cache, -1 for none
                auto entry = [&](int i) -> int {
                    const int c = (step0 + i) * per_step + lane;
                    if (i >= steps || lane >= per_step || c < c_lo || c > c_hi) return -1;
                    const int key = c << rsh;
                    int phys = __ldg(bt + (key >> bsh));
                    if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
                        atomicOr(p.status, kDevErrRange);
                        phys = 0;
                    }
                    return ((phys * p.num_kv_heads + head) << bsh) + (key & (p.block_size - 1));
                };
                auto copy = [&](const CUtensorMap* map, int y) {
                    constexpr int kRing = kFp8 ? C::kRaw : NS;
                    constexpr int kF = kFp8 ? static_cast<int>(kRawFull) : static_cast<int>(kFull);
                    constexpr int kE = kFp8 ? static_cast<int>(kRawEmpty) : static_cast<int>(kEmpty);
                    const int st = r % kRing;
                    if (!ok || (r >= kRing && !warp_wait_all(bar(kE + st), ((r / kRing) - 1) & 1, p.timeout_ns))) {
                        ok = false;
                        return;
                    }
                    const unsigned live = __ballot_sync(0xffffffffu, y >= 0);
                    const uint32_t full = bar(kF + st);
                    if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(live)) * ((kFp8 ? 128u : 256u) << rsh));
                    __syncwarp();
                    if (y >= 0) {
                        if constexpr (kFp8) {
                            tma_load_2d_hint(sbase + C::kOffRaw + st * kHalfBytes + (lane << rsh) * 128, map, 0, y, full, policy);
                        } else {
                            const uint32_t dst = sbase + C::kOffStage + st * kTileBytes + (lane << rsh) * 128;
                            tma_load_2d_hint(dst, map, 0, y, full, policy);
                            tma_load_2d_hint(dst + kHalfBytes, map, 64, y, full, policy);
                        }
                    }
                    ++r;
                };
                // K0, the queries, K1, then V(i), K(i + 2); the table's entries ahead of their use
                int y0 = entry(0), y1 = entry(1), y2 = entry(2);
                copy(&kmap, y0);
                for (int x = 0; x < (solo ? 1 : 2) && ok; ++x) {
                    // one copy of QT queries x G heads; those past the unit's are other rows or zeros and
                    // end in rows of S that nothing reads
                    const int b = solo ? (k - 1) & 1 : x;
                    if (q_used >> b & 1) {
                        if (!warp_wait_all(bar(kQEmpty + b), q_par >> b & 1, p.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        q_par ^= 1u << b;
                    }
                    q_used |= 1u << b;
                    q_sent ^= 1u << b;
                    const uint32_t landed = bar((kFp8 && QBf16 ? kQLand : kQFull) + b), dst = sbase + b * kTileBytes;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(landed, static_cast<uint32_t>(QT * G) * 256);
                        tma_load_3d(dst, &qmap, 0, head * G, row0 + x * QT, landed);
                        tma_load_3d(dst + kHalfBytes, &qmap, 64, head * G, row0 + x * QT, landed);
                    }
                    __syncwarp();
                }
                if (steps > 1) copy(&kmap, y1);
                for (int i = 0; i < steps && ok; ++i) {
                    const int y3 = entry(i + 3);
                    copy(&vmap, y0);
                    // (the tile's barrier is in its phase from here until the zeroing is done)
                    if (!kFp8 && ok && lane == 0 && edge_step(flags, tail, i)) mbar_arrive(bar(kIssued + (r - 1) % NS));
                    if (i + 2 < steps) copy(&kmap, y2);
                    y0 = y1;
                    y1 = y2;
                    y2 = y3;
                }
            }
            if (!ok) {
                if (lane == 0) atomicOr(p.status, kDevErrTimeout);
                // let the copies still in flight land before the CTA leaves
                constexpr int kRing = kFp8 ? C::kRaw : NS;
                constexpr int kF = kFp8 ? static_cast<int>(kRawFull) : static_cast<int>(kFull);
                for (int i = max(0, r - kRing); i < r; ++i) warp_wait_all(bar(kF + i % kRing), (i / kRing) & 1, p.timeout_ns);
                for (int b = 0; b < 2; ++b)
                    if (q_used >> b & 1) warp_wait_all(bar((kFp8 && QBf16 ? kQLand : kQFull) + b), (q_sent >> b & 1) ^ 1u, p.timeout_ns);
            }
        } else if (warp == 1) {
            // ================= MMA issuer =================
            // The whole warp walks along, so that addresses stay uniform and need no moves, and one
            // lane issues.  What it does between two products is time in which the tensor cores run
            // dry: places in the ring are counted on, not divided out, and the tiles of the next step
            // are waited for behind the last product of this one.
            constexpr uint32_t idS = umma_idesc_f16<kMmaBf16>(kRows, kKeys, false);
            constexpr uint32_t idPV = umma_idesc_f16<kMmaBf16>(kRows, kHeadDim, true);
            const bool leader = lane == 0;
            const uint32_t tiles = (sbase + C::kOffStage) >> 4, q_tiles = sbase >> 4;      // in units of 16 bytes
            int st = 0;                              // the next tile's stage, and the parity of its filling
            uint32_t ph = 0;
            auto wait = [&](uint32_t b, uint32_t par) -> bool {
                if (!warp_wait_all(b, par, p.timeout_ns)) ok = false;
                return ok;
            };
            auto advance = [&]() {
                if (++st == NS) {
                    st = 0;
                    ph ^= 1u;
                }
            };
            auto issue_s = [&](int x, int q, int stage_k) {
                if (leader) {
                    const uint32_t a = (q_tiles + q * (kTileBytes >> 4)) | (1u << 16);
                    const uint32_t b = (tiles + stage_k * (kTileBytes >> 4)) | (1u << 16);
#pragma unroll
                    for (int kk = 0; kk < kHeadDim / 16; ++kk) {
                        const uint32_t at = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
                        mma_ss(tS(x), a + at, b + at, idS, kk > 0);
                    }
                    umma_commit(bar(kSFull + x));
                }
            };
            // P.V over the step's keys; V is MN-major: d-halves kHalfBytes apart, 16 keys = 2 KiB
            auto issue_pv = [&](int x, int stage_v, bool first) {
                if (leader) {
                    const uint32_t b = (tiles + stage_v * (kTileBytes >> 4)) | ((kHalfBytes >> 4) << 16);
#pragma unroll
                    for (int e = 0; e < kKeys / 16; ++e) mma_ts(tO(x), tS(x) + 8 * e, b + e * 128, idPV, !first || e > 0);
                }
            };
            auto commit = [&](int b) {
                if (leader) umma_commit(bar(b));
            };
            // parities as bits: an array indexed at run time would live in local memory
            unsigned fixes = 0;                      // bit st: of the stage's zeroings
            unsigned q_par = 0, p_par = 0;           // bit x: of the buffer's fills, of the tile's P
            // P of tile x and whatever else the products need, asked for together: each test takes a
            // hundred cycles or so, side by side no more than one
            auto p_and = [&](int x, uint32_t b1, uint32_t par1, uint32_t b2, uint32_t par2) -> bool {
                const bool p0 = mbar_test(bar(kPFull + x), p_par >> x & 1), p1 = mbar_test(b1, par1), p2 = mbar_test(b2, par2);
                if (!__all_sync(0xffffffffu, p0 && p1 && p2) &&
                    !(wait(b1, par1) && wait(b2, par2) && wait(bar(kPFull + x), p_par >> x & 1)))
                    return false;
                p_par ^= 1u << x;
                tc_fence_after();
                return true;
            };
            int seg = 0;
            while (ok) {
                if (!wait(bar(kSegFull + seg % kSegs), (seg / kSegs) & 1)) break;
                const int* d = segs + (seg % kSegs) * kSegInts;
                const int n = __shfl_sync(0xffffffffu, d[kSegSteps], 0), flags = __shfl_sync(0xffffffffu, d[kSegFlags], 0);
                const int tail = __shfl_sync(0xffffffffu, d[kSegTail], 0);
                if (leader) mbar_arrive(bar(kSegEmpty + seg % kSegs));
                if (n == 0) break;
                const bool solo = flags & 1;
                const int qa = solo ? seg & 1 : 0, qb = solo ? qa : 1;
                if (!wait(bar(kQFull + qa), q_par >> qa & 1)) break;
                q_par ^= 1u << qa;
                if (!solo) {
                    if (!wait(bar(kQFull + 1), q_par >> 1 & 1)) break;
                    q_par ^= 2u;
                }
                auto q_free = [&]() {                // behind the segment's last S
                    commit(kQEmpty + qa);
                    if (!solo) commit(kQEmpty + 1);
                };
                // V of step i is at place v_st: its unseen rows have to be zeroed
                auto v_fixed = [&](int i, int v_st) -> bool {
                    if (!kFp8 && edge_step(flags, tail, i)) {
                        if (!wait(bar(kFixed + v_st), fixes >> v_st & 1)) return false;
                        fixes ^= 1u << v_st;
                    }
                    return true;
                };
                if (!wait(bar(kFull + st), ph)) break;
                tc_fence_after();
                issue_s(0, qa, st);
                if (!solo) issue_s(1, qb, st);
                commit(kEmpty + st);
                if (n == 1) q_free();
                advance();
                if (solo) {
                    if (n > 1) {
                        if (!wait(bar(kFull + st), ph)) break;
                        tc_fence_after();
                        issue_s(1, qa, st);
                        commit(kEmpty + st);
                        if (n == 2) q_free();
                        advance();
                    }
                    for (int i = 0; i < n; ++i) {
                        // V(i), then K(i + 2) for the same tile
                        const int v_st = st, x = i & 1;
                        const uint32_t v_bar = bar(kFull + st);
                        if (!v_fixed(i, v_st) || !p_and(x, v_bar, ph, v_bar, ph)) break;
                        issue_pv(x, v_st, i < 2);
                        commit(kEmpty + v_st);
                        advance();
                        if (i + 2 < n) {
                            if (!wait(bar(kFull + st), ph)) break;
                            tc_fence_after();
                            issue_s(x, qa, st);
                            commit(kEmpty + st);
                            if (i + 3 == n) q_free();
                            advance();
                        }
                    }
                    // (B's warps are in this segment too, if it has no step for them)
                    if (n == 1) {
                        if (!wait(bar(kPFull + 1), p_par >> 1 & 1)) break;
                        p_par ^= 2u;
                    }
                    if (!ok) break;
                    commit(kSegDone);
                } else {
                    for (int i = 0; i < n; ++i) {
                        // K(i + 1) and V(i), for both tiles
                        const bool more = i + 1 < n;
                        const int k_st = st;
                        const uint32_t k_bar = bar(kFull + st), k_ph = ph;
                        if (more) advance();
                        const int v_st = st;
                        const uint32_t v_bar = bar(kFull + st);
                        if (!v_fixed(i, v_st) || !p_and(0, more ? k_bar : v_bar, more ? k_ph : ph, v_bar, ph)) break;
                        issue_pv(0, v_st, i == 0);
                        if (more) issue_s(0, 0, k_st);
                        else commit(kSegDone);
                        if (!p_and(1, v_bar, ph, v_bar, ph)) break;
                        issue_pv(1, v_st, i == 0);
                        if (more) issue_s(1, 1, k_st);
                        commit(kEmpty + v_st);
                        if (more) commit(kEmpty + k_st);
                        if (i + 2 == n) q_free();
                        advance();
                    }
                }
                if (!ok) break;
                commit(kSegDone + 1);
                ++seg;
            }
            if (!ok && leader) atomicOr(p.status, kDevErrTimeout);
            __syncwarp();
        } else if (kFp8) {
            // ================= FP8: e4m3 rows to fp16 tiles, two of a tile's rows a thread =================
            const int part = warp - 2;
            int r = 0;
            Seg g;
            while (ok && next_seg(g)) {
                const int two = min(2, g.steps), both = 2 * max(g.steps - 2, 0);
                for (int it = 0; it < 2 * g.steps && ok; ++it, ++r) {
                    // the item's step, and whether it is V
                    int i = it;
                    bool is_v = false;
                    if (it >= two) {
                        const int e = it - two;
                        is_v = e >= both || !(e & 1);
                        i = (e < both ? e >> 1 : e - both / 2) + (is_v ? 0 : 2);
                    }
                    uint32_t seen[2] = {0xffffffffu, 0xffffffffu};     // keys 32 (2 e + part) .. that some row sees
                    const int key0 = (g.step + i) * kKeys;
                    if (is_v && edge_step(g.flags, g.tail, i)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) seen[e] = seen_keys(p, g, key0 + 32 * (2 * e + part), lane);
                    }
                    const int rs = r % C::kRaw, st = r % NS;
                    if (!warp_wait_all(bar(kRawFull + rs), (r / C::kRaw) & 1, p.timeout_ns) ||
                        (r >= NS && !warp_wait_all(bar(kEmpty + st), ((r / NS) - 1) & 1, p.timeout_ns))) {
                        ok = false;
                        break;
                    }
                    // a row's eight 16-byte chunks are read and its sixteen written at places that differ
                    // from row to row by an exclusive or with the row's low bits
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const int row = 32 * (2 * h + part) + lane;
                        const uint32_t swz = (row & 7) << 4;
                        const uint32_t src = sbase + C::kOffRaw + rs * kHalfBytes + row * 128;
                        const uint32_t dst = stage(r) + row * 128;
                        uint4 x8[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) x8[e] = ld_shared_16(src + ((e << 4) ^ swz));
                        if (!((h ? seen[1] : seen[0]) >> lane & 1)) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x8[e] = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t w[4] = {x8[e].x, x8[e].y, x8[e].z, x8[e].w};
                            uint32_t f16[8];
#pragma unroll
                            for (int a = 0; a < 4; ++a) widen4(w[a], f16[2 * a], f16[2 * a + 1]);
                            const uint32_t d = dst + (e >> 2) * kHalfBytes;
                            st_shared_16(d + ((((e & 3) * 2) << 4) ^ swz), make_uint4(f16[0], f16[1], f16[2], f16[3]));
                            st_shared_16(d + ((((e & 3) * 2 + 1) << 4) ^ swz), make_uint4(f16[4], f16[5], f16[6], f16[7]));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(kFull + st));
                        mbar_arrive(bar(kRawEmpty + rs));
                    }
                }
            }
            if (!ok && lane == 0) atomicOr(p.status, kDevErrTimeout);
        } else if (warp == 3) {
            // ================= 16-bit caches: V rows that no row sees =================
            int r0 = 0;
            unsigned issued = 0;                     // bit st: parity of the stage's edge copies
            Seg g;
            while (ok && next_seg(g)) {
                for (int i = 0; i < g.steps && ok; ++i) {
                    const int key0 = (g.step + i) * kKeys;
                    if (!edge_step(g.flags, g.tail, i)) continue;
                    const int r = r0 + item_v(g.steps, i);
                    uint32_t seen[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) seen[w] = seen_keys(p, g, key0 + 32 * w, lane);
                    // not before its copy is issued: the stage may still be a phase or two behind
                    if (!warp_wait_all(bar(kIssued + r % NS), issued >> (r % NS) & 1, p.timeout_ns) ||
                        !warp_wait_all(bar(kFull + r % NS), (r / NS) & 1, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    issued ^= 1u << (r % NS);
                    uint8_t* vst = sm + C::kOffStage + (r % NS) * kTileBytes;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int row = 32 * w + lane;
                        if (seen[w] >> lane & 1) continue;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            *reinterpret_cast<uint4*>(vst + row * 128 + 16 * c) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4*>(vst + kHalfBytes + row * 128 + 16 * c) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kFixed + r % NS));
                }
                r0 += 2 * g.steps;
            }
            if (!ok && lane == 0) atomicOr(p.status, kDevErrTimeout);
        }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        // ================= softmax: tile A's warps, then tile B's; two threads to a row =================
        constexpr int NC = kCols;
        const int x = (warp - 4) / 8;
        const int half = (warp - 4) / 4 % 2;           // the thread's keys of a step: NC half ..
        const int quarter = warp & 3;                  // tensor-memory lanes 32 quarter .. + 31
        const int r = quarter * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t s_addr = tS(x) + lane_off + NC * half;               // its scores
        const uint32_t p_addr = s_addr - NC / 2 * half;                     // its P, 16 bits each
        const int exch = (2 * x + half) * kRows + r;   // in row_smem; the row's other thread: exch ^ kRows
        // parities: 1 of S, 2 of the solos, 4 of the meetings, 8 and 16 of the Q buffers' copies
        unsigned par = 0;
        auto come = [&]() {                            // to a meeting of both threads of the row
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kPair + 4 * x + quarter));
        };
        auto met = [&]() -> bool {
            if (!warp_wait_all(bar(kPair + 4 * x + quarter), par >> 2 & 1, p.timeout_ns)) ok = false;
            par ^= 4u;
            return ok;
        };
        auto meet = [&]() -> bool {
            come();
            return met();
        };
        // Registers are short (a thread's scores take most of them, and a spill misses the little
        // L1 that is left; up to 48 bytes are spilled all the same): a segment's fields are read from shared memory where they are used,
        // and its slot is given back when its outputs are written.
        // What a segment's row needs from global memory is read ahead, while the products of the
        // segment before it end.
        RowView next_view;
        float next_kscale = 1.0f, next_slope2 = 0.f;
        bool next_live = false, more = false;
        auto look_ahead = [&]() {
            if (!warp_wait_all(bar(kSegFull + k % kSegs), (k / kSegs) & 1, p.timeout_ns)) {
                ok = more = false;
                return;
            }
            const int* d = segs + (k % kSegs) * kSegInts;
            more = d[kSegSteps] != 0;
            if (!more) return;
            const int jq = (d[kSegFlags] & 1 ? 0 : x * QT) + r / G;
            next_live = r < QT * G && jq < d[kSegNq];
            next_view = RowView{0, 0, INT_MAX};
            if (next_live)
                next_view = row_view(p, SeqView{d[kSegRow0] - d[kSegJ0], d[kSegQLen], d[kSegN], d[kSegPrefix]}, d[kSegJ0] + jq);
            if (kFp8) next_kscale = __ldg(p.k_scale + d[kSegHead] * p.scale_stride);
            if (kBiased && p.slopes)
                next_slope2 = next_live ? __ldg(p.slopes + d[kSegHead] * G + r % G) * 1.4426950408889634f : 0.f;
            if constexpr (kFp8 && QBf16) {
                // its queries, bf16 to fp16 as the widened codes: exact for magnitudes 2^-14 to 65504, 2^-25
                // off below, infinite above.  A pair's tile by its own warps, a solo's by all.
                const bool solo = d[kSegFlags] & 1;
                const int b = solo ? k & 1 : x;
                if (!warp_wait_all(bar(kQLand + b), par >> (3 + b) & 1, p.timeout_ns)) {
                    ok = more = false;
                    return;
                }
                par ^= solo ? 8u << b : 24u;
                uint4* q = reinterpret_cast<uint4*>(sm + b * kTileBytes);
                const int chunks = min(QT, d[kSegNq] - (solo ? 0 : x * QT)) * G * 8;      // of 16 bytes, in each half
#pragma unroll 1
                for (int c = (warp - 4 - (solo ? 0 : 8 * x)) * 32 + lane; c < chunks; c += solo ? 512 : 256) {
                    uint4 v[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) v[e] = q[e * (kHalfBytes / 16) + c];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
                        for (int a = 0; a < 4; ++a)
                            w[a] = pack2<false>(to_float<true>(w[a] & 0xffffu), to_float<true>(w[a] >> 16));
                        q[e * (kHalfBytes / 16) + c] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_n(bar(kQFull + b), solo ? 1 : 2);
            }
        };
        look_ahead();
        while (more) {
            const int* d = segs + (k % kSegs) * kSegInts;
            ++k;
            const bool solo = d[kSegFlags] & 1;
            const RowView view = next_view;
            const float kscale = next_kscale;
            [[maybe_unused]] const float slope2 = next_slope2;
            const bool live = next_live;
            const bool warp_live = __any_sync(0xffffffffu, live);
            // never 0: hidden scores are infinite, and stay so under it
            const float s_raw = p.scale_log2 * kscale;
            const float s_log2 = s_raw == 0.f ? 1e-30f : s_raw;
            [[maybe_unused]] auto k_cap = [&]() {       // of a score, to x / cap
                const float k = p.cap_scale * kscale;
                return k == 0.f ? 1e-30f : k;
            };
            float m_used = -INFINITY, l = 0.f;
            int key0 = (d[kSegStep] + (solo ? x : 0)) * kKeys + NC * half;
            for (int left_steps = solo ? (d[kSegSteps] + 1 - x) >> 1 : d[kSegSteps]; left_steps > 0;
                 --left_steps, key0 += (d[kSegFlags] & 1 ? 2 : 1) * kKeys) {
                if (!warp_wait_all(bar(kSFull + x), par & 1, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                par ^= 1u;
                if (!warp_live) {                       // rows past the unit's: nothing reads their P
                    if (lane == 0) mbar_arrive(bar(kPFull + x));
                    continue;
                }
                tc_fence_after();
                const bool need_mask = __any_sync(0xffffffffu, key0 < view.lo || key0 + NC > view.hi);
                // what the row sees of the thread's keys
                uint32_t vis[NC / 32];
#pragma unroll
                for (int w = 0; w < NC / 32; ++w) vis[w] = 0xffffffffu;
                if (need_mask) {
#pragma unroll
                    for (int w = 0; w < NC / 32; ++w) {
                        const int base = key0 + 32 * w;
                        const int a = max(view.lo - base, 0), b = min(view.hi - base, 32);
                        vis[w] = b <= a ? 0u : (0xffffffffu << a) & (0xffffffffu >> (32 - b));
                        if (p.masks && live) {
                            const size_t row = static_cast<size_t>(d[kSegRow0] + (solo ? 0 : x * QT) + r / G);
                            vis[w] |= tree_bits(p.masks + row * p.mask_words, d[kSegQLen], base - d[kSegCtx]);
                        }
                    }
                }
                __syncwarp();
                // the scores in registers: one tensor-memory round trip per step
                uint32_t sv[NC];
#pragma unroll
                for (int c = 0; c < NC / 32; ++c)
                    tmem_ld32(s_addr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * c));
                tmem_wait_ld();
                // The row's maximum, of what the maximum of the scores follows: a cap is monotone, so that
                // of the raw scores will do; biased scores are computed first.  (A negative scale turns
                // the order round.)  Hidden scores are infinite on the far side.
                const float mul = kBiased ? 1.0f : s_log2;
                const bool upward = kBiased || s_log2 >= 0.f;
                if constexpr (kBiased) {
                    // a cap first: a rare pair, so without the short polynomials (what stands in hidden
                    // places, keys that were never copied, stays there)
                    if (p.cap > 0.f) {
                        const float c2 = p.cap_log2, k1 = p.cap_scale * kscale;
#pragma unroll
                        for (int e = 0; e < NC; ++e)
                            sv[e] = __float_as_uint(capped<kWide>(__uint_as_float(sv[e]) * k1, c2));
                    }
                    const float by = p.cap > 0.f ? 1.0f : s_log2;
                    const uint64_t by2 = f2_pack(by, by);
                    if (__all_sync(0xffffffffu, !live || key0 + NC - 1 <= view.pos)) {
                        // every key at or before every row: the bias grows by slope2 from key to key, and
                        // is counted on for four pairs from a place that is computed
                        const uint64_t step2 = f2_pack(2.f * slope2, 2.f * slope2);
                        const float base = static_cast<float>(key0 - view.pos);
#pragma unroll
                        for (int c = 0; c < NC / 8; ++c) {
                            const float b0 = slope2 * (base + static_cast<float>(8 * c));
                            uint64_t b2 = f2_pack(b0, b0 + slope2);
#pragma unroll
                            for (int e = 8 * c; e < 8 * c + 8; e += 2) {
                                float a0, a1;
                                f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), by2, b2), a0, a1);
                                sv[e] = __float_as_uint(a0);
                                sv[e + 1] = __float_as_uint(a1);
                                b2 = f2_add(b2, step2);
                            }
                        }
                    } else {
                        const float base = static_cast<float>(key0 - view.pos);
#pragma unroll
                        for (int e = 0; e < NC; ++e)
                            sv[e] = __float_as_uint(fmaf(__uint_as_float(sv[e]), by, -slope2 * fabsf(base + static_cast<float>(e))));
                    }
                }
                if (need_mask) {
                    const float hidden = upward ? -INFINITY : INFINITY;
#pragma unroll
                    for (int e = 0; e < NC; ++e)
                        sv[e] = vis[e >> 5] >> (e & 31) & 1 ? sv[e] : __float_as_uint(hidden);
                }
                float mx;
                {
                    // four independent chains
                    float e4[4];
                    if (upward) {
                        e4[0] = e4[1] = e4[2] = e4[3] = -INFINITY;
#pragma unroll
                        for (int e = 0; e < NC; e += 2)
                            e4[(e >> 1) & 3] = max3f(e4[(e >> 1) & 3], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                        mx = fmaxf(fmaxf(e4[0], e4[1]), fmaxf(e4[2], e4[3]));
                    } else {
                        e4[0] = e4[1] = e4[2] = e4[3] = INFINITY;
#pragma unroll
                        for (int e = 0; e < NC; e += 2)
                            e4[(e >> 1) & 3] = min3f(e4[(e >> 1) & 3], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                        mx = fminf(fminf(e4[0], e4[1]), fminf(e4[2], e4[3]));
                    }
                    mx *= kCapped ? k_cap() : mul;
                }
                // The form of the tanh, one for the warp's part of the step: the shortest polynomial where
                // the largest x / cap of every row lies in [-0.1, 0.3] and the cap is 40 or more: what lies
                // below -0.3 then weighs e^-7.7 at most, and beyond the polynomial's range, where it falls
                // faster than the tanh, next to nothing.  Else by the largest |x / cap|.  Not the shortest where its
                // highest coefficient would leave float's range: 0 does not hide an infinite score.
                int tanh_form = 0;
                if constexpr (kCapped) {
                    const float k1 = k_cap();
                    if (__any_sync(0xffffffffu, live && !(mx >= -0.1f && mx <= kCapTiny)) || p.cap < 40.f || fabsf(k1) < p.cap_flat) {
                        float am = 0.f;
#pragma unroll
                        for (int e = 0; e < NC; ++e) {
                            const float v = fabsf(__uint_as_float(sv[e]));
                            am = fmaxf(am, v < INFINITY ? v : 0.f);
                        }
                        am = live ? fmaxf(am * fabsf(k1), mx) : 0.f;        // mx: an infinite score that is seen
                        tanh_form = __any_sync(0xffffffffu, am > kCapSmall) ? 2
                                    : __any_sync(0xffffffffu, am > kCapTiny || fabsf(k1) < p.cap_flat) ? 1 : 0;
                    }
                }
                // with the row's other thread, which has read its scores too: P may go over them
                row_smem[exch] = mx;
                tc_fence_before();
                if (!meet()) break;
                tc_fence_after();
                mx = fmaxf(mx, row_smem[exch ^ kRows]);
                if constexpr (kCapped) {
                    // the row's maximum capped (a reference: what matters is that both threads take the same)
                    const float c2 = p.cap_log2;
                    if (__any_sync(0xffffffffu, live && !(fabsf(mx) <= kCapTiny))) {
                        mx = mx == -INFINITY ? mx : capped_far(mx, c2);
                    } else {
                        const float u = mx * mx;
                        mx *= c2 * fmaf(u, fmaf(u, kTiny2, kTiny1), kTiny0);
                    }
                }
                const bool need = live && mx > m_used + kRescale;
                const bool resc = __any_sync(0xffffffffu, need && m_used > -INFINITY);
                const float m_new = need ? mx : m_used;
                // a row that has seen nothing yet: exponents against 0, all of hidden scores
                const float m_at = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = ex2_approx(m_used - m_at);    // 0 before the row's first key, 1 when kept
                const float neg_m = (kMmaBf16 ? 0.f : kLift) - m_at;
                m_used = m_new;
                // O is final for the products before: S(i) was issued behind them.  Rescaled
                // before any of P(i) is released, since P.V(i) accumulates into it.
                if (resc) {
#pragma unroll 1
                    for (int c = 0; c < kHeadDim / 32; ++c) {       // few registers beside the scores
                        const uint32_t o_addr = tO(x) + lane_off + kHeadDim / 2 * half + 16 * c;
                        uint32_t ov[16];
                        tmem_ld16(o_addr, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                        tmem_st16(o_addr, ov);
                    }
                }
                __syncwarp();          // (and nothing below is begun above: it would spill)
                // p = 2^(s * scale - m), rounded to the 16 bits that the tensor cores take beside V's
                // (bf16 2^-8 of it at most, fp16, FP8 caches' type too, 2^-11, times 2^kLift; their sum is of
                // the unrounded ones), written over the columns of S (keys 32 c .. +31 -> columns 16 c
                // .. +15).  P in two 16-bit parts would double the products of P.V.
                float sum;
                if constexpr (!kCapped) {
                    uint64_t sum2[2] = {0ull, 0ull};
                    const uint64_t negm2 = f2_pack(neg_m, neg_m), scale2 = f2_pack(mul, mul);
#pragma unroll
                    for (int c = 0; c < NC / 16; ++c) {
                        uint32_t pw[8];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const uint64_t v = f2_pack(__uint_as_float(sv[16 * c + e]), __uint_as_float(sv[16 * c + e + 1]));
                            float a0, a1;
                            f2_unpack(Form == kPlainScores ? f2_fma(v, scale2, negm2) : f2_add(v, negm2), a0, a1);
                            const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);     // hidden: 0
                            sum2[(e >> 1) & 1] = f2_add(sum2[(e >> 1) & 1], f2_pack(p0, p1));
                            pw[e >> 1] = pack2<kMmaBf16>(p0, p1);
                        }
                        tmem_st8(p_addr + 8 * c, pw);
                    }
                    float s0, s1, s2, s3;
                    f2_unpack(sum2[0], s0, s1);
                    f2_unpack(sum2[1], s2, s3);
                    sum = (s0 + s1) + (s2 + s3);
                } else {
                    // cap tanh(x / cap) less the maximum, x a score before the scale: a polynomial where |x /
                    // cap| is small, nearly always (caps lie far above most scores), four operations with
                    // the scale and the maximum folded in, or eight with its coefficients in the
                    // instructions; else by the exponential unit, which the softmax waits for too
                    // (tanh.approx is 2^-11 off, 0.02 of a score at a cap of 50).  One score at a time:
                    // packed pairs take twice the registers for what is the same in both, and spilled.
                    float sums[2] = {0.f, 0.f};
                    auto store_p = [&](auto exponent) {
#pragma unroll
                        for (int c = 0; c < NC / 16; ++c) {
                            uint32_t pw[8];
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                float a0, a1;
                                exponent(__uint_as_float(sv[16 * c + e]), __uint_as_float(sv[16 * c + e + 1]), a0, a1);
                                const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);     // hidden: 0
                                sums[0] += p0;
                                sums[1] += p1;
                                pw[e >> 1] = pack2<kMmaBf16>(p0, p1);
                            }
                            tmem_st8(p_addr + 8 * c, pw);
                        }
                    };
                    const float k1 = k_cap();
                    if (tanh_form == 0) {
                        const float d0 = kTiny0 * s_log2, d1 = kTiny1 * s_log2 * (k1 * k1), d2 = kTiny2 * s_log2 * (k1 * k1) * (k1 * k1);
                        const uint64_t c0 = f2_pack(d0, d0), c1 = f2_pack(d1, d1), c2 = f2_pack(d2, d2), negm2 = f2_pack(neg_m, neg_m);
                        store_p([&](float v0, float v1, float& a0, float& a1) {
                            const uint64_t v = f2_pack(v0, v1), u = f2_mul(v, v);
                            f2_unpack(f2_fma(v, f2_fma(u, f2_fma(u, c2, c1), c0), negm2), a0, a1);
                        });
                    } else if (tanh_form == 1) {
                        auto one = [&](float v) { return capped_near(v * k1, p.cap_log2, neg_m); };
                        store_p([&](float v0, float v1, float& a0, float& a1) {
                            a0 = one(v0);
                            a1 = one(v1);
                        });
                    } else {
                        auto one = [&](float v) {
                            const float t = capped<kWide>(v * k1, p.cap_log2) + neg_m;
                            return v * k1 == -INFINITY ? -INFINITY : t;
                        };
                        store_p([&](float v0, float v1, float& a0, float& a1) {
                            a0 = one(v0);
                            a1 = one(v1);
                        });
                    }
                    sum = sums[0] + sums[1];
                }
                tmem_wait_st();
                l = l * alpha + sum;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + x));
            }
            // ---- the segment's outputs ----
            if (solo && x == 1 && d[kSegSteps] == 1 && lane == 0) mbar_arrive(bar(kPFull + 1));
            const float vscale = kFp8 ? __ldg(p.v_scale + d[kSegHead] * p.scale_stride) : 1.0f;
            if (!ok) break;
            // The sum goes where the maximum of the last step stood: not before the row's other thread has
            // read that.  (Between two steps the scores are waited for, which come behind both threads' P.)
            if (warp_live) come();
            look_ahead();
            if (!ok) break;
            if (warp_live) {                           // the row's sum
                if (!met()) break;
                row_smem[exch] = l;
                if (!meet()) break;
                const float l2 = row_smem[exch ^ kRows];
                l = half ? l2 + l : l + l2;
                if (!meet()) break;                    // both have read: the places are free
            }
            if (!warp_wait_all(bar(kSegDone + x), (k - 1) & 1, p.timeout_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool whole = d[kSegFlags] & 2;
            const size_t slot = static_cast<size_t>(d[kSegSlot]);
            const size_t orow = (static_cast<size_t>(d[kSegRow0] + (solo ? 0 : x * QT) + r / G) * p.num_q_heads + d[kSegHead] * G + r % G) * kHeadDim;
            const int at_row = solo ? r : x * kRows + r;
            // 32 components from 32 c on: of the row itself, in whole sectors, or of its partial, in an
            // order in which a warp's rows lie side by side ([quad of components][row][4])
            auto put = [&](int c, const uint32_t (&ov)[32], float inv) {
                if (live && whole) {
                    uint16_t* dst = static_cast<uint16_t*>(p.out) + orow + 32 * c;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t w[8];
#pragma unroll
                        for (int a = 0; a < 8; ++a)
                            w[a] = pack2<QBf16>(__uint_as_float(ov[16 * e + 2 * a]) * inv, __uint_as_float(ov[16 * e + 2 * a + 1]) * inv);
                        if (p.out_sectors) {
                            st_global_32(dst + 16 * e, w);
                        } else {
                            reinterpret_cast<uint4*>(dst)[2 * e] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4*>(dst)[2 * e + 1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                } else if (live) {
                    float4* dst = p.partial + (slot * 32 + 8 * c) * (2 * kRows) + at_row;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e * 2 * kRows] = make_float4(__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                                                         __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3]));
                }
                __syncwarp();
            };
            float2* ml = p.ml + slot * (2 * kRows) + at_row;
            // No barrier gets two phases ahead of a warp: a segment's end waits for P, or as much, of
            // all of the tile's warps.
            if (!solo) {
                if (warp_live) {
                    const float inv = l == 0.f ? 0.f : vscale / l;
#pragma unroll 1
                    for (int c = 2 * half; c < 2 * half + 2; ++c) {
                        uint32_t ov[32];
                        tmem_ld32(tO(x) + lane_off + 32 * c, ov);
                        tmem_wait_ld();
                        put(c, ov, inv);
                    }
                    if (!whole && live && half == 0) *ml = make_float2(m_used, l);
                }
            } else {
                // A's steps and B's: both tiles hold the row in this lane; each of the row's four threads
                // writes a quarter of the components
                if (half == 0) {
                    row_smem[2 * x * kRows + r] = m_used;
                    row_smem[(2 * x + 1) * kRows + r] = l;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kMlReady));
                if (!warp_wait_all(bar(kMlReady), par >> 1 & 1, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                if (warp_live) {
                    const float ma = row_smem[r], la = row_smem[kRows + r];
                    const float mb = row_smem[2 * kRows + r], lb = row_smem[3 * kRows + r];
                    const float m = fmaxf(ma, mb), m_at = m == -INFINITY ? 0.f : m;
                    const float wa = ex2_approx(ma - m_at), wb = ex2_approx(mb - m_at);
                    const float sum = la * wa + lb * wb;
                    const float inv = sum == 0.f ? 0.f : vscale / sum;
                    const bool two = d[kSegSteps] > 1;  // else B has no products
                    const int c = 2 * x + half;
                    uint32_t ov[32];
                    tmem_ld32(tO(0) + lane_off + 32 * c, ov);
                    tmem_wait_ld();
                    if (two) {
                        uint32_t ob[32];
                        tmem_ld32(tO(1) + lane_off + 32 * c, ob);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ov[e] = __float_as_uint(fmaf(__uint_as_float(ov[e]), wa, __uint_as_float(ob[e]) * wb));
                    }
                    put(c, ov, inv);
                    if (!whole && live && c == 0) *ml = make_float2(m, sum);
                }
                // its products were read by both tiles' warps: the next may go over them when all are done
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kOFree));
                if (!warp_wait_all(bar(kOFree), par >> 1 & 1, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                par ^= 2u;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kSegEmpty + (k - 1) % kSegs));
        }
        if (!ok && lane == 0) atomicOr(p.status, kDevErrTimeout);
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Units that several CTAs share:
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   M = max_i m_i,
// over the partials (o_i, m_i in log2 units, l_i).  CTA (w, y) takes parts of the unit that main
// CTA w began and did not finish; its partials lie in w's second slot and in the first slots of
// the CTAs behind it up to `last`.  A part is up to 32 rows and 4 or 8 quads of their components;
// the threads that are left when the rows are few share out the partials, and their sums meet
// in shared memory.
template <bool OutBf16, bool Fp8>
__global__ void __launch_bounds__(256) scored_combine_kernel(const ScoredParams p) {
    __shared__ float4 acc_smem[256];
    __shared__ float2 ml_smem[256];
    grid_dependency_wait();
    grid_launch_dependents();
    const int w = blockIdx.x;
    const CombineRecord rec = p.records[w];
    if (rec.rows == 0) return;
    const int parts = rec.last - w + 1;
    const int QT = p.queries_per_tile, G = p.group;
    // threads: row (a power of two of them up to 32) x 4 quads x share of the partials
    int shift = 0;
    while (shift < 5 && (1 << shift) < rec.rows) ++shift;
    const int qs = parts <= 8 && shift == 5 ? 3 : 2;         // 8 quads where nothing is left to share out
    const int row = threadIdx.x & ((1 << shift) - 1), quad = threadIdx.x >> shift & ((1 << qs) - 1);
    const int share = threadIdx.x >> (shift + qs), shares = 256 >> (shift + qs);
    const int tasks = ((rec.rows + (1 << shift) - 1) >> shift) * (32 >> qs);
    for (int task = blockIdx.y; task < tasks; task += gridDim.y) {
        const int i = ((task >> (5 - qs)) << shift) + row;
        const int q4 = ((task & ((32 >> qs) - 1)) << qs) + quad;
        const bool live = i < rec.rows;
        const int query = i / G;
        const int at = rec.solo ? i : (query / QT) * kRows + (query % QT) * G + i % G;
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto fold = [&](float2 ml, float4 o) {
            const float mn = fmaxf(m, ml.x), m_at = mn == -INFINITY ? 0.f : mn;
            const float a = ex2_approx(m - m_at), b = ex2_approx(ml.x - m_at);
            acc = make_float4(acc.x * a + o.x * b, acc.y * a + o.y * b, acc.z * a + o.z * b, acc.w * a + o.w * b);
            l = l * a + ml.y * b;
            m = mn;
        };
        if (live) {
            for (int k0 = share; k0 < parts; k0 += 4 * shares) {
                float4 o[4];
                float2 ml[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int kk = k0 + e * shares;
                    ml[e] = make_float2(-INFINITY, 0.f);
                    o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (kk < parts) {
                        const size_t slot = kk == 0 ? 2 * w + 1 : 2 * (w + kk);
                        ml[e] = __ldcg(p.ml + slot * (2 * kRows) + at);
                        o[e] = __ldcg(p.partial + (slot * 32 + q4) * (2 * kRows) + at);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) fold(ml[e], o[e]);
            }
        }
        if (shares > 1 && parts > 1) {
            __syncthreads();
            acc_smem[threadIdx.x] = acc;
            ml_smem[threadIdx.x] = make_float2(m, l);
            __syncthreads();
            if (share == 0)
                for (int e = 1; e < min(shares, parts); ++e)
                    fold(ml_smem[threadIdx.x + (e << (shift + qs))], acc_smem[threadIdx.x + (e << (shift + qs))]);
        }
        if (live && share == 0) {
            const int head = rec.head0 + i % G;
            const float vscale = Fp8 ? __ldg(p.v_scale + rec.head0 / G * p.scale_stride) : 1.0f;
            const float inv = l == 0.f ? 0.f : vscale / l;
            uint16_t* dst = static_cast<uint16_t*>(p.out) +
                            (static_cast<size_t>(rec.row0 + query) * p.num_q_heads + head) * kHeadDim + 4 * q4;
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<OutBf16>(acc.x * inv, acc.y * inv), pack2<OutBf16>(acc.z * inv, acc.w * inv));
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

namespace {

template <int Kind, bool QBf16>
const void* scored_fn(ScoreForm form) {
    switch (form) {
        case kPlainScores: return reinterpret_cast<const void*>(&scored_kernel<Kind, QBf16, kPlainScores>);
        case kCappedScores: return reinterpret_cast<const void*>(&scored_kernel<Kind, QBf16, kCappedScores>);
        case kBiasedScores: return reinterpret_cast<const void*>(&scored_kernel<Kind, QBf16, kBiasedScores>);
        case kWideCappedScores: return reinterpret_cast<const void*>(&scored_kernel<Kind, QBf16, kWideCappedScores>);
        case kWideBiasedScores: return reinterpret_cast<const void*>(&scored_kernel<Kind, QBf16, kWideBiasedScores>);
    }
    return nullptr;
}

const void* scored_fn(CacheKind kind, bool q_bf16, ScoreForm form) {
    switch (kind) {
        case kKindBf16: return scored_fn<kKindBf16, true>(form);
        case kKindFp16: return scored_fn<kKindFp16, false>(form);
        case kKindFp8: return q_bf16 ? scored_fn<kKindFp8, true>(form) : scored_fn<kKindFp8, false>(form);
    }
    return nullptr;
}

size_t scored_smem(CacheKind kind) { return kind == kKindFp8 ? Cfg<kKindFp8>::kSmem : Cfg<kKindBf16>::kSmem; }

}  // namespace

ScoredLayout scored_layout(int sms) {
    ScoredLayout l;
    const size_t rows = static_cast<size_t>(sms) * 2 * 2 * kRows;        // two slots per CTA
    l.records_off = 256;
    l.ml_off = l.records_off + (static_cast<size_t>(sms) * sizeof(CombineRecord) + 255) / 256 * 256;
    l.partial_off = l.ml_off + rows * sizeof(float2);
    l.total = l.partial_off + rows * kHeadDim * sizeof(float);
    return l;
}

int scored_rows() { return kRows; }

cudaError_t scored_prepare(CacheKind kind, bool q_bf16, ScoreForm form) {
    return cudaFuncSetAttribute(scored_fn(kind, q_bf16, form), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(scored_smem(kind)));
}

cudaError_t launch_scored(CacheKind kind, bool q_bf16, ScoreForm form, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          const CUtensorMap& qmap, const ScoredParams& p, int sms, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = scored_smem(kind);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<CUtensorMap*>(&kmap), const_cast<CUtensorMap*>(&vmap), const_cast<CUtensorMap*>(&qmap),
                    const_cast<ScoredParams*>(&p)};
    return cudaLaunchKernelExC(&cfg, scored_fn(kind, q_bf16, form), args);
}

cudaError_t launch_scored_combine(bool out_bf16, bool fp8, const ScoredParams& p, int sms, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms), 16);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (out_bf16)
        return fp8 ? cudaLaunchKernelEx(&cfg, scored_combine_kernel<true, true>, p)
                   : cudaLaunchKernelEx(&cfg, scored_combine_kernel<true, false>, p);
    return fp8 ? cudaLaunchKernelEx(&cfg, scored_combine_kernel<false, true>, p)
               : cudaLaunchKernelEx(&cfg, scored_combine_kernel<false, false>, p);
}

}  // namespace pa
