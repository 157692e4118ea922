// The rotation and slot write of rope.cu for heads that are normed first and tokens whose
// positions have several axes (sm_103a).
//
// A query or key head x of 128 components becomes y = x / sqrt(mean(x^2) + eps) * (offset +
// weight), its pairs are turned as in rope.cu, pair i by row positions[axis of i] of the
// table, and keys and values go to their slots.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

// HBM-bound: q is read and written once, k and v are read once and written once.  The norm
// adds a sum over the head, which the eight threads that hold its row fold with three
// shuffles; nothing is read twice.
// As in rope.cu eight threads own a row (one head of one token), each two 16-byte pieces
// whose components are paired with one another, and a thread's eight pairs, with their
// cosines and sines, are the same in every row.  Two kernels: with few tokens one in which
// every row is a thread group's own, as short as its chain of loads (position, table row);
// with many one in which a warp copies whole tokens and their tables' rows into shared
// memory ahead of the others (below).

// What a thread does to its two pieces of a row.
struct RowPieces {
    int c;                      // the thread's place among the row's eight
    int o0, o1;                 // its pieces' first components
    bool turned;                // they are rotated

    template <bool Interleaved>
    __device__ __forceinline__ static RowPieces of(int c, int rot_dim) {
        RowPieces r;
        const int half = rot_dim >> 1;
        r.c = c;
        r.turned = Interleaved ? 16 * c < rot_dim : 8 * c < half;
        if (Interleaved) {
            r.o0 = 16 * c;
            r.o1 = r.o0 + 8;
        } else if (r.turned) {
            r.o0 = 8 * c;
            r.o1 = half + 8 * c;
        } else {
            r.o0 = rot_dim + 16 * (c - (half >> 3));
            r.o1 = r.o0 + 8;
        }
        return r;
    }
};

template <bool SrcBf16>
__device__ __forceinline__ void unpack_pieces(const uint4& a, const uint4& b, float (&f)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f[2 * e] = to_float<SrcBf16>(w[e] & 0xffffu);
        f[2 * e + 1] = to_float<SrcBf16>(w[e] >> 16);
    }
}

// The eight pairs' cosines and sines: `row(axis)` is the token's row of the table for an axis.
// Pairs of one axis come as 16-byte loads, pairs of several as single ones.
template <typename RowOf>
__device__ __forceinline__ void load_turns(const NormRopeParams& np, int c, int half, RowOf row, float (&cs)[8], float (&sn)[8]) {
    const unsigned w01 = c & 2 ? np.axis_word[1] : np.axis_word[0], w23 = c & 2 ? np.axis_word[3] : np.axis_word[2];
    const unsigned axes = (c & 4 ? w23 : w01) >> (16 * (c & 1));        // two bits for each of the eight pairs
    if (np.one_axis >> c & 1) {
        const float4* t = reinterpret_cast<const float4*>(row(axes & 3) + 8 * c);
        const float4* u = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(t) + half);
        const float4 a = t[0], b = t[1], d = u[0], e = u[1];
        cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w; cs[4] = b.x; cs[5] = b.y; cs[6] = b.z; cs[7] = b.w;
        sn[0] = d.x; sn[1] = d.y; sn[2] = d.z; sn[3] = d.w; sn[4] = e.x; sn[5] = e.y; sn[6] = e.z; sn[7] = e.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float* t = row(axes >> (2 * e) & 3) + 8 * c;
            cs[e] = t[e];
            sn[e] = t[half + e];
        }
    }
}

// The sum of a row's squares over its eight threads, as the factor of the norm.
__device__ __forceinline__ float norm_factor(const NormRopeParams& np, const float (&f)[16], unsigned row_lanes) {
    uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        const uint64_t v = f2_pack(f[e], f[e + 1]);
        sum2[(e >> 1) & 1] = f2_fma(v, v, sum2[(e >> 1) & 1]);
    }
    float s0, s1;
    f2_unpack(f2_add(sum2[0], sum2[1]), s0, s1);
    float sum = s0 + s1;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(row_lanes, sum, o);
    return rsqrtf(fmaf(sum, 1.0f / kHeadDim, np.eps));
}

// Rotation of a thread's pieces: products by the sines rounded, the others fused.
template <bool Interleaved>
__device__ __forceinline__ void turn_pieces(const float (&cs)[8], const float (&sn)[8], float (&f)[16]) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const int a0 = Interleaved ? 2 * e : e, a1 = Interleaved ? 2 * e + 2 : e + 1;
        const int b0 = Interleaved ? 2 * e + 1 : 8 + e, b1 = Interleaved ? 2 * e + 3 : 9 + e;
        const uint64_t a = f2_pack(f[a0], f[a1]), b = f2_pack(f[b0], f[b1]);
        const uint64_t c = f2_pack(cs[e], cs[e + 1]), s = f2_pack(sn[e], sn[e + 1]), m = f2_pack(-sn[e], -sn[e + 1]);
        f2_unpack(f2_fma(a, c, f2_mul(b, m)), f[a0], f[a1]);
        f2_unpack(f2_fma(b, c, f2_mul(a, s)), f[b0], f[b1]);
    }
}

// Two e4m3 codes by the slot-write rule, x / scale rounded once to 32 bits (IEEE) and then to
// e4m3.  With y the reciprocal of the scale, itself rounded to nearest, and q = x y, the
// remainder x - q scale is exact in a fused operation and q + remainder y is the quotient
// correctly rounded (Markstein's division): four operations and a bound on q against overflow
// (what lies beyond becomes 448 all the same), where a division takes a dozen and a branch.
// Scales whose reciprocal or products could leave the normal range take the division.
__device__ __forceinline__ uint32_t e4m3_codes(float a, float b, float scale, float y, bool plain) {
    auto quotient = [&](float x) {
        if (!plain) return __fdiv_rn(x, scale);
        const float q = fminf(fmaxf(x * y, -1e6f), 1e6f);
        return copysignf(fmaf(fmaf(-q, scale, x), y, q), q);       // -0 + 0 would lose a zero's sign
    };
    uint16_t code;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(code) : "f"(quotient(b)), "f"(quotient(a)));
    return code;
}

// Stores a thread's pieces of a row of 16-bit elements: as they came, or changed.
template <bool SrcBf16>
__device__ __forceinline__ void store_halves(uint16_t* dst, const RowPieces& rp, bool changed, const uint4& x0, const uint4& x1,
                                             const float (&f)[16]) {
    uint4 y0 = x0, y1 = x1;
    if (changed) {
        y0 = make_uint4(pack2<SrcBf16>(f[0], f[1]), pack2<SrcBf16>(f[2], f[3]), pack2<SrcBf16>(f[4], f[5]), pack2<SrcBf16>(f[6], f[7]));
        y1 = make_uint4(pack2<SrcBf16>(f[8], f[9]), pack2<SrcBf16>(f[10], f[11]), pack2<SrcBf16>(f[12], f[13]), pack2<SrcBf16>(f[14], f[15]));
    }
    *reinterpret_cast<uint4*>(dst + rp.o0) = y0;
    *reinterpret_cast<uint4*>(dst + rp.o1) = y1;
}

// The same as e4m3 codes.  A stored value's NaN keeps the sign of its source, one of the norm's
// or the rotation's is positive: the conversion makes every NaN 0x7f, a code that nothing else
// gets, so they are looked for by fours.
__device__ __forceinline__ void store_codes(uint8_t* dst, const RowPieces& rp, bool changed, const uint4& x0, const uint4& x1,
                                            const float (&f)[16], float scale) {
    const float y = __frcp_rn(scale);
    const bool plain = fabsf(scale) > 0x1p-60f && fabsf(scale) < 0x1p60f;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        w[e] = e4m3_codes(f[4 * e], f[4 * e + 1], scale, y, plain) | e4m3_codes(f[4 * e + 2], f[4 * e + 3], scale, y, plain) << 16;
        if (((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) {
            const uint32_t src[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            const uint32_t signs = changed ? 0u
                                           : (src[2 * e] >> 8 & 0x80u) | (src[2 * e] >> 16 & 0x8000u) |
                                                 (src[2 * e + 1] << 8 & 0x800000u) | (src[2 * e + 1] & 0x80000000u);
#pragma unroll
            for (int b = 0; b < 32; b += 8)
                if ((w[e] >> b & 0x7fu) == 0x7fu) w[e] = (w[e] & ~(0x80u << b)) | (signs & (0x80u << b));
        }
    }
    *reinterpret_cast<uint2*>(dst + rp.o0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(dst + rp.o1) = make_uint2(w[2], w[3]);
}

// A head's row at a slot of a cache, in elements.
__device__ __forceinline__ size_t slot_row(const RopeParams& p, long long slot, int h) {
    return (((static_cast<size_t>(slot >> p.block_shift) * p.num_kv_heads + h) << p.block_shift) +
            static_cast<size_t>(slot & ((1 << p.block_shift) - 1))) * kHeadDim;
}

// ---- few tokens: a thread group per row ----
constexpr int kNormThreads = 128;

template <bool SrcBf16, bool Fp8, bool Interleaved>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams np) {
    const RopeParams& p = np.rope;
    grid_dependency_wait();
    grid_launch_dependents();
    const int heads = p.num_q_heads + p.num_kv_heads;       // rows that are normed and rotated
    const unsigned grp = blockIdx.x * (kNormThreads / 8) + (threadIdx.x >> 3);
    const unsigned tok = grp / static_cast<unsigned>(heads + p.num_kv_heads);
    const int row = static_cast<int>(grp % static_cast<unsigned>(heads + p.num_kv_heads));
    if (tok >= static_cast<unsigned>(p.num_tokens)) return;     // all eight threads of a row alike
    const RowPieces rp = RowPieces::of<Interleaved>(threadIdx.x & 7, p.rot_dim);
    const bool is_q = row < p.num_q_heads, is_v = row >= heads;
    const int h = row - (is_q ? 0 : is_v ? heads : p.num_q_heads);

    long long pos[kMaxAxes];
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a)
        pos[a] = a < np.num_axes ? p.positions[static_cast<size_t>(a) * p.num_tokens + tok] : 0;
    const long long slot = p.slots[tok];
    const uint16_t* src = (is_q ? p.q + tok * p.q_stride : is_v ? p.v + tok * p.v_stride : p.k + tok * p.k_stride) + h * kHeadDim;
    const uint4 x0 = *reinterpret_cast<const uint4*>(src + rp.o0), x1 = *reinterpret_cast<const uint4*>(src + rp.o1);
    const uint16_t* weight = is_v ? nullptr : is_q ? np.q_weight : np.k_weight;
    uint4 g0 = make_uint4(0, 0, 0, 0), g1 = g0;
    if (weight) {
        g0 = __ldg(reinterpret_cast<const uint4*>(weight + rp.o0));
        g1 = __ldg(reinterpret_cast<const uint4*>(weight + rp.o1));
    }
    bool padding = false, beyond = false;
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) {
        padding |= pos[a] < 0;
        beyond |= pos[a] >= p.max_positions;
    }
    if (padding) return;                                    // nothing of the token is written
    const long long limit = static_cast<long long>(p.num_blocks) << p.block_shift;
    if (beyond || slot >= limit) {
        if (row == 0 && rp.c == 0 && p.status) atomicOr(p.status, kDevErrRange);
        if (beyond) return;
    }
    if (!is_q && (slot < 0 || slot >= limit)) return;
    const bool turns = rp.turned && !is_v;
    float cs[8], sn[8];
    if (turns) {
        load_turns(np, rp.c, p.rot_dim >> 1, [&](unsigned axis) {
            const long long y = axis & 2 ? (axis & 1 ? pos[3] : pos[2]) : (axis & 1 ? pos[1] : pos[0]);
            return p.cos_sin + static_cast<size_t>(y) * p.rot_dim;
        }, cs, sn);
    }
    float f[16];
    unpack_pieces<SrcBf16>(x0, x1, f);
    if (weight) {
        const float r = norm_factor(np, f, 0xffu << (threadIdx.x & 24));
        float g[16];
        unpack_pieces<SrcBf16>(g0, g1, g);
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] *= r * (np.weight_offset + g[e]);
    }
    if (turns) turn_pieces<Interleaved>(cs, sn, f);
    const bool changed = weight != nullptr || turns;
    if (is_q) {
        store_halves<SrcBf16>(p.q_out + tok * p.q_out_stride + h * kHeadDim, rp, changed, x0, x1, f);
    } else if constexpr (!Fp8) {
        store_halves<SrcBf16>(static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) + slot_row(p, slot, h), rp, changed, x0, x1, f);
    } else {
        store_codes(static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + slot_row(p, slot, h), rp, changed, x0, x1, f,
                    __ldg((is_v ? p.v_scale : p.k_scale) + h * p.scale_stride));
    }
}

// ---- many tokens: copies run ahead ----
// A CTA takes every gridDim-th token.  Its last warp copies a token's q, k and v and its rows
// of the table (bulk copies) into a ring of stages, several tokens ahead, with the tokens'
// positions and slots fetched 32 at a time before; the other warps norm and turn one stage
// after the other in place, eight threads to a row, and the copying warp brings the worked rows
// back (bulk copies again; FP8 codes are written by their threads).  So nothing waits for a
// chain of loads, and the table's rows are read once for a token whatever axes its pairs
// follow: 16384 tokens of 32/8 heads in bf16 (0.41 GB) take 66 us with three axes, 6.2 TB/s,
// as one row per group 110, with rows stored by their threads 78.
//
// Four CTAs of four working warps to an SM, or three of six: the fewer tokens are in flight, the
// less HBM turns between reading and writing, so the three for 16-bit caches whose data do not fit L2
// (16384 tokens 66 against 74 us, 8192 34.1 against 38.0, but 4096 18.1 against 16.7); FP8
// codes are bound by the work, which four CTAs spread better (1040 tokens of 64/8 heads 10.3
// against 12.4; a row per group 13.9).
constexpr int stream_ctas(int warps) { return warps == 4 ? 4 : 3; }
constexpr int kMaxStages = 8;
constexpr unsigned long long kStreamTimeoutNs = 1000ull * 1000ull * 1000ull;    // bound of every wait

struct StreamShape {
    int rows;                   // of a token: q, k, v heads
    int stage_bytes, table_off; // a stage: rows x 256 bytes, then the table's rows
    int stages;
};

template <bool SrcBf16, bool Fp8, bool Interleaved, int Warps>
__global__ void __launch_bounds__(32 * (Warps + 1), stream_ctas(Warps))
    norm_rope_stream_kernel(const __grid_constant__ NormRopeParams np, const StreamShape sh) {
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages];
    __shared__ long long slots[kMaxStages];                 // of a stage's token; -2: nothing of it is written
    // of q and k, the offset added: [four of a thread's components][thread of a row][4], so that a
    // row's threads read side by side
    __shared__ __align__(16) float weights[2 * kHeadDim];
    const RopeParams& p = np.rope;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kMaxStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < sh.stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, Warps);
        }
        fence_barrier_init();
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    const int first = blockIdx.x, step = gridDim.x;
    const int mine = first < p.num_tokens ? (p.num_tokens - 1 - first) / step + 1 : 0;      // this CTA's tokens
    const long long limit = static_cast<long long>(p.num_blocks) << p.block_shift;
    int st = 0;
    uint32_t ph = 0;
    auto advance = [&]() {
        if (++st == sh.stages) {
            st = 0;
            ph ^= 1u;
        }
    };
    if (warp == Warps) {
        const int row_bytes = p.rot_dim * 4;
        long long pos[kMaxAxes], slot = 0;
        int done = 0;
        // the worked rows of the CTA's i-th token, in stage st, to where they belong
        auto flush = [&](int i) {
            const long long s = slots[st];
            const uint32_t src = smem_addr(sm) + st * sh.stage_bytes;
            if (s >= -1 && lane == 0)
                bulk_store(p.q_out + (first + static_cast<long long>(i) * step) * p.q_out_stride, src, p.num_q_heads * 256);
            if (!Fp8 && s >= 0) {
                for (int r = lane; r < 2 * p.num_kv_heads; r += 32) {
                    const bool is_v = r >= p.num_kv_heads;
                    uint16_t* cache = static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache);
                    bulk_store(cache + slot_row(p, s, is_v ? r - p.num_kv_heads : r), src + (p.num_q_heads + r) * 256, 256);
                }
            }
            bulk_store_wait_read();
            __syncwarp();
        };
        for (; done < mine; ++done) {
            if ((done & 31) == 0) {
                // the next 32 tokens' places, a lane each
                const int t = first + min(done + lane, mine - 1) * step;
#pragma unroll
                for (int a = 0; a < kMaxAxes; ++a)
                    pos[a] = a < np.num_axes ? p.positions[static_cast<size_t>(a) * p.num_tokens + t] : 0;
                slot = p.slots[t];
            }
            if (done >= sh.stages) {
                if (!warp_wait_all(empty + 8 * st, ph ^ 1u, kStreamTimeoutNs)) break;
                flush(done - sh.stages);
            }
            const int src = done & 31;
            const int t = first + done * step;
            const long long s = __shfl_sync(0xffffffffu, slot, src);
            bool padding = false, beyond = false;
            long long at[kMaxAxes];
#pragma unroll
            for (int a = 0; a < kMaxAxes; ++a) {
                at[a] = __shfl_sync(0xffffffffu, pos[a], src);
                padding |= at[a] < 0;
                beyond |= at[a] >= p.max_positions;
            }
            if (lane == 0) {
                if (!padding && (beyond || s >= limit) && p.status) atomicOr(p.status, kDevErrRange);
                const bool skip = padding || beyond;
                slots[st] = skip ? -2 : s < 0 || s >= limit ? -1 : s;
                if (skip) {
                    mbar_arrive(full + 8 * st);
                } else {
                    const uint32_t dst = smem_addr(sm) + st * sh.stage_bytes;
                    mbar_arrive_expect_tx(full + 8 * st, sh.rows * 256 + np.num_axes * row_bytes);
                    bulk_load(dst, p.q + t * p.q_stride, p.num_q_heads * 256, full + 8 * st);
                    bulk_load(dst + p.num_q_heads * 256, p.k + t * p.k_stride, p.num_kv_heads * 256, full + 8 * st);
                    bulk_load(dst + (p.num_q_heads + p.num_kv_heads) * 256, p.v + t * p.v_stride, p.num_kv_heads * 256, full + 8 * st);
#pragma unroll
                    for (int a = 0; a < kMaxAxes; ++a)
                        if (a < np.num_axes)
                            bulk_load(dst + sh.table_off + a * row_bytes, p.cos_sin + at[a] * p.rot_dim, row_bytes, full + 8 * st);
                }
            }
            __syncwarp();
            advance();
        }
        bool ok = done == mine;
        for (int i = max(0, mine - sh.stages); i < mine && ok; ++i) {
            if (mine < sh.stages) {
                st = i;
                ph = 1u;
            }
            ok = warp_wait_all(empty + 8 * st, ph ^ 1u, kStreamTimeoutNs);
            if (ok) flush(i);
            advance();
        }
        if (!ok) {
            // a wait gave up: let the copies in flight land before the CTA leaves
            if (lane == 0 && p.status) atomicOr(p.status, kDevErrTimeout);
            for (int i = max(0, done - sh.stages); i < done; ++i)
                warp_wait_all(full + 8 * (i % sh.stages), (i / sh.stages) & 1, kStreamTimeoutNs);
        }
        return;
    }
    const RowPieces rp = RowPieces::of<Interleaved>(threadIdx.x & 7, p.rot_dim);
    const unsigned row_lanes = 0xffu << (threadIdx.x & 24);
    const int heads = p.num_q_heads + p.num_kv_heads;
    for (int i = threadIdx.x; i < 2 * kHeadDim; i += 32 * Warps) {
        const uint16_t* w = i < kHeadDim ? np.q_weight : np.k_weight;
        const RowPieces of = RowPieces::of<Interleaved>(i >> 2 & 7, p.rot_dim);
        const int e = (i >> 5 & 3) * 4 + (i & 3);
        weights[i] = w ? np.weight_offset + to_float<SrcBf16>(w[e < 8 ? of.o0 + e : of.o1 + e - 8]) : 1.0f;
    }
    named_barrier_sync(1, 32 * Warps);
    for (int i = 0; i < mine; ++i) {
        if (!warp_wait_all(full + 8 * st, ph, kStreamTimeoutNs)) {
            if (lane == 0 && p.status) atomicOr(p.status, kDevErrTimeout);
            break;
        }
        const long long slot = slots[st];
        if (slot >= -1) {
            uint8_t* stage = sm + st * sh.stage_bytes;
            float cs[8], sn[8];
            if (rp.turned) {
                const float* table = reinterpret_cast<const float*>(stage + sh.table_off);
                load_turns(np, rp.c, p.rot_dim >> 1, [&](unsigned axis) { return table + axis * p.rot_dim; }, cs, sn);
            }
            // (16-bit values stay as they came)
            for (int row = threadIdx.x >> 3; row < (Fp8 ? sh.rows : heads); row += 4 * Warps) {
                const bool is_q = row < p.num_q_heads, is_v = row >= heads;
                if (!is_q && slot < 0) break;
                const int h = row - (is_q ? 0 : is_v ? heads : p.num_q_heads);
                uint16_t* src = reinterpret_cast<uint16_t*>(stage) + row * kHeadDim;
                const uint4 x0 = *reinterpret_cast<const uint4*>(src + rp.o0), x1 = *reinterpret_cast<const uint4*>(src + rp.o1);
                const bool norm = !is_v && (is_q ? np.q_weight : np.k_weight) != nullptr, turns = rp.turned && !is_v;
                float f[16];
                unpack_pieces<SrcBf16>(x0, x1, f);
                const float r = norm_factor(np, f, row_lanes);      // of every row: a branch here costs 8%
                if (norm) {
                    const float* g = weights + (is_q ? 0 : kHeadDim) + 4 * rp.c;
                    const uint64_t r2 = f2_pack(r, r);
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(g + 8 * e);
                        f2_unpack(f2_mul(f2_mul(f2_pack(f[e], f[e + 1]), r2), f2_pack(w.x, w.y)), f[e], f[e + 1]);
                        f2_unpack(f2_mul(f2_mul(f2_pack(f[e + 2], f[e + 3]), r2), f2_pack(w.z, w.w)), f[e + 2], f[e + 3]);
                    }
                }
                if (turns) turn_pieces<Interleaved>(cs, sn, f);
                if (!Fp8 || is_q) {
                    if (norm || turns) store_halves<SrcBf16>(src, rp, true, x0, x1, f);
                } else if constexpr (Fp8) {
                    store_codes(static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + slot_row(p, slot, h), rp, norm || turns,
                                x0, x1, f, __ldg((is_v ? p.v_scale : p.k_scale) + h * p.scale_stride));
                }
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * st);
        advance();
    }
}

// warps: of the kernel for many tokens, 0 for the one for few
template <bool SrcBf16, bool Fp8, bool Interleaved>
const void* norm_rope_fn(int warps) {
    if (warps == 0) return reinterpret_cast<const void*>(&norm_rope_kernel<SrcBf16, Fp8, Interleaved>);
    if constexpr (!Fp8) {
        if (warps == 6) return reinterpret_cast<const void*>(&norm_rope_stream_kernel<SrcBf16, Fp8, Interleaved, 6>);
    }
    return reinterpret_cast<const void*>(&norm_rope_stream_kernel<SrcBf16, Fp8, Interleaved, 4>);
}

template <bool SrcBf16, bool Fp8>
const void* norm_rope_fn(bool interleaved, int warps) {
    return interleaved ? norm_rope_fn<SrcBf16, Fp8, true>(warps) : norm_rope_fn<SrcBf16, Fp8, false>(warps);
}

const void* norm_rope_fn(bool src_bf16, bool fp8, bool interleaved, int warps) {
    if (src_bf16) return fp8 ? norm_rope_fn<true, true>(interleaved, warps) : norm_rope_fn<true, false>(interleaved, warps);
    return fp8 ? norm_rope_fn<false, true>(interleaved, warps) : norm_rope_fn<false, false>(interleaved, warps);
}

constexpr int kStreamSmem = 54 * 1024;                      // of a CTA's stages: four CTAs to an SM (three: the same)

}  // namespace

cudaError_t norm_rope_prepare() {
    for (int i = 0; i < 16; ++i) {
        const cudaError_t e = cudaFuncSetAttribute(norm_rope_fn(i & 1, i & 2, i & 4, i & 8 ? 6 : 4),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_norm_rope_cache(const NormRopeParams& p, bool src_bf16, bool fp8, bool interleaved, int sms,
                                   cudaStream_t stream) {
    StreamShape sh;
    sh.rows = p.rope.num_q_heads + 2 * p.rope.num_kv_heads;
    sh.table_off = sh.rows * 2 * kHeadDim;
    sh.stage_bytes = (sh.table_off + p.num_axes * p.rope.rot_dim * 4 + 127) / 128 * 128;
    sh.stages = kStreamSmem / sh.stage_bytes < kMaxStages ? kStreamSmem / sh.stage_bytes : kMaxStages;
    const long long total = static_cast<long long>(p.rope.num_tokens) * sh.rows;
    // the streaming kernel where there are a few tokens for each of its CTAs and stages to run ahead
    // (1024 tokens of 32/8 heads 7.7 us against 7.2, 2048 10.3 against 11.8)
    const bool many = sh.stages >= 2 && total > 512ll * sms;
    // rows that take 512 bytes of L2 each, in and out (130 MB in all)
    const int warps = !many ? 0 : !fp8 && total > (160ll << 20) / 512 ? 6 : 4;
    cudaLaunchConfig_t cfg = {};
    if (many) {
        const int ctas = stream_ctas(warps) * sms;
        cfg.gridDim = dim3(static_cast<unsigned>(p.rope.num_tokens < ctas ? p.rope.num_tokens : ctas));
        cfg.blockDim = dim3(32 * (warps + 1));
        cfg.dynamicSmemBytes = static_cast<size_t>(sh.stages) * sh.stage_bytes;
    } else {
        constexpr int kPerCta = kNormThreads / 8;
        cfg.gridDim = dim3(static_cast<unsigned>((total + kPerCta - 1) / kPerCta));
        cfg.blockDim = dim3(kNormThreads);
    }
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<NormRopeParams*>(&p), &sh};
    return cudaLaunchKernelExC(&cfg, norm_rope_fn(src_bf16, fp8, interleaved, warps), args);
}

}  // namespace pa
