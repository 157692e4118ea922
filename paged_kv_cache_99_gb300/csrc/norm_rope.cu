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
// whose components are paired with one another, and a thread's eight pairs are the same in
// every row, so that their cosines and sines are loaded once for all the rows (Rows) that
// the thread takes of its token.  Pairs of one axis come as two 16-byte loads each of
// cosines and sines; pairs of several as single loads from their axes' rows (those of a
// token are read by all its groups and stay in L1).
constexpr int kNormThreads = 128;

template <bool SrcBf16, bool Fp8, bool Interleaved, int Rows>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams np) {
    const RopeParams& p = np.rope;
    grid_dependency_wait();
    grid_launch_dependents();
    const unsigned grp = blockIdx.x * (kNormThreads / 8) + (threadIdx.x >> 3);
    const unsigned tok = grp / static_cast<unsigned>(p.groups);
    const int gi = static_cast<int>(grp % static_cast<unsigned>(p.groups));
    if (tok >= static_cast<unsigned>(p.num_tokens)) return;     // all eight threads of a row alike
    const unsigned row_lanes = 0xffu << (threadIdx.x & 24);
    const int c = threadIdx.x & 7;
    const int heads = p.num_q_heads + p.num_kv_heads;       // rows that are normed and rotated
    const int rows = heads + p.num_kv_heads;
    const int half = p.rot_dim >> 1;
    const bool turned = Interleaved ? 16 * c < p.rot_dim : 8 * c < half;
    int o0, o1;                                             // the thread's two pieces of a row
    if (Interleaved) {
        o0 = 16 * c;
        o1 = o0 + 8;
    } else if (turned) {
        o0 = 8 * c;
        o1 = half + 8 * c;
    } else {
        o0 = p.rot_dim + 16 * (c - (half >> 3));
        o1 = o0 + 8;
    }

    long long pos[kMaxAxes];
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a)
        pos[a] = a < np.num_axes ? p.positions[static_cast<size_t>(a) * p.num_tokens + tok] : 0;
    const long long slot = p.slots[tok];
    uint4 x0[Rows], x1[Rows];
#pragma unroll
    for (int j = 0; j < Rows; ++j) {
        const int row = gi + j * p.groups;
        if (row < rows) {
            const uint16_t* src = row < p.num_q_heads ? p.q + tok * p.q_stride + row * kHeadDim
                                : row < heads ? p.k + tok * p.k_stride + (row - p.num_q_heads) * kHeadDim
                                              : p.v + tok * p.v_stride + (row - heads) * kHeadDim;
            x0[j] = *reinterpret_cast<const uint4*>(src + o0);
            x1[j] = *reinterpret_cast<const uint4*>(src + o1);
        }
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
        if (gi == 0 && c == 0 && p.status) atomicOr(p.status, kDevErrRange);
        if (beyond) return;
    }
    float cs[8], sn[8];
    if (turned && gi < heads) {
        const unsigned w01 = c & 2 ? np.axis_word[1] : np.axis_word[0], w23 = c & 2 ? np.axis_word[3] : np.axis_word[2];
        const unsigned axes = (c & 4 ? w23 : w01) >> (16 * (c & 1));        // two bits for each of the eight pairs
        auto at = [&](unsigned axis) -> const float* {
            const long long y = axis & 2 ? (axis & 1 ? pos[3] : pos[2]) : (axis & 1 ? pos[1] : pos[0]);
            return p.cos_sin + static_cast<size_t>(y) * p.rot_dim + 8 * c;
        };
        if (np.one_axis >> c & 1) {
            const float4* t = reinterpret_cast<const float4*>(at(axes & 3));
            const float4* u = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(t) + half);
            const float4 a = __ldg(t), b = __ldg(t + 1), d = __ldg(u), e = __ldg(u + 1);
            cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w; cs[4] = b.x; cs[5] = b.y; cs[6] = b.z; cs[7] = b.w;
            sn[0] = d.x; sn[1] = d.y; sn[2] = d.z; sn[3] = d.w; sn[4] = e.x; sn[5] = e.y; sn[6] = e.z; sn[7] = e.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float* t = at(axes >> (2 * e) & 3);
                cs[e] = __ldg(t + e);
                sn[e] = __ldg(t + half + e);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < Rows; ++j) {
        const int row = gi + j * p.groups;
        if (row >= rows) break;
        const bool is_q = row < p.num_q_heads, is_v = row >= heads;
        if (!is_q && (slot < 0 || slot >= limit)) continue;
        const int h = row - (is_v ? heads : p.num_q_heads);
        const uint16_t* weight = is_v ? nullptr : is_q ? np.q_weight : np.k_weight;
        const bool changed = !is_v && (weight != nullptr || turned);
        float f[16];
        if (!is_v) {
            const uint32_t w[8] = {x0[j].x, x0[j].y, x0[j].z, x0[j].w, x1[j].x, x1[j].y, x1[j].z, x1[j].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[2 * e] = to_float<SrcBf16>(w[e] & 0xffffu);
                f[2 * e + 1] = to_float<SrcBf16>(w[e] >> 16);
            }
            if (weight) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) sum = fmaf(f[e], f[e], sum);
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(row_lanes, sum, o);
                const float r = rsqrtf(fmaf(sum, 1.0f / kHeadDim, np.eps));
                const uint4 g0 = __ldg(reinterpret_cast<const uint4*>(weight + o0));
                const uint4 g1 = __ldg(reinterpret_cast<const uint4*>(weight + o1));
                const uint32_t g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[2 * e] = f[2 * e] * r * (np.weight_offset + to_float<SrcBf16>(g[e] & 0xffffu));
                    f[2 * e + 1] = f[2 * e + 1] * r * (np.weight_offset + to_float<SrcBf16>(g[e] >> 16));
                }
            }
            if (turned) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int ia = Interleaved ? 2 * e : e, ib = Interleaved ? 2 * e + 1 : 8 + e;
                    const float a = f[ia], b = f[ib];
                    f[ia] = __fsub_rn(__fmul_rn(a, cs[e]), __fmul_rn(b, sn[e]));
                    f[ib] = __fadd_rn(__fmul_rn(b, cs[e]), __fmul_rn(a, sn[e]));
                }
            }
        }
        if (!Fp8 || is_q) {
            uint16_t* dst;
            if (is_q) {
                dst = p.q_out + tok * p.q_out_stride + row * kHeadDim;
            } else {
                uint16_t* cache = static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache);
                dst = cache + (((static_cast<size_t>(slot >> p.block_shift) * p.num_kv_heads + h) << p.block_shift) +
                               static_cast<size_t>(slot & ((1 << p.block_shift) - 1))) * kHeadDim;
            }
            uint4 y0 = x0[j], y1 = x1[j];
            if (changed) {
                y0 = make_uint4(pack2<SrcBf16>(f[0], f[1]), pack2<SrcBf16>(f[2], f[3]), pack2<SrcBf16>(f[4], f[5]),
                                pack2<SrcBf16>(f[6], f[7]));
                y1 = make_uint4(pack2<SrcBf16>(f[8], f[9]), pack2<SrcBf16>(f[10], f[11]),
                                pack2<SrcBf16>(f[12], f[13]), pack2<SrcBf16>(f[14], f[15]));
            }
            *reinterpret_cast<uint4*>(dst + o0) = y0;
            *reinterpret_cast<uint4*>(dst + o1) = y1;
        } else {
            const float scale = __ldg((is_v ? p.v_scale : p.k_scale) + h * p.scale_stride);
            uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
            uint8_t* dst = cache + (((static_cast<size_t>(slot >> p.block_shift) * p.num_kv_heads + h) << p.block_shift) +
                                    static_cast<size_t>(slot & ((1 << p.block_shift) - 1))) * kHeadDim;
            uint2 y0, y1;
            if (changed) {
                y0 = make_uint2(e4m3_of(f[0], f[1], scale) | (e4m3_of(f[2], f[3], scale) << 16),
                                e4m3_of(f[4], f[5], scale) | (e4m3_of(f[6], f[7], scale) << 16));
                y1 = make_uint2(e4m3_of(f[8], f[9], scale) | (e4m3_of(f[10], f[11], scale) << 16),
                                e4m3_of(f[12], f[13], scale) | (e4m3_of(f[14], f[15], scale) << 16));
            } else {
                const uint4 a = x0[j], b = x1[j];
                y0 = make_uint2(e4m3_pair<SrcBf16>(a.x, scale) | (e4m3_pair<SrcBf16>(a.y, scale) << 16),
                                e4m3_pair<SrcBf16>(a.z, scale) | (e4m3_pair<SrcBf16>(a.w, scale) << 16));
                y1 = make_uint2(e4m3_pair<SrcBf16>(b.x, scale) | (e4m3_pair<SrcBf16>(b.y, scale) << 16),
                                e4m3_pair<SrcBf16>(b.z, scale) | (e4m3_pair<SrcBf16>(b.w, scale) << 16));
            }
            *reinterpret_cast<uint2*>(dst + o0) = y0;
            *reinterpret_cast<uint2*>(dst + o1) = y1;
        }
    }
}

template <bool SrcBf16, bool Fp8, int Rows>
const void* norm_rope_fn(bool interleaved) {
    return interleaved ? reinterpret_cast<const void*>(&norm_rope_kernel<SrcBf16, Fp8, true, Rows>)
                       : reinterpret_cast<const void*>(&norm_rope_kernel<SrcBf16, Fp8, false, Rows>);
}

template <int Rows>
const void* norm_rope_fn(bool src_bf16, bool fp8, bool interleaved) {
    if (src_bf16) return fp8 ? norm_rope_fn<true, true, Rows>(interleaved) : norm_rope_fn<true, false, Rows>(interleaved);
    return fp8 ? norm_rope_fn<false, true, Rows>(interleaved) : norm_rope_fn<false, false, Rows>(interleaved);
}

}  // namespace

cudaError_t launch_norm_rope_cache(NormRopeParams p, bool src_bf16, bool fp8, bool interleaved, int sms,
                                   cudaStream_t stream) {
    const int rows = p.rope.num_q_heads + 2 * p.rope.num_kv_heads;
    // one row per thread group up to a few waves of CTAs, where a call is as long as its
    // chains of loads; four rows beyond, for the loads in flight (as in rope.cu)
    const int per = static_cast<long long>(p.rope.num_tokens) * rows <= 2048ll * sms ? 1 : 4;
    p.rope.groups = (rows + per - 1) / per;
    constexpr int kPerCta = kNormThreads / 8;
    const long long ctas = (static_cast<long long>(p.rope.num_tokens) * p.rope.groups + kPerCta - 1) / kPerCta;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kNormThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&p};
    const void* fn = per == 1 ? norm_rope_fn<1>(src_bf16, fp8, interleaved) : norm_rope_fn<4>(src_bf16, fp8, interleaved);
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace pa
