// Rotary positions for sm_103a: the table of cosines and sines, and the rotation of
// a step's new queries and keys fused with the slot write.
//
// A rotary embedding turns pairs of a head's first rot_dim components by an angle
// that grows with the token's position p:
//   u = a cos(p f_i) - b sin(p f_i),   v = b cos(p f_i) + a sin(p f_i),
// where (a, b) are components (i, i + rot_dim / 2) in the half layout and
// (2i, 2i + 1) in the interleaved one; the other components stay as they are.
#include <cuda_runtime.h>

#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

// ---- the table -----------------------------------------------------------------
// cos_sin[p][i] = a cos(p f_i), cos_sin[p][rot / 2 + i] = a sin(p f_i).
//
// At position 10^5 an angle in 32 bits is off by up to 4e-3 rad, and FP64 runs at
// two operations per SM and clock here, far under the rate the stores go out at.
// So angles are kept as turns in 64-bit fixed point, f_i / 2 pi x 2^64 modulo 2^64:
// the whole turns fall off the top by themselves, the product with a position is an
// integer product, and the next position of a thread is one 64-bit addition.  The
// nearest quarter turn (two bits) picks sine or cosine and sign; the rest, in
// [-1/2, 1/2) quarter turns, goes to polynomials in 32-bit floats as the sum of two, so
// that a sine near zero (a slow component at the first positions) is as exact relative
// to itself as any other.
struct RopeTurns {
    unsigned long long turn[kHeadDim / 2];     // f_i / 2 pi in units of 2^-64 turns
};

// sine and cosine of y = a + b quarter turns, |a| <= 1/2 a multiple of 2^-23 and |b| at
// most half of one: Taylor polynomials in y with (pi / 2)^n / n! folded into the
// coefficients, to y^9 and y^10 (the first terms left out are under 2.5e-9 and 1.7e-10 of
// the result).  pi / 2 times a, most of the sine, is added last and so rounded once, with
// pi / 2 itself in two floats: both results are within 2.2 x 2^-24 of themselves (in one
// float, with 32 bits of y, the rest cut off: 28 units in the last place at the slowest
// component of base 10^4, thousands for slower ones).
__device__ __forceinline__ void sincos_quarter(float a, float b, float& sn, float& cs) {
    const float y = a + b;
    const float z = y * y;
    float p = 1.6044118e-4f;                    // (pi/2)^9 / 9!
    p = fmaf(p, z, -4.6817541e-3f);             // (pi/2)^7 / 7!
    p = fmaf(p, z, 7.9692626e-2f);              // (pi/2)^5 / 5!
    p = fmaf(p, z, -6.4596410e-1f);             // (pi/2)^3 / 3!
    const float rest = fmaf(p, y * z, fmaf(b, 1.5707964f, a * -4.3711388e-8f));
    sn = fmaf(a, 1.5707964f, rest);             // 1.5707964f - 4.3711388e-8 = pi/2
    float q = -2.5202042e-5f;                   // (pi/2)^10 / 10!
    q = fmaf(q, z, 9.1926027e-4f);              // (pi/2)^8 / 8!
    q = fmaf(q, z, -2.0863481e-2f);             // (pi/2)^6 / 6!
    q = fmaf(q, z, 2.5366951e-1f);              // (pi/2)^4 / 4!
    q = fmaf(q, z, -1.2337006e+0f);             // (pi/2)^2 / 2!
    cs = fmaf(q, z, 1.0f);
}

// A thread owns four frequencies and every `step`-th position, so that it writes 16
// bytes of cosines and 16 of sines at a time and a row goes out in whole lines.  Bound by
// the stores and, as closely, by instruction issue: 524288 positions of 128 (268 MB) take
// 41.0 us, 6.5 TB/s; 32768 (16.8 MB, it stays in L2) 4.5.  (With the rest of a quarter turn
// in one float, cut to 32 bits, 37.2 and 4.2.)  Two CTAs per SM: four take 40.6 and 5.5.
__global__ void __launch_bounds__(256) rope_table_kernel(float* __restrict__ cos_sin, int max_positions, int rot_dim,
                                                         const __grid_constant__ RopeTurns turns, float attention) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int quads = rot_dim / 8;                  // threads across a row
    const int rows = 256 / quads;                   // positions a CTA covers at a time
    const int i = threadIdx.x % quads, r = threadIdx.x / quads;
    if (r >= rows) return;
    const int step = gridDim.x * rows;
    int p = blockIdx.x * rows + r;
    unsigned long long phase[4], inc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const unsigned long long t = turns.turn[4 * i + e];
        phase[e] = t * static_cast<unsigned long long>(p);
        inc[e] = t * static_cast<unsigned long long>(step);
    }
    for (; p < max_positions; p += step) {
        float c[4], s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned hi = static_cast<unsigned>(phase[e] >> 32), lo = static_cast<unsigned>(phase[e]);
            // half a quarter turn up, and half of 2^-23 more: the top two bits are the quarter,
            // the next 23 the nearest multiple of 2^-23 quarter turns to the rest (a float
            // exactly), and of what is left 32 bits are kept
            const unsigned quarter = hi + (1u << 29) + 64u;
            const int left = static_cast<int>(__funnelshift_r(lo, hi, 7));
            float sn, cs;
            sincos_quarter(fmaf(static_cast<float>(quarter & 0x3fffff80u), 0x1p-30f, -0.5f),
                           static_cast<float>(left) * 0x1p-55f, sn, cs);
            const bool swap = quarter & (1u << 30);
            const float x = swap ? sn : cs, y = swap ? cs : sn;
            // cosine is negative in quarters 1 and 2, sine in 2 and 3
            c[e] = __uint_as_float(__float_as_uint(x) ^ ((quarter + (1u << 30)) & 0x80000000u)) * attention;
            s[e] = __uint_as_float(__float_as_uint(y) ^ (quarter & 0x80000000u)) * attention;
            phase[e] += inc[e];
        }
        float* row = cos_sin + static_cast<size_t>(p) * rot_dim + 4 * i;
        *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<float4*>(row + rot_dim / 2) = make_float4(s[0], s[1], s[2], s[3]);
        if (p > max_positions - step) break;        // p + step may not fit in 32 bits
    }
}

// ---- rotation and slot write ----------------------------------------------------
// HBM-bound: q is read and written once, k and v are read once and written once (16384
// tokens of 32/8 heads in bf16, 0.41 GB, take 62.3 us: 6.6 TB/s).
// Eight threads own a row (one head of one token): each holds two 16-byte pieces of it,
// the two whose components are paired with one another (half layout: pieces 8c and
// rot / 2 + 8c; interleaved: 16c and 16c + 8; past the rotated part: what is left, two
// by two).  A thread's columns are the same in every row, so it loads its 8 cosines and
// sines once and uses them for all the rows of its token that it takes (Rows of them,
// their loads all in flight together).  With few tokens a thread takes one row, so
// that the call is as short as its chain of loads (position, table row).
// The rotation is two products and a sum, each rounded to 32 bits, then one rounding to
// the type stored: what separate 32-bit operations give, bit for bit.
constexpr int kRopeThreads = 128;           // 256: 64.0 us on the 16384 tokens, 12.7 on 1040 (below)

template <bool SrcBf16, bool Fp8, bool Interleaved, int Rows>
__global__ void __launch_bounds__(kRopeThreads) rope_cache_kernel(const RopeParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const unsigned grp = blockIdx.x * (kRopeThreads / 8) + (threadIdx.x >> 3);
    const unsigned tok = grp / static_cast<unsigned>(p.groups);
    const int gi = static_cast<int>(grp % static_cast<unsigned>(p.groups));
    if (tok >= static_cast<unsigned>(p.num_tokens)) return;
    const int c = threadIdx.x & 7;
    const int heads = p.num_q_heads + p.num_kv_heads;       // rows that are rotated
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

    const long long pos = p.positions[tok];
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
    if (pos < 0) return;                                    // padding: nothing of the token is written
    const long long limit = static_cast<long long>(p.num_blocks) << p.block_shift;
    if (pos >= p.max_positions || slot >= limit) {
        if (gi == 0 && c == 0 && p.status) atomicOr(p.status, kDevErrRange);
        if (pos >= p.max_positions) return;
    }
    float cs[8], sn[8];
    if (turned && gi < heads) {
        const float4* t = reinterpret_cast<const float4*>(p.cos_sin + static_cast<size_t>(pos) * p.rot_dim + 8 * c);
        const float4* u = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(t) + half);
        const float4 a = __ldg(t), b = __ldg(t + 1), d = __ldg(u), e = __ldg(u + 1);
        cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w; cs[4] = b.x; cs[5] = b.y; cs[6] = b.z; cs[7] = b.w;
        sn[0] = d.x; sn[1] = d.y; sn[2] = d.z; sn[3] = d.w; sn[4] = e.x; sn[5] = e.y; sn[6] = e.z; sn[7] = e.w;
    }
#pragma unroll
    for (int j = 0; j < Rows; ++j) {
        const int row = gi + j * p.groups;
        if (row >= rows) break;
        const bool is_q = row < p.num_q_heads, is_v = row >= heads;
        if (!is_q && (slot < 0 || slot >= limit)) continue;
        const int h = row - (is_v ? heads : p.num_q_heads);
        const bool rot = turned && !is_v;
        float f[16];
        if (rot) {
            const uint32_t w[8] = {x0[j].x, x0[j].y, x0[j].z, x0[j].w, x1[j].x, x1[j].y, x1[j].z, x1[j].w};
            float in[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                in[2 * e] = to_float<SrcBf16>(w[e] & 0xffffu);
                in[2 * e + 1] = to_float<SrcBf16>(w[e] >> 16);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int ia = Interleaved ? 2 * e : e, ib = Interleaved ? 2 * e + 1 : 8 + e;
                f[ia] = __fsub_rn(__fmul_rn(in[ia], cs[e]), __fmul_rn(in[ib], sn[e]));
                f[ib] = __fadd_rn(__fmul_rn(in[ib], cs[e]), __fmul_rn(in[ia], sn[e]));
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
            if (rot) {
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
            if (rot) {
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
const void* rope_cache_fn(bool interleaved) {
    return interleaved ? reinterpret_cast<const void*>(&rope_cache_kernel<SrcBf16, Fp8, true, Rows>)
                       : reinterpret_cast<const void*>(&rope_cache_kernel<SrcBf16, Fp8, false, Rows>);
}

template <int Rows>
const void* rope_cache_fn(bool src_bf16, bool fp8, bool interleaved) {
    if (src_bf16) return fp8 ? rope_cache_fn<true, true, Rows>(interleaved) : rope_cache_fn<true, false, Rows>(interleaved);
    return fp8 ? rope_cache_fn<false, true, Rows>(interleaved) : rope_cache_fn<false, false, Rows>(interleaved);
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

}  // namespace

void rope_frequencies(double* freqs, int rot_dim, double base, int scaling, double factor, double trained,
                      double low_turns, double high_turns) {
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == kRopeLinear) {
            freqs[i] = f / factor;
        } else if (scaling == kRopeByParts) {
            double keep = (trained * f / kTwoPi - low_turns) / (high_turns - low_turns);
            keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
            freqs[i] = keep * f + (1.0 - keep) * f / factor;
        } else {
            freqs[i] = f;
        }
    }
}

cudaError_t launch_rope_table(float* cos_sin, int max_positions, int rot_dim, const double* freqs, float attention,
                              int sms, cudaStream_t stream) {
    RopeTurns turns = {};
    for (int i = 0; i < rot_dim / 2; ++i) {
        // |f| / 2 pi modulo one turn: the quotient is rounded once (2^-53, as an angle p f in
        // 64 bits would be), its fraction is exact (of a negative quotient it would not be:
        // 1 - 2^-60 is no double), and the product with 2^64 is cut; the sign comes last
        const double t = std::fabs(freqs[i]) / kTwoPi;
        const unsigned long long turn = static_cast<unsigned long long>((t - std::floor(t)) * 0x1p64);
        turns.turn[i] = std::signbit(freqs[i]) ? 0ull - turn : turn;
    }
    const int rows = 256 / (rot_dim / 8);
    const long long want = (static_cast<long long>(max_positions) + rows - 1) / rows;
    const long long cap = 2ll * sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < cap ? want : cap));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_table_kernel, cos_sin, max_positions, rot_dim, turns, attention);
}

cudaError_t launch_rope_cache(RopeParams p, bool src_bf16, bool fp8, bool interleaved, int sms, cudaStream_t stream) {
    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    // one row per thread group up to a few waves of CTAs, where a call is as long as its
    // chains of loads (1040 tokens of 64/8 heads into an FP8 cache: 12.0 us, with four rows
    // 13.5); four rows beyond, for the loads in flight (16384 tokens of 32/8 heads: 62.3 us,
    // with one 66.8, with two 65.9)
    const int per = static_cast<long long>(p.num_tokens) * rows <= 2048ll * sms ? 1 : 4;
    p.groups = (rows + per - 1) / per;
    constexpr int kPerCta = kRopeThreads / 8;
    const long long ctas = (static_cast<long long>(p.num_tokens) * p.groups + kPerCta - 1) / kPerCta;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&p};
    const void* fn = per == 1 ? rope_cache_fn<1>(src_bf16, fp8, interleaved) : rope_cache_fn<4>(src_bf16, fp8, interleaved);
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace pa
