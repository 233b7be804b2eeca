// RMS norm of each query and key head with the position rotation, and its gradient: the
// step between the projections and the attention of layers that normalise their heads.
//
// Forward, per token t and head, in fp32 and rounded once to bf16:
//   r = 1 / sqrt(mean_c x_c^2 + eps),  n_c = w_c x_c r   (n = x without the norm)
//   y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin     for every rotated pair (a, b)
// Gradient, with g = the rotation by the opposite angle of dy and xh = x r:
//   dw_c = sum over tokens and heads of g_c xh_c,
//   dx   = r (g w - xh mean_c(g w xh)).
//
// Both are bound by HBM: every row is read and written once.  A lane holds eight columns of
// a row as two 8-byte chunks that contain whole pairs (halves: the chunks lie rot/2 apart),
// so that no lane needs another's columns, and the arithmetic runs on packed fp32 pairs; a
// warp instruction covers a "row group" of 32 / (d / 8) rows, and a warp keeps several
// groups in flight.  A warp takes one token and walks its query heads' groups, then its key
// heads', so that the token's cosines and sines (in the forward with the norm weights
// multiplied in) stay in registers for all of them; with few tokens a token's row groups
// are spread over several warps instead (see qk_grid in lazyflash.cu).
// 32,768 tokens, 32/8 heads of 128, on one B200: forward 131 us (81 % of the measured copy
// bandwidth), gradient 208 us (76 %).  With one 16-byte chunk per lane and partners fetched
// by shuffles it was 162 and 348 us: 100 and 145 registers left 16 and 8 warps per SM.
//
// The weight gradients are summed in a fixed order: each lane over its rows, the warp and
// the block in shared memory, one partial row per block in the workspace, and a second
// kernel over the blocks.  No atomics: the same inputs give the same bits.
#pragma once

#include "lf_device.cuh"

namespace lf {

constexpr int kQkThreads = 256;
constexpr int kQkUnroll = 4;
constexpr int kQkUnrollBwd = 4;
constexpr int kQkBlocksFwd = 3, kQkBlocksBwd = 2;   // resident blocks per SM (their registers)
constexpr int kQkMaxBlocks = 148 * kQkBlocksBwd;    // blocks of the backward, one partial row each

struct QkParams {
    int T, hq, hkv, nseq, npos, rot, weights_bf16, zero_tail;
    int per_unit, units_per_token;   // row groups per unit, units per token
    const int32_t* cu;               // segment table, or null: every row counts
    const int32_t* positions;        // [T], or null: the row's index in its segment
    const float* cos_sin;            // [npos][rot]: rot/2 cosines, rot/2 sines
    float eps;
    const void *qw, *kw;             // [d] norm weights, or null: ones
    const __nv_bfloat16 *q, *k;
    int64_t qs, ks;                  // elements between tokens
    const __nv_bfloat16 *gq, *gk;    // backward: gradients of the outputs
    int64_t gqs, gks;
    __nv_bfloat16 *oq, *ok;          // outputs: rotated heads, or the inputs' gradients
    int64_t oqs, oks;
    float* partial;                  // backward: [blocks][2][d], or null
};

// Four bf16 of a row as two packed pairs.
struct Four {
    float2 lo, hi;
};
__device__ __forceinline__ uint2 ld_row8(const __nv_bfloat16* p) {
    // not the read-only path: outputs may be the inputs' own memory
    uint2 r;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ Four unpack4(uint2 v) { return {unpack2(v.x), unpack2(v.y)}; }
__device__ __forceinline__ uint2 pack4(const Four& x) {
    return make_uint2(pack_bf16(x.lo.x, x.lo.y), pack_bf16(x.hi.x, x.hi.y));
}
__device__ __forceinline__ Four operator*(const Four& a, const Four& b) {
    return {f2_mul(a.lo, b.lo), f2_mul(a.hi, b.hi)};
}
__device__ __forceinline__ Four operator*(const Four& a, float s) {
    const float2 s2 = make_float2(s, s);
    return {f2_mul(a.lo, s2), f2_mul(a.hi, s2)};
}
__device__ __forceinline__ Four fma4(const Four& a, const Four& b, const Four& c) {
    return {f2_fma(a.lo, b.lo, c.lo), f2_fma(a.hi, b.hi, c.hi)};
}
__device__ __forceinline__ Four fma4(const Four& a, float s, const Four& c) {
    const float2 s2 = make_float2(s, s);
    return {f2_fma(a.lo, s2, c.lo), f2_fma(a.hi, s2, c.hi)};
}
__device__ __forceinline__ Four neg4(const Four& a) {
    return {make_float2(-a.lo.x, -a.lo.y), make_float2(-a.hi.x, -a.hi.y)};
}
__device__ __forceinline__ Four swap4(const Four& a) {   // the other member of each neighbouring pair
    return {make_float2(a.lo.y, a.lo.x), make_float2(a.hi.y, a.hi.x)};
}
__device__ __forceinline__ Four zero4() { return {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}; }
__device__ __forceinline__ float sum4(const Four& a) { return (a.lo.x + a.lo.y) + (a.hi.x + a.hi.y); }
__device__ __forceinline__ Four ld4(const float* p) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
}

// A lane holds two chunks of four columns, A and B, of its row.  Halves: A lies in the
// rotated columns' first half and B holds the partners, rot/2 further, so that a lane
// rotates without the others; the columns past rot follow in chunk pairs.  Neighbouring
// pairs: eight consecutive columns.
struct LaneColumns {
    int a, b;
    bool on;   // its columns are rotated
};
template <bool kPairs>
__device__ __forceinline__ LaneColumns lane_columns(int l, int rot) {
    const bool on = l * 8 < rot;
    if (kPairs || !on) return {l * 8, l * 8 + 4, on};
    return {l * 4, rot / 2 + l * 4, on};
}

// cos and sin of a lane's pairs as multipliers: rotated A = A ca + P(A) sa, where P(A) is
// the other members: B (halves) or A swapped (pairs), and likewise for B.
template <bool kPairs>
struct LaneAngles {
    Four ca, sa;   // of chunk A
    Four cb, sb;   // of chunk B (kPairs; halves share the cosines and negate the sines)
    // back: the opposite angle
    __device__ void load(const float* row, int l, int rot, bool on, bool back) {
        const float sg = back ? -1.f : 1.f;
        const float2 one = make_float2(1.f, 1.f);
        ca = cb = {one, one};
        sa = sb = zero4();
        if (!on) return;
        if (kPairs) {
            const Four c = ld4(row + l * 4), s = ld4(row + rot / 2 + l * 4);
            ca = {make_float2(c.lo.x, c.lo.x), make_float2(c.lo.y, c.lo.y)};
            cb = {make_float2(c.hi.x, c.hi.x), make_float2(c.hi.y, c.hi.y)};
            sa = {make_float2(-sg * s.lo.x, sg * s.lo.x), make_float2(-sg * s.lo.y, sg * s.lo.y)};
            sb = {make_float2(-sg * s.hi.x, sg * s.hi.x), make_float2(-sg * s.hi.y, sg * s.hi.y)};
        } else {
            ca = cb = ld4(row + l * 4);
            sb = ld4(row + rot / 2 + l * 4) * sg;
            sa = neg4(sb);
        }
    }
};

// Multiplies chunk (a, b) by (ma, mb) and adds the partners times (na, nb).
template <bool kPairs>
__device__ __forceinline__ void turn(Four& a, Four& b, const Four& ma, const Four& na, const Four& mb,
                                     const Four& nb) {
    const Four pa = kPairs ? swap4(a) : b, pb = kPairs ? swap4(b) : a;
    a = fma4(pa, na, a * ma);
    b = fma4(pb, nb, b * mb);
}

// The lane's norm weights of one chunk.
__device__ __forceinline__ Four load_weights4(const void* w, int bf16, int c) {
    const float2 one = make_float2(1.f, 1.f);
    if (!w) return {one, one};
    if (bf16) return unpack4(*reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + c));
    return ld4(static_cast<const float*>(w) + c);
}

// Position of token t for the rotation, or -1 when the row takes no part (behind the last
// segment).  The whole warp calls it, converged.
__device__ __forceinline__ int token_position(const QkParams& p, int t, int t_end, bool& bad) {
    bad = false;
    if (t >= t_end) return -1;
    if (p.rot == 0) return 0;
    int pos;
    if (p.positions) {
        pos = p.positions[t];
    } else {
        const int s = segment_of_unit(p.cu, p.nseq, t, 0);
        pos = s < 0 ? -1 : t - p.cu[s];
        bad = s < 0;
    }
    if (pos < 0 || pos >= p.npos) bad = true;
    return bad ? -1 : pos;
}

// One kind of head (q or k) of a token: row groups [g0, g1) of 32 / (D / 8) rows each.
struct QkRows {
    const __nv_bfloat16* x;   // this lane's row 0 (token and lane's sub-row applied)
    const __nv_bfloat16* g;
    __nv_bfloat16* o;
    int heads;
};

template <int D, bool kNorm, bool kPairs>
__device__ __forceinline__ void qk_forward_rows(const QkRows& r, int g0, int g1, const LaneColumns& col, int sub,
                                                bool live, float eps, const LaneAngles<kPairs>& an, Four wa,
                                                Four wb) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = kQkUnroll;
    // the weights go into the angles once per token: n_c cos = x_c r (w_c cos)
    Four ma = an.ca, na = an.sa, mb = an.cb, nb = an.sb;
    if (kNorm) {
        na = na * (kPairs ? swap4(wa) : wb);
        nb = nb * (kPairs ? swap4(wb) : wa);
        ma = ma * wa;
        mb = mb * wb;
    }
    for (int gb = g0; gb < g1; gb += U) {
        uint2 ra[U], rb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (gb + u) * RPW + sub;
            ra[u] = rb[u] = make_uint2(0u, 0u);
            if (live && gb + u < g1 && h < r.heads) {
                ra[u] = ld_row8(r.x + h * D + col.a);
                rb[u] = ld_row8(r.x + h * D + col.b);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (gb + u >= g1) break;
            const int h = (gb + u) * RPW + sub;
            Four a = unpack4(ra[u]), b = unpack4(rb[u]);
            float scale = 1.f;
            if (kNorm) {
                float ss = sum4(fma4(a, a, b * b));
#pragma unroll
                for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                scale = rsqrtf(ss * (1.f / D) + eps);
            }
            const Four a0 = a, b0 = b;
            turn<kPairs>(a, b, ma, na, mb, nb);
            if (!kNorm && !col.on) {   // not even 0 * inf may reach a column that is not rotated
                a = a0;
                b = b0;
            }
            if (kNorm) {
                a = a * scale;
                b = b * scale;
            }
            if (h < r.heads) {
                *reinterpret_cast<uint2*>(r.o + h * D + col.a) = live ? pack4(a) : make_uint2(0u, 0u);
                *reinterpret_cast<uint2*>(r.o + h * D + col.b) = live ? pack4(b) : make_uint2(0u, 0u);
            }
        }
    }
}

template <int D, bool kNorm, bool kPairs>
__device__ __forceinline__ void qk_backward_rows(const QkRows& r, int g0, int g1, const LaneColumns& col, int sub,
                                                 bool live, float eps, const LaneAngles<kPairs>& an, const Four& wa,
                                                 const Four& wb, Four& acc_a, Four& acc_b) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = kQkUnrollBwd;
    for (int gb = g0; gb < g1; gb += U) {
        uint2 xa[U], xb[U], ga[U], gc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = (gb + u) * RPW + sub;
            xa[u] = xb[u] = ga[u] = gc[u] = make_uint2(0u, 0u);
            if (live && gb + u < g1 && h < r.heads) {
                ga[u] = ld_row8(r.g + h * D + col.a);
                gc[u] = ld_row8(r.g + h * D + col.b);
                if (kNorm) {
                    xa[u] = ld_row8(r.x + h * D + col.a);
                    xb[u] = ld_row8(r.x + h * D + col.b);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (gb + u >= g1) break;
            const int h = (gb + u) * RPW + sub;
            Four a = unpack4(ga[u]), b = unpack4(gc[u]);
            const Four a0 = a, b0 = b;
            turn<kPairs>(a, b, an.ca, an.sa, an.cb, an.sb);
            if (!kNorm && !col.on) {
                a = a0;
                b = b0;
            }
            if (kNorm) {
                const Four x = unpack4(xa[u]), y = unpack4(xb[u]);
                const Four ha = a * wa, hb = b * wb;
                float ss = sum4(fma4(x, x, y * y)), sd = sum4(fma4(ha, x, hb * y));
#pragma unroll
                for (int off = LPR / 2; off > 0; off >>= 1) {
                    ss += __shfl_xor_sync(0xffffffffu, ss, off);
                    sd += __shfl_xor_sync(0xffffffffu, sd, off);
                }
                const float rs = rsqrtf(ss * (1.f / D) + eps);
                const Four xr = x * rs, yr = y * rs;
                acc_a = fma4(a, xr, acc_a);
                acc_b = fma4(b, yr, acc_b);
                const float back = -(sd * (1.f / D)) * rs * rs;   // mean(g w xh) r, applied to xh
                a = fma4(xr, back, ha * rs);
                b = fma4(yr, back, hb * rs);
            }
            if (h < r.heads) {
                *reinterpret_cast<uint2*>(r.o + h * D + col.a) = live ? pack4(a) : make_uint2(0u, 0u);
                *reinterpret_cast<uint2*>(r.o + h * D + col.b) = live ? pack4(b) : make_uint2(0u, 0u);
            }
        }
    }
}

template <int D, bool kNorm, bool kPairs, bool kBack>
__global__ void __launch_bounds__(kQkThreads, kBack ? kQkBlocksBwd : kQkBlocksFwd) qk_norm_rope_kernel(QkParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, kWarps = kQkThreads / 32;
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    const int ngq = (p.hq + RPW - 1) / RPW, ng = ngq + (p.hkv + RPW - 1) / RPW;
    const long long units = (long long)p.T * p.units_per_token;
    const long long step = (long long)gridDim.x * kWarps;
    const int t_end = p.cu ? min(p.T, max(p.cu[p.nseq], 0)) : p.T;
    const LaneColumns col = lane_columns<kPairs>(l, p.rot);
    Four acc_qa = zero4(), acc_qb = zero4(), acc_ka = zero4(), acc_kb = zero4();
    long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    bool bad = false;
    int pos = unit < units ? token_position(p, static_cast<int>(unit / p.units_per_token), t_end, bad) : -1;
    while (unit < units) {
        const int t = static_cast<int>(unit / p.units_per_token);
        const int g0 = static_cast<int>(unit - (long long)t * p.units_per_token) * p.per_unit;
        const int g1 = min(ng, g0 + p.per_unit);
        const bool live = pos >= 0, skip = !live && (bad || !p.zero_tail);
        if (bad && lane == 0) {
            report_error(60, kErrBadPosition);
            mirror_error();
        }
        LaneAngles<kPairs> an;
        an.load(p.cos_sin + (size_t)max(pos, 0) * p.rot, l, p.rot, col.on && live, kBack);
        // the next unit's position is on its way while this unit's rows are
        const long long next = unit + step;
        bool next_bad = false;
        const int next_pos =
            next < units ? token_position(p, static_cast<int>(next / p.units_per_token), t_end, next_bad) : -1;
        if (!skip) {
            // an element offset: 64 bits, as the rows may lie far apart
            QkRows q, k;
            q.heads = p.hq;
            k.heads = p.hkv;
            q.x = p.q + (int64_t)t * p.qs;
            k.x = p.k + (int64_t)t * p.ks;
            q.g = p.gq + (int64_t)t * p.gqs;
            k.g = p.gk + (int64_t)t * p.gks;
            q.o = p.oq + (int64_t)t * p.oqs;
            k.o = p.ok + (int64_t)t * p.oks;
            if (g0 < ngq) {
                const Four wa = load_weights4(p.qw, p.weights_bf16, col.a), wb = load_weights4(p.qw, p.weights_bf16, col.b);
                if (kBack)
                    qk_backward_rows<D, kNorm, kPairs>(q, g0, min(g1, ngq), col, sub, live, p.eps, an, wa, wb, acc_qa, acc_qb);
                else
                    qk_forward_rows<D, kNorm, kPairs>(q, g0, min(g1, ngq), col, sub, live, p.eps, an, wa, wb);
            }
            if (g1 > ngq) {
                const int k0 = max(g0 - ngq, 0);
                const Four wa = load_weights4(p.kw, p.weights_bf16, col.a), wb = load_weights4(p.kw, p.weights_bf16, col.b);
                if (kBack)
                    qk_backward_rows<D, kNorm, kPairs>(k, k0, g1 - ngq, col, sub, live, p.eps, an, wa, wb, acc_ka, acc_kb);
                else
                    qk_forward_rows<D, kNorm, kPairs>(k, k0, g1 - ngq, col, sub, live, p.eps, an, wa, wb);
            }
        }
        unit = next;
        pos = next_pos;
        bad = next_bad;
    }
    if (kBack && kNorm && p.partial) {
        // lanes holding the same columns, then the block's warps, in a fixed order
        __shared__ float part[kWarps][2][D];
        const Four acc[4] = {acc_qa, acc_qb, acc_ka, acc_kb};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[4] = {acc[i].lo.x, acc[i].lo.y, acc[i].hi.x, acc[i].hi.y};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int off = LPR; off < 32; off <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], off);
                if (sub == 0) part[threadIdx.x >> 5][i >> 1][((i & 1) ? col.b : col.a) + e] = v[e];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += kQkThreads) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) a += part[w][i / D][i % D];
            p.partial[(size_t)blockIdx.x * 2 * D + i] = a;
        }
    }
}

// dqw and dkw [D] = the sums of the blocks' partial rows [n][2][D].  One block of 32 x 32
// threads per 32 columns; strip y takes rows y, y + 32, ...
__global__ void __launch_bounds__(1024) qk_weight_grad_kernel(const float* __restrict__ partial, int n, int D,
                                                              float* __restrict__ dqw, float* __restrict__ dkw) {
    __shared__ float part[32][33];
    const int x = threadIdx.x, y = threadIdx.y, col = blockIdx.x * 32 + x;
    float a = 0.f;
#pragma unroll 4
    for (int i = y; i < n; i += 32) a += partial[(size_t)i * 2 * D + col];
    part[y][x] = a;
    __syncthreads();
    if (y == 0) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += part[i][x];
        float* out = col < D ? dqw : dkw;
        if (out) out[col < D ? col : col - D] = a;
    }
}

}  // namespace lf
