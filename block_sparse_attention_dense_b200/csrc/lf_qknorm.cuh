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
// Both are bound by HBM: every row is read and written once.  A row of d bf16 is d / 8
// lanes of 16 bytes, so a warp instruction covers a "row group" of 32 / (d / 8) rows, and
// a warp keeps kQkUnroll groups in flight, the query heads' groups first (a group never
// mixes query and key heads).  A warp takes one token and walks its heads, so
// that the token's position, cosines and sines and the weights stay in registers for all
// of them; with few tokens a token's row groups are spread over several warps instead (see
// launch_qk in lazyflash.cu).  The members of a pair lie rot/2 apart in the
// halves pairing: lanes exchange them by shuffles; neighbouring pairs lie in one lane.
//
// The weight gradients are summed in a fixed order: each lane over its rows, the warp and
// the block in shared memory, one partial row per block in the workspace, and a second
// kernel over the blocks.  No atomics: the same inputs give the same bits.
#pragma once

#include "lf_device.cuh"

namespace lf {

constexpr int kQkThreads = 256;
constexpr int kQkUnroll = 4;
constexpr int kQkMaxBlocks = 148 * 4;   // blocks of the backward, one partial row each

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

// A failure that the next call has to see: the flag, and its host-mapped copy at once
// (these kernels are not followed by the mirroring kernel).
__device__ __forceinline__ void report_error_now(int site, int kind) {
    report_error(site, kind);
    int* m = g_error_mirror;
    if (m) {
        *reinterpret_cast<volatile int*>(m) = (site << 8) | kind;
        __threadfence_system();
    }
}

__device__ __forceinline__ uint4 ld_row16(const __nv_bfloat16* p) {
    // not the read-only path: outputs may be the inputs' own memory
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
}

// The lane's eight norm weights.
__device__ __forceinline__ void load_weights8(const void* w, int bf16, int c8, float (&out)[8]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = 1.f;
    } else if (bf16) {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c8), out);
    } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c8);
        const float4 a = f[0], b = f[1];
        out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
        out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
    }
}

// One lane's part of a token's rotation: columns [c8, c8 + 8) of the head.
template <bool kPairs>
struct LaneRotation {
    float c[8], s[8];     // kPairs: c[0..3], s[0..3] of the lane's four pairs
    int partner;          // halves: the lane that holds the other members
    bool on;              // the lane's columns are rotated

    __device__ void init(int lane, int lpr, int rot) {
        const int l = lane % lpr;
        on = l * 8 < rot;
        partner = lane;
        if (!kPairs && on) partner = l * 16 < rot ? lane + rot / 16 : lane - rot / 16;
    }
    __device__ void load(const float* row, int l, int rot) {
        if (!on) return;
        if (kPairs) {
            const float4 a = *reinterpret_cast<const float4*>(row + l * 4);
            const float4 b = *reinterpret_cast<const float4*>(row + rot / 2 + l * 4);
            c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
            s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
        } else {
            const bool first = l * 16 < rot;
            const int i = first ? l * 8 : l * 8 - rot / 2;
            const float sg = first ? -1.f : 1.f;   // y_a = n_a c - n_b s, y_b = n_b c + n_a s
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 a = *reinterpret_cast<const float4*>(row + i + e);
                const float4 b = *reinterpret_cast<const float4*>(row + rot / 2 + i + e);
                c[e] = a.x; c[e + 1] = a.y; c[e + 2] = a.z; c[e + 3] = a.w;
                s[e] = sg * b.x; s[e + 1] = sg * b.y; s[e + 2] = sg * b.z; s[e + 3] = sg * b.w;
            }
        }
    }
    // Rotates the lane's eight values in place; kBack: by the opposite angle.  Every lane
    // of the warp calls it.
    template <bool kBack>
    __device__ void apply(float (&x)[8]) const {
        if (kPairs) {
            if (on) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float sn = kBack ? -s[e / 2] : s[e / 2], a = x[e], b = x[e + 1];
                    x[e] = a * c[e / 2] - b * sn;
                    x[e + 1] = b * c[e / 2] + a * sn;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float o = __shfl_sync(0xffffffffu, x[e], partner);
                const float sn = kBack ? -s[e] : s[e];
                if (on) x[e] = x[e] * c[e] + o * sn;
            }
        }
    }
};

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

template <int D, bool kNorm, bool kPairs>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(QkParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = kQkUnroll;
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR, c8 = l * 8;
    const int ngq = (p.hq + RPW - 1) / RPW, ng = ngq + (p.hkv + RPW - 1) / RPW;
    const long long units = (long long)p.T * p.units_per_token;
    const long long nwarps = (long long)gridDim.x * (kQkThreads / 32);
    const int t_end = p.cu ? min(p.T, max(p.cu[p.nseq], 0)) : p.T;
    LaneRotation<kPairs> rot;
    rot.init(lane, LPR, p.rot);
    float wq[8], wk[8];
    if (kNorm) {
        load_weights8(p.qw, p.weights_bf16, c8, wq);
        load_weights8(p.kw, p.weights_bf16, c8, wk);
    }
    for (long long unit = (long long)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5); unit < units;
         unit += nwarps) {
        const int t = static_cast<int>(unit / p.units_per_token);
        const int g0 = static_cast<int>(unit % p.units_per_token) * p.per_unit;
        const int g1 = min(ng, g0 + p.per_unit);
        bool bad;
        const int pos = token_position(p, t, t_end, bad);
        if (bad && lane == 0) report_error_now(60, kErrBadPosition);
        const bool live = pos >= 0;
        if (!live && (bad || !p.zero_tail)) continue;
        if (live && p.rot > 0) rot.load(p.cos_sin + (size_t)pos * p.rot, l, p.rot);
        const __nv_bfloat16* qrow = p.q + (int64_t)t * p.qs + c8;
        const __nv_bfloat16* krow = p.k + (int64_t)t * p.ks + c8;
        __nv_bfloat16* oq = p.oq + (int64_t)t * p.oqs + c8;
        __nv_bfloat16* ok = p.ok + (int64_t)t * p.oks + c8;
        for (int gb = g0; gb < g1; gb += U) {
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int gi = gb + u;
                const bool is_k = gi >= ngq;
                const int h = (is_k ? gi - ngq : gi) * RPW + sub;
                raw[u] = make_uint4(0u, 0u, 0u, 0u);
                if (live && gi < g1 && h < (is_k ? p.hkv : p.hq))
                    raw[u] = ld_row16((is_k ? krow : qrow) + h * D);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int gi = gb + u;
                if (gi >= g1) break;
                const bool is_k = gi >= ngq;
                const int h = (is_k ? gi - ngq : gi) * RPW + sub;
                float x[8];
                unpack8(raw[u], x);
                if (kNorm) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                    for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                    const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (is_k ? wk[e] : wq[e]);
                }
                if (p.rot > 0) rot.template apply<false>(x);
                if (h < (is_k ? p.hkv : p.hq))
                    *reinterpret_cast<uint4*>((is_k ? ok : oq) + h * D) =
                        live ? pack8(x) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
}

template <int D, bool kNorm, bool kPairs>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_bwd_kernel(QkParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = kQkUnroll;
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR, c8 = l * 8;
    const int ngq = (p.hq + RPW - 1) / RPW, ng = ngq + (p.hkv + RPW - 1) / RPW;
    const long long units = (long long)p.T * p.units_per_token;
    const long long nwarps = (long long)gridDim.x * (kQkThreads / 32);
    const int t_end = p.cu ? min(p.T, max(p.cu[p.nseq], 0)) : p.T;
    LaneRotation<kPairs> rot;
    rot.init(lane, LPR, p.rot);
    float wq[8], wk[8], aq[8], ak[8];
    if (kNorm) {
        load_weights8(p.qw, p.weights_bf16, c8, wq);
        load_weights8(p.kw, p.weights_bf16, c8, wk);
#pragma unroll
        for (int e = 0; e < 8; ++e) aq[e] = ak[e] = 0.f;
    }
    for (long long unit = (long long)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5); unit < units;
         unit += nwarps) {
        const int t = static_cast<int>(unit / p.units_per_token);
        const int g0 = static_cast<int>(unit % p.units_per_token) * p.per_unit;
        const int g1 = min(ng, g0 + p.per_unit);
        bool bad;
        const int pos = token_position(p, t, t_end, bad);
        if (bad && lane == 0) report_error_now(61, kErrBadPosition);
        const bool live = pos >= 0;
        if (!live && (bad || !p.zero_tail)) continue;
        if (live && p.rot > 0) rot.load(p.cos_sin + (size_t)pos * p.rot, l, p.rot);
        const __nv_bfloat16* qrow = kNorm ? p.q + (int64_t)t * p.qs + c8 : nullptr;
        const __nv_bfloat16* krow = kNorm ? p.k + (int64_t)t * p.ks + c8 : nullptr;
        const __nv_bfloat16* gq = p.gq + (int64_t)t * p.gqs + c8;
        const __nv_bfloat16* gk = p.gk + (int64_t)t * p.gks + c8;
        __nv_bfloat16* oq = p.oq + (int64_t)t * p.oqs + c8;
        __nv_bfloat16* ok = p.ok + (int64_t)t * p.oks + c8;
        for (int gb = g0; gb < g1; gb += U) {
            uint4 raw[U], grad[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int gi = gb + u;
                const bool is_k = gi >= ngq;
                const int h = (is_k ? gi - ngq : gi) * RPW + sub;
                raw[u] = grad[u] = make_uint4(0u, 0u, 0u, 0u);
                if (live && gi < g1 && h < (is_k ? p.hkv : p.hq)) {
                    grad[u] = ld_row16((is_k ? gk : gq) + h * D);
                    if (kNorm) raw[u] = ld_row16((is_k ? krow : qrow) + h * D);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int gi = gb + u;
                if (gi >= g1) break;
                const bool is_k = gi >= ngq;
                const int h = (is_k ? gi - ngq : gi) * RPW + sub;
                float g[8];
                unpack8(grad[u], g);
                if (p.rot > 0) rot.template apply<true>(g);
                if (kNorm) {
                    float x[8], ss = 0.f, sd = 0.f;
                    unpack8(raw[u], x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        ss = fmaf(x[e], x[e], ss);
                        sd = fmaf(g[e] * (is_k ? wk[e] : wq[e]), x[e], sd);
                    }
#pragma unroll
                    for (int off = LPR / 2; off > 0; off >>= 1) {
                        ss += __shfl_xor_sync(0xffffffffu, ss, off);
                        sd += __shfl_xor_sync(0xffffffffu, sd, off);
                    }
                    const float r = rsqrtf(ss * (1.f / D) + p.eps);
                    const float back = sd * r * r * (1.f / D);   // mean(g w xh) r, applied to x
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float gx = g[e] * x[e] * r;
                        if (is_k) ak[e] += gx; else aq[e] += gx;
                        g[e] = r * (g[e] * (is_k ? wk[e] : wq[e]) - x[e] * back);
                    }
                }
                if (h < (is_k ? p.hkv : p.hq))
                    *reinterpret_cast<uint4*>((is_k ? ok : oq) + h * D) =
                        live ? pack8(g) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
    if (kNorm && p.partial) {
        // lanes holding the same columns, then the block's warps, in a fixed order
        __shared__ float part[kQkThreads / 32][2][D];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int off = LPR; off < 32; off <<= 1) {
                aq[e] += __shfl_xor_sync(0xffffffffu, aq[e], off);
                ak[e] += __shfl_xor_sync(0xffffffffu, ak[e], off);
            }
            if (sub == 0) {
                part[threadIdx.x >> 5][0][c8 + e] = aq[e];
                part[threadIdx.x >> 5][1][c8 + e] = ak[e];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += kQkThreads) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < kQkThreads / 32; ++w) a += part[w][i / D][i % D];
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
