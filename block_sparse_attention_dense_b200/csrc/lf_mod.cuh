// Modified scores: what the attention kernels do to S = <q_t, k_u> between the two matrix
// products.  In units of log2 (the softmax runs in the exp2 domain), with s2 = scale log2 e:
//   y = C tanh(S a), a = scale / cap, C = cap log2 e       (kCap; else y = S s2)
//   z = y - slope_h log2(e) |t - u|                        (kBias; kPositions: position_t - u to
//                                                           prefix keys u)
//   z = -inf unless the mask lets row t see key u          (kMask)
// and in the gradient dy = P (dP - D), dS = dy (1 - (y / C)^2) scale.
//
// Mask, per segment, rows and keys counted from its start: a row t sees its own keys
// [row_start[t], t] and the prefix keys u < P (with prefix_causal only those u <= t).
// row_start never decreases, which is what makes the tiles that a query tile needs two runs
// (the prefix, and a run that ends at the diagonal), and the rows that see a key one run.
#pragma once

#include "lf_device.cuh"

namespace lf {

enum { kModCap = 1, kModBias = 2, kModMask = 4, kModPositions = 8 };   // the last with kModBias | kModMask only

// tanh(x) = x p(x^2), p a relative minimax fit (iterated weighted least squares on Chebyshev
// nodes, in double).  tanh.approx (2^-11) would cost the scores three digits, and exp and a
// reciprocal two more operations of the unit that the softmax already fills.
//  * kCapFused: |x| <= 0.7, degree four, off by 3.1e-7 of tanh.  The scale goes into the
//    coefficients (C a^(2k+1) c_k, powers of s), which holds while those stay normal numbers
//    (the host sets fused_max to 0 where they would not): six packed operations a pair
//    instead of the uncapped one.  Degree three (to 0.5) made the forward 6 % faster where
//    all scores lie within it, and three times slower where some do not (16,384 tokens,
//    scores of deviation 2: cap 50 2.22 against 2.36 ms, cap 14 6.4 against 2.8 ms).
//  * kCapCoef: |x| <= 3/4, degree five, off by 2.9e-8, and 1.6e-7 in fp32; beyond,
//    1 - 2 / (1 + exp(2 |x|)), whose error is below 4e-7 of tanh there.
// A warp (or, in the gradient, a chunk of 16 columns) whose scores all lie within the first
// takes it, else the second for all of them.
constexpr int kCapFusedTerms = 5;
constexpr double kCapFused[kCapFusedTerms] = {0.999999697294, -0.333302129002, 0.132811125731,
                                              -0.050836235324, 0.013773709951};
constexpr double kCapFusedRange = 0.7;
constexpr float kCapRange = 0.75f;
constexpr int kCapTerms = 6;
constexpr double kCapCoef[kCapTerms] = {0.999999971014, -0.333329588792, 0.133254060138,
                                        -0.053344429950, 0.019582907796, -0.004716256973};

struct ModParams {
    float cap_in;                      // a
    float cap_damp;                    // -1 / C^2
    float cap_out;                     // C
    float cap_coef[kCapTerms];         // C times the wide fit's coefficients
    float cap_fused[kCapFusedTerms];   // C a^(2k+1) times the narrow fit's
    float fused_max;                   // the largest |s| of the narrow fit
    const float* slopes;               // [hq]
    const int32_t* prefix;             // [nseq], or null
    int prefix_causal;
    const int32_t* row_start;          // [T], or null
};

// C tanh(a s) / s of a pair within the narrow fit.
__device__ __forceinline__ float2 cap_fused_factor(const ModParams& m, float2 s) {
    const float2 w = f2_mul(s, s);
    float2 p = make_float2(m.cap_fused[kCapFusedTerms - 1], m.cap_fused[kCapFusedTerms - 1]);
#pragma unroll
    for (int i = kCapFusedTerms - 2; i >= 0; --i) p = f2_fma(p, w, make_float2(m.cap_fused[i], m.cap_fused[i]));
    return p;
}
__device__ __forceinline__ float cap_fused_one(const ModParams& m, float s) {
    const float w = s * s;
    float p = m.cap_fused[kCapFusedTerms - 1];
#pragma unroll
    for (int i = kCapFusedTerms - 2; i >= 0; --i) p = fmaf(p, w, m.cap_fused[i]);
    return p * s;
}

// C tanh(a s) of a pair, |a s| <= kCapRange.
__device__ __forceinline__ float2 cap_near(const ModParams& m, float2 s) {
    const float2 x = f2_mul(s, make_float2(m.cap_in, m.cap_in));
    const float2 w = f2_mul(x, x);
    float2 p = make_float2(m.cap_coef[kCapTerms - 1], m.cap_coef[kCapTerms - 1]);
#pragma unroll
    for (int i = kCapTerms - 2; i >= 0; --i) p = f2_fma(p, w, make_float2(m.cap_coef[i], m.cap_coef[i]));
    return f2_mul(p, x);
}
// The same for any s.
__device__ __forceinline__ float cap_far(const ModParams& m, float s) {
    const float x = s * m.cap_in;
    const float e = fast_exp2(fabsf(x) * 2.8853900817779268f);   // exp(2 |x|); inf is fine
    return copysignf(fmaf(-2.f * m.cap_out, __fdividef(1.f, 1.f + e), m.cap_out), x);
}
__device__ __forceinline__ float2 cap_any(const ModParams& m, float2 s) {
    const float2 y = cap_near(m, s);
    return make_float2(fabsf(s.x * m.cap_in) <= kCapRange ? y.x : cap_far(m, s.x),
                       fabsf(s.y * m.cap_in) <= kCapRange ? y.y : cap_far(m, s.y));
}

// The same with the derivative 1 - tanh^2.  It comes from r = 2 / (1 + exp(2 |x|)), as
// |tanh x| = 1 - r: the derivative is r (2 - r), to a few roundings of itself at every x.  From
// y it would be off by y's own rounding, about 1e-6, which is more than all of it for |x| above 7.
__device__ __forceinline__ float2 cap_any(const ModParams& m, float2 s, float2& damp) {
    const float2 x = f2_mul(s, make_float2(m.cap_in, m.cap_in)), y = cap_near(m, s);
    auto ratio = [](float v) { return __fdividef(2.f, 1.f + fast_exp2(fabsf(v) * 2.8853900817779268f)); };
    const float2 r = make_float2(ratio(x.x), ratio(x.y));
    damp = f2_mul(r, f2_sub(make_float2(2.f, 2.f), r));
    const float2 far = f2_fma(make_float2(-m.cap_out, -m.cap_out), r, make_float2(m.cap_out, m.cap_out));
    return make_float2(fabsf(x.x) <= kCapRange ? y.x : copysignf(far.x, x.x),
                       fabsf(x.y) <= kCapRange ? y.y : copysignf(far.y, x.y));
}

// The largest value, and the largest size, of a thread's 128 scores (three-input maxima,
// four independent chains).
__device__ __forceinline__ float row_max(const float (&s)[128]) {
    float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 128; e += 8) {
#pragma unroll
        for (int q = 0; q < 4; ++q) mq[q] = fmax3(mq[q], s[e + 2 * q], s[e + 2 * q + 1]);
    }
    return fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3]));
}
// max(|a|, |b|, |c|) in one instruction (three-input form).
__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float row_max_size(const float (&s)[128]) {
    float mq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 128; e += 8) {
#pragma unroll
        for (int q = 0; q < 4; ++q) mq[q] = fmax3_abs(mq[q], s[e + 2 * q], s[e + 2 * q + 1]);
    }
    return fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3]));
}

// The cap over a thread's 128 scores, whatever they are.
__device__ __forceinline__ void cap_scores(const ModParams& m, float (&s)[128]) {
    if (__any_sync(0xffffffffu, !(row_max_size(s) * m.cap_in <= kCapRange))) {
#pragma unroll
        for (int e = 0; e < 128; e += 2) {
            const float2 y = cap_any(m, make_float2(s[e], s[e + 1]));
            s[e] = y.x;
            s[e + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 128; e += 2) {
            const float2 y = cap_near(m, make_float2(s[e], s[e + 1]));
            s[e] = y.x;
            s[e + 1] = y.y;
        }
    }
}

// The prefix length of segment s within its length.
__device__ __forceinline__ int prefix_of(const ModParams& m, int s, int len, bool& bad) {
    if (!m.prefix) return 0;
    const int p = m.prefix[s];
    bad = p < 0;
    return min(max(p, 0), len);
}

// Row t's position within its bounds: the distance to the prefix keys that it sees, u < P and
// u <= t, is then never negative, nor more than that in rows.
__device__ __forceinline__ int bounded_position(int pos, int t, int P) { return min(max(pos, min(t, P - 1)), t); }

// The KV tiles that a pair of query tiles (2m, 2m+1) needs, in ascending order: slot i is KV
// tile i for i < n_prefix, then lo, lo + 1, ...  The forward takes the slots from the last to
// the first: a row then meets its own key, or prefix keys, in its first tile, so that it has
// a maximum from the start, and with a distance bias close to its last one.  A query tile
// has work in the slots whose tile lies in its own runs [0, np) and [lo, hi).
struct PairSlots {
    int n_prefix, lo;
    __device__ int tile(int i) const { return i < n_prefix ? i : lo + i - n_prefix; }
};
struct TileRuns {
    int np, lo, hi;
    // one past the last slot with work for this tile
    __device__ int slots(const PairSlots& p) const {
        return hi > p.lo ? p.n_prefix + hi - p.lo : max(np, hi);
    }
    // the slots below slots() without work are [np, idle_end)
    __device__ int idle_end(const PairSlots& p) const {
        return lo <= p.n_prefix ? max(lo, np) : p.n_prefix + max(lo - p.lo, 0);
    }
    // the tile after j, in the forward's order (below 0: none)
    __device__ int next(int j) const { return j - 1 < lo && j - 1 >= np ? np - 1 : j - 1; }
};
__device__ __forceinline__ TileRuns tile_runs(const ModParams& m, int qt, int seg0, int len, int P) {
    const int q0 = qt * 128;
    TileRuns r;
    const int seen = m.prefix_causal ? min(P, min(q0 + 128, len)) : P;
    r.np = (seen + 127) >> 7;
    r.lo = m.row_start ? min(max(m.row_start[seg0 + q0], 0), q0) >> 7 : 0;
    r.hi = qt + 1;
    return r;
}

// Last row of the segment that sees key u as its own: rows' starts ascend, so a bisection.
__device__ __forceinline__ int last_row_of_key(const int32_t* row_start, int seg0, int len, int u) {
    int lo = u, hi = len;   // the first row with a start behind u lies in (lo, hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row_start[seg0 + mid] <= u) lo = mid; else hi = mid;
    }
    return lo;
}

}  // namespace lf
