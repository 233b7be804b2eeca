// Dense attention forward on sm_100a (the LazyFlash forward is FlashAttention's,
// unchanged: article standfirst and section "Le passage arrière fait deux fois
// le travail du passage avant").
//
// One CTA computes two consecutive 128-row query tiles (2m, 2m+1) of one head
// of one segment, in ping-pong: while one softmax warpgroup turns its score
// tile into probabilities, the tensor core computes the other tile's scores
// and P.V products.
//   TMA:      both Q tiles once; K and V tiles through two-stage rings;
//   tcgen05:  S_t = Q_t K_j^T (SS, 128 x 128 fp32 in TMEM), O_t += P_t V_j
//             (TS: P_t read from TMEM, where the softmax wrote it over S_t);
//   softmax:  warpgroup t, thread r owns query row r (TMEM lane r): online
//             softmax in the exp2 domain with a stale-max rule (the reference
//             maximum moves only when the row maximum grows by more than 2^8,
//             and only then is O rescaled in TMEM); P is written in four
//             32-column chunks, and P.V starts once the first half is stored;
//   epilogue: O / l -> bf16, LSE = (m + log2 l) * ln 2.
// Roles (384 threads): warp 0 TMA producer, warps 1 and 2 MMA issuers of tile 0
// and tile 1 (whole warp, one elected lane issues; the two take turns so the
// tensor pipe sees the ping-pong order), warps 4-7 softmax of tile 0, warps
// 8-11 softmax of tile 1.
// Tensor memory (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+d),
// O1 [384,384+d); P_t (bf16, packed two per column) over S_t [0,64).  Reuse
// of a region by a later MMA relies on tcgen05.mma executing in issue order.
//
// kMod selects modified scores (lf_mod.cuh) at compile time: the tanh cap and the distance
// bias in the softmax warps, the masks also in the KV tiles that are visited.  KV tiles are
// then taken from the diagonal down, so that a row has its reference from its first tile.
// Under a mask the two query tiles of a CTA share one list of KV tiles (the prefix's, and a
// run up to the diagonal), and a tile that has nothing in a step only hands the step's
// stages back, so that a document's end between the two does not make the later one walk
// the earlier one's keys.  Distances to prefix keys may be counted from the rows' positions
// (kModPositions: a shared prompt's answers): a row's distances then have another start in the
// prefix's tiles, and in the one tile at the prefix's end a start per key.  A variant of its
// own, as the same code behind a runtime test made the biased masks 2-3 % slower.
// A row's softmax warp is bound by its own latency (under a cap the exp2 unit is busy 40 % of
// the time and the FMA pipes 23 %), so the cap and the bias are laid beside the exp2
// (capped_row; `fused`).  16,384 tokens, 32/8 heads of 128, causal, scores of deviation 2, ms in
// short runs (in brackets back to back, under the power cap): plain 1.76 (1.97), cap 50 2.29
// (2.51), cap 100, which keeps the running maximum, 2.74 (2.90), bias 2.00 (2.15), a mask that
// hides nothing 1.83 (2.05), cap and bias 2.45 (2.60), a window of 1,024 keys 0.45 (0.42).
// P is rounded to bf16, the type in which the tensor core takes it beside V; its sums stay in fp32.
#pragma once

#include <climits>
#include <type_traits>

#include "lf_device.cuh"
#include "lf_mod.cuh"

namespace lf {

struct FwdParams {
    const int32_t* cu_seqlens;
    int T, hq, hkv, causal, max_seqlen, nseq;
    float scale_log2;          // softmax_scale * log2(e)
    int tile_major;            // CTA order: 1 = KV head fastest (see the kernel)
    __nv_bfloat16* o;
    float* lse;
};
struct FwdModParams : FwdParams {
    ModParams mod;
    __nv_bfloat16* o_low;      // [T][hq][D] what rounding took from o, or null (bf16: 16 bits of O
                               // in all, which leaves D no error beside that of P's rounding)
};
struct FwdPositionsParams : FwdModParams {
    const int32_t* positions;  // [T] where distances to prefix keys are counted from
};
template <int kMod>
using FwdParamsOf =
    std::conditional_t<kMod == 0, FwdParams,
                       std::conditional_t<(kMod & kModPositions) != 0, FwdPositionsParams, FwdModParams>>;

template <int D>
struct FwdSmem {
    static constexpr int kPanels = D / 64;
    static constexpr uint32_t kTile = kPanels * kPanelBytes;     // one 128 x D bf16 tile
    static constexpr uint32_t kQ = 0;                            // 2 tiles
    static constexpr uint32_t kK = kQ + 2 * kTile;               // 2 stages
    static constexpr uint32_t kV = kK + 2 * kTile;               // 2 stages
    static constexpr uint32_t kBars = kV + 2 * kTile;
    static constexpr uint32_t kBytes = kBars + 256;
    static constexpr uint32_t kAlloc = kBytes + 1024;            // slack for 1024-B alignment
};

constexpr int kFwdThreads = 384;
constexpr int kFwdLaunchRegs = 168;     // 65536 / 384, rounded down to a multiple of 8
constexpr int kFwdCtrlRegs = 64;
constexpr int kFwdSoftmaxRegs = 216;
constexpr float kRescaleThreshold = 8.0f;   // log2 of the largest P before a rescale
constexpr float kBoundedCap = 80.0f;        // cap * log2(e) up to which rows need no maximum
constexpr float kFusedAbove = 40.0f;        // log2 of the largest P of a fused tile

// Adds a packed bf16 pair to a pair of fp32 sums.
__device__ __forceinline__ void add_packed(float2& sum, uint32_t packed) {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; add.f32.bf16 %0, l, %0; add.f32.bf16 %1, h, %1;}"
        : "+f"(sum.x), "+f"(sum.y)
        : "r"(packed));
}

// A row's sum of P, as computed and as rounded to bf16.
struct RowSums {
    float exact, rounded;
};

// The keys of a KV tile that a row sees, counted from the tile's first: [0, pre) and the
// own + 1 keys from `first` on (one unsigned compare for those: with two, the compiler
// spilled a quarter of the scores).
struct RowView {
    int pre, first;
    unsigned own;
    __device__ bool sees(int e) const { return e < pre || static_cast<unsigned>(e - first) <= own; }
};

// One row's softmax numerators over a KV tile, under a cap of at most kBoundedCap: P = 2^(C tanh(a s) + bias part) to TMEM over S, an arrival on `half` once its
// first 64 columns are stored (the caller does the second); returns the row's sums.
// A row is four chunks of 32 columns.  While chunk c goes through the exp2 unit, chunk c + 1
// is capped, chunk c - 1 summed and packed, and the range of chunk c + 2 looked at (its vote
// decides between the narrow fit and the general form two chunks ahead).
//   dist_bias: bias of column 0; bias2: its step from one column to the next, negated;
//   kHidden: the tile has keys that some row does not see (view: this row's).  A variant of
//   its own: a branch per chunk split the pairing above and cost 10 % on whole tiles.
template <bool kBias, bool kHidden>
__device__ __forceinline__ RowSums capped_row(const ModParams& m, uint32_t t_s, float dist_bias, float bias2,
                                            const float2 (&bias_in8)[4], const RowView& view, uint64_t* half) {
    float sv[128];
    uint32_t sr[8][16];
#pragma unroll
    for (int i = 0; i < 2; ++i) tmem_ld16_nowait(t_s + i * 16, sr[i]);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 2; ++i) tmem_regs_ready(sr[i]);
#pragma unroll
    for (int i = 2; i < 8; ++i) tmem_ld16_nowait(t_s + i * 16, sr[i]);
    auto take = [&](int i) {
#pragma unroll
        for (int e = 0; e < 16; ++e) sv[i * 16 + e] = __uint_as_float(sr[i][e]);
    };
    auto in_range = [&](int c) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            a = fmax3_abs(a, sv[c * 32 + e], sv[c * 32 + e + 1]);
            b = fmax3_abs(b, sv[c * 32 + e + 2], sv[c * 32 + e + 3]);
        }
        return !__any_sync(0xffffffffu, !(fmaxf(a, b) <= m.fused_max));
    };
    // the bias of columns [e, e + 1]: multiples of eight, and within eight
    auto bias_at = [&](int e) {
        const float at = fmaf(static_cast<float>(-(e / 8 * 8)), bias2, dist_bias);
        return f2_add(make_float2(at, at), bias_in8[(e % 8) / 2]);
    };
    auto narrow = [&](int e) {
        const float2 s2 = make_float2(sv[e], sv[e + 1]);
        const float2 p = cap_fused_factor(m, s2);
        float2 x;
        if constexpr (kBias)
            x = f2_fma(p, s2, bias_at(e));
        else
            x = f2_mul(p, s2);
        sv[e] = x.x;
        sv[e + 1] = x.y;
    };
    auto general = [&](int c) {
#pragma unroll
        for (int e = c * 32; e < c * 32 + 32; e += 2) {
            float2 x = cap_any(m, make_float2(sv[e], sv[e + 1]));
            if constexpr (kBias) x = f2_add(x, bias_at(e));
            sv[e] = x.x;
            sv[e + 1] = x.y;
        }
    };
    auto hide = [&](int c) {
#pragma unroll
        for (int e = c * 32; e < c * 32 + 32; ++e) sv[e] = view.sees(e) ? sv[e] : -INFINITY;
    };
    take(0);
    take(1);
    if (in_range(0)) {
#pragma unroll
        for (int e = 0; e < 32; e += 2) narrow(e);
    } else {
        general(0);
    }
    if (kHidden) hide(0);
    tmem_wait_ld();
#pragma unroll
    for (int i = 2; i < 8; ++i) {
        tmem_regs_ready(sr[i]);
        take(i);
    }
    bool fits = in_range(1);
    float p[2][32] = {};
    float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, rounded[2] = {rs[0], rs[0]};
    uint32_t pk[16];
    auto finish = [&](int c, int e) {   // sum and pack columns [e, e + 1] of chunk c
        const float2 q = make_float2(p[c & 1][e], p[c & 1][e + 1]);
        rs[(e >> 1) & 1] = f2_add(rs[(e >> 1) & 1], q);
        pk[e / 2] = pack_bf16(q.x, q.y);
        add_packed(rounded[(e >> 1) & 1], pk[e / 2]);
    };
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        auto exp2_pair = [&](int e) {
            p[c & 1][e] = fast_exp2(sv[c * 32 + e]);
            p[c & 1][e + 1] = fast_exp2(sv[c * 32 + e + 1]);
        };
        if (c < 3 && fits) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                exp2_pair(e);
                narrow((c + 1) * 32 + e);
                if (c > 0) finish(c - 1, e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                exp2_pair(e);
                if (c > 0) finish(c - 1, e);
            }
            if (c < 3) general(c + 1);
        }
        if (c < 3 && kHidden) hide(c + 1);
        if (c < 2) fits = in_range(c + 2);
        if (c > 0) tmem_st16(t_s + (c - 1) * 16, pk);
        if (c == 2) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(half);
        }
    }
#pragma unroll
    for (int e = 0; e < 32; e += 2) finish(3, e);
    tmem_st16(t_s + 48, pk);
    return {(rs[0].x + rs[0].y) + (rs[1].x + rs[1].y),
            (rounded[0].x + rounded[0].y) + (rounded[1].x + rounded[1].y)};
}

template <int D, int kMod>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, FwdParamsOf<kMod> prm) {
    using L = FwdSmem<D>;
    constexpr bool kCap = (kMod & kModCap) != 0, kBias = (kMod & kModBias) != 0, kMask = (kMod & kModMask) != 0,
                   kPositions = (kMod & kModPositions) != 0;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* bar_q = bars + 0;
    uint64_t* bar_k_full = bars + 1;    // [2]
    uint64_t* bar_k_empty = bars + 3;   // [2]
    uint64_t* bar_v_full = bars + 5;    // [2]
    uint64_t* bar_v_empty = bars + 7;   // [2]
    uint64_t* bar_s_full = bars + 9;    // [2] per query tile
    uint64_t* bar_p_ready = bars + 11;  // [2]
    uint64_t* bar_o_done = bars + 13;   // [2]
    uint64_t* bar_done = bars + 15;     // [2] per MMA issuer
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 17);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 18);
    volatile int* burst_seq = reinterpret_cast<volatile int*>(bars + 19);   // [2] bursts issued per MMA issuer
    uint64_t* bar_p_half = bars + 20;   // [2] per query tile: P columns [0, 64) written

    // blockIdx.x = pair * G + query head within the KV head's group, the pairs of
    // 256 query rows running over all segments, segment by segment; blockIdx.y = KV
    // head.  The G query heads that share a KV head run together, longest rows first
    // within each segment, so their K/V stay in L2 and each group's work outlasts its
    // heaviest CTA.  With few waves of CTAs (tile_major) the KV head runs fastest
    // instead, so that every KV head's longest rows start first rather than the last
    // head's running alone at the end.
    const int G = prm.hq / prm.hkv;
    int g, xr;
    if (prm.tile_major) {
        const int lin = static_cast<int>(blockIdx.x + blockIdx.y * gridDim.x);
        g = lin % static_cast<int>(gridDim.y);
        xr = lin / static_cast<int>(gridDim.y);
    } else {
        g = blockIdx.y;
        xr = blockIdx.x;
    }
    const int h = g * G + xr % G;
    const int pg = xr / G;
    const int s = segment_of_unit(prm.cu_seqlens, prm.nseq, pg, 8);
    if (s < 0) return;
    int seg0, len;
    if (!load_segment(prm.cu_seqlens, s, prm.T, prm.max_seqlen, seg0, len, 20)) {
        if (kMod != 0 && threadIdx.x == 0) mirror_error();
        return;
    }
    const int ntiles = (len + 127) >> 7;
    const int npairs = (ntiles + 1) >> 1;
    const int m = npairs - 1 - (pg - first_unit_of_segment(seg0, s, 8));   // longest rows first
    if (m < 0) return;
    const bool two = 2 * m + 1 < ntiles;                     // tile 1 exists
    // KV tiles each query tile needs (under a mask: its slots up to the last one with work)
    int nkv0 = prm.causal ? 2 * m + 1 : ntiles;
    int nkv1 = two ? (prm.causal ? 2 * m + 2 : ntiles) : 0;
    int P = 0;                       // prefix length
    PairSlots slots{};
    TileRuns runs0{}, runs1{};
    if constexpr (kMask) {
        bool bad = false;
        P = prefix_of(prm.mod, s, len, bad);
        if (bad && threadIdx.x == 0) {
            report_error(17, kErrBadMask);
            mirror_error();
        }
        runs0 = tile_runs(prm.mod, 2 * m, seg0, len, P);
        runs1 = two ? tile_runs(prm.mod, 2 * m + 1, seg0, len, P) : TileRuns{0, 0, 0};
        runs1.lo = max(runs1.lo, runs0.lo);   // starts never decrease; all roles rely on it
        slots.n_prefix = max(runs0.np, runs1.np);
        slots.lo = max(runs0.lo, slots.n_prefix);
        nkv0 = runs0.slots(slots);
        nkv1 = two ? runs1.slots(slots) : 0;
    }
    const int nkv = nkv0 > nkv1 ? nkv0 : nkv1;
    // the KV tile of step i: in ascending order, with modified scores in descending order
    auto kv_tile = [&](int i) { return kMask ? slots.tile(nkv - 1 - i) : kMod ? nkv - 1 - i : i; };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t s_base = smem_addr(smem);

    if (tid == 0) {
        mbar_init(bar_q, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_k_full[i], 1);
            mbar_init(&bar_k_empty[i], two ? 2 : 1);   // one commit per query tile
            mbar_init(&bar_v_full[i], 1);
            mbar_init(&bar_v_empty[i], two ? 2 : 1);
            mbar_init(&bar_s_full[i], 1);
            mbar_init(&bar_p_ready[i], 128);
            mbar_init(&bar_p_half[i], 128);
            mbar_init(&bar_o_done[i], 1);
        }
        mbar_init(&bar_done[0], 1);
        mbar_init(&bar_done[1], 1);
        *abort_flag = 0;
        burst_seq[0] = 0;
        burst_seq[1] = two ? 0 : INT_MAX;   // a lone tile never waits for its turn
        fence_barrier_init();
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // 384 threads x 168 registers at launch >= 128 x 64 (TMA, MMA, idle) + 256 x 216 (softmax)
    static_assert(128 * kFwdCtrlRegs + 256 * kFwdSoftmaxRegs <= kFwdThreads * kFwdLaunchRegs, "register split");
    if (warp < 4) {
        regs_release_to<kFwdCtrlRegs>();
        if (warp == 0) {
            // ===================== TMA producer =====================
            if (lane == 0) {
                const uint32_t qbytes = (two ? 2 : 1) * L::kTile;
                mbar_arrive_expect_tx(bar_q, qbytes);
                for (int t = 0; t < (two ? 2 : 1); ++t)
                    for (int c = 0; c < L::kPanels; ++c)
                        tma_load_3d(smem + L::kQ + t * L::kTile + c * kPanelBytes, &tm_q, bar_q, c * 64, h,
                                    seg0 + (2 * m + t) * 128);
                uint32_t kpar[2] = {0, 0}, vpar[2] = {0, 0};
                int kfill = 0, vfill = 0;   // loads issued (for the drain on abort)
                for (int j = 0; j < nkv; ++j) {
                    const int st = j & 1;
                    if (j >= 2 && !mbar_wait_or_abort(&bar_k_empty[st], ((j >> 1) - 1) & 1, 21, abort_flag)) break;
                    mbar_arrive_expect_tx(&bar_k_full[st], L::kTile);
                    for (int c = 0; c < L::kPanels; ++c)
                        tma_load_3d(smem + L::kK + st * L::kTile + c * kPanelBytes, &tm_k, &bar_k_full[st],
                                    c * 64, g, seg0 + kv_tile(j) * 128);
                    kpar[st] = (j >> 1) & 1;
                    ++kfill;
                    if (j >= 2 && !mbar_wait_or_abort(&bar_v_empty[st], ((j >> 1) - 1) & 1, 22, abort_flag)) break;
                    mbar_arrive_expect_tx(&bar_v_full[st], L::kTile);
                    for (int c = 0; c < L::kPanels; ++c)
                        tma_load_3d(smem + L::kV + st * L::kTile + c * kPanelBytes, &tm_v, &bar_v_full[st],
                                    c * 64, g, seg0 + kv_tile(j) * 128);
                    vpar[st] = (j >> 1) & 1;
                    ++vfill;
                }
                if (*abort_flag) {
                    // let this CTA's own copies land before the CTA exits (bounded)
                    mbar_wait(bar_q, 0, 23);
                    for (int st = 0; st < 2; ++st) {
                        if (kfill > st) mbar_wait(&bar_k_full[st], kpar[st], 23);
                        if (vfill > st) mbar_wait(&bar_v_full[st], vpar[st], 23);
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1 || warp == 2) {
            // ============ MMA issuers: warp 1 for query tile 0, warp 2 for tile 1 ============
            // The tensor pipe sees the bursts in the single-issuer order S0 S1 | PV0 S0' |
            // PV1 S1' | ..., so each tile's softmax overlaps the other tile's MMAs, but each
            // issuer clears its own barrier waits while the other one's burst runs.  A burst
            // waits for its turn on the other issuer's count of bursts issued.  The whole
            // warp runs this code (one elected lane issues); every wait result is made
            // warp-uniform.  Each commit tracks only the MMAs of the issuing lane.
            const int t = warp - 1;
            const int own_slots = t ? nkv1 : nkv0;
            const int nk = kMod && own_slots > 0 ? nkv : own_slots;   // steps this warp goes through
            if (nk > 0) {
                constexpr uint32_t kIdescS = idesc_bf16(128, 128, 0, 0);
                constexpr uint32_t kIdescO = idesc_bf16(128, D, 0, 1);
                const uint32_t qa = s_base + L::kQ + t * L::kTile;
                const uint32_t t_s = tmem + t * 128, t_o = tmem + 256 + t * 128;
                int nb = 0;   // bursts this warp has issued
                auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
                    return __all_sync(0xffffffffu, mbar_wait_or_abort(bar, parity, site, abort_flag));
                };
                auto my_turn = [&]() {
                    return __all_sync(0xffffffffu, spin_until_geq(&burst_seq[1 - t], nb + t, 19, abort_flag));
                };
                auto publish = [&](int v) {
                    __syncwarp();
                    if (lane == 0) burst_seq[t] = v;
                    __syncwarp();
                };
                auto issue_s = [&](int j) {
                    const uint32_t ka = s_base + L::kK + (j & 1) * L::kTile;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_bf16_ss_warp(t_s, desc_kmajor(qa, k), desc_kmajor(ka, k), kIdescS, k > 0);
                    mma_commit_warp(&bar_s_full[t]);
                    mma_commit_warp(&bar_k_empty[j & 1]);
                };
                // work: this tile computes in the current step (always in the plain kernel); ka
                // counts those steps, which its own barriers' phases follow, while the K/V
                // stages' phases follow the step itself
                const int idle_from = kMask ? (t ? runs1.np : runs0.np) : 0;
                const int idle_end = kMask ? (t ? runs1.idle_end(slots) : runs0.idle_end(slots)) : 0;
                auto has_work = [&](int step) {
                    const int i = nkv - 1 - step;   // the slot
                    return !kMod || (i < own_slots && (!kMask || i < idle_from || i >= idle_end));
                };
                bool work = has_work(0);
                bool ok = wait(bar_q, 0, 24) && (!work || wait(&bar_k_full[0], 0, 25)) && my_turn();
                if (ok) {
                    if (work) {
                        tc_fence_after();
                        issue_s(0);
                    }
                    publish(++nb);
                }
                int ka = 0;
                for (int j = 0; j < nk && ok; ++j) {
                    const int st = j & 1;
                    const bool next = j + 1 < nk && has_work(j + 1);
                    if (kMod && !work && !wait(&bar_k_full[st], (j >> 1) & 1, 25)) break;
                    if (!wait(&bar_v_full[st], (j >> 1) & 1, 26)) break;
                    if (next && !wait(&bar_k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, 28)) break;
                    if (work && !wait(&bar_p_half[t], ka & 1, 18)) break;
                    if (!my_turn()) break;
                    tc_fence_after();
                    if (work) {
                        // P.V over the first 64 keys while the softmax finishes the second half
                        const uint32_t va = s_base + L::kV + st * L::kTile;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ts_warp(t_o, t_s + k * 8, desc_mnmajor(va, k), kIdescO, (ka > 0 || k > 0) ? 1u : 0u);
                        if (!wait(&bar_p_ready[t], ka & 1, 27)) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 4; k < 8; ++k)
                            mma_bf16_ts_warp(t_o, t_s + k * 8, desc_mnmajor(va, k), kIdescO, 1u);
                        mma_commit_warp(&bar_o_done[t]);
                        mma_commit_warp(&bar_v_empty[st]);
                        ++ka;
                    } else {
                        mma_commit_warp(&bar_k_empty[st]);   // nothing of this tile reads the stages
                        mma_commit_warp(&bar_v_empty[st]);
                    }
                    if (next) issue_s(j + 1);
                    publish(++nb);
                    work = next;
                }
                publish(INT_MAX);   // finished (or aborted): never hold the other issuer
                mma_commit_warp(&bar_done[t]);
                // every MMA issued by this warp has finished (waits even after an abort)
                const bool drained = __all_sync(0xffffffffu, mbar_wait(&bar_done[t], 0, 29));
                if (kMod != 0 && !drained) *abort_flag = 1;
            }
        }
    } else {
        regs_grow_to<kFwdSoftmaxRegs>();
        // ============ softmax, one warpgroup per query tile (thread = row) ============
        const int t = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + t * 128 + lane_off;
        const uint32_t t_o = tmem + 256 + t * 128 + lane_off;
        const int nk = t ? nkv1 : nkv0;
        const int qt = 2 * m + t;
        const int q_local = qt * 128 + r;
        float m_ref = -INFINITY, l_run = 0.f;
        // kMod: the sum of P as rounded, which O is divided by.  P V with the rounded P over their
        // own sum is an average of V again, exactly V for a row that lies on one key; over the
        // exact sum it is off by that key's rounding, and so is D = <dO, O>, while dS = P (dP - D)
        // cancels: such rows got gradients as large as the rounding instead of none
        [[maybe_unused]] float l_rounded = 0.f;
        bool failed = false;
        int P_row = 0, from = 0;      // kMask: the prefix length, the row's first own key
        int all_prefix = 0, all_from = 0;   // keys that every row of the tile sees: below
                                            // all_prefix, and from all_from to the diagonal
        TileRuns runs{};
        if constexpr (kMask) {
            runs = t ? runs1 : runs0;
            P_row = P;
            all_prefix = prm.mod.prefix_causal ? min(P, qt * 128 + 1) : P;
            if (prm.mod.row_start && nk > 0) {
                const int32_t* rs = prm.mod.row_start + seg0;
                const int row = min(q_local, len - 1);
                from = rs[row];
                // starts lie in the row's own past and never decrease
                if (from < 0 || from > row || (row + 1 < len && rs[row + 1] < from)) {
                    report_error(16, kErrBadMask);
                    mirror_error();
                }
                from = min(max(from, 0), row);
                all_from = min(max(rs[min(qt * 128 + 127, len - 1)], 0), len - 1);
            }
        }
        // the row's index as its distances to prefix keys see it
        [[maybe_unused]] auto q_prefix = [&](bool check) {
            if constexpr (kPositions) {
                const int row = min(q_local, len - 1), given = prm.positions[seg0 + row];
                const int pos = bounded_position(given, row, P);
                if (check && pos != given) {
                    report_error(16, kErrBadMask);
                    mirror_error();
                }
                return pos + (q_local - row);
            } else {
                return q_local;
            }
        };
        if (kPositions && nk > 0) q_prefix(true);
        float bias2 = 0.f;   // per key of distance, in log2 units
        bool two_sided = false;
        if constexpr (kBias) {
            bias2 = prm.mod.slopes[h] * -1.4426950408889634f;
            two_sided = !prm.causal || (kMask && P > 0 && !prm.mod.prefix_causal);
        }
        // Capped scores lie in [-C, C], a bias with slope >= 0 only lowers them, and every row
        // sees its own key, which has none: the reference 0 will do, without a maximum and
        // without rescaling.  P then lies below 2^C and the row's sum above 2^-C, both far
        // inside fp32 and bf16 for C <= kBoundedCap; what falls out below is less than
        // 2^(C - 126) of the sum
        bool bounded = false;
        if constexpr (kCap) bounded = prm.mod.cap_out <= kBoundedCap && (!kBias || bias2 <= 0.f);
        const float grow = bounded ? INFINITY : kRescaleThreshold;
        if (bounded) m_ref = 0.f;
        // the bias of the columns within eight, by pairs
        float2 bias_in8[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) bias_in8[i] = make_float2(-bias2 * (2 * i), -bias2 * (2 * i + 1));
        int ka = 0;   // steps with work so far
        // the tile's KV tiles: all of them in ascending order; with modified scores in descending
        // order, under a mask those of its two runs
        for (int j = !kMod ? 0 : kMask && nk > 0 ? max(runs.np, runs.hi) - 1 : nk - 1; kMod ? j >= 0 : j < nk;
             j = kMask ? runs.next(j) : kMod ? j - 1 : j + 1) {
            // where the tile's distances are counted from (read anew for each tile: a register
            // held across the steps spilled); at the prefix's end that holds for its keys below P
            int q_dist = q_local;
            bool prefix_end = false;
            if (kPositions && j * 128 < P) {
                q_dist = q_prefix(false);
                prefix_end = j * 128 + 128 > P;
            }
            const bool got = mbar_wait_or_abort(&bar_s_full[t], ka & 1, 30, abort_flag);
            if (!__all_sync(0xffffffffu, got)) { failed = true; break; }
            tc_fence_after();
            const int kv0 = j * 128;
            const bool diag = !kMask && prm.causal && j == qt;
            const bool tail = !kMask && kv0 + 128 > len;
            // every row of the tile sees every key of the step
            const bool whole = kMask ? kv0 + 128 <= all_prefix || (kv0 >= all_from && j < qt) : !(diag || tail);
            // the row's visible keys of the tile (a padding row takes the last row's)
            RowView view{0, -kv0, static_cast<unsigned>(len - 1)};
            if constexpr (kMask) {
                const int row = min(q_local, len - 1);
                view.pre = (prm.mod.prefix_causal ? min(P_row, row + 1) : P_row) - kv0;
                view.first = from - kv0;
                view.own = row - from;
            } else if (diag) {
                view.own = min(q_local, len - 1);
            }
            if constexpr (kCap) {
                if (bounded && !(kBias && two_sided && j >= qt) && !prefix_end) {
                    // a tile under a cap: no maximum, no reference, and so the row is taken in
                    // chunks of 32 columns as they arrive
                    const float dist_bias = static_cast<float>(q_dist - kv0) * bias2;
                    const RowSums sums =
                        whole ? capped_row<kBias, false>(prm.mod, t_s, dist_bias, bias2, bias_in8, view, &bar_p_half[t])
                              : capped_row<kBias, true>(prm.mod, t_s, dist_bias, bias2, bias_in8, view, &bar_p_half[t]);
                    l_run += sums.exact;
                    l_rounded += sums.rounded;
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&bar_p_ready[t]);
                    ++ka;
                    continue;
                }
            }
            // the row's 128 score columns: eight loads in flight, one wait
            float sv[128];
            {
                uint32_t sr[8][16];
#pragma unroll
                for (int c = 0; c < 8; ++c) tmem_ld16_nowait(t_s + c * 16, sr[c]);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    tmem_regs_ready(sr[c]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) sv[c * 16 + e] = __uint_as_float(sr[c][e]);
                }
            }
            // fused: the bias is part of the exponents below, so that it runs in the shadow of the
            // exp2 unit.  The maximum of the raw scores plus the largest bias bounds the scores
            // from above; a tile for which the bound stays near the row's reference (which the
            // tiles before, nearer ones, have set) needs neither its own maximum nor another
            // reference: P <= 2^kFusedAbove is as exact as P <= 1
            bool fused = false;
            if constexpr (kBias && !kCap) {
                if (whole && !(two_sided && j >= qt) && !prefix_end && ka > 0) {
                    const float nearest = static_cast<float>(q_dist - kv0 - (bias2 <= 0.f ? 127 : 0));
                    const float bound = fmaf(nearest, bias2, row_max(sv) * prm.scale_log2);
                    fused = !__any_sync(0xffffffffu, !(bound <= m_ref + kFusedAbove));
                }
            }
            float mx = m_ref;
            if (!fused) {
                // raw scores are scaled in the exponent's FMA; capped ones come scaled
                const float to_log2 = kCap ? 1.f : prm.scale_log2;
                if constexpr (kCap) cap_scores(prm.mod, sv);
                if constexpr (kBias) {
                    // the distances t - u are exact in fp32 (below 2^24; relative to that beyond)
                    const float base = static_cast<float>(q_dist - kv0);
                    const float bias = kCap ? bias2 : bias2 / prm.scale_log2;
                    if ((two_sided && j >= qt) || prefix_end) {
                        const float own = static_cast<float>(q_local - kv0);
#pragma unroll
                        for (int e = 0; e < 128; ++e)
                            sv[e] = fmaf(fabsf((kPositions && kv0 + e >= P ? own : base) - e), bias, sv[e]);
                    } else {
                        const float2 b2 = make_float2(base, base), s2 = make_float2(bias, bias);
#pragma unroll
                        for (int e = 0; e < 128; e += 2) {
                            const float2 x = f2_fma(f2_add(b2, make_float2(-e, -e - 1)), s2, make_float2(sv[e], sv[e + 1]));
                            sv[e] = x.x;
                            sv[e + 1] = x.y;
                        }
                    }
                }
                if constexpr (kMod != 0) {
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 128; ++e) sv[e] = view.sees(e) ? sv[e] : -INFINITY;
                    }
                } else if (diag || tail) {
#pragma unroll
                    for (int e = 0; e < 128; ++e) {
                        const int kv = kv0 + e;
                        const bool valid = !(diag && kv > q_local) && kv < len;
                        sv[e] = valid ? sv[e] : -INFINITY;
                    }
                }
                // row maximum of the raw scores; the scale is positive, so scaling the maximum
                // gives the scaled maximum
                mx = row_max(sv) * to_log2;
            }
            // stale-max rule: keep the old reference unless the row maximum grew a lot
            float alpha = 1.f;
            bool rescale = false;
            if (ka == 0 && !bounded) {
                m_ref = mx;
            } else if (mx > m_ref + grow) {
                alpha = fast_exp2(m_ref - mx);
                m_ref = mx;
                rescale = true;
            }
            if (!fused && __any_sync(0xffffffffu, rescale)) {
                // O_t must hold the previous P.V product before it is rescaled (it does: S
                // of this step completed after it); no P.V of this step has started yet
                const bool got_o = mbar_wait_or_abort(&bar_o_done[t], (ka - 1) & 1, 31, abort_flag);
                if (!__all_sync(0xffffffffu, got_o)) { failed = true; break; }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float ov[32];
                    tmem_ld32(t_o + c * 32, ov);
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] *= alpha;
                    tmem_st32(t_o + c * 32, ov);
                }
            }
            // P = 2^(scale * S - m_ref), in four chunks of 32 columns, software-pipelined:
            // the exponentials of chunk c+1 are issued ahead of the row sums, the bf16
            // packing and the TMEM store of chunk c, so that one warp keeps the MUFU busy
            const float neg_m = -m_ref;
            // (scale and subtract, and the row sums, in packed pairs)
            const float to_log2 = kCap ? 1.f : prm.scale_log2;
            const float2 sc2 = make_float2(to_log2, to_log2);
            const float2 nm2 = make_float2(neg_m, neg_m);
            const float fused_base = kBias ? fmaf(static_cast<float>(q_dist - kv0), bias2, neg_m) : neg_m;
            auto exps = [&](int c, float (&p)[32], auto fuse) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 s2 = make_float2(sv[c * 32 + e], sv[c * 32 + e + 1]);
                    float2 x;
                    if constexpr (decltype(fuse)::value) {
                        float2 off = make_float2(fused_base, fused_base);
                        {
                            const float at = fmaf(static_cast<float>(-(c * 32 + e) / 8 * 8), bias2, fused_base);
                            off = f2_add(make_float2(at, at), bias_in8[(e % 8) / 2]);
                        }
                        x = f2_fma(s2, sc2, off);
                    } else {
                        x = f2_fma(s2, sc2, nm2);
                    }
                    p[e] = fast_exp2(x.x);
                    p[e + 1] = fast_exp2(x.y);
                }
            };
            float2 rsA = make_float2(0.f, 0.f), rsB = make_float2(0.f, 0.f);
            [[maybe_unused]] float2 roundedA = rsA, roundedB = rsA;
            auto finish = [&](int c, const float (&p)[32]) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (e & 1)
                        rsB = f2_add(rsB, make_float2(p[2 * e], p[2 * e + 1]));
                    else
                        rsA = f2_add(rsA, make_float2(p[2 * e], p[2 * e + 1]));
                    pk[e] = pack_bf16(p[2 * e], p[2 * e + 1]);
                    if constexpr (kMod != 0) add_packed((e & 1) ? roundedB : roundedA, pk[e]);
                }
                tmem_st16(t_s + c * 16, pk);   // P (packed) over S columns already read
            };
            auto probabilities = [&](auto fuse) {
                float pa[32], pb[32];
                exps(0, pa, fuse);
                exps(1, pb, fuse);
                finish(0, pa);
                exps(2, pa, fuse);
                finish(1, pb);
                // the first half of P (columns [0, 64), K = 0..63 of P.V) is in TMEM
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bar_p_half[t]);
                exps(3, pb, fuse);
                finish(2, pa);
                finish(3, pb);
            };
            if constexpr (kBias && !kCap) {
                if (fused) probabilities(std::true_type{});
                else probabilities(std::false_type{});
            } else {
                probabilities(std::false_type{});
            }
            const float rs_all = (rsA.x + rsA.y) + (rsB.x + rsB.y);
            l_run = l_run * alpha + rs_all;
            if constexpr (kMod != 0)
                l_rounded = l_rounded * alpha + ((roundedA.x + roundedA.y) + (roundedB.x + roundedB.y));
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bar_p_ready[t]);
            ++ka;
        }
        // ---- epilogue: O / l -> bf16, LSE ----
        bool have = !failed && nk > 0 && !*abort_flag;
        if (have) have = mbar_wait_or_abort(&bar_o_done[t], (ka - 1) & 1, 32, abort_flag);
        have = __all_sync(0xffffffffu, have);
        if (have) {
            tc_fence_after();
            const bool row_ok = q_local < len;
            const float inv_l = 1.f / (kMod ? l_rounded : l_run);
            const int tok = seg0 + q_local;
            __nv_bfloat16* orow = prm.o + ((size_t)tok * prm.hq + h) * D;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float ov[32];
                tmem_ld32(t_o + c * 32, ov);
                if (row_ok) {
#pragma unroll
                    for (int e8 = 0; e8 < 4; ++e8) {
                        uint4 pk;
                        pk.x = pack_bf16(ov[e8 * 8 + 0] * inv_l, ov[e8 * 8 + 1] * inv_l);
                        pk.y = pack_bf16(ov[e8 * 8 + 2] * inv_l, ov[e8 * 8 + 3] * inv_l);
                        pk.z = pack_bf16(ov[e8 * 8 + 4] * inv_l, ov[e8 * 8 + 5] * inv_l);
                        pk.w = pack_bf16(ov[e8 * 8 + 6] * inv_l, ov[e8 * 8 + 7] * inv_l);
                        *reinterpret_cast<uint4*>(orow + c * 32 + e8 * 8) = pk;
                        if constexpr (kMod != 0) {
                            if (prm.o_low) {
                                const uint32_t hi[4] = {pk.x, pk.y, pk.z, pk.w};
                                uint32_t low[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    low[i] = pack_bf16(fmaf(ov[e8 * 8 + 2 * i], inv_l, -__uint_as_float(hi[i] << 16)),
                                                       fmaf(ov[e8 * 8 + 2 * i + 1], inv_l,
                                                            -__uint_as_float(hi[i] & 0xffff0000u)));
                                *reinterpret_cast<uint4*>(prm.o_low + (orow - prm.o) + c * 32 + e8 * 8) =
                                    make_uint4(low[0], low[1], low[2], low[3]);
                            }
                        }
                    }
                }
            }
            if (row_ok)
                prm.lse[(size_t)h * prm.T + tok] = (m_ref + __log2f(l_run)) * 0.69314718055994531f;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (kMod != 0 && tid == 0 && *abort_flag) mirror_error();   // no mirroring kernel follows
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace lf
