// Host side of the LazyFlash C ABI (include/lazyflash.h): argument checks,
// workspace sizing, TMA tensor-map encoding and kernel launches.  Nothing
// here computes attention; every step of the path runs in the kernels of
// lf_fwd.cuh, lf_select.cuh, lf_bwd.cuh and lf_qknorm.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>
#include <mutex>
#include <type_traits>

#include "lazyflash.h"
#include "lf_bwd.cuh"
#include "lf_device.cuh"
#include "lf_fwd.cuh"
#include "lf_qknorm.cuh"
#include "lf_select.cuh"

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

lf_status check_desc(const lf_attn_desc* d) {
    if (!d) return LF_ERR_INVALID_ARG;
    if (d->nseq < 1 || !d->cu_seqlens || d->total_tokens < 0 || d->max_seqlen < 0)
        return LF_ERR_INVALID_ARG;
    if (d->hq < 1 || d->hkv < 1 || d->hq % d->hkv != 0) return LF_ERR_INVALID_ARG;
    if (d->hq > 65535 || d->hkv > 65535) return LF_ERR_UNSUPPORTED;
    if (!(d->softmax_scale > 0.f) || !std::isfinite(d->softmax_scale)) return LF_ERR_INVALID_ARG;
    if (d->causal != 0 && d->causal != 1) return LF_ERR_INVALID_ARG;
    if (d->d != 64 && d->d != 128) return LF_ERR_UNSUPPORTED;
    if (d->block_q != 64 && d->block_q != 128) return LF_ERR_UNSUPPORTED;
    if (d->nseq > 65535) return LF_ERR_UNSUPPORTED;
    // element offsets are computed in 64 bits; row indices in 32 bits
    if ((int64_t)d->total_tokens * d->hq > (int64_t)1 << 31) return LF_ERR_UNSUPPORTED;
    return LF_OK;
}

inline int nbmax_of(const lf_attn_desc* d) { return (d->max_seqlen + d->block_q - 1) / d->block_q; }
inline int ntiles_of(const lf_attn_desc* d) { return (d->max_seqlen + 127) / 128; }

// Backward workspace: fp32 accumulators dQ [hq][T][d] (head-major), dK and dV
// [T][hkv][d]
// (one contiguous, 256-byte aligned block, cleared by one memset), then D
// [hq][T] when the caller does not pass it.
struct BwdWs {
    size_t dq, dk, dv, acc_end, D, total;
};
inline size_t al256(size_t b) { return (b + 255) & ~size_t(255); }
BwdWs bwd_ws_layout(const lf_attn_desc* d, bool need_D) {
    BwdWs w{};
    w.dq = 0;
    w.dk = al256((size_t)d->total_tokens * d->hq * d->d * sizeof(float));
    w.dv = w.dk + al256((size_t)d->total_tokens * d->hkv * d->d * sizeof(float));
    w.acc_end = w.dv + al256((size_t)d->total_tokens * d->hkv * d->d * sizeof(float));
    w.D = w.acc_end;
    w.total = w.acc_end + (need_D ? al256((size_t)d->total_tokens * d->hq * sizeof(float)) : 0);
    return w;
}
size_t bwd_ws_bytes(const lf_attn_desc* d, bool need_D) { return bwd_ws_layout(d, need_D).total; }
// ... then, for modified scores with row_start, a row index per key
size_t key_last_offset(const lf_attn_desc* d) { return bwd_ws_bytes(d, true); }
size_t bwd_ws_bytes_mod(const lf_attn_desc* d) {
    return key_last_offset(d) + al256((size_t)d->total_tokens * sizeof(int32_t));
}

// [T][H][d] bf16 -> 3-D map (d, H, T), 64 x 1 x `rows` boxes, 128-byte swizzle.
bool make_thd_map(CUtensorMap* m, const void* base, int T, int H, int D, int rows = 128) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [T][H][d] fp32 accumulator -> 3-D map (d, H, T), 32 x 1 x 128 boxes (128 bytes of a
// row each), 128-byte swizzle: the layout the backward stages its dK/dV tiles in.
bool make_acc_map(CUtensorMap* m, float* base, int T, int H, int D) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 4, (cuuint64_t)H * D * 4};
    const cuuint32_t box[3] = {32, 1, 128};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline lf_status launch_status() {
    return cudaGetLastError() == cudaSuccess ? LF_OK : LF_ERR_CUDA;
}

lf_status check_mod(const lf_attn_desc* d, const lf_score_mod* m) {
    if (!m) return LF_ERR_INVALID_ARG;
    if (m->softcap != 0.f && !(m->softcap >= 1e-3f && m->softcap <= 1e6f)) return LF_ERR_INVALID_ARG;
    // read value by value: slices of longer arrays are fine
    for (const void* p : {static_cast<const void*>(m->alibi_slopes), static_cast<const void*>(m->prefix_len),
                          static_cast<const void*>(m->row_start), static_cast<const void*>(m->positions)})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return LF_ERR_INVALID_ARG;
    if (m->prefix_causal != 0 && m->prefix_causal != 1) return LF_ERR_INVALID_ARG;
    if (m->prefix_causal && !m->prefix_len) return LF_ERR_INVALID_ARG;
    if (m->positions && !m->prefix_len) return LF_ERR_INVALID_ARG;
    if (m->positions && !m->prefix_causal) return LF_ERR_UNSUPPORTED;   // a prefix's own rows see later keys
    // the masks say which keys a causal row sees besides, or no longer
    if ((m->prefix_len || m->row_start) && !d->causal) return LF_ERR_UNSUPPORTED;
    return LF_OK;
}

// The kernels' variant for a modifier, and its parameters.
int mod_variant(const lf_score_mod* m) {
    return !m ? 0 : (m->softcap != 0.f ? lf::kModCap : 0) | (m->alibi_slopes ? lf::kModBias : 0) |
                        (m->prefix_len || m->row_start ? lf::kModMask : 0) |
                        (m->alibi_slopes && m->positions ? lf::kModPositions : 0);
}
lf::ModParams mod_params(const lf_attn_desc* d, const lf_score_mod* m) {
    lf::ModParams p{};
    if (!m) return p;
    if (m->softcap != 0.f) {
        const double c = m->softcap * 1.4426950408889634;
        p.cap_in = static_cast<float>((double)d->softmax_scale / m->softcap);
        p.cap_out = static_cast<float>(c);
        p.cap_damp = static_cast<float>(-1.0 / (c * c));
        for (int i = 0; i < lf::kCapTerms; ++i) p.cap_coef[i] = static_cast<float>(c * lf::kCapCoef[i]);
        const double a = (double)d->softmax_scale / m->softcap;
        const bool fits = a >= 3e-4 && a <= 1e3;   // every C a^(2k+1) is a normal number
        for (int i = 0; i < lf::kCapFusedTerms; ++i)
            p.cap_fused[i] = fits ? static_cast<float>(c * lf::kCapFused[i] * std::pow(a, 2 * i + 1)) : 0.f;
        p.fused_max = fits ? static_cast<float>(lf::kCapFusedRange / a) : 0.f;
    }
    p.slopes = m->alibi_slopes;
    p.prefix = m->prefix_len;
    p.prefix_causal = m->prefix_causal;
    p.row_start = m->row_start;
    return p;
}

template <int D, int kMod>
lf_status launch_fwd(const lf_attn_desc* d, const lf_score_mod* mod, const void* q, const void* k,
                     const void* v, void* o, void* o_low, float* lse, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    if (!make_thd_map(&mq, q, d->total_tokens, d->hq, D) ||
        !make_thd_map(&mk, k, d->total_tokens, d->hkv, D) ||
        !make_thd_map(&mv, v, d->total_tokens, d->hkv, D))
        return LF_ERR_CUDA;
    lf::FwdParamsOf<kMod> p{};
    p.cu_seqlens = d->cu_seqlens;
    p.T = d->total_tokens;
    p.hq = d->hq;
    p.hkv = d->hkv;
    p.causal = d->causal;
    p.max_seqlen = d->max_seqlen;
    p.nseq = d->nseq;
    p.scale_log2 = d->softmax_scale * 1.4426950408889634f;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    if constexpr (kMod != 0) {
        p.mod = mod_params(d, mod);
        p.o_low = static_cast<__nv_bfloat16*>(o_low);
    }
    if constexpr ((kMod & lf::kModPositions) != 0) p.positions = mod->positions;
    const uint32_t smem = lf::FwdSmem<D>::kAlloc;
    if (cudaFuncSetAttribute(lf::attn_fwd_kernel<D, kMod>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess)
        return LF_ERR_CUDA;
    // The kernel's warpgroups resize their register budgets (setmaxnreg); the larger
    // budget can only be granted from the registers the block was launched with, so a
    // build that launches with fewer than the budgets add up to must not run (its
    // softmax warps would wait for registers that never come).
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, lf::attn_fwd_kernel<D, kMod>) != cudaSuccess) return LF_ERR_CUDA;
    const int launch_regs = (fa.numRegs + 7) / 8 * 8;
    if (launch_regs * lf::kFwdThreads < 128 * lf::kFwdCtrlRegs + 256 * lf::kFwdSoftmaxRegs)
        return LF_ERR_UNSUPPORTED;
    // one CTA per pair of query tiles; the query heads of one KV head together, their
    // longest pairs first within each segment (x = pair rank * group + head in group,
    // y = KV head)
    // (x: pairs of query tiles over all segments, flattened; see segment_of_unit)
    const long long pair_units = ((long long)d->total_tokens + 255ll * d->nseq) >> 8;
    dim3 grid(static_cast<unsigned>(pair_units * (d->hq / d->hkv)), d->hkv, 1);
    // up to eight waves: every KV head's longest rows first (the whole grid's K/V then
    // shares L2, which is small at these lengths)
    int dev = 0, nsm = 148;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return LF_ERR_CUDA;
    p.tile_major = (long long)grid.x * grid.y <= 8LL * nsm ? 1 : 0;
    lf::attn_fwd_kernel<D, kMod><<<grid, lf::kFwdThreads, smem, st>>>(mq, mk, mv, p);
    return launch_status();
}

template <int D>
lf_status launch_norms(const lf_attn_desc* d, const void* dout, const void* o, float* norms,
                       float* Dv, int write_norms, cudaStream_t st) {
    dim3 grid(nbmax_of(d), d->hq, d->nseq);
    lf::norms_rowdot_kernel<D><<<grid, lf::kNormThreads, 0, st>>>(
        d->cu_seqlens, d->total_tokens, d->max_seqlen, d->hq, d->block_q, nbmax_of(d),
        static_cast<const __nv_bfloat16*>(dout), static_cast<const __nv_bfloat16*>(o), norms, Dv,
        write_norms);
    return launch_status();
}

// The backward: prologue over kept blocks (dQ accumulator rows zeroed; D computed into
// the workspace when the caller passed none), attn_bwd_kernel, dQ conversion.
// key_last: scratch of a modifier with row_start.
template <int D, int kMod>
lf_status launch_bwd(const lf_attn_desc* d, const lf_score_mod* mod, int32_t* key_last, const void* o_low,
                     const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout, const float* Dgiven,
                     const float* w, const int32_t* kidx, const int32_t* kcnt, void* dq, void* dk,
                     void* dv, void* ws, cudaStream_t st) {
    // Q and dO also in 64-row boxes: a query tile with one live half loads only that half
    CUtensorMap mq, mk, mv, mdo, mq64, mdo64;
    if (!make_thd_map(&mq, q, d->total_tokens, d->hq, D) ||
        !make_thd_map(&mk, k, d->total_tokens, d->hkv, D) ||
        !make_thd_map(&mv, v, d->total_tokens, d->hkv, D) ||
        !make_thd_map(&mdo, dout, d->total_tokens, d->hq, D) ||
        !make_thd_map(&mq64, q, d->total_tokens, d->hq, D, 64) ||
        !make_thd_map(&mdo64, dout, d->total_tokens, d->hq, D, 64))
        return LF_ERR_CUDA;
    const BwdWs lay = bwd_ws_layout(d, false);
    uint8_t* base = static_cast<uint8_t*>(ws);
    float* dq_acc = reinterpret_cast<float*>(base + lay.dq);
    float* dk_acc = reinterpret_cast<float*>(base + lay.dk);
    float* dv_acc = reinterpret_cast<float*>(base + lay.dv);
    CUtensorMap mdvacc, mdkacc;
    if (!make_acc_map(&mdvacc, dv_acc, d->total_tokens, d->hkv, D) ||
        !make_acc_map(&mdkacc, dk_acc, d->total_tokens, d->hkv, D))
        return LF_ERR_CUDA;
    // one CTA per KV tile walks the whole query group of its KV head (up to
    // kMaxHeadsPerCta heads): dK/dV are then final in TMEM and go straight to the bf16
    // outputs, with no atomics; a larger group is split over CTAs (the largest divisor
    // of the group within the limit) whose dK/dV tiles meet in fp32 accumulators
    const int group = d->hq / d->hkv;
    int heads_per_cta = group;
    while (heads_per_cta > lf::kMaxHeadsPerCta || group % heads_per_cta != 0) --heads_per_cta;
    const bool kv_direct = heads_per_cta == group;
    // the outputs (direct) or the dK/dV accumulators zeroed whole: rows no CTA writes
    // (no kept block reaches them, or outside every segment) read as 0; the dQ
    // accumulator is zeroed only in the rows of kept blocks
    const size_t nkv = (size_t)d->total_tokens * d->hkv * D;
    if (kv_direct) {
        if (cudaMemsetAsync(dk, 0, nkv * 2, st) != cudaSuccess ||
            cudaMemsetAsync(dv, 0, nkv * 2, st) != cudaSuccess)
            return LF_ERR_CUDA;
    } else if (cudaMemsetAsync(base + lay.dk, 0, lay.acc_end - lay.dk, st) != cudaSuccess) {
        return LF_ERR_CUDA;
    }
    const dim3 blocks(nbmax_of(d), d->hq, d->nseq);
    float* Dw = Dgiven ? nullptr : reinterpret_cast<float*>(base + bwd_ws_layout(d, true).D);
    lf::bwd_prologue_kernel<D, kMod != 0><<<blocks, lf::kNormThreads, 0, st>>>(
        d->cu_seqlens, d->total_tokens, d->max_seqlen, d->hq, d->block_q, nbmax_of(d), w, dq_acc,
        static_cast<const __nv_bfloat16*>(dout), static_cast<const __nv_bfloat16*>(o), Dw,
        static_cast<const __nv_bfloat16*>(o_low), mod ? mod->row_start : nullptr, key_last);
    if (launch_status() != LF_OK) return LF_ERR_CUDA;
    const float* Dv = Dgiven ? Dgiven : Dw;
    lf::BwdParamsOf<kMod> p{};
    p.cu_seqlens = d->cu_seqlens;
    p.T = d->total_tokens;
    p.hq = d->hq;
    p.hkv = d->hkv;
    p.causal = d->causal;
    p.block_q = d->block_q;
    p.nbmax = nbmax_of(d);
    p.max_seqlen = d->max_seqlen;
    p.heads_per_cta = heads_per_cta;
    p.kv_out_direct = kv_direct ? 1 : 0;
    p.dk_out = static_cast<__nv_bfloat16*>(dk);
    p.dv_out = static_cast<__nv_bfloat16*>(dv);
    p.scale = d->softmax_scale;
    p.scale_log2 = d->softmax_scale * 1.4426950408889634f;
    p.lse = lse;
    p.Dvec = Dv;
    p.block_weight = w;
    p.kept_idx = kidx;
    p.kept_cnt = kcnt;
    p.dq_acc = dq_acc;
    if constexpr (kMod != 0) {
        p.mod = mod_params(d, mod);
        p.key_last = key_last;
    }
    if constexpr ((kMod & lf::kModPositions) != 0) p.positions = mod->positions;
    const uint32_t smem =
        (kMod & lf::kModPositions) != 0 ? lf::BwdSmem<D>::kAllocPositions : lf::BwdSmem<D>::kAlloc;
    // 64-row selection blocks: the variant that skips a tile's dropped half
    auto kern = d->block_q == 64 ? lf::attn_bwd_kernel<D, true, kMod> : lf::attn_bwd_kernel<D, false, kMod>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return LF_ERR_CUDA;
    dim3 grid(ntiles_of(d), d->hq / p.heads_per_cta, d->nseq);
    // up to eight waves of CTAs per segment (16K tokens at 8 KV heads): every head
    // group's heavy tiles first; longer segments run one group at a time, which keeps
    // the group's Q, dO and dQ accumulator in L2 (the other order was slower at 32K)
    int dev = 0, nsm = 148;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return LF_ERR_CUDA;
    p.tile_major = (long long)grid.x * grid.y <= 8LL * nsm ? 1 : 0;
    kern<<<grid, lf::kBwdThreads, smem, st>>>(mq, mk, mv, mdo, mdvacc, mdkacc, mq64, mdo64, p);
    if (launch_status() != LF_OK) return LF_ERR_CUDA;
    // fp32 accumulators -> bf16 results (dQ and dK take the softmax scale)
    const size_t nkv8 = (size_t)d->total_tokens * d->hkv * D / 8;
    const int bkv = (int)std::min<size_t>((nkv8 + 255) / 256, 148 * 16);
    lf::dq_acc_to_thd_kept_kernel<D><<<blocks, 256, 0, st>>>(d->cu_seqlens, d->total_tokens, d->max_seqlen,
                                                             d->hq, d->block_q, nbmax_of(d), w, dq_acc,
                                                             static_cast<uint4*>(dq), d->softmax_scale);
    if (!kv_direct) {
        lf::dq_convert_kernel<<<bkv, 256, 0, st>>>(reinterpret_cast<const float4*>(dk_acc),
                                                   static_cast<uint4*>(dk), nkv8, d->softmax_scale);
        lf::dq_convert_kernel<<<bkv, 256, 0, st>>>(reinterpret_cast<const float4*>(dv_acc),
                                                   static_cast<uint4*>(dv), nkv8, 1.0f);
    }
    return launch_status();
}

// f(head dim, variant of the modified scores) as compile-time constants.
template <typename F>
lf_status by_variant(const lf_attn_desc* d, const lf_score_mod* mod, F&& f) {
    auto by_d = [&](auto v) {
        return d->d == 128 ? f(std::integral_constant<int, 128>{}, v) : f(std::integral_constant<int, 64>{}, v);
    };
    switch (mod_variant(mod)) {
        case 0: return by_d(std::integral_constant<int, 0>{});
        case 1: return by_d(std::integral_constant<int, 1>{});
        case 2: return by_d(std::integral_constant<int, 2>{});
        case 3: return by_d(std::integral_constant<int, 3>{});
        case 4: return by_d(std::integral_constant<int, 4>{});
        case 5: return by_d(std::integral_constant<int, 5>{});
        case 6: return by_d(std::integral_constant<int, 6>{});
        case 7: return by_d(std::integral_constant<int, 7>{});
        case 14: return by_d(std::integral_constant<int, 14>{});   // positions come with bias and mask
        default: return by_d(std::integral_constant<int, 15>{});
    }
}
lf_status launch_fwd_any(const lf_attn_desc* d, const lf_score_mod* mod, const void* q, const void* k,
                         const void* v, void* o, void* o_low, float* lse, cudaStream_t st) {
    return by_variant(d, mod, [&](auto D, auto M) {
        return launch_fwd<decltype(D)::value, decltype(M)::value>(d, mod, q, k, v, o, o_low, lse, st);
    });
}
lf_status launch_bwd_any(const lf_attn_desc* d, const lf_score_mod* mod, int32_t* key_last, const void* o_low,
                         const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                         const float* Dgiven, const float* w, const int32_t* kidx, const int32_t* kcnt, void* dq,
                         void* dk, void* dv, void* ws, cudaStream_t st) {
    return by_variant(d, mod, [&](auto D, auto M) {
        return launch_bwd<decltype(D)::value, decltype(M)::value>(d, mod, key_last, o_low, q, k, v, o, lse, dout,
                                                                  Dgiven, w, kidx, kcnt, dq, dk, dv, ws, st);
    });
}

lf_status check_qk_desc(const lf_qk_desc* d) {
    if (!d) return LF_ERR_INVALID_ARG;
    if (d->total_tokens < 0 || d->hq < 1 || d->hkv < 1 || d->rot < 0) return LF_ERR_INVALID_ARG;
    if (d->d != 64 && d->d != 128) return LF_ERR_UNSUPPORTED;
    if (d->hq > 65535 || d->hkv > 65535) return LF_ERR_UNSUPPORTED;
    if (d->cu_seqlens && d->nseq < 1) return LF_ERR_INVALID_ARG;
    if (d->rot > d->d) return LF_ERR_INVALID_ARG;
    if (d->rot % 16 != 0) return LF_ERR_UNSUPPORTED;
    if (d->rot > 0 && (!d->cos_sin || d->npos < 1 || (!d->positions && !d->cu_seqlens)))
        return LF_ERR_INVALID_ARG;
    if (d->pairing != LF_ROPE_HALVES && d->pairing != LF_ROPE_PAIRS) return LF_ERR_INVALID_ARG;
    if (d->flags & ~(LF_QK_NORM | LF_QK_ZERO_TAIL)) return LF_ERR_INVALID_ARG;
    if (d->flags & LF_QK_NORM) {
        if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return LF_ERR_INVALID_ARG;
        if (d->weights_bf16 != 0 && d->weights_bf16 != 1) return LF_ERR_INVALID_ARG;
        if (!aligned16(d->q_weight) || !aligned16(d->k_weight)) return LF_ERR_INVALID_ARG;
    } else if (d->q_weight || d->k_weight || d->rot == 0) {
        return LF_ERR_INVALID_ARG;   // weights without the norm; or nothing to do
    }
    if (!aligned16(d->cos_sin)) return LF_ERR_INVALID_ARG;
    return LF_OK;
}

// A strided [T][heads][d] bf16 operand.
bool qk_operand_ok(const lf_qk_desc* d, const void* p, int64_t stride, int heads) {
    return p && aligned16(p) && stride % 8 == 0 && stride >= (int64_t)heads * d->d;
}

lf::QkParams qk_params(const lf_qk_desc* d) {
    lf::QkParams p{};
    p.T = d->total_tokens;
    p.hq = d->hq;
    p.hkv = d->hkv;
    p.nseq = d->nseq;
    p.npos = d->npos;
    p.rot = d->rot;
    p.weights_bf16 = d->weights_bf16;
    p.zero_tail = (d->flags & LF_QK_ZERO_TAIL) ? 1 : 0;
    p.cu = d->cu_seqlens;
    p.positions = d->positions;
    p.cos_sin = d->cos_sin;
    p.eps = d->eps;
    p.qw = d->q_weight;
    p.kw = d->k_weight;
    return p;
}

// The grid over units of row groups (see lf_qknorm.cuh).  A warp takes a token's whole
// list of row groups once there are tokens enough to give every SM 16 warps; with fewer
// tokens the list is cut so that the warps of the whole GPU share it.  Returns the blocks.
int qk_grid(const lf_qk_desc* d, lf::QkParams& p, bool bwd) {
    const int rpw = 32 / (d->d / 8);
    const int ng = (d->hq + rpw - 1) / rpw + (d->hkv + rpw - 1) / rpw;
    const long long cut = std::min<long long>(ng, (148ll * 16 + p.T - 1) / p.T);
    p.per_unit = static_cast<int>((ng + cut - 1) / cut);
    p.units_per_token = (ng + p.per_unit - 1) / p.per_unit;
    const long long units = (long long)p.T * p.units_per_token;
    return static_cast<int>(
        std::min<long long>((units + 7) / 8, 148 * (bwd ? lf::kQkBlocksBwd : lf::kQkBlocksFwd)));
}

template <int D, bool kNorm, bool kPairs>
lf_status launch_qk(const lf::QkParams& p, int blocks, bool bwd, cudaStream_t st) {
    if (bwd)
        lf::qk_norm_rope_kernel<D, kNorm, kPairs, true><<<blocks, lf::kQkThreads, 0, st>>>(p);
    else
        lf::qk_norm_rope_kernel<D, kNorm, kPairs, false><<<blocks, lf::kQkThreads, 0, st>>>(p);
    return launch_status();
}

lf_status launch_qk_any(const lf_qk_desc* d, const lf::QkParams& p, int blocks, bool bwd,
                        cudaStream_t st) {
    const bool norm = (d->flags & LF_QK_NORM) != 0, pairs = d->pairing == LF_ROPE_PAIRS;
    auto by_d = [&](auto n, auto pr) {
        constexpr bool N = decltype(n)::value, P = decltype(pr)::value;
        return d->d == 128 ? launch_qk<128, N, P>(p, blocks, bwd, st)
                           : launch_qk<64, N, P>(p, blocks, bwd, st);
    };
    if (norm) return pairs ? by_d(std::true_type{}, std::true_type{}) : by_d(std::true_type{}, std::false_type{});
    return pairs ? by_d(std::false_type{}, std::true_type{}) : by_d(std::false_type{}, std::false_type{});
}

}  // namespace

namespace lf {
// Failure-detection self-test: one thread waits, with the kernels' bounded wait,
// on a barrier phase that nothing completes.  The wait gives up after `limit`
// cycles and records a timeout in the device flag; nothing faults or traps.
__global__ void watchdog_selftest_kernel(long long limit) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) (void)mbar_wait(&bar, 0, 99, limit);
    __syncthreads();
}
// Enqueued at the end of every call that launches kernels: copies the failure flag,
// once set, into the host-mapped page, so that the next call sees it without a
// synchronization.
__global__ void mirror_error_kernel() { mirror_error(); }
}  // namespace lf

// Scratch of lf_attn_bwd_static_ws: one array per device, loaded with the
// library and kept until the process exits.  Host code must not use this name
// as a device address (it names a host-side stand-in); the device address comes
// from cudaGetSymbolAddress below.
static __device__ __align__(256) unsigned char lf_static_ws[LF_STATIC_WS_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_static_ws_mutex;
void* g_static_ws_ptr[kMaxDevices] = {};

// Device address of lf_static_ws on the current device (looked up once per device).
lf_status static_ws_address(void** out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return LF_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_static_ws_mutex);
    if (!g_static_ws_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, lf_static_ws) != cudaSuccess || !p) return LF_ERR_CUDA;
        g_static_ws_ptr[dev] = p;
    }
    *out = g_static_ws_ptr[dev];
    return LF_OK;
}

// Device-side errors (an expired bounded wait, a bad segment table) are recorded in
// lf::g_device_error on the device and, through lf::g_error_mirror, in this page of
// host memory, page-locked and mapped into the device address space.  Every entry
// point reads it (a plain host load, no synchronization) and reports an earlier
// call's failure before launching anything; lf_sync_status clears it.
alignas(4096) volatile int g_host_error_page[1024];
std::once_flag g_register_once;
bool g_page_mapped = false;
bool g_mirror_ready[kMaxDevices] = {};

// Once per process: map the page; once per device: tell the device where it is.
lf_status prepare_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return LF_ERR_CUDA;
    std::call_once(g_register_once, [] {
        g_page_mapped = cudaHostRegister(const_cast<int*>(g_host_error_page), sizeof(g_host_error_page),
                                         cudaHostRegisterMapped | cudaHostRegisterPortable) ==
                        cudaSuccess;
        if (!g_page_mapped) (void)cudaGetLastError();
    });
    std::lock_guard<std::mutex> lock(g_static_ws_mutex);
    if (!g_mirror_ready[dev]) {
        int* dptr = nullptr;
        if (g_page_mapped) {
            void* p = nullptr;
            if (cudaHostGetDevicePointer(&p, const_cast<int*>(g_host_error_page), 0) != cudaSuccess)
                return LF_ERR_CUDA;
            dptr = static_cast<int*>(p);
        }
        if (cudaMemcpyToSymbol(lf::g_error_mirror, &dptr, sizeof(dptr)) != cudaSuccess)
            return LF_ERR_CUDA;
        g_mirror_ready[dev] = true;
    }
    return LF_OK;
}

// The call's kernels, then the flag's copy to the host page (stream order).
lf_status mirror_after(lf_status launched, cudaStream_t s) {
    if (launched != LF_OK) return launched;
    lf::mirror_error_kernel<<<1, 1, 0, s>>>();
    return launch_status();
}

lf_status status_of_device_code(int code) {
    if (code == 0) return LF_OK;
    return (code & 0xff) == lf::kErrTimeout ? LF_ERR_TIMEOUT : LF_ERR_INVALID_ARG;
}

// An earlier call's device-side failure not yet cleared by lf_sync_status.
lf_status pending_device_error() { return status_of_device_code(g_host_error_page[0]); }

}  // namespace

extern "C" {

const char* lf_status_string(lf_status s) {
    switch (s) {
        case LF_OK: return "LF_OK";
        case LF_ERR_INVALID_ARG: return "LF_ERR_INVALID_ARG: invalid argument";
        case LF_ERR_UNSUPPORTED: return "LF_ERR_UNSUPPORTED: shape not supported by this build";
        case LF_ERR_WORKSPACE: return "LF_ERR_WORKSPACE: workspace too small";
        case LF_ERR_CUDA: return "LF_ERR_CUDA: CUDA call failed";
        case LF_ERR_TIMEOUT: return "LF_ERR_TIMEOUT: a device-side bounded wait expired";
    }
    return "unknown lf_status";
}

lf_status lf_workspace_size(const lf_attn_desc* desc, int which, size_t* bytes) {
    lf_status st = check_desc(desc);
    if (st != LF_OK) return st;
    if (!bytes) return LF_ERR_INVALID_ARG;
    switch (which) {
        case LF_WS_FWD: *bytes = 0; return LF_OK;
        case LF_WS_SELECT: *bytes = 0; return LF_OK;
        case LF_WS_BWD: *bytes = bwd_ws_bytes_mod(desc); return LF_OK;
    }
    return LF_ERR_INVALID_ARG;
}

static lf_status attn_fwd_impl(const lf_attn_desc* desc, const lf_score_mod* mod, const void* q,
                               const void* k, const void* v, void* o, void* o_low, float* lse,
                               lf_stream_t stream) {
    lf_status st = check_desc(desc);
    if (st != LF_OK) return st;
    if (!q || !k || !v || !o || !lse) return LF_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return LF_ERR_INVALID_ARG;
    if ((st = pending_device_error()) != LF_OK) return st;
    if (desc->total_tokens == 0 || desc->max_seqlen == 0) return LF_OK;
    if ((st = prepare_device()) != LF_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // an empty modifier runs the plain forward, which has no residual: 0, and its backward
    // takes D from o alone
    if (o_low && mod_variant(mod) == 0 &&
        cudaMemsetAsync(o_low, 0, (size_t)desc->total_tokens * desc->hq * desc->d * 2, s) != cudaSuccess)
        return LF_ERR_CUDA;
    st = launch_fwd_any(desc, mod, q, k, v, o, o_low, lse, s);
    // the variants with modified scores write the host page themselves: one launch fewer
    return mod_variant(mod) == 0 ? mirror_after(st, s) : st;
}

lf_status lf_attn_fwd(const lf_attn_desc* desc, const void* q, const void* k, const void* v,
                      void* o, float* lse, void* ws, size_t ws_bytes, lf_stream_t stream) {
    (void)ws;
    (void)ws_bytes;
    return attn_fwd_impl(desc, nullptr, q, k, v, o, nullptr, lse, stream);
}

lf_status lf_attn_fwd_mod(const lf_attn_desc* desc, const lf_score_mod* mod, const void* q,
                          const void* k, const void* v, void* o, void* o_low, float* lse,
                          lf_stream_t stream) {
    lf_status st = check_desc(desc);
    if (st == LF_OK) st = check_mod(desc, mod);
    if (st == LF_OK && !aligned16(o_low)) st = LF_ERR_INVALID_ARG;
    if (st == LF_OK && desc->total_tokens == 0) return pending_device_error();   // empty tensors have no address
    return st != LF_OK ? st : attn_fwd_impl(desc, mod, q, k, v, o, o_low, lse, stream);
}

static lf_status block_select_impl(const lf_attn_desc* desc, const void* dout, const void* o,
                                   int rule, double param, uint64_t seed, uint64_t step,
                                   uint32_t flags, float* block_norm, float* D, double* tau,
                                   float* block_weight, uint8_t* keep, int32_t* kept_idx,
                                   int32_t* kept_cnt, lf_stream_t stream) {
    lf_status st = check_desc(desc);
    if (st != LF_OK) return st;
    if (rule == LF_RULE_BUDGET) {
        if (!(param >= 0.0 && param < 1.0)) return LF_ERR_INVALID_ARG;
    } else if (rule == LF_RULE_FIXED_FRACTION || rule == LF_RULE_TOPK) {
        if (!(param > 0.0 && param <= 1.0)) return LF_ERR_INVALID_ARG;
    } else {
        return LF_ERR_INVALID_ARG;
    }
    if (flags & ~LF_SELECT_NORMS_GIVEN) return LF_ERR_INVALID_ARG;
    const bool norms_given = (flags & LF_SELECT_NORMS_GIVEN) != 0;
    // dout is needed for the norms, o only for D; empty tensors have no address
    const bool rows = desc->total_tokens > 0, blocks = desc->max_seqlen > 0;
    if ((rows && ((!norms_given && !dout) || (D && (!dout || !o)))) || !tau || !kept_cnt)
        return LF_ERR_INVALID_ARG;
    if ((rows || blocks) && (!block_norm || !block_weight || !keep || !kept_idx)) return LF_ERR_INVALID_ARG;
    const void* ptrs[] = {dout, o, block_norm, D, tau, block_weight, keep, kept_idx, kept_cnt};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return LF_ERR_INVALID_ARG;
    if ((st = pending_device_error()) != LF_OK) return st;
    if (!blocks) return LF_OK;
    const int nbmax = nbmax_of(desc);
    if ((size_t)nbmax * sizeof(double) > 200 * 1024) return LF_ERR_UNSUPPORTED;
    if ((st = prepare_device()) != LF_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int write_norms = norms_given ? 0 : 1;
    if (write_norms || D) {
        st = desc->d == 128 ? launch_norms<128>(desc, dout, o, block_norm, D, write_norms, s)
                            : launch_norms<64>(desc, dout, o, block_norm, D, write_norms, s);
        if (st != LF_OK) return st;
    }
    const size_t smem = (size_t)nbmax * sizeof(float);
    auto kern = rule == LF_RULE_BUDGET ? lf::select_kernel<0>
              : rule == LF_RULE_FIXED_FRACTION ? lf::select_kernel<1> : lf::select_kernel<2>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess)
        return LF_ERR_CUDA;
    dim3 grid(desc->hq, desc->nseq);
    kern<<<grid, lf::kSelectThreads, smem, s>>>(desc->cu_seqlens, desc->total_tokens, desc->max_seqlen, desc->hq,
                                desc->block_q, nbmax, block_norm, param, seed, step, tau,
                                block_weight, keep, kept_idx, kept_cnt);
    return mirror_after(launch_status(), s);
}

lf_status lf_block_select(const lf_attn_desc* desc, const void* dout, const void* o, double delta,
                          uint64_t seed, uint64_t step, uint32_t flags, float* block_norm,
                          float* D, double* tau, float* block_weight, uint8_t* keep,
                          int32_t* kept_idx, int32_t* kept_cnt, void* ws, size_t ws_bytes,
                          lf_stream_t stream) {
    (void)ws;
    (void)ws_bytes;
    return block_select_impl(desc, dout, o, LF_RULE_BUDGET, delta, seed, step, flags, block_norm,
                             D, tau, block_weight, keep, kept_idx, kept_cnt, stream);
}

lf_status lf_block_select_rule(const lf_attn_desc* desc, const void* dout, const void* o,
                               int rule, double param, uint64_t seed, uint64_t step,
                               uint32_t flags, float* block_norm, float* D, double* tau,
                               float* block_weight, uint8_t* keep, int32_t* kept_idx,
                               int32_t* kept_cnt, void* ws, size_t ws_bytes, lf_stream_t stream) {
    (void)ws;
    (void)ws_bytes;
    return block_select_impl(desc, dout, o, rule, param, seed, step, flags, block_norm, D, tau,
                             block_weight, keep, kept_idx, kept_cnt, stream);
}

static lf_status attn_bwd_impl(const lf_attn_desc* desc, const lf_score_mod* mod, const void* q,
                               const void* k, const void* v, const void* o, const void* o_low, const float* lse,
                               const void* dout, const float* D, const float* block_weight,
                               const int32_t* kept_idx, const int32_t* kept_cnt, void* dq, void* dk,
                               void* dv, void* ws, size_t ws_bytes, lf_stream_t stream) {
    lf_status st = check_desc(desc);
    if (st != LF_OK) return st;
    if (!q || !k || !v || !lse || !dout || !block_weight || !kept_idx || !kept_cnt || !dq ||
        !dk || !dv)
        return LF_ERR_INVALID_ARG;
    if (!D && !o) return LF_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, lse, dout, block_weight, kept_idx, kept_cnt, dq, dk, dv, ws};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return LF_ERR_INVALID_ARG;
    if ((o && !aligned16(o)) || (D && !aligned16(D))) return LF_ERR_INVALID_ARG;
    if ((st = pending_device_error()) != LF_OK) return st;
    if (desc->total_tokens == 0 || desc->max_seqlen == 0) return LF_OK;
    const bool starts = mod && mod->row_start;
    if (!ws || ws_bytes < (starts ? bwd_ws_bytes_mod(desc) : bwd_ws_bytes(desc, D == nullptr)))
        return LF_ERR_WORKSPACE;
    int32_t* key_last =
        starts ? reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + key_last_offset(desc)) : nullptr;
    if ((st = prepare_device()) != LF_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return mirror_after(launch_bwd_any(desc, mod, key_last, o_low, q, k, v, o, lse, dout, D, block_weight, kept_idx,
                                       kept_cnt, dq, dk, dv, ws, s),
                        s);
}

lf_status lf_attn_bwd(const lf_attn_desc* desc, const void* q, const void* k, const void* v,
                      const void* o, const float* lse, const void* dout, const float* D,
                      const float* block_weight, const int32_t* kept_idx,
                      const int32_t* kept_cnt, void* dq, void* dk, void* dv, void* ws,
                      size_t ws_bytes, lf_stream_t stream) {
    return attn_bwd_impl(desc, nullptr, q, k, v, o, nullptr, lse, dout, D, block_weight, kept_idx, kept_cnt, dq, dk, dv,
                         ws, ws_bytes, stream);
}

lf_status lf_attn_bwd_mod(const lf_attn_desc* desc, const lf_score_mod* mod, const void* q,
                          const void* k, const void* v, const void* o, const void* o_low,
                          const float* lse, const void* dout, const float* D, const float* block_weight,
                          const int32_t* kept_idx, const int32_t* kept_cnt, void* dq, void* dk,
                          void* dv, void* ws, size_t ws_bytes, lf_stream_t stream) {
    lf_status st = check_desc(desc);
    if (st == LF_OK) st = check_mod(desc, mod);
    if (st == LF_OK && (!aligned16(o_low) || (o_low && D))) st = LF_ERR_INVALID_ARG;
    if (st == LF_OK && desc->total_tokens == 0) return pending_device_error();
    return st != LF_OK ? st
                       : attn_bwd_impl(desc, mod, q, k, v, o, o_low, lse, dout, D, block_weight, kept_idx, kept_cnt, dq,
                                       dk, dv, ws, ws_bytes, stream);
}

lf_status lf_attn_bwd_static_ws(const lf_attn_desc* desc, const void* q, const void* k,
                                const void* v, const void* o, const float* lse, const void* dout,
                                const float* D, const float* block_weight,
                                const int32_t* kept_idx, const int32_t* kept_cnt, void* dq,
                                void* dk, void* dv, lf_stream_t stream) {
    lf_status st = check_desc(desc);
    if (st != LF_OK) return st;
    if (!q || !k || !v || !lse || !dout || !block_weight || !kept_idx || !kept_cnt || !dq ||
        !dk || !dv)
        return LF_ERR_INVALID_ARG;
    if (!D && !o) return LF_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, lse, dout, block_weight, kept_idx, kept_cnt, dq, dk, dv};
    for (const void* p : ptrs)
        if (!aligned16(p)) return LF_ERR_INVALID_ARG;
    if ((o && !aligned16(o)) || (D && !aligned16(D))) return LF_ERR_INVALID_ARG;
    const size_t need = bwd_ws_bytes(desc, D == nullptr);
    if (need > LF_STATIC_WS_BYTES) return LF_ERR_WORKSPACE;
    if ((st = pending_device_error()) != LF_OK) return st;
    if (desc->total_tokens == 0 || desc->max_seqlen == 0) return LF_OK;
    if ((st = prepare_device()) != LF_OK) return st;
    void* ws = nullptr;
    st = static_ws_address(&ws);
    if (st != LF_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // launch_bwd clears the accumulators it uses before the kernel
    return mirror_after(launch_bwd_any(desc, nullptr, nullptr, nullptr, q, k, v, o, lse, dout, D, block_weight, kept_idx,
                                       kept_cnt, dq, dk, dv, ws, s),
                        s);
}

lf_status lf_qk_norm_rope(const lf_qk_desc* desc, const void* q, int64_t q_stride, const void* k,
                          int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out,
                          int64_t k_out_stride, lf_stream_t stream) {
    lf_status st = check_qk_desc(desc);
    if (st != LF_OK) return st;
    if (desc->total_tokens == 0) return pending_device_error();
    if (!qk_operand_ok(desc, q, q_stride, desc->hq) || !qk_operand_ok(desc, k, k_stride, desc->hkv) ||
        !qk_operand_ok(desc, q_out, q_out_stride, desc->hq) ||
        !qk_operand_ok(desc, k_out, k_out_stride, desc->hkv))
        return LF_ERR_INVALID_ARG;
    if ((st = pending_device_error()) != LF_OK) return st;
    if ((st = prepare_device()) != LF_OK) return st;
    lf::QkParams p = qk_params(desc);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.qs = q_stride;
    p.ks = k_stride;
    p.oq = static_cast<__nv_bfloat16*>(q_out);
    p.ok = static_cast<__nv_bfloat16*>(k_out);
    p.oqs = q_out_stride;
    p.oks = k_out_stride;
    const int blocks = qk_grid(desc, p, false);
    return launch_qk_any(desc, p, blocks, false, reinterpret_cast<cudaStream_t>(stream));
}

lf_status lf_qk_workspace_size(const lf_qk_desc* desc, size_t* bytes) {
    lf_status st = check_qk_desc(desc);
    if (st != LF_OK) return st;
    if (!bytes) return LF_ERR_INVALID_ARG;
    *bytes = (size_t)lf::kQkMaxBlocks * 2 * desc->d * sizeof(float);
    return LF_OK;
}

lf_status lf_qk_norm_rope_bwd(const lf_qk_desc* desc, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, const void* dq_out,
                              int64_t dq_out_stride, const void* dk_out, int64_t dk_out_stride,
                              void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                              float* dqw, float* dkw, void* ws, size_t ws_bytes,
                              lf_stream_t stream) {
    lf_status st = check_qk_desc(desc);
    if (st != LF_OK) return st;
    const bool norm = (desc->flags & LF_QK_NORM) != 0, weights = dqw || dkw;
    if (weights && !norm) return LF_ERR_INVALID_ARG;
    const bool rows = desc->total_tokens > 0;
    if (rows && norm &&
        (!qk_operand_ok(desc, q, q_stride, desc->hq) || !qk_operand_ok(desc, k, k_stride, desc->hkv)))
        return LF_ERR_INVALID_ARG;
    if (rows && (!qk_operand_ok(desc, dq_out, dq_out_stride, desc->hq) ||
                 !qk_operand_ok(desc, dk_out, dk_out_stride, desc->hkv) ||
                 !qk_operand_ok(desc, dq, dq_stride, desc->hq) ||
                 !qk_operand_ok(desc, dk, dk_stride, desc->hkv)))
        return LF_ERR_INVALID_ARG;
    if (!aligned16(dqw) || !aligned16(dkw) || !aligned16(ws)) return LF_ERR_INVALID_ARG;
    if ((st = pending_device_error()) != LF_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!rows) {
        const size_t b = desc->d * sizeof(float);
        if ((dqw && cudaMemsetAsync(dqw, 0, b, s) != cudaSuccess) ||
            (dkw && cudaMemsetAsync(dkw, 0, b, s) != cudaSuccess))
            return LF_ERR_CUDA;
        return LF_OK;
    }
    size_t need = 0;
    if ((st = lf_qk_workspace_size(desc, &need)) != LF_OK) return st;
    if (weights && (!ws || ws_bytes < need)) return LF_ERR_WORKSPACE;
    if ((st = prepare_device()) != LF_OK) return st;
    lf::QkParams p = qk_params(desc);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.qs = q_stride;
    p.ks = k_stride;
    p.gq = static_cast<const __nv_bfloat16*>(dq_out);
    p.gk = static_cast<const __nv_bfloat16*>(dk_out);
    p.gqs = dq_out_stride;
    p.gks = dk_out_stride;
    p.oq = static_cast<__nv_bfloat16*>(dq);
    p.ok = static_cast<__nv_bfloat16*>(dk);
    p.oqs = dq_stride;
    p.oks = dk_stride;
    p.partial = weights ? static_cast<float*>(ws) : nullptr;
    // lanes that hold no row (a surplus head, a row behind the last segment) hold zeros: with
    // eps = 0 their root would be inf, and 0 * inf reach the weights' sums.  The least number
    // above 0 keeps it finite and is lost beside any row's mean square (a test per row cost 2 %)
    if (p.eps == 0.f) p.eps = std::numeric_limits<float>::denorm_min();
    const int blocks = qk_grid(desc, p, true);
    if ((st = launch_qk_any(desc, p, blocks, true, s)) != LF_OK) return st;
    if (weights) {
        lf::qk_weight_grad_kernel<<<2 * desc->d / 32, dim3(32, 32), 0, s>>>(p.partial, blocks, desc->d, dqw, dkw);
        return launch_status();
    }
    return LF_OK;
}

lf_status lf_watchdog_selftest(uint32_t limit_log2, lf_stream_t stream) {
    if (limit_log2 < 10 || limit_log2 > 31) return LF_ERR_INVALID_ARG;
    lf_status st = pending_device_error();
    if (st != LF_OK) return st;
    if ((st = prepare_device()) != LF_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    lf::watchdog_selftest_kernel<<<1, 32, 0, s>>>(1ll << limit_log2);
    return mirror_after(launch_status(), s);
}

lf_status lf_sync_status(lf_stream_t stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return LF_ERR_CUDA;
    int flag = 0;
    if (cudaMemcpyFromSymbol(&flag, lf::g_device_error, sizeof(int)) != cudaSuccess)
        return LF_ERR_CUDA;
    if (flag != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(lf::g_device_error, &zero, sizeof(int)) != cudaSuccess)
            return LF_ERR_CUDA;
    }
    // the page may also hold a failure recorded on another device
    const int host = g_host_error_page[0];
    g_host_error_page[0] = 0;
    return status_of_device_code(flag != 0 ? flag : host);
}

lf_status lf_check_device_error(lf_stream_t stream) { return lf_sync_status(stream); }

}  // extern "C"
