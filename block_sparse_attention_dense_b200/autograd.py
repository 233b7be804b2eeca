"""LazyFlash, and the norms and rotation before it, as torch.autograd.Functions
(argument marshalling only).

The forward is the exact dense attention (lf_attn_fwd); the backward selects
query blocks from the incoming output gradient (lf_block_select: budget delta,
Philox draw keyed on (seed, step)) and runs the block-sparse backward over the
kept blocks (lf_attn_bwd).  The returned gradients are the reweighted estimate:
unbiased in expectation, exactly the dense gradient at delta = 0 (LazyFlash
article, section "Un budget sur la masse de gradient, et un tirage qui garde le
gradient non biaisé").

Tensors use the THD layout of include/lazyflash.h: q [T, hq, d], k and v
[T, hkv, d] (bf16, CUDA, contiguous); cu_seqlens int32 CUDA [nseq + 1].
"""
from __future__ import annotations

import itertools
import math

import torch
from torch.autograd.function import once_differentiable

from . import (Buffers, lf_attn_bwd, lf_attn_bwd_mod, lf_attn_fwd, lf_attn_fwd_mod, lf_block_select,
               lf_qk_norm_rope, lf_qk_norm_rope_bwd, lf_qk_workspace_size, make_desc, make_qk_desc,
               make_score_mod)

_step_counter = itertools.count()


def _modified(softcap, alibi_slopes, prefix_len, prefix_causal, row_start, positions):
    return bool(softcap or prefix_causal or alibi_slopes is not None or prefix_len is not None
                or row_start is not None or positions is not None)


class LazyFlashAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, max_seqlen, delta, seed, step, causal, block_q,
                softmax_scale, selection_out, softcap=0.0, alibi_slopes=None, prefix_len=None,
                prefix_causal=False, row_start=None, positions=None):
        for t in (q, k, v):
            if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("q, k, v must be contiguous bf16 CUDA tensors")
        T, hq, d = q.shape
        hkv = k.shape[1]
        scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(d)
        desc = make_desc(cu_seqlens, max_seqlen, T, hq, hkv, d, scale, causal, block_q)
        o = torch.empty_like(q)
        lse = torch.empty(hq, T, dtype=torch.float32, device=q.device)
        if _modified(softcap, alibi_slopes, prefix_len, prefix_causal, row_start, positions):
            mod = make_score_mod(softcap, alibi_slopes, prefix_len, prefix_causal, row_start, positions)
            # O's rounding residual, kept for the backward's D (not when no gradient is asked for)
            o_low = torch.empty_like(q) if any(ctx.needs_input_grad) else None
            lf_attn_fwd_mod(desc, mod, q, k, v, o, lse, o_low)
            # the modifier's arrays are saved as cu_seqlens is, so that one written to between the
            # two passes is noticed: P comes from this pass's LSE and the backward's own scores
            ctx.save_for_backward(q, k, v, o, lse, cu_seqlens, o_low, alibi_slopes, prefix_len, row_start, positions)
            ctx.scalars = (softcap, prefix_causal)
        else:
            lf_attn_fwd(desc, q, k, v, o, lse)
            ctx.save_for_backward(q, k, v, o, lse, cu_seqlens)
        ctx.desc = desc
        ctx.delta = float(delta)
        ctx.seed = int(seed)
        ctx.step = int(next(_step_counter) if step is None else step)
        ctx.selection_out = selection_out
        return o

    @staticmethod
    def backward(ctx, grad_o):
        q, k, v, o, lse, cu_seqlens, *modifier = ctx.saved_tensors
        desc = ctx.desc
        mod = None
        if modifier:
            o_low, alibi_slopes, prefix_len, row_start, positions = modifier
            softcap, prefix_causal = ctx.scalars
            mod = make_score_mod(softcap, alibi_slopes, prefix_len, prefix_causal, row_start, positions)
        dout = grad_o.to(torch.bfloat16).contiguous()
        # the backward's own buffers only: o and lse are the forward's saved tensors
        bufs = Buffers(desc, device=q.device, forward=False)
        if desc.max_seqlen == 0:   # an empty batch: the selection writes nothing
            bufs.tau.zero_()
            bufs.kept_cnt.zero_()
        # with modified scores the backward computes D itself, from o and its residual
        D = bufs.D if mod is None else None
        lf_block_select(desc, dout, o, ctx.delta, ctx.seed, ctx.step, 0, bufs.norm, D,
                        bufs.tau, bufs.w, bufs.keep, bufs.kept_idx, bufs.kept_cnt)
        args = (q, k, v, o, lse, dout, D, bufs.w, bufs.kept_idx, bufs.kept_cnt, bufs.dq, bufs.dk,
                bufs.dv, bufs.ws)
        if mod is None:
            lf_attn_bwd(desc, *args)
        else:
            lf_attn_bwd_mod(desc, mod, *args, o_low)
        if ctx.selection_out is not None:
            ctx.selection_out.update(norm=bufs.norm, tau=bufs.tau, keep=bufs.keep,
                                     weight=bufs.w, kept_cnt=bufs.kept_cnt, step=ctx.step)
        return (bufs.dq, bufs.dk, bufs.dv) + (None,) * 15


def lazyflash_attention(q, k, v, cu_seqlens, max_seqlen, delta=0.1, seed=0, step=None,
                        causal=True, block_q=128, softmax_scale=None, selection_out=None,
                        softcap=0.0, alibi_slopes=None, prefix_len=None, prefix_causal=False,
                        row_start=None, positions=None):
    """Dense attention forward, LazyFlash block-sparse backward.

    ``step`` defaults to a process-wide counter, so every backward draws a
    fresh mask; pass it explicitly to replay a draw.  If ``selection_out`` is a
    dict, the backward stores in it the selection it drew: block norms ``norm``,
    thresholds ``tau``, ``keep``, block weights ``weight`` ([nseq, hq, nbmax]
    device tensors), ``kept_cnt`` and the Philox ``step`` used.

    ``softcap`` (scores capped by a tanh), ``alibi_slopes`` [hq] (a bias that falls with the
    distance; no gradient), ``prefix_len`` [nseq], ``prefix_causal`` and ``row_start`` [T]
    (prefix, document, window and shared-prompt masks) modify the scores of both directions:
    lf_score_mod in include/lazyflash.h says how, shared_prompt_tables makes the last's.  The
    bias counts rows of the packed segment: answers that share a prompt need ``positions`` [T]
    (the table's fourth) as well, from which it then counts the distance to the prompt's keys;
    without, an answer is too far from its prompt by the answers packed before it.  With
    modified scores the backward also keeps O's rounding residual, a second tensor of O's size
    (no gradient asked for: not allocated).

    Every row belongs to a segment (cu_seqlens[-1] = T): rows behind the last one are left
    unwritten in the result and the gradients."""
    if alibi_slopes is not None and alibi_slopes.requires_grad and torch.is_grad_enabled():
        raise ValueError("no gradient is computed for alibi_slopes: pass them detached")
    modifier = (softcap, alibi_slopes, prefix_len, prefix_causal, row_start, positions)
    return LazyFlashAttention.apply(q, k, v, cu_seqlens, max_seqlen, delta, seed, step, causal,
                                    block_q, softmax_scale, selection_out, *(modifier if _modified(*modifier) else ()))


class QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos_sin, cu_seqlens, positions, eps, norm, interleaved):
        # rows behind the last segment (a padded batch) come out as zeros, and so do their
        # gradients: every element of what this returns is defined
        desc = make_qk_desc(q, k, q_weight, k_weight, cos_sin, cu_seqlens, positions, eps, norm,
                            interleaved, zero_tail=True)
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        lf_qk_norm_rope(desc, q, k, q_out, k_out)
        # without the norm the gradient does not read the inputs
        ctx.save_for_backward(*((q, k) if norm else (None, None)), q_weight, k_weight, cos_sin,
                              cu_seqlens, positions)
        ctx.desc = desc
        return q_out, k_out

    @staticmethod
    @once_differentiable
    def backward(ctx, gq, gk):
        q, k, q_weight, k_weight = ctx.saved_tensors[:4]
        desc = ctx.desc
        gq = gq.to(torch.bfloat16).contiguous()
        gk = gk.to(torch.bfloat16).contiguous()
        dq, dk = torch.empty_like(gq), torch.empty_like(gk)

        def grad_of(w, needed):
            return torch.empty(desc.d, dtype=torch.float32, device=gq.device) if w is not None and needed else None

        dqw = grad_of(q_weight, ctx.needs_input_grad[2])
        dkw = grad_of(k_weight, ctx.needs_input_grad[3])
        ws = None
        if dqw is not None or dkw is not None:
            ws = torch.empty(lf_qk_workspace_size(desc), dtype=torch.uint8, device=gq.device)
        lf_qk_norm_rope_bwd(desc, q, k, gq, gk, dq, dk, dqw, dkw, ws)
        return (dq, dk, None if dqw is None else dqw.to(q_weight.dtype),
                None if dkw is None else dkw.to(k_weight.dtype), None, None, None, None, None, None)


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos_sin=None, cu_seqlens=None, positions=None,
                 eps=1e-6, norm=True, interleaved=False):
    """RMS norm of every query and key head, then the position rotation, in one pass; both
    differentiable (see lf_qk_norm_rope in include/lazyflash.h).

    q [T, hq, d], k [T, hkv, d] bf16; they may be slices of one fused projection's output
    (contiguous heads, any token stride).  The results are contiguous and go into
    lazyflash_attention.  cos_sin: rope_cos_sin(npos, rot), or None for the norm alone;
    norm=False rotates only.  A row's position is its index in its segment of cu_seqlens,
    or positions[row].  No gradient is computed for the table."""
    if cos_sin is not None and cos_sin.requires_grad and torch.is_grad_enabled():
        raise ValueError("no gradient is computed for cos_sin: pass it detached")
    return QkNormRope.apply(q, k, q_weight, k_weight, cos_sin, cu_seqlens, positions, eps, norm, interleaved)
