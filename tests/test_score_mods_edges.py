"""Attention with modified scores through autograd: arrays changed between the two passes,
empty batches, the function's own arguments, slopes that are parameters;
and rows whose scores all lie where the cap is flat."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_dense_b200 as lf
from block_sparse_attention_dense_b200 import build as lfbuild
from block_sparse_attention_dense_b200.autograd import LazyFlashAttention, lazyflash_attention
from test_score_mods import NAMED, B, U, dev, raw_desc

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    lfbuild.build()
    return lf.lib()


def attend(c, g, **kw):
    return lazyflash_attention(g["q"], g["k"], g["v"], g["cu"], max(c.lens), delta=c.delta, seed=3, step=0,
                               block_q=c.block, softcap=c.softcap, alibi_slopes=g["slopes"], prefix_len=g["prefix"],
                               prefix_causal=c.prefix_causal, row_start=g["start"], **kw)


@gpu
@pytest.mark.parametrize("name", ["slopes", "prefix", "start", "cu"])
def test_arrays_changed_between_the_passes_are_noticed(name):
    """The backward would recompute P with another mask or bias than the LSE's."""
    c = NAMED["everything"]
    g = dev(c.make(6))
    for x in ("q", "k", "v"):
        g[x].requires_grad_(True)
    o = attend(c, g)
    g[name].add_(0)   # the same values: what counts is that they were written
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.backward(g["dout"])


@gpu
@pytest.mark.parametrize("longest", [0, 200])
def test_training_step_of_an_empty_batch(longest):
    q, k, v = (torch.zeros(0, h, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True) for h in (4, 2, 2))
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    start = torch.zeros(0, dtype=torch.int32, device="cuda")
    drawn = {}
    o = lazyflash_attention(q, k, v, cu, longest, softcap=20.0, row_start=start, selection_out=drawn)
    o.backward(torch.zeros_like(o))
    lf.lf_sync_status()
    assert o.shape == q.shape and all(x.grad is not None and x.grad.shape == x.shape for x in (q, k, v))
    blocks = -(-longest // 128)
    assert drawn["norm"].shape == (2, 4, blocks) and (drawn["kept_cnt"] == 0).all() and (drawn["tau"] == 0).all()


def test_selection_of_no_rows_needs_no_token_tensors(L):
    """As the forward and the backward with modified scores: empty tensors have no address."""
    d = raw_desc(total_tokens=0, max_seqlen=0)
    p = 0x10000
    tail = [None, 0, None]
    # dout, o | norm, D, tau, weight, keep, kept_idx, kept_cnt
    assert L.lf_block_select(ctypes.byref(d), None, None, 0.1, 0, 0, 0, None, None, p, None, None, None, p, *tail) == 0
    for missing in (2, 6):   # tau and kept_cnt have nseq * hq elements whatever the rows
        outs = [None, None, p, None, None, None, p]
        outs[missing] = None
        assert L.lf_block_select(ctypes.byref(d), None, None, 0.1, 0, 0, 0, *outs, *tail) == lf.LF_ERR_INVALID_ARG
    rows = raw_desc()
    assert L.lf_block_select(ctypes.byref(rows), None, None, 0.1, 0, 0, 0, p, None, p, p, p, p, p, *tail) == lf.LF_ERR_INVALID_ARG


@gpu
def test_the_function_takes_the_arguments_of_the_plain_attention():
    """LazyFlashAttention.apply without a modifier: twelve arguments, as for the plain attention."""
    c = NAMED["cap"]
    g = dev(c.make())
    x = [[g[n].clone().requires_grad_(True) for n in ("q", "k", "v")] for _ in range(2)]
    o = LazyFlashAttention.apply(*x[0], g["cu"], max(c.lens), 0.2, 3, 0, True, 128, None, None)
    z = lazyflash_attention(*x[1], g["cu"], max(c.lens), delta=0.2, seed=3, step=0)
    o.backward(g["dout"])
    z.backward(g["dout"])
    assert torch.equal(o, z) and torch.equal(x[0][1].grad, x[1][1].grad) and torch.equal(x[0][2].grad, x[1][2].grad)
    assert (x[0][0].grad.float() - x[1][0].grad.float()).norm() <= B * x[1][0].grad.float().norm()


def test_slopes_are_refused_only_where_a_gradient_is_recorded():
    x, slopes = torch.zeros(4, 2, 64), torch.zeros(2, requires_grad=True)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # only the device is wrong
        lazyflash_attention(x, x, x, torch.tensor([0, 4]), 4, alibi_slopes=slopes)


@gpu
def test_slopes_that_are_a_parameter_without_grad():
    c = NAMED["everything"]
    g = dev(c.make())
    want = attend(c, g)
    with torch.no_grad():
        got = attend(c, dict(g, slopes=torch.nn.Parameter(g["slopes"])))
    assert torch.equal(got, want)


@gpu
@pytest.mark.parametrize("d,block,prefix", [(128, 128, None), (64, 64, 40)])
def test_rows_whose_scores_are_all_saturated(d, block, prefix):
    """|x| / cap between 7 and 12 for every score, where 1 - tanh^2 = 4 e / (1 + e)^2, e = exp(2 |x| / cap),
    is 3e-6 to 1e-10: the gradient is that small, and right.

    Off by (u = 2^-24, b = 2^-8): x by d u scale sum|q_i k_i| + 4 u |x| (ex), which changes the
    derivative by 2 ex / cap of itself and every z by less than 1e-6 cap (tanh as computed), P
    by twice that and 1e-6 (ep); the derivative's own operations (two roundings of an exponent
    below 40, exp2, a sum, a reciprocal, a product) by 2 * 40 u + 16 u of itself.  D, dP and
    the sums as in test_score_mods.py."""
    n, hq, hkv, cap, scale = 300, 2, 1, 1.0, 1.0 / math.sqrt(d)
    gen = torch.Generator().manual_seed(0)
    axis = torch.randn(d, generator=gen).sign()
    # q = s axis + noise, k = axis + noise: x = +-(7 to 12)
    size = 8.0 + 3.0 * torch.rand(n, hq, 1, generator=gen)
    sign = torch.randn(n, hq, 1, generator=gen).sign()
    q = (sign * size / math.sqrt(d) * axis + 0.02 * torch.randn(n, hq, d, generator=gen)).bfloat16()
    k = (axis + 0.02 * torch.randn(n, hkv, d, generator=gen)).bfloat16()
    v, do = (torch.randn(n, h, d, generator=gen).bfloat16() for h in (hkv, hq))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    leaves = [t.cuda().requires_grad_(True) for t in (q, k, v)]
    plen = None if prefix is None else torch.tensor([prefix], dtype=torch.int32, device="cuda")
    o = lazyflash_attention(*leaves, cu, n, delta=0.0, block_q=block, softcap=cap, softmax_scale=scale, prefix_len=plen)
    o.backward(do.cuda())
    lf.lf_sync_status()
    see = torch.ones(n, n).tril().bool()
    if prefix is not None:
        see[:, :prefix] = True
    kd, vd = k[:, 0].double(), v[:, 0].double()
    dk, tk = torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, d, dtype=torch.float64)
    for h in range(hq):
        qd, dod = q[:, h].double(), do[:, h].double()
        x = qd @ kd.T * scale
        assert x.abs().min() > 7 * cap and x.abs().max() < 12 * cap
        ex = d * U * scale * (qd.abs() @ kd.abs().T) + 4 * U * x.abs()
        p = torch.softmax((cap * torch.tanh(x / cap)).masked_fill(~see, -math.inf), 1)
        ep = 2 * (1e-6 * cap) + 1e-6
        e = torch.exp(2 * x.abs() / cap)
        damp = 4 * e / (1 + e).square()
        edamp = 2 * ex / cap + (2 * 40 + 16) * U
        out = p @ vd
        dp, D = dod @ vd.T, (dod * out).sum(1, keepdim=True)
        ds = p * (dp - D) * damp
        edp = d * U * (dod.abs() @ vd.abs().T)
        eD = 2 * (B + ep) * (p * (dp - D).abs()).sum(1, keepdim=True) + edp.amax(1, keepdim=True)
        eD += (B * B + d * U) * (dod.abs() * out.abs()).sum(1, keepdim=True)
        eds = (B + ep + edamp + 4 * U) * ds.abs() + p * damp * (eD + edp) + n * hq * U * ds.abs()
        want, tol = scale * ds @ kd, scale * eds @ kd.abs()
        got = leaves[0].grad[:, h].double().cpu()
        assert ((got - want).abs() <= tol + B * want.abs()).all(), float(((got - want).abs() / (tol + B * want.abs())).max())
        dk += scale * ds.T @ qd
        tk += scale * eds.T @ qd.abs()
    got = leaves[1].grad[:, 0].double().cpu()
    assert ((got - dk).abs() <= tk + B * dk.abs()).all(), float(((got - dk).abs() / (tk + B * dk.abs())).max())
