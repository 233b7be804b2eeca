"""Attention with a distance bias whose distances to prefix keys are counted from positions:
answers that share a prompt, computed once, are as far from it as in copies of their own.
Formulas in 64 bits; the tolerances are those of test_score_mods.py, with the distance as it
is counted here."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_dense_b200 as lf
from block_sparse_attention_dense_b200 import build as lfbuild
from block_sparse_attention_dense_b200.autograd import lazyflash_attention
from test_score_mods import B, P, U, bwd_args, fwd_args, raw_desc, window

gpu = pytest.mark.gpu


class Case:
    """Segments as (prefix length, row_start, positions), or as (prompt length, answers' lengths)."""

    def __init__(self, name, segments, hq=4, hkv=2, d=128, block=128, softcap=0.0, spread=1.5, delta=0.2,
                 rising=False, steep=0.7, tail=0):
        self.__dict__.update(locals())
        del self.__dict__["self"]
        self.parts = []
        for seg in segments:
            if len(seg) == 2:
                _, plen, start, pos = lf.shared_prompt_tables([seg[0]], [seg[1]], device="cpu")
                seg = (int(plen[0]), start.numpy(), pos.numpy())
            self.parts.append(seg)
        self.lens = [len(s[1]) for s in self.parts]
        self.scale = 1.0 / math.sqrt(d)

    def make(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        T = sum(self.lens) + self.tail

        def normal(h, s=1.0):
            return (torch.randn(T, h, self.d, generator=g) * s).to(torch.bfloat16)

        m = dict(q=normal(self.hq, self.spread), k=normal(self.hkv), v=normal(self.hkv), dout=normal(self.hq), T=T)
        slopes = torch.tensor([self.steep * 2.0 ** (-4 * h / self.hq) for h in range(self.hq)])
        if self.rising:
            slopes[1::2] *= -0.1
        m["slopes"] = slopes
        m["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(self.lens)]), dtype=torch.int32)
        m["prefix"] = torch.tensor([s[0] for s in self.parts], dtype=torch.int32)
        behind = np.full(self.tail, -5)   # not read
        for n, i in (("start", 1), ("pos", 2)):
            m[n] = torch.tensor(np.concatenate([s[i] for s in self.parts] + [behind]), dtype=torch.int32)
        return m


def mod_of(c, g, **kw):
    return lf.make_score_mod(**dict(dict(softcap=c.softcap, alibi_slopes=g["slopes"], prefix_len=g["prefix"],
                                         prefix_causal=True, row_start=g["start"], positions=g["pos"]), **kw))


def run(c, g, seed=3, **kw):
    desc = lf.make_desc(g["cu"], max(c.lens), g["T"], c.hq, c.hkv, c.d, c.scale, True, c.block)
    mod, b = mod_of(c, g, **kw), lf.Buffers(desc)
    o_low = torch.empty_like(b.o)
    for t in (b.o, b.dq, b.dk, b.dv, b.lse):
        t.fill_(float("nan"))
    b.ws.fill_(255)
    lf.lf_attn_fwd_mod(desc, mod, g["q"], g["k"], g["v"], b.o, b.lse, o_low)
    lf.lf_block_select(desc, g["dout"], b.o, c.delta, seed, 0, 0, b.norm, None, b.tau, b.w, b.keep, b.kept_idx, b.kept_cnt)
    lf.lf_attn_bwd_mod(desc, mod, g["q"], g["k"], g["v"], b.o, b.lse, g["dout"], None, b.w, b.kept_idx, b.kept_cnt,
                       b.dq, b.dk, b.dv, b.ws, o_low)
    lf.lf_sync_status()
    return b


def reference(c, m, w):
    """O, LSE, dQ, dK, dV and how far the kernels' may be off (test_score_mods.py has the reasons)."""
    q, k, v, do = (m[x].double() for x in ("q", "k", "v", "dout"))
    out = {x: torch.zeros_like(m[y].double()) for x, y in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
    out["lse"] = torch.zeros(c.hq, m["T"], dtype=torch.float64)
    tol = {x: t.clone() for x, t in out.items()}
    G, at = c.hq // c.hkv, 0
    for i, n in enumerate(c.lens):
        r = slice(at, at + n)
        at += n
        if n == 0:
            continue
        prefix, start, pos = c.parts[i]
        t, u = np.arange(n)[:, None], np.arange(n)[None]
        see = torch.from_numpy((u <= t) & ((u >= np.asarray(start)[:, None]) | (u < prefix)))
        far = torch.from_numpy(np.where(u < prefix, np.asarray(pos)[:, None], t) - u).double().abs()
        for h in range(c.hq):
            g = h // G
            qh, kh, vh, dor = q[r, h], k[r, g], v[r, g], do[r, h]
            x = qh @ kh.T * c.scale
            ez = c.d * U * c.scale * (qh.abs() @ kh.abs().T) + 8 * U * x.abs()
            z, damp = x, torch.ones_like(x)
            if c.softcap:
                th = torch.tanh(x / c.softcap)
                z, damp = c.softcap * th, 1 - th * th
                ez = ez * damp + 1e-6 * z.abs()
            bias = float(m["slopes"][h]) * far
            z, ez = (z - bias).masked_fill(~see, -math.inf), ez + 8 * U * bias.abs()
            ez = ez.masked_fill(~see, 0.0).amax(1, keepdim=True)
            lse = torch.logsumexp(z, 1, keepdim=True)
            p, ep = torch.exp(z - lse), 2 * ez + 1e-6
            o = p @ vh
            out["o"][r, h], out["lse"][h, r] = o, lse[:, 0]
            tol["o"][r, h] = 2 * (B + ep) * (p @ vh.square() - o.square()).clamp(min=0).sqrt() + (B + 8 * U) * o.abs()
            tol["lse"][h, r] = (ez + 16 * U * lse.abs() + 1e-6)[:, 0]
            wr = w[i, h, torch.arange(n) // c.block].double()[:, None]
            dp, D = dor @ vh.T, (dor * o).sum(1, keepdim=True)
            ds, wp = wr * p * (dp - D) * damp, wr * p
            edp = c.d * U * (dor.abs() @ vh.abs().T)
            eD = 2 * (B + ep) * (p * (dp - D).abs()).sum(1, keepdim=True) + edp.amax(1, keepdim=True)
            eD += (B * B + c.d * U) * (dor.abs() * o.abs()).sum(1, keepdim=True)
            sums = n * c.hq * U
            eds = (B + ep + 4 * U + sums) * ds.abs() + wp * damp * (eD + edp)
            if c.softcap:
                eds = eds + wp * (dp - D).abs() * 2 * (ez / c.softcap + 1e-6)
            out["dq"][r, h] = c.scale * ds @ kh
            out["dk"][r, g] += c.scale * ds.T @ qh
            out["dv"][r, g] += wp.T @ dor
            tol["dq"][r, h] = c.scale * eds @ kh.abs()
            tol["dk"][r, g] += c.scale * eds.T @ qh.abs()
            tol["dv"][r, g] += ((B + ep + sums) * wp).T @ dor.abs()
    for x in ("dq", "dk", "dv"):
        tol[x] += B * out[x].abs() + 1e-30
    return out, tol


def halfway(n, prefix):
    """Positions halfway between the least allowed and the row itself."""
    t = np.arange(n)
    return (np.minimum(t, prefix - 1) + t + 1) // 2


CASES = [
    Case("prompt", [(150, (40, 129, 1, 200))]),
    Case("prompt_steep", [(1000, (150,) * 6)], hq=2, hkv=1, steep=0.2),   # answers up to 750 rows from their place
    Case("prompt_at_a_tile", [(256, (70, 300))], d=64, block=64, delta=0.4),
    Case("prompt_inside_one_tile", [(5, (100, 1, 60))], d=64),
    Case("prompt_of_one", [(1, (1, 1, 200))], hq=2, hkv=2),
    Case("prompts", [(150, (40, 70)), (0, (60, 200)), (130, (3,)), (20, ())], hq=6, hkv=2, tail=50),
    Case("prompt_cap", [(150, (40, 129, 1, 200))], softcap=7.0, spread=3.0),
    Case("prompt_cap_64", [(300, (200, 90))], d=64, block=64, softcap=20.0),
    Case("prompt_high_cap", [(150, (40, 129))], hq=2, hkv=2, softcap=100.0, spread=3.0),
    Case("prompt_rising", [(150, (140, 129))], rising=True),
    Case("prompt_rising_cap", [(140, (140, 29))], d=64, rising=True, softcap=9.0),
    Case("prompt_split_group", [(140, (50, 90))], hq=40, hkv=1, d=64),
    # rows whose own keys begin inside the prefix: a tile that all rows see whole has keys of both kinds
    Case("window_over_the_prefix", [(200, window(700, 400), halfway(700, 200))]),
    Case("window_over_the_prefix_cap", [(200, window(700, 400), halfway(700, 200))], softcap=10.0, block=64),
    Case("nothing_hidden", [(150, np.zeros(400), np.maximum(np.arange(400) - 150, np.minimum(np.arange(400), 149)))], d=64),
]
each = pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)


def dev(m):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in m.items()}


@gpu
@each
def test_training_step_matches_the_formula(c):
    m = c.make()
    b = run(c, dev(m))
    ref, tol = reference(c, m, b.w.cpu())
    live = m["T"] - c.tail
    for x in ("o", "lse", "dq", "dk", "dv"):
        off = (getattr(b, x).double().cpu() - ref[x]).abs()
        bad = off - tol[x]
        bad = bad[:, :live] if x == "lse" else bad[:live]
        assert (bad <= 0).all(), (c.name, x, float(bad.nan_to_num(nan=1e9).max()), float(off.max()))


@gpu
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_answers_equal_those_of_separate_copies(softcap):
    """A prompt computed once, against a copy of it in front of every answer: outputs and the
    whole gradient."""
    hq, hkv, d, prompt, answers = 4, 2, 128, 150, (40, 129, 1, 200)
    gen = torch.Generator(device="cuda").manual_seed(0)
    cu, plen, start, pos = lf.shared_prompt_tables([prompt], [answers])
    T = int(cu[-1])
    x = [torch.randn(T, h, d, device="cuda", generator=gen).bfloat16() for h in (hq, hkv, hkv)]
    dout = torch.randn(T, hq, d, device="cuda", generator=gen).bfloat16()
    slopes = torch.tensor([0.5, 0.1, 0.02, 0.004], device="cuda")
    leaves = [t.clone().requires_grad_(True) for t in x]
    o = lazyflash_attention(*leaves, cu, T, delta=0.0, softcap=softcap, alibi_slopes=slopes, prefix_len=plen,
                            prefix_causal=True, row_start=start, positions=pos)
    o.backward(dout)
    rows, grads, lens, at = [], [], [], prompt
    for i, n in enumerate(answers):
        rows.append(torch.cat([torch.arange(prompt), torch.arange(at, at + n)]).cuda())
        grads.append(dout[rows[-1]].clone())
        if i:
            grads[-1][:prompt] = 0   # the prompt's own rows count once
        lens.append(prompt + n)
        at += n
    cu2 = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    copies = [t.clone().requires_grad_(True) for t in x]
    index = torch.cat(rows)
    o2 = lazyflash_attention(*(t[index] for t in copies), cu2, max(lens), delta=0.0, softcap=softcap, alibi_slopes=slopes)
    o2.backward(torch.cat(grads))
    last = {int(r): i for i, r in enumerate(index.tolist())}
    pick = torch.tensor([last[r] for r in range(T)], device="cuda")
    # O: P is rounded to bf16 at other references m, and O once on either side; a gradient passes
    # through bf16 once here and once for each copy
    assert (o.detach().float() - o2.detach()[pick].float()).abs().max() <= 4 * B * float(x[2].abs().max())
    for a, z in zip(leaves, copies):
        assert (a.grad.float() - z.grad.float()).norm() <= 4 * B * z.grad.float().norm()


@gpu
def test_positions_without_slopes_change_nothing():
    c = CASES[0]
    g = dev(c.make())
    a, z = run(c, g, alibi_slopes=None), run(c, g, alibi_slopes=None, positions=None)
    for x in ("o", "lse", "dk", "dv"):
        assert torch.equal(getattr(a, x), getattr(z, x))


@gpu
def test_a_captured_step_reads_the_positions_of_its_replay():
    """... and positions written between the two passes are noticed by autograd."""
    c = CASES[6]
    g = dev(c.make())
    want = run(c, g)
    desc = lf.make_desc(g["cu"], max(c.lens), g["T"], c.hq, c.hkv, c.d, c.scale, True, c.block)
    mod, o, lse = mod_of(c, g), torch.empty_like(want.o), torch.empty_like(want.lse)
    dq, dk, dv = (torch.empty_like(t) for t in (want.dq, want.dk, want.dv))
    given = g["pos"].clone()
    g["pos"].copy_(torch.arange(c.lens[0], device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lf.lf_attn_fwd_mod(desc, mod, g["q"], g["k"], g["v"], o, lse)
        lf.lf_attn_bwd_mod(desc, mod, g["q"], g["k"], g["v"], o, lse, g["dout"], None, want.w, want.kept_idx,
                           want.kept_cnt, dq, dk, dv, want.ws)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(o, want.o)
    g["pos"].copy_(given)
    graph.replay()
    lf.lf_sync_status()
    assert torch.equal(o, want.o) and torch.equal(lse, want.lse) and torch.equal(dv, want.dv)
    leaves = [g[x].clone().requires_grad_(True) for x in ("q", "k", "v")]
    out = lazyflash_attention(*leaves, g["cu"], max(c.lens), softcap=c.softcap, alibi_slopes=g["slopes"],
                              prefix_len=g["prefix"], prefix_causal=True, row_start=g["start"], positions=g["pos"])
    assert torch.equal(out, want.o)
    g["pos"].add_(0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward(g["dout"])


@gpu
@pytest.mark.parametrize("row,value", [(3, 2), (3, 4), (300, 148), (300, 301), (5, -1)])
def test_positions_that_break_their_rule_are_reported(row, value):
    c = CASES[0]
    m = c.make()
    m["pos"][row] = value
    g = dev(m)
    desc = lf.make_desc(g["cu"], max(c.lens), g["T"], c.hq, c.hkv, c.d, c.scale, True, c.block)
    o, lse = torch.empty_like(g["q"]), torch.empty(c.hq, m["T"], device="cuda")
    lf.lf_attn_fwd_mod(desc, mod_of(c, g), g["q"], g["k"], g["v"], o, lse)
    torch.cuda.synchronize()
    with pytest.raises(lf.LfError) as e:
        lf.lf_attn_fwd_mod(desc, mod_of(c, g), g["q"], g["k"], g["v"], o, lse)
    assert e.value.code == lf.LF_ERR_INVALID_ARG
    with pytest.raises(lf.LfError):
        lf.lf_sync_status()
    lf.lf_sync_status()


@gpu
def test_binding_refuses_positions_that_do_not_fit():
    c = CASES[0]
    g = dev(c.make())
    for bad in (g["pos"].long(), g["pos"].cpu(), torch.stack([g["pos"]] * 2, 1)[:, 0]):
        with pytest.raises(ValueError, match="positions"):
            mod_of(c, g, positions=bad)
    with pytest.raises(ValueError, match="positions"):
        run(c, g, positions=g["pos"][1:])


def test_positions_need_a_causal_prefix():
    lfbuild.build()
    L, d = lf.lib(), raw_desc()
    for mod, code in ((dict(positions=P), lf.LF_ERR_INVALID_ARG),
                      (dict(positions=P, prefix_len=P), lf.LF_ERR_UNSUPPORTED),
                      (dict(positions=P + 2, prefix_len=P, prefix_causal=1), lf.LF_ERR_INVALID_ARG)):
        m = lf.lf_score_mod(alibi_slopes=P, **mod)
        assert L.lf_attn_fwd_mod(ctypes.byref(d), ctypes.byref(m), *fwd_args(), None) == code
        assert L.lf_attn_bwd_mod(ctypes.byref(d), ctypes.byref(m), *bwd_args(), 1 << 30, None) == code
