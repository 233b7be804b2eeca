"""Attention with modified scores (tanh cap, distance bias, prefix / document / window /
shared-prompt masks), forward and block-sparse backward, against the formulas in 64 bits.

Tolerances, element by element, from the kernels' roundings.  u = 2^-24, b = 2^-8 (half a
step of bf16, relative).
 * A score is a sum of d products in fp32: off by at most d u sum|q_i k_i| scale, plus 8 u of
   itself and of the bias, plus, when capped, 1e-6 of the cap's derivative times score
   (ez in all).  So LSE is off by ez + 16 u |LSE| + 1e-6, and P by 2 ez + 1e-6 of itself (ep).
 * O is the average of V with weights P^ = P (1 + e), each e the rounding of P to bf16 (b)
   and ep, over their own sum: O - O_exact = sum (P^ - P) (V - O) is at most 2 (b + ep)
   sum P|V - O| <= 2 (b + ep) sqrt(sum P (V - O)^2), and rounding to bf16 adds b |O|.
 * D is <dO, O> with O's residual, so the same average of dP: off by 2 (b + ep) sum P|dP - D|
   and b^2 of |dO|.|O|; where the selection gives D, from the rounded O, by b |dO|.|O| too.
   dP is a sum of d products.  dS = w P (dP - D) (1 - tanh^2) is rounded to bf16: b + ep of
   itself, plus w P times the errors of dP and D.  dQ = scale dS K, dK = scale dS^T Q and
   dV = (w P)^T dO pass these through absolute values, add n u for their fp32 sums, and are
   rounded to bf16.
 * The plain forward divides by the exact sum of P instead: its O is off by (b + ep) sum P|V|
   + b |O|, and its D by |dO| times that.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_dense_b200 as lf
from block_sparse_attention_dense_b200 import build as lfbuild
from block_sparse_attention_dense_b200.autograd import lazyflash_attention, qk_norm_rope

U, B = 2.0 ** -24, 2.0 ** -8
gpu = pytest.mark.gpu


def documents(lens):
    """row_start of a segment made of documents of these lengths."""
    return np.concatenate([np.full(n, a) for a, n in zip(np.cumsum([0] + list(lens)), lens)] or [np.zeros(0)])


def window(n, w):
    return np.maximum(0, np.arange(n) - w + 1)


class Case:
    def __init__(self, name, lens, hq=4, hkv=2, d=128, block=128, softcap=0.0, alibi=False, prefix=None,
                 prefix_causal=False, start=None, causal=True, spread=1.5, tail=0, delta=0.2, rising=False):
        self.__dict__.update(locals())
        del self.__dict__["self"]

    @property
    def scale(self):
        return 1.0 / math.sqrt(self.d)

    def make(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        T = sum(self.lens) + self.tail

        def normal(h, s=1.0):
            return (torch.randn(T, h, self.d, generator=g) * s).to(torch.bfloat16)

        nb = max(1, max(-(-n // self.block) for n in self.lens))
        m = dict(q=normal(self.hq, self.spread), k=normal(self.hkv), v=normal(self.hkv), T=T)
        dout = torch.randn(T, self.hq, self.d, generator=g)
        size = torch.exp(1.5 * torch.randn(T // self.block + 1, self.hq, generator=g))
        m["dout"] = (dout * size[torch.arange(T) // self.block][..., None]).to(torch.bfloat16)
        m["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(self.lens)]), dtype=torch.int32)
        m["nb"] = nb
        m["slopes"] = torch.tensor([0.7 * 2.0 ** (-4 * h / self.hq) for h in range(self.hq)]) if self.alibi else None
        if self.rising:   # every other head's bias grows with the distance
            m["slopes"][1::2] *= -0.1
        m["prefix"] = None if self.prefix is None else torch.tensor(self.prefix, dtype=torch.int32)
        m["start"] = None
        if self.start is not None:
            rows = [np.asarray(s) for s in self.start] + [np.full(self.tail, -5)]   # behind the last segment: not read
            m["start"] = torch.tensor(np.concatenate(rows), dtype=torch.int32)
        return m

    def mod(self, m):
        return lf.make_score_mod(self.softcap, m["slopes"], m["prefix"], self.prefix_causal, m["start"])

    def desc(self, m, extra=0):
        return lf.make_desc(m["cu"], max(self.lens) + extra, m["T"], self.hq, self.hkv, self.d, self.scale,
                            self.causal, self.block)

    def visible(self, i):
        n = self.lens[i]
        t, u = np.arange(n)[:, None], np.arange(n)[None]
        if not self.causal:
            return torch.ones(n, n, dtype=torch.bool)
        own = u <= t
        if self.start is not None:
            own = own & (u >= np.asarray(self.start[i])[:, None])
        if self.prefix is not None:
            own = own | ((u < self.prefix[i]) & ((u <= t) if self.prefix_causal else True))
        return torch.from_numpy(own)


def reference(c, m, w=None, given_D=False, plain=False):
    """O, LSE, dQ, dK, dV of the formulas in 64 bits and how far the kernels' may be off.
    w [nseq][hq][nb]: block weights (None: forward only); given_D: D is the selection's;
    plain: the tolerances of the plain attention."""
    q, k, v, do = (m[x].double() for x in ("q", "k", "v", "dout"))
    out = {x: torch.zeros_like(m[y].double()) for x, y in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
    out["lse"] = torch.zeros(c.hq, m["T"], dtype=torch.float64)
    tol = {x: t.clone() for x, t in out.items()}
    G = c.hq // c.hkv
    at = 0
    for i, n in enumerate(c.lens):
        r = slice(at, at + n)
        at += n
        if n == 0:
            continue
        see = c.visible(i)
        far = (torch.arange(n)[:, None] - torch.arange(n)[None]).abs().double()
        for h in range(c.hq):
            qh, kh, vh, g = q[r, h], k[r, h // G], v[r, h // G], h // G
            x = qh @ kh.T * c.scale
            ez = c.d * U * c.scale * (qh.abs() @ kh.abs().T) + 8 * U * x.abs()
            z, damp = x, torch.ones_like(x)
            if c.softcap:
                th = torch.tanh(x / c.softcap)
                z, damp = c.softcap * th, 1 - th * th
                ez = ez * damp + 1e-6 * z.abs()
            if c.alibi:
                bias = float(m["slopes"][h]) * far
                z = z - bias
                ez = ez + 8 * U * bias
            z = z.masked_fill(~see, -math.inf)
            ez = ez.masked_fill(~see, 0.0).amax(1, keepdim=True)
            lse = torch.logsumexp(z, 1, keepdim=True)
            p = torch.exp(z - lse)
            ep = 2 * ez + 1e-6
            o = p @ vh
            out["o"][r, h], out["lse"][h, r] = o, lse[:, 0]
            if plain:
                eo = (B + ep) * (p @ vh.abs()) + B * o.abs()
            else:
                eo = 2 * (B + ep) * (p @ vh.square() - o.square()).clamp(min=0).sqrt() + (B + 8 * U) * o.abs()
            tol["o"][r, h] = eo
            tol["lse"][h, r] = (ez + 16 * U * lse.abs() + 1e-6)[:, 0]
            if w is None:
                continue
            wr = w[i, h, torch.arange(n) // c.block].double()[:, None]
            dor = do[r, h]
            dp, D = dor @ vh.T, (dor * o).sum(1, keepdim=True)
            ds = wr * p * (dp - D) * damp
            edp = c.d * U * (dor.abs() @ vh.abs().T)
            if plain:
                eD = (dor.abs() * eo).sum(1, keepdim=True)
            else:
                eD = 2 * (B + ep) * (p * (dp - D).abs()).sum(1, keepdim=True) + edp.amax(1, keepdim=True)
                eD += ((B if given_D else B * B) + c.d * U) * (dor.abs() * o.abs()).sum(1, keepdim=True)
            eds = (B + ep + 4 * U) * ds.abs() + wr * p * damp * (eD + edp)
            if c.softcap:
                eds = eds + wr * p * (dp - D).abs() * 2 * (ez / c.softcap + 1e-6)
            wp = wr * p
            out["dq"][r, h] = c.scale * ds @ kh
            out["dk"][r, g] += c.scale * ds.T @ qh
            out["dv"][r, g] += wp.T @ dor
            sums = n * c.hq * U
            tol["dq"][r, h] = c.scale * (eds + sums * ds.abs()) @ kh.abs()
            tol["dk"][r, g] += c.scale * (eds + sums * ds.abs()).T @ qh.abs()
            tol["dv"][r, g] += ((B + ep + sums) * wp).T @ dor.abs()
    for x in ("dq", "dk", "dv"):
        tol[x] += B * out[x].abs() + 1e-30
    return out, tol


def dev(m):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in m.items()}


def run(c, g, give_D=False, seed=3, extra=0):
    desc, mod = c.desc(g, extra), c.mod(g)
    b = lf.Buffers(desc)
    o_low = None if give_D else torch.empty_like(b.o)
    for t in (b.o, b.dq, b.dk, b.dv, b.lse):
        t.fill_(float("nan"))
    lf.lf_attn_fwd_mod(desc, mod, g["q"], g["k"], g["v"], b.o, b.lse, o_low)
    lf.lf_block_select(desc, g["dout"], b.o, c.delta, seed, 0, 0, b.norm, b.D if give_D else None, b.tau, b.w,
                       b.keep, b.kept_idx, b.kept_cnt)
    b.ws.fill_(255)
    lf.lf_attn_bwd_mod(desc, mod, g["q"], g["k"], g["v"], b.o, b.lse, g["dout"], b.D if give_D else None, b.w,
                       b.kept_idx, b.kept_cnt, b.dq, b.dk, b.dv, b.ws, o_low)
    lf.lf_sync_status()
    torch.cuda.synchronize()
    b.o_low = o_low
    return b


def check(c, m, b, parts=("o", "lse", "dq", "dk", "dv"), given_D=False):
    ref, tol = reference(c, m, b.w.cpu() if "dq" in parts else None, given_D)
    live = m["T"] - c.tail
    for x in parts:
        got, want, t = getattr(b, x).double().cpu(), ref[x], tol[x]
        if x == "lse":
            got, want, t = got[:, :live], want[:, :live], t[:, :live]
        else:
            got, want, t = got[:live], want[:live], t[:live]
        off = (got - want).abs()
        assert (off <= t).all(), (c.name, x, float((off - t).nan_to_num(nan=1e9).max()), float(off.max()))


PROMPT = np.concatenate([np.zeros(150), np.full(70, 150), np.full(1, 220), np.full(130, 221), np.full(128, 351)])
CASES = [
    Case("cap", (300, 1, 129), softcap=8.0, spread=3.0),
    Case("cap_beyond_the_fit", (257, 64), hq=2, hkv=2, d=64, softcap=2.0, spread=4.0),   # tanh near 1
    Case("cap_far_away", (200,), softcap=1e6),
    Case("cap_not_causal", (300, 200), hq=2, hkv=1, softcap=10.0, causal=False),
    Case("cap_64", (520,), d=64, block=64, softcap=6.0, delta=0.4),
    Case("bias", (300, 1, 129), alibi=True),
    Case("bias_not_causal", (300, 200), hq=4, hkv=1, d=64, alibi=True, causal=False),
    Case("bias_64", (400,), hq=8, hkv=2, block=64, alibi=True, delta=0.4),
    Case("prefix", (300, 300, 129, 260, 5, 131), prefix=(100, 0, 129, 128, 1, 1000)),
    Case("prefix_across_tiles", (700, 390), d=64, prefix=(530, 129)),
    Case("prefix_64", (500,), block=64, prefix=(333,), delta=0.4),
    Case("prefix_bias", (400, 300), hq=2, hkv=2, alibi=True, prefix=(200, 257)),
    Case("prefix_cap", (400, 300), d=64, softcap=5.0, prefix=(131, 127)),
    Case("documents", (700, 256), start=(documents((1, 127, 128, 129, 200, 3, 112)), documents((128, 128)))),
    Case("documents_64", (700,), d=64, block=64, start=(documents((300, 60, 1, 1, 338)),), delta=0.4),
    Case("window_1", (260,), start=(window(260, 1),)),
    Case("window", (700, 129), start=(window(700, 37), window(129, 300))),
    Case("window_tile", (600,), d=64, start=(window(600, 128),), softcap=4.0, spread=3.0),
    Case("window_wide_bias", (900,), hq=2, hkv=1, start=(window(900, 300),), alibi=True),
    Case("window_and_kept_prefix", (800, 300), prefix=(4, 140), prefix_causal=True,
         start=(window(800, 200), window(300, 20))),
    Case("prompt", (479,), prefix=(150,), prefix_causal=True, start=(PROMPT,)),
    Case("prompt_twice", (479, 300), hq=6, hkv=2, d=64, prefix=(150, 0), prefix_causal=True,
         start=(PROMPT, documents((100, 200)))),
    Case("prompt_64", (479,), block=64, prefix=(150,), prefix_causal=True, start=(PROMPT,), delta=0.4),
    Case("prefix_seen_whole_and_documents", (479,), prefix=(150,), start=(PROMPT,)),
    Case("everything", (479, 257), softcap=7.0, alibi=True, prefix=(150, 60), prefix_causal=True,
         start=(PROMPT, window(257, 90)), spread=3.0),
    Case("everything_64", (479, 257), d=64, block=64, softcap=7.0, alibi=True, prefix=(150, 60),
         start=(PROMPT, window(257, 90)), delta=0.4),
    Case("split_group", (300, 170), hq=40, hkv=1, d=64, softcap=6.0, prefix=(20, 5), prefix_causal=True,
         start=(window(300, 100), window(170, 64)), alibi=True),
    Case("odd_group", (333, 200), hq=6, hkv=2, softcap=9.0, alibi=True),
    Case("many_segments", (0, 1, 127, 128, 129, 256, 300, 5) * 5, hq=2, hkv=1, d=64, block=64, softcap=5.0,
         start=[window(n, 70) for n in (0, 1, 127, 128, 129, 256, 300, 5) * 5]),
    Case("rising_bias", (400, 129), alibi=True, rising=True),
    Case("rising_bias_capped", (300, 260), d=64, alibi=True, rising=True, softcap=9.0, start=(window(300, 200), documents((130, 130)))),
    Case("high_cap_bias", (300, 200), alibi=True, softcap=100.0, spread=3.0, prefix=(20, 150)),
    Case("high_cap", (520,), hq=2, hkv=2, softcap=60.0, spread=6.0, start=(window(520, 256),)),
    Case("padded", (200, 100), alibi=True, start=(window(200, 150), documents((50, 50))), tail=90),
]
# every compiled variant: which modifiers x head dim x block rows
for bits in range(1, 8):
    for d in (64, 128):
        for blk in (64, 128):
            CASES.append(Case("variant_%d_%d_%d" % (bits, d, blk), (290, 150), hq=4, hkv=2, d=d, block=blk,
                              softcap=6.0 if bits & 1 else 0.0, alibi=bool(bits & 2), spread=2.5, delta=0.3,
                              **(dict(prefix=(70, 0), prefix_causal=True,
                                      start=(documents((130, 100, 60)), window(150, 33))) if bits & 4 else {})))
each = pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
NAMED = {c.name: c for c in CASES}


@gpu
@each
def test_forward_matches_the_formula(c):
    m = c.make()
    g = dev(m)
    desc = c.desc(g)
    o = torch.full_like(g["q"], 7.0)
    lse = torch.full((c.hq, m["T"]), 7.0, device="cuda")
    lf.lf_attn_fwd_mod(desc, c.mod(g), g["q"], g["k"], g["v"], o, lse)
    lf.lf_sync_status()

    class Got:
        pass

    Got.o, Got.lse = o, lse
    check(c, m, Got, ("o", "lse"))
    if c.tail:   # rows behind the last segment stay as they were
        assert (o[-c.tail:] == 7).all() and (lse[:, -c.tail:] == 7).all()


@gpu
@each
def test_training_step_matches_the_formula(c):
    m = c.make(1)
    check(c, m, run(c, dev(m)))


@gpu
@pytest.mark.parametrize("c", [NAMED["cap"], NAMED["window_and_kept_prefix"], NAMED["prompt_64"], NAMED["everything_64"]], ids=lambda c: c.name)
def test_row_products_given_by_the_selection(c):
    m = c.make(2)
    check(c, m, run(c, dev(m), give_D=True), given_D=True)


@gpu
@pytest.mark.parametrize("c", [NAMED["cap"], NAMED["bias"], NAMED["documents"], NAMED["everything"]], ids=lambda c: c.name)
def test_residual_of_the_rounding(c):
    """o + o_low is the unrounded O, o a nearest bf16 of it: o_low is at most half a step of o
    (a power of two, so its own rounding to bf16 cannot pass it; on the tie o + o_low may
    round to the other neighbour, which is why the sum is not compared with o)."""
    m = c.make(9)
    b = run(c, dev(m))
    live = m["T"] - c.tail
    o, low = b.o[:live].double(), b.o_low[:live].double()
    half_step = torch.exp2(torch.floor(torch.log2(o.abs())) - 8)
    assert (low.abs() <= half_step).all()
    assert (low != 0).double().mean() > 0.9


@gpu
def test_a_row_on_one_key_gets_no_gradient():
    """Softmax over one visible key is 1 whatever its score: dQ = 0, O = v, and dS = 0 but
    for the errors of fp32 (D and dP are two sums of the same products)."""
    c = Case("one", (40,), start=(np.arange(40),), softcap=20.0, alibi=True, spread=4.0)
    m = c.make()
    b = run(c, dev(m))
    assert torch.equal(b.o.cpu(), m["v"].repeat_interleave(2, 1))
    exact = (m["dout"].double().abs() * m["v"].double().abs().repeat_interleave(2, 1)).sum(2)   # [T, hq]
    k = m["k"].double().abs().repeat_interleave(2, 1).amax(2)
    w = torch.cat([b.w[0].cpu().double().T[[0]]] * 40)
    assert (b.dq.double().cpu().abs().amax(2) <= 2 * c.d * U * w * exact * k * c.scale).all()


@gpu
@pytest.mark.parametrize("c", [NAMED["documents"], NAMED["prompt"], NAMED["many_segments"]], ids=lambda c: c.name)
def test_max_seqlen_above_the_longest_segment(c):
    m = c.make(3)
    check(c, m, run(c, dev(m), extra=333))


@gpu
def test_a_mask_that_hides_nothing_is_the_plain_attention():
    c = Case("plain", (300, 129), start=(np.zeros(300), np.zeros(129)), delta=0.0)
    m = c.make()
    g = dev(m)
    b = run(c, g)
    desc = c.desc(g)
    p = lf.Buffers(desc)
    lf.lazyflash_step(desc, g["q"], g["k"], g["v"], g["dout"], 0.0, 3, 0, p)
    # the same scores, but the tiles in another order: the row's reference m differs, and with
    # it where bf16 rounds each P, so each side has its own tolerance; in the row's sum of n <= 300 positive terms, kept in fp32, each addition, each exp2 (4 u) and
    # each exponent (60 u of 1, |z - m| < 60) is off by as much on either side
    ours, plain = reference(c, m, b.w.cpu())[1], reference(c, m, b.w.cpu(), plain=True)[1]
    assert ((b.o.double() - p.o.double()).abs().cpu() <= ours["o"] + plain["o"]).all()
    assert ((b.lse - p.lse).abs() <= 2 * (300 + 64) * U + 8 * U * p.lse.abs()).all()
    for x in ("dq", "dk", "dv"):   # dQ is summed by atomics, in any order
        # dS and P of the backward come from LSE and D; D from O (see the tolerances above)
        a, z = getattr(b, x).double().cpu(), getattr(p, x).double().cpu()
        assert ((a - z).abs() <= ours[x] + plain[x]).all()


@gpu
@pytest.mark.parametrize("c", [NAMED["documents"], NAMED["window"], NAMED["window_and_kept_prefix"], NAMED["prompt"], NAMED["everything"]], ids=lambda c: c.name)
def test_hidden_keys_do_not_matter(c):
    """Bit for bit: keys and values that a row does not see may be anything finite, and the
    output gradient of rows that do not see a key does not reach it."""
    m = c.make(4)
    g = dev(m)
    row, seg = c.lens[0] - 1, 0
    see = c.visible(seg)
    hidden = (~see[row]).nonzero()[:, 0].cuda()
    assert len(hidden)
    first = run(c, g)
    h = dict(g, k=g["k"].clone(), v=g["v"].clone())
    h["k"][hidden] = 300.0
    h["v"][hidden] = -1e4
    o, lse = torch.empty_like(first.o), torch.empty_like(first.lse)
    lf.lf_attn_fwd_mod(c.desc(h), c.mod(h), h["q"], h["k"], h["v"], o, lse)
    assert torch.equal(o[row], first.o[row]) and torch.equal(lse[:, row], first.lse[:, row])
    # all rows but those that see key 0 get another gradient
    key = int(hidden[-1])
    blind = (~see[:, key]).nonzero()[:, 0].cuda()
    h = dict(g, dout=g["dout"].clone())
    h["dout"][blind] *= 1.5
    desc, mod = c.desc(g), c.mod(g)
    got = []
    for x in (g, h):
        ones = torch.ones_like(first.w)
        nb = first.w.shape[2]
        idx = torch.arange(nb, dtype=torch.int32, device="cuda").expand_as(first.kept_idx).contiguous()
        cnt = torch.tensor([-(-n // c.block) for n in c.lens], dtype=torch.int32, device="cuda")[:, None]
        dq, dk, dv = (torch.empty_like(t) for t in (first.dq, first.dk, first.dv))
        lf.lf_attn_bwd_mod(desc, mod, x["q"], x["k"], x["v"], first.o, first.lse, x["dout"], None, ones, idx,
                           cnt.expand(-1, c.hq).contiguous(), dq, dk, dv, first.ws)
        got.append((dk[key].clone(), dv[key].clone()))
    lf.lf_sync_status()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@gpu
@pytest.mark.parametrize("c", [NAMED["cap"], NAMED["bias_not_causal"], NAMED["prefix_bias"], NAMED["everything"]], ids=lambda c: c.name)
def test_gradient_matches_differences(c):
    """The weighted sum sum(w dO O) along a direction that agrees with the kernel's gradient
    in every sign, by central differences of the formula in 64 bits (their own error is the
    third derivative's, under 1e-5 of the sum at this step)."""
    m = c.make(5)
    b = run(c, dev(m))
    ref, tol = reference(c, m, b.w.cpu())
    weight = torch.zeros(m["T"], c.hq, dtype=torch.float64)
    at = 0
    for i, n in enumerate(c.lens):
        weight[at:at + n] = b.w[i].cpu().double().T[torch.arange(n) // c.block]
        at += n
    wdo = m["dout"].double() * weight[..., None]
    gen = torch.Generator().manual_seed(1)
    for x, dx in (("q", b.dq), ("k", b.dk), ("v", b.dv)):
        dx = dx.cpu().double()
        v = torch.rand(dx.shape, generator=gen, dtype=torch.float64) * dx.sign()
        step = 1e-4
        f = [(wdo * reference(c, {**m, x: m[x].double() + s * v})[0]["o"]).sum() for s in (step, -step)]
        want = (f[0] - f[1]) / (2 * step)
        assert abs((dx * v).sum() - want) <= (tol["d" + x] * v.abs()).sum() + 1e-5 * (dx * v).abs().sum()


@gpu
def test_layer_with_a_shared_prompt_equals_separate_copies():
    """Norms, rotation, attention and the whole gradient of a batch whose answers share one
    prompt, against the same batch with the prompt repeated in front of every answer."""
    torch.manual_seed(0)
    hq, hkv, d, prompt, answers = 4, 2, 128, 150, (40, 129, 1, 200)
    cu, plen, start, pos = lf.shared_prompt_tables([prompt], [answers])
    T = int(cu[-1])
    assert T == prompt + sum(answers)
    qkv = torch.randn(T, hq + 2 * hkv, d, device="cuda").bfloat16()
    dout = torch.randn(T, hq, d, device="cuda").bfloat16()
    table = lf.rope_cos_sin(1024, d)
    weights = [(1 + 0.2 * torch.randn(d, device="cuda")).requires_grad_(True) for _ in range(2)]

    def layer(x, cu, longest, positions, **mask):
        q, k = qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], *weights, table, cu, positions)
        return lazyflash_attention(q, k, x[:, hq + hkv:].contiguous(), cu, longest, delta=0.0, softcap=20.0, **mask)

    x = qkv.clone().requires_grad_(True)
    o = layer(x, cu, T, pos, prefix_len=plen, prefix_causal=True, row_start=start)
    # the prompt repeated: its own rows' output gradient counts in the first copy only
    rows, grads, lens = [], [], []
    at = prompt
    for i, n in enumerate(answers):
        rows.append(torch.cat([torch.arange(prompt), torch.arange(at, at + n)]))
        gr = dout[rows[-1].cuda()].clone()
        if i:
            gr[:prompt] = 0
        grads.append(gr)
        lens.append(prompt + n)
        at += n
    index = torch.cat(rows).cuda()
    y = qkv.clone().requires_grad_(True)
    cu2 = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    o2 = layer(y[index], cu2, max(lens), None)
    last = {int(r): i for i, r in enumerate(index.tolist())}
    pick = torch.tensor([last[r] for r in range(T)], device="cuda")
    # the same keys, in tiles of another place: P is rounded the same, sums are in another order
    assert (o.detach().float() - o2.detach()[pick].float()).abs().max() <= 2 * B * float(o.detach().abs().max())
    o.backward(dout)
    wg = [w.grad.clone() for w in weights]
    for w in weights:
        w.grad = None
    o2.backward(torch.cat(grads))
    # a gradient passes through bf16 dQ, dK once here, and there once for each copy
    for a, z in ((x.grad, y.grad), (wg[0], weights[0].grad), (wg[1], weights[1].grad)):
        assert (a.float() - z.float()).norm() <= 2 * B * z.float().norm() * 2


@gpu
def test_an_empty_modifier_is_the_plain_attention():
    c = Case("empty", (200, 57))
    m = c.make()
    g = dev(m)
    b, desc = run(c, g), c.desc(g)
    p = lf.Buffers(desc)
    lf.lazyflash_step(desc, g["q"], g["k"], g["v"], g["dout"], c.delta, 3, 0, p)
    assert torch.equal(b.o, p.o) and torch.equal(b.lse, p.lse) and (b.o_low == 0).all()
    assert torch.equal(b.dk, p.dk) and torch.equal(b.dv, p.dv)
    assert (b.dq.float() - p.dq.float()).norm() <= B * p.dq.float().norm()


@gpu
def test_slices_of_longer_arrays_and_two_streams_at_once():
    """The modifier's arrays need only four bytes of alignment, and two calls with buffers of
    their own may run at the same time."""
    c = NAMED["everything"]
    m = c.make()
    g = dev(m)
    want = run(c, g)
    for x in ("slopes", "start", "prefix"):
        g[x] = torch.cat([g[x][:1], g[x]])[1:]
        assert g[x].data_ptr() % 16
    desc, mod = c.desc(g), c.mod(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            b = lf.Buffers(desc)
            low = torch.empty_like(b.o)
            for _ in range(3):
                lf.lf_attn_fwd_mod(desc, mod, g["q"], g["k"], g["v"], b.o, b.lse, low)
                lf.lf_attn_bwd_mod(desc, mod, g["q"], g["k"], g["v"], b.o, b.lse, g["dout"], None, want.w,
                                   want.kept_idx, want.kept_cnt, b.dq, b.dk, b.dv, b.ws, low)
            outs.append(b)
    torch.cuda.synchronize()
    lf.lf_sync_status()
    for b in outs:
        assert torch.equal(b.o, want.o) and torch.equal(b.lse, want.lse)
        assert torch.equal(b.dk, want.dk) and torch.equal(b.dv, want.dv)
        assert (b.dq.float() - want.dq.float()).norm() <= B * want.dq.float().norm()


@gpu
def test_autograd_passes_the_modifier_on():
    c = NAMED["everything"]
    m = c.make(6)
    g = dev(m)
    q, k, v = (g[x].clone().requires_grad_(True) for x in ("q", "k", "v"))
    o = lazyflash_attention(q, k, v, g["cu"], max(c.lens), delta=c.delta, seed=3, step=0, block_q=c.block,
                            softcap=c.softcap, alibi_slopes=g["slopes"], prefix_len=g["prefix"],
                            prefix_causal=c.prefix_causal, row_start=g["start"])
    o.backward(g["dout"])
    b = run(c, g)
    assert torch.equal(o, b.o) and torch.equal(v.grad, b.dv) and torch.equal(k.grad, b.dk)
    assert (q.grad.float() - b.dq.float()).norm() <= B * b.dq.float().norm()


@gpu
def test_side_stream_and_captured_graph():
    c = NAMED["everything_64"]
    m = c.make(7)
    g = dev(m)
    b = run(c, g)
    desc, mod = c.desc(g), c.mod(g)
    o, lse = torch.empty_like(b.o), torch.empty_like(b.lse)
    dq, dk, dv = (torch.empty_like(t) for t in (b.dq, b.dk, b.dv))

    def step():
        lf.lf_attn_fwd_mod(desc, mod, g["q"], g["k"], g["v"], o, lse)
        lf.lf_attn_bwd_mod(desc, mod, g["q"], g["k"], g["v"], o, lse, g["dout"], None, b.w, b.kept_idx, b.kept_cnt,
                           dq, dk, dv, b.ws)

    def same(want):
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        for a, z in zip((dq, dk, dv), want[2:]):
            assert (a.float() - z.float()).norm() <= 2 * B * z.float().norm()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    same((b.o, b.lse, b.dq, b.dk, b.dv))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g["q"].copy_(c.make(8)["q"])
    if g["start"] is not None:   # another mask in the same place
        g["start"][: c.lens[0]] = torch.from_numpy(window(c.lens[0], 50)).int().cuda()
    step()
    want = [t.clone() for t in (o, lse, dq, dk, dv)]
    for t in (o, lse, dq, dk, dv):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    same(want)


@gpu
@pytest.mark.parametrize("what", ["negative", "later", "falls", "prefix"])
def test_masks_that_break_their_rules_are_reported(what):
    c = Case("bad", (300,), prefix=(10,), prefix_causal=True, start=(window(300, 100),))
    m = c.make()
    if what == "negative":
        m["start"][5] = -1
    elif what == "later":
        m["start"][200] = 201
    elif what == "falls":
        m["start"][200] = 90
    else:
        m["prefix"][0] = -3
    g = dev(m)
    o, lse = torch.empty_like(g["q"]), torch.empty(c.hq, 300, device="cuda")
    lf.lf_attn_fwd_mod(c.desc(g), c.mod(g), g["q"], g["k"], g["v"], o, lse)
    torch.cuda.synchronize()
    with pytest.raises(lf.LfError) as e:   # the next call, without a synchronization
        lf.lf_attn_fwd_mod(c.desc(g), c.mod(g), g["q"], g["k"], g["v"], o, lse)
    assert e.value.code == lf.LF_ERR_INVALID_ARG
    with pytest.raises(lf.LfError):
        lf.lf_sync_status()
    lf.lf_sync_status()


@gpu
def test_long_windowed_rows():
    """12,000 rows: many steps per query tile with the two tiles' runs apart, sampled rows."""
    c = Case("long", (12000,), hq=2, hkv=1, prefix=(200,), prefix_causal=True, softcap=12.0, spread=3.0,
             start=(np.maximum(documents((5000, 40, 3000, 3960)), window(12000, 2500)),))
    m = c.make()
    g = dev(m)
    o, lse = torch.empty_like(g["q"]), torch.empty(c.hq, 12000, device="cuda")
    lf.lf_attn_fwd_mod(c.desc(g), c.mod(g), g["q"], g["k"], g["v"], o, lse)
    lf.lf_sync_status()
    q, k, v = (g[x].double() for x in ("q", "k", "v"))
    start = g["start"].long()
    u = torch.arange(12000, device="cuda")
    for t in (0, 127, 128, 199, 200, 255, 4999, 5000, 5039, 5040, 5041, 7600, 8039, 8040, 8192, 11999):
        see = ((u >= start[t]) & (u <= t)) | ((u < 200) & (u <= t))
        for h in range(2):
            x = (k[see, 0] @ q[t, h]) * c.scale
            z = 12.0 * torch.tanh(x / 12.0)
            ez = float(c.d * U * c.scale * (k[see, 0].abs() @ q[t, h].abs()).max()) + 2e-5
            assert abs(float(lse[h, t]) - float(torch.logsumexp(z, 0))) <= ez + 1e-5
            p = torch.softmax(z, 0)
            ref = p @ v[see, 0]
            assert ((o[t, h].double() - ref).abs() <= (B + 2 * ez) * (p @ v[see, 0].abs()) + B * ref.abs()).all()


# ---- refusals, on the host ----
@pytest.fixture(scope="module")
def L():
    lfbuild.build()
    return lf.lib()


P = 0x10000


def raw_desc(**kw):
    base = dict(nseq=1, cu_seqlens=0x1000, max_seqlen=256, total_tokens=256, hq=4, hkv=2, d=128,
                softmax_scale=0.088, causal=1, block_q=128)
    base.update(kw)
    return lf.lf_attn_desc(**base)


@pytest.mark.parametrize("mod,causal,code", [
    (dict(softcap=-1.0), 1, lf.LF_ERR_INVALID_ARG),
    (dict(softcap=1e-4), 1, lf.LF_ERR_INVALID_ARG),
    (dict(softcap=float("inf")), 1, lf.LF_ERR_INVALID_ARG),
    (dict(softcap=float("nan")), 1, lf.LF_ERR_INVALID_ARG),
    (dict(alibi_slopes=P + 2), 1, lf.LF_ERR_INVALID_ARG),
    (dict(row_start=P + 1), 1, lf.LF_ERR_INVALID_ARG),
    (dict(prefix_len=P, prefix_causal=2), 1, lf.LF_ERR_INVALID_ARG),
    (dict(prefix_causal=1), 1, lf.LF_ERR_INVALID_ARG),
    (dict(prefix_len=P), 0, lf.LF_ERR_UNSUPPORTED),
    (dict(row_start=P), 0, lf.LF_ERR_UNSUPPORTED),
])
def test_bad_modifiers_rejected(L, mod, causal, code):
    d, m = raw_desc(causal=causal), lf.lf_score_mod(**mod)
    assert L.lf_attn_fwd_mod(ctypes.byref(d), ctypes.byref(m), *fwd_args(), None) == code
    assert L.lf_attn_bwd_mod(ctypes.byref(d), ctypes.byref(m), *bwd_args(), 1 << 30, None) == code


def fwd_args(**kw):
    return list(dict(dict(q=P, k=P, v=P, o=P, o_low=P, lse=P), **kw).values())


def bwd_args(**kw):
    return list(dict(dict(q=P, k=P, v=P, o=P, o_low=P, lse=P, dout=P, D=None, w=P, idx=P, cnt=P, dq=P, dk=P, dv=P, ws=P),
                     **kw).values())


def test_missing_modifier_operands_and_workspace_rejected(L):
    d, m = raw_desc(), lf.lf_score_mod(softcap=5.0, row_start=P)

    def fwd(desc=d, mod=ctypes.byref(m), **kw):
        return L.lf_attn_fwd_mod(ctypes.byref(desc), mod, *fwd_args(**kw), None)

    def bwd(nbytes=1 << 30, desc=d, **kw):
        return L.lf_attn_bwd_mod(ctypes.byref(desc), ctypes.byref(m), *bwd_args(**kw), nbytes, None)

    assert fwd(mod=None) == lf.LF_ERR_INVALID_ARG
    for x in ("q", "k", "v", "o", "lse"):
        assert fwd(**{x: None}) == lf.LF_ERR_INVALID_ARG and fwd(**{x: P + 8}) == lf.LF_ERR_INVALID_ARG
    assert fwd(o_low=P + 8) == lf.LF_ERR_INVALID_ARG
    assert fwd(raw_desc(d=96)) == lf.LF_ERR_UNSUPPORTED
    for x in ("q", "k", "v", "o", "lse", "dout", "w", "idx", "cnt", "dq", "dk", "dv"):
        assert bwd(**{x: None}) == lf.LF_ERR_INVALID_ARG, x
    assert bwd(D=P) == lf.LF_ERR_INVALID_ARG                 # D and the residual it would be computed with
    assert bwd(o_low=P + 8) == lf.LF_ERR_INVALID_ARG
    n = ctypes.c_size_t(0)
    assert L.lf_workspace_size(ctypes.byref(d), lf.LF_WS_BWD, ctypes.byref(n)) == 0
    assert bwd(n.value - 1) == lf.LF_ERR_WORKSPACE and bwd(ws=None) == lf.LF_ERR_WORKSPACE
    none = raw_desc(total_tokens=0, max_seqlen=0)   # an empty batch, whose tensors have no address
    assert fwd(none, **dict.fromkeys(("q", "k", "v", "o", "o_low", "lse"))) == 0
    assert bwd(0, none, **dict.fromkeys(("q", "k", "v", "o", "o_low", "lse", "dout", "dq", "dk", "dv", "ws"))) == 0


def test_shared_prompt_tables_on_the_host():
    cu, plen, start, pos = lf.shared_prompt_tables([3, 0], [[2, 1], [2]], device="cpu")
    assert cu.tolist() == [0, 6, 8] and plen.tolist() == [3, 0]
    assert start.tolist() == [0, 0, 0, 3, 3, 5, 0, 0] and pos.tolist() == [0, 1, 2, 3, 4, 3, 0, 1]
    with pytest.raises(ValueError):
        lf.shared_prompt_tables([3], [[1], [2]], device="cpu")


def test_slopes_that_ask_for_a_gradient_are_refused():
    x, slopes = torch.zeros(4, 2, 64), torch.zeros(2, requires_grad=True)
    with pytest.raises(ValueError, match="slopes"):
        lazyflash_attention(x, x, x, torch.tensor([0, 4]), 4, alibi_slopes=slopes)


@gpu
def test_binding_refuses_what_does_not_fit():
    c = NAMED["everything"]
    g = dev(c.make())
    desc, mod = c.desc(g), c.mod(g)
    o, lse = torch.empty_like(g["q"]), torch.empty(c.hq, g["T"], device="cuda")
    for bad in (dict(q=g["q"].float()), dict(k=g["k"][:, :1]), dict(v=g["v"].transpose(0, 1).contiguous().transpose(0, 1)),
                dict(q=g["q"].cpu())):
        a = {**g, **bad}
        with pytest.raises(ValueError):
            lf.lf_attn_fwd_mod(desc, mod, a["q"], a["k"], a["v"], o, lse)
    for kw in (dict(alibi_slopes=g["slopes"][:2]), dict(row_start=g["start"][1:]), dict(prefix_len=g["prefix"][:1])):
        with pytest.raises(ValueError):
            lf.lf_attn_fwd_mod(desc, lf.make_score_mod(**kw), g["q"], g["k"], g["v"], o, lse)
    for kw in (dict(alibi_slopes=g["slopes"].double()), dict(row_start=g["start"].long()), dict(prefix_len=g["prefix"].cpu())):
        with pytest.raises(ValueError):
            lf.make_score_mod(**kw)
    with pytest.raises(ValueError):
        lf.lf_attn_fwd_mod(desc, mod, g["q"], g["k"], g["v"], o, lse.double())
    b = lf.Buffers(desc)
    args = [g["q"], g["k"], g["v"], o, lse, g["dout"], None, b.w, b.kept_idx, b.kept_cnt, b.dq, b.dk, b.dv, b.ws]
    for i, bad in ((6, b.D.double()), (7, b.w[:, :1]), (8, b.kept_idx.long()), (10, b.dk), (13, b.ws.cpu())):
        with pytest.raises(ValueError):
            lf.lf_attn_bwd_mod(desc, mod, *args[:i], bad, *args[i + 1:])
