"""Training steps with modified scores over thousands of rows and enough heads for more than
eight waves of CTAs, where the kernels walk their grids in the other order, against the
formulas in 64 bits: every row and key of sampled heads.

Tolerances as in test_score_mods.py, with what grows with the length n counted: a row's sum of
P is 32 additions in a lane and one per KV tile, so LSE and P are off by (64 + n / 128) u more;
dQ is a sum over n keys and dK, dV over n rows of every head of the group, in fp32."""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_dense_b200 as lf
from test_score_mods import B, U, window

gpu = pytest.mark.gpu


class Case:
    def __init__(self, name, n, hq, hkv, d, block, heads, softcap=0.0, alibi=False, prefix=0, start=None, pos=None):
        self.__dict__.update(locals())
        del self.__dict__["self"]
        self.scale = 1.0 / math.sqrt(d)


def prompt(p, answers):
    _, _, start, pos = lf.shared_prompt_tables([p], [answers], device="cpu")
    return dict(n=p + sum(answers), prefix=p, start=start.numpy(), pos=pos.numpy())


# heads: sampled, whole groups
CASES = [
    Case("cap", 10100, 32, 32, 64, 128, (0, 17), softcap=30.0),
    Case("all_window_and_kept_prefix", 9900, 32, 32, 64, 64, (3, 31), softcap=15.0, alibi=True, prefix=300, start=window(9900, 2500)),
    Case("window_and_kept_prefix", 19300, 32, 8, 128, 128, (8, 9, 10, 11), prefix=200, start=window(19300, 6000)),
    Case("prompt_bias_positions", hq=32, hkv=32, d=64, block=128, heads=(1, 30), alibi=True, **prompt(2000, (300,) * 20 + (1700, 5))),
]


def reference(c, m, b):
    """Yields name, result, value, tolerance of every sampled head (of the group for dK, dV)."""
    n, G = c.n, c.hq // c.hkv
    u = torch.arange(n, device="cuda")[None]
    row_err = (64 + n / 128) * U
    for g in sorted({h // G for h in c.heads}):
        k, v = m["k"][:, g].double(), m["v"][:, g].double()
        dk, dv, tk, tv = (torch.zeros(n, c.d, dtype=torch.float64, device="cuda") for _ in range(4))
        for h in range(g * G, g * G + G):
            for r0 in range(0, n, 2048):
                t = torch.arange(r0, min(n, r0 + 2048), device="cuda")[:, None]
                r = slice(r0, min(n, r0 + 2048))
                q, do = m["q"][r, h].double(), m["dout"][r, h].double()
                see = u <= t
                if c.start is not None:
                    see = see & ((u >= m["start"][r, None]) | (u < c.prefix))
                x = q @ k.T * c.scale
                ez = c.d * U * c.scale * (q.abs() @ k.abs().T) + 8 * U * x.abs()
                z, damp = x, 1.0
                if c.softcap:
                    th = torch.tanh(x / c.softcap)
                    z, damp = c.softcap * th, 1 - th * th
                    ez = ez * damp + 1e-6 * z.abs()
                if c.alibi:
                    far = t - u
                    if c.pos is not None:
                        far = torch.where(u < c.prefix, m["pos"][r, None] - u, far)
                    bias = float(m["slopes"][h]) * far
                    z, ez = z - bias, ez + 8 * U * bias.abs()
                z = z.masked_fill(~see, -math.inf)
                ez = ez.masked_fill(~see, 0.0).amax(1, keepdim=True)
                lse = torch.logsumexp(z, 1, keepdim=True)
                p, ep = torch.exp(z - lse), 2 * ez + 1e-6 + row_err
                o = p @ v
                yield "o", b.o[r, h], o, 2 * (B + ep) * (p @ v.square() - o.square()).clamp(min=0).sqrt() + (B + 8 * U) * o.abs()
                yield "lse", b.lse[h, r], lse[:, 0], (ez + 16 * U * lse.abs() + 1e-6 + row_err)[:, 0]
                w = b.w[0, h][t // c.block].double()
                dp, D = do @ v.T, (do * o).sum(1, keepdim=True)
                ds, wp = w * p * (dp - D) * damp, w * p
                edp = c.d * U * (do.abs() @ v.abs().T)
                eD = 2 * (B + ep) * (p * (dp - D).abs()).sum(1, keepdim=True) + edp.amax(1, keepdim=True)
                eD += (B * B + c.d * U) * (do.abs() * o.abs()).sum(1, keepdim=True)
                eds = (B + ep + 4 * U) * ds.abs() + wp * damp * (eD + edp)
                if c.softcap:
                    eds = eds + wp * (dp - D).abs() * 2 * (ez / c.softcap + 1e-6)
                dq = c.scale * ds @ k
                yield "dq", b.dq[r, h], dq, c.scale * (eds + n * U * ds.abs()) @ k.abs() + B * dq.abs() + 1e-30
                dk += c.scale * ds.T @ q
                dv += wp.T @ do
                tk += c.scale * (eds + n * G * U * ds.abs()).T @ q.abs()
                tv += ((B + ep + n * G * U) * wp).T @ do.abs()
        yield "dk", b.dk[:, g], dk, tk + B * dk.abs() + 1e-30
        yield "dv", b.dv[:, g], dv, tv + B * dv.abs() + 1e-30


@gpu
@pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)
def test_long_training_step_matches_the_formula(c):
    G = c.hq // c.hkv
    # CTAs of the forward (pairs of 128-row tiles) and of the backward (a KV tile and a group)
    assert -(-c.n // 256) * c.hq > 8 * 148 and -(-c.n // 128) * c.hkv > 8 * 148
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(h, s=1.0):
        return (torch.randn(c.n, h, c.d, device="cuda", generator=gen) * s).bfloat16()

    m = dict(q=normal(c.hq, 1.5), k=normal(c.hkv), v=normal(c.hkv))
    size = torch.exp(1.5 * torch.randn(c.n // c.block + 1, c.hq, device="cuda", generator=gen))
    m["dout"] = (normal(c.hq).float() * size[torch.arange(c.n, device="cuda") // c.block][..., None]).bfloat16()
    m["slopes"] = torch.tensor([0.3 * 2.0 ** (-8 * h / c.hq) for h in range(c.hq)], device="cuda") if c.alibi else None
    i32 = dict(dtype=torch.int32, device="cuda")
    m["start"] = None if c.start is None else torch.tensor(np.asarray(c.start), **i32)
    m["pos"] = None if c.pos is None else torch.tensor(np.asarray(c.pos), **i32)
    prefix = torch.tensor([c.prefix], **i32) if c.prefix else None
    desc = lf.make_desc(torch.tensor([0, c.n], **i32), c.n, c.n, c.hq, c.hkv, c.d, c.scale, True, c.block)
    mod = lf.make_score_mod(c.softcap, m["slopes"], prefix, prefix is not None, m["start"], m["pos"])
    b = lf.Buffers(desc)
    o_low = torch.empty_like(b.o)
    for t in (b.o, b.dq, b.dk, b.dv, b.lse):
        t.fill_(float("nan"))
    b.ws.fill_(255)
    lf.lf_attn_fwd_mod(desc, mod, m["q"], m["k"], m["v"], b.o, b.lse, o_low)
    lf.lf_block_select(desc, m["dout"], b.o, 0.3, 3, 0, 0, b.norm, None, b.tau, b.w, b.keep, b.kept_idx, b.kept_cnt)
    lf.lf_attn_bwd_mod(desc, mod, m["q"], m["k"], m["v"], b.o, b.lse, m["dout"], None, b.w, b.kept_idx, b.kept_cnt,
                       b.dq, b.dk, b.dv, b.ws, o_low)
    lf.lf_sync_status()
    assert 0.1 < float((b.w > 0).float().mean()) < 0.9
    assert all(h // G in {x // G for x in c.heads} for h in c.heads)
    for name, got, want, tol in reference(c, m, b):
        off = (got.double() - want).abs()
        assert (off <= tol).all(), (name, float((off - tol).nan_to_num(nan=1e9).max()), float(off.max()))
