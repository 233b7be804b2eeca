"""Norms of query and key heads with the position rotation, and their gradient, against
the formulas in 64 bits.

Tolerances.  An output is rounded once to bf16: at most 2^-8 of its value.  Before that
the kernels compute in fp32; with u = 2^-24 the sum of d squares is off by at most 16 u
(eight terms in a lane, four exchanges, each one rounding), its root's reciprocal by half
of that and 2 u more, and every value then passes at most six roundings, so each product
n_a cos, n_b sin is off by less than 32 u, and the terms of the gradient, which hold one
more such sum, by less than 64 u of their own sizes.  A weight gradient's addends each
carry 32 u, and no chain of additions in these cases is longer than 256.
"""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_attention_dense_b200 as lf
from block_sparse_attention_dense_b200 import build as lfbuild
from block_sparse_attention_dense_b200.autograd import qk_norm_rope

U = 2.0 ** -24
BF16 = 2.0 ** -8


def pair_index(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, cs, rot, interleaved):
    """x [T, H, d] turned by the angles of cs [T, rot]; also the sum of the terms' sizes."""
    a, b = pair_index(rot, interleaved)
    c, s = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    y, size = x.clone(), x.abs()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    size[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, size


def ref_forward(x, w, cs, rot, interleaved, eps, norm):
    x = x.double()
    n = x
    if norm:
        n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
        if w is not None:
            n = n * w.double()
    return rotate(n, cs.double(), rot, interleaved) if rot else (n, n.abs())


def ref_backward(x, w, cs, rot, interleaved, eps, norm, dy):
    """(dx, sizes of dx's terms, dw, sum of the sizes of dw's terms) by the formulas."""
    dy = dy.double()
    g, gsize = dy, dy.abs()
    if rot:
        back = cs.double().clone()
        back[:, rot // 2:] *= -1
        g, gsize = rotate(dy, back, rot, interleaved)
    if not norm:
        return g, gsize, None, None
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    r = 1.0 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    xh = x * r
    dx = r * (g * w - xh * (g * w * xh).mean(-1, keepdim=True))
    size = r * (gsize * w.abs() + xh.abs() * (gsize * w.abs() * xh.abs()).mean(-1, keepdim=True))
    return dx, size, (g * xh).sum((0, 1)), (gsize * xh.abs()).sum((0, 1))


class Case:
    def __init__(self, name, lens, hq, hkv, d, rot, interleaved=False, norm=True, weights="bf16",
                 fused=True, given=False, tail=0):
        self.__dict__.update(locals())
        del self.__dict__["self"]

    def make(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        T = sum(self.lens) + self.tail
        qkv = torch.randn(T, self.hq + 2 * self.hkv, self.d, generator=g).to(torch.bfloat16)
        # rows of very different sizes, one of them all zeros
        qkv *= torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g)).to(torch.bfloat16)
        if T:
            qkv[T // 2] = 0
        q, k = qkv[:, : self.hq], qkv[:, self.hq: self.hq + self.hkv]
        if not self.fused:
            q, k = q.contiguous(), k.contiguous()
        qw = kw = None
        if self.norm and self.weights:
            wt = torch.bfloat16 if self.weights == "bf16" else torch.float32
            qw, kw = ((1 + 0.3 * torch.randn(self.d, generator=g)).to(wt) for _ in range(2))
        npos = 4096
        cos_sin = lf.rope_cos_sin(npos, self.rot, device="cpu") if self.rot else None
        pos = torch.cat([torch.arange(n) for n in self.lens] + [torch.zeros(self.tail, dtype=torch.long)])
        if self.given:
            pos = torch.randint(0, npos, (T,), generator=g)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(self.lens)]), dtype=torch.int32)
        return dict(q=q, k=k, qw=qw, kw=kw, cos_sin=cos_sin, cu=cu, pos=pos, T=T, qkv=qkv,
                    dyq=torch.randn(T, self.hq, self.d, generator=g).to(torch.bfloat16),
                    dyk=torch.randn(T, self.hkv, self.d, generator=g).to(torch.bfloat16))

    def dev(self, m):
        out = {n: t.cuda() if torch.is_tensor(t) else t for n, t in m.items()}
        if self.fused:
            out["q"], out["k"] = out["qkv"][:, : self.hq], out["qkv"][:, self.hq: self.hq + self.hkv]
        return out

    def desc(self, m, **kw):
        return lf.make_qk_desc(m["q"], m["k"], m["qw"], m["kw"], m["cos_sin"], cu_seqlens=m["cu"],
                               positions=m["pos"].int() if self.given else None, norm=self.norm,
                               interleaved=self.interleaved, **kw)


CASES = [
    Case("token", (1,), 32, 8, 128, 128),
    Case("token_one_head", (1,), 1, 1, 64, 64, weights="fp32", fused=False),
    Case("segments", (1, 130, 0, 257, 64), 4, 2, 128, 128),
    Case("given_positions", (300,), 8, 2, 64, 64, given=True),
    Case("pairs", (97, 33), 5, 3, 128, 128, interleaved=True, weights="fp32"),
    Case("pairs_partly", (61,), 3, 1, 64, 32, interleaved=True, given=True, fused=False),
    Case("partly", (200,), 7, 1, 128, 48),
    Case("least_rotated", (45, 4), 2, 2, 64, 16),
    Case("no_rotation", (77,), 6, 2, 128, 0),
    Case("no_weights", (77,), 6, 2, 64, 64, weights=None),
    Case("rotation_only", (150, 31), 9, 3, 128, 128, norm=False),
    Case("rotation_only_pairs", (150,), 4, 4, 64, 48, norm=False, interleaved=True, fused=False),
    Case("padded", (100, 20), 4, 2, 128, 64, tail=37),
    Case("many_rows", (1500, 1300), 32, 8, 128, 128),   # whole tokens per warp, several per warp
]
gpu = pytest.mark.gpu
each = pytest.mark.parametrize("c", CASES, ids=lambda c: c.name)


def cs_rows(c, m):
    return m["cos_sin"][m["pos"]] if c.rot else None


def check_forward(c, m, x, w, y):
    live = m["T"] - c.tail
    ref, size = ref_forward(x, w, cs_rows(c, m), c.rot, c.interleaved, 1e-6, c.norm)
    fp32 = 32 * U * size
    bad = (y.cpu().double() - ref).abs() - (BF16 * (ref.abs() + fp32) + fp32)
    assert bad[:live].max() <= 0, float(bad[:live].max())


@gpu
@each
def test_forward_matches_the_formula(c):
    m = c.make()
    g = c.dev(m)
    yq = torch.full((m["T"], c.hq, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    yk = torch.full((m["T"], c.hkv, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lf.lf_qk_norm_rope(c.desc(g), g["q"], g["k"], yq, yk)
    lf.lf_sync_status()
    check_forward(c, m, m["q"], m["qw"], yq)
    check_forward(c, m, m["k"], m["kw"], yk)
    if c.tail:   # rows behind the last segment stay as they were
        assert (yq[-c.tail:] == 7).all() and (yk[-c.tail:] == 7).all()
        lf.lf_qk_norm_rope(c.desc(g, zero_tail=True), g["q"], g["k"], yq, yk)
        assert (yq[-c.tail:] == 0).all() and (yk[-c.tail:] == 0).all()


def check_dx(ref, size, dx, live):
    fp32 = 64 * U * size
    bad = (dx.cpu().double() - ref).abs() - (BF16 * (ref.abs() + fp32) + fp32)
    assert bad[:live].max() <= 0, float(bad[:live].max())


@gpu
@each
def test_backward_matches_the_formula(c):
    m = c.make(1)
    g = c.dev(m)
    live = m["T"] - c.tail
    # gradients of the inputs go into slices of the fused projection's gradient
    dqkv = torch.full_like(g["qkv"], 7.0)
    dq, dk = dqkv[:, : c.hq], dqkv[:, c.hq: c.hq + c.hkv]
    dqw, dkw = (torch.full((c.d,), 7.0, device="cuda") for _ in range(2))
    desc = c.desc(g)
    ws = torch.full((lf.lf_qk_workspace_size(desc),), 255, dtype=torch.uint8, device="cuda")
    if c.norm:
        lf.lf_qk_norm_rope_bwd(desc, g["q"], g["k"], g["dyq"], g["dyk"], dq, dk, dqw, dkw, ws)
    else:
        lf.lf_qk_norm_rope_bwd(desc, None, None, g["dyq"], g["dyk"], dq, dk)
    lf.lf_sync_status()
    assert (dqkv[:, c.hq + c.hkv:] == 7).all()
    if c.tail:
        assert (dq[-c.tail:] == 7).all() and (dk[-c.tail:] == 7).all()
    cs = cs_rows(c, m)
    cs = cs[:live] if cs is not None else None
    for x, w, dy, dx, dw in ((m["q"], m["qw"], m["dyq"], dq, dqw), (m["k"], m["kw"], m["dyk"], dk, dkw)):
        ref, size, rdw, wsize = ref_backward(x[:live], w, cs, c.rot, c.interleaved, 1e-6, c.norm, dy[:live])
        check_dx(ref, size, dx[:live], live)
        if c.norm:
            assert ((dw.cpu().double() - rdw).abs() <= (256 + 32) * U * wsize).all()


@gpu
@pytest.mark.parametrize("c", [CASES[2], CASES[4], CASES[10]], ids=lambda c: c.name)
def test_gradient_matches_differences(c):
    """sum(dy * y) along a direction that agrees with the gradient in every sign, by central
    differences of the formula in 64 bits: the kernel's sum is off by 2^-8 of itself at
    most (each element's rounding), the differences by the third derivative, about h^2."""
    m = c.make(2)
    g = c.dev(m)
    # rows of one size, so that one step suits all of them
    for n, h in (("q", c.hq), ("k", c.hkv)):
        m[n] = torch.randn(m["T"], h, c.d, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
        g[n] = m[n].cuda()
    dq, dk = torch.empty_like(g["q"]), torch.empty_like(g["k"])
    lf.lf_qk_norm_rope_bwd(c.desc(g), g["q"], g["k"], g["dyq"], g["dyk"], dq, dk)
    gen = torch.Generator().manual_seed(3)
    for x, w, dy, dx in ((m["q"], m["qw"], m["dyq"], dq), (m["k"], m["kw"], m["dyk"], dk)):
        dx = dx.cpu().double()
        v = torch.randn(x.shape, generator=gen, dtype=torch.float64).abs() * dx.sign()

        def f(step):
            y = ref_forward(x.double() + step * v, w, cs_rows(c, m), c.rot, c.interleaved, 1e-6, c.norm)[0]
            return (y * dy.double()).sum()

        h = 1e-4
        want = (f(h) - f(-h)) / (2 * h)
        assert abs((dx * v).sum() - want) <= (BF16 + 1e-6) * (dx * v).sum()


@gpu
def test_in_place_and_reproducible():
    c = CASES[2]
    m = c.make(3)
    g = c.dev(m)
    desc = c.desc(g)
    yq, yk = torch.empty(m["T"], c.hq, c.d, dtype=torch.bfloat16, device="cuda"), torch.empty_like(g["dyk"])
    lf.lf_qk_norm_rope(desc, g["q"], g["k"], yq, yk)
    q2, k2 = g["q"].clone(), g["k"].contiguous()
    fused = g["qkv"].clone()
    lf.lf_qk_norm_rope(desc, q2, k2, q2, k2)
    assert torch.equal(q2, yq) and torch.equal(k2, yk)
    fq, fk = fused[:, : c.hq], fused[:, c.hq: c.hq + c.hkv]
    lf.lf_qk_norm_rope(desc, fq, fk, fq, fk)
    assert torch.equal(fq, yq) and torch.equal(fk, yk)
    assert torch.equal(fused[:, c.hq + c.hkv:], g["qkv"][:, c.hq + c.hkv:])
    ws = torch.empty(lf.lf_qk_workspace_size(desc), dtype=torch.uint8, device="cuda")
    got = []
    for gq, gk in ((torch.empty_like(yq), torch.empty_like(yk)), (g["dyq"].clone(), g["dyk"].clone())):
        same = len(got) == 1    # the second time over the incoming gradient
        dw = torch.empty(2, c.d, device="cuda")
        lf.lf_qk_norm_rope_bwd(desc, g["q"], g["k"], gq if same else g["dyq"], gk if same else g["dyk"],
                               gq, gk, dw[0], dw[1], ws)
        got.append((gq, gk, dw))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@gpu
def test_far_positions_and_far_rows():
    """Positions near 2^20 keep their angles; token offsets pass 2^31 elements."""
    rot, d, T = 16, 64, 66000
    cos_sin = lf.rope_cos_sin(1 << 20, rot)
    row = 33000
    assert row * (T - 1) > 2 ** 31
    buf = torch.zeros(T * row, dtype=torch.bfloat16, device="cuda").view(T, row)[:, : 3 * d].unflatten(1, (3, d))
    q, k = buf[:, :2], buf[:, 2:]
    with pytest.raises(lf.LfError):   # a token stride that is no multiple of 16 bytes
        odd = torch.zeros(2 * 129, dtype=torch.bfloat16, device="cuda").as_strided((2, 2, d), (129, d, 1))
        lf.lf_qk_norm_rope(lf.make_qk_desc(odd, odd, cos_sin=cos_sin, positions=torch.zeros(2, dtype=torch.int32, device="cuda")),
                           odd, odd, torch.empty(2, 2, d, dtype=torch.bfloat16, device="cuda"),
                           torch.empty(2, 2, d, dtype=torch.bfloat16, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(0)
    buf.copy_(torch.randn(T, 3, d, generator=g, device="cuda"))
    pos = torch.arange((1 << 20) - T, 1 << 20, dtype=torch.int32, device="cuda")
    yq, yk = torch.empty(T, 2, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, 1, d, dtype=torch.bfloat16, device="cuda")
    lf.lf_qk_norm_rope(lf.make_qk_desc(q, k, cos_sin=cos_sin, positions=pos), q, k, yq, yk)
    lf.lf_sync_status()
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    for t in (0, 1, T // 2, T - 1):
        a = (float((1 << 20) - T + t) * inv)[None]
        cs = torch.cat([a.cos(), a.sin()], 1)
        for x, y in ((q, yq), (k, yk)):
            ref, size = ref_forward(x[t:t + 1].cpu(), None, cs, rot, False, 1e-6, True)
            tol = 33 * U * size   # the table's rounding is one more
            assert ((y[t:t + 1].cpu().double() - ref).abs() <= BF16 * (ref.abs() + tol) + tol).all()


@gpu
def test_bad_position_is_reported_and_its_row_left():
    c = Case("bad", (40,), 2, 1, 64, 64, given=True)
    m = c.make()
    m["pos"][3], m["pos"][17] = -1, 4096
    g = c.dev(m)
    yq = torch.full((40, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    yk = torch.full((40, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lf.lf_qk_norm_rope(c.desc(g), g["q"], g["k"], yq, yk)
    torch.cuda.synchronize()
    with pytest.raises(lf.LfError) as e:   # the next call of any entry point, with no synchronization
        lf.lf_qk_norm_rope(c.desc(g), g["q"], g["k"], yq, yk)
    assert e.value.code == lf.LF_ERR_INVALID_ARG
    with pytest.raises(lf.LfError):
        lf.lf_sync_status()
    lf.lf_sync_status()
    keep = torch.ones(40, dtype=torch.bool)
    keep[[3, 17]] = False
    assert (yq[~keep.cuda()] == 7).all() and (yk[~keep.cuda()] == 7).all()
    m["pos"][[3, 17]] = 0
    ref, _ = ref_forward(m["q"], m["qw"], cs_rows(c, m), 64, False, 1e-6, True)
    assert (yq.cpu().double() - ref)[keep].abs().max() < 0.1


@gpu
def test_side_stream_and_captured_graph():
    c = CASES[3]
    m = c.make()
    g = c.dev(m)
    desc = c.desc(g)
    ws = torch.empty(lf.lf_qk_workspace_size(desc), dtype=torch.uint8, device="cuda")
    out = [torch.zeros_like(g["dyq"]), torch.zeros_like(g["dyk"]), torch.zeros_like(g["dyq"]), torch.zeros_like(g["dyk"]),
           torch.zeros(c.d, device="cuda"), torch.zeros(c.d, device="cuda")]

    def both(o):
        lf.lf_qk_norm_rope(desc, g["q"], g["k"], o[0], o[1])
        lf.lf_qk_norm_rope_bwd(desc, g["q"], g["k"], g["dyq"], g["dyk"], *o[2:], ws)

    both(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [torch.zeros_like(t) for t in out]
    with torch.cuda.stream(side):
        both(got)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(got)
    g["qkv"].copy_(torch.randn_like(g["qkv"].float()))
    both(out)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, out))


@gpu
@pytest.mark.parametrize("c", [CASES[2], CASES[9], CASES[10], CASES[12]], ids=lambda c: c.name)
def test_autograd(c):
    m = c.make(4)
    g = c.dev(m)
    qkv = g["qkv"].clone().requires_grad_(True)
    ws = [None if w is None else w.clone().requires_grad_(True) for w in (g["qw"], g["kw"])]
    pos = g["pos"].int() if c.given else None
    yq, yk = qk_norm_rope(qkv[:, : c.hq], qkv[:, c.hq: c.hq + c.hkv], *ws, g["cos_sin"], g["cu"], pos,
                          norm=c.norm, interleaved=c.interleaved)
    (yq.float() * g["dyq"].float()).sum().add((yk.float() * g["dyk"].float()).sum()).backward()
    want = [torch.zeros_like(g["dyq"]), torch.zeros_like(g["dyk"])]
    dw = torch.zeros(2, c.d, device="cuda")
    desc = c.desc(g)
    lf.lf_qk_norm_rope_bwd(desc, g["q"], g["k"], g["dyq"], g["dyk"], *want,
                           *((dw[0], dw[1]) if ws[0] is not None else ()),
                           ws=torch.empty(lf.lf_qk_workspace_size(desc), dtype=torch.uint8, device="cuda"))
    assert torch.equal(qkv.grad[:, : c.hq], want[0]) and torch.equal(qkv.grad[:, c.hq: c.hq + c.hkv], want[1])
    for w, d in zip(ws, dw):
        assert w is None or torch.equal(w.grad, d.to(w.dtype))
    if c.tail:
        assert (yq[-c.tail:] == 0).all() and (qkv.grad[-c.tail:] == 0).all()


# ---- refusals, on the host ----
@pytest.fixture(scope="module")
def L():
    lfbuild.build()
    return lf.lib()


def raw_desc(**kw):
    base = dict(total_tokens=4, hq=4, hkv=2, d=128, nseq=1, cu_seqlens=0x1000, positions=None, cos_sin=0x1000,
                npos=16, rot=128, pairing=0, flags=lf.LF_QK_NORM, eps=1e-6, q_weight=0x1000, k_weight=0x1000,
                weights_bf16=1)
    base.update(kw)
    return lf.lf_qk_desc(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(total_tokens=-1), lf.LF_ERR_INVALID_ARG),
    (dict(hq=0), lf.LF_ERR_INVALID_ARG),
    (dict(d=96), lf.LF_ERR_UNSUPPORTED),
    (dict(nseq=0), lf.LF_ERR_INVALID_ARG),
    (dict(rot=144), lf.LF_ERR_INVALID_ARG),
    (dict(rot=8), lf.LF_ERR_UNSUPPORTED),
    (dict(rot=-16), lf.LF_ERR_INVALID_ARG),
    (dict(cos_sin=None), lf.LF_ERR_INVALID_ARG),
    (dict(cos_sin=0x1004), lf.LF_ERR_INVALID_ARG),
    (dict(npos=0), lf.LF_ERR_INVALID_ARG),
    (dict(cu_seqlens=None), lf.LF_ERR_INVALID_ARG),
    (dict(pairing=2), lf.LF_ERR_INVALID_ARG),
    (dict(flags=0x11), lf.LF_ERR_INVALID_ARG),
    (dict(eps=-1e-6), lf.LF_ERR_INVALID_ARG),
    (dict(eps=float("nan")), lf.LF_ERR_INVALID_ARG),
    (dict(weights_bf16=2), lf.LF_ERR_INVALID_ARG),
    (dict(q_weight=0x1002), lf.LF_ERR_INVALID_ARG),
    (dict(flags=0), lf.LF_ERR_INVALID_ARG),                                    # weights without the norm
    (dict(flags=0, q_weight=None, k_weight=None, rot=0), lf.LF_ERR_INVALID_ARG),   # nothing to do
])
def test_bad_descriptors_rejected(L, kw, code):
    n = ctypes.c_size_t(0)
    d = raw_desc(**kw)
    assert L.lf_qk_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code
    p = 0x10000
    assert L.lf_qk_norm_rope(ctypes.byref(d), p, 512, p, 256, p, 512, p, 256, None) == code


def test_bad_operands_rejected(L):
    d, p = raw_desc(), 0x10000
    good = [p, 512, p, 256, p, 512, p, 256]
    for i, v in ((0, None), (2, p + 8), (1, 511), (1, 504), (3, 0), (5, 516), (7, 248), (6, None)):
        args = list(good)
        args[i] = v
        assert L.lf_qk_norm_rope(ctypes.byref(d), *args, None) == lf.LF_ERR_INVALID_ARG, (i, v)
    back = good + [p, 512, p, 256]
    assert L.lf_qk_norm_rope_bwd(ctypes.byref(d), *back, p, p, p, 16, None) == lf.LF_ERR_WORKSPACE
    assert L.lf_qk_norm_rope_bwd(ctypes.byref(d), *back, p, p, None, 0, None) == lf.LF_ERR_WORKSPACE
    assert L.lf_qk_norm_rope_bwd(ctypes.byref(d), *back, p + 4, p, p, 1 << 20, None) == lf.LF_ERR_INVALID_ARG
    for i in (0, 4, 6, 8, 10):
        args = list(back)
        args[i] = None
        assert L.lf_qk_norm_rope_bwd(ctypes.byref(d), *args, None, None, None, 0, None) == lf.LF_ERR_INVALID_ARG, i
    plain = raw_desc(flags=0, q_weight=None, k_weight=None)
    assert L.lf_qk_norm_rope_bwd(ctypes.byref(plain), *back, p, None, p, 1 << 20, None) == lf.LF_ERR_INVALID_ARG


def test_no_rows_is_a_noop(L):
    d = raw_desc(total_tokens=0)
    assert L.lf_qk_norm_rope(ctypes.byref(d), None, 0, None, 0, None, 0, None, 0, None) == 0
    assert L.lf_qk_norm_rope_bwd(ctypes.byref(d), *[None, 0] * 6, None, None, None, 0, None) == 0


def test_binding_refuses_what_does_not_fit():
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lf.make_qk_desc(q, k)                      # not on a GPU
    with pytest.raises(ValueError):
        lf.make_qk_desc(q, k[:3])
    with pytest.raises(ValueError):
        lf.make_qk_desc(q, k[..., :32])


@gpu
def test_binding_refuses_other_types_shapes_and_devices():
    q, k = (torch.zeros(4, h, 64, dtype=torch.bfloat16, device="cuda") for h in (2, 1))
    w = torch.ones(64, device="cuda")
    cs = lf.rope_cos_sin(8, 64)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for kw in (dict(q_weight=w, k_weight=w.bfloat16()), dict(q_weight=w[:32]), dict(cos_sin=cs.double()),
               dict(cos_sin=cs, positions=pos.long()), dict(cos_sin=cs, positions=pos[:3]),
               dict(cos_sin=cs.cpu(), positions=pos), dict(cos_sin=cs.t()[:, :4], positions=pos),
               dict(cos_sin=cs[0], positions=pos)):
        with pytest.raises(ValueError):
            lf.make_qk_desc(q, k, **kw)
    desc = lf.make_qk_desc(q, k, w, w, cs, positions=pos)
    for bad in (q.float(), q[:3], q.cpu(), q.transpose(0, 1).contiguous().transpose(0, 1), q[:, :1]):
        with pytest.raises(ValueError):
            lf.lf_qk_norm_rope(desc, bad, k, q, k)
        with pytest.raises(ValueError):
            lf.lf_qk_norm_rope(desc, q, k, bad, k)


@gpu
def test_empty_batch():
    q, k = (torch.zeros(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (2, 1))
    w = torch.ones(64, device="cuda", requires_grad=True)
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    q.requires_grad_(True)
    yq, yk = qk_norm_rope(q, k, w, None, lf.rope_cos_sin(8, 64), cu)
    yq.sum().backward()
    assert yq.shape == q.shape and (w.grad == 0).all()
