"""What the attention layer's operators around the block-sparse backward cost.

Four operators, each through the package's public calls (``own``) or written out in elementary
torch operations:

* ``norm_rope``: RMS norm of every query and key head with the position rotation;
* ``norm_rope_bwd``: its gradient (inputs and norm weights);
* ``attn_fwd``: attention with modified scores (tanh cap, distance bias, prefix / document / shared
  prefix / window masks), output and log-sum-exp;
* ``attn_train``: the same forward followed by the block-sparse backward over given kept blocks.

Tensors are packed ([tokens, heads, head dim], bf16) with segments given by cu_seqlens.
"""
import math
import random

import numpy as np
import torch

own = False

LOG2E = 1.4426950408889634
MASKS = ("causal", "prefix", "shared", "window")


# ----------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------
def _norm(name, op, tokens, segments, hq, hkv, d, rot, interleaved, weights, fused, positions):
    return dict(name=name, op=op, tokens=tokens, segments=segments, hq=hq, hkv=hkv, d=d, rot=rot,
                interleaved=interleaved, weights=weights, fused=fused, positions=positions)


def _attn(name, op, tokens, segments, hq, hkv, d, block, softcap, alibi, mask, spread, kept=1.0):
    return dict(name=name, op=op, tokens=tokens, segments=segments, hq=hq, hkv=hkv, d=d, block=block,
                softcap=softcap, alibi=alibi, mask=mask, spread=spread, kept=kept)


def listed():
    return [
        # one new token of one request: a call whose latency counts
        _norm("norm_rope token", "norm_rope", 1, 1, 32, 8, 128, 128, False, "bf16", True, "given"),
        # the headline layer's packed batch, slices of one fused projection
        _norm("norm_rope headline", "norm_rope", 32768, 1, 32, 8, 128, 128, False, "bf16", True, "segment"),
        # a small ragged batch with partly rotated heads, neighbouring pairs
        _norm("norm_rope_bwd ragged", "norm_rope_bwd", 700, 3, 8, 2, 64, 32, True, "fp32", False, "given"),
        # the headline layer's gradient
        _norm("norm_rope_bwd headline", "norm_rope_bwd", 32768, 1, 32, 8, 128, 128, False, "bf16", True, "segment"),
        # capped scores, the smallest training layer of the repository
        _attn("attn_train tiny cap", "attn_train", 512, 1, 2, 2, 64, 64, 30.0, False, "causal", 2.0, 0.6),
        # capped scores at the mid and long layers, the share of blocks that the selection keeps there
        _attn("attn_fwd long cap", "attn_fwd", 16384, 1, 32, 8, 128, 128, 50.0, False, "causal", 2.0),
        _attn("attn_train mid cap", "attn_train", 4096, 1, 32, 8, 128, 128, 50.0, False, "causal", 3.0, 0.4),
        # one of four tensor-parallel shards of the headline layer, capped, windowed
        _attn("attn_train shard cap window", "attn_train", 32768, 1, 8, 2, 128, 128, 30.0, False, "window", 2.0, 0.29),
        # a packed batch of several documents with a distance bias
        _attn("attn_fwd varlen bias", "attn_fwd", 15001, 5, 32, 8, 64, 128, 0.0, True, "causal", 1.5),
        _attn("attn_train long bias", "attn_train", 16384, 1, 32, 8, 128, 128, 0.0, True, "causal", 1.5, 0.3),
        # prefix language model: every document's first part is seen whole
        _attn("attn_train varlen prefix", "attn_train", 8192, 3, 16, 4, 128, 128, 0.0, False, "prefix", 1.5, 0.5),
        # many answers to one prompt, which is packed and computed once
        _attn("attn_train shared prompt", "attn_train", 12288, 1, 32, 8, 128, 128, 0.0, False, "shared", 1.5, 0.35),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("norm_rope", "norm_rope_bwd", "attn_fwd", "attn_train"))
    d = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 3, 4))
    if op.startswith("norm"):
        tokens = size(1, 32768)
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d])
        c = _norm("", op, tokens, min(tokens, rng.randint(1, 8)), hq, hkv, d, rot, rng.random() < 0.5,
                  rng.choice(("bf16", "fp32")), rng.random() < 0.5, rng.choice(("given", "segment")))
    else:
        tokens = size(64, 16384)
        c = _attn("", op, tokens, rng.randint(1, 6), hq, hkv, d, rng.choice((64, 128)),
                  rng.choice((0.0, round(rng.uniform(15.0, 50.0), 1))), rng.random() < 0.3,
                  rng.choice(MASKS), round(rng.uniform(1.0, 4.0), 2),
                  round(rng.uniform(0.1, 1.0), 2) if op == "attn_train" else 1.0)
        if not c["softcap"] and not c["alibi"] and c["mask"] == "causal":
            c["softcap"] = 30.0
        most = max(work(x)["flops"] for x in listed())
        while work(c)["flops"] > most:   # no dearer than the dearest of the listed ones
            c["tokens"] = size(64, c["tokens"])
    del c["name"]
    return c


def _lengths(total, parts, lo=1):
    """`parts` ragged lengths, at least `lo` each, that add up to `total`; the same for the same sizes."""
    r = random.Random(total * 1009 + parts)
    parts = max(1, min(parts, total // max(1, lo)))
    shares = [r.uniform(0.3, 1.7) for _ in range(parts)]
    got = [max(lo, int(total * s / sum(shares))) for s in shares]
    got[got.index(max(got))] += total - sum(got)
    return got


def _layout(case):
    """cu_seqlens, and for attention each segment's prefix length and each row's first own key (both
    counted from the segment's start; None where the mask has none), as numpy int32."""
    lens = _lengths(case["tokens"], case["segments"])
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    mask = case.get("mask", "causal")
    prefix = start = None
    if mask == "prefix":
        prefix = np.array([max(1, n * 2 // 5) for n in lens], np.int32)
    elif mask == "window":
        width = max(1, case["tokens"] // 16)
        start = np.concatenate([np.maximum(0, np.arange(n) - width + 1) for n in lens]).astype(np.int32)
    elif mask == "shared":
        prefix = np.array([max(1, n // 3) for n in lens], np.int32)
        rows = []
        for n, p in zip(lens, prefix):
            at = int(p)
            rows.append(np.zeros(at, np.int64))
            for m in _lengths(n - at, 12) if n > at else []:
                rows.append(np.full(m, at))
                at += m
        start = np.concatenate(rows).astype(np.int32)
    return cu, prefix, start


# ----------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _cos_sin(npos, rot):
    """fp32 [npos, rot]: the cosines, then the sines, of pos * 10000^(-2i/rot), angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(npos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def prepare(case, seed):
    g = _gen(seed)
    T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    cu, prefix, start = _layout(case)
    s = dict(case=case, lens=np.diff(cu).tolist(), cu=torch.from_numpy(cu).cuda())
    if case["op"].startswith("norm"):
        if case["fused"]:   # slices of the fused projection's output, as the layer has them
            qkv = _normal(g, T, hq + 2 * hkv, d)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            s["q"], s["k"] = _normal(g, T, hq, d), _normal(g, T, hkv, d)
        wt = torch.bfloat16 if case["weights"] == "bf16" else torch.float32
        s["qw"], s["kw"] = ((1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(wt) for _ in range(2))
        npos = 4 * T + 64
        s["cos_sin"] = _cos_sin(npos, case["rot"])
        s["positions"] = None
        if case["positions"] == "given":
            s["positions"] = torch.randint(0, npos, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(T, hkv, d, dtype=torch.bfloat16, device="cuda")
        if case["op"] == "norm_rope_bwd":
            s["dq_out"], s["dk_out"] = _normal(g, T, hq, d), _normal(g, T, hkv, d)
            s["dqw"], s["dkw"] = (torch.empty(d, dtype=torch.float32, device="cuda") for _ in range(2))
        return s
    s["q"] = _normal(g, T, hq, d, std=case["spread"])   # scores of this standard deviation
    s["k"], s["v"] = _normal(g, T, hkv, d), _normal(g, T, hkv, d)
    s["prefix"] = None if prefix is None else torch.from_numpy(prefix).cuda()
    s["start"] = None if start is None else torch.from_numpy(start).cuda()
    s["slopes"] = None
    if case["alibi"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda")
    if case["op"] == "attn_train":
        # the kept blocks of one step: a fixed share of each head's blocks, weights as 1/p has them,
        # and an output gradient whose size differs from block to block
        n, B = len(s["lens"]), case["block"]
        nb = [-(-m // B) for m in s["lens"]]
        nbmax = max(nb)
        count = torch.tensor(nb, device="cuda")
        live = torch.arange(nbmax, device="cuda") < count[:, None]
        u = torch.rand(n, hq, nbmax, generator=g, device="cuda").masked_fill(~live[:, None], 2.0)
        cnt = (count * case["kept"]).ceil().long()
        rank = u.argsort(-1).argsort(-1)
        keep = rank < cnt[:, None, None]
        w = (1.0 + torch.rand(n, hq, nbmax, generator=g, device="cuda") / case["kept"]) * keep
        s["weight"] = w.contiguous()
        key = torch.where(keep, torch.arange(nbmax, device="cuda"), nbmax).sort(-1).values
        s["kept_idx"] = torch.where(key < nbmax, key, -1).int().contiguous()
        s["kept_cnt"] = cnt[:, None].expand(n, hq).int().contiguous()
        s["seg"] = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(s["lens"], device="cuda"))
        s["blk"] = torch.cat([torch.arange(m, device="cuda") // B for m in s["lens"]])
        size = torch.exp(1.5 * torch.randn(n, hq, nbmax, generator=g, device="cuda"))
        dout = torch.randn(T, hq, d, generator=g, device="cuda") * size[s["seg"], :, s["blk"]][..., None]
        s["dout"] = dout.to(torch.bfloat16)
    return s


# ----------------------------------------------------------------------------------------------
# the norm and the rotation
# ----------------------------------------------------------------------------------------------
def _pos_plain(s):
    if s["positions"] is not None:
        return s["positions"].long()
    return torch.cat([torch.arange(m, device="cuda") for m in s["lens"]])


def _pairs(case):
    """Indices of the first and second member of each rotated pair."""
    rot = case["rot"]
    i = torch.arange(rot // 2, device="cuda")
    return (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)


def _rotate(case, x, cos, sin):
    a, b = _pairs(case)
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


EPS = 1e-6


def _norm_rope_plain(s):
    case = s["case"]
    half = case["rot"] // 2
    cs = s["cos_sin"][_pos_plain(s)]
    cos, sin = cs[:, None, :half], cs[:, None, half:]

    def fwd(x, w):
        x = x.float()
        xn = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        return _rotate(case, xn * w.float(), cos, sin).to(torch.bfloat16)

    def bwd(x, w, dy):
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xn = x * r
        g = _rotate(case, dy.float(), cos, -sin)
        dw = (g * xn).double().sum((0, 1)).float()
        gw = g * w.float()
        dx = r * (gw - xn * (gw * xn).mean(-1, keepdim=True))
        return dx.to(torch.bfloat16), dw

    if case["op"] == "norm_rope":
        return fwd(s["q"], s["qw"]), fwd(s["k"], s["kw"])
    dq, dqw = bwd(s["q"], s["qw"], s["dq_out"])
    dk, dkw = bwd(s["k"], s["kw"], s["dk_out"])
    return dq, dk, dqw, dkw


def _norm_rope_own(s):
    import block_sparse_attention_dense_b200 as lf
    case = s["case"]
    if "desc" not in s:   # the layer's descriptor, kept from step to step
        s["desc"] = lf.make_qk_desc(s["q"], s["k"], s["qw"], s["kw"], s["cos_sin"], cu_seqlens=s["cu"],
                                    positions=s["positions"], eps=EPS, interleaved=case["interleaved"])
    desc = s["desc"]
    if case["op"] == "norm_rope":
        lf.lf_qk_norm_rope(desc, s["q"], s["k"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    if "ws" not in s:
        s["ws"] = torch.empty(lf.lf_qk_workspace_size(desc), dtype=torch.uint8, device="cuda")
    lf.lf_qk_norm_rope_bwd(desc, s["q"], s["k"], s["dq_out"], s["dk_out"], s["q_out"], s["k_out"],
                           s["dqw"], s["dkw"], s["ws"])
    return s["q_out"], s["k_out"], s["dqw"], s["dkw"]


def _norm_rope_exact(s):
    """By complex multiplication and torch's own derivative, in 64 bits."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    cs = s["cos_sin"][_pos_plain(s)].double()
    turn = torch.complex(cs[:, None, :half], cs[:, None, half:])

    def fwd(x, w):
        y = x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * w
        z, rest = y[..., :rot], y[..., rot:]
        if case["interleaved"]:
            z = torch.view_as_real(torch.view_as_complex(z.unflatten(-1, (half, 2)).contiguous()) * turn).flatten(-2)
        else:
            z = torch.complex(z[..., :half].contiguous(), z[..., half:].contiguous()) * turn
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, rest], -1)

    if case["op"] == "norm_rope":
        return fwd(s["q"].double(), s["qw"].double()), fwd(s["k"].double(), s["kw"].double())
    got = []
    for x, w, dy in ((s["q"], s["qw"], s["dq_out"]), (s["k"], s["kw"], s["dk_out"])):
        x, w = x.double().detach().requires_grad_(True), w.double().detach().requires_grad_(True)
        got.append(torch.autograd.grad(fwd(x, w), (x, w), dy.double()))
    return got[0][0], got[1][0], got[0][1], got[1][1]


# ----------------------------------------------------------------------------------------------
# attention with modified scores
# ----------------------------------------------------------------------------------------------
def _visible(s, i, a, n):
    """[n, n]: whether row t (down) of segment i, of n rows from row a on, sees key u (across)."""
    t = torch.arange(n, device="cuda")[:, None]
    u = torch.arange(n, device="cuda")[None]
    own_keys = u <= t
    if s["start"] is not None:
        own_keys = own_keys & (u >= s["start"][a:a + n, None])
    if s["prefix"] is None:
        return own_keys
    in_prefix = u < s["prefix"][i]
    if s["case"]["mask"] == "shared":
        in_prefix = in_prefix & (u <= t)
    return own_keys | in_prefix


def _attn_plain(s):
    case = s["case"]
    T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    G, scale, cap = hq // hkv, 1.0 / math.sqrt(d), case["softcap"]
    o = torch.empty(T, hq, d, device="cuda")
    lse = torch.empty(hq, T, device="cuda")
    train = case["op"] == "attn_train"
    if train:
        dq = torch.empty(T, hq, d, device="cuda")
        dk, dv = torch.zeros(T, hkv, d, device="cuda"), torch.zeros(T, hkv, d, device="cuda")
        wrow = s["weight"][s["seg"], :, s["blk"]]   # [T, hq]
    a = 0
    for i, n in enumerate(s["lens"]):
        r = slice(a, a + n)
        hidden = ~_visible(s, i, a, n)
        if case["alibi"]:
            at = torch.arange(n, device="cuda", dtype=torch.float32)
            far = (at[:, None] - at[None]).abs()
        for h in range(hq):
            q, k, v = s["q"][r, h].float(), s["k"][r, h // G].float(), s["v"][r, h // G].float()
            z = (q @ k.T) * scale
            if cap:
                th = torch.tanh(z / cap)
                z = cap * th
            if case["alibi"]:
                z = z - s["slopes"][h] * far
            z.masked_fill_(hidden, float("-inf"))
            top = z.amax(1, keepdim=True)
            p = torch.exp(z - top)
            total = p.sum(1, keepdim=True)
            lse[h, r] = (top + torch.log(total))[:, 0]
            p = p / total
            oh = p @ v
            o[r, h] = oh
            if train:
                do = s["dout"][r, h].float() * wrow[r, h, None]
                dv[r, h // G] += p.T @ do
                dz = p * (do @ v.T - (do * oh).sum(1, keepdim=True))
                if cap:
                    dz = dz * (1.0 - th * th)
                dq[r, h] = (dz @ k) * scale
                dk[r, h // G] += (dz.T @ q) * scale
        a += n
    if not train:
        return o.to(torch.bfloat16), lse
    return tuple(x.to(torch.bfloat16) for x in (o,)) + (lse,) + tuple(x.to(torch.bfloat16) for x in (dq, dk, dv))


def _attn_own(s):
    import block_sparse_attention_dense_b200 as lf
    case = s["case"]
    T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    if "bufs" not in s:   # the layer's plan: descriptors and buffers, kept from step to step
        s["desc"] = lf.make_desc(s["cu"], max(s["lens"]), T, hq, hkv, d, 1.0 / math.sqrt(d), True, case["block"])
        s["mod"] = lf.make_score_mod(softcap=case["softcap"], alibi_slopes=s["slopes"], prefix_len=s["prefix"],
                                     prefix_causal=case["mask"] == "shared", row_start=s["start"])
        s["bufs"] = lf.Buffers(s["desc"]) if case["op"] == "attn_train" else None
        s["o"] = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(hq, T, dtype=torch.float32, device="cuda")
        s["o_low"] = torch.empty_like(s["o"]) if case["op"] == "attn_train" else None
    lf.lf_attn_fwd_mod(s["desc"], s["mod"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["o_low"])
    if case["op"] == "attn_fwd":
        return s["o"], s["lse"]
    b = s["bufs"]
    lf.lf_attn_bwd_mod(s["desc"], s["mod"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], None,
                       s["weight"], s["kept_idx"], s["kept_cnt"], b.dq, b.dk, b.dv, b.ws, s["o_low"])
    return s["o"], s["lse"], b.dq, b.dk, b.dv


def _attn_exact(s):
    """From the definition, one segment's head at a time, by torch's own derivative in 64 bits."""
    case = s["case"]
    G, train = case["hq"] // case["hkv"], case["op"] == "attn_train"
    q, k, v = (s[x].double().transpose(0, 1) for x in "qkv")   # [heads, tokens, d]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    edges = np.concatenate([[0], np.cumsum(s["lens"])]).tolist()
    for i, (a, b) in enumerate(zip(edges, edges[1:])):
        seen = _visible(s, i, a, b - a)
        dist = torch.arange(b - a, device="cuda", dtype=torch.float64)
        for h in range(case["hq"]):
            qh, kh, vh = (x[j, a:b].detach().requires_grad_(train) for x, j in ((q, h), (k, h // G), (v, h // G)))
            with torch.set_grad_enabled(train):
                z = torch.einsum("td,ud->tu", qh, kh) / case["d"] ** 0.5
                if case["softcap"]:
                    z = torch.tanh(z / case["softcap"]) * case["softcap"]
                if case["alibi"]:
                    z = z - s["slopes"][h].double() * (dist[:, None] - dist).abs()
                z = torch.where(seen, z, float("-inf"))
                total = torch.logsumexp(z, 1)
                out = torch.exp(z - total[:, None]) @ vh
            o[h, a:b], lse[h, a:b] = out.detach(), total.detach()
            if train:
                w = s["weight"][i, h].double()[torch.arange(b - a, device="cuda") // case["block"]]
                grads = torch.autograd.grad(out, (qh, kh, vh), s["dout"][a:b, h].double() * w[:, None])
                dq[h, a:b] = grads[0]
                dk[h // G, a:b] += grads[1]
                dv[h // G, a:b] += grads[2]
            del z, out, total
    o, dq, dk, dv = (x.transpose(0, 1).contiguous() for x in (o, dq, dk, dv))
    return (o, lse, dq, dk, dv) if train else (o, lse)


# ----------------------------------------------------------------------------------------------
def run(state):
    norm = state["case"]["op"].startswith("norm")
    if own:
        return _norm_rope_own(state) if norm else _attn_own(state)
    return _norm_rope_plain(state) if norm else _attn_plain(state)


def exact(case, seed):
    s = prepare(case, seed)
    return _norm_rope_exact(s) if case["op"].startswith("norm") else _attn_exact(s)


def _pairs_seen(case):
    """(row, key) pairs that the mask leaves, over all segments."""
    cu, prefix, start = _layout(case)
    total = 0
    for i in range(len(cu) - 1):
        n = int(cu[i + 1] - cu[i])
        t = np.arange(n, dtype=np.int64)
        lo = np.zeros(n, np.int64) if start is None else start[cu[i]:cu[i + 1]].astype(np.int64)
        if prefix is None:
            total += int((t - lo + 1).sum())
            continue
        e = np.minimum(int(prefix[i]), t + 1) if case["mask"] == "shared" else np.full(n, int(prefix[i]))
        # keys [0, e) and [lo, t], counted once
        total += int((e + np.maximum(0, t + 1 - np.maximum(lo, e))).sum())
    return total


def work(case):
    T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    x = T * (hq + hkv) * d
    if case["op"].startswith("norm"):
        wb = 2 * d * (2 if case["weights"] == "bf16" else 4)
        table = T * case["rot"] * 4 + 4 * T
        if case["op"] == "norm_rope":
            return {"bytes": 2 * 2 * x + table + wb, "flops": 7 * x}
        return {"bytes": 3 * 2 * x + table + wb + 2 * d * 4, "flops": 16 * x}
    pairs = _pairs_seen(case) * hq
    byt = 2 * T * d * (2 * hq + 2 * hkv) + 4 * T * hq
    flops = 4 * d * pairs
    if case["op"] == "attn_train":
        byt += 2 * T * d * (2 * hq + 2 * hkv)
        flops += int(10 * d * pairs * case["kept"])
    return {"bytes": byt, "flops": flops}
