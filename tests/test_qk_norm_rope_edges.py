"""Head norms with rotation: eps = 0 with lanes and rows that hold nothing, and tables that
ask for a gradient.  References and tolerances are those of test_qk_norm_rope.py."""
import pytest
import torch

import block_sparse_attention_dense_b200 as lf
from block_sparse_attention_dense_b200.autograd import qk_norm_rope
from test_qk_norm_rope import U, Case, check_dx, cs_rows, ref_backward

gpu = pytest.mark.gpu


# a warp instruction covers 2 (d = 128) or 4 (d = 64) heads: head counts that are no multiple
# of it leave lanes without a row
@gpu
@pytest.mark.parametrize("c", [
    Case("one_kv_head", (70, 9), 4, 1, 128, 128),
    Case("six_and_two_heads", (70, 9), 6, 2, 64, 64, weights="fp32"),
    Case("odd_heads_without_rotation", (40,), 5, 3, 128, 0),
    Case("pairs_padded", (70, 9), 4, 1, 64, 32, interleaved=True, tail=21),
    Case("padded", (70, 9), 4, 2, 128, 128, tail=21),
], ids=lambda c: c.name)
def test_weight_gradients_without_eps(c):
    """Rows of non-zero values need no eps; what is behind the last segment adds nothing."""
    m = c.make(11)
    assert (m["qkv"][m["T"] // 2] == 0).all()
    m["qkv"][m["T"] // 2] = torch.randn(m["qkv"].shape[1:], generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    g = c.dev(m)
    live = m["T"] - c.tail
    cs = cs_rows(c, m)
    cs = cs[:live] if cs is not None else None
    refs = [ref_backward(x[:live], w, cs, c.rot, c.interleaved, 0.0, True, dy[:live])
            for x, w, dy in ((m["q"], m["qw"], m["dyq"]), (m["k"], m["kw"], m["dyk"]))]
    for zero_tail in (False, True):
        desc = c.desc(g, eps=0.0, zero_tail=zero_tail)
        dq, dk = torch.empty_like(g["dyq"]), torch.empty_like(g["dyk"])
        dqw, dkw = torch.empty(2, c.d, device="cuda")
        ws = torch.full((lf.lf_qk_workspace_size(desc),), 255, dtype=torch.uint8, device="cuda")
        lf.lf_qk_norm_rope_bwd(desc, g["q"], g["k"], g["dyq"], g["dyk"], dq, dk, dqw, dkw, ws)
        lf.lf_sync_status()
        for (ref, size, rdw, wsize), dx, dw in zip(refs, (dq, dk), (dqw, dkw)):
            check_dx(ref, size, dx[:live], live)
            assert ((dw.cpu().double() - rdw).abs() <= (256 + 32) * U * wsize).all()
    # the autograd function, which always writes the rows behind the last segment
    x = g["qkv"].clone().requires_grad_(True)
    weights = [w.clone().requires_grad_(True) for w in (g["qw"], g["kw"])]
    y = qk_norm_rope(x[:, : c.hq], x[:, c.hq: c.hq + c.hkv], *weights, g["cos_sin"], g["cu"], eps=0.0,
                     interleaved=c.interleaved)
    torch.autograd.backward(y, (g["dyq"], g["dyk"]))
    for w, dw in zip(weights, (dqw, dkw)):
        assert torch.equal(w.grad, dw.to(w.dtype))


@gpu
def test_rows_of_tiny_values_without_eps():
    """Squares near the least normal number, 2^-126: nothing but the row's own mean square counts.
    Each square is off by half of 2^-149 at most, 2^-143 for 128 of them, which is 2^-28 of their
    sum: less than one rounding."""
    c = Case("tiny", (40,), 4, 2, 128, 128)
    m = c.make(12)
    gen = torch.Generator().manual_seed(2)
    m["qkv"].copy_(torch.randn(m["qkv"].shape, generator=gen) * 2.0 ** -61)
    g = c.dev(m)
    cs = cs_rows(c, m)
    desc = c.desc(g, eps=0.0)
    dq, dk = torch.empty_like(g["dyq"]), torch.empty_like(g["dyk"])
    dqw, dkw = torch.empty(2, c.d, device="cuda")
    ws = torch.empty(lf.lf_qk_workspace_size(desc), dtype=torch.uint8, device="cuda")
    lf.lf_qk_norm_rope_bwd(desc, g["q"], g["k"], g["dyq"], g["dyk"], dq, dk, dqw, dkw, ws)
    lf.lf_sync_status()
    for x, w, dy, dx, dw in ((m["q"], m["qw"], m["dyq"], dq, dqw), (m["k"], m["kw"], m["dyk"], dk, dkw)):
        ref, size, rdw, wsize = ref_backward(x, w, cs, c.rot, c.interleaved, 0.0, True, dy)
        check_dx(ref, size, dx, m["T"])
        assert ((dw.cpu().double() - rdw).abs() <= (256 + 32) * U * wsize).all()


def test_a_table_that_asks_for_a_gradient_is_refused():
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    table = lf.rope_cos_sin(8, 64, device="cpu").requires_grad_(True)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="cos_sin"):
        qk_norm_rope(q, k, None, None, table, cu)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # no gradient is asked for: only the device is wrong
        qk_norm_rope(q, k, None, None, table, cu)
