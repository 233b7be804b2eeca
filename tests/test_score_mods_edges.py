"""Attention with modified scores through autograd: arrays changed between the two passes."""
import pytest

from block_sparse_attention_dense_b200.autograd import lazyflash_attention
from test_score_mods import NAMED, dev

gpu = pytest.mark.gpu


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
