"""Softmax scales so small that every visible key counts the same, in the attention over shared prefixes."""
import pytest
import torch

from test_gpu_prefix_attention import check, make, msa, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("scale", [1e-9, 1e-20, 1e-38, 1e-45])
def test_scales_next_to_nothing(msa, kv, scale):
    """With queries as they are, of zeros, and of the type's least values: hidden keys stay hidden, the others weigh the same."""
    c = make([300], [[(0, 6), (50, 6)]], 8, 2, kv, seed=71)
    c["q"][1::4] = 0.0
    c["q"][2::4] *= torch.finfo(c["q"].dtype).tiny
    for kw in (dict(), dict(groups=False), dict(groups=False, causal=False)):
        check(c, *run(msa, c, softmax_scale=scale, **kw), scale=scale, causal=kw.get("causal", True))
    c = make([0, 0], [[(700, 4)], [(3, 2)]], 8, 2, kv, seed=72)
    c["q"][1::4] = 0.0
    c["q"][2::4] *= torch.finfo(c["q"].dtype).tiny
    check(c, *run(msa, c, softmax_scale=scale, groups=False, max_seqlen_q=4), scale=scale)
