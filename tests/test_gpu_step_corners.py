"""Calls of the serving step's operators at the edges of what their documentation allows."""
import pytest
import torch

import test_gpu_tree_attention as tree

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def msa():
    import block_sparse_top_msa_gb300 as m
    m.build()
    m.lib()
    return m


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
def test_tree_refuses_a_query_with_strides(msa, kv):
    """A slice of a packed projection, a transposed and an expanded query: refused, by the call and by the prepared form."""
    c = tree.make([5, 3], [300, 140], 8, 2, 2, kv, garbage=False)
    d = {n: t.to(DEV) for n, t in c.items()}
    t, hq = c["q"].shape[:2]
    packed = torch.randn(t, hq + 4, 128, device=DEV).to(c["q"].dtype)
    strided = [packed[:, :hq], packed[:, 2 : 2 + hq], torch.randn(hq, t, 128, device=DEV).to(c["q"].dtype).transpose(0, 1), packed[:1, :hq].expand(t, hq, 128),
               packed[:, :1].expand(t, hq, 128)]
    for q in strided:
        for call in (msa.msa_tree_attention, msa.TreeAttentionRunner):
            with pytest.raises(ValueError, match="q must be contiguous"):
                call(q, d["k"], d["v"], d["q2k"], d["cu"], d["mask"], page_table=d["table"], seqused_k=d["used"], max_seqlen_q=5)
        c["q"] = q.contiguous().cpu()
        tree.check(c, *tree.run(msa, c))
