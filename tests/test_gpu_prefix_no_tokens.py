"""The attention over shared prefixes of a step without tokens: called and prepared."""
import pytest
import torch

from test_gpu_prefix_attention import msa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [False, True])
def test_no_tokens(msa, groups):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 2, 128, 128, dtype=torch.bfloat16, device="cuda")
    kw = dict(page_table=i32([[0], [1]]), seqused_k=i32([5, 7]), return_softmax_lse=True)
    if groups:
        kw.update(group_rows=i32([0, 1]), cu_groups=i32([0, 2, 2]), group_blocks=i32([0, 0]))
    out, lse = msa.msa_prefix_attention(q, k, k, i32([0, 0, 0]), **kw)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    runner = msa.PrefixAttentionRunner(q, k, k, i32([0, 0, 0]), **kw)
    runner.run()
    assert runner.out.shape == (0, 8, 128) and runner.lse.shape == (0, 8)
    torch.cuda.synchronize()
    assert msa.msa_read_device_fault() == 0
