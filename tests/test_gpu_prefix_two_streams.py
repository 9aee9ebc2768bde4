"""Two calls of the attention over shared prefixes at once, each on a stream and with a workspace of its own."""
import pytest
import torch

from parity_util import fault_clear
from test_gpu_prefix_attention import DEV, check, make, msa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kinds", [("bf16", "e4m3"), ("fp16", "fp16")])
def test_two_calls_at_once(msa, kinds):
    cases = [make([3000, 300], [[(i * 11, 2) for i in range(9)], [(3, 1), (80, 4)]], 16, 2, kinds[0], seed=111),
             make([0] * 20, [[(i * 90, 1)] for i in range(20)], 16, 2, kinds[1], seed=112)]
    calls = []
    for c, groups in zip(cases, (True, False)):
        d = {n: t.to(DEV) for n, t in c.items()}
        kw = dict(group_rows=d["rows"], cu_groups=d["ends"], group_blocks=d["blocks"]) if groups else dict(max_seqlen_q=1)
        calls.append(lambda d=d, kw=kw: msa.msa_prefix_attention(d["q"], d["k"], d["v"], d["cu"], page_table=d["table"], seqused_k=d["used"], return_softmax_lse=True, **kw))
    want = [f() for f in calls]
    for c, (out, lse) in zip(cases, want):
        check(c, out, lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        assert all(torch.equal(w[0], g[0]) and torch.equal(w[1], g[1]) for g in gs)
    fault_clear(msa)
