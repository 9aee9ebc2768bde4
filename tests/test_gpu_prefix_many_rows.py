"""The attention over shared prefixes with more rows than its CTAs have places for the parts of cut units, and no groups."""
import pytest
import torch

from test_gpu_prefix_attention import DEV, check, make, msa, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("samples,hq,hkv", [([(500, 700)], 64, 1), ([(3000, 250), (0, 200), (700, 210)], 64, 2), ([(90, 1300)], 32, 1)])
def test_prompts(msa, samples, hq, hkv, kv):
    c = make([0] * len(samples), [[s] for s in samples], hq, hkv, kv, seed=101)
    assert c["q"].shape[0] * hq > 152 * 256
    out, lse = run(msa, c, groups=False)
    check(c, out, lse)
    again, lse2 = run(msa, c, groups=False)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_thousands_of_requests_of_few_rows(msa, kv):
    """Units of 16 rows: 2600 requests of one to sixteen rows of one KV head, some of long runs."""
    b, g = 2600, torch.Generator().manual_seed(7)
    c = make([0], [[(6000, 1)]], 16, 1, kv, seed=102)
    pages = c["k"].shape[0]
    used = torch.randint(1, 400, (b,), generator=g).to(torch.int32)
    used[::97] = 6001
    table = torch.randint(0, pages, (b, 47), generator=g).to(torch.int32)
    live = torch.randn(pages, 1, 128, 128, generator=g)
    c["k"], c["v"] = live.to(c["k"].dtype), live.flip(0).to(c["v"].dtype)
    c.update(q=torch.randn(b, 16, 128, generator=g).to(c["q"].dtype), cu=torch.arange(b + 1, dtype=torch.int32), table=table, used=used)
    out, lse = run(msa, c, groups=False, max_seqlen_q=1)
    some = torch.cat([torch.arange(0, b, 97), torch.arange(5, b, 53)])
    part = dict(c, q=c["q"][some], cu=torch.arange(len(some) + 1, dtype=torch.int32), table=table[some], used=used[some])
    check(part, out[some.to(DEV)], lse[some.to(DEV)])
