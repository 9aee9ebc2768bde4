"""Calls of the operators of a step of samples that lie at the edge of what they allow: counters that overflow, the most requests,
many rows, the largest numbers, two calls at once."""
import math

import pytest
import torch

import samples_util as S
from parity_util import fault_clear
from test_gpu_prefix_attention import check as check_attention
from test_gpu_sample import check, normal, run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def msa():
    import block_sparse_top_msa_gb300 as m
    m.build()
    m.lib()
    return m


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [57343, 57345, 61441, 200019, 1 << 19])
def test_flat_rows_of_many_tokens(dtype, vocab):
    """One logit tens of thousands of times over: the whole part of u times the number kept, whole numbers all the way."""
    u = [0.0, 0.13, 0.5, 0.77, 0.999]
    x = torch.full((5, vocab), -2.5).to(dtype)
    x[3, 1::2] = -math.inf
    tokens, logprobs = run(x, u)
    kept = [vocab] * 5
    kept[3] = (vocab + 1) // 2
    want = [math.floor(f32(a) * n) for a, n in zip(u, kept)]
    want[3] *= 2
    assert tokens.tolist() == want
    assert torch.allclose(logprobs.double(), -torch.tensor(kept).double().log(), rtol=2**-21, atol=0)
    tokens, _ = run(x[:3], u[:3], top_k=[vocab - 1, 4097, 60000])
    assert tokens.tolist() == [math.floor(f32(a) * min(k, vocab)) for a, k in zip(u, [vocab - 1, 4097, 60000])]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_both_zeros_many_times_over(dtype):
    """Zeros of either sign are one logit, also where both counters overflow; a few others stand beside them."""
    n = 150001
    x = torch.zeros(3, n)
    x[:, 1::2] = -0.0
    x[1, 100] = 3.0
    x[2, ::5] = -1.0
    x = x.to(dtype)
    assert bool(torch.signbit(x[0, 1])) and not bool(torch.signbit(x[0, 0]))
    check(x, [0.731, 0.602, 0.987], top_k=[0, 90001, 0], temperature=[1.0, 0.9, 1.1])


def test_the_largest_numbers():
    """Differences that overflow, temperatures at both ends, logits next to the type's largest."""
    big = torch.finfo(torch.float32).max
    x = torch.tensor([[big, -big, 0.0, big / 2], [-big, -big, -big, -big * 0.5], [1e30, 2e30, -1e30, 0.0], [1e-40, 0.0, -1e-40, 3e-39]])
    # By hand: all weight at the largest; the same; e^1, e^2, e^-1, 1 at T = 1e30; four equal weights.
    tokens, logprobs = run(x, [0.999, 0.999, 0.2, 0.99], temperature=[1.0, 1.0, 1e35, 1.0])
    w = [math.exp(v) for v in (1, 2, -1, 0)]
    assert tokens.tolist()[:2] == [0, 3] and logprobs[0] == 0 and logprobs[1] == 0
    assert tokens[2] == 1 and abs(float(logprobs[2]) - math.log(w[1] / sum(w))) < 1e-6
    assert abs(float(logprobs[3]) + math.log(4)) < 1e-6
    for dtype in (torch.bfloat16, torch.float16):
        top = torch.finfo(dtype).max
        y = torch.tensor([[top, -top, 0.0], [-top, -top, -top], [math.inf, top, math.inf], [-math.inf, math.nan, -top]]).to(dtype)
        tokens, logprobs = run(y, [0.99, 0.5, 0.6, 0.9])
        assert tokens.tolist() == [0, 1, 2, 2]
        assert logprobs[0] == 0 and logprobs[3] == 0 and abs(float(logprobs[2]) + math.log(2)) < 1e-6


def test_cuts_that_are_no_numbers():
    """NaN as top_p or min_p is above nothing and below nothing: no cut."""
    x = normal(4, 2003, seed=21)
    u = [0.9, 0.8, 0.7, 0.95]
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        want, _ = run(y, u)
        got, _ = run(y, u, top_p=[math.nan] * 4, min_p=[math.nan] * 4)
        assert got.tolist() == want.tolist()
        got, _ = run(y, u, top_p=[math.inf, 2.0, 1.0, 1.5], min_p=[-math.inf, -1.0, 0.0, -0.0], top_k=[-(2**31), 2**31 - 1, 0, -1])
        assert got.tolist() == want.tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_rows_and_slices_at_their_ends(dtype):
    """Thousands of rows; vocabularies around whole slices, from an aligned place and from others."""
    x = normal(7, 130, dtype, seed=31)
    u = [0.11, 0.36, 0.5, 0.62, 0.77, 0.81, 0.93]
    want = [S.sample_row(x[i].float(), f32(u[i]))[0] for i in range(7)]
    import block_sparse_top_msa_gb300 as msa
    got = msa.msa_sample(x.to(DEV).repeat(3000, 1), torch.tensor(u, device=DEV).repeat(3000))
    assert torch.equal(got.view(3000, 7).cpu(), torch.tensor(want, dtype=torch.int32).expand(3000, 7))
    for rows, vocab in ((2, 2048), (2, 2045), (2, 2046), (40, 8192 * 8), (40, 8192 * 8 - 3), (38, 8192 * 8 - 2), (38, 8192 * 8 + 1)):
        flat = normal(1, rows * vocab + 8, dtype, seed=vocab)[0].to(DEV)
        a = torch.rand(rows, generator=torch.Generator().manual_seed(rows)).to(DEV)
        for lo in (0, 1, 3):
            y = flat[lo : lo + rows * vocab].view(rows, vocab)
            got = msa.msa_sample(y, a)
            for i in (0, 1, rows - 1):
                w = S.sample_row(y[i].cpu().float(), float(a[i]))
                assert not w[2] or int(got[i]) == w[0], (rows, vocab, lo, i)
    fault_clear(msa)


def test_two_calls_at_once(msa):
    """Two streams, each with its own workspace, over and over."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    x = [normal(40, 30011, torch.float32, seed=1).to(DEV), normal(200, 30011, torch.bfloat16, seed=2).to(DEV)]
    u = [torch.rand(len(y), generator=torch.Generator().manual_seed(3)).to(DEV) for y in x]
    want = [msa.msa_sample(a, b, return_logprobs=True) for a, b in zip(x, u)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(msa.msa_sample(x[i], u[i], return_logprobs=True))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1])
    fault_clear(msa)


@pytest.mark.parametrize("shared", [True, False])
def test_the_most_requests_of_the_attention(msa, shared):
    """16384 requests of one token; all of them behind one page, or none."""
    g = torch.Generator().manual_seed(17)
    b, pages = 16384, 600
    table = torch.randint(0, pages, (b, 2), generator=g).to(torch.int32)
    used = torch.randint(1, 140, (b,), generator=g).to(torch.int32)
    if shared:
        table[:, 0] = 5
        used += 128
        used.clamp_(max=200)
    k, v = (torch.randn(pages, 1, 128, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(b, 1, 128, generator=g).to(torch.bfloat16)
    ints = lambda x: x.to(DEV)  # noqa: E731
    kw = {}
    ones = torch.ones(b, dtype=torch.int32, device=DEV)
    t = msa.msa_step_tables(ints(table), ints(used), torch.arange(b, dtype=torch.int32, device=DEV), ones, total_q=b, num_pages=pages)
    if shared:
        assert t.cu_groups.tolist()[1] == b and t.group_blocks.tolist()[0] == 1
        kw = dict(group_rows=t.group_rows, cu_groups=t.cu_groups, group_blocks=t.group_blocks)
    out, lse = msa.msa_prefix_attention(q.to(DEV), k.to(DEV), v.to(DEV), t.cu_seqlens_q, page_table=t.page_table, seqused_k=t.seqused_k, max_seqlen_q=1, return_softmax_lse=True, **kw)
    fault_clear(msa)
    # The plain form, for every 37th request.
    some = torch.arange(0, b, 37)
    cu = torch.arange(len(some) + 1, dtype=torch.int32)
    c = dict(q=q[some], k=k, v=v, cu=cu, table=table[some], used=used[some])
    check_attention(c, out[some.to(DEV)], lse[some.to(DEV)])
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
