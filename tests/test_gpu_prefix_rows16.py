"""The attention over shared prefixes in units of 16 rows: requests without groups, the bound on whose tokens times the query heads
of a KV head is at most 16. Tolerances are those of test_gpu_prefix_attention.py."""
import pytest
import torch

from test_gpu_prefix_attention import DEV, check, make, msa, run  # noqa: F401

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "fp16", "e4m3"]


def small(c):
    """The bound that a caller knows: the most tokens of a request."""
    most = int((c["cu"][1:] - c["cu"][:-1]).max())
    assert 0 < most * (c["q"].shape[1] // c["k"].shape[1]) <= 16
    return most


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("requests,hq,hkv", [
    ([(0, 1)], 16, 1), ([(127, 1)], 8, 8), ([(128, 1), (0, 1)], 12, 3),
    # One to sixteen heads a KV head, one to sixteen tokens: full tiles and others.
    ([(300, 16), (5, 3), (0, 16)], 2, 2), ([(300, 2), (129, 1), (700, 2)], 16, 2), ([(300, 1), (129, 1), (700, 1)], 32, 2), ([(260, 5), (100, 4)], 9, 3), ([(77, 3)], 5, 1), ([(200, 2), (90, 2)], 7, 1),
    # Empty requests between, a request of nothing but its new tokens, more tokens than keys are not given here.
    ([(50, 0), (0, 4), (0, 0), (200, 2)], 4, 1),
    # Many requests a CTA, each of a block or two.
    ([(i * 3 % 250, 1 + i % 2) for i in range(400)], 8, 2),
])
def test_requests(msa, requests, hq, hkv, kv):
    c = make([0] * len(requests), [[r] for r in requests], hq, hkv, kv, seed=81 + hq)
    check(c, *run(msa, c, groups=False, max_seqlen_q=small(c)))
    check(c, *run(msa, c, groups=False, max_seqlen_q=small(c), causal=False, softmax_scale=0.15), causal=False, scale=0.15)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("hq,hkv,new", [(16, 1, 1), (8, 1, 2), (2, 2, 8)])
def test_long_runs_and_short_ones_beside_them(msa, kv, hq, hkv, new):
    """Runs of hundreds of blocks, cut over many CTAs, whose pieces pass 32 blocks where the CTAs have more: a long request beside
    many others, so that a piece is long too."""
    c = make([0, 0, 0], [[(33000, new)], [(5, 1)], [(2500, new)]], hq, hkv, kv, seed=91)
    check(c, *run(msa, c, groups=False, max_seqlen_q=small(c)))


@pytest.mark.parametrize("kv", KINDS)
def test_pieces_of_more_than_32_blocks(msa, kv):
    """40 requests of 160 blocks of the same pages: 42 blocks a CTA."""
    n, lk = 40, 20450
    c = make([0], [[(lk - 1, 1)]], 16, 1, kv, seed=92)
    g = torch.Generator().manual_seed(5)
    for x in ("table", "used"):
        c[x] = c[x].repeat(n, *[1] * (c[x].dim() - 1))
    c["used"] -= torch.randint(0, 3000, (n,), generator=g).to(torch.int32)
    c["q"], c["cu"] = c["q"].repeat(n, 1, 1) * (1 + torch.arange(n) / n).to(c["q"].dtype)[:, None, None], torch.arange(n + 1, dtype=torch.int32)
    assert n * 160 > 32 * 152
    out, lse = run(msa, c, groups=False, max_seqlen_q=1)
    for lo in (0, 17, n - 1):
        one = dict(c, q=c["q"][lo : lo + 1], cu=c["cu"][:2], table=c["table"][lo : lo + 1], used=c["used"][lo : lo + 1])
        check(one, out[lo : lo + 1], lse[lo : lo + 1])


@pytest.mark.parametrize("kv", KINDS)
def test_pages_that_are_not_there(msa, kv):
    c = make([0] * 4, [[(1500, 2)], [(200, 3)], [(40, 1)], [(127, 3)]], 10, 2, kv, seed=93)
    long = int(c["used"].argmax())
    c["table"][long, 0] = -1
    c["table"][long, 3:5] = c["k"].shape[0]
    c["table"][long, 11] = 2**31 - 1
    c["table"][long, 7] = -(2**31)
    c["table"][int((c["used"] == 41).nonzero()[0]), 0] = -7  # all of a request's
    out, lse = run(msa, c, groups=False, max_seqlen_q=small(c))
    check(c, out, lse)
    assert int((lse == -float("inf")).sum()) == 10
    c["table"] = c["table"][:, :2].contiguous()  # rows that end before their requests do
    check(c, *run(msa, c, groups=False, max_seqlen_q=small(c)))


def test_more_tokens_than_keys(msa):
    for kv in KINDS:
        c = make([0, 0], [[(0, 5)], [(20, 2)]], 3, 1, kv, seed=94)
        c["used"][:] = torch.where(c["used"] == 5, 2, c["used"])
        out, lse = run(msa, c, groups=False, max_seqlen_q=small(c))
        check(c, out, lse)
        assert int((lse == -float("inf")).sum()) == 9


def test_same_bits_on_a_stream_prepared_and_replayed(msa):
    for kv in KINDS:
        c = make([0] * 5, [[(n, 2)] for n in (5000, 300, 0, 127, 1000)], 16, 2, kv, seed=95, extra=3)
        out, lse = run(msa, c, groups=False, max_seqlen_q=2)
        for _ in range(3):
            again, lse2 = run(msa, c, groups=False, max_seqlen_q=2)
            assert torch.equal(out[:10], again[:10]) and torch.equal(lse[:10], lse2[:10])
        d = {n: t.to(DEV) for n, t in c.items()}
        runner = msa.PrefixAttentionRunner(d["q"], d["k"], d["v"], d["cu"], page_table=d["table"], seqused_k=d["used"], max_seqlen_q=2, return_softmax_lse=True,
                                           out=torch.full_like(d["q"], 3.0), lse=torch.full(d["q"].shape[:2], 3.0, device=DEV))
        runner.workspace.fill_(0xFF)
        graph = torch.cuda.CUDAGraph()
        runner.run()
        with torch.cuda.graph(graph):
            runner.run()
        graph.replay()
        assert torch.equal(out[:10], runner.out[:10]) and torch.equal(lse[:10], runner.lse[:10])
        assert (runner.out[10:] == 3).all() and (runner.lse[10:] == 3).all()
        d["used"] -= 1
        graph.replay()
        torch.cuda.synchronize()
        check(dict(c, used=c["used"] - 1), runner.out, runner.lse)
