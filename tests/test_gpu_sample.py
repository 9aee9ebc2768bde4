"""Sampling against a walk through the sorted tokens in 64 bits."""
import math

import pytest
import torch

import samples_util as S

pytestmark = pytest.mark.gpu
INF = math.inf


def run(x, u, device="cuda", **cuts):
    import block_sparse_top_msa_gb300 as msa
    types = {"top_k": torch.int32}
    cuts = {n: torch.tensor(c, dtype=types.get(n, torch.float32), device=device) for n, c in cuts.items()}
    tokens, logprobs = msa.msa_sample(x.to(device), torch.tensor(u, dtype=torch.float32, device=device), return_logprobs=True, **cuts)
    assert msa.msa_read_device_fault() == 0
    return tokens.cpu(), logprobs.cpu()


def check(x, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """Every row against 64 bits. A border that the weights' rounding may move is a fault of the inputs."""
    cuts = {n: c for n, c in dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p).items() if c is not None}
    f32 = lambda c, i, other: other if c is None else float(torch.tensor(c[i], dtype=torch.float32))  # noqa: E731
    want = [S.sample_row(x[i].float(), float(torch.tensor(u[i], dtype=torch.float32)), f32(temperature, i, 1.0), top_k[i] if top_k else 0, f32(top_p, i, 1.0), f32(min_p, i, 0.0)) for i in range(len(u))]
    assert all(w[2] for w in want), [i for i, w in enumerate(want) if not w[2]]
    tokens, logprobs = run(x, u, **cuts)
    assert tokens.tolist() == [w[0] for w in want]
    for got, (_, lp, _) in zip(logprobs.tolist(), want):
        # The difference to the maximum, its product with 1 / T, the logarithm and their difference: a rounding each.
        assert got == lp or abs(got - lp) <= 6 * 2**-24 * max(1.0, abs(lp)) + 2**-22


def normal(rows, vocab, dtype=torch.float32, spread=2.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(rows, vocab, generator=g)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 300, 4099, 32001, 131072, 200019])
def test_cuts_of_random_rows(vocab, dtype):
    n = 12
    u = [(37 * i + 5) % 101 / 101 for i in range(n)]
    check(normal(n, vocab, dtype, seed=vocab), u, temperature=[1.0, 0.7, 1.3, 1.0] * 3, top_k=[0, 1, 5, 50, 1000, -3, vocab, vocab + 1, 0, 2, 3, 100],
          top_p=[0.9, 1.0, 0.5, 0.95, 0.99, 0.3, 1.0, 0.999, 0.01, 1.0, 0.6, 0.8], min_p=[0.0, 0.0, 0.02, 0.0, 0.001, 0.1, 0.0, 0.0, 0.5, 0.3, 0.0, 0.05])


@pytest.mark.parametrize("cuts", [dict(), dict(top_k=[40] * 6), dict(top_p=[0.9] * 6), dict(min_p=[0.03] * 6), dict(temperature=[0.1, 0.5, 2.0, 10.0, 1e-4, 100.0])])
@pytest.mark.parametrize("spread", [0.01, 0.3, 4.0, 30.0])
def test_each_cut_by_itself(cuts, spread):
    check(normal(6, 5003, spread=spread, seed=3), [0.03, 0.2, 0.41, 0.6, 0.83, 0.97], **cuts)


@pytest.mark.parametrize("vocab", [5, 1000, 50000])
def test_equal_logits_go_by_their_number(vocab):
    """Flat rows: all weights are 1, and the token is the whole part of u times the number that is kept."""
    u = [0.0, 0.1, 0.5, 0.77, 0.999, 0.25]
    x = torch.full((6, vocab), -3.25)
    tokens, logprobs = run(x, u)
    assert tokens.tolist() == [int(float(torch.tensor(a)) * vocab) for a in u]
    assert torch.allclose(logprobs, torch.full((6,), -math.log(vocab)), rtol=2**-21, atol=0)
    k = max(1, vocab // 3)
    tokens, _ = run(x, u, top_k=[k] * 6)
    assert tokens.tolist() == [int(float(torch.tensor(a)) * k) for a in u]
    tokens, _ = run(x, u, top_p=[0.5] * 6)
    half = (vocab + 1) // 2
    assert tokens.tolist() == [int(float(torch.tensor(a)) * half) for a in u]


def test_few_distinct_logits():
    """Ties everywhere: cuts and samples end inside runs of equal tokens."""
    g = torch.Generator().manual_seed(8)
    x = torch.randint(-3, 4, (10, 30011), generator=g).float()
    check(x, [i / 10 + 0.037 for i in range(10)], temperature=[0.9] * 10, top_k=[0, 7, 4000, 5000, 0, 0, 12000, 1, 300, 20000], top_p=[1, 1, 1, 0.7, 0.41, 0.87, 0.5, 0.5, 0.9, 0.99])


def test_zeros_of_both_signs_are_equal():
    x = torch.tensor([[0.0, -0.0, -1.0, 0.0], [-0.0, 0.0, -1.0, -0.0]])
    tokens, _ = run(x, [0.0, 0.0])
    assert tokens.tolist() == [0, 0]
    tokens, _ = run(x, [0.5, 0.5], top_k=[3, 3])
    assert tokens.tolist() == [1, 1]


def test_masked_tokens_infinities_and_nan():
    n = 500
    x = normal(8, n, seed=5)
    x[0, ::2] = -INF
    x[1, 1:] = -INF
    x[2] = -INF
    x[3, 7] = math.nan
    x[4] = math.nan
    x[5, 400], x[5, 30] = INF, INF
    x[6, 100:] = torch.finfo(torch.float32).min
    x[7, :] = torch.finfo(torch.float32).min
    u = [0.4, 0.9, 0.5, 0.7, 0.5, 0.6, 0.99, 0.5]
    tokens, logprobs = run(x, u, top_p=[1.0, 0.9, 0.9, 1.0, 1.0, 1.0, 1.0, 1.0], min_p=[0.0, 0.5, 0.1, 0.0, 0.0, 0.3, 0.0, 0.0])
    want = [S.sample_row(x[i], u[i]) for i in (0, 3, 6)]
    assert tokens.tolist() == [want[0][0], 0, -1, want[1][0], -1, 400, want[2][0], 250]
    assert logprobs[1] == 0 and logprobs[2] == -INF and logprobs[4] == -INF
    assert abs(float(logprobs[5]) + math.log(2)) < 1e-6 and abs(float(logprobs[7]) + math.log(n)) < 1e-5


def test_the_numbers_that_leave_nothing_to_choose():
    x = normal(12, 3001, seed=6)
    best = x.argmax(1).tolist()
    tokens, logprobs = run(x, [0.999] * 12, temperature=[0.0, -1.0, math.nan, 1e-6] + [1.0] * 8, top_k=[0] * 4 + [1] + [0] * 7, top_p=[1.0] * 5 + [0.0, -0.5, 1e-7] + [1.0] * 4,
                           min_p=[0.0] * 8 + [1.0, 7.0, 0.0, 0.0])
    assert tokens.tolist()[:10] == best[:10]
    lse = torch.logsumexp(x.double(), 1)
    for i in range(10):
        assert abs(float(logprobs[i]) - float(x[i].double().max() - lse[i])) < 1e-5
    # Numbers outside [0, 1): the first token, the last that has a weight.
    tokens, _ = run(x, [-1.0, 1.0, math.nan] * 4)
    for i in range(12):
        assert tokens[i] == (int(x[i].argmax()) if i % 3 == 0 else int(x[i].argmin()))
    cold = x.clone()
    cold[:, 10:] -= 1000.0
    tokens, _ = run(cold, [1.0] * 12, temperature=[0.5] * 12)
    assert all(int(t) == int(cold[i, :10].argmin()) for i, t in enumerate(tokens))


def test_rows_at_a_distance_and_odd_places():
    """Rows of a wider tensor, that begin anywhere within 16 bytes."""
    wide = normal(5, 1013, torch.bfloat16, seed=9)
    u = [0.1, 0.3, 0.5, 0.7, 0.9]
    import block_sparse_top_msa_gb300 as msa
    dev = wide.cuda()
    for lo, n in ((0, 1000), (1, 1000), (3, 77), (7, 1), (5, 1008), (9, 16)):
        got = msa.msa_sample(dev[:, lo : lo + n], torch.tensor(u, device="cuda"))
        want = [S.sample_row(wide[i, lo : lo + n].float(), float(torch.tensor(u[i]))) for i in range(5)]
        assert got.tolist() == [w[0] for w in want], (lo, n)
    flat = normal(1, 4100, seed=2)[0].cuda()
    for lo in range(4):
        got = msa.msa_sample(flat[lo : lo + 4001][None], torch.tensor([0.6], device="cuda"))
        assert got.item() == S.sample_row(flat[lo : lo + 4001].cpu(), float(torch.tensor(0.6)))[0]


def test_no_rows_and_the_largest_vocabulary():
    import block_sparse_top_msa_gb300 as msa
    assert msa.msa_sample(torch.empty(0, 50, device="cuda"), torch.empty(0, device="cuda")).shape == (0,)
    x = normal(2, 1 << 19, seed=12)
    check(x, [0.31, 0.86], top_p=[0.9, 1.0])
    x = normal(2, 1 << 19, torch.float16, spread=0.2, seed=13)
    check(x, [0.31, 0.86], top_k=[0, 100000])


def test_many_rows_alike_captured_and_on_another_stream():
    """The same row many times over gives the same token, eagerly, on a side stream and in a replayed graph with new numbers."""
    import block_sparse_top_msa_gb300 as msa
    x = normal(1, 20011, seed=4).cuda().expand(700, -1)
    u = torch.full((700,), 0.618, device="cuda")
    want = S.sample_row(x[0].cpu(), float(torch.tensor(0.618)), 1.0, 0, float(torch.tensor(0.95)))[0]
    p = torch.full((700,), 0.95, device="cuda")
    dense = x.contiguous()
    assert msa.msa_sample(dense, u, top_p=p).eq(want).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = msa.msa_sample(dense, u, top_p=p, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert out.eq(want).all()
    tokens, lps = torch.empty(700, dtype=torch.int32, device="cuda"), torch.empty(700, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_sample(dense, u, top_p=p, tokens=tokens, logprobs=lps)
    for a in (0.618, 0.05, 0.93):
        u.fill_(a)
        graph.replay()
        assert tokens.eq(S.sample_row(x[0].cpu(), float(torch.tensor(a)), 1.0, 0, float(torch.tensor(0.95)))[0]).all()
    assert msa.msa_read_device_fault() == 0


def test_frequencies_follow_the_probabilities():
    """Numbers spread evenly over [0, 1): each token comes as often as its share says, to one number at each of its ends."""
    import block_sparse_top_msa_gb300 as msa
    n = 4096
    x = normal(1, 12, seed=1)
    u = ((torch.arange(n) + 0.5) / n).cuda()
    got = torch.bincount(msa.msa_sample(x.cuda().expand(n, -1).contiguous(), u).long().cpu(), minlength=12)
    assert bool(((got - torch.softmax(x[0].double(), 0) * n).abs() <= 2).all())
