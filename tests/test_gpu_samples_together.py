"""A serving loop of samples, operator after operator: prompts, their forks, steps of one token and a step of drafted chains, each
operator held to what it got: tables, paths, tokens and lengths exactly, attention by the tolerances of its own tests (queries and
keys are normalised here, so that a logit's sum of magnitudes stays below 16 as it does there)."""
import pytest
import torch

import samples_util as S
import workloads
from parity_util import fault_clear
from step_util import DT, Tables, accept, bits, rope_table, tree_bits
from test_gpu_prefix_attention import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HQ, HKV, ROWS, MAX_PAGES, PAGES, VOCAB = 8, 2, 7, 6, 24, 700


@pytest.fixture(scope="module")
def msa():
    import block_sparse_top_msa_gb300 as m
    m.build()
    m.lib()
    return m


class Loop:
    """One layer whose q, k and v are read from a table by token, and whose logits are its output's first values."""

    def __init__(self, msa, kv, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.msa, self.dtype = msa, torch.float16 if kv == "fp16" else torch.bfloat16
        self.plain = Tables(ROWS, MAX_PAGES, PAGES)
        self.table, self.used, self.refs = self.plain.tensors(DEV)
        self.k, self.v = (torch.zeros(PAGES, HKV, 128, 128, device=DEV).to(DT[kv]) for _ in range(2))
        self.embed = torch.randn(VOCAB, HQ + 2 * HKV, 128, generator=g).to(self.dtype).to(DEV)
        self.angles, self.ones = rope_table(MAX_PAGES * 128, 64).to(DEV), torch.ones(128, device=DEV)

    def tables(self, rows, counts, total, out=None):
        return self.msa.msa_step_tables(self.table, self.used, rows, counts, total_q=total, num_pages=PAGES, out=out)

    def attend(self, tokens, t, most, stream=None):
        x = self.embed[tokens.long()]
        q = self.msa.msa_qk_norm_rope_append(x[:, :HQ], x[:, HQ : HQ + HKV], x[:, HQ + HKV :], self.ones, self.ones, self.angles, t.positions, t.cu_seqlens_q, self.k, self.v,
                                             page_table=t.page_table, seqused_k=t.seqused_k, stream=stream)
        out, lse = self.msa.msa_prefix_attention(q, self.k, self.v, t.cu_seqlens_q, page_table=t.page_table, seqused_k=t.seqused_k, group_rows=t.group_rows,
                                                 cu_groups=t.cu_groups, group_blocks=t.group_blocks, max_seqlen_q=most, return_softmax_lse=True, stream=stream)
        return q, out, lse

    def logits(self, out):
        return 6 * out.flatten(1)[:, :VOCAB].float()

    def step(self, rows, counts, tokens, u, cuts):
        """Extends the rows, runs the step and checks it; returns the tables and each token's sample."""
        lengths = [self.plain.used[r] + n for r, n in zip(rows, counts)]
        got = self.msa.msa_cache_extend(self.table, self.used, self.refs, S.ints(rows), S.ints(lengths))
        assert got.tolist() == self.plain.extend(rows, lengths) == [0] * len(rows)
        total = sum(counts) + 2  # two tokens of padding
        t = self.tables(S.ints(rows), S.ints(counts), total)
        want = S.step_tables(self.plain.table, self.plain.used, rows, counts, total, PAGES)
        assert [x.tolist() for x in t] == list(want)
        tokens = torch.cat([tokens, torch.zeros(2, dtype=torch.int32, device=DEV)])
        q, out, lse = self.attend(tokens, t, max(counts))
        fault_clear(self.msa)
        c = dict(q=q.cpu(), k=self.k.cpu(), v=self.v.cpu(), cu=t.cu_seqlens_q.cpu(), table=t.page_table.cpu(), used=t.seqused_k.cpu())
        check(c, out, lse)
        n = sum(counts)
        x = self.logits(out[:n])
        picked, logprobs = self.msa.msa_sample(x, u[:n], return_logprobs=True, **{m: v.expand(n).contiguous() for m, v in cuts.items()})
        plain = [S.sample_row(row, float(a), *(float(cuts[m][0]) if m != "top_k" else int(cuts[m][0]) for m in ("temperature", "top_k", "top_p", "min_p")))
                 for row, a in zip(x.cpu(), u.cpu())]
        assert all(p[2] for p in plain)
        assert picked.tolist() == [p[0] for p in plain]
        assert torch.allclose(logprobs.cpu().double(), torch.tensor([p[1] for p in plain], dtype=torch.float64), rtol=6 * 2.0**-24, atol=2.0**-21)
        return t, picked


def cuts_of(t, k, p, m):
    return dict(temperature=torch.tensor([t], device=DEV), top_k=S.ints([k]), top_p=torch.tensor([p], device=DEV), min_p=torch.tensor([m], device=DEV))


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
def test_samples_of_two_prompts_and_their_drafts(msa, kv):
    loop = Loop(msa, kv)
    g = torch.Generator().manual_seed(5)
    tokens = lambda n: torch.randint(0, VOCAB, (n,), generator=g).to(torch.int32).to(DEV)  # noqa: E731
    u = lambda n: torch.rand(n, generator=g).to(DEV)  # noqa: E731
    # Both prompts in one step; then samples of them, each with the page that it writes to of its own.
    _, first = loop.step([0, 1], [300, 131], tokens(431), u(431), cuts_of(1.0, 50, 0.95, 0.0))
    last = {0: first[299], 1: first[430]}
    got = msa.msa_cache_fork([loop.k, loop.v], loop.table, loop.used, loop.refs, S.ints([0, 0, 1]), S.ints([2, 5, 4]))
    assert got.tolist() == loop.plain.fork([0, 0, 1], [2, 5, 4]) == [0, 0, 0]
    last.update({2: last[0], 5: last[0], 4: last[1]})
    order = [5, 1, 0, 4, 2]
    for cuts in (cuts_of(1.0, 0, 0.9, 0.0), cuts_of(0.8, 40, 1.0, 0.02), cuts_of(0.0, 0, 1.0, 0.0)):
        t, picked = loop.step(order, [1] * 5, torch.stack([last[r] for r in order]), u(5), cuts)
        assert t.group_blocks.tolist()[:2] == [2, 1]  # whole blocks of 300 and 131 tokens
        last = dict(zip(order, picked))
    # Chains of drafts behind each row's token; of some the next ones are what was sampled.
    counts = [4, 1, 3, 6, 2]
    drafts = tokens(sum(counts))
    cu = workloads.cu_from_lengths(counts)
    for i, r in enumerate(order):
        drafts[cu[i]] = last[r]
    t, picked = loop.step(order, counts, drafts, u(16), cuts_of(0.0, 0, 1.0, 0.0))
    known = drafts.clone()
    known[1:3], known[9:13] = picked[0:2], picked[8:12]  # two of the first row's, four of the fourth's
    mask = torch.cat([tree_bits([i - 1 for i in range(n)]) for n in counts]).to(DEV)
    path, path_len, after = msa.msa_draft_path(picked, known, mask, t.cu_seqlens_q, max_path=6)
    want = S.draft_path(picked.tolist(), known.tolist(), [[int(w) for w in row] for row in mask.tolist()], cu.tolist(), 6, 16)
    assert (path.tolist(), path_len.tolist(), after.tolist()) == tuple(want)
    assert path_len.tolist()[0] >= 3 and path_len.tolist()[3] >= 5
    mirror = [bits(x.cpu()) for x in (loop.k, loop.v)]
    lengths = msa.msa_cache_accept([loop.k, loop.v], t.page_table, t.seqused_k, t.cu_seqlens_q, path, path_len)
    assert lengths.tolist() == accept(mirror, t.page_table.cpu(), t.seqused_k.cpu(), cu, path.cpu(), path_len.cpu())
    assert all(torch.equal(bits(x.cpu()), y) for x, y in zip((loop.k, loop.v), mirror))
    loop.used[torch.tensor(order, device=DEV)] = lengths
    for r, n in zip(order, lengths.tolist()):
        loop.plain.used[r] = n
    loop.step(order, [1] * 5, after, u(5), cuts_of(1.3, 0, 0.99, 0.0))
    fault_clear(msa)


def test_a_captured_step_replayed_and_on_a_side_stream(msa):
    """One graph of a whole step, replayed over a growing cache, gives what the calls give one by one; so does a side stream."""
    def start():
        loop = Loop(msa, "bf16", seed=3)
        g = torch.Generator().manual_seed(9)
        loop.step([0], [260], torch.randint(0, VOCAB, (260,), generator=g).to(torch.int32).to(DEV), torch.rand(260, generator=g).to(DEV), cuts_of(1.0, 0, 1.0, 0.0))
        msa.msa_cache_fork([loop.k, loop.v], loop.table, loop.used, loop.refs, S.ints([0] * 3), S.ints([1, 2, 3]))
        state = dict(rows=S.ints([2, 0, 3, 1]), counts=S.ints([1] * 4), tokens=S.ints([5, 6, 7, 8]), u=torch.rand(4, generator=g).to(DEV), p=torch.full((4,), 0.9, device=DEV))
        return loop, state

    def one(loop, s, stream=None):
        at = s["rows"].long()
        msa.msa_cache_extend(loop.table, loop.used, loop.refs, s["rows"], (loop.used[at] + 1).to(torch.int32), stream=stream)
        t = msa.msa_step_tables(loop.table, loop.used, s["rows"], s["counts"], total_q=4, num_pages=PAGES, stream=stream)
        _, out, lse = loop.attend(s["tokens"], t, 1, stream)
        picked = msa.msa_sample(loop.logits(out), s["u"], top_p=s["p"], stream=stream)
        s["tokens"].copy_(picked)
        s["u"].mul_(0.83)
        return out, lse, picked

    want = []
    loop, s = start()
    for _ in range(6):
        want.append([x.clone() for x in one(loop, s)])
    # Captured: a replay reads the tables as they are then. The cache is begun anew, so the first call is the graph's.
    loop, s = start()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one(loop, s)
    for i in range(6):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
    loop, s = start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(6):
            got = one(loop, s)
            assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
    torch.cuda.current_stream().wait_stream(side)
    fault_clear(msa)
