"""A serving loop of drafted trees, operator after operator: pages for the prompts, their K and V, a fork, then steps of extension,
append, attention over the drafts and acceptance, with a row freed in between, against the plain forms. Each operator is held to
what it got: tables, counts and moved rows to the byte, appended rows and outputs by the tolerances of their own tests (one
rounding behind 2^-20 of the magnitudes; a probability's rounding and 2^-13)."""
import pytest
import torch

import workloads
from parity_util import fault_clear
from step_util import DT, Tables, accept, bits, half_step, norm_rope, pad_words, rope_table, tree_attention, tree_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HQ, HKV, LAYERS, ROWS, MAX_PAGES, PAGES, TOPK = 16, 2, 2, 5, 6, 20, 3
CHAIN = 2.0**-20
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0**-25, torch.float8_e4m3fn: 2.0**-10}


@pytest.fixture(scope="module")
def msa():
    import block_sparse_top_msa_gb300 as m
    m.build()
    m.lib()
    return m


class Loop:
    def __init__(self, msa, kv, seed=0):
        self.msa, self.kv = msa, kv
        self.g = torch.Generator().manual_seed(seed)
        self.dtype = torch.float16 if kv == "fp16" else torch.bfloat16
        self.plain = Tables(ROWS, MAX_PAGES, PAGES)
        self.table, self.used, self.refs = self.plain.tensors(DEV)
        self.pools = torch.zeros(2 * LAYERS, PAGES, HKV, 128, 128, device=DEV).to(DT[kv])
        self.angles = rope_table(MAX_PAGES * 128, 64)
        self.w = 1 + 0.3 * torch.randn(2, 128, generator=self.g)

    def same_tables(self):
        self.plain.check(self.table, self.used, self.refs)

    def extend(self, rows, lengths):
        got = self.msa.msa_cache_extend(self.table, self.used, self.refs, torch.tensor(rows, dtype=torch.int32, device=DEV),
                                        torch.tensor(lengths, dtype=torch.int32, device=DEV))
        assert got.tolist() == self.plain.extend(rows, lengths)
        self.same_tables()

    def fork(self, src, dst):
        mirror = [bits(p.cpu()) for p in self.pools]
        got = self.msa.msa_cache_fork(self.pools, self.table, self.used, self.refs, torch.tensor(src, dtype=torch.int32, device=DEV),
                                      torch.tensor(dst, dtype=torch.int32, device=DEV))
        assert got.tolist() == self.plain.fork(src, dst, mirror)
        self.same_tables()
        assert all(torch.equal(bits(p.cpu()), m) for p, m in zip(self.pools, mirror))

    def free(self, rows):
        self.msa.msa_cache_free(self.table, self.used, self.refs, torch.tensor(rows, dtype=torch.int32, device=DEV))
        self.plain.free(rows)
        self.same_tables()

    def batch(self, rows, counts):
        """Rows of the tables as a batch of so many new tokens each."""
        at = torch.tensor(rows, device=DEV)
        cu = workloads.cu_from_lengths(counts).to(DEV)
        return self.table[at].contiguous(), self.used[at].contiguous(), cu

    def append(self, layer, batch, positions):
        table, used, cu = batch
        x = torch.randn(len(positions), HQ + 2 * HKV, 128, generator=self.g).to(self.dtype)
        q, k, v = x[:, :HQ], x[:, HQ : HQ + HKV], x[:, HQ + HKV :]
        dev = x.to(DEV)
        before = bits(self.pools.cpu()).clone()
        out = self.msa.msa_qk_norm_rope_append(dev[:, :HQ], dev[:, HQ : HQ + HKV], dev[:, HQ + HKV :], self.w[0].to(DEV), self.w[1].to(DEV),
                                               self.angles.to(DEV), positions.to(DEV), cu, self.pools[2 * layer], self.pools[2 * layer + 1],
                                               page_table=table, seqused_k=used)
        yq, mq = norm_rope(q, self.w[0], self.angles, positions, False)
        yk, mk = norm_rope(k, self.w[1], self.angles, positions, False)
        assert ((out.cpu().double() - yq).abs() <= half_step(self.dtype) * (yq.abs() + CHAIN * mq) + CHAIN * mq + TINY[self.dtype]).all()
        after, pools = bits(self.pools.cpu()), self.pools.cpu()
        rows, cu, table = used.tolist(), cu.tolist(), table.tolist()
        step = half_step(DT[self.kv])
        for b, n in enumerate(rows):
            for t in range(cu[b], cu[b + 1]):
                p = n - cu[b + 1] + t
                page, row = table[b][p // 128], p % 128
                got = pools[2 * layer, page, :, row].double()
                assert ((got - yk[t]).abs() <= step * (yk[t].abs() + CHAIN * mk[t]) + CHAIN * mk[t] + TINY[DT[self.kv]]).all()
                want = v[t].float().clamp(-448, 448).to(DT[self.kv]) if self.kv == "e4m3" else v[t]
                assert torch.equal(bits(pools[2 * layer + 1, page, :, row].contiguous()), bits(want.contiguous()))
                before[2 * layer : 2 * layer + 2, page, :, row] = after[2 * layer : 2 * layer + 2, page, :, row]
        assert torch.equal(before, after)  # nothing else was written
        return out

    def attend(self, layer, q, batch, parents):
        table, used, cu = batch
        lens = (cu[1:] - cu[:-1]).tolist()
        mask = torch.cat([pad_words(tree_bits(p), 1) for p in parents if p])
        lists = torch.full((HKV, q.shape[0], TOPK), -1, dtype=torch.int32)
        t = 0
        for b, n in enumerate(lens):
            last = (int(used[b]) + 127) // 128
            for _ in range(n):
                for h in range(HKV):
                    near = sorted({max(0, int(used[b]) - n) // 128, last - 1})
                    rest = [x for x in torch.randperm(last, generator=self.g).tolist() if x not in near]
                    ids = sorted((near + rest)[:TOPK])
                    lists[h, t, : len(ids)] = torch.tensor(ids, dtype=torch.int32)
                t += 1
        out, lse = self.msa.msa_tree_attention(q, self.pools[2 * layer], self.pools[2 * layer + 1], lists.to(DEV), cu, mask.to(DEV), page_table=table,
                                               seqused_k=used, max_seqlen_q=max(lens), return_softmax_lse=True)
        ref, rl, size = tree_attention(q.cpu(), self.pools[2 * layer].float().cpu(), self.pools[2 * layer + 1].float().cpu(), lists, cu.cpu(), mask,
                                       table.cpu(), used.cpu(), 128**-0.5)
        # Weighted keys here reach twice the unit normal's logits: twice the 2^-13 of 16.
        tol = half_step(self.dtype) * (size + ref.abs()) * 1.01 + 2.0**-12 * size
        if self.dtype == torch.float16:
            tol += TOPK * 128 * 2.0**-25 * 6 + 2.0**-25
        assert ((out.double().cpu() - ref).abs() <= tol).all()
        assert ((lse.double().cpu() - rl).abs() <= 2.0**-12 + rl.abs() * 2.0**-21).all()

    def accept(self, rows, batch, path, path_len):
        table, used, cu = batch
        mirror = [bits(p.cpu()) for p in self.pools]
        got = self.msa.msa_cache_accept(self.pools, table, used, cu, path.to(DEV), path_len.to(DEV))
        want = accept(mirror, table.cpu(), used.cpu(), cu.cpu(), path, path_len)
        assert got.tolist() == want
        assert all(torch.equal(bits(p.cpu()), m) for p, m in zip(self.pools, mirror))
        self.used[torch.tensor(rows, device=DEV)] = got
        for r, n in zip(rows, want):
            self.plain.used[r] = n

    def drafted(self, rows, sizes):
        """A step: drafts of random trees, a random chain of each kept."""
        start = [self.plain.used[r] for r in rows]
        self.extend(rows, [s + n for s, n in zip(start, sizes)])
        batch = self.batch(rows, sizes)
        parents, positions, paths = [], [], []
        for s, n in zip(start, sizes):
            p = [int(torch.randint(-1, i, (1,), generator=self.g)) if i else -1 for i in range(n)]
            depth = []
            for i in range(n):
                depth.append(0 if p[i] < 0 else depth[p[i]] + 1)
            chain, at = [], int(torch.randint(0, n, (1,), generator=self.g))
            while at >= 0:
                chain.insert(0, at)
                at = p[at]
            parents.append(p)
            positions += [s + d for d in depth]
            paths.append(chain)
        positions = torch.tensor(positions, dtype=torch.int32)
        for layer in range(LAYERS):
            self.attend(layer, self.append(layer, batch, positions), batch, parents)
        path = torch.full((len(rows), max(sizes)), -1, dtype=torch.int32)
        for b, c in enumerate(paths):
            path[b, : len(c)] = torch.tensor(c, dtype=torch.int32)
        self.accept(rows, batch, path, torch.tensor([len(c) for c in paths], dtype=torch.int32))


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
def test_a_loop_of_steps(msa, kv):
    loop = Loop(msa, kv)
    prompts = [300, 127, 5]
    loop.extend([0, 1, 2], prompts)
    batch = loop.batch([0, 1, 2], prompts)
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in prompts])
    for layer in range(LAYERS):
        loop.append(layer, batch, positions)
    loop.fork([0, 2], [3, 4])
    loop.drafted([0, 1, 2, 3, 4], [7, 9, 1, 12, 3])
    loop.drafted([3, 0, 2], [2, 16, 5])  # some rows, in another order
    loop.free([0])
    loop.fork([1], [0])
    loop.drafted([0, 1, 2, 3, 4], [1, 1, 1, 1, 1])  # one token each
    loop.drafted([1, 4], [30, 20])
    loop.free([0, 1, 2, 3, 4])
    assert loop.refs.eq(0).all()
    fault_clear(msa)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_captured_step(msa, kv):
    """Extension, append, attention and acceptance of one shape captured once: replays continue the sequences as the calls do."""
    rows, n = 3, 6
    gen = torch.Generator().manual_seed(3)
    prompts = torch.tensor([250, 120, 3], dtype=torch.int32)
    x = torch.randn(3, rows * n, HQ + 2 * HKV, 128, generator=gen).to(torch.bfloat16).to(DEV)  # per step
    mask = torch.cat([tree_bits([-1, 0, 0, 1, 2, 2])] * rows).to(DEV)
    depth = torch.tensor([0, 1, 1, 2, 2, 2] * rows, dtype=torch.int32, device=DEV)
    path = torch.tensor([[0, 2, 5], [0, 1, -1], [-1, -1, -1]], dtype=torch.int32, device=DEV)
    path_len = torch.tensor([3, 2, 0], dtype=torch.int32, device=DEV)
    lists = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV).expand(HKV, rows * n, TOPK).contiguous()
    cu = torch.arange(rows + 1, dtype=torch.int32, device=DEV) * n
    angles, w = rope_table(MAX_PAGES * 128, 128).to(DEV), torch.ones(2, 128, device=DEV)
    which = torch.arange(rows, dtype=torch.int32, device=DEV)

    def state():
        plain = Tables(rows, MAX_PAGES, PAGES)
        plain.extend([0, 1, 2], prompts.tolist())
        g = torch.Generator().manual_seed(4)
        pools = torch.randn(2, PAGES, HKV, 128, 128, generator=g).to(DT[kv]).to(DEV)
        return (*plain.tensors(DEV), pools, x[0].clone(), torch.zeros(rows * n, HQ, 128, dtype=torch.bfloat16, device=DEV))

    def step(table, used, refs, pools, x, out):
        first = used.clone()
        lengths = used + n
        msa.msa_cache_extend(table, used, refs, which, lengths)
        positions = first.repeat_interleave(n, output_size=rows * n) + depth
        q = msa.msa_qk_norm_rope_append(x[:, :HQ], x[:, HQ : HQ + HKV], x[:, HQ + HKV :], w[0], w[1], angles, positions, cu, pools[0], pools[1],
                                        page_table=table, seqused_k=used)
        msa.msa_tree_attention(q, pools[0], pools[1], lists, cu, mask, page_table=table, seqused_k=used, max_seqlen_q=n, out=out)
        used.copy_(msa.msa_cache_accept(pools, table, used, cu, path, path_len))

    eager, seen = state(), []
    for i in range(3):
        eager[4].copy_(x[i])
        step(*eager)
        seen.append([t.clone() for t in eager[:4]] + [eager[5].clone()])
    held = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*state())  # first launches outside the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*held)
    for i in range(3):
        held[4].copy_(x[i])
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip([*held[:4], held[5]], seen[i]):
            same = torch.equal(got, want) if got.dtype == torch.int32 else torch.equal(bits(got), bits(want))
            assert same
    fault_clear(msa)
