"""Pages of a cache: extended, forked, freed, copied, and accepted drafts moved, against plain lists. All of it is copies and whole
numbers: results are equal."""
import pytest
import torch

from step_util import DT, Tables, accept, bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def msa():
    import block_sparse_top_msa_gb300 as m
    m.build()
    m.lib()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Both:
    """The tables as plain lists and on the GPU, with pools, each operation on both and compared."""

    def __init__(self, msa, rows, max_pages, num_pages, pools=3, shape=(2, 128, 16), dtype="bf16", seed=0, offset=0):
        self.msa, self.plain = msa, Tables(rows, max_pages, num_pages)
        g = torch.Generator().manual_seed(seed)
        self.pools = [torch.randn(num_pages, *shape, generator=g).to(DT[dtype]) for _ in range(pools)]
        self.gpu_pools = [p.to(DEV) for p in self.pools]
        self.offset = offset
        self.push()

    def push(self):
        t, u, r = self.plain.tensors(DEV)
        if self.offset:  # counts that do not start on a 16-byte boundary
            r = torch.cat([r.new_zeros(self.offset), r])[self.offset :]
        self.t, self.u, self.r = t, u, r

    def check(self):
        self.plain.check(self.t, self.u, self.r)
        for a, b in zip(self.pools, self.gpu_pools):
            assert torch.equal(bits(a), bits(b.cpu()))

    def extend(self, rows, lengths):
        want = self.plain.extend(rows, lengths)
        got = self.msa.msa_cache_extend(self.t, self.u, self.r, i32(rows), i32(lengths))
        assert got.tolist() == want
        self.check()
        return want

    def fork(self, src, dst):
        want = self.plain.fork(src, dst, [bits(p) for p in self.pools])
        got = self.msa.msa_cache_fork(self.gpu_pools, self.t, self.u, self.r, i32(src), i32(dst))
        assert got.tolist() == want
        self.check()
        return want

    def free(self, rows):
        self.plain.free(rows)
        self.msa.msa_cache_free(self.t, self.u, self.r, i32(rows))
        self.check()


@pytest.mark.parametrize("offset", [0, 1])
def test_life_of_a_batch(msa, offset):
    c = Both(msa, 6, 4, 11, offset=offset)
    assert c.extend([0, 1, 2], [300, 128, 1]) == [0, 0, 0]
    assert c.extend([0, 1, 2], [300, 129, 128]) == [0, 0, 0]  # no change, one more page, none
    assert c.fork([0, 0, 1], [3, 4, 5]) == [0, 0, 0]
    c.free([0, 4])
    assert c.fork([3], [0]) == [0]
    c.free([5, 5, 1])
    assert c.extend([1, 5, 4], [512, 100, 40]) == [0, 0, 0]
    assert c.extend([2, 4], [300, 129]) == [2, 2]  # not a page left
    c.free([0, 1, 2, 3, 4, 5])
    assert c.plain.refs == [0] * 11


def test_refusals(msa):
    c = Both(msa, 5, 3, 20)
    c.extend([0, 1], [200, 384])
    assert c.extend([0, 0, -1, 5, 1, 2, 3], [210, 220, 5, 5, 385, -1, 0]) == [0, 1, 1, 1, 1, 1, 0]
    assert c.extend([0], [100]) == [1]
    # twice to one row, a row onto itself, a chain, onto a row with tokens, out of range
    assert c.fork([0, 1, 2, 3, 0, 9, 0], [2, 2, 3, 3, 1, 4, -1]) == [0, 1, 1, 1, 1, 1, 1]
    assert c.fork([4], [3]) == [0]  # an empty row
    # a row without tokens that holds a page
    c.plain.table[3][2], c.plain.refs[17] = 17, 1
    c.push()
    assert c.fork([0], [3]) == [1]
    c.free([3, 100, -1])


def test_too_few_pages(msa):
    """Served in order until one does not fit; those that need no page still are."""
    c = Both(msa, 8, 4, 6)
    assert c.extend([0, 1, 2, 3, 4], [256, 300, 300, 0, 1]) == [0, 0, 2, 0, 2]
    c.free([0])
    assert c.fork([1, 1, 1, 1], [5, 6, 7, 0]) == [0, 0, 0, 2]
    c.free([1, 5, 6, 7])
    assert c.plain.refs == [0] * 6


def test_pages_out_of_range_or_missing(msa):
    """Entries that name no page are passed over everywhere."""
    c = Both(msa, 4, 4, 9)
    c.extend([0], [500])
    c.plain.table[0][1], c.plain.refs[1] = 9, 0
    c.plain.table[0][3], c.plain.refs[3] = -1, 0
    c.push()
    assert c.fork([0], [1]) == [0]
    assert c.extend([0], [512]) == [0]
    c.free([0, 1])
    assert c.plain.refs == [0] * 9


def test_many_rows_and_pages(msa):
    """More requests than a block has threads, more pages than one step of the search, with holes between."""
    g = torch.Generator().manual_seed(2)
    rows, pages = 2300, 40001
    c = Both(msa, rows, 17, pages, pools=1, shape=(1, 1, 8))
    c.plain.refs = [int(x) for x in (torch.rand(pages, generator=g) < 0.55)]
    held = list(c.plain.refs)
    c.push()
    order = torch.randperm(rows, generator=g)[:1500].tolist()
    lengths = torch.randint(0, 17 * 128 + 1, (1500,), generator=g).tolist()
    want = c.extend(order, lengths)
    assert want.count(0) > 1300 and (2 in want or sum((n + 127) // 128 for n in lengths) <= held.count(0))
    empty = [r for r in range(rows) if c.plain.used[r] == 0 and r not in order]
    full = [r for r in order if c.plain.used[r] > 0]
    c.fork([full[i % 40] for i in range(len(empty))], empty)
    c.free(list(range(rows)) * 2)
    assert c.plain.refs == held


@pytest.mark.parametrize("dtype,shape,count", [("bf16", (3, 128, 128), 2), ("e4m3", (1, 128, 128), 300), ("e4m3", (1, 1, 48), 1), ("bf16", (5, 128, 128), 1)])
def test_copies(msa, dtype, shape, count):
    """Pages of several sizes and more pools than one launch takes; pairs that clash are passed over."""
    pages = 9 if count < 100 else 5
    g = torch.Generator().manual_seed(5)
    pools = [torch.randn(pages, *shape, generator=g).to(DT[dtype]) for _ in range(count)]
    gpu = [p.to(DEV) for p in pools]
    src, dst = ([0, 1, 2, 8, 9, -1, 3], [4, 5, 5, 8, 6, 7, 0]) if count < 100 else ([0, 1, 1, 2], [4, 3, 3, 2])
    msa.msa_cache_copy_pages(gpu, i32(src), i32(dst))
    for p, got in zip(pools, gpu):
        if count < 100:  # 0 -> 4 reads a destination (0), 1 -> 5 comes again as 2 -> 5, 3 -> 0 stands
            bits(p)[5], bits(p)[0] = bits(p)[2].clone(), bits(p)[3].clone()
        else:
            bits(p)[4], bits(p)[3] = bits(p)[0].clone(), bits(p)[1].clone()
        assert torch.equal(bits(p), bits(got.cpu()))


def test_stacked_pools_and_streams(msa):
    """One tensor over all pools, with room between them, on another stream, captured and replayed."""
    g = torch.Generator().manual_seed(6)
    whole = torch.randn(4, 2, 10, 1, 128, 16, generator=g).to(torch.bfloat16)
    gpu = whole.to(DEV)[:, 1]
    t = Tables(3, 2, 10)
    t.extend([0], [130])
    tt, uu, rr = t.tensors(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st = msa.msa_cache_fork(gpu, tt, uu, rr, i32([0]), i32([1]), stream=side)
    side.synchronize()
    assert st.tolist() == t.fork([0], [1], [bits(p) for p in whole[:, 1]])
    t.check(tt, uu, rr)
    assert torch.equal(bits(gpu.cpu().contiguous()), bits(whole[:, 1].contiguous()))
    graph = torch.cuda.CUDAGraph()
    rows, lengths = i32([2]), i32([200])
    with torch.cuda.graph(graph):
        msa.msa_cache_free(tt, uu, rr, rows)
        status = msa.msa_cache_extend(tt, uu, rr, rows, lengths)
    for n in (200, 50):
        lengths.fill_(n)
        graph.replay()
        t.free([2])
        assert status.tolist() == t.extend([2], [n])
        t.check(tt, uu, rr)


@pytest.mark.parametrize("dtype,hkv,layers", [("bf16", 4, 3), ("fp16", 1, 1), ("e4m3", 3, 130)])
def test_accept(msa, dtype, hkv, layers):
    """Paths within a page and across pages, the whole draft, none of it, long ones, ones that stop ascending or leave the drafts,
    lengths out of range, requests without drafts or with fewer keys than drafts, pages missing."""
    lens = [8, 5, 100, 200, 3, 0, 4, 6, 9, 7]
    used = [300, 130, 230, 400, 3, 50, 260, 4, 133, 137]
    paths = [[0, 2, 5, 7], [1, 3, 4], list(range(0, 100, 1)), list(range(1, 200, 2)) + [199], [0, 1], [], [2, 1, 3], [3, 4, 5], [0, 4, 9], [1, 2, 5]]
    paths[2][50:] = range(50, 100)
    plen = [4, 3, 100, 1000, -2, 3, 3, 3, 3, 3]
    g = torch.Generator().manual_seed(7)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    width = max(map(len, paths))
    path = torch.tensor([p + [-1] * (width - len(p)) for p in paths], dtype=torch.int32)
    need = [(n + 127) // 128 for n in used]
    table = torch.full((len(lens), 4), -1, dtype=torch.int32)
    perm, off = torch.randperm(sum(need), generator=g).to(torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[off : off + n]
        off += n
    table[9, 1] = 10_000
    pools = torch.randn(2 * layers, sum(need), hkv, 128, 128 if layers < 100 else 16, generator=g).to(DT[dtype])
    gpu = pools.to(DEV)
    seq, ln = torch.tensor(used, dtype=torch.int32), torch.tensor(plen, dtype=torch.int32)
    out = msa.msa_cache_accept(gpu, table.to(DEV), seq.to(DEV), cu.to(DEV), path.to(DEV), ln.to(DEV))
    want = accept([bits(p) for p in pools], table, seq, cu, path, ln)
    assert out.tolist() == want
    assert torch.equal(bits(gpu.cpu()), bits(pools))
    listed = [p.to(DEV) for p in pools]
    again = msa.msa_cache_accept(listed, table.to(DEV), out, cu.to(DEV), path.to(DEV), torch.zeros_like(ln).to(DEV))
    assert again.tolist() == [max(0, n - m) for n, m in zip(want, lens)]


def test_offsets_past_32_bits(msa):
    """The last pages of pools over 4 GiB: a copy, an accepted row and an appended token land where they should."""
    pages, hkv = 33000, 4  # 4.3 GB a pool
    pools = torch.zeros(2, pages, hkv, 128, 128, dtype=torch.bfloat16, device=DEV)
    last = pages - 1
    pools[0, last] = 1
    pools[1, last] = 2
    msa.msa_cache_copy_pages(pools, i32([last]), i32([last - 1]))
    assert (pools[0, last - 1] == 1).all() and (pools[1, last - 1] == 2).all()
    pools[:, last, :, 5] = 3
    out = msa.msa_cache_accept(pools, i32([[last]]), i32([7]), i32([0, 3]), i32([[1]]), i32([1]))
    assert out.tolist() == [5] and (pools[:, last, :, 4] == 3).all()
    x = torch.ones(1, 6, 128, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(128, device=DEV)
    msa.msa_qk_norm_rope_append(x, x[:, :4], x[:, :4] * 9, w, w, None, i32([0]), i32([0, 1]), pools[0], pools[1], page_table=i32([[last]]), seqused_k=i32([128]))
    assert (pools[0, last, :, 127] == 1).all() and (pools[1, last, :, 127] == 9).all()
    assert int((pools[0].view(torch.int16) != 0).sum()) == 2 * hkv * 128 * 128
