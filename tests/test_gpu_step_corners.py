"""Calls of the serving step's operators at the edges of what their documentation allows."""
import ctypes as C
import threading

import pytest
import torch

import test_gpu_cache_pages as pages
import test_gpu_qk_norm_rope as rope
import test_gpu_tree_attention as tree
from parity_util import fault_clear
from step_util import DT, half_step, norm_rope_bwd, tree_attention

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


@pytest.mark.parametrize("captured", [False, True])
def test_a_step_behind_a_forward_whose_splits_come_to_nothing(msa, captured):
    """A forward with room to split its units but short lists, and right behind it an append and accepted rows that overwrite what it
    reads: every time the forward's results of the caches before."""
    batch, lq, hq, hkv, topk = 4, 3, 64, 4, 16
    g = torch.Generator().manual_seed(4)
    used = [700 + 128 * b for b in range(batch)]
    width = (max(used) + 127) // 128
    pages = batch * width
    table = torch.randperm(pages, generator=g).to(torch.int32).view(batch, width).to(DEV)
    lists = torch.full((hkv, batch * lq, topk), -1, dtype=torch.int32)
    lists[:, :, 0] = 1  # one listed block of sixteen
    lists, cu = lists.to(DEV), torch.arange(0, batch * lq + 1, lq, dtype=torch.int32, device=DEV)
    seq = torch.tensor(used, dtype=torch.int32, device=DEV)
    pools = torch.randn(2, pages, hkv, 128, 128, generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn(batch * lq, hq, 128, generator=g).to(torch.bfloat16).to(DEV)
    x = torch.randn(batch * lq, hq + 2 * hkv, 128, generator=g).to(torch.bfloat16).to(DEV)
    w, pos = torch.ones(128, device=DEV), torch.zeros(batch * lq, dtype=torch.int32, device=DEV)
    # The tokens' cache rows are the listed block's, so that the append overwrites keys that the forward reads.
    at = torch.full((batch,), 256, dtype=torch.int32, device=DEV)
    path, plen = torch.tensor([[1, 2]] * batch, dtype=torch.int32, device=DEV), torch.full((batch,), 2, dtype=torch.int32, device=DEV)
    work = torch.empty(msa.msa_sparse_attention_workspace_size(batch, batch * lq, hq, hkv, 128, topk, lq, True) + 256, dtype=torch.uint8, device=DEV)
    out, kept = torch.empty_like(q), (pools.clone(), q.clone())

    def step():
        msa.msa_sparse_attention_fwd(q, pools[0], pools[1], lists, cu, causal=True, page_table=table, seqused_k=seq, max_seqlen_q=lq, out=out, workspace=work)
        msa.msa_qk_norm_rope_append(x[:, :hq], x[:, hq : hq + hkv], x[:, hq + hkv :], w, w, None, pos, cu, pools[0], pools[1], page_table=table, seqused_k=at, q_out=q)
        return msa.msa_cache_accept(pools, table, at, cu, path, plen)

    step()
    torch.cuda.synchronize()
    pools.copy_(kept[0])
    q.copy_(kept[1])
    msa.msa_sparse_attention_fwd(q, pools[0], pools[1], lists, cu, causal=True, page_table=table, seqused_k=seq, max_seqlen_q=lq, out=out, workspace=work)
    want = out.clone()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for _ in range(50):
        pools.copy_(kept[0])
        q.copy_(kept[1])
        out.fill_(7)
        graph.replay() if captured else step()
        assert torch.equal(out, want)
    fault_clear(msa)


@pytest.mark.parametrize("kv,hq,hkv,lo,hi", [("fp16", 40, 4, 4, 7), ("bf16", 64, 4, 1, 16), ("e4m3", 64, 4, 1, 16), ("e4m3", 32, 4, 1, 16)])
def test_tree_gives_the_same_bits(msa, kv, hq, hkv, lo, hi):
    """Units of one tile and of two in one call, keys that grow so that rows are rescaled from half a block to the next: near 64 bits,
    and the same bits in every run, alone and with runs right behind one another."""
    lens = [lo + (5 * i) % (hi - lo + 1) for i in range(20)]
    used = [900 + 77 * i for i in range(20)]
    c = tree.make(lens, used, hq, hkv, 8, kv, seed=12, garbage=False)
    kf = c["k"].float()
    for b, n in enumerate(used):
        for i in range((n + 127) // 128):
            kf[c["table"][b, i]] *= 1 + 2 * ((torch.arange(128) + 128 * i) / n).clamp(max=1)[None, :, None]
    c["k"] = kf.to(DT[kv])
    d = {n: t.to(DEV) for n, t in c.items()}

    def run():
        return msa.msa_tree_attention(d["q"], d["k"], d["v"], d["q2k"], d["cu"], d["mask"], page_table=d["table"], seqused_k=d["used"], max_seqlen_q=max(lens),
                                      return_softmax_lse=True)

    first = run()
    ref, rl, size = tree_attention(c["q"], c["k"].float(), c["v"].float(), c["q2k"], c["cu"], c["mask"], c["table"], c["used"], tree.SCALE)
    # A logit is off by at most 128 roundings of 2^-24 of L = max sum |q k| scale, a probability by twice that and by the
    # exponent's argument's three roundings: 2 (2^-17 + 9 2^-24) L < 2^-15.8 L.
    most = max((c["q"].float().abs().reshape(-1, hkv, hq // hkv, 128).amax(2)[:, h] @ c["k"].float()[:, h].abs().reshape(-1, 128).T).max().item() for h in range(hkv)) * tree.SCALE
    tol = half_step(c["q"].dtype) * (size + ref.abs()) * 1.01 + 2.0**-15.8 * most * size
    if kv == "fp16":
        tol += 8 * 128 * 2.0**-25 * 6 + 2.0**-25
    assert ((first[0].double().cpu() - ref).abs() <= tol).all()
    for _ in range(20):
        runs = [run() for _ in range(10)]
        assert all(torch.equal(o, first[0]) and torch.equal(l, first[1]) for o, l in runs)
    fault_clear(msa)


@pytest.mark.parametrize("hq,hkv", [(1, 2048), (2048, 1), (4, 1300)])
def test_gradient_of_unlike_head_counts(msa, hq, hkv):
    """Both sides' gradients, where nearly all rows are of one side."""
    tokens = 13
    _, q, k, _, w, table, pos = rope.inputs(tokens, hq, hkv, 64, "bf16", seed=3, packed=False)
    g = torch.Generator().manual_seed(8)
    dq, dk = (torch.randn(t.shape, generator=g).to(t.dtype) for t in (q, k))
    got = msa.msa_qk_norm_rope_bwd(*(t.to(DEV) for t in (dq, dk, q, k, w[0], w[1], table, pos)))
    for i, (x, d) in enumerate(((q, dq), (k, dk))):
        dx, mag, dw, terms = norm_rope_bwd(x, w[i], d, table, pos, False)
        rope.near(got[i], dx, mag, x.dtype, rope.CHAIN_BWD)
        assert ((got[2 + i].double().cpu() - dw).abs() <= rope.SUMS * terms).all()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_extend_to_the_longest_row(msa):
    """A row that ends within the last 128 tokens of what an int counts gets its last pages."""
    table = torch.full((1, 1 << 24), -1, dtype=torch.int32, device=DEV)
    used, refs = i32([2**31 - 300]), torch.zeros(5, dtype=torch.int32, device=DEV)
    first = (2**31 - 300) // 128
    table[0, first] = 4
    refs[4] = 1
    assert msa.msa_cache_extend(table, used, refs, i32([0]), i32([2**31 - 1])).tolist() == [0]
    assert used.tolist() == [2**31 - 1] and refs.tolist() == [1, 1, 0, 0, 1]
    assert table[0, first - 2 :].tolist() == [-1, -1, 4, 0, 1]


def test_rows_that_lack_more_pages_than_an_int_counts(msa):
    """2^24 pages wanted by each of 130 rows: the sum is past 2^31. None is granted, those that need none are done."""
    rows = 132
    table = torch.full((rows, 1 << 24), -1, dtype=torch.int32, device=DEV)
    used, refs = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.zeros(100, dtype=torch.int32, device=DEV)
    lengths = [0] + [2**31 - 1] * 130 + [1]
    status = msa.msa_cache_extend(table, used, refs, i32(range(rows)), i32(lengths))
    assert status.tolist() == [0] + [2] * 131
    assert (used == 0).all() and (refs == 0).all() and int(table.max()) == -1
    assert msa.msa_cache_extend(table, used, refs, i32([131, 130]), i32([1, 129])).tolist() == [0, 0]
    assert refs[:4].tolist() == [1, 1, 1, 0] and table[131, :2].tolist() == [0, -1] and table[130, :3].tolist() == [1, 2, -1]


def test_fork_of_whole_pages_with_the_first_page_free(msa):
    """A source that ends with its page has no begun one: the free page 0 goes to the first fork that needs one, and holds the copy of
    its source's begun page."""
    c = pages.Both(msa, 7, 4, 12)
    c.extend([0, 1, 2, 3], [1, 256, 300, 128])
    c.free([0])
    assert c.plain.refs[0] == 0
    assert c.fork([1, 2, 3, 2], [4, 5, 0, 6]) == [0, 0, 0, 0]
    assert c.plain.table[5][2] == 0 and torch.equal(c.gpu_pools[0][0], c.gpu_pools[0][c.plain.table[2][2]])


def test_calls_of_several_threads_at_once(msa):
    """Calls that need different amounts of shared memory, each thread on its stream with its own tables: none fails to launch."""
    L = msa.lib()
    sizes = [range(8000 + i, 16384, 7) for i in range(4)]
    state, bad = [], []
    for i in range(4):
        most = 16384
        state.append((torch.full((most, 1), -1, dtype=torch.int32, device=DEV), torch.zeros(most, dtype=torch.int32, device=DEV),
                      torch.zeros(64, dtype=torch.int32, device=DEV), i32([3]), i32([100]), i32([9]),
                      torch.empty(4096, dtype=torch.uint8, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def calls(i):
        table, used, refs, rows, lengths, status, ws, stream = state[i]
        p = [C.c_void_p(t.data_ptr()) for t in (table, used, refs, rows, lengths, status, ws)]
        for n in sizes[i]:
            st = L.msa_cache_extend(p[0], 1, n, p[1], p[2], 64, p[3], p[4], 1, p[5], p[6], 4096, C.c_void_p(stream.cuda_stream))
            if st != 0:
                bad.append((i, n, st))

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad
    for table, used, refs, _, _, status, _, _ in state:
        assert status.tolist() == [0] and used[3].item() == 100 and table[3].tolist() == [0] and int(refs.sum()) == 1
