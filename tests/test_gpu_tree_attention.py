"""Attention of drafted trees over a paged cache against 64 bits.

Tolerances, from the arithmetic, with A = sum of p |v| over the keys: a probability is off by its rounding to V's type (half a
step; in fp16 also 2^-25 absolute, with the largest at least 1 before the division) and by its logit's error. A logit is a float32
sum of 128 products, off by at most 128 roundings of 2^-24 of sum |q k| scale; for the unit normal values here that sum is below
16, so 2^-13 covers the numerator and the denominator together. The output is rounded once more. The normaliser's logarithm is off
by the logits' error and float32 roundings of its own size."""
import pytest
import torch

import workloads
from parity_util import fault_clear
from step_util import DT, half_step, pad_words, tree_attention, tree_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 128**-0.5


@pytest.fixture(scope="module")
def msa():
    import block_sparse_top_msa_gb300 as m
    m.build()
    m.lib()
    return m


def make(lens, used, hq, hkv, topk, kv, seed=0, words=None, garbage=True):
    """Ragged trees of drafts: parents at random, lists of random blocks with the drafts' own, NaN and infinities past each end."""
    g = torch.Generator().manual_seed(seed)
    qt = torch.float16 if kv == "fp16" else torch.bfloat16
    cu = workloads.cu_from_lengths(lens)
    pages = [(n + 127) // 128 for n in used]
    num = sum(pages) + 3
    perm, off = torch.randperm(num, generator=g).to(torch.int32), 0
    table = torch.full((len(used), max(1, max(pages))), -1, dtype=torch.int32)
    for b, n in enumerate(pages):
        table[b, :n] = perm[off : off + n]
        off += n
    k, v = (torch.randn(num, hkv, 128, 128, generator=g) for _ in range(2))
    if garbage:
        live = torch.zeros(num, 128, dtype=torch.bool)
        for b, n in enumerate(used):
            for p in range(n):
                live[table[b, p // 128], p % 128] = True
        junk = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38])[torch.randint(0, 4, (num, hkv, 128, 128), generator=g)]
        if kv == "e4m3":
            junk = torch.full_like(junk, float("nan"))
        k, v = (torch.where(live[:, None, :, None], x, junk) for x in (k, v))
    k, v = k.to(DT[kv]), v.to(DT[kv])
    words = words or max(1, (max(lens) + 31) // 32)
    mask = [pad_words(tree_bits([int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(n)]), words) for n in lens if n]
    q2k = torch.full((hkv, sum(lens), topk), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range(n):
            for h in range(hkv):
                own = sorted({max(0, used[b] - n) // 128, max(0, used[b] - 1) // 128})
                rest = [x for x in torch.randperm(max(1, pages[b]), generator=g).tolist() if x not in own]
                ids = sorted((own + rest)[:topk])
                q2k[h, cu[b] + i, : len(ids)] = torch.tensor(ids, dtype=torch.int32)
    return dict(q=torch.randn(sum(lens), hq, 128, generator=g).to(qt), k=k, v=v, q2k=q2k, cu=cu, mask=torch.cat(mask) if mask else torch.zeros(0, words, dtype=torch.int32),
                table=table, used=torch.tensor(used, dtype=torch.int32))


def run(msa, c, max_q=None, **kw):
    d = {n: t.to(DEV) for n, t in c.items()}
    got = msa.msa_tree_attention(d["q"], d["k"], d["v"], d["q2k"], d["cu"], d["mask"], page_table=d["table"], seqused_k=d["used"],
                                 max_seqlen_q=max_q or max(1, int((c["cu"][1:] - c["cu"][:-1]).max())), return_softmax_lse=True, **kw)
    torch.cuda.synchronize()
    fault_clear(msa)
    return got


def check(c, out, lse):
    ref, rl, size = tree_attention(c["q"], c["k"].float(), c["v"].float(), c["q2k"], c["cu"], c["mask"], c["table"], c["used"], SCALE)
    n = int(c["cu"][-1])
    out, lse, ref, rl, size = out.double().cpu()[:n], lse.double().cpu()[:n], ref[:n], rl[:n], size[:n]
    step = half_step(c["q"].dtype)
    tol = step * (size + ref.abs()) * 1.01 + 2.0**-13 * size
    if c["q"].dtype == torch.float16:
        tol += c["q2k"].shape[2] * 128 * 2.0**-25 * 6 + 2.0**-25
    empty = rl == -float("inf")
    assert torch.equal(lse == -float("inf"), empty)
    assert (out[empty] == 0).all()
    bad = (out - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), ((out - ref).abs() / tol.clamp(min=1e-30)).max().item())
    assert ((lse - rl).abs()[~empty] <= 2.0**-13 + rl.abs()[~empty] * 2.0**-21).all()


CASES = [
    # one token each: the one-token form, its longest lists and the sorted ones; a sequence of one key
    ([1, 1, 1], [1, 700, 129], 16, 1, 4, "bf16"),
    ([1] * 3, [5000, 1, 128], 8, 8, 33, "fp16"),
    # drafts inside one block, across a page's end, from position 0 on, and with fewer keys than tokens
    ([5, 8, 7, 6], [133, 132, 7, 4], 8, 2, 3, "bf16"),
    ([9, 17], [1000, 140], 32, 2, 5, "fp16"),
    ([33, 2, 64], [290, 400, 64], 16, 2, 6, "bf16"),
    # more drafts than a block holds, three words a row, several tiles a request
    ([150, 70], [600, 1100], 12, 3, 7, "bf16"),
    # G = 1 (128 tokens a tile), G = 128 (one), G = 40
    ([20, 31], [400, 900], 3, 3, 6, "bf16"),
    ([4, 2], [300, 257], 128, 1, 3, "bf16"),
    ([3, 6], [500, 380], 40, 1, 4, "fp16"),
    # an E4M3 cache, converted in the kernel, and (the short one) decoded to bf16 first
    ([5, 1, 12], [1200, 300, 140], 16, 2, 4, "e4m3"),
    ([70, 64], [128, 100], 16, 2, 1, "e4m3"),
    ([130], [640], 8, 1, 4, "e4m3"),
]


@pytest.mark.parametrize("lens,used,hq,hkv,topk,kv", CASES)
def test_trees(msa, lens, used, hq, hkv, topk, kv):
    c = make(lens, used, hq, hkv, topk, kv, seed=len(lens) + hq)
    check(c, *run(msa, c))


def test_lists_and_masks_of_any_kind(msa):
    """Lists unsorted, repeated, with -1 inside and ids past the end, pages missing, rows that see nothing by list or by mask, a mask
    without a token's own bit or with bits past the drafts, more words than needed, a request without tokens."""
    c = make([6, 0, 4], [700, 50, 260], 8, 2, 5, "bf16", words=3)
    c["q2k"][0, 0] = torch.tensor([5, 2, 5, -1, 0])
    c["q2k"][1, 1] = torch.tensor([-7, 9, 5, 100000, 1])
    c["q2k"][0, 2] = -1
    c["mask"][3] = 0
    c["q2k"][:, 3] = torch.tensor([5, -1, -1, -1, -1])  # block 5 holds keys 640..699: the six drafts and 54 before
    c["q2k"][:, 7] = torch.tensor([2, -1, -1, -1, -1])  # keys 256..259, all drafts
    c["mask"][7] = torch.tensor([0, -1, -1])
    c["mask"][8] = torch.tensor([-1, -1, -1])
    c["table"][0, 1] = -1
    c["table"][2, 0] = c["k"].shape[0]
    check(c, *run(msa, c))
    assert (run(msa, c)[1][7] == -float("inf")).all()


def test_a_chain_is_the_causal_forward(msa):
    """Lower-triangular bits: the forward's own causal results (the same products and sums: the same bits)."""
    lens, used = [9, 4, 16], [500, 132, 1025]
    c = make(lens, used, 32, 4, 5, "bf16", garbage=False)
    c["mask"] = torch.cat([tree_bits([i - 1 for i in range(n)]) for n in lens])
    out, lse = run(msa, c)
    d = {n: t.to(DEV) for n, t in c.items()}
    want, wl = msa.msa_sparse_attention_fwd(d["q"], d["k"], d["v"], d["q2k"], d["cu"], causal=True, page_table=d["table"], seqused_k=d["used"], max_seqlen_q=16,
                                            return_softmax_lse=True)
    torch.testing.assert_close(out.float(), want.float(), rtol=2.0**-7, atol=2.0**-9)
    torch.testing.assert_close(lse, wl, rtol=0, atol=2.0**-13)


def test_rows_behind_the_last_sequence(msa):
    """A padded batch: the rows past cu_seqlens_q[-1] keep what they held."""
    c = make([5, 3], [200, 140], 8, 2, 2, "bf16")
    for n, dim in (("q", 0), ("mask", 0), ("q2k", 1)):
        c[n] = torch.cat([c[n], c[n].narrow(dim, 0, 4)], dim)
    out = torch.full((12, 8, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((12, 8), 5.0, device=DEV)
    run(msa, c, max_q=8, out=out, lse=lse)
    check(c, out, lse)
    assert (out[8:] == 5).all() and (lse[8:] == 5).all()


def test_many_units_and_bounds(msa):
    """Whole and split units together, and a bound on the tokens well above them."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(1, 6, (40,), generator=g).tolist()
    used = [n + int(torch.randint(0, 300, (1,), generator=g)) for n in lens]
    c = make(lens, used, 16, 4, 3, "bf16", words=2)
    check(c, *run(msa, c))
    check(c, *run(msa, c, max_q=64))


def test_runner_captured(msa):
    """The prepared form, replayed on new contents; two graphs, each with its workspace."""
    c = make([7, 4], [300, 420], 16, 2, 3, "bf16")
    d = {n: t.to(DEV) for n, t in c.items()}
    runners = [msa.TreeAttentionRunner(d["q"], d["k"], d["v"], d["q2k"], d["cu"], d["mask"], page_table=d["table"], seqused_k=d["used"], max_seqlen_q=7,
                                       return_softmax_lse=True) for _ in range(2)]
    graphs = []
    for r in runners:
        r.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            r.run()
    c["q"] = c["q"].flip(0)
    d["q"].copy_(c["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs[0].replay()
    with torch.cuda.stream(side):
        graphs[1].replay()
    torch.cuda.synchronize()
    fault_clear(msa)
    for r in runners:
        check(c, r.out, r.lse)


def test_no_tokens(msa):
    c = make([0, 0], [300, 20], 16, 2, 3, "bf16")
    out, lse = run(msa, c, max_q=1)
    assert out.shape == (0, 16, 128) and lse.shape == (0, 16)


def test_other_routes_leave_it_alone(msa):
    c = make([9, 4], [300, 420], 16, 2, 3, "bf16")
    try:
        msa.msa_set_prefill_route(2)
        check(c, *run(msa, c))
    finally:
        msa.msa_set_prefill_route(0)


ODD = [
    ([9, 17], [1000, 140], 32, 2, 5, "fp16"),
    ([33, 2, 64], [290, 400, 64], 16, 2, 6, "bf16"),
    ([5, 1, 12], [1200, 300, 140], 16, 2, 4, "e4m3"),
    ([70, 64], [190, 640], 16, 2, 2, "e4m3"),
    ([1, 1], [3000, 129], 8, 8, 20, "bf16"),
    # blocks of one unit over several ranges
    ([20], [5000], 32, 2, 36, "bf16"),
    ([20], [5000], 32, 2, 36, "e4m3"),
]


@pytest.mark.parametrize("where", ["k", "v", "block"])
@pytest.mark.parametrize("lens,used,hq,hkv,topk,kv", ODD)
def test_what_a_row_does_not_see_may_be_anything(msa, lens, used, hq, hkv, topk, kv, where):
    """Keys and values that are not finite, in a draft's row or in a block that one token lists: whoever does not see them is as
    near its 64-bit result as ever, whoever does gets the formula's NaN or infinity."""
    c = make(lens, used, hq, hkv, topk, kv, seed=5, garbage=False)
    nan, inf = float("nan"), float("nan") if kv == "e4m3" else float("inf")
    kf, vf = c["k"].float(), c["v"].float()
    for b, n in enumerate(lens):
        lo, first = int(c["cu"][b]), used[b] - n
        if where == "block":
            blk = 0
            c["q2k"][:, lo + 1 : lo + n] = torch.where(c["q2k"][:, lo + 1 : lo + n] == blk, -1, c["q2k"][:, lo + 1 : lo + n])
            page = int(c["table"][b, blk])
            kf[page, :, 3] = nan
            vf[page, :, 5, 7] = inf
        else:
            p = first + n // 2
            page, row = int(c["table"][b, p // 128]), p % 128
            if where == "k":
                kf[page, :, row] = nan
                vf[page, :, row] = -inf
            else:
                vf[page, :, row, 9] = inf
                vf[page, :, row, 64:] = nan
    c["k"], c["v"] = kf.to(DT[kv]), vf.to(DT[kv])
    out, lse = (x.double().cpu() for x in run(msa, c))
    ref, rl, size = tree_attention(c["q"], c["k"].float(), c["v"].float(), c["q2k"], c["cu"], c["mask"], c["table"], c["used"], SCALE)
    finite = ref.isfinite()
    assert not finite.all() and (finite.any() or max(lens) == 1)
    assert torch.equal(out.isnan(), ref.isnan()) and torch.equal(out.isinf(), ref.isinf()) and torch.equal(lse.isnan(), rl.isnan())
    assert torch.equal(out[ref.isinf()], ref[ref.isinf()])
    tol = half_step(c["q"].dtype) * (size + ref.abs()) * 1.01 + 2.0**-13 * size
    if kv == "fp16":
        tol += topk * 128 * 2.0**-25 * 6 + 2.0**-25
    assert ((out - ref).abs() <= tol)[finite].all()
    ok = rl.isfinite()
    assert ((lse - rl).abs()[ok] <= 2.0**-13 + rl.abs()[ok] * 2.0**-21).all()


GROWN = [
    ([9, 17], [1000, 640], 32, 2, 7, "fp16"),
    ([33, 64], [1290, 900], 16, 2, 9, "bf16"),
    ([5, 1, 12], [1200, 900, 640], 16, 2, 8, "e4m3"),
    ([20], [5000], 32, 2, 36, "bf16"),
    ([70], [3000], 16, 2, 20, "e4m3"),
    # lists of the greatest length, 128 tokens a tile and one
    ([30], [9000], 2, 2, 64, "bf16"),
    ([3], [9000], 128, 1, 64, "fp16"),
]


@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("lens,used,hq,hkv,topk,kv", GROWN)
def test_logits_that_grow_and_fall(msa, lens, used, hq, hkv, topk, kv, down):
    """Keys that grow with their place, so that the running maximum moves from half a block to the next (or never after the
    first), with a row of Q of zeros and one below every normal f16. The logits' error grows with L = max sum |q k| scale: 128 roundings of 2^-24
    of the sum, and three of the exponent's argument, below 2 L log2(e): a probability is off by 2 (2^-17 + 9 2^-24) L < 2^-15.8 L
    over numerator and denominator."""
    c = make(lens, used, hq, hkv, topk, kv, seed=9, garbage=False)
    kf = c["k"].float()
    for b, n in enumerate(used):
        for i in range((n + 127) // 128):
            at = (torch.arange(128) + 128 * i) / n
            kf[c["table"][b, i]] *= (6 * (1 - at if down else at)).clamp(min=0)[None, :, None]
    c["k"] = kf.to(DT[kv])
    c["q"][0] = 0
    c["q"][1] *= 2.0**-24 if kv == "fp16" else 2.0**-60
    out, lse = (x.double().cpu() for x in run(msa, c))
    ref, rl, size = tree_attention(c["q"], c["k"].float(), c["v"].float(), c["q2k"], c["cu"], c["mask"], c["table"], c["used"], SCALE)
    big = max((c["q"].float().abs().reshape(-1, hkv, hq // hkv, 128).amax(2)[:, h] @ c["k"].float()[:, h].abs().reshape(-1, 128).T).max().item() for h in range(hkv)) * SCALE
    off = 2.0**-15.8 * big
    tol = half_step(c["q"].dtype) * (size + ref.abs()) * 1.01 + off * size
    if kv == "fp16":
        tol += topk * 128 * 2.0**-25 * 6 + 2.0**-25
    bad = (out - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), ((out - ref).abs() / tol.clamp(min=1e-30)).max().item())
    assert ((lse - rl).abs() <= off + rl.abs() * 2.0**-21 + 2.0**-20).all()


@pytest.mark.parametrize("kv,hq,hkv", [("fp16", 40, 4), ("bf16", 64, 4), ("e4m3", 32, 2)])
def test_slow_caches_change_nothing(msa, kv, hq, hkv):
    """Long lists read from memory and not from L2, so that blocks arrive later than their place in the pipeline: the bits of a
    call whose caches are warm, in units of one tile and of two."""
    lens = [4 + (7 * i) % 13 for i in range(24)]
    used = [2200 + 61 * i for i in range(24)]
    c = make(lens, used, hq, hkv, 16, kv, seed=3)
    warm = run(msa, c)
    check(c, *warm)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    d = {n: t.to(DEV) for n, t in c.items()}
    for i in range(6):
        flush.fill_(i)
        out, lse = msa.msa_tree_attention(d["q"], d["k"], d["v"], d["q2k"], d["cu"], d["mask"], page_table=d["table"], seqused_k=d["used"],
                                          max_seqlen_q=max(lens), return_softmax_lse=True)
        assert torch.equal(out, warm[0]) and torch.equal(lse, warm[1])
    fault_clear(msa)


def test_hundreds_of_requests(msa):
    """More sequences than a block of the union kernel reads at once, some of them empty."""
    lens = [(5 * i) % 3 for i in range(600)]
    used = [n + (37 * i) % 200 for i, n in enumerate(lens)]
    c = make(lens, used, 4, 2, 2, "bf16", seed=6)
    check(c, *run(msa, c))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_past_32_bits(msa, kv):
    """Pages whose elements lie past 2^32, written by the append and read by the attention."""
    g = torch.Generator().manual_seed(8)
    hkv, hq, num, lens, used = 4, 16, 70000, [6, 9], [300, 140]
    assert (num - 10) * hkv * 128 * 128 > 2**32
    k, v = (torch.empty(num, hkv, 128, 128, dtype=DT[kv], device=DEV) for _ in range(2))
    table = torch.tensor([[num - 1, num - 5, num - 2], [num - 7, num - 3, -1]], dtype=torch.int32)
    small = torch.tensor([[0, 1, 2], [3, 4, -1]], dtype=torch.int32)
    pages = table[small >= 0].long().to(DEV)
    fill = torch.randn(2, 5, hkv, 128, 128, generator=g).to(DT[kv])
    k[pages], v[pages] = fill[0].to(DEV), fill[1].to(DEV)
    c = make(lens, used, hq, hkv, 3, kv, seed=8, garbage=False)
    x = torch.randn(sum(lens), hq + 2 * hkv, 128, generator=g).to(torch.bfloat16).to(DEV)
    w = torch.ones(128, device=DEV)
    pos = torch.zeros(sum(lens), dtype=torch.int32, device=DEV)
    c["table"] = table
    q = msa.msa_qk_norm_rope_append(x[:, :hq], x[:, hq : hq + hkv], x[:, hq + hkv :], w, w, None, pos, c["cu"].to(DEV), k, v, page_table=table.to(DEV),
                                    seqused_k=c["used"].to(DEV))
    d = {n: t.to(DEV) for n, t in c.items()}
    out, lse = msa.msa_tree_attention(q, k, v, d["q2k"], d["cu"], d["mask"], page_table=d["table"], seqused_k=d["used"], max_seqlen_q=9, return_softmax_lse=True)
    fault_clear(msa)
    kept, near = (t[pages].cpu() for t in (k, v)), x[:, hq + hkv :].float().cpu()
    c["k"], c["v"] = kept
    for b in range(2):
        for t in range(int(c["cu"][b]), int(c["cu"][b + 1])):
            p = used[b] - int(c["cu"][b + 1]) + t
            assert torch.equal(c["v"][small[b, p // 128], :, p % 128].float(), near[t].to(DT[kv]).float())
    c["q"], c["table"] = q.cpu(), small
    check(c, out, lse)
