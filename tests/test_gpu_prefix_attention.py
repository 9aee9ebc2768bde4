"""Attention over shared prefixes against 64 bits.

Tolerances, from the arithmetic, with A = sum of p |v| over the keys: a probability is off by its rounding to the products' type
(half a step of bf16; of fp16, as which E4M3 is multiplied too, also 2^-25 absolute, with the largest of a part at least 1 and a
part's weight at most 1) and by its logit's error. A logit is a float32 sum of 128 products, off by at most 128 roundings of 2^-24
of sum |q k| scale; for the unit normal values here that sum is below 16, so 2^-13 covers the numerator and the denominator
together. The output is rounded once more. The normaliser's logarithm is off by the logits' error and float32 roundings of its own
size; joining parts adds a few roundings of 2^-22, which 2^-13 covers too."""
import pytest
import torch

import samples_util as S
import workloads
from parity_util import fault_clear
from step_util import DT, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 128**-0.5


@pytest.fixture(scope="module")
def msa():
    import block_sparse_top_msa_gb300 as m
    m.build()
    m.lib()
    return m


def make(prompts, samples, hq, hkv, kv, seed=0, garbage=True, extra=0):
    """Groups of samples [(own tokens, new tokens), ...] of prompts, the requests in an order of their own; NaN and infinities in
    every row of the pool that no request holds. `extra` rows of q follow the last request's."""
    g = torch.Generator().manual_seed(seed)
    qt = torch.float16 if kv == "fp16" else torch.bfloat16
    flat = [(p, n, new) for p, group in zip(prompts, samples) for n, new in group]
    b = len(flat)
    at = torch.randperm(b, generator=g).tolist()  # the request that sample i is
    used, lens = [0] * b, [0] * b
    for i, (p, n, new) in enumerate(flat):
        used[at[i]], lens[at[i]] = p + n + new, new
    cu = workloads.cu_from_lengths(lens)
    width = max(1, max((n + 127) // 128 for n in used))
    num = sum(p // 128 for p in prompts) + sum((p + n + new + 127) // 128 - p // 128 for p, n, new in flat) + 3
    perm, off = torch.randperm(num, generator=g).to(torch.int32), 0
    table = torch.full((b, width), -1, dtype=torch.int32)
    rows, ends, blocks, i = [], [0], [], 0
    for p, group in zip(prompts, samples):
        shared = perm[off : off + p // 128]
        off += p // 128
        members = []
        for n, new in group:
            r, pages = at[i], (p + n + new + 127) // 128
            own = pages - p // 128
            table[r, : p // 128] = shared
            table[r, p // 128 : pages] = perm[off : off + own]
            off += own
            members.append(r)
            i += 1
        rows += sorted(members)
        ends.append(len(rows))
        blocks.append(p // 128)
    pad = b - len(prompts)
    k, v = (torch.randn(num, hkv, 128, 128, generator=g) for _ in range(2))
    if garbage:
        live = torch.zeros(num, 128, dtype=torch.bool)
        for r in range(b):
            pos = torch.arange(used[r])
            live[table[r].long()[pos // 128], pos % 128] = True
        junk = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38])[torch.randint(0, 4, (num, hkv, 128, 128), generator=g)]
        if kv == "e4m3":
            junk = torch.full_like(junk, float("nan"))
        k, v = (torch.where(live[:, None, :, None], x, junk) for x in (k, v))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return dict(q=torch.randn(sum(lens) + extra, hq, 128, generator=g).to(qt), k=k.to(DT[kv]), v=v.to(DT[kv]), cu=cu, table=table, used=i32(used), rows=i32(rows),
                ends=i32(ends + [b] * pad), blocks=i32(blocks + [0] * pad))


def run(msa, c, groups=True, **kw):
    d = {n: t.to(DEV) for n, t in c.items()}
    if groups:
        kw = dict(kw, group_rows=d["rows"], cu_groups=d["ends"], group_blocks=d["blocks"])
    got = msa.msa_prefix_attention(d["q"], d["k"], d["v"], d["cu"], page_table=d["table"], seqused_k=d["used"], return_softmax_lse=True, **kw)
    torch.cuda.synchronize()
    fault_clear(msa)
    return got


def check(c, out, lse, causal=True, scale=SCALE):
    ref, rl, size = S.prefix_attention(c["q"], c["k"].float(), c["v"].float(), c["cu"], c["table"], c["used"], scale, causal)
    n = int(c["cu"][-1])
    out, lse, ref, rl, size = out.double().cpu()[:n], lse.double().cpu()[:n], ref[:n], rl[:n], size[:n]
    step = half_step(c["q"].dtype)
    tol = step * (size + ref.abs()) * 1.01 + 2.0**-13 * size
    if c["q"].dtype == torch.float16 or c["k"].dtype == torch.float8_e4m3fn:
        tol += int(c["used"].max()) * 2.0**-25 * 6 + 2.0**-25
    empty = rl == -float("inf")
    assert torch.equal(lse == -float("inf"), empty)
    assert (out[empty] == 0).all()
    bad = ~((out - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), ((out - ref).abs() / tol.clamp(min=1e-30)).max().item())
    assert ((lse - rl).abs()[~empty] <= 2.0**-13 + rl.abs()[~empty] * 2.0**-21).all()


CASES = [
    # one key; one request by itself; a pair that shares two blocks
    ([0], [[(0, 1)]], 16, 1, "bf16"),
    ([700], [[(30, 1)]], 8, 2, "fp16"),
    ([300], [[(0, 1), (77, 1)]], 16, 1, "bf16"),
    # several prompts, one without a whole block, a request alone, one that ends with its prompt, drafts
    ([300, 100, 513, 40], [[(0, 1), (130, 3), (5, 2)], [(20, 1), (9, 1)], [(300, 4)], [(0, 1), (1, 1)]], 8, 2, "fp16"),
    ([256, 640], [[(0, 5), (127, 5), (128, 7)], [(129, 1), (0, 9), (250, 2)]], 12, 3, "bf16"),
    # heads without sharing, 96 and 128 to one, 40
    ([400], [[(3, 2), (60, 1), (200, 17)]], 3, 3, "bf16"),
    ([260], [[(10, 2), (100, 3)]], 128, 1, "bf16"),
    ([260, 128], [[(10, 1), (100, 3)], [(0, 1), (0, 2)]], 96, 1, "fp16"),
    ([390], [[(50, 3), (1, 1), (300, 2)]], 40, 1, "bf16"),
    # rows of several tiles of 16, 128 and 256, own runs of more than one block
    ([520], [[(i * 13, 3) for i in range(20)]], 16, 2, "bf16"),
    ([256], [[(i, 1 + i % 4) for i in range(24)], ], 32, 2, "fp16"),
    ([130], [[(5, 150), (0, 70)]], 4, 2, "bf16"),
    ([384], [[(0, 260), (100, 33)]], 16, 4, "fp16"),
    # an E4M3 cache
    ([300, 0], [[(0, 1), (130, 3), (5, 2)], [(400, 1)]], 16, 2, "e4m3"),
    ([520], [[(i * 13, 3) for i in range(14)]], 16, 2, "e4m3"),
    ([256], [[(3, 140), (0, 1)]], 8, 1, "e4m3"),
]


@pytest.mark.parametrize("prompts,samples,hq,hkv,kv", CASES)
def test_samples_of_prompts(msa, prompts, samples, hq, hkv, kv):
    c = make(prompts, samples, hq, hkv, kv, seed=hq + len(prompts))
    check(c, *run(msa, c))
    check(c, *run(msa, c, groups=False))


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
def test_not_causal(msa, kv):
    c = make([300, 70], [[(0, 4), (130, 9)], [(60, 3)]], 8, 2, kv, seed=3)
    check(c, *run(msa, c, causal=False), causal=False)
    check(c, *run(msa, c, groups=False, causal=False, softmax_scale=0.2), causal=False, scale=0.2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_long_runs_split_over_many_ctas(msa, kv):
    c = make([20000], [[(900, 1), (0, 1), (17, 1)]], 8, 1, kv, seed=5)
    check(c, *run(msa, c))
    c = make([0, 0], [[(33000, 2)], [(5, 1)]], 4, 1, kv, seed=6)
    check(c, *run(msa, c, groups=False))


def test_empty_requests_few_keys_and_pages_that_are_not_there(msa):
    """Requests without tokens or keys, fewer keys than tokens, groups of which some have no tokens, missing pages in the shared and
    in the own run, a group that names more blocks than its requests have before their new tokens."""
    c = make([384, 300], [[(0, 2), (140, 0), (9, 3)], [(0, 1), (200, 2)]], 8, 2, "bf16", seed=7)
    c["table"][c["rows"][:3].long(), 1] = -1
    c["table"][c["rows"][4].long(), 3] = c["k"].shape[0]
    check(c, *run(msa, c))
    c["blocks"][:2] = 50
    shared = c["table"][c["rows"][0].long()]
    assert all(torch.equal(c["table"][r, :3], shared[:3]) for r in c["rows"][:3].tolist())
    # Blocks that not all have in common lie behind the last whole block before the shortest one's new tokens (384 + 0 -> 3; 300 -> 2).
    check(c, *run(msa, c))
    c = make([0, 0, 0], [[(0, 3)], [(5, 0)], [(0, 0)]], 4, 2, "bf16", seed=8)
    c["used"][:] = torch.where(c["used"] == 3, 2, c["used"])  # three tokens, two keys
    out, lse = run(msa, c)
    check(c, out, lse)
    first = int(c["cu"][int((c["used"] == 2).nonzero()[0])])
    assert (lse[first] == -float("inf")).all() and (out[first] == 0).all()


def test_what_a_token_does_not_see(msa):
    """NaN and infinities in later tokens' keys and values leave the earlier tokens as they are; who sees one gets NaN."""
    for kv in ("bf16", "fp16", "e4m3"):
        c = make([300], [[(0, 6), (50, 6)]], 8, 1, kv, seed=11, garbage=False)
        bad = float("nan")
        for r in range(2):
            pos = int(c["used"][r]) - 2  # of the last but one token
            page = int(c["table"][r, pos // 128])
            (c["k"] if r else c["v"])[page, 0, pos % 128, 5] = bad
        out, lse = run(msa, c)
        ref, rl, _ = S.prefix_attention(c["q"], c["k"].float(), c["v"].float(), c["cu"], c["table"], c["used"], SCALE)
        assert torch.equal(out.isnan().cpu(), ref.isnan()) and torch.equal(lse.isnan().cpu(), rl.isnan())
        early = [int(c["cu"][r]) + i for r in range(2) for i in range(4)]
        clean = make([300], [[(0, 6), (50, 6)]], 8, 1, kv, seed=11, garbage=False)
        ref, rl, size = S.prefix_attention(clean["q"], clean["k"].float(), clean["v"].float(), clean["cu"], clean["table"], clean["used"], SCALE)
        tol = half_step(c["q"].dtype) * (size + ref.abs()) * 1.01 + 2.0**-13 * size + 512 * 2.0**-25 * 6
        assert ((out.double().cpu() - ref).abs() <= tol)[early].all()


def test_rows_behind_the_last_request_stay(msa):
    c = make([300], [[(0, 2), (50, 1)]], 8, 2, "bf16", seed=12, extra=5)
    out, lse = torch.full_like(c["q"], 7.0, device=DEV), torch.full(c["q"].shape[:2], 7.0, device=DEV)
    run(msa, c, out=out, lse=lse)
    check(c, out, lse)
    assert (out[3:] == 7).all() and (lse[3:] == 7).all()


def test_same_bits_stream_plan_and_graph(msa):
    """Twice the same; on another stream; prepared; captured and replayed with other lengths and groups."""
    c = make([1000, 300], [[(i * 11, 1) for i in range(9)], [(3, 1), (80, 1)]], 16, 2, "bf16", seed=13)
    out, lse = run(msa, c)
    again, lse2 = run(msa, c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    d = {n: t.to(DEV) for n, t in c.items()}
    groups = dict(group_rows=d["rows"], cu_groups=d["ends"], group_blocks=d["blocks"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = msa.msa_prefix_attention(d["q"], d["k"], d["v"], d["cu"], page_table=d["table"], seqused_k=d["used"], stream=side, **groups)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, other)
    runner = msa.PrefixAttentionRunner(d["q"], d["k"], d["v"], d["cu"], page_table=d["table"], seqused_k=d["used"], return_softmax_lse=True, **groups)
    runner.workspace.fill_(0xFF)
    graph = torch.cuda.CUDAGraph()
    runner.run()
    with torch.cuda.graph(graph):
        runner.run()
    graph.replay()
    assert torch.equal(out, runner.out) and torch.equal(lse, runner.lse)
    d["used"] -= 7
    d["blocks"][0] = 2
    c["used"] -= 7
    c["blocks"][0] = 2
    graph.replay()
    torch.cuda.synchronize()
    check(c, runner.out, runner.lse)
    fault_clear(msa)


def test_groups_of_the_steps_tables(msa):
    """The groups as msa_step_tables finds them, of rows of a cache with others between, and a captured step that makes both."""
    c = make([700, 260, 40], [[(i * 9, 2) for i in range(5)], [(1, 1), (140, 3)], [(0, 1)]], 8, 2, "bf16", seed=14)
    b = len(c["used"])
    table, used = torch.full((3 * b, c["table"].shape[1]), -1, dtype=torch.int32), torch.zeros(3 * b, dtype=torch.int32)
    at = torch.arange(b) * 3 + 1
    table[at], used[at] = c["table"], c["used"]
    t = msa.msa_step_tables(table.to(DEV), used.to(DEV), at.to(torch.int32).to(DEV), (c["cu"][1:] - c["cu"][:-1]).to(DEV), total_q=int(c["cu"][-1]), num_pages=c["k"].shape[0])
    assert torch.equal(t.cu_seqlens_q.cpu(), c["cu"]) and torch.equal(t.page_table.cpu(), c["table"])
    by = {frozenset(c["rows"][lo:hi].tolist()): int(n) for lo, hi, n in zip(c["ends"], c["ends"][1:], c["blocks"]) if hi > lo}
    got = {frozenset(t.group_rows[lo:hi].tolist()): int(n) for lo, hi, n in zip(t.cu_groups, t.cu_groups[1:], t.group_blocks) if hi > lo}
    assert {g: n for g, n in got.items() if len(g) > 1} == {g: n for g, n in by.items() if len(g) > 1 and n > 0}
    d = {n: x.to(DEV) for n, x in c.items()}
    out, lse = msa.msa_prefix_attention(d["q"], d["k"], d["v"], t.cu_seqlens_q, page_table=t.page_table, seqused_k=t.seqused_k, group_rows=t.group_rows, cu_groups=t.cu_groups,
                                        group_blocks=t.group_blocks, return_softmax_lse=True)
    check(c, out, lse)


def test_hundreds_of_requests_and_pages_past_32_bits(msa):
    """Many requests of one prompt in a pool whose pages lie past 2^32 elements."""
    hkv, n = 4, 300
    pages = 70000  # of 65536 elements
    table = torch.full((n, 5), -1, dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    perm = torch.randperm(pages, generator=g)[: 3 + 2 * n].to(torch.int32)
    perm[:3] = torch.tensor([pages - 1, 65600, 7], dtype=torch.int32)
    table[:, :3] = perm[:3]
    table[:, 3] = perm[3 : 3 + n]
    table[:, 4] = perm[3 + n :]
    used = torch.randint(385, 640, (n,), generator=g).to(torch.int32)
    k = torch.empty(pages, hkv, 128, 128, dtype=torch.float8_e4m3fn, device=DEV)
    v = torch.empty_like(k)
    held = perm.long().unique().to(DEV)
    gg = torch.Generator(DEV).manual_seed(3)
    for x in (k, v):
        x[held] = torch.randn(len(held), hkv, 128, 128, generator=gg, device=DEV).to(x.dtype)
    q = torch.randn(n, 32, 128, generator=g).to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cu = torch.arange(n + 1, dtype=torch.int32)
    out, lse = msa.msa_prefix_attention(q.to(DEV), k, v, cu.to(DEV), page_table=table.to(DEV), seqused_k=used.to(DEV), group_rows=cu[:n].to(DEV).contiguous(), cu_groups=i32([0] + [n] * n),
                                        group_blocks=i32([3] + [0] * (n - 1)), return_softmax_lse=True)
    fault_clear(msa)
    # The pages held, renumbered for the check.
    small = torch.full((pages,), -1, dtype=torch.int32)
    small[held.cpu()] = torch.arange(len(held), dtype=torch.int32)
    some = [0, 1, 137, n - 1]
    c = dict(q=q[some], k=k[held].cpu(), v=v[held].cpu(), cu=torch.arange(len(some) + 1, dtype=torch.int32), table=torch.where(table[some] >= 0, small[table[some].long().clamp(min=0)], -1),
             used=used[some])
    check(c, out[some], lse[some])


@pytest.mark.parametrize("prompts,samples,hq,hkv,kv", [([1300], [[(0, 1), (150, 1)]], 16, 2, "fp16"), ([300, 260], [[(0, 1), (40, 1)], [(5, 1), (200, 1)]], 4, 1, "bf16"),
                                                       ([400], [[(0, 4), (140, 4), (3, 5)]], 2, 2, "e4m3"), ([520, 40], [[(0, 0), (7, 2), (9, 1)], [(0, 1)]], 12, 3, "bf16")])
def test_few_rows_in_all(msa, prompts, samples, hq, hkv, kv):
    """At most 16 rows for each KV head in all: units of 256 rows with the groups, of 16 without."""
    c = make(prompts, samples, hq, hkv, kv, seed=20 + hq)
    assert int(c["cu"][-1]) * (hq // hkv) <= 16
    check(c, *run(msa, c))
    check(c, *run(msa, c, groups=False, max_seqlen_q=5))
    check(c, *run(msa, c, causal=False), causal=False)
