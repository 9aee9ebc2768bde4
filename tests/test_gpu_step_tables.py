"""A step's tables and drafted paths against plain lists."""
import random

import pytest
import torch

import samples_util as S
import step_util as U

pytestmark = pytest.mark.gpu


def tables(table, used, rows, lens, total, pages, **kw):
    import block_sparse_top_msa_gb300 as msa
    got = msa.msa_step_tables(S.ints(table), S.ints(used), S.ints(rows), S.ints(lens), total_q=total, num_pages=pages, **kw)
    assert msa.msa_read_device_fault() == 0
    return got


def check(table, used, rows, lens, total, pages):
    got = tables(table, used, rows, lens, total, pages)
    for name, x, want in zip(got._fields, got, S.step_tables(table, used, rows, lens, total, pages)):
        assert x.tolist() == want, name


def random_cache(rng, rows, width, prompts):
    """Rows that share the first pages of some prompts and go on with pages of their own; some with holes or pages out of range."""
    nxt, heads = 0, []
    for _ in range(prompts):
        n = rng.randint(1, width)
        heads.append(list(range(nxt, nxt + n)))
        nxt += n
    table, used = [], []
    for _ in range(rows):
        head = rng.choice(heads)
        keep = rng.randint(0, len(head))
        row = head[:keep] + list(range(nxt, nxt + width - keep))
        nxt += width - keep
        if rng.random() < 0.1:
            row[rng.randrange(width)] = rng.choice([-1, -5, 10**6])
        n = rng.choice([0, 1, 127, 128, 129, rng.randint(0, 128 * width), 128 * width])
        table.append([p if 128 * j < n else -1 for j, p in enumerate(row)])
        used.append(n)
    return table, used, nxt


@pytest.mark.parametrize("rows,width,batch,prompts", [(1, 1, 1, 1), (3, 2, 3, 1), (40, 7, 33, 3), (200, 65, 150, 9), (60, 300, 60, 4), (2500, 3, 1500, 40)])
def test_random_caches(rows, width, batch, prompts):
    rng = random.Random(rows * 7 + width)
    table, used, pages = random_cache(rng, rows, width, prompts)
    pick = rng.sample(range(rows), batch) if batch <= rows else [rng.randrange(rows) for _ in range(batch)]
    pick = [r if rng.random() < 0.95 else rng.choice([-1, rows, 10**9]) for r in pick]
    lens = [rng.choice([0, 1, 1, 1, 5, 130, -2]) for _ in range(batch)]
    total = sum(max(0, n) for n in lens)
    check(table, used, pick, lens, total, pages)
    check(table, used, pick, lens, total + 77, pages)
    check(table, used, pick, lens, total // 2, pages)
    check(table, used, pick, lens, 0, pages)


def test_a_row_given_twice_and_all_rows_alike():
    table, used = [[5, 6, 7, -1], [5, 6, 8, 9]], [300, 512]
    check(table, used, [0, 0, 1, 0], [1, 2, 3, 0], 10, 10)
    n = 3000
    check([[1, 2, 3]] * n, [384] * n, list(range(n)), [1] * n, n, 4)
    check([[i, 2, 3] for i in range(n)], [384] * n, list(range(n)), [1] * n, n, n)


def test_the_most_requests():
    n = 16384
    rng = random.Random(2)
    table = [[rng.randrange(500), i] for i in range(n)]
    check(table, [200] * n, list(range(n)), [rng.randint(0, 2) for _ in range(n)], 2 * n, n)


def test_lengths_whose_sum_passes_32_bits():
    n = 4
    table, used = [[0]] * n, [2**31 - 1] * n
    got = tables(table, used, list(range(n)), [2**30] * n, 8, 1)
    assert got.cu_seqlens_q.tolist() == [0] * 5 and got.token_rows.tolist() == [-1] * 8
    got = tables(table, used, list(range(n)), [3, 2**31 - 1, 2**31 - 1, 1], 8, 1)
    assert got.cu_seqlens_q.tolist() == [0, 3, 3, 3, 3] and got.positions.tolist() == [2**31 - 4, 2**31 - 3, 2**31 - 2] + [-1] * 5
    assert got.slots.tolist() == [-1] * 8


def test_written_in_place_captured_and_replayed():
    import block_sparse_top_msa_gb300 as msa
    rng = random.Random(4)
    table, used, pages = random_cache(rng, 30, 9, 3)
    t, u, rows, lens = S.ints(table), S.ints(used), S.ints(list(range(20))), S.ints([1] * 20)
    out = msa.msa_step_tables(t, u, rows, lens, total_q=40, num_pages=pages)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = msa.msa_step_tables(t, u, rows, lens, total_q=40, num_pages=pages, out=out, workspace=ws)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(out, again))
    for shift in range(3):
        pick = [(i * 3 + shift) % 30 for i in range(20)]
        n = [(i + shift) % 4 for i in range(20)]
        rows.copy_(S.ints(pick))
        lens.copy_(S.ints(n))
        ws.fill_(0xA5)
        graph.replay()
        for name, x, want in zip(out._fields, out, S.step_tables(table, used, pick, n, 40, pages)):
            assert x.tolist() == want, name


def tree(rng, n, reach):
    return [-1] + [max(0, c - rng.randint(1, reach)) for c in range(1, n)]


@pytest.mark.parametrize("batch,lo,hi,reach,words", [(1, 1, 1, 1, 1), (5, 0, 8, 3, 1), (9, 20, 40, 2, 2), (3, 100, 200, 4, 7), (150, 1, 64, 5, 3)])
def test_paths(batch, lo, hi, reach, words):
    import block_sparse_top_msa_gb300 as msa
    rng = random.Random(batch * 31 + hi)
    sampled, drafts, mask, cu = [], [], [], [0]
    for _ in range(batch):
        n = rng.randint(lo, hi)
        parent = tree(rng, n, reach) if n else []
        if n:
            mask += S.mask_rows(parent, words).tolist()
        d = [rng.randint(0, 3) for _ in range(n)]
        drafts += d
        sampled += [rng.choice([d[c] for c in range(n) if parent[c] == i] or [9]) if rng.random() < 0.9 else rng.randint(0, 3) for i in range(n)]
        cu.append(len(drafts))
    for most in (32 * words, 3, 1):
        t = lambda x: S.ints(x) if x else torch.empty(0, dtype=torch.int32, device="cuda")  # noqa: E731
        m = torch.tensor(mask, dtype=torch.int32, device="cuda").view(-1, words)
        got = msa.msa_draft_path(t(sampled), t(drafts), m, S.ints(cu), max_path=None if most == 32 * words else most)
        want = S.draft_path(sampled, drafts, [[w & 0xFFFFFFFF for w in r] for r in mask], cu, most, len(drafts))
        assert [x.tolist() for x in got] == [list(w) for w in want], most
    assert msa.msa_read_device_fault() == 0


def test_paths_of_trees_longer_than_their_mask_and_of_several_roots():
    import block_sparse_top_msa_gb300 as msa
    # 40 nodes in one word: nodes past the 31st are seen by nobody's mask; those behind it still name parents in it.
    n = 40
    rows = [(1 << c) - 1 if c < 31 else (1 << 31) - 1 for c in range(n)]  # ancestors 0 .. min(c, 31) - 1: a chain
    rows = [[r | (1 << c if c < 32 else 0)] for c, r in enumerate(rows)]
    drafts, sampled = [1] * n, [1] * n
    want = S.draft_path(sampled, drafts, rows, [0, n], n, n)
    signed = [[r[0] - (1 << 32) if r[0] >= 1 << 31 else r[0]] for r in rows]
    got = msa.msa_draft_path(S.ints(sampled), S.ints(drafts), S.ints(signed), S.ints([0, n]), max_path=n)
    assert [x.tolist() for x in got] == [list(w) for w in want]
    # A second root is on nobody's path, nor are its children.
    rows = S.mask_rows([-1, -1, 0, 1]).tolist()
    got = msa.msa_draft_path(S.ints([5, 5, 6, 7]), S.ints([5, 5, 5, 5]), S.ints(rows), S.ints([0, 4]))
    assert got[0].tolist()[0][:3] == [0, 2, -1] and got[1].tolist() == [2] and got[2].tolist() == [6]
