"""NaN that a token sees, in the attention over shared prefixes: wherever its keys' runs are cut into parts, the token gets NaN."""
import pytest
import torch

import samples_util as S
from test_gpu_prefix_attention import SCALE, make, msa, run  # noqa: F401

pytestmark = pytest.mark.gpu
NAN = float("nan")


def check_nan(c, out, lse):
    """NaN where 64 bits have it, and nowhere else."""
    ref, rl, _ = S.prefix_attention(c["q"], c["k"].float(), c["v"].float(), c["cu"], c["table"], c["used"], SCALE)
    assert torch.equal(lse.isnan().cpu(), rl.isnan())
    assert torch.equal(out.isnan().cpu(), ref.isnan())


def nan_page(c, request, block, head):
    c["k"][int(c["table"][request, block]), head] = NAN


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
def test_a_query_of_nan_over_many_parts(msa, kv):
    """Each part of the row has nothing but NaN for scores, in every one of its 16 keys."""
    c = make([0] * 3, [[(4095, 1)], [(6399, 1)], [(500, 1)]], 8, 2, kv, seed=31, garbage=False)
    c["q"][0, :4] = NAN
    c["q"][1] = NAN
    for most in (1, None):
        out, lse = run(msa, c, groups=False, max_seqlen_q=most)
        check_nan(c, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
def test_a_page_of_nan_wherever_a_part_begins(msa, kv):
    """Requests of 25 blocks, one page of each NaN in one head: among them pages that begin a CTA's piece of a run."""
    n = 25
    c = make([0] * n, [[(3199, 1)] for _ in range(n)], 4, 2, kv, seed=32, garbage=False)
    for r in range(n):
        nan_page(c, r, r, r % 2)
    for most in (1, None):
        out, lse = run(msa, c, groups=False, max_seqlen_q=most)
        check_nan(c, out, lse)
        assert lse.isnan().sum() == 2 * n
    # One long request, more parts than a join's half-warps take at once.
    for first in range(8):
        c = make([0], [[(20479, 1)]], 4, 1, kv, seed=33, garbage=False)
        for block in range(first, 160, 8):
            nan_page(c, 0, block, 0)
        out, lse = run(msa, c, groups=False, max_seqlen_q=1)
        check_nan(c, out, lse)


def pieces(blocks, cost, before, grid=152, least=16, unit=12):
    """The blocks of the last unit on the line as its CTAs have them; `before` is what lies before it there."""
    total = before + unit + cost * blocks
    n = max(1, min(total // least, grid))
    where = [before + (unit + cost * j if j else 0) for j in range(blocks)]
    starts = [total * i // n for i in range(n + 1)]
    got = [[j for j, at in enumerate(where) if starts[i] <= at < starts[i + 1]] for i in range(n)]
    return [p for p in got if p]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("turn", [0, 1, 2, 3])
def test_parts_of_nan_that_one_half_warp_joins(msa, kv, turn):
    """Few rows of a long prefix: several half-warps join a row's parts by turns. All parts of one turn are NaN."""
    c = make([20000], [[(0, 1), (17, 1)]], 4, 1, kv, seed=34, garbage=False)
    cut = pieces(156, 3, 2 * 15)
    assert len(cut) >= 16
    for p in cut[turn::4]:
        for block in p:
            nan_page(c, int(c["rows"][0]), block, 0)
    out, lse = run(msa, c)
    check_nan(c, out, lse)
    assert bool(lse.isnan().all())
