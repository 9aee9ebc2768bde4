"""Outputs of the operators of a step of samples that share memory with an input or with another output, wherever they begin: refused
on the host before any CUDA call (CPU only)."""
import ctypes as C

import pytest

from test_step_host_samples import (INVALID, L, OK, PATH, PATH_GOOD, PREFIX, PREFIX_GOOD, SAMPLE, SAMPLE_GOOD, TABLES, TABLES_GOOD, TOO_SMALL, at,  # noqa: F401
                                    call)


def by(i, n):
    """n bytes from where argument i begins."""
    return C.c_void_p(0x100000 + 0x1000 * i + n)


# Of 2 requests, 3 tokens, rows of 4 pages and a cache of 8 rows; no call of these comes as far as a launch: the workspace is too small.
@pytest.mark.parametrize("clash", [dict(pto=by(0, 124)), dict(pto=by(0, -28)), dict(suo=by(1, 28)), dict(cu=by(2, 4)), dict(gr=by(3, 4)), dict(cu=by(5, 4)), dict(sl=by(8, -8)), dict(sl=by(7, 8)),
                                   dict(cg=by(12, -8)), dict(ws=C.c_void_p(0x10000), pt=C.c_void_p(0x10080)), dict(ws=C.c_void_p(0x10000), gb=C.c_void_p(0x100fc))])
def test_step_tables(L, clash):
    assert call(L.msa_step_tables, TABLES, TABLES_GOOD, **clash) == INVALID


@pytest.mark.parametrize("apart", [dict(pto=by(0, 128)), dict(pto=by(0, -32)), dict(suo=by(1, 32)), dict(cu=by(2, 8)), dict(sl=by(7, 16)), dict(cg=by(12, -12))])
def test_step_tables_side_by_side(L, apart):
    assert call(L.msa_step_tables, TABLES, TABLES_GOOD, wb=16, **apart) == TOO_SMALL


# Three rows of 100 (fp32), 120 apart.
GOOD = dict(SAMPLE_GOOD, rows=3, stride=120)


@pytest.mark.parametrize("clash", [dict(out=by(0, 396)), dict(out=by(0, 392)), dict(out=by(0, 472)), dict(out=by(0, 960 + 396)), dict(out=by(0, -8)), dict(out=by(1, 8)), dict(lp=by(2, 8)), dict(lp=by(2, -8)),
                                   dict(out=by(5, 4), k=by(5, 0)), dict(lp=by(5, 4), p=by(5, 8)), dict(out=by(0, 476)), dict(ws=C.c_void_p(0x10000), u=C.c_void_p(0x10010))])
def test_sample(L, clash):
    assert call(L.msa_sample, SAMPLE, GOOD, **clash) == INVALID


@pytest.mark.parametrize("apart", [dict(out=by(0, 400)), dict(out=by(0, 468)), dict(out=by(0, 880)), dict(out=by(0, 960 + 400)), dict(out=by(0, -12)), dict(lp=by(2, 12)), dict(out=by(1, 12))])
def test_sample_between_the_rows_and_beside(L, apart):
    assert call(L.msa_sample, SAMPLE, GOOD, wb=16, **apart) == TOO_SMALL


# One request of four nodes, a path of four.
@pytest.mark.parametrize("clash", [dict(path=by(0, 12)), dict(path=by(1, -12)), dict(path=by(2, 8)), dict(len=by(3, 4)), dict(nxt=by(4, 12)), dict(len=by(4, 4)), dict(path=by(6, -12))])
def test_draft_path(L, clash):
    assert call(L.msa_draft_path, PATH, PATH_GOOD, **clash) == INVALID


# One token of 8 heads: 2048 bytes; a pool of four pages: 2^18.
FAR = dict(k=C.c_void_p(0x1000000), v=C.c_void_p(0x2000000), ws=C.c_void_p(0x10000000))


@pytest.mark.parametrize("clash", [dict(out=by(0, 2032)), dict(out=by(0, -2032)), dict(out=by(0, 1024)), dict(lse=by(9, 2044)), dict(lse=by(0, 4)), dict(lse=by(3, 4)), dict(out=by(4, 0)), dict(out=by(5, -2032)),
                                   dict(lse=by(6, -28)), dict(lse=by(7, 4)), dict(lse=by(8, 0)), dict(out=C.c_void_p(0x1000000 + (1 << 18) - 16)), dict(out=C.c_void_p(0x2000000 - 2032)),
                                   dict(ws=by(0, 1024)), dict(ws=by(9, 256))])
def test_prefix_attention(L, clash):
    good = dict(PREFIX_GOOD, t=1, **FAR)
    assert call(L.msa_prefix_attention, PREFIX, good, **clash) == INVALID
    plan = C.c_void_p()
    assert call(L.msa_prefix_attention_prepare, PREFIX[:-1] + ["plan"], dict(good, plan=C.byref(plan)), **clash) == INVALID and plan.value is None


def test_prefix_attention_of_no_tokens_covers_nothing(L):
    assert call(L.msa_prefix_attention, PREFIX, dict(PREFIX_GOOD, t=0), out=by(0, 16)) == OK


def test_prefix_attention_workspace_without_groups(L):
    """Only units that a range cuts leave parts: two pieces of 256 rows a CTA, and eight bytes a token."""
    size = L.msa_prefix_attention_workspace_size
    assert size(1, 32768, 64, 4, 128, 0) < 50 << 20
    assert size(1, 1 << 20, 64, 4, 128, 0) - size(1, 32768, 64, 4, 128, 0) == 8 * ((1 << 20) - 32768)
    assert size(4, 600, 64, 4, 128, 0) < size(4, 700, 64, 4, 128, 0)
