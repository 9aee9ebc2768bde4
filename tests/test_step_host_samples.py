"""What the entry points of a step of samples refuse, decided on the host before any CUDA call (CPU only)."""
import ctypes as C

import pytest

OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3
P = C.c_void_p(0x10000)      # never followed: the call ends before
ODD = C.c_void_p(0x10002)


def at(i):
    return C.c_void_p(0x100000 + 0x1000 * i)


@pytest.fixture(scope="module")
def L():
    import block_sparse_top_msa_gb300 as msa
    msa.build()
    return msa.lib()


def call(fn, names, good, **changed):
    return fn(*[changed.get(n, good[n]) for n in names])


TABLES = "pt mp nr su np rows lens b t cu suo pto tr pos sl gr cg gb ws wb s".split()
TABLES_GOOD = dict(pt=at(0), mp=4, nr=8, su=at(1), np=10, rows=at(2), lens=at(3), b=2, t=3, cu=at(4), suo=at(5), pto=at(6), tr=at(7), pos=at(8), sl=at(9), gr=at(10), cg=at(11),
                   gb=at(12), ws=P, wb=1 << 20, s=None)


@pytest.mark.parametrize("bad,status", [(dict(pt=None), INVALID), (dict(su=ODD), INVALID), (dict(rows=None), INVALID), (dict(lens=ODD), INVALID), (dict(cu=None), INVALID),
                                        (dict(suo=None), INVALID), (dict(pto=ODD), INVALID), (dict(tr=None), INVALID), (dict(sl=C.c_void_p(0x10004)), INVALID), (dict(gr=None), INVALID),
                                        (dict(cg=None), INVALID), (dict(gb=ODD), INVALID), (dict(mp=0), INVALID), (dict(nr=0), INVALID), (dict(np=0), INVALID), (dict(b=0), INVALID),
                                        (dict(t=-1), INVALID), (dict(pto=at(0)), INVALID), (dict(suo=at(1)), INVALID), (dict(cu=at(3)), INVALID), (dict(gr=at(12)), INVALID),
                                        (dict(b=16385), UNSUPPORTED), (dict(wb=16), TOO_SMALL), (dict(ws=None), TOO_SMALL), (dict(ws=C.c_void_p(0x10010)), INVALID)])
def test_step_tables_refuses(L, bad, status):
    assert call(L.msa_step_tables, TABLES, TABLES_GOOD, **bad) == status


def test_step_tables_workspace(L):
    assert L.msa_step_tables_workspace_size(0) == 0 and L.msa_step_tables_workspace_size(16385) == 0
    assert L.msa_step_tables_workspace_size(1) == 256 and L.msa_step_tables_workspace_size(16384) == 16 * 16384


SAMPLE = "x dt stride rows vocab u t k p m out lp ws wb s".split()
SAMPLE_GOOD = dict(x=at(0), dt=3, stride=100, rows=0, vocab=100, u=at(1), t=None, k=None, p=None, m=None, out=at(2), lp=None, ws=P, wb=1 << 30, s=None)


@pytest.mark.parametrize("bad,status", [(dict(), OK), (dict(x=None, u=None, out=None), OK), (dict(rows=1, x=None), INVALID), (dict(rows=1, u=None), INVALID),
                                        (dict(rows=1, out=None), INVALID), (dict(x=ODD), INVALID), (dict(x=ODD, dt=0), OK), (dict(x=C.c_void_p(0x10001), dt=1), INVALID),
                                        (dict(t=ODD), INVALID), (dict(k=ODD), INVALID), (dict(p=ODD), INVALID), (dict(m=ODD), INVALID), (dict(lp=ODD), INVALID),
                                        (dict(rows=-1), INVALID), (dict(vocab=0), INVALID), (dict(stride=99), INVALID), (dict(dt=2), UNSUPPORTED), (dict(dt=4), UNSUPPORTED),
                                        (dict(vocab=(1 << 19) + 1, stride=1 << 20), UNSUPPORTED), (dict(rows=(1 << 24) + 1), UNSUPPORTED), (dict(out=at(1)), INVALID),
                                        (dict(lp=at(2)), INVALID), (dict(lp=at(3), t=at(3)), INVALID),
                                        (dict(rows=1, ws=None), TOO_SMALL), (dict(rows=1, wb=100), TOO_SMALL), (dict(rows=1, ws=C.c_void_p(0x10010)), INVALID)])
def test_sample_refuses(L, bad, status):
    assert call(L.msa_sample, SAMPLE, SAMPLE_GOOD, **bad) == status


def test_sample_workspace(L):
    size = L.msa_sample_workspace_size
    assert size(-1, 5, 3) == 0 and size(1, 0, 3) == 0 and size(1, (1 << 19) + 1, 3) == 0 and size(1, 5, 2) == 0 and size(1 << 25, 5, 0) == 0
    assert size(0, 5, 3) == 0 and size(512, 200019, 0) == 256 and 2 * 512 * 200019 < size(512, 200019, 3) < 1 << 28  # two bytes a token


PATH = "sa dr mask words cu b t w path len nxt s".split()
PATH_GOOD = dict(sa=at(0), dr=at(1), mask=at(2), words=1, cu=at(3), b=1, t=4, w=4, path=at(4), len=at(5), nxt=at(6), s=None)


@pytest.mark.parametrize("bad", [dict(sa=None), dict(dr=ODD), dict(mask=None), dict(words=0), dict(cu=None), dict(b=0), dict(t=-1), dict(w=0), dict(path=None), dict(len=ODD),
                                 dict(nxt=None), dict(path=at(0)), dict(len=at(6)), dict(nxt=at(3))])
def test_draft_path_refuses(L, bad):
    assert call(L.msa_draft_path, PATH, PATH_GOOD, **bad) == INVALID


def test_binding_refuses_before_the_library():
    import torch

    import block_sparse_top_msa_gb300 as msa
    i, f = torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    with pytest.raises(ValueError):
        msa.msa_step_tables(torch.zeros(2, 3, dtype=torch.int32), i, i, i, total_q=3, num_pages=4)
    with pytest.raises(ValueError):
        msa.msa_sample(torch.zeros(3, 10), f)
    with pytest.raises(TypeError):
        msa.msa_sample([1.0], f)
    with pytest.raises(ValueError):
        msa.msa_draft_path(i, i, torch.zeros(3, 1, dtype=torch.int32), i)


def test_fp32_is_no_type_of_the_attention(L):
    """The code of a logit's type, given to the operators that do not know it."""
    assert L.msa_sparse_attention_fwd(P, 3, P, P, 3, P, 4, P, P, None, 0, 0, None, 1, 0, 128, 4, 2, 128, 32, 1, C.c_float(0.0), P, None, P, 1 << 30, None) == UNSUPPORTED


PREFIX = "q dt k v kdt cu pt mp np su rows ends blocks b t hq hkv d mq causal scale out lse ws wb s".split()
PREFIX_GOOD = dict(q=at(0), dt=0, k=at(1), v=at(2), kdt=0, cu=at(3), pt=at(4), mp=4, np=4, su=at(5), rows=at(6), ends=at(7), blocks=at(8), b=1, t=0, hq=8, hkv=2, d=128, mq=0, causal=1, scale=C.c_float(0.0),
                   out=at(9), lse=None, ws=P, wb=1 << 30, s=None)


@pytest.mark.parametrize("bad,status", [(dict(), OK), (dict(rows=None, ends=None, blocks=None), OK), (dict(kdt=2), OK), (dict(dt=1, kdt=1), OK), (dict(q=None), INVALID),
                                        (dict(k=ODD), INVALID), (dict(v=None), INVALID), (dict(cu=ODD), INVALID), (dict(pt=None), INVALID), (dict(su=None), INVALID),
                                        (dict(rows=None), INVALID), (dict(ends=None), INVALID), (dict(blocks=None), INVALID), (dict(rows=ODD), INVALID), (dict(b=0), INVALID),
                                        (dict(t=-1), INVALID), (dict(mq=-1), INVALID), (dict(mp=0), INVALID), (dict(np=0), INVALID), (dict(hq=9), INVALID), (dict(hkv=0), INVALID), (dict(out=None), INVALID),
                                        (dict(t=1, out=at(0)), INVALID), (dict(lse=ODD), INVALID), (dict(ws=C.c_void_p(0x10010)), INVALID), (dict(d=64), UNSUPPORTED),
                                        (dict(hq=258), UNSUPPORTED), (dict(b=16385), UNSUPPORTED), (dict(mp=(1 << 23) + 1), UNSUPPORTED), (dict(kdt=1), UNSUPPORTED),
                                        (dict(dt=1, kdt=2), UNSUPPORTED), (dict(dt=3), UNSUPPORTED), (dict(kdt=3), UNSUPPORTED), (dict(t=1 << 28), UNSUPPORTED),
                                        (dict(wb=100), TOO_SMALL), (dict(ws=None), TOO_SMALL)])
def test_prefix_attention_refuses(L, bad, status):
    assert call(L.msa_prefix_attention, PREFIX, PREFIX_GOOD, **bad) == status
    plan = C.c_void_p()
    names = PREFIX[:-1] + ["plan"]
    assert call(L.msa_prefix_attention_prepare, names, dict(PREFIX_GOOD, plan=C.byref(plan)), **bad) == status
    assert (plan.value is not None) == (status == OK)
    L.msa_sparse_attention_plan_free(plan)


def test_prefix_attention_workspace(L):
    size = L.msa_prefix_attention_workspace_size
    assert size(0, 5, 8, 2, 128, 0) == 0 and size(1, 5, 8, 3, 128, 0) == 0 and size(1, 5, 8, 2, 64, 0) == 0 and size(16385, 5, 8, 2, 128, 1) == 0
    assert size(4, 100, 64, 4, 128, 1) - size(4, 100, 64, 4, 128, 0) == 100 * 64 * 520
