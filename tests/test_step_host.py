"""What the C entry points of the serving step refuse, decided on the host before any CUDA call (CPU only)."""
import ctypes as C

import pytest

OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3
P = C.c_void_p(0x10000)      # never followed: the call ends before
ODD = C.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    import block_sparse_top_msa_gb300 as msa
    msa.build()
    return msa.lib()


def call(fn, names, good, **changed):
    return fn(*[changed.get(n, good[n]) for n in names])


ROPE = "q qs k ks dt wq wk eps cs most rd il pos t hq hkv d qo ko s".split()
ROPE_GOOD = dict(q=P, qs=1024, k=P, ks=256, dt=0, wq=P, wk=P, eps=1e-6, cs=P, most=10, rd=64, il=0, pos=P, t=0, hq=8, hkv=2, d=128, qo=P, ko=P, s=None)
APPEND = "q qs k ks v vs dt wq wk eps cs most rd il pos cu b pt mp np su t hq hkv d qo kp vp kdt s".split()
APPEND_GOOD = dict(ROPE_GOOD, v=P, vs=256, cu=P, b=1, pt=P, mp=1, np=1, su=P, kp=P, vp=P, kdt=0)
BWD = "dqo dko q qs k ks dt wq wk eps cs most rd il pos t hq hkv d dq dqs dk dks dwq dwk ws wb s".split()
BWD_GOOD = dict(ROPE_GOOD, dqo=P, dko=P, dq=P, dqs=1024, dk=P, dks=256, dwq=P, dwk=P, ws=P, wb=1 << 20)

BAD_ROPE = [(dict(q=None, t=1), INVALID), (dict(k=ODD), INVALID), (dict(wq=None), INVALID), (dict(wk=ODD), INVALID), (dict(pos=None, t=1), INVALID), (dict(cs=None), INVALID),
            (dict(qs=1016), INVALID), (dict(qs=1028), INVALID), (dict(ks=248), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
            (dict(eps=float("inf")), INVALID), (dict(eps=-1e-6), INVALID), (dict(most=0), INVALID), (dict(t=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=0), INVALID),
            (dict(d=64), UNSUPPORTED), (dict(dt=2), UNSUPPORTED), (dict(rd=24), UNSUPPORTED), (dict(rd=144), UNSUPPORTED), (dict(rd=-16), UNSUPPORTED),
            (dict(t=2**31 - 1), UNSUPPORTED)]


@pytest.mark.parametrize("bad,status", BAD_ROPE)
def test_norm_rope_refuses(L, bad, status):
    assert call(L.msa_qk_norm_rope, ROPE, ROPE_GOOD, **bad) == status
    assert call(L.msa_qk_norm_rope_append, APPEND, APPEND_GOOD, **bad) == status
    assert call(L.msa_qk_norm_rope_bwd, BWD, BWD_GOOD, **bad) == status


def test_norm_rope_accepts_no_tokens(L):
    assert call(L.msa_qk_norm_rope, ROPE, ROPE_GOOD) == OK
    assert call(L.msa_qk_norm_rope, ROPE, ROPE_GOOD, rd=0, cs=None) == OK
    assert call(L.msa_qk_norm_rope, ROPE, ROPE_GOOD, q=None, k=None, pos=None, qo=None, ko=None) == OK
    assert call(L.msa_qk_norm_rope_append, APPEND, APPEND_GOOD) == OK
    assert call(L.msa_qk_norm_rope_append, APPEND, APPEND_GOOD, kdt=2) == OK


@pytest.mark.parametrize("bad,status", [(dict(v=None, t=1), INVALID), (dict(vs=250), INVALID), (dict(qo=None, t=1), INVALID), (dict(kp=None), INVALID), (dict(vp=ODD), INVALID),
                                        (dict(cu=None), INVALID), (dict(pt=ODD), INVALID), (dict(su=None), INVALID), (dict(b=0), INVALID), (dict(mp=0), INVALID),
                                        (dict(np=0), INVALID), (dict(kdt=1), UNSUPPORTED), (dict(dt=1, kdt=2), UNSUPPORTED)])
def test_append_refuses(L, bad, status):
    assert call(L.msa_qk_norm_rope_append, APPEND, APPEND_GOOD, **bad) == status


@pytest.mark.parametrize("bad,status", [(dict(dqo=None, t=1), INVALID), (dict(dko=ODD), INVALID), (dict(dq=None, t=1), INVALID), (dict(dks=200), INVALID), (dict(dwq=None), INVALID),
                                        (dict(ws=None), TOO_SMALL), (dict(wb=100), TOO_SMALL), (dict(ws=C.c_void_p(0x10010)), INVALID)])
def test_backward_refuses(L, bad, status):
    assert call(L.msa_qk_norm_rope_bwd, BWD, BWD_GOOD, **bad) == status


def test_workspace_sizes(L):
    assert L.msa_qk_norm_rope_bwd_workspace_size(-1, 8, 2) == 0
    assert L.msa_qk_norm_rope_bwd_workspace_size(0, 8, 2) > 0
    assert L.msa_qk_norm_rope_bwd_workspace_size(10**6, 64, 8) <= 1 << 20
    assert L.msa_cache_workspace_size(-1, 5) == 0 and L.msa_cache_workspace_size(3, 0) == 0
    assert L.msa_cache_workspace_size(3, 100) == 256 + 512


TREE = "q dt k v kdt lists topk cu mask words pt mp np su b t hq hkv d mq scale out lse ws wb s".split()
TREE_GOOD = dict(q=P, dt=0, k=P, v=P, kdt=0, lists=P, topk=16, cu=P, mask=P, words=1, pt=P, mp=4, np=4, su=P, b=1, t=0, hq=8, hkv=2, d=128, mq=32, scale=0.0, out=P, lse=None,
                 ws=P, wb=1 << 30, s=None)


@pytest.mark.parametrize("bad,status", [(dict(), OK), (dict(mask=None), INVALID), (dict(mask=ODD), INVALID), (dict(words=0), INVALID), (dict(mq=33), INVALID),
                                        (dict(words=2, mq=64), OK), (dict(pt=None), INVALID), (dict(su=None), INVALID), (dict(mp=0), INVALID), (dict(hq=9), INVALID),
                                        (dict(topk=65), UNSUPPORTED), (dict(d=64), UNSUPPORTED), (dict(kdt=1), UNSUPPORTED), (dict(dt=1, kdt=2), UNSUPPORTED),
                                        (dict(wb=0), TOO_SMALL), (dict(hq=258, hkv=2), UNSUPPORTED)])
def test_tree_refuses(L, bad, status):
    assert call(L.msa_tree_attention, TREE, TREE_GOOD, **bad) == status
    plan = C.c_void_p()
    names = TREE[:-1] + ["plan"]
    assert call(L.msa_tree_attention_prepare, names, dict(TREE_GOOD, plan=C.byref(plan)), **bad) == status
    assert (plan.value is not None) == (status == OK)
    L.msa_sparse_attention_plan_free(plan)


def test_pages_refuse(L):
    pools = (C.c_void_p * 2)(0x10000, 0x20000)
    odd = (C.c_void_p * 2)(0x10000, 0x20008)
    ext = "pt mp nr su refs np rows lens n st ws wb s".split()
    good = dict(pt=P, mp=4, nr=8, su=P, refs=P, np=10, rows=P, lens=P, n=0, st=P, ws=P, wb=1 << 20, s=None)
    both = [(dict(pt=None), INVALID), (dict(su=ODD), INVALID), (dict(refs=None), INVALID), (dict(mp=0), INVALID), (dict(nr=0), INVALID), (dict(np=0), INVALID),
            (dict(n=-1), INVALID), (dict(nr=16385), UNSUPPORTED), (dict(n=16385), UNSUPPORTED), (dict(), OK)]
    few = [(dict(n=1, ws=None), TOO_SMALL), (dict(n=1, wb=16), TOO_SMALL), (dict(n=1, ws=C.c_void_p(0x10010)), INVALID), (dict(n=1, st=None), INVALID),
           (dict(n=1, rows=None), INVALID)]
    for bad, status in both + few + [(dict(n=1, lens=ODD), INVALID)]:
        assert call(L.msa_cache_extend, ext, good, **bad) == status
    for bad, status in both + [(dict(n=1, rows=None), INVALID)]:
        assert call(L.msa_cache_free, "pt mp nr su refs np rows n s".split(), good, **bad) == status
    fork = "pools k bytes pt mp nr su refs np rows lens n st ws wb s".split()
    fgood = dict(good, pools=pools, k=2, bytes=64)
    for bad, status in both + few + [(dict(pools=odd), INVALID), (dict(k=0), INVALID), (dict(bytes=24), INVALID), (dict(bytes=0), INVALID), (dict(pools=None), INVALID)]:
        assert call(L.msa_cache_fork, fork, fgood, **bad) == status
    copy = "pools k bytes np src dst n s".split()
    cgood = dict(pools=pools, k=2, bytes=64, np=3, src=P, dst=P, n=0, s=None)
    for bad, status in [(dict(), OK), (dict(n=1, src=None), INVALID), (dict(n=1, dst=ODD), INVALID), (dict(n=-1), INVALID), (dict(n=4097), UNSUPPORTED), (dict(np=0), INVALID),
                        (dict(pools=odd), INVALID)]:
        assert call(L.msa_cache_copy_pages, copy, cgood, **bad) == status
    acc = "pools k rb hkv pt mp np b su cu path plen w out s".split()
    agood = dict(pools=pools, k=2, rb=256, hkv=2, pt=P, mp=4, np=10, b=1, su=P, cu=P, path=P, plen=P, w=3, out=C.c_void_p(0x20000), s=None)
    for bad, status in [(dict(out=P), INVALID), (dict(out=None), INVALID), (dict(rb=100), INVALID), (dict(hkv=0), INVALID), (dict(b=0), INVALID), (dict(w=0), INVALID),
                        (dict(mp=0), INVALID), (dict(path=None), INVALID), (dict(plen=ODD), INVALID), (dict(cu=None), INVALID), (dict(b=16385), UNSUPPORTED),
                        (dict(hkv=1025), UNSUPPORTED), (dict(rb=8192), UNSUPPORTED), (dict(pools=odd), INVALID)]:
        assert call(L.msa_cache_accept, acc, agood, **bad) == status


def test_binding_refuses_before_the_library():
    """Shapes, types and places of tensors, before anything is launched."""
    import torch

    import block_sparse_top_msa_gb300 as msa
    x = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    w, pos = torch.ones(128), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        msa.msa_qk_norm_rope(x, x, w, w, None, pos)
    with pytest.raises(ValueError):
        msa.msa_cache_free(torch.zeros(2, 3, dtype=torch.int32), pos, pos, pos)
    with pytest.raises(ValueError):
        msa.msa_cache_copy_pages([], pos, pos)
    with pytest.raises(ValueError):
        msa.msa_tree_attention(x, x, x, pos, pos, pos, page_table=pos, seqused_k=pos)


def test_accept_refuses_a_pool_given_twice(L):
    names = "pools n row hkv pt mp np b su cu path len most out s".split()
    good = dict(pools=(C.c_void_p * 3)(0x10000, 0x20000, 0x10000), n=3, row=256, hkv=2, pt=P, mp=1, np=1, b=1, su=P, cu=P, path=P, len=P, most=1, out=C.c_void_p(0x30000), s=None)
    assert call(L.msa_cache_accept, names, good) == INVALID
