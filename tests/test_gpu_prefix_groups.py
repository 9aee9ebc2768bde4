"""Group arrays of the attention over shared prefixes that are not as they should be: nothing outside the tensors is touched, and
requests that no group takes are attended by themselves."""
import pytest
import torch

import samples_util as S
from parity_util import fault_clear
from test_gpu_prefix_attention import DEV, check, make, msa  # noqa: F401

pytestmark = pytest.mark.gpu
GUARD = 1 << 16


def run_guarded(msa, c):
    """A call whose workspace lies between guards, as its outputs do."""
    t, hq, hkv, b = c["q"].shape[0], c["q"].shape[1], c["k"].shape[1], len(c["used"])
    d = {n: x.to(DEV) for n, x in c.items()}
    size = msa.lib().msa_prefix_attention_workspace_size(b, t, hq, hkv, 128, 1)
    raw = torch.full((size + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=DEV)
    wide = torch.full((t + 256, hq, 128), 7.0, dtype=c["q"].dtype, device=DEV)
    long = torch.full((t + 256, hq), 7.0, device=DEV)
    out, lse = wide[128 : 128 + t], long[128 : 128 + t]
    msa.msa_prefix_attention(d["q"], d["k"], d["v"], d["cu"], page_table=d["table"], seqused_k=d["used"], group_rows=d["rows"], cu_groups=d["ends"], group_blocks=d["blocks"],
                             out=out, lse=lse, workspace=raw[GUARD : GUARD + size])
    torch.cuda.synchronize()
    fault_clear(msa)
    assert bool((raw[:GUARD] == 0xA5).all()) and bool((raw[GUARD + size :] == 0xA5).all())
    assert bool((wide[:128] == 7).all()) and bool((wide[128 + t :] == 7).all()) and bool((long[:128] == 7).all()) and bool((long[128 + t :] == 7).all())
    return out, lse


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("first", [1, 2, 3, 6, 10**9])
def test_groups_that_do_not_begin_at_0(msa, kv, first):
    """Requests listed before the first group are in none; the last group's tokens end with the last request's."""
    c = make([512, 300], [[(0, 3), (140, 2), (9, 9), (30, 1)], [(0, 1), (200, 2)]], 8, 2, kv, seed=61)
    b = len(c["used"])
    c["ends"][:] = torch.tensor([first] + [b] * b)
    c["blocks"][:] = 0
    if first < b:
        same = c["rows"][first:].tolist()
        lead = c["table"][same[0]]
        c["blocks"][0] = min(int((c["table"][r] == lead).int().cumprod(0).sum()) for r in same) if len(same) > 1 else 2
    check(c, *run_guarded(msa, c))


@pytest.mark.parametrize("seed", range(12))
def test_arrays_of_any_numbers(msa, seed):
    """Groups that begin anywhere, requests listed over and over or not at all, more blocks than there are."""
    g = torch.Generator().manual_seed(seed)
    c = make([512, 300, 20], [[(0, 3), (140, 2), (9, 30), (30, 1)], [(0, 1), (200, 2), (7, 70)], [(100, 4)]], 8, 2, "e4m3" if seed % 3 == 2 else "bf16", seed=62, extra=4)
    b = len(c["used"])
    any_of = lambda lo, hi, n: torch.randint(lo, hi, (n,), generator=g).to(torch.int32)  # noqa: E731
    c["ends"][:] = any_of(-2, b + 3, b + 1)
    if seed % 2:
        c["rows"][:] = any_of(-1, b + 1, b)
    c["blocks"][:] = any_of(-1, 9, b)
    if seed > 7:
        c["rows"][:] = int((c["cu"][1:] - c["cu"][:-1]).argmax())
        c["ends"][:] = c["ends"].sort(descending=True).values
    run_guarded(msa, c)


def test_a_long_request_listed_thousands_of_times(msa):
    """The tokens listed sum up to more than 2^32; those past the tokens there are are left out."""
    b, t = 16384, 300000
    c = make([0], [[(100, 5)]], 1, 1, "bf16", seed=63)
    d = {n: x.to(DEV) for n, x in c.items()}
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cu = torch.full((b + 1,), t, dtype=torch.int32, device=DEV)
    cu[0] = 0
    table = torch.zeros(b, 1, dtype=torch.int32, device=DEV)
    used = torch.full((b,), 100, dtype=torch.int32, device=DEV)
    rows = torch.zeros(b, dtype=torch.int32, device=DEV)
    ends = torch.full((b + 1,), b, dtype=torch.int32, device=DEV)
    ends[0] = 0
    blocks = torch.zeros(b, dtype=torch.int32, device=DEV)
    q = torch.randn(t, 1, 128, dtype=torch.bfloat16, device=DEV)
    out, lse = msa.msa_prefix_attention(q, d["k"], d["v"], cu, page_table=table, seqused_k=used, group_rows=rows, cu_groups=ends, group_blocks=blocks, return_softmax_lse=True)
    torch.cuda.synchronize()
    fault_clear(msa)
    last = dict(q=q[-3:].cpu(), k=c["k"], v=c["v"], cu=i32([0, 3]).cpu(), table=table[:1].cpu(), used=used[:1].cpu())
    check(last, out[-3:], lse[-3:])
