"""What later tokens hold, in the attention over shared prefixes: their values may be NaN or infinite and leave the tokens before
them as they are; who sees them gets what 64 bits give; and a cache that has them takes no longer."""
import pytest
import torch

import samples_util as S
from step_util import half_step
from test_gpu_prefix_attention import DEV, SCALE, make, msa, run  # noqa: F401

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def check(c, out, lse, infinite=True):
    """Finite where 64 bits are, by the attention's own tolerances, and the same infinities and NaN elsewhere (`infinite` false: NaN
    may stand for an infinity whose probability is 0 in the products' type)."""
    ref, rl, size = S.prefix_attention(c["q"], c["k"].float(), c["v"].float(), c["cu"], c["table"], c["used"], SCALE)
    out, lse = out.double().cpu(), lse.double().cpu()
    fine = ref.isfinite()
    assert torch.equal(out.isfinite(), fine)
    if infinite:
        assert torch.equal(out[~fine].nan_to_num(7.0), ref[~fine].nan_to_num(7.0))
    tol = half_step(c["q"].dtype) * (size + ref.abs()) * 1.01 + 2.0**-13 * size
    if c["q"].dtype == torch.float16 or c["k"].dtype == torch.float8_e4m3fn:
        tol += int(c["used"].max()) * 2.0**-25 * 6 + 2.0**-25
    assert ((out - ref).abs() <= tol)[fine].all()
    good = rl.isfinite()
    assert torch.equal(lse.isfinite(), good) and ((lse - rl).abs() <= 2.0**-13 + rl.abs() * 2.0**-21)[good].all()


def spoil(c, request, back, columns, value, heads=slice(None)):
    """A value in some columns of the key that stands `back` before the request's end."""
    pos = int(c["used"][request]) - 1 - back
    c["v"][int(c["table"][request, pos // 128]), heads, pos % 128, columns] = value


# Units of 16 rows and of 256, of one tile and of two; the last tokens in one block, in two and in three; own runs that are cut.
SHAPES = [
    ([0], [[(200, 6)]], 2, 1, 6), ([0], [[(122, 9), (300, 4)]], 3, 3, 9), ([0], [[(70, 16)]], 4, 4, 16), ([0], [[(5000, 5)]], 3, 1, 5), ([0, 0], [[(0, 8)], [(3, 2)]], 2, 1, 8),
    ([300], [[(0, 6), (50, 6)]], 8, 1, None), ([130], [[(5, 40), (100, 30)]], 8, 1, None), ([260], [[(10, 12), (120, 20)]], 16, 1, None), ([0], [[(100, 300)]], 1, 1, None),
    ([128], [[(64, 150), (7, 3)]], 4, 2, None), ([0], [[(6000, 20)]], 8, 1, None),
]


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("prompts,samples,hq,hkv,most", SHAPES)
def test_values_of_later_tokens(msa, prompts, samples, hq, hkv, most, kv):
    values = [NAN] if kv == "e4m3" else [NAN, INF, -INF]
    flat = [new for group in samples for _, new in group]
    for turn, value in enumerate(values):
        c = make(prompts, samples, hq, hkv, kv, seed=40 + turn)
        lens = (c["cu"][1:] - c["cu"][:-1]).tolist()
        assert sorted(lens) == sorted(flat)
        for r, n in enumerate(lens):
            # The last token's in all columns; in the middle a few; the first token's none, so that it is finite.
            spoil(c, r, 0, slice(None), value)
            if n > 2:
                spoil(c, r, n // 2, slice(5, 9), value)
                spoil(c, r, n // 2, slice(127, 128), value, 0)
            if n > 4:
                spoil(c, r, 1, slice(64, 66), value)
        for groups in ([False] if most else [True, False]):
            out, lse = run(msa, c, groups=groups, max_seqlen_q=most)
            check(c, out, lse, infinite=max(lens) * (hq // hkv) <= 256)
            assert out[c["cu"][0]].isfinite().all()


@pytest.mark.parametrize("kv", ["bf16", "fp16", "e4m3"])
def test_keys_and_values_of_later_tokens_in_many_units_at_once(msa, kv):
    """Requests enough that a CTA has units with such values and without, one behind the other."""
    b = 300
    c = make([0] * b, [[(i % 140, 1 + i % 5)] for i in range(b)], 3, 1, kv, seed=51)
    for r in range(0, b, 7):
        spoil(c, r, 0, slice(r % 128, r % 128 + 1), NAN)
        pos = int(c["used"][r]) - 1
        c["k"][int(c["table"][r, pos // 128]), 0, pos % 128, 3] = NAN
    for most in (5, None):
        check(c, *run(msa, c, groups=False, max_seqlen_q=most))


def test_opposite_infinities(msa):
    """Both in one column are NaN to who sees both, infinite to who sees one."""
    for most in (4, None):
        c = make([0], [[(150, 4)]], 4, 1, "bf16", seed=52)
        spoil(c, 0, 2, slice(10, 12), INF)
        spoil(c, 0, 1, slice(11, 13), -INF)
        out, lse = run(msa, c, groups=False, max_seqlen_q=most)
        check(c, out, lse)
        assert out[0].isfinite().all() and out[1, 0, 11] == INF and out[2, 0, 11].isnan() and out[2, 0, 12] == -INF


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("most", [4, None])
def test_a_length_next_to_2_31_of_a_short_table(msa, kv, most):
    """Keys behind the table's last block are not there, however long the request is said to be; with a NaN among those that are."""
    c = make([0], [[(300, 4)]], 4, 1, kv, seed=53)
    c["used"][0] = 384
    live = torch.randn(c["v"].shape, generator=torch.Generator().manual_seed(1))
    c["k"], c["v"] = live.to(c["k"].dtype), (2 * live).to(c["v"].dtype)
    c["v"][int(c["table"][0, 1]), 0, 5, 7] = NAN
    c["used"][0] = 2**31 - 1
    check(c, *run(msa, c, groups=False, max_seqlen_q=most))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_nan_takes_no_time(msa, kv):
    """One NaN near the beginning, seen by all tokens of a prompt, and one in each of its last tokens: no more than twice the time."""
    lq, lk = 1024, 4096
    c = make([0], [[(lk - lq, lq)]], 16, 1, kv, seed=54, garbage=False)

    def time(c):
        d = {n: t.to(DEV) for n, t in c.items()}
        at = []
        for _ in range(8):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            for _ in range(4):
                msa.msa_prefix_attention(d["q"], d["k"], d["v"], d["cu"], page_table=d["table"], seqused_k=d["used"])
            end.record()
            torch.cuda.synchronize()
            at.append(begin.elapsed_time(end))
        return min(at)

    clean = time(c)
    spoil(c, 0, lk - 6, slice(3, 4), NAN)
    seen = time(c)
    for back in range(0, lq, 3):
        spoil(c, 0, back, slice(back % 128, back % 128 + 1), NAN)
    assert seen <= 2 * clean and time(c) <= 2 * clean
