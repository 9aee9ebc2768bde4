"""Norm and rotation of q and k, forward, appending to a cache, and backward, against 64 bits.

Tolerances, from the arithmetic: the float32 chain of the forward (a sum of 128 squares in a tree, the inverse root, two products,
the two products and the sum of the rotation) is within 16 roundings of 2^-24 of the magnitudes that make an element, 2^-20; then
one rounding to the type, half a step relative to the value. fp16 below its normal range is off by at most 2^-25. The backward's
chain is within 64 roundings, 2^-18; the weights' gradients add up to 256 sums in a row, 2^-16 of the terms' magnitudes."""
import pytest
import torch

from step_util import DT, bits, half_step, norm_rope, norm_rope_bwd, rope_table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CHAIN, CHAIN_BWD, SUMS = 2.0**-20, 2.0**-18, 2.0**-16
TINY = {torch.float16: 2.0**-25, torch.bfloat16: 0.0, torch.float8_e4m3fn: 2.0**-10}


@pytest.fixture(scope="module")
def msa():
    import block_sparse_top_msa_gb300 as m
    m.build()
    m.lib()
    return m


def near(got, ref, mag, dtype, chain):
    """Within one rounding to the type and the float32 chain before it."""
    got = got.double().cpu()
    tol = half_step(dtype) * (ref.abs() + chain * mag) + chain * mag + TINY[dtype]
    bad = (got - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), ((got - ref).abs() / tol).max().item())


def inputs(tokens, hq, hkv, rotary, dtype, seed=0, packed=True, length=50):
    g = torch.Generator().manual_seed(seed)
    heads = hq + 2 * hkv
    x = torch.randn(tokens, heads, 128, generator=g) * (0.2 + 5 * torch.rand(tokens, 1, 1, generator=g))
    x = x.to(DT[dtype])
    q, k, v = x[:, :hq], x[:, hq : hq + hkv], x[:, hq + hkv :]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = 1 + 0.3 * torch.randn(2, 128, generator=g)
    pos = torch.randint(0, length, (tokens,), generator=g).to(torch.int32)
    if tokens > 3:
        pos[1], pos[2], pos[3] = -1, length, 2**31 - 1  # padding
    return x, q, k, v, w, rope_table(length, rotary) if rotary else None, pos


def on_gpu(x, hq, hkv, packed):
    x = x.to(DEV)
    parts = x[:, :hq], x[:, hq : hq + hkv], x[:, hq + hkv :]
    return parts if packed else tuple(p.contiguous() for p in parts)


def gpu(t):
    return None if t is None else t.to(DEV)


SHAPES = [(1, 1, 1, 128, "bf16", False, True), (4, 64, 4, 128, "bf16", False, True), (33, 12, 3, 96, "fp16", True, True), (257, 8, 8, 64, "bf16", True, False),
          (130, 5, 5, 16, "fp16", False, True), (65, 40, 4, 112, "bf16", False, True), (19, 7, 1, 0, "bf16", False, True), (3, 3, 2, 80, "fp16", True, False)]


@pytest.mark.parametrize("tokens,hq,hkv,rotary,dtype,interleaved,packed", SHAPES)
def test_forward(msa, tokens, hq, hkv, rotary, dtype, interleaved, packed):
    x, q, k, v, w, table, pos = inputs(tokens, hq, hkv, rotary, dtype, packed=packed)
    if rotary == 0:
        pos = pos.clamp(max=49)
    gq, gk, _ = on_gpu(x, hq, hkv, packed)
    oq, ok = msa.msa_qk_norm_rope(gq, gk, w[0].to(DEV), w[1].to(DEV), gpu(table), pos.to(DEV), eps=1e-6, interleaved=interleaved)
    for got, src, wt in ((oq, q, w[0]), (ok, k, w[1])):
        ref, mag = norm_rope(src, wt, table, pos, interleaved)
        near(got, ref, mag, DT[dtype], CHAIN)


def test_forward_in_place_and_extremes(msa):
    """Contiguous inputs may be the outputs; rows of zeros, of the largest eps, of infinities and NaN keep to themselves."""
    x, q, k, v, w, table, pos = inputs(9, 4, 2, 128, "bf16", packed=False)
    pos = torch.arange(9, dtype=torch.int32)
    q[0] = 0
    q[2, 1] = float("inf")
    q[3, 0, 5] = float("nan")
    gq, gk = q.to(DEV), k.to(DEV)
    oq, ok = msa.msa_qk_norm_rope(gq, gk, w[0].to(DEV), w[1].to(DEV), table.to(DEV), pos.to(DEV), eps=4.0, q_out=gq, k_out=gk)
    assert oq.data_ptr() == gq.data_ptr() and ok.data_ptr() == gk.data_ptr()
    ref, mag = norm_rope(q, w[0], table, pos, False, eps=4.0)
    odd = torch.zeros(9, 4, dtype=torch.bool)
    odd[2, 1], odd[3, 0] = True, True
    assert oq.cpu()[odd].isnan().all()
    near(oq.cpu()[~odd], ref[~odd], mag[~odd], torch.bfloat16, CHAIN)
    assert (oq[0] == 0).all()


@pytest.mark.parametrize("tokens,hq,hkv,rotary,dtype,interleaved,packed", SHAPES)
def test_backward(msa, tokens, hq, hkv, rotary, dtype, interleaved, packed):
    x, q, k, v, w, table, pos = inputs(tokens, hq, hkv, rotary, dtype, packed=packed)
    if rotary == 0:
        pos = pos.clamp(max=49)
    g = torch.Generator().manual_seed(9)
    dq, dk = (torch.randn(tokens, n, 128, generator=g).to(DT[dtype]) for n in (hq, hkv))
    gq, gk, _ = on_gpu(x, hq, hkv, packed)
    into = torch.full((tokens, hq + 2 * hkv, 128), 7.0, dtype=DT[dtype], device=DEV)
    args = (dq.to(DEV), dk.to(DEV), gq, gk, w[0].to(DEV), w[1].to(DEV), gpu(table), pos.to(DEV))
    got = msa.msa_qk_norm_rope_bwd(*args, eps=1e-6, interleaved=interleaved, dq=into[:, :hq], dk=into[:, hq : hq + hkv])
    again = msa.msa_qk_norm_rope_bwd(*args, eps=1e-6, interleaved=interleaved)
    assert all(torch.equal(bits(a.contiguous()), bits(b.contiguous())) for a, b in zip(got[:2], again[:2]))
    assert torch.equal(got[2], again[2]) and torch.equal(got[3], again[3])
    assert (into[:, hq + hkv :] == 7).all()  # the packed gradient's other part
    for dx, dw, src, wt, d in ((got[0], got[2], q, w[0], dq), (got[1], got[3], k, w[1], dk)):
        ref, mag, rw, terms = norm_rope_bwd(src, wt, d, table, pos, interleaved)
        near(dx, ref, mag, DT[dtype], CHAIN_BWD)
        assert ((dw.double().cpu() - rw).abs() <= SUMS * terms).all()


def test_backward_against_differences(msa):
    """The kernel's gradients along a direction against central differences of the 64-bit forward: h = 1e-5, whose truncation
    (h^2 times third derivatives of order one) and cancellation (2^-53 / h) are below 1e-9 of the terms."""
    x, q, k, v, w, table, pos = inputs(21, 6, 2, 64, "fp16")
    g = torch.Generator().manual_seed(4)
    d = torch.randn(21, 6, 128, generator=g).to(torch.float16)
    dk = torch.zeros(21, 2, 128, dtype=torch.float16)
    got = msa.msa_qk_norm_rope_bwd(d.to(DEV), dk.to(DEV), x.to(DEV)[:, :6], x.to(DEV)[:, 6:8], w[0].to(DEV), w[1].to(DEV), table.to(DEV), pos.to(DEV), interleaved=True)
    ux = torch.randn(21, 6, 128, generator=g).double()
    uw = torch.randn(128, generator=g).double()

    def f(h, which):
        y, _ = norm_rope(q.double() + (h * ux if which == 0 else 0), w[0].double() + (h * uw if which == 1 else 0), table, pos, True)
        return (y * d.double()).sum()

    ref, mag, _, terms = norm_rope_bwd(q, w[0], d, table, pos, True)
    for which, grad, u, tol in ((0, got[0], ux, half_step(torch.float16) * ref.abs() + 2 * CHAIN_BWD * mag + 2.0**-25), (1, got[2], uw, SUMS * terms)):
        slope = (f(1e-5, which) - f(-1e-5, which)) / 2e-5
        along = (grad.double().cpu() * u).sum()
        assert (along - slope).abs() <= (tol * u.abs()).sum() + 1e-6 * (mag * ux.abs()).sum()
    assert (got[1] == 0).all() and (got[3] == 0).all()


def test_no_tokens(msa):
    z = torch.zeros(0, 4, 128, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(128, device=DEV)
    pos = torch.zeros(0, dtype=torch.int32, device=DEV)
    q, k = msa.msa_qk_norm_rope(z, z, w, w, None, pos)
    assert q.shape == k.shape == z.shape
    got = msa.msa_qk_norm_rope_bwd(z, z, z, z, w, w, None, pos)
    assert (got[2] == 0).all() and (got[3] == 0).all()


@pytest.mark.parametrize("hq,hkv,rotary,dtype,kv,interleaved", [(8, 2, 128, "bf16", "bf16", False), (12, 3, 64, "fp16", "fp16", True), (64, 4, 64, "bf16", "e4m3", False),
                                                                (1, 1, 96, "bf16", "e4m3", True)])
def test_append(msa, hq, hkv, rotary, dtype, kv, interleaved):
    """Ragged sequences whose tokens cross pages, one without tokens, pages missing or out of range, padding tokens, and rows behind
    the last sequence: what is not written stays as it was, byte for byte."""
    lens, used = [3, 0, 9, 1, 40, 5], [128, 77, 133, 1, 300, 3]  # the last has more tokens than keys
    total, tail = sum(lens), 4
    x, q, k, v, w, table, pos = inputs(total + tail, hq, hkv, rotary, dtype)
    v[5, 0, :4] = torch.tensor([1000.0, -500.0, 448.0, 464.0])
    x[:, hq + hkv :] = v
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    pages = 9
    pt = torch.tensor([[4, -1, -1], [0, -1, -1], [8, 2, -1], [1, 3, -1], [5, pages, 6], [7, -1, -1]], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    kp, vp = (torch.randn(pages, hkv, 128, 128, generator=g).to(DT[kv]) for _ in range(2))
    gk_pool, gv_pool = kp.to(DEV), vp.to(DEV)
    out = torch.full((total + tail, hq, 128), 3.0, dtype=DT[dtype], device=DEV)
    gx = x.to(DEV)
    msa.msa_qk_norm_rope_append(gx[:, :hq], gx[:, hq : hq + hkv], gx[:, hq + hkv :], w[0].to(DEV), w[1].to(DEV), table.to(DEV), pos.to(DEV), cu.to(DEV), gk_pool, gv_pool,
                                page_table=pt.to(DEV), seqused_k=torch.tensor(used, dtype=torch.int32, device=DEV), interleaved=interleaved, q_out=out)
    ref, mag = norm_rope(q, w[0], table, pos, interleaved)
    near(out[:total], ref[:total], mag[:total], DT[dtype], CHAIN)
    assert (out[total:] == 3).all()
    rk, mk = norm_rope(k, w[1], table, pos, interleaved)
    touched = torch.zeros(pages, 128, dtype=torch.bool)
    gk_pool, gv_pool = gk_pool.cpu(), gv_pool.cpu()
    for b, n in enumerate(lens):
        for i in range(n):
            t, p = int(cu[b]) + i, used[b] - n + i
            if not 0 <= int(pos[t]) < 50 or p < 0 or not 0 <= int(pt[b, p // 128]) < pages:
                continue
            page, row = int(pt[b, p // 128]), p % 128
            touched[page, row] = True
            want = rk[t].clamp(-448, 448) if kv == "e4m3" else rk[t]
            near(gk_pool[page, :, row].float(), want, mk[t], DT[kv], CHAIN)
            val = v[t].float().clamp(-448, 448).to(DT[kv]) if kv == "e4m3" else v[t]
            assert torch.equal(bits(gv_pool[page, :, row].contiguous()), bits(val.contiguous()))
    assert touched.sum() > 40
    for got, was in ((gk_pool, kp), (gv_pool, vp)):
        assert torch.equal(bits(got).transpose(1, 2)[~touched], bits(was).transpose(1, 2)[~touched])


def test_append_many_sequences(msa):
    """More sequences than one search step, of uneven lengths, an E4M3 value halfway between two codes among them."""
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 4, (700,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).to(torch.int32)
    total = int(cu[-1])
    x, q, k, v, w, table, _ = inputs(total, 2, 1, 32, "bf16")
    pos = torch.zeros(total, dtype=torch.int32)
    v[0, 0, 0] = 17.0  # between 16 and 18: to the even code, 16
    used = (lens + torch.randint(0, 120, (700,), generator=g)).to(torch.int32)
    pt = torch.randperm(700, generator=g).to(torch.int32)[:, None]
    kp, vp = (torch.zeros(700, 1, 128, 128, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    msa.msa_qk_norm_rope_append(q.to(DEV), k.to(DEV), v.to(DEV), w[0].to(DEV), w[1].to(DEV), table.to(DEV), pos.to(DEV), cu.to(DEV), kp, vp, page_table=pt.to(DEV),
                                seqused_k=used.to(DEV))
    b = torch.repeat_interleave(torch.arange(700), lens)
    row = (used[b] - lens[b]).long() + torch.arange(total) - cu[b].long()
    got = vp.cpu().float()[pt[b, 0].long(), 0, row]
    assert torch.equal(got, v[:, 0].to(torch.float8_e4m3fn).float())
    ref, mag = norm_rope(k, w[1], table, pos, False)
    near(kp.cpu().float()[pt[b, 0].long(), 0, row], ref[:, 0], mag[:, 0], torch.float8_e4m3fn, CHAIN)
    assert int((bits(vp) != 0).any(-1).sum()) <= total


def test_captured_and_on_another_stream(msa):
    x, q, k, v, w, table, pos = inputs(50, 8, 2, 64, "bf16", packed=False)
    a = (q.to(DEV), k.to(DEV), w[0].to(DEV), w[1].to(DEV), table.to(DEV), pos.to(DEV))
    want = msa.msa_qk_norm_rope(*a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = msa.msa_qk_norm_rope(*a, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    d = torch.randn_like(a[0]), torch.randn_like(a[1])
    with torch.cuda.graph(graph):
        again = msa.msa_qk_norm_rope(*a)
        grads = msa.msa_qk_norm_rope_bwd(*d, *a)
    a[0].copy_(a[0].flip(0))
    d[0].copy_(d[0].flip(0))
    graph.replay()
    want, grads_want = msa.msa_qk_norm_rope(*a), msa.msa_qk_norm_rope_bwd(*d, *a)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(again + grads, want + grads_want))


def test_rows_of_zeros_and_a_tiny_eps(msa):
    """r = eps^(-1/2) is 2^50 for a row of zeros, r^3 beyond float32: the gradient is r g all the same."""
    x, q, k, v, w, table, pos = inputs(6, 4, 2, 64, "bf16")
    eps, pos = 2.0**-100, pos.clamp(0, 49)
    x[2] = 0
    x[4, 1] = 0
    gq, gk, _ = on_gpu(x, 4, 2, True)
    dq, dk = (torch.randn(6, n, 128, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16) for n in (4, 2))
    args = gq, gk, w[0].to(DEV), w[1].to(DEV), gpu(table), pos.to(DEV)
    oq, ok = msa.msa_qk_norm_rope(*args, eps=eps)
    gdq, gdk, gwq, gwk = msa.msa_qk_norm_rope_bwd(dq.to(DEV), dk.to(DEV), *args, eps=eps)
    for y, src, wt, dx, dy, dw in ((oq, q, w[0], gdq, dq, gwq), (ok, k, w[1], gdk, dk, gwk)):
        ref, mag = norm_rope(src, wt, table, pos, False, eps)
        near(y, ref, mag, torch.bfloat16, CHAIN)
        rx, xm, rw, wm = norm_rope_bwd(src, wt, dy, table, pos, False, eps)
        near(dx, rx, xm, torch.bfloat16, CHAIN_BWD)
        assert ((dw.double().cpu() - rw).abs() <= SUMS * wm).all()
