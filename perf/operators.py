"""The operators of a serving step with drafted tokens over a paged cache, as they are measured: the per-head norm and rotation
of queries and keys (forward, appending to the cache, backward), attention of a tree of drafted tokens over listed blocks, the
acceptance of drafted rows and the forking of sequences. `own` says whose form runs: the plain one below, or the framework's."""
import math

import torch

own = False

BLK, DIM = 128, 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # One decode step of four requests: the latency of the smallest call.
        dict(name="append_decode_4", op="append", batch=4, nq_lo=1, nq_hi=1, hq=64, hkv=4, rotary=128, interleaved=False, dtype="bf16", kv="bf16", kv_hi=1024),
        # A batch of drafted trees written to an E4M3 cache, ragged, partial rotation.
        dict(name="append_drafts_e4m3", op="append", batch=128, nq_lo=4, nq_hi=32, hq=64, hkv=4, rotary=64, interleaved=False, dtype="bf16", kv="e4m3", kv_hi=1500),
        # The prefill of two long sequences out of a packed projection.
        dict(name="rope_prefill_65536", op="rope", tokens=65536, hq=32, hkv=4, rotary=128, interleaved=False, dtype="bf16"),
        # Training: the gradient of a long packed batch, and a small odd one in the other pairing and type.
        dict(name="rope_bwd_32768", op="rope_bwd", tokens=32768, hq=64, hkv=8, rotary=64, interleaved=False, dtype="bf16"),
        dict(name="rope_bwd_odd_fp16", op="rope_bwd", tokens=1037, hq=12, hkv=3, rotary=96, interleaved=True, dtype="fp16"),
        # One request's eight drafted tokens: the latency of verification for a single user.
        dict(name="tree_one_request_fp16", op="tree", batch=1, nq_lo=8, nq_hi=8, hq=32, hkv=4, topk=16, kv="fp16", kv_lo=8192, kv_hi=16384),
        # An ordinary serving batch.
        dict(name="tree_batch_32", op="tree", batch=32, nq_lo=16, nq_hi=16, hq=64, hkv=4, topk=16, kv="bf16", kv_lo=8192, kv_hi=65536),
        # A large batch of ragged trees over an E4M3 cache.
        dict(name="tree_batch_128_e4m3", op="tree", batch=128, nq_lo=8, nq_hi=32, hq=64, hkv=4, topk=16, kv="e4m3", kv_lo=8192, kv_hi=131072),
        # A drafted step's end: the drafts of every layer written, then the accepted path moved up.
        dict(name="accept_small", op="accept", batch=3, nq_lo=5, nq_hi=9, hq=8, hkv=2, rotary=128, interleaved=False, dtype="bf16", kv="bf16", kv_hi=700, layers=2),
        dict(name="accept_batch_96", op="accept", batch=96, nq_lo=8, nq_hi=24, hq=32, hkv=4, rotary=64, interleaved=False, dtype="bf16", kv="bf16", kv_hi=600, layers=6),
        # Beams or samples dropped and forked anew: tables, counts and the partial pages of every layer.
        dict(name="fork_small", op="fork", rows=8, forks=2, hkv=1, layers=2, kv_hi=900, max_pages=64, grow=5, kv="bf16"),
        dict(name="fork_batch_96", op="fork", rows=224, forks=96, hkv=4, layers=8, kv_hi=640, max_pages=1024, grow=16, kv="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rope", "rope_bwd", "tree", "accept", "fork"])
    hq, hkv = rng.choice([(64, 4), (64, 8), (32, 4), (16, 1), (12, 3), (8, 8), (40, 4), (4, 1)])
    rope = dict(hq=hq, hkv=hkv, rotary=rng.choice([32, 64, 96, 128]), interleaved=rng.random() < 0.4, dtype=rng.choice(["bf16", "fp16"]))
    lo = _spread(rng, 1, 24)
    hi = lo + rng.randint(0, 16)
    if op in ("append", "accept"):
        kv = "e4m3" if rope["dtype"] == "bf16" and rng.random() < 0.4 else rope["dtype"]
        batch = _spread(rng, 1, 96)
        c = dict(op=op, batch=batch, nq_lo=lo, nq_hi=hi, kv=kv, kv_hi=rng.randint(1, 800), **rope)
        return dict(c, layers=rng.randint(1, 6)) if op == "accept" else c
    if op in ("rope", "rope_bwd"):
        most = 65536 * 36 // (hq + hkv) // (2 if op == "rope_bwd" else 1)
        return dict(op=op, tokens=_spread(rng, 1, min(most, 100000)), **rope)
    if op == "tree":
        top = _spread(rng, 300, 60000)
        return dict(op=op, batch=_spread(rng, 1, 64), nq_lo=lo, nq_hi=hi, hq=hq, hkv=hkv, topk=rng.choice([1, 4, 8, 16, 20, 32] if hkv < 8 else [1, 4, 8, 16]),
                    kv=rng.choice(["bf16", "fp16", "e4m3"]), kv_lo=rng.randint(1, top), kv_hi=top)
    rows = _spread(rng, 2, 200)
    return dict(op=op, rows=rows, forks=rng.randint(1, max(1, rows // 2)), hkv=min(hkv, 4), layers=rng.randint(1, 6), kv_hi=rng.randint(1, 700), max_pages=rng.randint(16, 800),
                grow=rng.randint(0, 40), kv=rng.choice(["bf16", "e4m3"]))


# ------------------------------------------------------------------------------------------------------------------- the inputs
def _gens(seed):
    h, g = torch.Generator("cpu"), torch.Generator("cuda")
    h.manual_seed(int(seed) * 2 + 1)
    g.manual_seed(int(seed) * 2)
    return h, g


def _normal(g, shape, dtype):
    """Standard normal values of a type, a slab at a time."""
    x = torch.empty(shape, dtype=dtype, device="cuda")
    flat = x.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        b = min(flat.numel(), a + (1 << 28))
        flat[a:b] = torch.randn(b - a, generator=g, device="cuda").to(dtype)
    return x


def _lengths(h, n, lo, hi):
    """Lengths spread evenly over a range, in an order of the seed's: their sum is the case's."""
    at = torch.linspace(lo, hi, n, dtype=torch.float64).round().long() if n > 1 else torch.tensor([(lo + hi) // 2])
    return at[torch.randperm(n, generator=h)]


def _cu(lengths):
    return torch.cat([torch.zeros(1, dtype=torch.long), lengths.cumsum(0)])


def _rope_table(rotary, length):
    """cos and sin of each position's angles side by side, computed in 64 bits and kept in 32."""
    f = 1e4 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _weights(g, *shape):
    return 1 + 0.2 * torch.randn(*shape, generator=g, device="cuda")


def _table(h, used, total, width):
    """Page tables over one shuffled pool: each request's pages where the others' lie between, with some that no one holds."""
    pages = (used + BLK - 1) // BLK
    at = torch.arange(width)[None] < pages[:, None]
    table = torch.full((len(used), width), -1, dtype=torch.int32)
    table[at] = torch.randperm(total, generator=h)[: int(pages.sum())].to(torch.int32)
    return table


def _trees(h, nq, lines):
    """A tree of drafted tokens for each request: parents of nodes by nearness, the ancestors of each as bits, the depths."""
    b, n = len(nq), int(nq.max())
    back = torch.randint(1, 9, (b, n), generator=h)
    parent = (torch.arange(n)[None] - back).clamp(min=-1)
    parent[:, 1:] = parent[:, 1:].clamp(min=0)  # the first node is the root
    eye = torch.eye(n, dtype=torch.bool)
    up = eye[parent.clamp(min=0)] & (parent >= 0)[..., None]
    anc = eye | up
    step = up.float()
    for _ in range(max(1, n.bit_length())):
        step = (step @ step + step > 0).float()
        anc = eye | (step > 0)
    words = (n + 31) // 32
    bits = torch.zeros(b, n, words * 32, dtype=torch.long)
    bits[:, :, :n] = anc.long()
    mask = (bits.view(b, n, words, 32) << torch.arange(32)).sum(-1)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    depth = anc.sum(-1) - 1
    live = torch.arange(n)[None] < nq[:, None]
    return parent, mask[live], depth, live


def _prepare_rope(c, g, h, layers=None):
    t = c["tokens"]
    heads = c["hq"] + 2 * c["hkv"]
    s = {"op": c["op"], "hq": c["hq"], "hkv": c["hkv"], "interleaved": c["interleaved"]}
    lead = () if layers is None else (layers,)
    # A projection's output: every token's scale is its own, as in a residual stream.
    s["qkv"] = (_normal(g, lead + (t, heads, DIM), torch.float32 if t < 4096 else DTYPES[c["dtype"]]) * (0.3 + 3 * torch.rand(lead + (t, 1, 1), generator=g, device="cuda"))).to(DTYPES[c["dtype"]])
    s["wq"], s["wk"] = _weights(g, *lead, DIM), _weights(g, *lead, DIM)
    length = max(4096, t) if c["op"] in ("rope", "rope_bwd") else c["kv_hi"] + c["nq_hi"] + 8
    s["cos_sin"] = _rope_table(c["rotary"], length)
    return s, length


def prepare(case, seed):
    h, g = _gens(seed)
    c = dict(case)
    if c["op"] in ("rope", "rope_bwd"):
        s, length = _prepare_rope(c, g, h)
        cuts = torch.randint(0, c["tokens"], (1,), generator=h)  # two sequences, one after the other
        p = torch.arange(c["tokens"])
        s["positions"] = torch.where(p < cuts, p, p - cuts).to(torch.int32).cuda()
        if c["op"] == "rope_bwd":
            s["dq"], s["dk"] = _normal(g, (c["tokens"], c["hq"], DIM), DTYPES[c["dtype"]]), _normal(g, (c["tokens"], c["hkv"], DIM), DTYPES[c["dtype"]])
        return s
    if c["op"] == "fork":
        return _prepare_fork(c, g, h)
    nq = _lengths(h, c["batch"], c["nq_lo"], c["nq_hi"])
    cu = _cu(nq)
    kept = _lengths(h, c["batch"], c.get("kv_lo", 1), c["kv_hi"])
    used = kept + nq
    pages = int(((kept + c["nq_hi"] + BLK - 1) // BLK).sum())
    table = _table(h, used, pages, (c["kv_hi"] + c["nq_hi"] + BLK - 1) // BLK)
    parent, mask, depth, live = _trees(h, nq, c["batch"])
    common = {"cu": cu.to(torch.int32).cuda(), "used": used.to(torch.int32).cuda(), "table": table.cuda(), "nq_hi": c["nq_hi"]}
    if c["op"] == "tree":
        return dict(_prepare_tree(c, g, nq, used, live, pages), mask=mask.cuda(), **common)
    c["tokens"] = int(cu[-1])
    layers = c.get("layers")
    s, _ = _prepare_rope(c, g, h, layers)
    s["positions"] = ((used - nq)[:, None] + depth)[live].to(torch.int32).cuda()
    s.update(common)
    lead = (1,) if layers is None else (layers,)
    s["pools"] = _normal(g, lead + (2, pages, c["hkv"], BLK, DIM), DTYPES[c["kv"]])
    s["q_out"] = torch.empty(lead + (c["tokens"], c["hq"], DIM), dtype=DTYPES[c["dtype"]], device="cuda")
    if c["op"] == "accept":
        # The accepted path: from the root down to a node drawn near the front.
        n = int(nq.max())
        end = (torch.rand(c["batch"], generator=h) ** 2 * nq).long()
        on = torch.zeros(c["batch"], n, dtype=torch.bool)
        for _ in range(n):
            on |= torch.nn.functional.one_hot(end.clamp(min=0), n).bool() & (end >= 0)[:, None]
            end = torch.where(end >= 0, parent.gather(1, end.clamp(min=0)[:, None])[:, 0], end)
        s["path"] = torch.where(on, torch.arange(n)[None], n).sort(1).values.to(torch.int32).cuda()
        s["path_len"] = on.sum(1).to(torch.int32).cuda()
    return s


def _prepare_tree(c, g, nq, used, live, pages):
    """Block lists whose tokens agree for the most part, as drafted tokens of one text do: every token of a request takes the first
    block, the blocks that hold the drafts and others of a common set half as large again as a list."""
    kv = DTYPES[c["kv"]]
    qt = torch.float16 if c["kv"] == "fp16" else torch.bfloat16
    b, n, hkv, topk = c["batch"], int(nq.max()), c["hkv"], c["topk"]
    blocks = ((used + BLK - 1) // BLK).cuda()
    width = int(blocks.max())
    col = torch.arange(width, device="cuda")
    seen = col < blocks[:, None]
    forced = seen & ((col == 0) | (col >= ((used - nq).cuda() // BLK)[:, None]))
    key = torch.rand(hkv, b, width, generator=g, device="cuda") + 2 * forced
    key = torch.where(seen, key, -1.0)
    common = key.topk(min(width, topk + (topk + 1) // 2), dim=-1)
    kc = torch.where(common.values < 0, -1.0, torch.where(common.values >= 2, 2.0, 1.0))
    pick = torch.where(kc[:, :, None] < 0, -1.0, kc[:, :, None] + torch.rand(hkv, b, n, kc.shape[-1], generator=g, device="cuda"))
    top = pick.topk(min(topk, kc.shape[-1]), dim=-1)
    ids = common.indices[:, :, None].expand(-1, -1, n, -1).gather(-1, top.indices)
    ids = torch.where(top.values < 0, 1 << 30, ids).sort(-1).values
    ids = torch.where(ids == 1 << 30, -1, ids).to(torch.int32)
    lists = torch.full((hkv, int(nq.sum()), topk), -1, dtype=torch.int32, device="cuda")
    lists[:, :, : ids.shape[-1]] = ids[:, live.cuda()]
    q = _normal(g, (int(nq.sum()), c["hq"], DIM), qt)
    return {"op": "tree", "q": q, "k": _normal(g, (pages, hkv, BLK, DIM), kv), "v": _normal(g, (pages, hkv, BLK, DIM), kv), "lists": lists}


def _prepare_fork(c, g, h):
    """Rows of a batch with their pages and counts; the last `forks` of them are dropped and forked anew from others, in each pass."""
    n = c["forks"]
    used = _lengths(h, c["rows"], 1, c["kv_hi"])
    pages = int(((used + BLK - 1) // BLK).sum()) + n * (2 + (c["kv_hi"] + c["grow"] + BLK - 1) // BLK)
    table = _table(h, used, pages, c["max_pages"])
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    src = torch.randint(0, c["rows"] - n, (n,), generator=h) if c["rows"] > n else torch.zeros(n, dtype=torch.long)
    dst = torch.arange(c["rows"] - n, c["rows"])
    return {"op": "fork", "pools": _normal(g, (2 * c["layers"], pages, c["hkv"], BLK, DIM), DTYPES[c["kv"]]), "table": table.cuda(), "used": used.to(torch.int32).cuda(),
            "refs": refs.cuda(), "src": src.to(torch.int32).cuda(), "dst": dst.to(torch.int32).cuda(), "longer": (used[src] + c["grow"]).to(torch.int32).cuda()}


# ------------------------------------------------------------------------------------------------------------------- plain forms
def _split(s):
    return s["qkv"].narrow(-2, 0, s["hq"]), s["qkv"].narrow(-2, s["hq"], s["hkv"]), s["qkv"].narrow(-2, s["hq"] + s["hkv"], s["hkv"])


def _pairs(x, half, interleaved):
    return (x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]) if interleaved else (x[..., :half], x[..., half : 2 * half])


def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    a, b = _pairs(x, half, interleaved)
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * half :]], -1)


def _angles(s):
    row = s["cos_sin"][s["positions"].long()][:, None]
    return row.chunk(2, -1)


def _inverse(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _norm_rope(x, w, cos, sin, interleaved):
    x = x.float()
    return _rotate(x * _inverse(x) * w, cos, sin, interleaved)


def _norm_rope_bwd(x, w, d, cos, sin, interleaved):
    f = x.float()
    r = _inverse(f)
    u = _rotate(d.float(), cos, -sin, interleaved)
    dw = (u * f * r).sum((0, 1))
    a = u * w
    return (r * (a - f * r.square() * (a * f).mean(-1, keepdim=True))).to(x.dtype), dw


def _held(x, dtype):
    return x.clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _bits(x):
    return x.view(torch.uint8 if x.element_size() == 1 else torch.int16)


def _requests(s, tokens):
    """Of each token: its request and its place in the cache."""
    cu = s["cu"].long()
    at = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cu[1:], at, right=True)
    return b, s["used"].long()[b] - cu[b + 1] + at


def _append(s):
    q, k, v = _split(s)
    layered = q.dim() == 4
    cos, sin = _angles(s)
    shape = (lambda w: w[:, None, None]) if layered else (lambda w: w)
    s["q_out"].copy_(_norm_rope(q, shape(s["wq"]), cos, sin, s["interleaved"]).view(s["q_out"].shape))
    kv = torch.stack([_norm_rope(k, shape(s["wk"]), cos, sin, s["interleaved"]), v.float()], -4).view(-1, *k.shape[-3:])
    pools = s["pools"].flatten(0, 1)
    b, pos = _requests(s, q.shape[-3])
    page = s["table"].long()[b, pos // BLK]
    _bits(pools)[:, page, :, pos % BLK] = _bits(_held(kv, pools.dtype)).transpose(0, 1)
    return {"q": s["q_out"], "pools": s["pools"]}


def _tree(s):
    q, lists, dev = s["q"], s["lists"].long(), "cuda"
    t, hq, _ = q.shape
    hkv, _, topk = lists.shape
    b, pos = _requests(s, t)
    cu, used = s["cu"].long(), s["used"].long()
    first = (used - (cu[1:] - cu[:-1]))[b]
    page = s["table"].long()[b[None, :, None], lists.clamp(min=0)].clamp(min=0)
    head = torch.arange(hkv, device=dev)[:, None, None]
    key = lists[..., None] * BLK + torch.arange(BLK, device=dev)
    node = key - first[None, :, None, None]
    words = s["mask"].long().expand(hkv, -1, -1)
    word = words.gather(2, (node >> 5).clamp(0, words.shape[2] - 1).view(hkv, t, -1)).view(node.shape)
    see = (lists >= 0)[..., None] & (key < used[b][None, :, None, None]) & ((node < 0) | ((word >> (node & 31)) & 1).bool())
    qh = q.float().view(t, hkv, 1, hq // hkv, DIM).transpose(0, 1)
    x = (qh @ s["k"][page, head].float().transpose(-1, -2)) * DIM**-0.5
    x = x.masked_fill(~see[:, :, :, None], -math.inf)
    m = x.amax((2, 4), keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = e.sum((2, 4))
    o = (e @ s["v"][page, head].float()).sum(2) / torch.where(l > 0, l, 1.0)[..., None]
    lse = m[:, :, 0, :, 0] + torch.log(l)
    return {"out": o.transpose(0, 1).reshape(t, hq, DIM).to(q.dtype), "lse": lse.transpose(0, 1).reshape(t, hq)}


def _accept(s):
    _append(s)
    pools = _bits(s["pools"].flatten(0, 1))
    cu, used, path = s["cu"].long(), s["used"].long(), s["path"].long()
    first = (used - (cu[1:] - cu[:-1]))[:, None]
    j = torch.arange(path.shape[1], device="cuda")
    live = j < s["path_len"][:, None]
    src, dst = first + torch.where(live, path, path[:, :1]), first + torch.where(live, j, 0)
    table = s["table"].long()
    pools[:, table.gather(1, dst // BLK), :, dst % BLK] = pools[:, table.gather(1, src // BLK), :, src % BLK].clone()
    return {"q": s["q_out"], "pools": s["pools"], "used": (first[:, 0] + s["path_len"]).to(torch.int32)}


def _count(refs, pages, by):
    refs.scatter_add_(0, pages.clamp(min=0).reshape(-1), by.reshape(-1).to(torch.int32))


def _fork(s):
    table, used, refs, pools = s["table"], s["used"], s["refs"], _bits(s["pools"])
    src, dst = s["src"].long(), s["dst"].long()
    # Dropped: the rows' pages lose a holder.
    old = table[dst].long()
    _count(refs, old, -(old >= 0).int())
    # Forked: whole pages are shared, a begun one is copied to a free one.
    ours, length = table[src].long(), used[src].long()
    at, whole = torch.arange(table.shape[1], device="cuda"), (length // BLK)[:, None]
    shared, begun = at < whole, length % BLK > 0
    _count(refs, ours, shared)
    free = torch.argsort((refs != 0).int(), stable=True)
    page = ours.gather(1, whole.clamp(max=table.shape[1] - 1))[:, 0].clamp(min=0)
    new = torch.where(begun, free[(begun.cumsum(0) - 1).clamp(min=0)], page)
    _count(refs, new, begun)
    pools[:, new] = pools[:, page]
    ours = torch.where(shared, ours, torch.where((at == whole) & begun[:, None], new[:, None], -1))
    # Extended: room for the next tokens.
    want = (at < ((s["longer"].long() + BLK - 1) // BLK)[:, None]) & (ours < 0)
    free = torch.argsort((refs != 0).int(), stable=True)
    fresh = free[(want.view(-1).cumsum(0) - 1).clamp(0, free.numel() - 1)].view(want.shape)
    _count(refs, fresh, want)
    table[dst] = torch.where(want, fresh, ours).to(torch.int32)
    used[dst] = s["longer"]
    done = torch.zeros(2, len(dst), dtype=torch.int32, device="cuda")
    return {"table": table, "used": used, "refs": refs, "pools": pools, "forked": done[0], "extended": done[1]}


# ------------------------------------------------------------------------------------------------------------------- the passes
def _own(s):
    import block_sparse_top_msa_gb300 as msa

    rope = {"eps": EPS, "interleaved": s.get("interleaved", False)}
    if s["op"] == "rope":
        q, k, _ = _split(s)
        return dict(zip("qk", msa.msa_qk_norm_rope(q, k, s["wq"], s["wk"], s["cos_sin"], s["positions"], **rope)))
    if s["op"] == "rope_bwd":
        q, k, _ = _split(s)
        return dict(zip(("q", "k", "wq", "wk"), msa.msa_qk_norm_rope_bwd(s["dq"], s["dk"], q, k, s["wq"], s["wk"], s["cos_sin"], s["positions"], **rope)))
    if s["op"] == "tree":
        return dict(zip(("out", "lse"), msa.msa_tree_attention(s["q"], s["k"], s["v"], s["lists"], s["cu"], s["mask"], page_table=s["table"], seqused_k=s["used"], max_seqlen_q=min(s["nq_hi"], 32 * s["mask"].shape[1]),
                                                              return_softmax_lse=True)))
    if s["op"] == "fork":
        msa.msa_cache_free(s["table"], s["used"], s["refs"], s["dst"])
        forked = msa.msa_cache_fork(s["pools"], s["table"], s["used"], s["refs"], s["src"], s["dst"])
        extended = msa.msa_cache_extend(s["table"], s["used"], s["refs"], s["dst"], s["longer"])
        return {"table": s["table"], "used": s["used"], "refs": s["refs"], "pools": _bits(s["pools"]), "forked": forked, "extended": extended}

    def append(q, k, v, wq, wk, pools, q_out):
        msa.msa_qk_norm_rope_append(q, k, v, wq, wk, s["cos_sin"], s["positions"], s["cu"], pools[0], pools[1], page_table=s["table"], seqused_k=s["used"], q_out=q_out, **rope)

    if s["op"] == "append":
        append(*_split(s), s["wq"], s["wk"], s["pools"][0], s["q_out"][0])
        return {"q": s["q_out"], "pools": s["pools"]}
    list(map(append, *_split(s), s["wq"], s["wk"], s["pools"], s["q_out"]))
    used = msa.msa_cache_accept(s["pools"].flatten(0, 1), s["table"], s["used"], s["cu"], s["path"], s["path_len"])
    return {"q": s["q_out"], "pools": s["pools"], "used": used}


def run(state):
    if own:
        return _own(state)
    s = state
    if s["op"] == "rope":
        q, k, _ = _split(s)
        cos, sin = _angles(s)
        return {"q": _norm_rope(q, s["wq"], cos, sin, s["interleaved"]).to(q.dtype), "k": _norm_rope(k, s["wk"], cos, sin, s["interleaved"]).to(k.dtype)}
    if s["op"] == "rope_bwd":
        q, k, _ = _split(s)
        cos, sin = _angles(s)
        (dq, dwq), (dk, dwk) = _norm_rope_bwd(q, s["wq"], s["dq"], cos, sin, s["interleaved"]), _norm_rope_bwd(k, s["wk"], s["dk"], cos, sin, s["interleaved"])
        return {"q": dq, "k": dk, "wq": dwq, "wk": dwk}
    return {"append": _append, "tree": _tree, "accept": _accept, "fork": _fork}[s["op"]](s)


# ------------------------------------------------------------------------------------------------------------------- work
def _mean(c):
    return (c["nq_lo"] + c["nq_hi"]) / 2 * c["batch"]


def work(case):
    c = case
    if c["op"] == "fork":
        pages = c["forks"] * (1 - 1 / BLK)
        size = 2 if c["kv"] == "bf16" else 1
        copied = 2 * pages * 2 * c["layers"] * c["hkv"] * BLK * DIM * size
        return {"bytes": copied + 4 * (3 * c["forks"] * c["max_pages"] + c["rows"]), "flops": 0}
    if c["op"] == "tree":
        t, size = _mean(c), 1 if c["kv"] == "e4m3" else 2
        lists = [min(c["topk"], math.ceil(x / BLK)) for x in range(c["kv_lo"], c["kv_hi"] + 1, max(1, (c["kv_hi"] - c["kv_lo"]) // 64))]
        each = sum(lists) / len(lists)
        union = min(1.5 * c["topk"], math.ceil(c["kv_hi"] / BLK)) * (1 - (1 - each / max(each, 1.5 * c["topk"])) ** (t / c["batch"]))
        seen = max(each, union) * c["batch"] * c["hkv"] * BLK
        return {"bytes": 2 * seen * DIM * size + t * c["hq"] * (4 * DIM + 4), "flops": 4 * t * c["hq"] * each * BLK * DIM}
    t, rows = c.get("tokens") or _mean(c), c["hq"] + c["hkv"]
    table = t * c["rotary"] * 4
    if c["op"] == "rope":
        return {"bytes": t * rows * DIM * 4 + table, "flops": 7 * t * rows * DIM}
    if c["op"] == "rope_bwd":
        return {"bytes": t * rows * DIM * 6 + table, "flops": 14 * t * rows * DIM}
    size = 1 if c["kv"] == "e4m3" else 2
    layer = t * (c["hq"] * DIM * 4 + 2 * c["hkv"] * DIM * (2 + size)) + table
    moved = 4 * c["batch"] * 2 * 2 * c["hkv"] * DIM * size if c["op"] == "accept" else 0
    return {"bytes": c.get("layers", 1) * (layer + moved), "flops": c.get("layers", 1) * 7 * t * rows * DIM}


# ------------------------------------------------------------------------------------------------------------------- 64 bits
def _exact_rope(x, w, turn, interleaved):
    """The same rotation as products of complex numbers."""
    x = x.double()
    n = x / torch.sqrt((x * x).sum(-1, keepdim=True) / DIM + EPS) * w.double()
    r = 2 * turn.shape[-1]
    z = n[..., :r].unflatten(-1, (-1, 2)) if interleaved else n[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, n[..., r:]], -1)


def _turns(s):
    c, n = s["cos_sin"].double()[s["positions"].long()].chunk(2, -1)
    return torch.complex(c, n)[:, None]


def _exact_cache(s, c):
    """Queries, pools and lengths after the drafts were appended and, for an accepted path, moved: each layer, request and node by itself."""
    turn, pools, qs = _turns(s), s["pools"].double(), []
    q, k, v = (x if x.dim() == 4 else x[None] for x in _split(s))
    wq, wk = (x if x.dim() == 2 else x[None] for x in (s["wq"], s["wk"]))
    cu, used, table = s["cu"].tolist(), s["used"].tolist(), s["table"].tolist()
    token, page, row = [], [], []
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        path = s["path"][b, : int(s["path_len"][b])].tolist() if "path" in s else []
        for j in range(hi - lo):
            pos = used[b] - (hi - lo) + j
            token.append(lo + (path[j] if j < len(path) else j))
            page.append(table[b][pos // BLK])
            row.append(pos % BLK)
    token, page, row = (torch.tensor(x, device="cuda") for x in (token, page, row))
    for i in range(q.shape[0]):
        qs.append(_exact_rope(q[i], wq[i], turn, s["interleaved"]))
        pools[i, 0][page, :, row] = _exact_rope(k[i], wk[i], turn, s["interleaved"])[token]
        pools[i, 1][page, :, row] = v[i].double()[token]
    if c["kv"] == "e4m3":
        pools.clamp_(-448, 448)
    return {"q": torch.stack(qs), "pools": pools, **({"used": None} if "path" in s else {})}


def _exact_tree(s):
    """Each request by itself, its tokens' keys one after the other."""
    cu, used = s["cu"].tolist(), s["used"].tolist()
    hkv, _, topk = s["lists"].shape
    t, hq, _ = s["q"].shape
    out, lse = torch.zeros(t, hq, DIM, dtype=torch.float64, device="cuda"), torch.full((t, hq), -math.inf, dtype=torch.float64, device="cuda")
    heads = torch.arange(hkv, device="cuda")[:, None]
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        first = used[b] - (hi - lo)
        for i in range(lo, hi):
            ids = s["lists"][:, i].long()
            page = s["table"][b].long()[ids.clamp(min=0)].clamp(min=0)
            keys = (ids[..., None] * BLK + torch.arange(BLK, device="cuda")).flatten(1)
            node = keys - first
            bit = torch.zeros(32 * s["mask"].shape[1], dtype=torch.bool, device="cuda")
            bit[:] = ((s["mask"][i].long()[:, None] >> torch.arange(32, device="cuda")) & 1).flatten().bool()
            see = (ids >= 0).repeat_interleave(BLK, 1) & (keys < used[b]) & ((node < 0) | bit[node.clamp(0, bit.numel() - 1)])
            k, v = (s[x][page, heads].double().flatten(1, 2) for x in "kv")
            x = s["q"][i].double().view(hkv, -1, DIM) @ k.transpose(1, 2) / math.sqrt(DIM)
            x = x.masked_fill(~see[:, None], -math.inf)
            z = torch.logsumexp(x, -1, keepdim=True)
            out[i] = (torch.exp(x - z).nan_to_num() @ v).view(hq, DIM)
            lse[i] = z.view(hq)
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "fork":
        return None  # copies and whole numbers
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] in ("append", "accept"):
        return _exact_cache(s, case)
    turn = _turns(s)
    q, k, _ = _split(s)
    if case["op"] == "rope":
        return {"q": _exact_rope(q, s["wq"], turn, s["interleaved"]), "k": _exact_rope(k, s["wk"], turn, s["interleaved"])}
    got = {}
    for name, x, w, d in (("q", q, s["wq"], s["dq"]), ("k", k, s["wk"], s["dk"])):
        w = w.double().requires_grad_()
        dx, dw = torch.empty(x.shape, dtype=torch.float64, device="cuda"), 0
        for a in range(0, x.shape[0], 8192):
            part = x[a : a + 8192].double().requires_grad_()
            gx, gw = torch.autograd.grad(_exact_rope(part, w, turn[a : a + 8192], s["interleaved"]), (part, w), d[a : a + 8192].double())
            dx[a : a + 8192], dw = gx, dw + gw
        got[name], got["w" + name] = dx, dw
    return got
