"""The operators of a serving step whose requests are samples of shared prompts, as they are measured: the step's tables built from
request lengths, attention that computes a shared prefix once for all, sampling from given random numbers, and the path that the
samples take through a tree of drafts. `own` says whose form runs: the plain one below, or the framework's."""
import math

import torch

own = False

BLK, DIM = 128, 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # A decode step's tables: the latency of the smallest call.
        dict(name="tables_decode_16", op="tables", rows=64, batch=16, group=4, nq_lo=1, nq_hi=1, kv_hi=6000, max_pages=64),
        # Many ragged requests of a large cache, some padded.
        dict(name="tables_batch_2048", op="tables", rows=4096, batch=2048, group=16, nq_lo=1, nq_hi=9, kv_hi=40000, max_pages=1024),
        # Two samples of a short prompt, one token each: latency.
        dict(name="attend_pair_fp16", op="attend", groups=1, group=2, nq_lo=1, nq_hi=1, hq=32, hkv=4, kv="fp16", prompt_lo=1300, prompt_hi=1300, own_hi=200),
        # Eight samples of a long prompt: the prefix fills one tile of query rows.
        dict(name="attend_8_samples", op="attend", groups=1, group=8, nq_lo=1, nq_hi=1, hq=64, hkv=4, kv="bf16", prompt_lo=32768, prompt_hi=32768, own_hi=700),
        # Many samples with drafted tokens over one prompt: products bound it.
        dict(name="attend_drafts_64", op="attend", groups=1, group=64, nq_lo=4, nq_hi=12, hq=64, hkv=4, kv="bf16", prompt_lo=32000, prompt_hi=32000, own_hi=1000),
        # Several prompts with many samples each, one token a request, an E4M3 cache.
        dict(name="attend_prompts_128_e4m3", op="attend", groups=4, group=32, nq_lo=1, nq_hi=1, hq=64, hkv=4, kv="e4m3", prompt_lo=8192, prompt_hi=32768, own_hi=2000),
        # Requests that share nothing: the whole cache is read, memory bounds it.
        dict(name="attend_apart_32", op="attend", groups=32, group=1, nq_lo=1, nq_hi=1, hq=64, hkv=4, kv="bf16", prompt_lo=4096, prompt_hi=65536, own_hi=1),
        # One user's next token.
        dict(name="sample_one", op="sample", rows=1, vocab=131072, dtype="fp32", cuts="kpm", spread=2.5),
        # An ordinary batch with each request's own settings, some greedy, some with masked tokens.
        dict(name="sample_batch_64", op="sample", rows=64, vocab=131072, dtype="fp32", cuts="kp", spread=2.5),
        # Every node of a batch of draft trees, 16-bit logits of an odd vocabulary, no bound on the count.
        dict(name="sample_nodes_512_bf16", op="sample", rows=512, vocab=200019, dtype="bf16", cuts="pm", spread=2.0),
        # The accepted path of a few trees, and of a large batch.
        dict(name="path_8", op="path", batch=8, nq_lo=8, nq_hi=8),
        dict(name="path_batch_256", op="path", batch=256, nq_lo=8, nq_hi=64),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "attend", "attend", "sample", "sample", "path"])
    lo = _spread(rng, 1, 16)
    hi = lo + rng.randint(0, 12)
    if op == "tables":
        batch = _spread(rng, 1, 2048)
        return dict(op=op, rows=batch + _spread(rng, 1, 2000), batch=batch, group=_spread(rng, 1, 40), nq_lo=lo, nq_hi=hi, kv_hi=_spread(rng, 1, 40000), max_pages=rng.randint(315, 1000))
    if op == "path":
        return dict(op=op, batch=_spread(rng, 1, 256), nq_lo=lo, nq_hi=hi + rng.randint(0, 36))
    if op == "sample":
        vocab = _spread(rng, 300, 200019)
        return dict(op=op, rows=_spread(rng, 1, min(512, 50_000_000 // vocab + 1)), vocab=vocab, dtype=rng.choice(["fp32", "bf16", "fp16"]), cuts=rng.choice(["", "k", "p", "m", "kp", "kpm", "pm"]),
                    spread=rng.choice([0.3, 1.0, 2.0, 2.5, 4.0]))
    hq, hkv = rng.choice([(64, 4), (64, 8), (32, 4), (16, 1), (12, 3), (8, 8), (40, 4), (4, 1), (96, 1)])
    group, nq = _spread(rng, 1, 48), _spread(rng, 1, 8)
    groups = _spread(rng, 1, max(1, 64 // group))
    most = min(4_000_000 // (groups * group * hkv), 1_000_000_000 // (groups * group * (nq + 2) * hq))
    top = _spread(rng, 200, max(201, min(65536, most)))
    return dict(op=op, groups=groups, group=group, nq_lo=nq, nq_hi=nq + rng.randint(0, 4), hq=hq, hkv=hkv, kv=rng.choice(["bf16", "fp16", "e4m3"]), prompt_lo=rng.randint(1, top), prompt_hi=top,
                own_hi=_spread(rng, 1, 1500))


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


def _ints(x):
    return x.to(torch.int32).cuda()


def _blocks(n):
    return (n + BLK - 1) // BLK


def _forked(h, prompts, group, lengths, width):
    """Page tables of the samples of some prompts, forked and grown: whole pages of a prompt are its samples' in common, the others
    each one's own. Returns the table (a prompt's samples side by side) and the number of pages."""
    shared = prompts // BLK
    n = len(prompts) * group
    col = torch.arange(width)[None]
    common = torch.cat([torch.zeros(1, dtype=torch.long), shared.cumsum(0)])
    rest = _blocks(lengths) - shared.repeat_interleave(group)
    own_at = common[-1] + torch.cat([torch.zeros(1, dtype=torch.long), rest.cumsum(0)])
    s = shared.repeat_interleave(group)[:, None]
    table = torch.where(col < s, common[:-1].repeat_interleave(group)[:, None] + col, own_at[:n, None] + col - s)
    pages = int(own_at[-1])
    table = torch.where(col < _blocks(lengths)[:, None], torch.randperm(pages, generator=h)[table.clamp(0, pages - 1)], -1)
    return table, pages


def _prepare_tables(c, h):
    """A cache of many rows; the step's requests lie anywhere among them, a few padded (row -1)."""
    n = -(-c["rows"] // c["group"])
    prompts = torch.randint(1, max(2, c["kv_hi"] * 3 // 4), (n,), generator=h)
    lengths = (prompts.repeat_interleave(c["group"]) + c["nq_hi"] + torch.randint(0, max(1, c["kv_hi"] // 4), (n * c["group"],), generator=h)).clamp(max=c["max_pages"] * BLK)
    table, pages = _forked(h, prompts, c["group"], lengths, c["max_pages"])
    rows = torch.randperm(n * c["group"], generator=h)[: c["rows"]].sort().values
    order = torch.randperm(len(rows), generator=h)
    pick = order[: c["batch"]]
    at = torch.randint(0, c["batch"], (c["batch"] // 50,), generator=h)
    pick[at] = -1
    nq = _lengths(h, c["batch"], c["nq_lo"], c["nq_hi"])
    return {"op": "tables", "table": _ints(table[rows]), "used": _ints(lengths[rows]), "rows": _ints(pick), "nq": _ints(nq), "total": int(nq.sum()), "pages": pages}


def _prepare_attend(c, g, h):
    kv, qt = DTYPES[c["kv"]], torch.float16 if c["kv"] == "fp16" else torch.bfloat16
    b = c["groups"] * c["group"]
    nq = _lengths(h, b, c["nq_lo"], c["nq_hi"])
    prompts = _lengths(h, c["groups"], c["prompt_lo"], c["prompt_hi"])
    used = prompts.repeat_interleave(c["group"]) + _lengths(h, b, 0, c["own_hi"] - 1) + nq
    table, pages = _forked(h, prompts, c["group"], used, int(_blocks(used.max())))
    at = torch.randperm(b, generator=h)  # the request that each sample is: a prompt's are anywhere in the batch
    s = {"op": "attend", "nq_hi": c["nq_hi"], "cu": None, "groups": None}
    place = lambda x: torch.empty_like(x).index_copy_(0, at, x)  # noqa: E731
    cu = _cu(place(nq))
    s["cu"], s["used"], s["table"] = _ints(cu), _ints(place(used)), _ints(place(table))
    s["q"] = _normal(g, (int(cu[-1]), c["hq"], DIM), qt)
    s["k"], s["v"] = _normal(g, (pages, c["hkv"], BLK, DIM), kv), _normal(g, (pages, c["hkv"], BLK, DIM), kv)
    if c["group"] > 1:
        ends = torch.full((b + 1,), b)
        ends[: c["groups"]] = torch.arange(c["groups"]) * c["group"]
        blocks = torch.zeros(b, dtype=torch.long)
        blocks[: c["groups"]] = prompts // BLK
        s["groups"] = {"group_rows": _ints(at.view(c["groups"], -1).sort(1).values.view(-1)), "cu_groups": _ints(ends), "group_blocks": _ints(blocks)}
    s["members"] = c["group"]
    s["rest"] = int((_blocks(used) - (prompts // BLK).repeat_interleave(c["group"])).max()) if c["group"] > 1 else table.shape[1]
    return s


def _prepare_sample(c, g, h):
    """Logits as a model's: a bulk, and some tokens that stand out of it; a third of the rows has tokens masked by -inf. Each row has
    its own temperature (0 picks the largest) and cuts."""
    n, v = c["rows"], c["vocab"]
    x = c["spread"] * torch.randn(n, v, generator=g, device="cuda")
    peaks = torch.randint(0, v, (n, 12), generator=g, device="cuda")
    x.scatter_add_(1, peaks, 3 * c["spread"] * torch.rand(n, 12, generator=g, device="cuda"))
    masked = torch.rand(n, generator=h) < 1 / 3
    x.masked_fill_((torch.rand(n, v, generator=g, device="cuda") < 0.3) & masked.cuda()[:, None], -math.inf)
    t = torch.tensor([0.7, 1.0, 1.0, 1.3, 0.0])[torch.randint(0, 5, (n,), generator=h)] if n > 1 else torch.full((1,), 0.8)
    s = {"op": "sample", "logits": x.to(DTYPES[c["dtype"]]), "u": torch.rand(n, generator=h).cuda(), "temperature": t.cuda(), "top_k": None, "top_p": None, "min_p": None}
    if "k" in c["cuts"]:
        s["top_k"] = _ints(torch.tensor([0, 1, 20, 50, 50, 1000])[torch.randint(0, 6, (n,), generator=h)] if n > 1 else torch.full((1,), 50))
    if "p" in c["cuts"]:
        s["top_p"] = torch.tensor([0.5, 0.9, 0.95, 0.95, 0.99, 1.0])[torch.randint(0, 6, (n,), generator=h)].cuda()
    if "m" in c["cuts"]:
        s["min_p"] = torch.tensor([0.0, 0.02, 0.05, 0.1])[torch.randint(0, 4, (n,), generator=h)].cuda()
    return s


def _prepare_path(c, h):
    """Trees of drafted tokens and what the model made of each node: most often one of the node's children."""
    nq = _lengths(h, c["batch"], c["nq_lo"], c["nq_hi"])
    b, n = c["batch"], int(nq.max())
    back = torch.randint(1, 5, (b, n), generator=h)
    parent = (torch.arange(n)[None] - back).clamp(min=-1)
    parent[:, 1:] = parent[:, 1:].clamp(min=0)  # the first node is the root
    eye = torch.eye(n, dtype=torch.bool)
    step = (eye[parent.clamp(min=0)] & (parent >= 0)[..., None]).float()
    for _ in range(max(1, n.bit_length())):
        step = (step @ step + step > 0).float()
    words = (n + 31) // 32
    bits = torch.zeros(b, n, words * 32, dtype=torch.long)
    bits[:, :, :n] = (eye | (step > 0)).long()
    mask = (bits.view(b, n, words, 32) << torch.arange(32)).sum(-1)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    drafts = torch.randint(0, 40, (b, n), generator=h)
    child = (torch.arange(n)[None] + torch.randint(1, 5, (b, n), generator=h)).clamp(max=n - 1)
    follows = (parent.gather(1, child) == torch.arange(n)[None]) & (torch.rand(b, n, generator=h) < 0.9)
    sampled = torch.where(follows, drafts.gather(1, child), torch.randint(0, 40, (b, n), generator=h))
    live = torch.arange(n)[None] < nq[:, None]
    return {"op": "path", "sampled": _ints(sampled[live]), "drafts": _ints(drafts[live]), "mask": mask[live].cuda(), "cu": _ints(_cu(nq)), "most": n}


def prepare(case, seed):
    h, g = _gens(seed)
    c = dict(case)
    if c["op"] == "tables":
        return _prepare_tables(c, h)
    if c["op"] == "attend":
        return _prepare_attend(c, g, h)
    return _prepare_sample(c, g, h) if c["op"] == "sample" else _prepare_path(c, h)


# ------------------------------------------------------------------------------------------------------------------- plain forms
def _tables(s):
    rows, dev = s["rows"].long(), "cuda"
    b, width = len(rows), s["table"].shape[1]
    real = (rows >= 0) & (rows < s["table"].shape[0])
    used = torch.where(real, s["used"].long()[rows.clamp(min=0)], 0)
    nq = torch.where(real, torch.minimum(s["nq"].long().clamp(min=0), used), 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), nq.cumsum(0)])
    col = torch.arange(width, device=dev)
    table = s["table"].long()[rows.clamp(min=0)]
    table = torch.where((col < _blocks(used)[:, None]) & (table < s["pages"]), table, -1)
    t = torch.arange(s["total"], device=dev)
    req = torch.searchsorted(cu[1:], t, right=True)
    live = t < cu[-1]
    req = req.clamp(max=b - 1)
    pos = used[req] - cu[req + 1] + t
    page = table[req, (pos // BLK).clamp(0, width - 1)]
    slots = torch.where(live & (page >= 0), page * BLK + pos % BLK, -1)
    # Groups: requests with the same first page, led by the first of them.
    joins = (table[:, 0] >= 0) & (nq > 0)
    same = (table[:, 0][:, None] == table[:, 0]) & joins[:, None] & joins
    leader = torch.where(joins, same.int().argmax(1), torch.arange(b, device=dev))
    order = torch.argsort(leader, stable=True)
    heads = leader == torch.arange(b, device=dev)
    number = heads.cumsum(0) - 1  # of each leader's group
    group = number[leader]
    size = torch.zeros(b, dtype=torch.long, device=dev).scatter_add_(0, group, torch.ones_like(group))
    cu_groups = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), size.cumsum(0)])
    alike = ((table == table[leader]) & (table >= 0)).long().cumprod(1).sum(1)
    most = torch.minimum(alike, (used - nq) // BLK)
    blocks = torch.full((b,), width, dtype=torch.long, device=dev).scatter_reduce_(0, group, most, "amin")
    blocks = torch.where(size > 1, blocks, 0)
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"cu": i32(cu), "used": i32(used), "table": i32(table), "token_rows": i32(torch.where(live, req, -1)), "positions": i32(torch.where(live, pos, -1)), "slots": slots,
            "group_rows": i32(order), "cu_groups": i32(cu_groups), "group_blocks": i32(blocks)}


def _part(q, k, v, see):
    """Running parts of a softmax: q (n, hkv, rows, DIM), k and v (n, keys, hkv, DIM), see broadcast to (n, hkv, rows, keys)."""
    x = (q @ k.permute(0, 2, 3, 1)) * DIM**-0.5
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    return m, e.sum(-1, keepdim=True), e @ v.transpose(1, 2)


def _keys(pool, pages):
    """(n, blocks) pages as (n, keys, hkv, DIM) in 32 bits."""
    return pool[pages.clamp(min=0)].float().transpose(2, 3).flatten(1, 2)


def _attend(s):
    q, cu, used, table, dev = s["q"], s["cu"].long(), s["used"].long(), s["table"].long(), "cuda"
    t, hq, _ = q.shape
    hkv, b = s["k"].shape[1], len(used)
    ratio = hq // hkv
    nq = cu[1:] - cu[:-1]
    i = torch.arange(s["nq_hi"], device=dev)
    token = torch.where(i < nq[:, None], cu[:-1, None] + i, t)  # (b, nq_hi), t where there is none
    qp = torch.cat([q.float(), torch.zeros(1, hq, DIM, device=dev)])
    shaped = lambda ids: qp[ids].view(ids.shape[0], ids.shape[1], hkv, ratio, DIM).transpose(1, 2).flatten(2, 3)  # noqa: E731
    skip = torch.zeros(b, dtype=torch.long, device=dev)  # blocks of each request that its group attends
    if s["groups"] is not None:
        n = b // s["members"]
        rows, blocks = s["groups"]["group_rows"].long().view(n, -1), s["groups"]["group_blocks"].long()[:n]
        skip[rows] = blocks[:, None]
        width = int(table.shape[1])
        ids = token[rows].flatten(1)
        key = torch.arange(width * BLK, device=dev)
        first = table[rows[:, 0]]
        pm, pl, po = _part(shaped(ids), _keys(s["k"], first), _keys(s["v"], first), (key < blocks[:, None] * BLK)[:, None, None])
        back = lambda x: x.unflatten(2, (-1, s["nq_hi"] * ratio)).transpose(1, 2).flatten(0, 1)  # noqa: E731
        turn = torch.argsort(rows.view(-1))
        pm, pl, po = (back(x)[turn] for x in (pm, pl, po))
    # The rest of each request by itself.
    blk = skip[:, None] + torch.arange(s["rest"], device=dev)
    page = torch.where(blk < table.shape[1], table.gather(1, blk.clamp(max=table.shape[1] - 1)), -1)
    key = (blk[..., None] * BLK + torch.arange(BLK, device=dev)).flatten(1)
    limit = (used - nq)[:, None] + i
    see = (key[:, None] <= limit[..., None]) & (page >= 0).repeat_interleave(BLK, 1)[:, None] & (key < used[:, None])[:, None]
    m, l, o = _part(shaped(token), _keys(s["k"], page), _keys(s["v"], page), see.repeat_interleave(ratio, 1)[:, None])
    if s["groups"] is not None:
        top = torch.maximum(m, pm)
        ref = torch.where(top == -math.inf, 0.0, top)
        f, p = torch.exp(m - ref), torch.exp(pm - ref)
        m, l, o = top, l * f + pl * p, o * f + po * p
    o = o / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l))[..., 0]
    live = (token < t).view(-1)
    o = o.unflatten(2, (-1, ratio)).transpose(1, 2).reshape(-1, hq, DIM)[live]
    lse = lse.unflatten(2, (-1, ratio)).transpose(1, 2).reshape(-1, hq)[live]
    return {"out": o.to(q.dtype), "lse": lse}


def _sample(s):
    """In 64 bits, as a border may lie anywhere: the tokens by falling logits (equal ones by their number), cut to a first few, and
    the first of these whose running sum passes u times the sum of all of them."""
    x, v = s["logits"].double(), s["logits"].shape[1]
    t = s["temperature"].double()[:, None]
    greedy = t < 1e-5
    val, order = x.sort(dim=1, descending=True, stable=True)
    y = torch.where(val == -math.inf, -math.inf, (val - val[:, :1]) / torch.where(greedy, 1.0, t))
    w = torch.exp(y)
    run = w.cumsum(1)
    n = torch.full_like(t, v, dtype=torch.long)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        n = torch.where((k > 0) & (k < v), k, n)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        cut = (run < p * run.gather(1, n - 1)).sum(1, keepdim=True) + 1
        n = torch.where(p < 1, torch.minimum(n, cut), n)
    if s["min_p"] is not None:
        n = torch.minimum(n, (w >= s["min_p"].double()[:, None]).sum(1, keepdim=True))
    n = torch.where(greedy, 1, n)
    at = (run <= s["u"].double()[:, None] * run.gather(1, n - 1)).sum(1, keepdim=True)
    at = torch.minimum(at, n - 1)
    return {"tokens": order.gather(1, at)[:, 0].to(torch.int32), "logprobs": (y.gather(1, at) - torch.log(run[:, -1:]))[:, 0].float()}


def _path(s):
    """A node is on the path where each of its ancestors is the first child of its parent that the parent's sample names."""
    cu, n, dev = s["cu"].long(), s["most"], "cuda"
    b = len(cu) - 1
    i = torch.arange(n, device=dev)
    live = i < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(live, cu[:-1, None] + i, 0)
    anc = ((s["mask"].long()[at][..., i // 32] >> (i % 32)) & 1).bool() & live[:, :, None]  # (b, node, ancestor)
    parent = torch.where(anc & (i < i[:, None]), i, -1).amax(2)
    named = live & (parent >= 0) & (s["drafts"].long()[at] == s["sampled"].long()[at].gather(1, parent.clamp(min=0)))
    first = torch.full((b, n + 1), n, dtype=torch.long, device=dev).scatter_reduce_(1, torch.where(named, parent, n), i.expand(b, n), "amin")
    chosen = (named & (first.gather(1, parent.clamp(min=0)) == i)) | (i == 0)
    on = live & ~(anc & ~chosen[:, None]).any(2)
    count = on.sum(1)
    path = torch.where(on, i, n).sort(1).values
    last = path.gather(1, (count - 1).clamp(min=0)[:, None])[:, 0].clamp(max=n - 1)
    after = torch.where(count > 0, s["sampled"].long()[at].gather(1, last[:, None])[:, 0], -1)
    return {"path": torch.where(i < count[:, None], path, -1).to(torch.int32), "path_len": count.to(torch.int32), "next": after.to(torch.int32)}


# ------------------------------------------------------------------------------------------------------------------- the passes
def _own(s):
    import block_sparse_top_msa_gb300 as msa

    if s["op"] == "tables":
        t = msa.msa_step_tables(s["table"], s["used"], s["rows"], s["nq"], total_q=s["total"], num_pages=s["pages"])
        return {"cu": t.cu_seqlens_q, "used": t.seqused_k, "table": t.page_table, "token_rows": t.token_rows, "positions": t.positions, "slots": t.slots,
                "group_rows": t.group_rows, "cu_groups": t.cu_groups, "group_blocks": t.group_blocks}
    if s["op"] == "attend":
        out, lse = msa.msa_prefix_attention(s["q"], s["k"], s["v"], s["cu"], page_table=s["table"], seqused_k=s["used"], max_seqlen_q=s["nq_hi"], return_softmax_lse=True, **(s["groups"] or {}))
        return {"out": out, "lse": lse}
    if s["op"] == "sample":
        return dict(zip(("tokens", "logprobs"), msa.msa_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], return_logprobs=True)))
    return dict(zip(("path", "path_len", "next"), msa.msa_draft_path(s["sampled"], s["drafts"], s["mask"], s["cu"], max_path=s["most"])))


def run(state):
    if own:
        return _own(state)
    return {"tables": _tables, "attend": _attend, "sample": _sample, "path": _path}[state["op"]](state)


# ------------------------------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    nq = (c.get("nq_lo", 0) + c.get("nq_hi", 0)) / 2
    if c["op"] == "tables":
        return {"bytes": c["batch"] * (2 * 4 * c["max_pages"] + 4 * 8 + nq * 16), "flops": 0}
    if c["op"] == "path":
        return {"bytes": c["batch"] * (nq * (8 + 4 * math.ceil(c["nq_hi"] / 32)) + 4 * c["nq_hi"] + 12), "flops": 0}
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (c["vocab"] * (4 if c["dtype"] == "fp32" else 2) + 28), "flops": 4 * c["rows"] * c["vocab"]}
    b, size = c["groups"] * c["group"], 1 if c["kv"] == "e4m3" else 2
    prompt, rest = (c["prompt_lo"] + c["prompt_hi"]) / 2, (c["own_hi"] - 1) / 2 + nq
    keys = c["groups"] * prompt + b * rest
    t = b * nq
    return {"bytes": 2 * keys * c["hkv"] * DIM * size + t * c["hq"] * (4 * DIM + 4), "flops": 4 * t * c["hq"] * DIM * (prompt + rest)}


# ------------------------------------------------------------------------------------------------------------------- 64 bits
def _exact_attend(s):
    """Each request by itself over all of its keys."""
    cu, used = s["cu"].tolist(), s["used"].tolist()
    t, hq, _ = s["q"].shape
    hkv = s["k"].shape[1]
    out, lse = torch.zeros(t, hq, DIM, dtype=torch.float64, device="cuda"), torch.zeros(t, hq, dtype=torch.float64, device="cuda")
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        page = s["table"][b, : _blocks(used[b])].long()
        k, v = (s[x][page].double().transpose(0, 1).reshape(hkv, -1, DIM)[:, : used[b]] for x in "kv")
        x = s["q"][lo:hi].double().view(hi - lo, hkv, -1, DIM).permute(1, 2, 0, 3) @ k[:, None].transpose(2, 3) / math.sqrt(DIM)
        hidden = torch.arange(used[b], device="cuda") > torch.arange(used[b] - (hi - lo), used[b], device="cuda")[:, None]
        x.masked_fill_(hidden, -math.inf)
        z = torch.logsumexp(x, -1, keepdim=True)
        out[lo:hi] = (torch.exp(x - z) @ v[:, None]).permute(2, 0, 1, 3).reshape(hi - lo, hq, DIM)
        lse[lo:hi] = z[..., 0].permute(2, 0, 1).reshape(hi - lo, hq)
    return {"out": out, "lse": lse}


def _exact_sample(s):
    """The chosen tokens' log probabilities, of tokens that a walk row by row chooses."""
    got = []
    for r in range(len(s["u"])):
        t = float(s["temperature"][r])
        x = s["logits"][r].double() / (t if t >= 1e-5 else 1.0)
        ids = torch.argsort(x, descending=True, stable=True)
        p = torch.softmax(x, 0)
        k = int(s["top_k"][r]) if s["top_k"] is not None else 0
        if t < 1e-5:
            k = 1
        keep = ids[:k] if 0 < k < len(ids) else ids
        if s["top_p"] is not None and float(s["top_p"][r]) < 1:
            q = p[keep] / p[keep].sum()
            keep = keep[q.cumsum(0) - q < float(s["top_p"][r])]
        if s["min_p"] is not None:
            keep = keep[p[keep] >= float(s["min_p"][r]) * p[ids[0]]]
        run = p[keep].cumsum(0)
        at = min(int(torch.searchsorted(run, float(s["u"][r]) * run[-1], right=True)), len(keep) - 1)
        got.append(torch.log(p[keep[at]]))
    return {"tokens": None, "logprobs": torch.stack(got)}


def exact(case, seed):
    if case["op"] in ("tables", "path"):
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_attend(s) if case["op"] == "attend" else _exact_sample(s)
