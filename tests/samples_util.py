"""Plain forms of the operators of a step of samples, on the CPU: a step's tables, drafted paths, sampling and attention over
shared prefixes."""
import math

import torch

import step_util as U


def step_tables(table, used, rows, new_lens, total_q, num_pages):
    """The nine tables as lists."""
    width, batch = len(table[0]), len(rows)
    cu, lens, out, full = [0], [], [], False
    counts = []
    for b in range(batch):
        r = rows[b]
        real = 0 <= r < len(table)
        lk = max(0, used[r]) if real else 0
        n = min(max(0, new_lens[b]), lk) if real else 0
        full = full or cu[-1] + n > total_q
        n = 0 if full else n
        cu.append(cu[-1] + n)
        counts.append(n)
        lens.append(lk)
        out.append([p if real and 128 * j < lk and 0 <= p < num_pages else -1 for j, p in enumerate(table[r] if real else [-1] * width)])
    token_rows, positions, slots = [-1] * total_q, [-1] * total_q, [-1] * total_q
    for b in range(batch):
        for i in range(counts[b]):
            t, pos = cu[b] + i, lens[b] - counts[b] + i
            page = out[b][pos // 128] if pos // 128 < width else -1
            token_rows[t], positions[t], slots[t] = b, pos, page * 128 + pos % 128 if page >= 0 else -1
    groups, place = [], {}
    for b in range(batch):
        p = out[b][0] if counts[b] > 0 else -1
        if p >= 0 and p in place:
            groups[place[p]].append(b)
            continue
        if p >= 0:
            place[p] = len(groups)
        groups.append([b])
    blocks = []
    for g in groups:
        most = 0
        if len(g) > 1:
            most = min((lens[b] - counts[b]) // 128 for b in g)
            lead = out[g[0]]
            for b in g:
                n = 0
                while n < width and out[b][n] >= 0 and out[b][n] == lead[n]:
                    n += 1
                most = min(most, n)
        blocks.append(most)
    cu_groups = [0]
    for g in groups:
        cu_groups.append(cu_groups[-1] + len(g))
    pad = batch - len(groups)
    return cu, lens, out, token_rows, positions, slots, [b for g in groups for b in g], cu_groups + [batch] * pad, blocks + [0] * pad


def draft_path(sampled, drafts, mask, cu, max_path, total):
    paths, lens, after = [], [], []
    words = len(mask[0]) if mask else 1
    for lo, hi in zip(cu, cu[1:]):
        n = min(hi, total) - lo
        parent = []
        for c in range(n):
            up = [j for j in range(min(c, 32 * words)) if (mask[lo + c][j // 32] >> (j % 32)) & 1]
            parent.append(max(up) if up else -1)
        path = [0] if n > 0 else []
        while path and len(path) < max_path:
            named = [c for c in range(path[-1] + 1, n) if parent[c] == path[-1] and drafts[lo + c] == sampled[lo + path[-1]]]
            if not named:
                break
            path.append(named[0])
        lens.append(len(path))
        after.append(sampled[lo + path[-1]] if path else -1)
        paths.append(path + [-1] * (max_path - len(path)))
    return paths, lens, after


def sample_row(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, its log probability before the cuts, whether no border is near) of one row in 64 bits. With weights that are off by
    2^-34 of themselves and 2^-45 of the largest, a sum of n of them is off by 2^-34 of it and n 2^-45, and so is what it is
    compared with: a border is clear where the two differ by more than both together."""
    x = torch.where(x.isnan(), -math.inf, x.double())
    val, order = x.sort(descending=True, stable=True)
    if val[0] == -math.inf:
        return -1, -math.inf, True
    greedy = not t >= 1e-5
    t = 1.0 if greedy else min(t, 1e30)
    y = torch.where(val == val[0], 0.0, torch.where(val == -math.inf, -math.inf, (val - val[0]) / t))
    w = torch.exp(y)
    w = torch.where(val == -math.inf, 0.0, w)
    run = w.cumsum(0)
    z, clear = float(run[-1]), True
    off = 2 * (z * 2**-34 + len(x) * 2**-45)
    n = len(x)
    if 0 < k < n:
        n = k
    if p < 1:
        want = max(p, 0.0) * float(run[n - 1])
        clear = clear and (want == 0 or float((run[:n] - want).abs().min()) > off)
        n = max(1, min(n, int((run[:n] < want).sum()) + 1))
    if m > 0:
        m = min(m, 1.0)
        clear = clear and (not bool((w < 1).any()) or float((w - m).abs()[w < 1].min()) > 2**-33)
        n = min(n, int((w >= m).sum()))
    if greedy:
        n, clear = 1, True
    at = 0
    if n > 1:
        want = min(max(u, 0.0), 1.0) * float(run[n - 1])
        if u < 1:
            clear = clear and float((run[: n - 1] - want).abs().min()) > off
            at = min(int((run[:n] <= want).sum()), n - 1)
        else:
            at = int((w[:n] > 0).sum()) - 1
    return int(order[at]), float(y[at] - math.log(z)), clear


def prefix_attention(q, k, v, cu, table, used, scale, causal=True):
    """(out, lse, A) in 64 bits, each request by itself; A = sum p |v| / l per element. Rows behind the last request are NaN."""
    t, hq, d = q.shape
    hkv, num_pages = k.shape[1], k.shape[0]
    group = hq // hkv
    out = torch.full((t, hq, d), math.nan, dtype=torch.float64)
    size, lse = out.clone(), torch.full((t, hq), math.nan, dtype=torch.float64)
    for b in range(len(used)):
        lo, hi, lk = int(cu[b]), int(cu[b + 1]), int(used[b])
        pos = torch.arange(min(lk, 128 * table.shape[1]))
        page = table[b].long()[pos // 128]
        here = (page >= 0) & (page < num_pages)
        pos, page = pos[here], page[here]
        kd, vd = k[page, :, pos % 128].double(), v[page, :, pos % 128].double()
        for i in range(lo, hi):
            see = pos <= lk - (hi - lo) + (i - lo) if causal else torch.ones_like(pos, dtype=torch.bool)
            for h in range(hkv):
                g = slice(h * group, (h + 1) * group)
                if not bool(see.any()):
                    out[i, g], size[i, g], lse[i, g] = 0.0, 0.0, -math.inf
                    continue
                s = q[i, g].double() @ kd[see, h].T * scale
                lse[i, g] = torch.logsumexp(s, 1)
                p = torch.exp(s - lse[i, g, None])
                out[i, g], size[i, g] = p @ vd[see, h], p @ vd[see, h].abs()
    return out, lse, size


def ints(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def mask_rows(parents, words=None):
    rows = U.tree_bits(parents)
    return rows if words is None else U.pad_words(rows, words)
