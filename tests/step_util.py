"""Plain 64-bit forms of the operators around the attention of a serving step, on the CPU, and
inputs for their tests."""
import math

import torch

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


def half_step(dtype):
    """The largest error of rounding to a type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def rope_table(length, rotary, seed=0):
    f = 1e4 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(rotary, 1))
    a = torch.arange(length, dtype=torch.float64)[:, None] * f + seed
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(x, cos, sin, interleaved):
    """x (T, H, 128) turned pair by pair; also the sum of the magnitudes that make each element."""
    y, mag = x.clone(), x.abs()
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[:, None, i], sin[:, None, i]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def table_rows(cos_sin, positions):
    """(known, cos, sin) of each token, zeros where the position is padding."""
    if cos_sin is None:
        e = torch.zeros(len(positions), 0, dtype=torch.float64)
        return (positions >= 0), e, e
    known = (positions >= 0) & (positions < cos_sin.shape[0])
    row = cos_sin.double()[positions.long().clamp(0, cos_sin.shape[0] - 1)]
    return known, *row.chunk(2, 1)


def norm_rope(x, w, cos_sin, positions, interleaved, eps=EPS):
    """The operator's rows in 64 bits and the magnitudes that its roundings are relative to."""
    known, cos, sin = table_rows(cos_sin, positions)
    x = x.double()
    n = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w.double()
    y, mag = rotate(n, cos, sin, interleaved)
    live = known[:, None, None]
    return torch.where(live, y, 0.0), torch.where(live, mag, 0.0)


def norm_rope_bwd(x, w, dy, cos_sin, positions, interleaved, eps=EPS):
    """(dx, its magnitudes, dw, the sum of its terms' magnitudes)."""
    known, cos, sin = table_rows(cos_sin, positions)
    live = known[:, None, None]
    x, w = x.double(), w.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    u, umag = rotate(dy.double(), cos, -sin, interleaved)
    u, umag = torch.where(live, u, 0.0), torch.where(live, umag, 0.0)
    g, gmag = u * w, umag * w.abs()
    dx = r * (g - x * r.square() * (g * x).mean(-1, keepdim=True))
    mag = r * (gmag + x.abs() * r.square() * (gmag * x.abs()).mean(-1, keepdim=True))
    terms = u * x * r
    return dx, mag, terms.sum((0, 1)), (umag * x.abs() * r).sum((0, 1))


def tree_bits(parents):
    """(n, words) int32 rows of a tree's mask: each node's ancestors and itself."""
    n = len(parents)
    rows = torch.zeros(n, (n + 31) // 32, dtype=torch.int64)
    for i in range(n):
        j = i
        while j >= 0:
            rows[i, j // 32] |= 1 << (j % 32)
            j = parents[j]
    return torch.where(rows >= 1 << 31, rows - (1 << 32), rows).to(torch.int32)


def pad_words(rows, words):
    return torch.nn.functional.pad(rows, (0, words - rows.shape[1]))


def bit(row, j):
    return j < 32 * len(row) and (int(row[j // 32]) >> (j % 32)) & 1 == 1


def tree_attention(q, k, v, lists, cu, mask, table, used, scale):
    """(out, lse, A) in 64 bits, A = sum p |v| / l per element; rows behind the last sequence are NaN."""
    t, hq, d = q.shape
    hkv, num_pages = lists.shape[0], k.shape[0]
    group = hq // hkv
    out = torch.full((t, hq, d), math.nan, dtype=torch.float64)
    size, lse = out.clone(), torch.full((t, hq), math.nan, dtype=torch.float64)
    qd, kd, vd = q.double(), k.double(), v.double()
    for b in range(len(used)):
        lo, hi = int(cu[b]), int(cu[b + 1])
        lk = int(used[b])
        first = lk - (hi - lo)
        for i in range(lo, hi):
            for h in range(hkv):
                at = []
                for blk in sorted(set(int(x) for x in lists[h, i])):
                    if blk < 0 or blk * 128 >= lk or blk >= table.shape[1]:
                        continue
                    page = int(table[b, blk])
                    if not 0 <= page < num_pages:
                        continue
                    for p in range(blk * 128, min(lk, blk * 128 + 128)):
                        if p < first or bit(mask[i], p - first):
                            at.append((page, p % 128))
                g = slice(h * group, (h + 1) * group)
                if not at:
                    out[i, g], size[i, g], lse[i, g] = 0.0, 0.0, -math.inf
                    continue
                page, row = (torch.tensor(x) for x in zip(*at))
                s = qd[i, g] @ kd[page, h, row].T * scale
                lse[i, g] = torch.logsumexp(s, 1)
                p = torch.exp(s - lse[i, g, None])
                out[i, g], size[i, g] = p @ vd[page, h, row], p @ vd[page, h, row].abs()
    return out, lse, size


class Tables:
    """The cache's tables as plain lists, with the operators on them."""

    def __init__(self, rows, max_pages, num_pages):
        self.table = [[-1] * max_pages for _ in range(rows)]
        self.used = [0] * rows
        self.refs = [0] * num_pages

    def tensors(self, device):
        return tuple(torch.tensor(x, dtype=torch.int32, device=device) for x in (self.table, self.used, self.refs))

    def check(self, table, used, refs):
        assert table.tolist() == self.table
        assert used.tolist() == self.used
        assert refs.tolist() == self.refs

    def _grant(self, wants):
        """Statuses and pages of requests for so many pages each (None: refused)."""
        free = [p for p, n in enumerate(self.refs) if n == 0]
        status, pages, taken = [], [], 0
        for want in wants:
            if want is None:
                status.append(1)
                pages.append([])
                continue
            taken += want
            fits = want == 0 or taken <= len(free)
            status.append(0 if fits else 2)
            pages.append(free[taken - want : taken] if fits else [])
        return status, pages

    def extend(self, rows, lengths):
        wants, seen = [], set()
        for r, n in zip(rows, lengths):
            ok = 0 <= r < len(self.table) and r not in seen and self.used[r] <= n <= 128 * len(self.table[0])
            seen.add(r)
            wants.append(sum(self.table[r][t] < 0 for t in range(self.used[r] // 128, (n + 127) // 128)) if ok else None)
        status, pages = self._grant(wants)
        for r, n, st, got in zip(rows, lengths, status, pages):
            if st == 0:
                for t in range(self.used[r] // 128, (n + 127) // 128):
                    if self.table[r][t] < 0:
                        self.table[r][t] = got.pop(0)
                        self.refs[self.table[r][t]] = 1
                self.used[r] = n
        return status

    def fork(self, src, dst, pools=()):
        rows, pages, wants, seen = len(self.table), len(self.refs), [], set()
        for s, r in zip(src, dst):
            ok = 0 <= r < rows and r not in seen and 0 <= s < rows and s not in dst
            ok = ok and self.used[r] == 0 and all(p < 0 for p in self.table[r])
            seen.add(r)
            n = self.used[s] if ok else 0
            wants.append(int(n % 128 != 0 and 0 <= self.table[s][n // 128] < pages) if ok else None)
        status, got = self._grant(wants)
        for s, r, st, fresh in zip(src, dst, status, got):
            if st != 0:
                continue
            whole = self.used[s] // 128
            for t in range(whole):
                p = self.table[s][t]
                if 0 <= p < pages:
                    self.table[r][t] = p
                    self.refs[p] += 1
            if fresh:
                self.table[r][whole] = fresh[0]
                self.refs[fresh[0]] = 1
                for pool in pools:
                    pool[fresh[0]] = pool[self.table[s][whole]]
            self.used[r] = self.used[s]
        return status

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.table):
                for p in self.table[r]:
                    if 0 <= p < len(self.refs):
                        self.refs[p] -= 1
                self.table[r] = [-1] * len(self.table[r])
                self.used[r] = 0


def accept(pools, table, used, cu, path, path_len):
    """Moves rows of (num_pages, Hkv, 128, d) pools in place; returns the lengths."""
    lengths = []
    for b in range(len(used)):
        n = int(cu[b + 1]) - int(cu[b])
        first = int(used[b]) - n
        kept = []
        for j in range(max(0, min(int(path_len[b]), path.shape[1]))):
            p = int(path[b, j])
            if p < 0 or p >= n or (kept and p <= kept[-1]):
                break
            kept.append(p)
        for j, p in enumerate(kept):
            s, d = first + p, first + j
            if s == d or d < 0 or s >= 128 * table.shape[1]:
                continue
            sp, dp = int(table[b, s // 128]), int(table[b, d // 128])
            for pool in pools:
                if 0 <= sp < pool.shape[0] and 0 <= dp < pool.shape[0]:
                    pool[dp, :, d % 128] = pool[sp, :, s % 128].clone()
        lengths.append(max(0, first + len(kept)))
    return lengths


def bits(x):
    """A tensor's bytes as whole numbers, for comparing copies."""
    return x.view(torch.uint8 if x.element_size() == 1 else torch.int16)
