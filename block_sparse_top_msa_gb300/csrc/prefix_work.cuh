// The work list of the attention over shared prefixes, as its kernels walk it:
// lines of units' blocks cut into ranges.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace msa {

// The partition of a line's [0, total) into the CTAs' ranges.
struct Ranges {
  long long total;
  int n;
  MSA_DEV long long start(int i) const { return total * i / n; }
  // The range that position p < total is in: the last i with start(i) <= p.
  MSA_DEV int holder(long long p) const { return (int)((p * n + n - 1) / total); }
};
MSA_DEV Ranges ranges_of(const PrefixArgs& a, int line) {
  const long long total = __ldcg(a.start + line * (2 * a.batch + 1) + 2 * a.batch);
  const long long most = total / (line ? a.big_range : a.small_range);
  const int grid = line ? a.big_grid : a.small_grid;
  return {total, (int)(most < 1 ? 1 : most < grid ? most : grid)};
}

// A piece of a unit: blocks [j0, j0 + n) of one entry's tile with one KV head.
struct Piece {
  int n;          // blocks; 0: no more
  int b, h, j0;   // page row, KV head, first block
  int row0, rows; // rows of the entry
  int tau;        // the entry's first token
  int hidden, lk; // row r sees keys below min(lk, hidden + r / G + 1)
  int place;      // of row 0's parts: its own, or (below 0) the CTA's
  int keys;       // keys from j0 on that some row sees
};

// Walks a CTA's range, piece by piece.
struct Walk {
  const PrefixArgs& a;
  int line;
  long long at, end;
  int e;
  MSA_DEV Walk(const PrefixArgs& args, int l, const Ranges& r, int cta) : a(args), line(l), at(0), end(0), e(0) {
    if (r.total <= 0 || cta >= r.n) return;
    at = r.start(cta), end = r.start(cta + 1);
    const long long* start = a.start + line * (2 * a.batch + 1);
    int lo = 0;  // the last entry that begins at or before `at`
    for (int hi = 2 * a.batch; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (__ldcg(start + mid) <= at) lo = mid; else hi = mid;
    }
    e = lo;
  }
  MSA_DEV bool next(Piece& p) {
    p.n = 0;
    while (at < end && p.n == 0) step(p);
    return p.n > 0;
  }
  // The piece at `at`, which may hold no block's first position.
  MSA_DEV void step(Piece& p) {
    const long long* start = a.start + line * (2 * a.batch + 1);
    while (__ldcg(start + e + 1) <= at) ++e;
    const int4 x = __ldcg(a.work + 2 * e), y = __ldcg(a.work + 2 * e + 1);
    const int G = a.num_qo_heads / a.num_kv_heads, tile_rows = line ? kBigRows : kSmallRows;
    const int w = prefix_weight(line, x.y);
    const long long len = (long long)y.x * w, rel = at - __ldcg(start + e);
    const long long unit = rel / len;
    const int in = (int)(rel - unit * len);
    const long long unit_end = at - in + len, stop = unit_end < end ? unit_end : end;
    // Block j belongs to the range that its first position is in.
    const int j0 = (in + w - 1) / w, j1 = (int)((stop - (at - in) + w - 1) / w);
    const int tile = (int)(unit / a.num_kv_heads);
    at = stop;
    p.n = j1 - j0;
    p.b = x.z, p.h = (int)(unit - (long long)tile * a.num_kv_heads);
    p.j0 = x.w + j0;
    p.row0 = tile * tile_rows, p.rows = min(tile_rows, x.y - p.row0);
    p.tau = x.x;
    p.hidden = y.y, p.lk = y.z;
    p.place = j0 == 0 ? (e >= a.batch ? a.total_q : 0) + x.x : -1;
    const long long last = min((long long)y.z, (long long)y.y + (p.row0 + p.rows - 1) / G + 1) - (long long)p.j0 * kBlk;
    p.keys = (int)max(0ll, min(last, (long long)p.n * kBlk));
  }
};

}  // namespace msa
