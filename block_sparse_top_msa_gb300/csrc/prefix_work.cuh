// The work of the attention over shared prefixes, as its kernels walk it: a line
// of units' blocks, cut into ranges, one per CTA.
#pragma once

#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "softmax.cuh"

namespace msa {

// Costs: a block, and what a unit takes besides its blocks (its Q, its
// epilogue, the change of units), in halves of a block of 16 rows, or in
// quarters of a block of two tiles of 128.
MSA_DEV int block_cost(const PrefixArgs& a, int rows) { return a.small ? 2 : rows > 128 ? 4 : 3; }
MSA_DEV int unit_cost(const PrefixArgs& a) { return a.small ? kSmallUnitCost : kBigUnitCost; }
MSA_DEV int tile_rows_of(const PrefixArgs& a) { return a.small ? kSmallRows : kBigRows; }
// Where block j of a unit lies on the line, from the unit's beginning: what the
// unit takes besides counts with its first block.
MSA_DEV int block_at(const PrefixArgs& a, int cost, int j) { return j == 0 ? 0 : unit_cost(a) + j * cost; }
// The first block that lies at or after `in`.
MSA_DEV int block_from(const PrefixArgs& a, int cost, int in) {
  return in <= 0 ? 0 : max(1, (in - unit_cost(a) + cost - 1) / cost);
}

// The partition of the line's [0, total) into the CTAs' ranges. A range is never
// shorter than a unit's first block, so each CTA between those of a unit's first
// and last block holds one of its blocks.
struct Ranges {
  long long total;
  int n;
  MSA_DEV long long start(int i) const { return total * i / n; }
  // The range that position p < total is in: the last i with start(i) <= p.
  MSA_DEV int holder(long long p) const { return (int)((p * n + n - 1) / total); }
};
MSA_DEV Ranges ranges_of(const PrefixArgs& a, int entries) {
  const long long total = __ldcg(a.start + entries);
  const long long most = total / (a.small ? kSmallRange : kBigRange);
  return {total, (int)(most < 1 ? 1 : most < a.grid ? most : a.grid)};
}
// The last of n ascending numbers, the first of them at most `at`, that is at
// most `at`; by a whole warp.
template <class T>
MSA_DEV int last_upto(const T* v, int n, T at) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const unsigned under = __ballot_sync(0xffffffffu, i < hi && __ldcg(v + (i < hi ? i : lo)) <= at);
    const int k = 31 - __clz(under);  // lane 0 is under
    hi = min(hi, lo + (k + 1) * step);
    lo += k * step;
  }
  return lo;
}

// A piece of a unit: some blocks of one entry's tile with one KV head.
struct Piece {
  int n;           // blocks; -1: no more
  int whole;       // all of the unit's
  int b, h, j0;    // page row, KV head, first block
  int row0, rows;  // rows of the entry
  int tau;         // the entry's first token
  int hidden, lk;  // row r sees keys below min(lk, hidden + r / G + 1)
  int place;       // of row 0's parts: its own, or (below 0) the CTA's
  int keys;        // keys from j0 on that some row sees
  int e, tile_head;  // the unit: entry, tile * heads + head
  int alone;       // a request's own run, without a group's before it
};

// Walks a CTA's range, piece by piece; by a whole warp, whose lanes agree. The
// next entry is read while this one's units are handed out.
struct Walk {
  const PrefixArgs& a;
  int list;
  long long at, end, unit_at;
  int e, tile, h, len, cost, tiles;
  int4 x, y, nx, ny;
  MSA_DEV void ahead() {
    const int4* w = a.work + 2 * min(e + 1, list - 1);
    nx = __ldcg(w), ny = __ldcg(w + 1);
  }
  MSA_DEV void open() {
    cost = block_cost(a, x.y);
    len = unit_cost(a) + y.x * cost;
    tiles = (x.y + tile_rows_of(a) - 1) / tile_rows_of(a);
  }
  MSA_DEV Walk(const PrefixArgs& args, int cta) : a(args), list(__ldcg(args.meta)), at(0), end(0) {
    const Ranges r = ranges_of(a, list);
    if (r.total <= 0 || cta >= r.n) return;
    at = r.start(cta), end = r.start(cta + 1);
    e = last_upto(a.start, list, at);
    const int4* w = a.work + 2 * e;
    x = __ldcg(w), y = __ldcg(w + 1);
    open();
    ahead();
    const long long first = __ldcg(a.start + e);
    const int unit = (int)((at - first) / len);
    unit_at = first + (long long)unit * len;
    tile = unit / a.num_kv_heads;
    h = unit - tile * a.num_kv_heads;
  }
  MSA_DEV bool next(Piece& p) {
    p.n = -1;
    while (at < end && p.n < 0) step(p);
    return p.n >= 0;
  }
  MSA_DEV void step(Piece& p) {
    const int in = (int)(at - unit_at);
    const bool ends = unit_at + len <= end;  // within the range
    const int j0 = block_from(a, cost, in), j1 = ends ? y.x : min(y.x, block_from(a, cost, (int)(end - unit_at)));
    if (j1 > j0 || in == 0) {
      const int G = a.num_qo_heads / a.num_kv_heads;
      p.n = j1 - j0;
      p.whole = j0 == 0 && j1 == y.x;
      p.b = x.z, p.h = h, p.j0 = (x.w & ~kGroupRun) + j0;
      p.row0 = tile * tile_rows_of(a), p.rows = min(tile_rows_of(a), x.y - p.row0);
      p.tau = x.x;
      p.hidden = y.y, p.lk = y.z;
      p.place = j0 == 0 ? ((x.w & kGroupRun) ? a.total_q : 0) + x.x : -1;
      const long long last = min((long long)y.z, (long long)y.y + (p.row0 + p.rows - 1) / G + 1) - (long long)p.j0 * kBlk;
      p.keys = (int)max(0ll, min(last, (long long)p.n * kBlk));
      p.e = e, p.tile_head = tile * a.num_kv_heads + h;
      p.alone = y.w < 0 && !(x.w & kGroupRun);
    }
    at = ends ? unit_at + len : end;
    if (ends) {
      unit_at = at;
      if (++h == a.num_kv_heads) {
        h = 0;
        if (++tile == tiles) {
          tile = 0, ++e;
          x = nx, y = ny;
          open();
          ahead();
        }
      }
    }
  }
};

// Where the parts of a unit are: at the rows' own places, and at those of the
// `n` CTAs from c0 + 1 on.
struct Parts {
  int c0, n;
};
// Of a unit of entry e, which has these rows and blocks.
MSA_DEV Parts parts_of(const PrefixArgs& a, const Ranges& r, int e, int rows, int blocks, int tile_head) {
  const int cost = block_cost(a, rows), len = unit_cost(a) + blocks * cost;
  const long long at = __ldcg(a.start + e) + (long long)tile_head * len;
  const int c0 = r.holder(at), c1 = blocks > 1 ? r.holder(at + block_at(a, cost, blocks - 1)) : c0;
  return {c0, c1 - c0};
}

// The parts of a group's run that rows of one of its requests join: of no more
// rows side by side than a tile has, which lie in one of its tiles or two.
struct Before {
  int on;        // the request has a group's run before its own
  int row0;      // of the group's entry: its row of row 0
  int tile;      // and the tile of that row
  Parts parts[2];  // of this tile and the next
};
// Where the first of a unit's pieces leaves a row's parts: at the row's own place,
// or in CTA c0's row `row` of the tile.
MSA_DEV size_t first_part(const PrefixArgs& a, size_t own_row, int c0, int row) {
  return a.at_cta ? (size_t)c0 * tile_rows_of(a) + row : own_row;
}
// By a whole warp.
MSA_DEV Before before_of(const PrefixArgs& a, const Ranges& ranges, int group, int tau, int row0, int rows, int h) {
  Before f{};
  const int e = group < 0 ? -1 : __ldcg(a.group + group), tile_rows = tile_rows_of(a);
  if (e < 0) return f;
  const int4* w = a.work + 2 * e;
  const int4 x = __ldcg(w);
  const int blocks = __ldcg(&w[1].x), G = a.num_qo_heads / a.num_kv_heads;
  f.on = 1;
  f.row0 = (tau - x.x) * G + row0;
  f.tile = f.row0 / tile_rows;
  const int lane = threadIdx.x & 31, last = (f.row0 + rows - 1) / tile_rows;
  const Parts mine = parts_of(a, ranges, e, x.y, blocks, min(f.tile + (lane & 1), last) * a.num_kv_heads + h);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    f.parts[i] = {__shfl_sync(0xffffffffu, mine.c0, i), __shfl_sync(0xffffffffu, mine.n, i)};
  return f;
}

// Of two 16-bit values: all bits of those that are not finite.
template <bool F16>
MSA_DEV uint32_t not_finite2(uint32_t x) {
  constexpr uint32_t kExp = F16 ? 0x7c007c00u : 0x7f807f80u;
  return __vcmpeq2(x & kExp, kExp);
}

// (m, l) of a part as it is joined: the part of a row that saw NaN has a sum of
// NaN, and a maximum that is a number, as -inf says that it saw nothing and
// maxima of parts drop NaN.
MSA_DEV float2 part_of_sum(float m, float l) { return make_float2(m > -INFINITY || l == 0.f ? m : 0.f, l); }

// Running sum of eight columns of a row's parts, by one thread.
struct Joined {
  float m = -INFINITY, l = 0.f, o[8] = {};
  MSA_DEV void add(float2 ml, const float (&v)[8]) {
    if (ml.x == -INFINITY) return;  // a part without a visible key may hold anything
    const float top = fmaxf(m, ml.x), f = m == -INFINITY ? 0.f : ex2(m - top), p = ex2(ml.x - top);
    m = top;
    l = fmaf(l, f, p * ml.y);
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = fmaf(p, v[c], o[c] * f);
  }
  // Those at `first`, then those of the CTAs, from the from-th in steps; loads of
  // AHEAD at a time.
  template <int kAhead>
  MSA_DEV void add_some(const PrefixArgs& a, size_t first, int row, Parts parts, int col, int from, int step) {
    for (int i0 = from; i0 <= parts.n; i0 += kAhead * step) {
      float2 ml[kAhead];
      float4 v[kAhead][2];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = min(i0 + u * step, parts.n);
        const size_t at = i == 0 ? first : a.part_rows + (size_t)(parts.c0 + i) * tile_rows_of(a) + row;
        ml[u] = __ldcg(a.part_ml + at);
        const float4* from = reinterpret_cast<const float4*>(a.part_o + at * kHeadDim + col);
        v[u][0] = __ldcg(from), v[u][1] = __ldcg(from + 1);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (i0 + u * step > parts.n) break;
        const float x[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w, v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
        add(ml[u], x);
      }
    }
  }
  // Row `row` of its tile.
  MSA_DEV void add_parts(const PrefixArgs& a, size_t first, int row, Parts parts, int col, int from = 0, int step = 1) {
    if (parts.n < 2 * step) add_some<2>(a, first, row, parts, col, from, step);
    else add_some<8>(a, first, row, parts, col, from, step);
  }
  MSA_DEV void add_before(const PrefixArgs& a, const Before& f, int r, size_t own_row, int col, int from = 0, int step = 1) {
    if (!f.on) return;
    const int row = f.row0 + r, tile = row / tile_rows_of(a), second = tile - f.tile;
    add_parts(a, (size_t)a.total_q * a.num_qo_heads + own_row, row - tile * tile_rows_of(a),
              Parts{second ? f.parts[1].c0 : f.parts[0].c0, second ? f.parts[1].n : f.parts[0].n}, col, from, step);
  }
  // Output row `orow` (token and head of q).
  MSA_DEV void write(const PrefixArgs& a, size_t orow, int col) const {
    const bool has = l != 0.f;
    const float inv = has ? 1.f / l : 0.f;
    auto pack = [&](float x, float y) { return a.f16 ? pack_f16x2(x, y) : pack_bf16x2(x, y); };
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * kHeadDim + col) =
        make_uint4(pack(o[0] * inv, o[1] * inv), pack(o[2] * inv, o[3] * inv), pack(o[4] * inv, o[5] * inv),
                   pack(o[6] * inv, o[7] * inv));
    if (col == 0 && a.lse != nullptr) a.lse[orow] = has ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
};

}  // namespace msa
