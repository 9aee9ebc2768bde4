// Tokens from logits: temperature, the largest k, the smallest set of mass p,
// the least share of the largest's probability, and one given random number a
// row.
//
// With x a row, m its maximum and w = e^((x - m) / T), the tokens stand in the
// order of falling x, equal ones in that of their numbers, and S(n) is the sum
// of the first n of their w. Each cut keeps a beginning of that order, so what
// is kept is one, of n tokens, and the token taken is the first whose S passes
// u S(n). All questions are thus of one kind: where does the running count or
// sum pass a number. They are answered without sorting: a histogram of w's
// exponent (32 parts an octave, with counts and sums) says in which part, and
// the few tokens in it are brought together, ordered and summed; a part with
// many is divided again by the logits' bits, down to tokens that are equal.
//
// A row's choice at a border goes by sums of up to 2^19 terms, so these are
// exact: w is a whole number of 2^-44 (to 35 bits of its own value, by a table
// of 2^(i / 1024) and a cubic), and whole numbers add up to the same in any
// order. That makes the result the same from run to run, whichever block or
// thread adds first.
//
// Logits of 32 bits: three kernels, each launched under the tail of the one
// before. The first finds the largest of each slice of a row. The second weighs
// a slice's tokens, adds them to the row's histogram and leaves the slice's order
// by parts (16 bits a token): a part's tokens are a run of each slice's order
// then, and no question but which of many equal ones reads the row again. In the third a block answers for
// its row. A slice is sorted by counting: what an addition to a part's counter
// returns is the token's place in it, so that one such addition a token is all,
// and the weights are added up along the order, a thread 16 neighbours.
//
// 64 rows of 131072: 68 to 71 us (alone 11, 48 and 17); one row 17 to 20 (4, 9,
// 28). Neither memory nor one pipe bounds them: a slice of 8192 goes through its
// steps one after the other, 27000 clocks with another beside it, 10500 of them
// the weights, with issue slots 55% busy at 135 instructions a token; one row's
// answer is a chain of searches. With parts down to 2^-16 only, a row whose
// largest logits stand far above the others had its borders among 100000 tokens of
// one part: 95 to 250 us by the kind of rows.
//
// 16-bit logits, of which there are few, have a form of their own (sample_16.cu).
#include "sample.cuh"

namespace msa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kOrderCap = 256;  // tokens that are ordered at once
constexpr int kStarts = kSampleStarts;
static_assert(kBins == 2 * kThreads, "a thread for two parts");
using Row32 = Values<2>;

struct Histogram {
  uint32_t cnt[kBins + 1], lo[kBins + 1], hi[kBins + 1];
  MSA_DEV void clear() {
    for (int i = threadIdx.x; i <= kBins; i += blockDim.x) cnt[i] = lo[i] = hi[i] = 0u;
    __syncthreads();
  }
  MSA_DEV void add_mass(int part, u64 w) {
    const uint32_t low = (uint32_t)w, old = atomicAdd(&lo[part], low);
    const uint32_t high = (uint32_t)(w >> 32) + (old + low < old ? 1u : 0u);
    if (high) atomicAdd(&hi[part], high);
  }
  MSA_DEV void add(int part, u64 w) {
    atomicAdd(&cnt[part], 1u);
    add_mass(part, w);
  }
  MSA_DEV Mark at(int part) const { return {cnt[part], ((u64)hi[part] << 32) + lo[part]}; }
  // To the row's.
  MSA_DEV void flush(const SampleArgs& a, int row) const {
    for (int i = threadIdx.x; i <= kBins; i += blockDim.x) {
      const Mark m = at(i);
      if (m.count == 0) continue;
      atomicAdd(a.parts_count + (size_t)row * kSampleParts + i, (uint32_t)m.count);
      atomicAdd(a.parts_mass + (size_t)row * kSampleParts + i, m.mass);
    }
  }
};
// Two numbers of each thread, added up or their largest, known to all of the block.
template <bool MAX>
MSA_DEV Mark block_join(u64 a, u64 b, u64 (*sw)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  a = MAX ? warp_max64(a) : warp_add(a);
  b = MAX ? warp_max64(b) : warp_add(b);
  __syncthreads();
  if (lane == 0) sw[warp][0] = a, sw[warp][1] = b;
  __syncthreads();
  a = lane < kWarps ? sw[lane][0] : 0ull;
  b = lane < kWarps ? sw[lane][1] : 0ull;
  return {MAX ? warp_max64(a) : warp_add(a), MAX ? warp_max64(b) : warp_add(b)};
}

// A row's own settings, and its scale.
struct Settings {
  float t;
  int k;
  bool none, one;  // no token at all; the largest is taken
  uint32_t top_key;
  int top_idx;
  Scale scale;
};
MSA_DEV Settings settings_of(const SampleArgs& a, int row) {
  Settings s{};
  u64 best = 0;
  for (int i = threadIdx.x & 31; i < a.slices; i += 32) {
    const u64 x = __ldcg(a.best + (size_t)row * a.slices + i);
    best = x > best ? x : best;
  }
  best = warp_max64(best);
  s.top_key = (uint32_t)(best >> 32);
  s.top_idx = (int)~(uint32_t)best;
  const bool greedy = temperature_of(a, row, s.t);
  s.k = a.top_k != nullptr ? __ldg(a.top_k + row) : 0;
  s.none = s.top_key <= kKeyNegInf;
  s.one = s.none || greedy || s.k == 1;
  s.scale = scale_of(value_of(s.top_key), s.t);
  return s;
}

// The largest value of a slice and its first token: (key, ~token) as one
// number. The row's histogram is emptied.
__global__ void __launch_bounds__(kThreads) sample_top_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ __align__(16) u64 sw[kWarps][2];
  const int slice = blockIdx.x % a.slices, row = blockIdx.x / a.slices;
  grid_dependency_wait();
  grid_dependents_launch();
  for (int i = slice * kThreads + threadIdx.x; i < kSampleParts; i += a.slices * kThreads) {
    a.parts_count[(size_t)row * kSampleParts + i] = 0u;
    a.parts_mass[(size_t)row * kSampleParts + i] = 0ull;
  }
  const int begin = min(slice * a.slice, a.vocab);
  const Row32 v{row_of<2>(a, row), begin, min(begin + a.slice, a.vocab)};
  uint32_t key = 0u;
  int idx = 0;
  v.each([&](float f, int i) {
    const uint32_t k = key_of(f);
    if (k > key) key = k, idx = i;
  });
  const Mark m = block_join<true>(((u64)key << 32) | (uint32_t)~idx, 0, sw);
  if (threadIdx.x == 0) a.best[(size_t)row * a.slices + slice] = m.count;
}

template <int GROUPS>
struct __align__(16) SortShared {
  static constexpr int kTokens = kThreads * 4 * GROUPS;
  // In the order, a word left out behind each thread's: neighbours' words lie in
  // other banks (without: 10500 of a slice's 27000 clocks in the weights).
  float value[kTokens + kThreads];
  uint16_t order[kTokens];
  u64 table[1024];
  Histogram h;
  uint16_t start[kStarts];
  int upto[kWarps];
};

// A slice's histogram and order, GROUPS groups of 16 bytes a thread.
template <int GROUPS>
__global__ void __launch_bounds__(kThreads, 2) sample_sort_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ uint4 sort_memory[];
  auto& sm = *reinterpret_cast<SortShared<GROUPS>*>(sort_memory);
  constexpr int kPer = 4 * GROUPS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slice = blockIdx.x % a.slices, row = blockIdx.x / a.slices;
  for (int i = tid; i < 1024; i += kThreads) sm.table[i] = kPowers.at[i];
  sm.h.clear();
  grid_dependency_wait();
  grid_dependents_launch();
  const Row32 v{row_of<2>(a, row), 0, a.vocab};
  const int at0 = v.first() + slice * kThreads * kPer;  // the slice's first place
  // Value g * 4 + j of a thread stands at at0 + (g * kThreads + tid) * 4 + j.
  float f[kPer];
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    const int at = at0 + (g * kThreads + tid) * 4;
    if (v.inside(at)) {
      const uint4 x = v.load(at);
      f[4 * g] = __uint_as_float(x.x), f[4 * g + 1] = __uint_as_float(x.y);
      f[4 * g + 2] = __uint_as_float(x.z), f[4 * g + 3] = __uint_as_float(x.w);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[4 * g + j] = at + j >= 0 && at + j < a.vocab ? Row32::value(v.row + (long long)(at + j) * 4) : -INFINITY;
    }
  }
  const Settings s = settings_of(a, row);
  if (s.none || (s.one && a.logprobs == nullptr)) return;
  if (s.one) {  // all that is asked for is the sum
    u64 mass = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mass += s.scale.weight(sm.table, f[i]);
    mass = warp_add(mass);
    if (lane == 0 && mass > 0) atomicAdd(a.parts_mass + (size_t)row * kSampleParts + kBins, mass);
    return;
  }
  // Each token's part, and its place in it. Tokens that are never taken, and
  // places beside the row, are left out; those of the last part, which may be
  // nearly all, are counted by the warp.
  uint32_t place[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool live = f[i] > -INFINITY;
    const int part = s.scale.part(f[i]);
    const bool rest = live && part >= kBins;
    const unsigned rests = __ballot_sync(0xffffffffu, rest);
    place[i] = 0xffffffffu;
    if (rests != 0u) {
      uint32_t first = 0u;
      if (lane == 0) first = atomicAdd(&sm.h.cnt[kBins], (uint32_t)__popc(rests));
      first = __shfl_sync(0xffffffffu, first, 0);
      if (rest) place[i] = ((uint32_t)kBins << 16) | (first + __popc(rests & ((1u << lane) - 1u)));
    }
    if (live && !rest) place[i] = ((uint32_t)part << 16) | atomicAdd(&sm.h.cnt[part], 1u);
  }
  __syncthreads();
  const int own = (int)sm.h.cnt[2 * tid], two = own + (int)sm.h.cnt[2 * tid + 1];
  int upto = two;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) sm.upto[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += sm.upto[w];
  sm.start[2 * tid] = (uint16_t)(upto - two);
  sm.start[2 * tid + 1] = (uint16_t)(upto - two + own);
  if (tid == kThreads - 1) sm.start[kBins] = (uint16_t)upto, sm.start[kBins + 1] = (uint16_t)(upto + (int)sm.h.cnt[kBins]);
  __syncthreads();
  const int total = sm.start[kBins + 1];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (place[i] == 0xffffffffu) continue;
    const int to = sm.start[place[i] >> 16] + (int)(place[i] & 0xffffu);
    sm.value[to + to / kPer] = f[i];
    sm.order[to] = (uint16_t)(((i >> 2) * kThreads + tid) * 4 + (i & 3));
  }
  __syncthreads();
  // The weights, along the order. A thread adds up those of its first part and
  // of its last, as most have one or two; what lies between goes one by one.
  const int from = tid * kPer, n = min(total - from, kPer);
  if (n > 0) {
    const int p0 = s.scale.part(sm.value[from + tid]), p1 = s.scale.part(sm.value[from + tid + n - 1]);
    u64 m0 = 0, m1 = 0;
#pragma unroll 4
    for (int i = 0; i < kPer; ++i) {
      if (i >= n) break;
      const float x = sm.value[from + tid + i];
      const int p = s.scale.part(x);
      const u64 w = s.scale.weight(sm.table, x);
      if (p == p0) m0 += w;
      else if (p == p1) m1 += w;
      else sm.h.add_mass(p, w);
    }
    sm.h.add_mass(p0, m0);
    if (p1 != p0) sm.h.add_mass(p1, m1);
  }
  uint4* order = reinterpret_cast<uint4*>(a.order + ((size_t)row * a.slices + slice) * SortShared<GROUPS>::kTokens);
  for (int i = tid; i * 8 < total; i += kThreads) order[i] = reinterpret_cast<const uint4*>(sm.order)[i];
  uint16_t* starts = a.starts + ((size_t)row * a.slices + slice) * kStarts;
  for (int i = tid; i < kBins + 2; i += kThreads) starts[i] = sm.start[i];
  __syncthreads();
  sm.h.flush(a, row);
}

struct __align__(16) Shared {
  u64 table[1024];
  Histogram h;
  Mark top[kBins + 1];  // the row's histogram as running sums
  Mark sub[kBins + 1];  // that of a part
  __align__(16) u64 warp[kWarps][2];
  uint32_t counts[kWarps];
  uint32_t order_n;
  u64 brought[kOrderCap];  // (key, ~token)
  int rank[kOrderCap];
  u64 sorted[kOrderCap];
  u64 sorted_w[kOrderCap];
  Answer answer;
};

struct Row {
  Shared& sm;
  const SampleArgs& a;
  int row;
  Row32 values;
  const Scale& scale;
  uint32_t top_key;

  // The keys of the logits in a part: from the lowest whose part is not above it
  // up to the last below the next part's.
  MSA_DEV uint32_t lowest_key(int part) {
    if (part >= kBins) return 0u;
    uint32_t lo = kKeyNegInf, hi = top_key;  // the part of lo is above, that of hi is not
    while (hi - lo > 1u) {
      const uint32_t step = (hi - lo + kThreads - 1) / kThreads, at = lo + (threadIdx.x + 1) * step;
      const int above = __syncthreads_count(at > lo && at < hi && scale.part(value_of(at)) > part);
      lo += above * step;
      hi = hi - lo > step ? lo + step : hi;
    }
    return hi;
  }
  struct Keys {
    uint32_t lo, hi;
  };
  MSA_DEV Keys keys_of(int part) { return {lowest_key(part), part > 0 ? lowest_key(part - 1) - 1u : top_key}; }

  // The tokens of parts p0 to p1 with these keys: f(value, key, token). A warp
  // takes the runs of every kWarps-th slice as one list.
  template <class F>
  MSA_DEV void tokens(int p0, int p1, Keys k, F f) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = values.first(), tokens = a.slice;
    for (int s0 = warp; s0 < a.slices; s0 += 32 * kWarps) {
      const int slice = s0 + lane * kWarps;
      int from = 0, upto = 0;
      if (slice < a.slices) {
        const uint16_t* starts = a.starts + ((size_t)row * a.slices + slice) * kStarts;
        from = __ldcg(starts + p0), upto = __ldcg(starts + p1 + 1) - from;
      }
      const int n = upto;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      const int all = __shfl_sync(0xffffffffu, upto, 31);
      from -= upto - n;  // a token's place in its slice's order is its place in the list and this
      constexpr int kAhead = 4;
      for (int i0 = 0; i0 < all; i0 += 32 * kAhead) {
        int at[kAhead];  // token, or -1
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          // Its slice: the first lane whose list ends behind it.
          const int i = i0 + 32 * u + lane;
          int l = 0;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1)
            if (__shfl_sync(0xffffffffu, upto, l + d - 1) <= i) l += d;
          const int sl = s0 + l * kWarps, base = __shfl_sync(0xffffffffu, from, l);
          at[u] = -1;
          if (i < all) at[u] = first + sl * tokens + (int)__ldcg(a.order + ((size_t)row * a.slices + sl) * tokens + base + i);
        }
        float x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) x[u] = at[u] >= 0 ? Row32::value(values.row + (size_t)at[u] * 4) : 0.f;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (at[u] < 0) continue;
          const uint32_t key = key_of(x[u]);
          if (key >= k.lo && key <= k.hi) f(value_of(key), key, at[u]);
        }
      }
    }
  }

  // Running sums of the parts, of which a thread has two; the last one's is all.
  MSA_DEV void run(Mark* to, Mark m, Mark next, Mark last) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Mark upto{m.count + next.count, m.mass + next.mass};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, upto.count, d), y = __shfl_up_sync(0xffffffffu, upto.mass, d);
      if (lane >= d) upto.count += x, upto.mass += y;
    }
    __syncthreads();
    if (lane == 31) sm.warp[warp][0] = upto.count, sm.warp[warp][1] = upto.mass;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto.count += sm.warp[w][0], upto.mass += sm.warp[w][1];
    to[2 * threadIdx.x] = {upto.count - next.count, upto.mass - next.mass};
    to[2 * threadIdx.x + 1] = upto;
    if (threadIdx.x == kThreads - 1) to[kBins] = {upto.count + last.count, upto.mass + last.mass};
    __syncthreads();
  }

  // The first part of `marks` whose running sum, with `base`, passes; the last one if none before does.
  MSA_DEV int locate(const Mark* marks, Mark base, Kind kind, u64 t) {
    auto at = [&](int i) { return passes(kind, t, Mark{base.count + marks[i].count, base.mass + marks[i].mass}); };
    const int thread = kThreads - __syncthreads_count(at(2 * threadIdx.x + 1));
    return thread == kThreads ? kBins : 2 * thread + !at(2 * thread);
  }

  // Where the row's order passes t (which it does, or its end is told).
  MSA_DEV Answer find(Kind kind, u64 t) {
    const int part = locate(sm.top, Mark{0, 0}, kind, t);
    Mark base = part > 0 ? sm.top[part - 1] : Mark{0, 0}, upto = sm.top[part];
    if (kind == kCount && upto.count <= t) return {upto.count, upto.mass, 0u, 0};
    Keys k{0u, 0xffffffffu};
    for (bool all = true;; all = false) {
      if (!all && k.lo >= k.hi) return equals(kind, t, base, k.hi);
      const u64 many = upto.count - base.count;
      if (kind != kMassGt && many == 1) return {upto.count, upto.mass, 0u, 0};
      if (many <= kOrderCap) {
        if (threadIdx.x == 0) sm.order_n = 0u;
        __syncthreads();
        tokens(part, part, k, [&](float, uint32_t key, int idx) {
          const uint32_t n = atomicAdd(&sm.order_n, 1u);
          if (n < kOrderCap) sm.brought[n] = ((u64)key << 32) | (uint32_t)~idx;
        });
        __syncthreads();
        return order(kind, t, base);
      }
      // Too many: by their keys.
      if (all) k = keys_of(part);
      if (k.lo >= k.hi) continue;
      int shift = 0;
      while (((k.hi - k.lo) >> shift) >= (uint32_t)kBins) ++shift;
      sm.h.clear();
      tokens(part, part, k, [&](float v, uint32_t key, int) { sm.h.add((int)((k.hi - key) >> shift), scale.weight(sm.table, v)); });
      __syncthreads();
      run(sm.sub, sm.h.at(2 * threadIdx.x), sm.h.at(2 * threadIdx.x + 1), Mark{0, 0});
      const int p = min(locate(sm.sub, base, kind, t), kBins - 1);
      const Mark start = base;
      if (p > 0) base = {start.count + sm.sub[p - 1].count, start.mass + sm.sub[p - 1].mass};
      upto = {start.count + sm.sub[p].count, start.mass + sm.sub[p].mass};
      k.hi -= (uint32_t)p << shift;
      const uint32_t width = (1u << shift) - 1u;
      k.lo = max(k.lo, k.hi - min(k.hi, width));
      __syncthreads();
    }
  }

  // The tokens brought together, in their order, their running sum, and where it
  // passes t. Two threads count how many stand before one of them.
  MSA_DEV Answer order(Kind kind, u64 t, Mark base) {
    const int n = (int)min(sm.order_n, (uint32_t)kOrderCap), i = threadIdx.x, mine = i & (kOrderCap - 1), half = (n + 1) / 2;
    static_assert(kThreads == 2 * kOrderCap, "two threads for each");
    int before = 0;
    if (mine < n) {
      const u64 x = sm.brought[mine];
      const int from = i < kOrderCap ? 0 : half, to = i < kOrderCap ? half : n;
#pragma unroll 8
      for (int j = from; j < to; ++j) before += sm.brought[j] > x;
      if (i >= kOrderCap) sm.rank[mine] = before;
    }
    if (i == 0) sm.answer = {base.count, base.mass, 0u, -1};
    __syncthreads();
    if (i < n) {
      const u64 x = sm.brought[i];
      const int to = before + sm.rank[i];
      sm.sorted[to] = x;
      sm.sorted_w[to] = scale.weight(sm.table, value_of((uint32_t)(x >> 32)));
    }
    __syncthreads();
    if (i < 32) {
      u64 sum = base.mass;
      for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + i;
        u64 s = j < n ? sm.sorted_w[j] : 0ull;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const u64 o = __shfl_up_sync(0xffffffffu, s, d);
          if (i >= d) s += o;
        }
        s += sum;
        const Mark m{base.count + j + 1, s};
        const unsigned hit = __ballot_sync(0xffffffffu, j < n && (passes(kind, t, m) || j == n - 1));
        if (hit) {
          if (i == __ffs(hit) - 1) sm.answer = {m.count, m.mass, (uint32_t)(sm.sorted[j] >> 32), (int)~(uint32_t)sm.sorted[j]};
          break;
        }
        sum = __shfl_sync(0xffffffffu, s, 31);
      }
    }
    __syncthreads();
    const Answer got = sm.answer;
    __syncthreads();
    return got;
  }

  // Tokens of one key: how many of them, and which is the last.
  MSA_DEV Answer equals(Kind kind, u64 t, Mark base, uint32_t key) {
    const u64 w = scale.weight(sm.table, value_of(key)), r = equals_upto(kind, t, base, w);
    Answer got{base.count + r, base.mass + r * w, key, -1};
    if (kind != kMassGt) return got;
    if (threadIdx.x == 0) sm.answer = got;
    got.idx = nth_of_key<2, kWarps>(values, key, (unsigned)r, sm.counts, &sm.answer.idx);
    __syncthreads();
    return got;
  }
};

// A block for each row: its cuts, and its token.
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ uint4 answer_memory[];
  Shared& sm = *reinterpret_cast<Shared*>(answer_memory);
  const int tid = threadIdx.x, row = blockIdx.x;
  for (int i = tid; i < 1024; i += kThreads) sm.table[i] = kPowers.at[i];
  grid_dependency_wait();
  grid_dependents_launch();
  const Settings s = settings_of(a, row);
  if (s.none || (s.one && a.logprobs == nullptr)) {
    if (tid == 0) {
      a.tokens[row] = s.none ? -1 : s.top_idx;
      if (a.logprobs != nullptr) a.logprobs[row] = -INFINITY;
    }
    return;
  }
  Row r{sm, a, row, {row_of<2>(a, row), 0, a.vocab}, s.scale, s.top_key};
  {
    const uint32_t* count = a.parts_count + (size_t)row * kSampleParts;
    const u64* mass = a.parts_mass + (size_t)row * kSampleParts;
    r.run(sm.top, Mark{__ldcg(count + 2 * tid), __ldcg(mass + 2 * tid)}, Mark{__ldcg(count + 2 * tid + 1), __ldcg(mass + 2 * tid + 1)},
          Mark{__ldcg(count + kBins), __ldcg(mass + kBins)});
  }
  const u64 z = sm.top[kBins].mass;
  int token = s.top_idx;
  float chosen = s.scale.m;
  if (!s.one) {
    u64 sum = z, n = (u64)a.vocab;
    if (s.k > 0 && s.k < a.vocab) {
      const Answer x = r.find(kCount, (u64)s.k);
      sum = x.s, n = x.n;
    }
    const float p = a.top_p != nullptr ? __ldg(a.top_p + row) : 1.f;
    if (p < 1.f) {
      const Answer x = r.find(kMassGe, max(share_of(sum, fmaxf(p, 0.f), true), 1ull));
      sum = x.s, n = x.n;
    }
    const float min_p = a.min_p != nullptr ? __ldg(a.min_p + row) : 0.f;
    if (min_p > 0.f) {
      const float mp = fminf(min_p, 1.f);
      const u64 least = max(share_of(kOne, mp, true), 1ull);
      // The parts that the border may be in, token by token.
      const int mid = (int)fminf(log2f(mp) * -(float)kOctaveBins, (float)kBins), p0 = max(mid - 1, 0), p1 = min(mid + 1, kBins);
      const Mark before = p0 > 0 ? sm.top[p0 - 1] : Mark{0, 0};
      u64 count = 0, mass = 0;
      r.tokens(p0, p1, {0u, 0xffffffffu}, [&](float v, uint32_t, int) {
        const u64 w = s.scale.weight(sm.table, v);
        if (w >= least) mass += w, ++count;
      });
      const Mark m = block_join<false>(count, mass, sm.warp);
      if (before.count + m.count < n) n = before.count + m.count, sum = before.mass + m.mass;
    }
    const float u = __ldg(a.uniforms + row);
    const Answer x = r.find(kMassGt, u < 1.f ? min(share_of(sum, fmaxf(u, 0.f), false), sum - 1) : sum - 1);
    token = x.idx;
    chosen = value_of(x.key);
  }
  if (tid == 0) {
    a.tokens[row] = token;
    if (a.logprobs != nullptr) a.logprobs[row] = (s.scale.at_inf ? 0.f : (chosen - s.scale.m) / s.t) - logf((float)z * 0x1p-44f);
  }
}

template <int GROUPS>
cudaError_t launch_sort(const SampleArgs& a, dim3 slices, cudaStream_t s) {
  cudaError_t e = set_smem_limit((const void*)sample_sort_kernel<GROUPS>, sizeof(SortShared<GROUPS>));
  if (e == cudaSuccess) e = launch_dependent(sample_sort_kernel<GROUPS>, slices, kThreads, sizeof(SortShared<GROUPS>), s, a);
  return e;
}

}  // namespace

// 32 bits: slices of 8192 values, or of 2048 while those of 8192 do not fill
// the SMs twice (one row of 131072 in slices of 2048 keeps 64 SMs busy, of 8192
// 16). A row's first group may begin up to three values before it,
// unless rows are aligned.
SampleSlices sample_slices(int rows, int vocab, bool wide, bool aligned) {
  if (!wide) return {vocab, 0};
  const int slice = (long long)rows * ((vocab + 3 + 8191) / 8192) >= 304 ? 8192 : 2048;  // aligned or not
  return {slice, (vocab + (aligned ? 0 : 3) + slice - 1) / slice};
}

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  if (a.type != 2) return launch_sample_16(a, s);
  const dim3 slices((unsigned)a.rows * a.slices);
  cudaError_t e = launch_dependent(sample_top_kernel, slices, kThreads, 0, s, a);
  if (e != cudaSuccess) return e;
  e = a.slice == 2048 ? launch_sort<1>(a, slices, s) : launch_sort<4>(a, slices, s);
  if (e != cudaSuccess) return e;
  e = set_smem_limit((const void*)sample_kernel, sizeof(Shared));
  if (e != cudaSuccess) return e;
  return launch_dependent(sample_kernel, dim3(a.rows), kThreads, sizeof(Shared), s, a);
}

}  // namespace msa
