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
// Three kernels, each launched under the tail of the one before: the largest
// of each slice of a row; the slices' histograms, added up in the row's; and a
// block a row that answers. In 16 bits there are few logits: a slice counts how
// often each of the 65536 comes, one addition a token, and weighs those that
// come. In 32 bits each token is weighed, and the slice lists its first tokens
// for the last kernel, which reads the row again for what the lists do not hold.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace msa {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kOctaveBins = 32, kBins = kSampleParts - 1;  // of the first 16 octaves below the maximum; then one for the rest
constexpr int kCountThreads = 1024;
constexpr int kOrderCap = 256;       // tokens that are ordered at once
constexpr float kNoWeight = -45.5f;  // 2^y below half of 2^-44
constexpr u64 kOne = 1ull << 44;
constexpr uint32_t kKeyNegInf = 0x007fffffu;
static_assert(kBins == kThreads, "a thread for each part");

// 2^(i / 1024) times 2^44, rounded: products of 2^(1 / 2), 2^(1 / 4), ...
// 2^(1 / 1024), which are held times 2^63.
struct Powers {
  u64 at[1024];
};
constexpr Powers make_powers() {
  constexpr u64 roots[10] = {0xb504f333f9de6484ull, 0x9837f0518db8a96full, 0x8b95c1e3ea8bd6e7ull, 0x85aac367cc487b15ull,
                             0x82cd8698ac2ba1d7ull, 0x8164d1f3bc030773ull, 0x80b1ed4fd999ab6cull, 0x8058d7d2d5e5f6b1ull,
                             0x802c6436d0e04f51ull, 0x8016302f17467628ull};
  Powers p{};
  for (int i = 0; i < 1024; ++i) {
    u64 t = 1ull << 63;
    for (int j = 0; j < 10; ++j)
      if (i & (512 >> j)) {
        // The upper half of the product of two 64-bit numbers, by 32-bit halves.
        const u64 a = t >> 32, b = t & 0xffffffffu, c = roots[j] >> 32, d = roots[j] & 0xffffffffu;
        const u64 mid = a * d + ((b * d) >> 32), low = (mid & 0xffffffffu) + b * c;
        t = (a * c + (mid >> 32) + (low >> 32)) << 1;
      }
    p.at[i] = (t + (1ull << 18)) >> 19;
  }
  return p;
}
__device__ const Powers kPowers = make_powers();

// What the passes ask for.
enum Kind { kCount, kMassGe, kMassGt };  // n >= k, S(n) >= t, S(n) > t
struct Answer {
  u64 n, s;      // how many tokens up to it, and their sum
  uint32_t key;  // kMassGt: the last of them
  int idx;
};
struct __align__(16) Mark {
  u64 count, mass;
};
struct Histogram {
  uint32_t cnt[kBins + 1], lo[kBins + 1], hi[kBins + 1];
  MSA_DEV void clear() {
    for (int i = threadIdx.x; i <= kBins; i += blockDim.x) cnt[i] = lo[i] = hi[i] = 0u;
    __syncthreads();
  }
  MSA_DEV void add(int part, u64 w, uint32_t n = 1u) {
    atomicAdd(&cnt[part], n);
    const uint32_t low = (uint32_t)w, old = atomicAdd(&lo[part], low);
    const uint32_t high = (uint32_t)(w >> 32) + (old + low < old ? 1u : 0u);
    if (high) atomicAdd(&hi[part], high);
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

MSA_DEV uint32_t key_of(float f) {
  if (f != f) return kKeyNegInf;  // NaN: never taken
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 is 0
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
MSA_DEV float value_of(uint32_t key) { return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu)); }

// Of a row: its maximum and log2(e) / T in two parts.
struct Scale {
  float m, ch, cl;
  bool at_inf;  // the maximum is infinite: those tokens share all mass
  // 1024 times log2 of w, rounded; never rises as f falls. f is not NaN; `far`
  // at least where the weight is 0.
  static constexpr int kFar = 1 << 20;
  MSA_DEV int steps(float f) const {
    const float y = fmaxf((f - m) * ch, -1000.f);
    return at_inf ? (f == m ? 0 : -kFar) : __float_as_int(fmaf(y, 1024.f, 12582912.f)) - 0x4b400000;
  }
  // What part of the histogram it is in.
  MSA_DEV int part(float f) const { return min(-steps(f) >> 5, kBins); }
  // w in 2^-44. x - m and its product with log2(e) / T in two floats each, so
  // that what is left for the cubic is exact to 2^-36.
  MSA_DEV u64 weight(const u64* table, float f) const {
    const float dh = f - m, yh = dh * ch;
    if (at_inf) return f == m ? kOne : 0ull;
    if (!(yh > kNoWeight)) return 0ull;
    const float b = dh - f, dl = (f - (dh - b)) - (m + b);
    const float yl = fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch);
    const float magic = 12582912.f, kf = yh * 1024.f + magic;
    const int k = __float_as_int(kf) - 0x4b400000;
    const float r = fmaf(kf - magic, -1.f / 1024.f, yh) + yl;
    const float q = r * fmaf(r, fmaf(r, 0.05550410866f, 0.2402265070f), 0.6931471806f);
    const u64 t = table[k & 1023];
    const int qi = __float2int_rn(q * 137438953472.f);  // 2^37
    const u64 x = t + (u64)(((long long)(int)(t >> 14) * qi) >> 23);
    return (((x << 1) >> -(k >> 10)) + 1) >> 1;
  }
};

// Values [begin, end) of a row, in 16-byte groups of its memory; the first and
// last group may hold less of it.
template <int TYPE>  // 0 bf16, 1 fp16, 2 fp32
struct Values {
  static constexpr int kGroup = TYPE == 2 ? 4 : 8, kSize = 16 / kGroup;
  const uint8_t* row;
  int begin, end;
  static MSA_DEV float value(const uint8_t* p) {
    if constexpr (TYPE == 2) return __ldg(reinterpret_cast<const float*>(p));
    const unsigned short w = __ldg(reinterpret_cast<const unsigned short*>(p));
    return TYPE == 1 ? __half2float(__ushort_as_half(w)) : __uint_as_float((uint32_t)w << 16);
  }
  static MSA_DEV float element(const uint32_t (&w)[4], int j) {
    if constexpr (TYPE == 2) return __uint_as_float(w[j]);
    if constexpr (TYPE == 1) return __half2float(__ushort_as_half((unsigned short)(w[j >> 1] >> (16 * (j & 1)))));
    return __uint_as_float((j & 1) ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
  }
  // Token of the first value of group 0, which begins on 16 bytes at or before `begin`.
  MSA_DEV int first() const {
    return begin - (int)((reinterpret_cast<uintptr_t>(row + (size_t)begin * kSize) & 15) / kSize);
  }
  MSA_DEV int groups() const { return (end - first() + kGroup - 1) / kGroup; }
  MSA_DEV bool inside(int at) const { return at >= begin && at + kGroup <= end; }
  MSA_DEV uint4 load(int at) const { return __ldg(reinterpret_cast<const uint4*>(row + (long long)at * kSize)); }
  // Calls f(value, token) for the values from `at` on, which are of one group:
  // those in v, where all of them are there.
  template <class F>
  MSA_DEV void group(int at, const uint4& v, F f) const {
    if (inside(at)) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < kGroup; ++j) f(element(w, j), at + j);
    } else {
#pragma unroll 1
      for (int j = 0; j < kGroup; ++j)
        if (at + j >= begin && at + j < end) f(value(row + (long long)(at + j) * kSize), at + j);
    }
  }
  // Groups g0, g0 + step, ... below n, four loads at a time; tokens ascend.
  template <class F>
  MSA_DEV void steps(int g0, int n, int step, F f) const {
    const int at0 = first();
    for (int g = g0; g < n; g += 4 * step) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = at0 + (g + u * step) * kGroup;
        v[u] = g + u * step < n && inside(at) ? load(at) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (g + u * step < n) group(at0 + (g + u * step) * kGroup, v[u], f);
    }
  }
  // Of a thread's groups.
  template <class F>
  MSA_DEV void each(F f) const {
    steps(threadIdx.x, groups(), blockDim.x, f);
  }
};

template <class T>
MSA_DEV T warp_add(T v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
MSA_DEV u64 warp_max64(u64 v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const u64 o = __shfl_xor_sync(0xffffffffu, v, d);
    v = o > v ? o : v;
  }
  return v;
}
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
  s.t = a.temperature != nullptr ? __ldg(a.temperature + row) : 1.f;
  const bool greedy = !(s.t >= 1e-5f);
  if (greedy) s.t = 1.f;
  s.t = fminf(s.t, 1e30f);
  s.k = a.top_k != nullptr ? __ldg(a.top_k + row) : 0;
  s.none = s.top_key <= kKeyNegInf;
  s.one = s.none || greedy || s.k == 1;
  // log2(e) / T in two floats: log2(e) is the first of these and 1.92596e-8.
  const float lh = 1.44269502162933349609375f, ll = 1.925963033500e-8f;
  const float ch = lh / s.t, rest = fmaf(-ch, s.t, lh), top = value_of(s.top_key);
  s.scale = {top, ch, (rest + ll) / s.t, top == INFINITY};
  return s;
}
template <int TYPE>
MSA_DEV const uint8_t* row_of(const SampleArgs& a, int row) {
  return static_cast<const uint8_t*>(a.logits) + (size_t)row * (size_t)a.stride * Values<TYPE>::kSize;
}

// The largest value of a slice and its first token: (key, ~token) as one
// number. The row's histogram is emptied.
template <int TYPE>
__global__ void __launch_bounds__(kThreads) sample_top_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ __align__(16) u64 sw[kWarps][2];
  const int slice = blockIdx.x % a.slices, row = blockIdx.x / a.slices;
  grid_dependency_wait();
  grid_dependents_launch();
  for (int i = slice * kThreads + threadIdx.x; i < kSampleParts; i += a.slices * kThreads) {
    a.parts_count[(size_t)row * kSampleParts + i] = 0u;
    a.parts_mass[(size_t)row * kSampleParts + i] = 0ull;
  }
  const int begin = slice * a.slice;
  const Values<TYPE> v{row_of<TYPE>(a, row), begin, min(begin + a.slice, a.vocab)};
  uint32_t key = 0u;
  int idx = 0;
  v.each([&](float f, int i) {
    const uint32_t k = key_of(f);
    if (k > key) key = k, idx = i;
  });
  const Mark m = block_join<true>(((u64)key << 32) | (uint32_t)~idx, 0, sw);
  if (threadIdx.x == 0) a.best[(size_t)row * a.slices + slice] = m.count;
}

// A slice's histogram, of 32-bit logits, and the list of the tokens in its first
// parts: as many parts as fill its share of the row's list.
__global__ void __launch_bounds__(kThreads, 2) sample_weigh_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ u64 table[1024];
  __shared__ Histogram h;
  __shared__ int s_upto[kWarps];
  __shared__ uint32_t s_n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slice = blockIdx.x % a.slices, row = blockIdx.x / a.slices;
  for (int i = tid; i < 1024; i += kThreads) table[i] = kPowers.at[i];
  if (tid == 0) s_n = 0u;
  h.clear();
  grid_dependency_wait();
  grid_dependents_launch();
  const Settings s = settings_of(a, row);
  if (s.none || (s.one && a.logprobs == nullptr)) return;
  const int begin = slice * a.slice;
  const Values<2> v{row_of<2>(a, row), begin, min(begin + a.slice, a.vocab)};
  u64 rest_mass = 0;
  uint32_t rest_count = 0;
  v.each([&](float f, int) {
    if (!(f > -INFINITY)) {
      ++rest_count;
      return;
    }
    const u64 w = s.scale.weight(table, f);
    const int part = s.scale.part(f);
    if (part < kBins && !s.one) h.add(part, w);
    else rest_mass += w, ++rest_count;
  });
  rest_mass = warp_add(rest_mass), rest_count = warp_add(rest_count);
  if (lane == 0 && rest_count > 0) h.add(kBins, rest_mass, rest_count);
  __syncthreads();
  h.flush(a, row);
  if (s.one) return;
  // Where the running count passes what the list holds.
  int upto = (int)h.cnt[tid];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) s_upto[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += s_upto[w];
  const int parts = __syncthreads_count(upto <= a.listed);
  uint2* list = a.list + ((size_t)row * a.slices + slice) * a.listed;
  v.each([&](float f, int i) {
    if (!(f > -INFINITY) || s.scale.part(f) >= parts) return;
    const uint32_t n = atomicAdd(&s_n, 1u);
    if (n < (uint32_t)a.listed) list[n] = make_uint2(key_of(f), (uint32_t)i);
  });
  __syncthreads();
  if (tid == 0) a.list_info[(size_t)row * a.slices + slice] = make_int2((int)min(s_n, (uint32_t)a.listed), parts);
}

// A slice's histogram, of 16-bit logits: how often each comes, two counters to a
// word (a slice has fewer than 65536), then the weight of each that comes.
template <int TYPE>
__global__ void __launch_bounds__(kCountThreads, 1) sample_count_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ uint4 counts[];  // 65536 times 16 bits
  __shared__ u64 table[1024];
  __shared__ Histogram h;
  const int tid = threadIdx.x, lane = tid & 31;
  const int slice = blockIdx.x % a.slices, row = blockIdx.x / a.slices;
  uint32_t* words = reinterpret_cast<uint32_t*>(counts);
  for (int i = tid; i < 8192; i += kCountThreads) counts[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int i = tid; i < 1024; i += kCountThreads) table[i] = kPowers.at[i];
  h.clear();
  grid_dependency_wait();
  grid_dependents_launch();
  const Settings s = settings_of(a, row);
  if (s.none || (s.one && a.logprobs == nullptr)) return;
  const int begin = slice * a.slice, end = min(begin + a.slice, a.vocab);
  const Values<TYPE> v{row_of<TYPE>(a, row), begin, end};
  auto count = [&](uint32_t bits) { atomicAdd(words + (bits >> 1), (bits & 1u) ? 65536u : 1u); };
  const int n = v.groups(), at0 = v.first();
  for (int g = tid; g < n; g += 4 * kCountThreads) {
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = g + u * kCountThreads, at = at0 + k * 8;
      x[u] = k < n && v.inside(at) ? v.load(at) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = g + u * kCountThreads, at = at0 + k * 8;
      if (k >= n) break;
      if (v.inside(at)) {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) count(w[j] & 0xffffu), count(w[j] >> 16);
      } else {
        for (int j = 0; j < 8; ++j)
          if (at + j >= begin && at + j < end)
            count(__ldg(reinterpret_cast<const unsigned short*>(v.row + (long long)(at + j) * 2)));
      }
    }
  }
  __syncthreads();
  u64 rest_mass = 0;
  uint32_t rest_count = 0;
  for (int i = tid; i < 8192; i += kCountThreads) {
    const uint4 c = counts[i];
    if ((c.x | c.y | c.z | c.w) == 0u) continue;
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
      const uint32_t times = (w[j >> 1] >> (16 * (j & 1))) & 0xffffu, bits = 8u * i + j;
      if (times == 0u) continue;
      const float f = TYPE == 1 ? __half2float(__ushort_as_half((unsigned short)bits)) : __uint_as_float(bits << 16);
      if (!(f > -INFINITY)) {
        rest_count += times;
        continue;
      }
      const u64 mass = s.scale.weight(table, f) * times;
      const int part = s.scale.part(f);
      if (part < kBins && !s.one) h.add(part, mass, times);
      else rest_mass += mass, rest_count += times;
    }
  }
  rest_mass = warp_add(rest_mass), rest_count = warp_add(rest_count);
  if (lane == 0 && rest_count > 0) h.add(kBins, rest_mass, rest_count);
  __syncthreads();
  h.flush(a, row);
}

struct Shared {
  u64 table[1024];
  Histogram h;
  Mark top[kBins + 1];  // the row's histogram as running sums
  Mark sub[kBins + 1];  // that of a part
  __align__(16) u64 warp[kWarps][2];
  int listed;  // the parts below this one are in the lists
  uint32_t order_n;
  uint32_t order_key[kOrderCap];
  int order_idx[kOrderCap];
  uint32_t sort_key[kOrderCap];
  int sort_idx[kOrderCap];
  u64 sort_w[kOrderCap];
  u64 ask;
  Answer answer;
};

template <int TYPE>
struct Row {
  Shared& sm;
  const SampleArgs& a;
  int row;
  Values<TYPE> values;
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
  MSA_DEV Keys keys_of(int part) {
    Keys k{lowest_key(part), part > 0 ? lowest_key(part - 1) - 1u : top_key};
    // Of 16-bit logits, only those that there are: the low bits are all 0, below
    // zero all 1.
    if constexpr (TYPE != 2) {
      constexpr uint32_t low = TYPE == 0 ? 0xffffu : 0x1fffu;
      k.lo = k.lo >= 0x80000000u ? (k.lo + low) & ~low : k.lo | low;
      if (k.hi >= 0x80000000u) k.hi &= ~low;
      else if ((k.hi & low) != low) k.hi = k.hi > low ? (k.hi & ~low) - 1u : 0u;
    }
    return k;
  }

  // The tokens with these keys, which are of one part: f(value, key, token).
  template <class F>
  MSA_DEV void tokens(int part, Keys k, F f) const {
    if (part < sm.listed) {
      // Loads of four steps at a time; what stands behind a list's end is not looked at.
      constexpr int kAhead = 4;
      const uint2* list = a.list + (size_t)row * a.slices * a.listed;
      const int2* info = a.list_info + (size_t)row * a.slices;
      const int all = a.slices * a.listed;
      for (int i0 = threadIdx.x; i0 < all; i0 += kAhead * kThreads) {
        uint2 x[kAhead];
        int n[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int i = i0 + u * kThreads;
          n[u] = i < all ? __ldcg(&info[i / a.listed].x) : 0;
          x[u] = i < all ? __ldcg(list + i) : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if ((i0 + u * kThreads) % a.listed >= n[u] || x[u].x < k.lo || x[u].x > k.hi) continue;
          f(value_of(x[u].x), x[u].x, (int)x[u].y);
        }
      }
    } else {
      values.each([&](float v, int i) {
        const uint32_t key = key_of(v);
        if (key >= k.lo && key <= k.hi) f(value_of(key), key, i);
      });
    }
  }

  // Running sums of the parts; the last one's is all.
  MSA_DEV void run(Mark* to, Mark m, Mark last) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, m.count, d), y = __shfl_up_sync(0xffffffffu, m.mass, d);
      if (lane >= d) m.count += x, m.mass += y;
    }
    __syncthreads();
    if (lane == 31) sm.warp[warp][0] = m.count, sm.warp[warp][1] = m.mass;
    __syncthreads();
    for (int w = 0; w < warp; ++w) m.count += sm.warp[w][0], m.mass += sm.warp[w][1];
    to[threadIdx.x] = m;
    if (threadIdx.x == kThreads - 1) to[kBins] = {m.count + last.count, m.mass + last.mass};
    __syncthreads();
  }

  static MSA_DEV bool passes(Kind kind, u64 t, Mark m) {
    return kind == kCount ? m.count >= t : kind == kMassGe ? m.mass >= t : m.mass > t;
  }
  // The first part of `marks` whose running sum, with `base`, passes; the last one if none before does.
  MSA_DEV int locate(const Mark* marks, Mark base, Kind kind, u64 t) {
    auto at = [&](int i) { return passes(kind, t, Mark{base.count + marks[i].count, base.mass + marks[i].mass}); };
    return kBins - __syncthreads_count(at(threadIdx.x));
  }

  // Where the row's order passes t (which it does).
  MSA_DEV Answer find(Kind kind, u64 t) {
    const int part = locate(sm.top, Mark{0, 0}, kind, t);
    Mark base = part > 0 ? sm.top[part - 1] : Mark{0, 0}, upto = sm.top[part];
    if (kind == kCount && upto.count == t) return {upto.count, upto.mass, 0u, 0};
    if (kind != kMassGt && upto.count - base.count == 1) return {upto.count, upto.mass, 0u, 0};
    Keys k = keys_of(part);
    while (true) {
      if (k.lo >= k.hi) return equals(kind, t, base, k.hi);
      const u64 many = upto.count - base.count;
      if (kind != kMassGt && many == 1) return {upto.count, upto.mass, 0u, 0};
      if (many <= kOrderCap) {
        if (threadIdx.x == 0) sm.order_n = 0u;
        __syncthreads();
        tokens(part, k, [&](float, uint32_t key, int idx) {
          const uint32_t n = atomicAdd(&sm.order_n, 1u);
          if (n < kOrderCap) sm.order_key[n] = key, sm.order_idx[n] = idx;
        });
        __syncthreads();
        return order(kind, t, base);
      }
      // Too many: by their keys.
      int shift = 0;
      while (((k.hi - k.lo) >> shift) >= (uint32_t)kBins) ++shift;
      sm.h.clear();
      tokens(part, k, [&](float v, uint32_t key, int) { sm.h.add((int)((k.hi - key) >> shift), scale.weight(sm.table, v)); });
      __syncthreads();
      run(sm.sub, sm.h.at(threadIdx.x), Mark{0, 0});
      const int p = min(locate(sm.sub, base, kind, t), kBins - 1);
      const Mark start = base;
      if (p > 0) base = {start.count + sm.sub[p - 1].count, start.mass + sm.sub[p - 1].mass};
      upto = {start.count + sm.sub[p].count, start.mass + sm.sub[p].mass};
      k.hi -= (uint32_t)p << shift;
      const uint32_t width = (1u << shift) - 1u;
      k.lo = max(k.lo, k.hi - min(k.hi, width));
      if constexpr (TYPE != 2) {  // down to one logit in 16 bits
        constexpr uint32_t low = TYPE == 0 ? 0xffffu : 0x1fffu;
        if (k.hi - k.lo <= low) k.lo = k.hi = k.hi >= 0x80000000u ? k.hi & ~low : k.lo | low;
      }
      __syncthreads();
    }
  }

  // The tokens brought together, in their order, their running sum, and where it passes t.
  MSA_DEV Answer order(Kind kind, u64 t, Mark base) {
    const int n = (int)min(sm.order_n, (uint32_t)kOrderCap), i = threadIdx.x;
    if (i < n) {
      const uint32_t key = sm.order_key[i];
      const int idx = sm.order_idx[i];
      int place = 0;
      for (int j = 0; j < n; ++j) place += sm.order_key[j] > key || (sm.order_key[j] == key && sm.order_idx[j] < idx);
      sm.sort_key[place] = key;
      sm.sort_idx[place] = idx;
      sm.sort_w[place] = scale.weight(sm.table, value_of(key));
    }
    if (i == 0) sm.answer = {base.count, base.mass, 0u, -1};
    __syncthreads();
    if (i < 32) {
      u64 sum = base.mass;
      for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + i;
        u64 s = j < n ? sm.sort_w[j] : 0ull;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const u64 o = __shfl_up_sync(0xffffffffu, s, d);
          if (i >= d) s += o;
        }
        s += sum;
        const Mark m{base.count + j + 1, s};
        const unsigned hit = __ballot_sync(0xffffffffu, j < n && (passes(kind, t, m) || j == n - 1));
        if (hit) {
          if (i == __ffs(hit) - 1) sm.answer = {m.count, m.mass, sm.sort_key[j], sm.sort_idx[j]};
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
    const u64 w = scale.weight(sm.table, value_of(key));
    const u64 r = kind == kCount ? t - base.count : w == 0 ? 1 : kind == kMassGe ? (t - base.mass + w - 1) / w : (t - base.mass) / w + 1;
    Answer got{base.count + r, base.mass + r * w, key, -1};
    if (kind != kMassGt) return got;
    // The r-th of them by number, in the row itself: each warp counts them in a
    // sixteenth, and the one that has it is cut up in the same way, down to 32
    // groups of values, a lane each.
    if (threadIdx.x == 0) sm.answer = got;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int g0 = 0, g1 = values.groups();
    unsigned left = (unsigned)r;
    while (g1 - g0 > 32) {
      const int each = (g1 - g0 + kWarps - 1) / kWarps, from = min(g0 + warp * each, g1), to = min(from + each, g1);
      unsigned mine = 0;
      values.steps(from + lane, to, 32, [&](float f, int) { mine += key_of(f) == key; });
      mine = warp_add(mine);
      __syncthreads();
      if (lane == 0) sm.warp[warp][0] = mine;
      __syncthreads();
      unsigned before = 0;
      int w = 0;
      while (w < kWarps - 1 && before + (unsigned)sm.warp[w][0] < left) before += (unsigned)sm.warp[w++][0];
      left -= before;
      g0 = min(g0 + w * each, g1), g1 = min(g0 + each, g1);
    }
    if (warp == 0) {
      const int at = values.first() + (g0 + lane) * Values<TYPE>::kGroup;
      const bool there = g0 + lane < g1;
      const uint4 v = there && values.inside(at) ? values.load(at) : make_uint4(0u, 0u, 0u, 0u);
      unsigned n = 0;
      if (there) values.group(at, v, [&](float f, int) { n += key_of(f) == key; });
      unsigned upto = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      if (left <= upto && left > upto - n) {
        unsigned k = left - (upto - n);
        values.group(at, v, [&](float f, int idx) {
          if (key_of(f) == key && --k == 0u) sm.answer.idx = idx;
        });
      }
    }
    __syncthreads();
    got = sm.answer;
    __syncthreads();
    return got;
  }
};

// A block for each row: its cuts, and its token.
template <int TYPE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ Shared sm;
  const int tid = threadIdx.x, row = blockIdx.x;
  for (int i = tid; i < 1024; i += kThreads) sm.table[i] = kPowers.at[i];
  if (tid == 0) sm.listed = TYPE == 2 ? kBins : 0;
  __syncthreads();
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
  Row<TYPE> r{sm, a, row, {row_of<TYPE>(a, row), 0, a.vocab}, s.scale, s.top_key};
  {
    const uint32_t* count = a.parts_count + (size_t)row * kSampleParts;
    const u64* mass = a.parts_mass + (size_t)row * kSampleParts;
    if (TYPE == 2 && !s.one)
      for (int i = tid; i < a.slices; i += kThreads)
        atomicMin(&sm.listed, __ldcg(&a.list_info[(size_t)row * a.slices + i].y));
    r.run(sm.top, Mark{__ldcg(count + tid), __ldcg(mass + tid)}, Mark{__ldcg(count + kBins), __ldcg(mass + kBins)});
  }
  const u64 z = sm.top[kBins].mass;
  int token = s.top_idx;
  float chosen = s.scale.m;
  if (!s.one) {
    // What one thread works out in 64 bits, for all.
    auto ask = [&](auto f) -> u64 {
      if (tid == 0) sm.ask = f();
      __syncthreads();
      const u64 t = sm.ask;
      __syncthreads();
      return t;
    };
    u64 sum = z, n = (u64)a.vocab;
    if (s.k > 0 && s.k < a.vocab) {
      const Answer x = r.find(kCount, (u64)s.k);
      sum = x.s, n = x.n;
    }
    const float p = a.top_p != nullptr ? __ldg(a.top_p + row) : 1.f;
    if (p < 1.f) {
      const u64 t = ask([&] { return max((u64)ceil((double)fmaxf(p, 0.f) * (double)sum), 1ull); });
      const Answer x = r.find(kMassGe, t);
      sum = x.s, n = x.n;
    }
    const float mp = a.min_p != nullptr ? fminf(__ldg(a.min_p + row), 1.f) : 0.f;
    if (mp > 0.f) {
      const u64 least = ask([&] { return max((u64)ceil((double)mp * (double)kOne), 1ull); });
      // The parts that the border may be in, token by token.
      const int mid = (int)fminf(log2f(mp) * -(float)kOctaveBins, (float)kBins), p0 = max(mid - 1, 0), p1 = min(mid + 1, kBins);
      const Mark before = p0 > 0 ? sm.top[p0 - 1] : Mark{0, 0};
      u64 count = 0, mass = 0;
      for (int part = p0; part <= p1; ++part) {
        if (sm.top[part].count == (part > 0 ? sm.top[part - 1].count : 0ull)) continue;
        r.tokens(part, r.keys_of(part), [&](float v, uint32_t, int) {
          const u64 w = s.scale.weight(sm.table, v);
          if (w >= least) mass += w, ++count;
        });
      }
      const Mark m = block_join<false>(count, mass, sm.warp);
      if (before.count + m.count < n) n = before.count + m.count, sum = before.mass + m.mass;
    }
    const float u = __ldg(a.uniforms + row);
    const u64 at = ask([&] { return u < 1.f ? min((u64)floor((double)fmaxf(u, 0.f) * (double)sum), sum - 1) : sum - 1; });
    const Answer x = r.find(kMassGt, at);
    token = x.idx;
    chosen = value_of(x.key);
  }
  if (tid == 0) {
    a.tokens[row] = token;
    if (a.logprobs != nullptr) a.logprobs[row] = (s.scale.at_inf ? 0.f : (chosen - s.scale.m) / s.t) - logf((float)z * 0x1p-44f);
  }
}

template <int TYPE>
cudaError_t launch_t(const SampleArgs& a, cudaStream_t s) {
  const dim3 slices((unsigned)a.rows * a.slices);
  cudaError_t e = launch_dependent(sample_top_kernel<TYPE>, slices, kThreads, 0, s, a);
  if (e != cudaSuccess) return e;
  if constexpr (TYPE == 2) {
    e = launch_dependent(sample_weigh_kernel, slices, kThreads, 0, s, a);
  } else {
    e = set_smem_limit((const void*)sample_count_kernel<TYPE>, 131072);
    if (e != cudaSuccess) return e;
    e = launch_dependent(sample_count_kernel<TYPE>, slices, kCountThreads, 131072, s, a);
  }
  if (e != cudaSuccess) return e;
  return launch_dependent(sample_kernel<TYPE>, dim3(a.rows), kThreads, 0, s, a);
}

}  // namespace

// 16 bits: slices of 65528 values at most, and of a quarter of that at least,
// as each takes 65536 counters to clear and look through. 32 bits: of 32768,
// and 2048. Smaller ones while the row's slices do not fill the SMs.
SampleSlices sample_slices(int rows, int vocab, bool wide) {
  const int most = wide ? 32768 : 65528, least = wide ? 2048 : 16384, fill = wide ? 608 : 304;
  int n = (vocab + most - 1) / most;
  while ((long long)rows * n < fill && (vocab + 2 * n - 1) / (2 * n) >= least) n *= 2;
  const int slice = ((vocab + n - 1) / n + 7) / 8 * 8;
  n = (vocab + slice - 1) / slice;
  return {slice, n, wide ? max(32, min(256, 4096 / n)) : 0};
}

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  return a.type == 2 ? launch_t<2>(a, s) : a.type == 1 ? launch_t<1>(a, s) : launch_t<0>(a, s);
}

}  // namespace msa
