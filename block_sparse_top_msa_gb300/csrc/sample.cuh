// What the kernels of sampling share: exact weights, a row's values, the walk
// to the r-th of equal tokens. Their mathematics is in sample.cu.
#pragma once
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace msa {
namespace {

using u64 = unsigned long long;

constexpr int kOctaveBins = 32, kBins = kSampleParts - 1;  // of the first 32 octaves below the maximum; then one for the rest
constexpr float kNoWeight = -45.5f;  // 2^y below half of 2^-44
constexpr u64 kOne = 1ull << 44;
constexpr uint32_t kKeyNegInf = 0x007fffffu;

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
  int idx;       // (or which it is of its equals)
};
struct __align__(16) Mark {
  u64 count, mass;
};
MSA_DEV bool passes(Kind kind, u64 t, Mark m) {
  return kind == kCount ? m.count >= t : kind == kMassGe ? m.mass >= t : m.mass > t;
}
// How many tokens of weight w, behind `base`, until it passes t: at most 2^19,
// so that the quotient of two floats is off by one at most.
MSA_DEV u64 equals_upto(Kind kind, u64 t, Mark base, u64 w) {
  if (kind == kCount) return t - base.count;
  if (w == 0) return 1;
  const u64 rest = t - base.mass;
  u64 n = (u64)((float)rest / (float)w);
  while (n > 0 && n * w > rest) --n;
  while ((n + 1) * w <= rest) ++n;
  return kind == kMassGe ? n + (n * w < rest) : n + 1;  // at least, or more than, the rest
}
// f times the sum, f in [0, 1], rounded down, or up: exact.
MSA_DEV u64 share_of(u64 sum, float f, bool up) {
  const uint32_t bits = __float_as_uint(f);
  const int e = (int)(bits >> 23) & 255, shift = 150 - max(e, 1);  // f = m 2^-shift, shift >= 23
  const u64 m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u), lo = sum * m, hi = __umul64hi(sum, m);
  if (shift >= 128) return up && m != 0 && sum != 0 ? 1 : 0;  // hi has 24 bits
  if (shift >= 64) return (hi >> (shift - 64)) + (up && (lo | (hi & ((1ull << (shift - 64)) - 1))) != 0 ? 1 : 0);
  return ((hi << (64 - shift)) | (lo >> shift)) + (up && (lo & ((1ull << shift) - 1)) != 0 ? 1 : 0);
}

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
MSA_DEV Scale scale_of(float top, float t) {
  // log2(e) / T in two floats: log2(e) is the first of these and 1.92596e-8.
  const float lh = 1.44269502162933349609375f, ll = 1.925963033500e-8f;
  const float ch = lh / t, rest = fmaf(-ch, t, lh);
  return {top, ch, (rest + ll) / t, top == INFINITY};
}
// A row's temperature, as it counts, and whether its largest token is taken.
MSA_DEV bool temperature_of(const SampleArgs& a, int row, float& t) {
  t = a.temperature != nullptr ? __ldg(a.temperature + row) : 1.f;
  const bool greedy = !(t >= 1e-5f);
  t = greedy ? 1.f : fminf(t, 1e30f);
  return greedy;
}

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
template <int TYPE>
MSA_DEV const uint8_t* row_of(const SampleArgs& a, int row) {
  return static_cast<const uint8_t*>(a.logits) + (size_t)row * (size_t)a.stride * Values<TYPE>::kSize;
}

// The left-th token with this key, in the row itself: WARPS warps count them in
// a part of it, each in its share, until they have come to it; the share that
// has it is cut up in the same way, down to 32 groups of values, a lane each.
// counts: a word a warp; the block waits before and after.
template <int TYPE, int WARPS>
MSA_DEV int nth_of_key(const Values<TYPE>& v, uint32_t key, unsigned left, uint32_t* counts, int* answer) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float f = value_of(key);
  uint32_t pat, mask;  // a value is one of them where (value ^ pat) & mask is 0; zeros of both signs are
  if constexpr (TYPE == 2) {
    pat = __float_as_uint(f), mask = f == 0.f ? 0x7fffffffu : 0xffffffffu;
  } else {
    pat = TYPE == 0 ? __float_as_uint(f) >> 16 : __half_as_ushort(__float2half_rn(f));
    pat |= pat << 16, mask = f == 0.f ? 0x7fff7fffu : 0xffffffffu;
  }
  auto count = [&](int at, const uint4& x) -> unsigned {
    unsigned n = 0;
    if (v.inside(at)) {
      const uint32_t d[4] = {(x.x ^ pat) & mask, (x.y ^ pat) & mask, (x.z ^ pat) & mask, (x.w ^ pat) & mask};
      if constexpr (TYPE != 2) {  // none of the eight, mostly
        const uint32_t least = __vminu2(__vminu2(d[0], d[1]), __vminu2(d[2], d[3]));
        if ((least & 0xffffu) != 0u && (least >> 16) != 0u) return 0u;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (TYPE == 2) n += d[j] == 0u;
        else n += ((d[j] & 0xffffu) == 0u) + ((d[j] >> 16) == 0u);
      }
    } else {
      v.group(at, x, [&](float g, int) { n += g == f; });
    }
    return n;
  };
  constexpr int kAhead = 8;
  const int at0 = v.first();
  int g0 = 0, g1 = v.groups();
  while (g1 - g0 > 32) {
    const int each = min((g1 - g0 + WARPS - 1) / WARPS, 32 * kAhead), from = min(g0 + warp * each, g1), to = min(from + each, g1);
    unsigned mine = 0;
    {
      const int g = from + lane;
      uint4 x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int at = at0 + (g + 32 * u) * Values<TYPE>::kGroup;
        x[u] = g + 32 * u < to && v.inside(at) ? v.load(at) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (g + 32 * u < to) mine += count(at0 + (g + 32 * u) * Values<TYPE>::kGroup, x[u]);
    }
    mine = warp_add(mine);
    __syncthreads();
    if (lane == 0) counts[warp] = mine;
    __syncthreads();
    unsigned upto = lane < WARPS ? counts[lane] : 0u;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const int w = __popc(__ballot_sync(0xffffffffu, upto < left));  // warps that end before it
    const unsigned before = __shfl_sync(0xffffffffu, upto, max(w - 1, 0));
    if (w > 0) left -= before;
    if (w < 32) g0 = min(g0 + w * each, g1), g1 = min(g0 + each, g1);
    else g0 = min(g0 + WARPS * each, g1);  // not in this part
  }
  __syncthreads();
  if (warp == 0) {
    const int at = at0 + (g0 + lane) * Values<TYPE>::kGroup;
    const bool there = g0 + lane < g1;
    const uint4 x = there && v.inside(at) ? v.load(at) : make_uint4(0u, 0u, 0u, 0u);
    const unsigned n = there ? count(at, x) : 0u;
    unsigned upto = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    if (left <= upto && left > upto - n) {
      unsigned k = left - (upto - n);
      v.group(at, x, [&](float g, int idx) {
        if (g == f && --k == 0u) *answer = idx;
      });
    }
  }
  __syncthreads();
  return *answer;
}

}  // namespace
}  // namespace msa
