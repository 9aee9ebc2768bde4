// Tokens from 16-bit logits (the questions and their mathematics: sample.cu).
//
// There are 65536 different logits, so a block counts how often each comes in
// its row, in 16-bit counters in shared memory, and has the row sorted by that:
// one addition a token is all the work that grows with the row. Counters stand
// in the order of falling logits, 64 to a chunk, and the chunks' running counts
// and sums (a weight for each logit that comes) answer each question in two
// steps, which chunk and which logit in it, without another look at the row.
// Only the token itself, as the r-th of its equals, takes one: from L2. 512 rows
// of 200019 (bf16): 177 us, 1.16 TB/s. Bound by the counting, 36000 clocks a row:
// an addition of 32 lanes takes 5.7 passes through the banks. Slices counted apart,
// and the row read again for each cut, took 797 us.
#include "sample.cuh"

namespace msa {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kChunks = 1024;  // of 64 counters
constexpr int kAhead = 7;      // groups of eight values that a thread has on their way
// A counter that has come to kSpill is put into a list and begins anew. Between
// two looks at the counters kAhead * 8 * kThreads values are counted, so that a
// counter, and those of both zeros together, stay below 2 kSpill + 57344 = 2^16.
constexpr uint32_t kSpill = 4096;
constexpr int kSpilled = kMaxVocab / kSpill;
static_assert(kChunks == kThreads && 2 * kSpill + kAhead * 8 * kThreads == 65536, "16-bit counters");

// Logits as places in their falling order, and back.
MSA_DEV uint32_t places_of(uint32_t two) { return two ^ (((~two >> 15) & 0x00010001u) * 0x7fffu); }
template <int TYPE>
MSA_DEV float logit_at(uint32_t place) {
  const uint32_t bits = place ^ ((place & 0x8000u) ? 0u : 0x7fffu);
  return TYPE == 1 ? __half2float(__ushort_as_half((unsigned short)bits)) : __uint_as_float(bits << 16);
}

struct Shared16 {
  u64 table[1024];
  Mark run[kChunks];  // running counts and sums of the chunks
  __align__(16) u64 warp[kWarps][2];
  uint32_t counts[kWarps];
  uint32_t spilled;
  uint32_t spilled_at[kSpilled], spilled_n[kSpilled];
  uint32_t top;
  Answer answer;
  int idx;
  uint32_t some[kChunks / 32];  // chunks with any logit, a bit each
  uint16_t list[kChunks];
  uint32_t listed;
};

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 1) sample_16_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ uint4 counters[];  // 65536 of 16 bits
  __shared__ Shared16 sm;
  constexpr uint32_t kFirst = TYPE == 0 ? 0x007fu : 0x03ffu;  // of +inf; before it NaN
  constexpr uint32_t kEnd = TYPE == 0 ? 0xff80u : 0xfc00u;    // of -inf; behind it NaN
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.x;
  uint32_t* words = reinterpret_cast<uint32_t*>(counters);
  for (int i = tid; i < 8192; i += kThreads) counters[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int i = tid; i < 1024; i += kThreads) sm.table[i] = kPowers.at[i];
  if (tid == 0) sm.spilled = 0u, sm.top = ~0u, sm.idx = 0, sm.listed = 0u;
  if (tid < kChunks / 32) sm.some[tid] = 0u;
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_launch();
  float t;
  const bool greedy = temperature_of(a, row, t);
  const int top_k = a.top_k != nullptr ? __ldg(a.top_k + row) : 0;
  const bool one = greedy || top_k == 1;  // the largest is taken
  const Values<TYPE> v{row_of<TYPE>(a, row), 0, a.vocab};
  const int n = v.groups(), at0 = v.first();

  if (one && a.logprobs == nullptr) {
    uint32_t key = 0u;
    int idx = 0;
    v.each([&](float f, int i) {
      const uint32_t k = key_of(f);
      if (k > key) key = k, idx = i;
    });
    const u64 best = warp_max64(((u64)key << 32) | (uint32_t)~idx);
    if (lane == 0) sm.warp[warp][0] = best;
    __syncthreads();
    if (warp == 0) {
      const u64 all = warp_max64(sm.warp[lane][0]);
      if (lane == 0) a.tokens[row] = (uint32_t)(all >> 32) <= kKeyNegInf ? -1 : (int)~(uint32_t)all;
    }
    return;
  }

  // ------------------------------------------------------------------- counts
  {
    uint4 x[kAhead];
    auto load = [&](int g) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = g + u * kThreads, at = at0 + k * 8;
        x[u] = k < n && v.inside(at) ? v.load(at) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    auto count = [&](uint32_t place) { atomicAdd(words + (place >> 1), (place & 1u) ? 65536u : 1u); };
    load(tid);
    for (int g0 = 0;; g0 += kAhead * kThreads) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = g0 + tid + u * kThreads, at = at0 + k * 8;
        if (k >= n) break;
        if (v.inside(at)) {
          const uint32_t w[4] = {places_of(x[u].x), places_of(x[u].y), places_of(x[u].z), places_of(x[u].w)};
#pragma unroll
          for (int j = 0; j < 4; ++j) count(w[j] & 0xffffu), count(w[j] >> 16);
        } else {
          for (int j = 0; j < 8; ++j)
            if (at + j >= 0 && at + j < a.vocab)
              count(places_of(__ldg(reinterpret_cast<const unsigned short*>(v.row + (long long)(at + j) * 2))) & 0xffffu);
        }
      }
      if (g0 + kAhead * kThreads >= n) break;
      load(g0 + kAhead * kThreads + tid);
      __syncthreads();
      for (int i = tid; i < 8192; i += kThreads) {
        uint4 c = counters[i];
        if (((c.x | c.y | c.z | c.w) & 0xf000f000u) == 0u) continue;
        uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
          const uint32_t many = (w[j >> 1] >> (16 * (j & 1))) & 0xffffu;
          if (many < kSpill) continue;
          const uint32_t to = atomicAdd(&sm.spilled, 1u), place = 8u * i + j;
          if (to < kSpilled) sm.spilled_at[to] = place == 0x8000u ? 0x7fffu : place, sm.spilled_n[to] = many;
          w[j >> 1] &= (j & 1) ? 0xffffu : 0xffff0000u;
        }
        counters[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncthreads();
    }
  }
  __syncthreads();
  // -0 is 0.
  if (tid == 0) words[0x3fff] += words[0x4000] << 16, words[0x4000] &= 0xffff0000u;
  const int spilled = (int)sm.spilled;
  __syncthreads();
  {
    uint32_t top = ~0u;
#pragma unroll
    for (int i = tid; i < 8192; i += kThreads) {
      const uint4 c = counters[i];
      const bool any = (c.x | c.y | c.z | c.w) != 0u;
      const unsigned bits = __ballot_sync(0xffffffffu, any);  // of four chunks, eight lanes each
      if (bits != 0u && lane < 4 && (bits >> (8 * lane) & 0xffu)) atomicOr(&sm.some[i >> 8], 1u << (((i >> 5) * 4 + lane) & 31));
      if (!any || 8u * i > top) continue;
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int j = 7; j >= 0; --j) {
        const uint32_t place = 8u * i + j;
        if (((w[j >> 1] >> (16 * (j & 1))) & 0xffffu) != 0u && place >= kFirst && place < kEnd) top = min(top, place);
      }
    }
    if (tid < spilled) atomicOr(&sm.some[sm.spilled_at[tid] >> 11], 1u << (sm.spilled_at[tid] >> 6 & 31));
    if (tid < spilled && sm.spilled_at[tid] >= kFirst && sm.spilled_at[tid] < kEnd) top = min(top, sm.spilled_at[tid]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = min(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0 && top != ~0u) atomicMin(&sm.top, top);
  }
  __syncthreads();
  const uint32_t top = sm.top;
  if (top == ~0u) {
    if (tid == 0) {
      a.tokens[row] = -1;
      if (a.logprobs != nullptr) a.logprobs[row] = -INFINITY;
    }
    return;
  }
  const Scale scale = scale_of(logit_at<TYPE>(top), t);

  // ------------------------------------------------------------ running sums
  // A lane's two logits of a chunk: how often they come, and their weights.
  struct Two {
    uint32_t n[2];
    u64 w[2];
  };
  auto two_of = [&](int chunk) -> Two {
    const uint32_t word = words[chunk * 32 + lane], place = (uint32_t)chunk * 64u + 2u * lane;
    Two x{{word & 0xffffu, word >> 16}, {0ull, 0ull}};
    for (int e = 0; e < spilled; ++e)
      if (sm.spilled_at[e] == place) x.n[0] += sm.spilled_n[e];
      else if (sm.spilled_at[e] == place + 1u) x.n[1] += sm.spilled_n[e];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (place + j < kFirst || place + j >= kEnd) x.n[j] = 0u;
      if (x.n[j] != 0u) x.w[j] = scale.weight(sm.table, logit_at<TYPE>(place + j));
    }
    return x;
  };
  // Sums of the warp's lanes by 26 bits at a time, so that 32 of them fit in 32.
  auto add_lanes = [](u64 x) -> u64 {
    const u64 low = __reduce_add_sync(0xffffffffu, (uint32_t)x & 0x3ffffffu), mid = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 26) & 0x3ffffffu);
    return low + (mid << 26) + ((u64)__reduce_add_sync(0xffffffffu, (uint32_t)(x >> 52)) << 52);
  };
  sm.run[tid] = {0, 0};
  if (sm.some[warp] >> lane & 1u) sm.list[atomicAdd(&sm.listed, 1u)] = (uint16_t)tid;
  __syncthreads();
  for (int i = warp; i < (int)sm.listed; i += kWarps) {
    const int chunk = sm.list[i];
    const Two x = two_of(chunk);
    const u64 mass = add_lanes(x.n[0] * x.w[0] + x.n[1] * x.w[1]);
    const uint32_t count = __reduce_add_sync(0xffffffffu, x.n[0] + x.n[1]);
    if (lane == 0) sm.run[chunk] = {count, mass};
  }
  __syncthreads();
  {
    Mark m = sm.run[tid];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const u64 x = __shfl_up_sync(0xffffffffu, m.count, d), y = __shfl_up_sync(0xffffffffu, m.mass, d);
      if (lane >= d) m.count += x, m.mass += y;
    }
    if (lane == 31) sm.warp[warp][0] = m.count, sm.warp[warp][1] = m.mass;
    __syncthreads();
    for (int w = 0; w < warp; ++w) m.count += sm.warp[w][0], m.mass += sm.warp[w][1];
    sm.run[tid] = m;
  }
  __syncthreads();
  const u64 z = sm.run[kChunks - 1].mass;

  // ---------------------------------------------------------------- questions
  // Where the row's order passes p. One warp looks into the chunk.
  auto find = [&](Kind kind, u64 p) -> Answer {
    const int chunk = kChunks - __syncthreads_count(passes(kind, p, sm.run[tid]));
    if (chunk == kChunks) return {sm.run[kChunks - 1].count, z, 0u, 0};
    if (warp == 0) {
      const Two x = two_of(chunk);
      const Mark base = chunk > 0 ? sm.run[chunk - 1] : Mark{0, 0};
      Mark upto{x.n[0] + x.n[1], x.n[0] * x.w[0] + x.n[1] * x.w[1]};
      const Mark own = upto;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 c = __shfl_up_sync(0xffffffffu, upto.count, d), m = __shfl_up_sync(0xffffffffu, upto.mass, d);
        if (lane >= d) upto.count += c, upto.mass += m;
      }
      upto.count += base.count, upto.mass += base.mass;
      const unsigned hits = __ballot_sync(0xffffffffu, passes(kind, p, upto));
      if (lane == __ffs(hits) - 1) {
        Mark before{upto.count - own.count, upto.mass - own.mass};
        const Mark mid{before.count + x.n[0], before.mass + x.n[0] * x.w[0]};
        const int j = passes(kind, p, mid) ? 0 : 1;
        if (j == 1) before = mid;
        const u64 w = j == 0 ? x.w[0] : x.w[1], r = equals_upto(kind, p, before, w);
        sm.answer = {before.count + r, before.mass + r * w, (uint32_t)chunk * 64u + 2u * lane + j, (int)r};
      }
    }
    __syncthreads();
    const Answer got = sm.answer;
    __syncthreads();
    return got;
  };
  uint32_t place = top;
  unsigned which = 1;  // of its equals
  if (!one) {
    u64 sum = z, kept = (u64)a.vocab;
    if (top_k > 0 && top_k < a.vocab) {
      const Answer x = find(kCount, (u64)top_k);
      sum = x.s, kept = x.n;
    }
    const float p = a.top_p != nullptr ? __ldg(a.top_p + row) : 1.f;
    if (p < 1.f) {
      const Answer x = find(kMassGe, max(share_of(sum, fmaxf(p, 0.f), true), 1ull));
      sum = x.s, kept = x.n;
    }
    const float min_p = a.min_p != nullptr ? __ldg(a.min_p + row) : 0.f;
    if (min_p > 0.f) {
      const float mp = fminf(min_p, 1.f);
      const u64 least = max(share_of(kOne, mp, true), 1ull);
      // The last chunk whose first logit has that weight, and those of its logits.
      const uint32_t first = 64u * tid;
      const int chunk =
          __syncthreads_count(first <= top || (first < kEnd && scale.weight(sm.table, logit_at<TYPE>(first)) >= least)) - 1;
      const Two x = two_of(chunk);
      u64 count = 0, mass = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (x.w[j] >= least) count += x.n[j], mass += x.n[j] * x.w[j];
      count = warp_add(count), mass = add_lanes(mass);
      if (chunk > 0) count += sm.run[chunk - 1].count, mass += sm.run[chunk - 1].mass;
      if (count < kept) kept = count, sum = mass;
    }
    const float u = __ldg(a.uniforms + row);
    const Answer x = find(kMassGt, u < 1.f ? min(share_of(sum, fmaxf(u, 0.f), false), sum - 1) : sum - 1);
    place = x.key, which = (unsigned)x.idx;
  }
  const float chosen = logit_at<TYPE>(place);
  const int token = nth_of_key<TYPE, kWarps>(v, key_of(chosen), which, sm.counts, &sm.idx);
  if (tid == 0) {
    a.tokens[row] = token;
    if (a.logprobs != nullptr) a.logprobs[row] = (scale.at_inf ? 0.f : (chosen - scale.m) / t) - logf((float)z * 0x1p-44f);
  }
}

template <int TYPE>
cudaError_t launch_t(const SampleArgs& a, cudaStream_t s) {
  cudaError_t e = set_smem_limit((const void*)sample_16_kernel<TYPE>, 131072);
  if (e == cudaSuccess) e = launch_dependent(sample_16_kernel<TYPE>, dim3(a.rows), kThreads, 131072, s, a);
  return e;
}

}  // namespace

cudaError_t launch_sample_16(const SampleArgs& a, cudaStream_t s) {
  return a.type == 1 ? launch_t<1>(a, s) : launch_t<0>(a, s);
}

}  // namespace msa
