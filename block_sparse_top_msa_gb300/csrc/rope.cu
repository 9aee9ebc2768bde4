// Norms of queries and keys for each head with the position rotation, in one
// pass, forward (dense, or appending K and V to a paged cache) and backward.
//
// A row is the 128 values x of one (token, head). With r = (mean x^2 +
// eps)^(-1/2) the forward is y = R(x r w): R turns the pairs of the first
// `rotary` elements by the angles of the token's position, (a, b) -> (a c -
// b s, b c + a s). The backward with dy: u = R^T dy, dw = sum over tokens and
// heads of u x r, and with g = u w, dx = r (g - x r^2 mean(g x)).
//
// A team of 16 lanes holds a row in registers, eight elements a lane: the first
// and second elements A[0..3], B[0..3] of four pairs. With paired halves lane
// l of the rotary / 8 turned lanes takes elements 4l.. as A and rotary / 2 +
// 4l.. as B; with adjacent pairs 8l, 8l + 2, .. and 8l + 1, 8l + 3, ..; lanes
// past the rotary elements take 8l.. and 8l + 4... A turned lane's cosines are
// entries 4l..4l+3 of the position's table row, and only the sums over a row
// cross lanes. The weight is taken into the cosines and sines once for the
// heads of a token that a team turns: y = r (A wc - B ws', B wc' + A ws).
//
// The kernels are bound by memory, if the arithmetic is kept down (one
// operation at a time instead of pairs: 17 instructions an element, 58% of the
// issue slots, a tenth slower) and loads are not held up: forward 65536 tokens
// of 32 + 4 heads (1.24 GB in and out) take 200 us, 91% of the measured copy
// bandwidth; backward 32768 of 64 + 8 (1.82 GB) 285 us, 94%. 16-byte accesses by
// 8 lanes a row were slower (by 12% and 5%), as were loads one unit ahead in the
// backward (by a fifth: its registers).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace msa {
namespace {

constexpr int kTeam = 16;             // lanes per row
constexpr int kThreads = 256;
constexpr int kTeams = kThreads / kTeam;
constexpr int kBwdResident = 2;  // backward blocks an SM holds

// A lane's eight elements: A and B of pairs 0, 1 and of pairs 2, 3.
struct Own {
  float2 a0, a1, b0, b1;
};

MSA_DEV float2 mul2(float2 x, float2 y) { return __fmul2_rn(x, y); }
MSA_DEV float2 fma2(float2 x, float2 y, float2 z) { return __ffma2_rn(x, y, z); }
MSA_DEV float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }
MSA_DEV float2 both(float x) { return make_float2(x, x); }

template <bool F16>
MSA_DEV float2 unpack2(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// Two groups of four elements as they lie in memory, to and from pairs.
template <bool F16, bool ADJ>
MSA_DEV Own unpack(uint2 lo, uint2 hi, bool adj) {
  const float2 x0 = unpack2<F16>(lo.x), x1 = unpack2<F16>(lo.y), x2 = unpack2<F16>(hi.x), x3 = unpack2<F16>(hi.y);
  if (ADJ && adj)
    return {make_float2(x0.x, x1.x), make_float2(x2.x, x3.x), make_float2(x0.y, x1.y), make_float2(x2.y, x3.y)};
  return {x0, x1, x2, x3};
}
template <bool ADJ>
MSA_DEV void groups(const Own& y, bool adj, float2 (&g)[4]) {
  if (ADJ && adj) {
    g[0] = make_float2(y.a0.x, y.b0.x), g[1] = make_float2(y.a0.y, y.b0.y);
    g[2] = make_float2(y.a1.x, y.b1.x), g[3] = make_float2(y.a1.y, y.b1.y);
  } else {
    g[0] = y.a0, g[1] = y.a1, g[2] = y.b0, g[3] = y.b1;
  }
}
template <bool F16>
MSA_DEV uint2 pack4(float2 x, float2 y) {
  return make_uint2(pack_x2<F16>(x.x, x.y), pack_x2<F16>(y.x, y.y));
}
// Four values as E4M3 codes, round to nearest even, magnitudes above 448 as
// 448 (NaN stays NaN).
MSA_DEV uint32_t pack4_e4m3(float2 x, float2 y) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

MSA_DEV float team_sum(float v) {
#pragma unroll
  for (int s = kTeam / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}
MSA_DEV float dot_of(const Own& x, const Own& y) {
  const float2 s = fma2(x.a0, y.a0, fma2(x.a1, y.a1, fma2(x.b0, y.b0, mul2(x.b1, y.b1))));
  return s.x + s.y;
}
MSA_DEV Own scaled(const Own& x, float f) {
  const float2 g = both(f);
  return {mul2(x.a0, g), mul2(x.a1, g), mul2(x.b0, g), mul2(x.b1, g)};
}
MSA_DEV Own product(const Own& x, const Own& y) {
  return {mul2(x.a0, y.a0), mul2(x.a1, y.a1), mul2(x.b0, y.b0), mul2(x.b1, y.b1)};
}

// Where a lane's two groups of four elements lie, whether they turn, and
// whether their pairs are adjacent.
struct Place {
  int o0, o1;
  bool turned, adj;
};
template <bool ADJ>
MSA_DEV Place place_of(int l, int rotary) {
  const bool turned = 8 * l < rotary;
  if (turned && !ADJ) return {4 * l, rotary / 2 + 4 * l, true, false};
  return {8 * l, 8 * l + 4, turned, ADJ};
}
// The weight's elements, in pairs.
template <bool ADJ>
MSA_DEV Own weight_of(const float* w, const Place& at) {
  const float4 x = __ldg(reinterpret_cast<const float4*>(w + at.o0));
  const float4 y = __ldg(reinterpret_cast<const float4*>(w + at.o1));
  if (ADJ && at.adj)
    return {make_float2(x.x, x.z), make_float2(y.x, y.z), make_float2(x.y, x.w), make_float2(y.y, y.w)};
  return {make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(y.x, y.y), make_float2(y.z, y.w)};
}
// Cosines and sines of the lane's four pairs.
struct Angles {
  float2 c0, c1, s0, s1;
};
template <class Args>
MSA_DEV Angles angles_of(const Args& a, int l, int pos, bool turned) {
  if (!turned) return {both(1.f), both(1.f), both(0.f), both(0.f)};
  const float* row = a.cos_sin + (size_t)pos * a.rotary + 4 * l;
  const float4 c = __ldg(reinterpret_cast<const float4*>(row));
  const float4 s = __ldg(reinterpret_cast<const float4*>(row + a.rotary / 2));
  return {make_float2(c.x, c.y), make_float2(c.z, c.w), make_float2(s.x, s.y), make_float2(s.z, s.w)};
}

// Cache row of token t (right-aligned in its sequence): its page, row within
// the page, or page -1 where it has none. Tokens at or past cu_q[batch]
// belong to no sequence. The team's lanes probe together: first the place
// that equal lengths would give, then kTeam places a step.
MSA_DEV int cache_page(const RopeArgs& a, int l, int t, bool live, int& row) {
  const unsigned lane0 = (threadIdx.x & 31) & ~(kTeam - 1);
  const unsigned mask = ((1u << kTeam) - 1u) << lane0;
  int lo = min(a.batch - 1, (int)((long long)t * a.batch / a.tokens));
  int begin = __ldg(a.cu_q + lo), end = __ldg(a.cu_q + lo + 1);
  if (!(begin <= t && t < end)) {
    // The last lo with cu_q[lo] <= t (0 where there is none).
    int hi = a.batch;
    lo = 0;
    while (hi - lo > 1) {
      const int step = (hi - lo + kTeam) / (kTeam + 1);
      const int at = lo + (l + 1) * step;
      const bool below = at < hi && __ldg(a.cu_q + min(at, a.batch)) <= t;
      const int n = __popc(__ballot_sync(mask, below) & mask);
      lo += n * step;
      hi = min(hi, lo + step);
    }
    begin = __ldg(a.cu_q + lo), end = __ldg(a.cu_q + lo + 1);
  }
  if (!live || t < begin || t >= end) return -1;
  const long long pos = (long long)__ldg(a.seqused_k + lo) - end + t;
  if (pos < 0 || pos >= (long long)a.max_pages * kBlk) return -1;
  row = (int)(pos % kBlk);
  const int page = __ldg(a.page_table + (size_t)lo * a.max_pages + pos / kBlk);
  return page < a.num_pages ? page : -1;
}

// KV: 0 K to a dense output, 1 K and V to 16-bit pools, 2 to E4M3 pools.
// A team takes up to R heads of one token, all of Q, of K or of V, with every
// row's loads issued before the first is used.
template <bool F16, bool ADJ, int KV, int R>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int l = threadIdx.x % kTeam;
  const unsigned cq = (a.hq + R - 1) / R, ck = (a.hkv + R - 1) / R;
  const unsigned id = blockIdx.x * kTeams + threadIdx.x / kTeam;
  unsigned t_u, c;  // the token, and the team within it: Q's, then K's and V's
  if (KV) {
    // All tokens' K and V first: where they go takes several loads one after
    // the other to find, which then is under the work on Q.
    const unsigned kv = a.tokens * 2u * ck;
    const bool q = id >= kv;
    const unsigned per = q ? cq : 2u * ck, rest = q ? id - kv : id;
    t_u = rest / per;
    c = rest - t_u * per + (q ? 0u : cq);
  } else {
    t_u = id / (cq + ck);
    c = id - t_u * (cq + ck);
  }
  const bool live = t_u < (unsigned)a.tokens;
  const int t = live ? (int)t_u : 0;
  const int side = !live || c < cq ? 0 : c < cq + ck ? 1 : 2;
  const int h0 = (int)(side == 0 ? (live ? c : 0u) : side == 1 ? c - cq : c - cq - ck) * R;
  const int n = live ? min(R, (side == 0 ? a.hq : a.hkv) - h0) : 0;
  const uint16_t* src = static_cast<const uint16_t*>(side == 0 ? a.q : side == 1 ? a.k : a.v) +
                        (long long)t * (side == 0 ? a.q_stride : side == 1 ? a.k_stride : a.v_stride) +
                        h0 * kHeadDim;
  Place at = place_of<ADJ>(l, a.rotary);
  if (KV && side == 2) at = {8 * l, 8 * l + 4, false, ADJ};
  uint2 raw[R][2];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < n) {
      raw[i][0] = __ldcs(reinterpret_cast<const uint2*>(src + i * kHeadDim + at.o0));
      raw[i][1] = __ldcs(reinterpret_cast<const uint2*>(src + i * kHeadDim + at.o1));
    } else {
      raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
    }
  }
  const int pos = __ldg(a.positions + t);
  const bool known = pos >= 0 && pos < a.max_position;
  const Angles g = angles_of(a, l, pos, at.turned && known);
  // The weight times cosines, and times sines (of the other element's term).
  Own wc, ws;
  if (side < 2) {
    const Own w = weight_of<ADJ>(side == 0 ? a.wq : a.wk, at);
    wc = {mul2(w.a0, g.c0), mul2(w.a1, g.c1), mul2(w.b0, g.c0), mul2(w.b1, g.c1)};
    ws = {mul2(w.a0, g.s0), mul2(w.a1, g.s1), neg2(mul2(w.b0, g.s0)), neg2(mul2(w.b1, g.s1))};
  }
  // Destination: a dense row, or the cache row's address for head 0.
  int page = 0, crow = 0;
  bool write = live;
  if (KV) {
    if (side == 0) {
      write = live && t < __ldg(a.cu_q + a.batch);
    } else {
      page = cache_page(a, l, t, live && known, crow);
      write = page >= 0;
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const Own x = unpack<F16, ADJ>(raw[i][0], raw[i][1], at.adj);
    const float r = rsqrtf(team_sum(dot_of(x, x)) * (1.f / kHeadDim) + a.eps);
    Own y = x;
    if (!KV || side < 2) {
      if (at.turned) {
        y = scaled({fma2(x.a0, wc.a0, mul2(x.b0, ws.b0)), fma2(x.a1, wc.a1, mul2(x.b1, ws.b1)),
                    fma2(x.b0, wc.b0, mul2(x.a0, ws.a0)), fma2(x.b1, wc.b1, mul2(x.a1, ws.a1))}, r);
      } else {
        y = scaled(product(x, wc), r);
      }
    }
    if (i >= n || !write) continue;
    float2 e[4];
    groups<ADJ>(y, at.adj, e);
    if (side < 2 && !known) e[0] = e[1] = e[2] = e[3] = both(0.f);
    if (side == 0 || KV == 0) {
      uint16_t* dst = static_cast<uint16_t*>(side == 0 ? a.q_out : a.k_out) +
                      ((size_t)t * (side == 0 ? a.hq : a.hkv) + h0 + i) * kHeadDim;
      __stcs(reinterpret_cast<uint2*>(dst + at.o0), pack4<F16>(e[0], e[1]));
      __stcs(reinterpret_cast<uint2*>(dst + at.o1), pack4<F16>(e[2], e[3]));
    } else {
      const size_t row = ((size_t)page * a.hkv + h0 + i) * kBlk + crow;
      void* pool = side == 1 ? a.k_pool : a.v_pool;
      if (KV == 2) {
        uint8_t* dst = static_cast<uint8_t*>(pool) + row * kHeadDim;
        *reinterpret_cast<uint32_t*>(dst + at.o0) = pack4_e4m3(e[0], e[1]);
        *reinterpret_cast<uint32_t*>(dst + at.o1) = pack4_e4m3(e[2], e[3]);
      } else {
        uint16_t* dst = static_cast<uint16_t*>(pool) + row * kHeadDim;
        *reinterpret_cast<uint2*>(dst + at.o0) = side == 2 ? raw[i][0] : pack4<F16>(e[0], e[1]);
        *reinterpret_cast<uint2*>(dst + at.o1) = side == 2 ? raw[i][1] : pack4<F16>(e[2], e[3]);
      }
    }
  }
}

// Backward. Blocks [0, q_blocks) take Q rows, the others K rows, so that a
// thread's eight weight sums belong to one weight. Units are R heads of one
// token; a block strides over its side's units and leaves one row of 128
// partial sums, summed over its teams in a fixed order.
template <bool F16, bool ADJ, int R>
__global__ void __launch_bounds__(kThreads, kBwdResident) rope_bwd_kernel(const __grid_constant__ RopeBwdArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int l = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
  const bool kside = (int)blockIdx.x >= a.q_blocks;
  const int heads = kside ? a.hkv : a.hq;
  const unsigned chunks = (heads + R - 1) / R;
  const unsigned units = (unsigned)a.tokens * chunks;  // below 2^31, as tokens * heads are
  const unsigned blk = kside ? blockIdx.x - a.q_blocks : blockIdx.x;
  const unsigned blocks = kside ? gridDim.x - a.q_blocks : a.q_blocks;
  const uint16_t* x = static_cast<const uint16_t*>(kside ? a.k : a.q);
  const uint16_t* dy = static_cast<const uint16_t*>(kside ? a.dk_out : a.dq_out);
  uint16_t* dx = static_cast<uint16_t*>(kside ? a.dk : a.dq);
  const long long xs = kside ? a.k_stride : a.q_stride, ds = kside ? a.dk_stride : a.dq_stride;
  const Place at = place_of<ADJ>(l, a.rotary);
  const Own w = weight_of<ADJ>(kside ? a.wk : a.wq, at);
  Own dw = {both(0.f), both(0.f), both(0.f), both(0.f)};
  // Both teams of a warp walk the same number of units (the sums over a row
  // are warp shuffles).
  for (unsigned u0 = blk * kTeams; u0 < units; u0 += blocks * kTeams) {
    const unsigned u = u0 + team;
    const bool live = u < units;
    const unsigned t = live ? u / chunks : 0u;
    const int h0 = live ? (int)(u - t * chunks) * R : 0;
    const int n = live ? min(R, heads - h0) : 0;
    const uint16_t* xp = x + t * xs + h0 * kHeadDim;
    const uint16_t* dp = dy + ((size_t)t * heads + h0) * kHeadDim;
    uint2 rx[R][2], rd[R][2];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < n) {
        rx[i][0] = __ldcs(reinterpret_cast<const uint2*>(xp + i * kHeadDim + at.o0));
        rx[i][1] = __ldcs(reinterpret_cast<const uint2*>(xp + i * kHeadDim + at.o1));
        rd[i][0] = __ldcs(reinterpret_cast<const uint2*>(dp + i * kHeadDim + at.o0));
        rd[i][1] = __ldcs(reinterpret_cast<const uint2*>(dp + i * kHeadDim + at.o1));
      } else {
        rx[i][0] = rx[i][1] = rd[i][0] = rd[i][1] = make_uint2(0u, 0u);
      }
    }
    const int pos = __ldg(a.positions + t);
    const bool known = pos >= 0 && pos < a.max_position;
    const Angles g = angles_of(a, l, pos, at.turned && known);
    // The rows' sums first, all of them under way together.
    Own v[R];
    float ss[R], dot[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const Own f = unpack<F16, ADJ>(rx[i][0], rx[i][1], at.adj);
      v[i] = unpack<F16, ADJ>(rd[i][0], rd[i][1], at.adj);
      if (at.turned)
        v[i] = {fma2(v[i].a0, g.c0, mul2(v[i].b0, g.s0)), fma2(v[i].a1, g.c1, mul2(v[i].b1, g.s1)),
                fma2(v[i].b0, g.c0, neg2(mul2(v[i].a0, g.s0))), fma2(v[i].b1, g.c1, neg2(mul2(v[i].a1, g.s1)))};
      ss[i] = dot_of(f, f);
      dot[i] = dot_of(product(v[i], f), w);
    }
#pragma unroll
    for (int d = kTeam / 2; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], d);
        dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], d);
      }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const Own f = unpack<F16, ADJ>(rx[i][0], rx[i][1], at.adj);
      const float r = rsqrtf(ss[i] * (1.f / kHeadDim) + a.eps);
      const float k = -(r * dot[i]) * r * r * (1.f / kHeadDim);  // a row of zeros has dot 0, however large r
      if (known && i < n) {
        const Own fr = scaled(f, r);
        dw = {fma2(v[i].a0, fr.a0, dw.a0), fma2(v[i].a1, fr.a1, dw.a1), fma2(v[i].b0, fr.b0, dw.b0),
              fma2(v[i].b1, fr.b1, dw.b1)};
      }
      if (i < n) {
        const Own h = scaled(product(v[i], w), r);
        const float2 k2 = both(k);
        float2 e[4];
        groups<ADJ>({fma2(f.a0, k2, h.a0), fma2(f.a1, k2, h.a1), fma2(f.b0, k2, h.b0), fma2(f.b1, k2, h.b1)}, at.adj, e);
        if (!known) e[0] = e[1] = e[2] = e[3] = both(0.f);
        uint16_t* out = dx + t * ds + (h0 + i) * kHeadDim;
        __stcs(reinterpret_cast<uint2*>(out + at.o0), pack4<F16>(e[0], e[1]));
        __stcs(reinterpret_cast<uint2*>(out + at.o1), pack4<F16>(e[2], e[3]));
      }
    }
  }
  __shared__ float sums[kTeams][kHeadDim];
  {
    float2 e[4];
    groups<ADJ>(dw, at.adj, e);
    *reinterpret_cast<float4*>(&sums[team][at.o0]) = make_float4(e[0].x, e[0].y, e[1].x, e[1].y);
    *reinterpret_cast<float4*>(&sums[team][at.o1]) = make_float4(e[2].x, e[2].y, e[3].x, e[3].y);
  }
  __syncthreads();
  if (threadIdx.x < kHeadDim) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kTeams; ++i) s += sums[i][threadIdx.x];
    a.partials[(size_t)blockIdx.x * kHeadDim + threadIdx.x] = s;
  }
}

// Sums the blocks' partials, always in the same order: block (side, column
// group of 32), 32 rows of threads each taking every 32nd partial, then those
// 32 sums one after the other.
__global__ void __launch_bounds__(1024) rope_bwd_sum_kernel(const __grid_constant__ RopeBwdArgs a, int blocks) {
  grid_dependency_wait();
  grid_dependents_launch();
  const bool kside = blockIdx.x >= 4;
  const int col = (blockIdx.x & 3) * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  const int first = kside ? a.q_blocks : 0, last = kside ? blocks : a.q_blocks;
  float s = 0.f;
#pragma unroll 8
  for (int i = first + g; i < last; i += 32) s += a.partials[(size_t)i * kHeadDim + col];
  __shared__ float sums[32][32];
  sums[g][threadIdx.x & 31] = s;
  __syncthreads();
  if (g == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sums[i][threadIdx.x];
    (kside ? a.dwk : a.dwq)[col] = s;
  }
}

// Heads of a token in flight per team. Forward 4 / 6 / 8: 208 / 200 / 204 us on
// the size above. Backward, with the blocks an SM holds: 1 row 363, 2 rows 337
// (4 blocks), 4 rows 285 (2 blocks); more blocks than an SM holds gain nothing.
constexpr int kFwdRows = 6, kAppendRows = 4;
constexpr int kBwdRows = 4;

template <bool F16, bool ADJ, int KV>
cudaError_t launch_rope_r(const RopeArgs& a, cudaStream_t s) {
  constexpr int R = KV ? kAppendRows : kFwdRows;
  const long long per_token = (a.hq + R - 1) / R + (KV ? 2 : 1) * (long long)((a.hkv + R - 1) / R);
  const long long teams = (long long)a.tokens * per_token;
  return launch_dependent(rope_kernel<F16, ADJ, KV, R>, dim3((unsigned)((teams + kTeams - 1) / kTeams)), kThreads, 0, s,
                          a);
}
template <bool F16, int KV>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t s) {
  return a.interleaved ? launch_rope_r<F16, true, KV>(a, s) : launch_rope_r<F16, false, KV>(a, s);
}
template <bool F16>
cudaError_t launch_rope_bwd_t(const RopeBwdArgs& a, int blocks, cudaStream_t s) {
  return launch_dependent(a.interleaved ? rope_bwd_kernel<F16, true, kBwdRows> : rope_bwd_kernel<F16, false, kBwdRows>,
                          dim3(blocks), kThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  if (a.tokens == 0) return cudaSuccess;
  if (a.kv == 0) return a.f16 ? launch_rope_t<true, 0>(a, s) : launch_rope_t<false, 0>(a, s);
  if (a.kv == 2) return launch_rope_t<false, 2>(a, s);
  return a.f16 ? launch_rope_t<true, 1>(a, s) : launch_rope_t<false, 1>(a, s);
}

RopeBwdGrid rope_bwd_grid(long long tokens, int hq, int hkv) {
  // Enough blocks to fill the GPU, shared between the sides by their rows (each
  // side with rows has one), but no more than have a unit each.
  constexpr long long kMost = 152 * kBwdResident;
  const long long uq = tokens * ((hq + kBwdRows - 1) / kBwdRows), uk = tokens * ((hkv + kBwdRows - 1) / kBwdRows);
  const long long bq = (uq + kTeams - 1) / kTeams, bk = (uk + kTeams - 1) / kTeams;
  RopeBwdGrid g{(int)bq, (int)bk};
  if (bq + bk > kMost) {
    g.k_blocks = (int)std::min((kMost * uk + uq + uk - 1) / (uq + uk), kMost - 1);
    g.q_blocks = (int)(kMost - g.k_blocks);
  }
  return g;
}

cudaError_t launch_rope_bwd(const RopeBwdArgs& a, int k_blocks, cudaStream_t s) {
  const int blocks = a.q_blocks + k_blocks;
  if (blocks > 0) {
    const cudaError_t e = a.f16 ? launch_rope_bwd_t<true>(a, blocks, s) : launch_rope_bwd_t<false>(a, blocks, s);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(rope_bwd_sum_kernel, dim3(8), 1024, 0, s, a, blocks);
}

}  // namespace msa
