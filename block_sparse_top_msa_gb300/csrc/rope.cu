// Norms of queries and keys for each head with the position rotation, in one
// pass, forward (dense, or appending K and V to a paged cache) and backward.
//
// A row is the 128 values x of one (token, head). With r = (mean x^2 +
// eps)^(-1/2) the forward is y = R(x r w): R turns the pairs of the first
// `rotary` elements by the angles of the token's position, (a, b) -> (a c -
// b s, b c + a s). The backward with dy: u = R^T dy, dw = sum over tokens and
// heads of u x r, and with g = u w, dx = r (g - x r^2 mean(g x)).
//
// A team of 16 lanes holds a row in registers, eight elements a lane in two
// groups of four, placed so that both elements of a pair are the lane's own:
// with paired halves lane l of the rotary / 8 turned lanes takes elements 4l..
// and rotary / 2 + 4l.., otherwise (adjacent pairs, or elements past the
// rotary ones) 8l.. and 8l + 4... Either way a turned lane's cosines are
// entries 4l..4l+3 of the position's table row, and only the sums over a row
// cross lanes.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace msa {
namespace {

constexpr int kTeam = 16;             // lanes per row
constexpr int kThreads = 256;
constexpr int kTeams = kThreads / kTeam;

struct Row {
  float e[8];
};

template <bool F16>
MSA_DEV void unpack4(uint2 w, float* e) {
  if (F16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    e[0] = a.x, e[1] = a.y, e[2] = b.x, e[3] = b.y;
  } else {
    e[0] = __uint_as_float(w.x << 16), e[1] = __uint_as_float(w.x & 0xffff0000u);
    e[2] = __uint_as_float(w.y << 16), e[3] = __uint_as_float(w.y & 0xffff0000u);
  }
}
template <bool F16>
MSA_DEV uint2 pack4(const float* e) {
  return make_uint2(pack_x2<F16>(e[0], e[1]), pack_x2<F16>(e[2], e[3]));
}
// Four values as E4M3 codes, round to nearest even, magnitudes above 448 as
// 448 (NaN stays NaN).
MSA_DEV uint32_t pack4_e4m3(const float* e) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(e[0], e[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(e[2], e[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

MSA_DEV float team_sum(float v) {
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// Where a lane's two groups of four elements lie, and whether they turn.
struct Place {
  int o0, o1;
  bool turned;
};
MSA_DEV Place place_of(int l, int rotary, int interleaved) {
  const bool turned = 8 * l < rotary;
  if (turned && !interleaved) return {4 * l, rotary / 2 + 4 * l, true};
  return {8 * l, 8 * l + 4, turned};
}

// Turns the lane's four pairs by (c, s).
MSA_DEV void turn(Row& y, float4 c, float4 s, int interleaved) {
  const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
  auto pair = [&](int ia, int ib, int j) {
    const float p = y.e[ia], q = y.e[ib];
    y.e[ia] = p * cc[j] - q * ss[j];
    y.e[ib] = q * cc[j] + p * ss[j];
  };
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) pair(2 * j, 2 * j + 1, j);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) pair(j, j + 4, j);
  }
}

// Cache row of token t (right-aligned in its sequence): its page, row within
// the page, or page -1 where it has none. Tokens at or past cu_q[batch]
// belong to no sequence.
MSA_DEV int cache_page(const RopeArgs& a, int t, int& row) {
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.cu_q + mid) <= t) lo = mid; else hi = mid - 1;
  }
  const int end = __ldg(a.cu_q + lo + 1);
  if (t < __ldg(a.cu_q + lo) || t >= end) return -1;
  const long long pos = (long long)__ldg(a.seqused_k + lo) - end + t;
  if (pos < 0 || pos >= (long long)a.max_pages * kBlk) return -1;
  row = (int)(pos % kBlk);
  const int page = __ldg(a.page_table + (size_t)lo * a.max_pages + pos / kBlk);
  return page < a.num_pages ? page : -1;
}

// KV: 0 K to a dense output, 1 K and V to 16-bit pools, 2 to E4M3 pools.
// A team takes up to R heads of one token, all of Q, of K or of V, with every
// row's loads issued before the first is used.
template <bool F16, int KV, int R>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  const int l = threadIdx.x % kTeam;
  const int cq = (a.hq + R - 1) / R, ck = (a.hkv + R - 1) / R;
  const int per_token = cq + (KV ? 2 : 1) * ck;
  const unsigned id = blockIdx.x * kTeams + threadIdx.x / kTeam;
  const unsigned t_u = id / (unsigned)per_token;
  const bool live = t_u < (unsigned)a.tokens;
  const int t = live ? (int)t_u : 0;
  const int c = live ? (int)(id - t_u * per_token) : 0;
  const int side = c < cq ? 0 : c < cq + ck ? 1 : 2;
  const int h0 = (side == 0 ? c : side == 1 ? c - cq : c - cq - ck) * R;
  const int n = live ? min(R, (side == 0 ? a.hq : a.hkv) - h0) : 0;
  const uint16_t* src = static_cast<const uint16_t*>(side == 0 ? a.q : side == 1 ? a.k : a.v) +
                        (long long)t * (side == 0 ? a.q_stride : side == 1 ? a.k_stride : a.v_stride) +
                        h0 * kHeadDim;
  Place at = place_of(l, a.rotary, a.interleaved);
  if (side == 2) at = {8 * l, 8 * l + 4, false};
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
  float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at.turned && known) {
    const float* tab = a.cos_sin + (size_t)pos * a.rotary + 4 * l;
    cs = __ldg(reinterpret_cast<const float4*>(tab));
    sn = __ldg(reinterpret_cast<const float4*>(tab + a.rotary / 2));
  }
  float w[8];
  if (side < 2) {
    const float* wp = side == 0 ? a.wq : a.wk;
    const float4 w0 = __ldg(reinterpret_cast<const float4*>(wp + at.o0));
    const float4 w1 = __ldg(reinterpret_cast<const float4*>(wp + at.o1));
    w[0] = w0.x, w[1] = w0.y, w[2] = w0.z, w[3] = w0.w;
    w[4] = w1.x, w[5] = w1.y, w[6] = w1.z, w[7] = w1.w;
  }
  // Destination: a dense row, or the cache row's address for head 0.
  int page = 0, crow = 0;
  bool write = live;
  if (KV) {
    if (side == 0) {
      write = live && t < __ldg(a.cu_q + a.batch);
    } else {
      page = live && known ? cache_page(a, t, crow) : -1;
      write = page >= 0;
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    Row y;
    unpack4<F16>(raw[i][0], y.e);
    unpack4<F16>(raw[i][1], y.e + 4);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(y.e[j], y.e[j], ss);
    ss = team_sum(ss);
    if (side < 2) {
      const float r = rsqrtf(ss * (1.f / kHeadDim) + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) y.e[j] = y.e[j] * r * w[j];
      if (at.turned) turn(y, cs, sn, a.interleaved);
      if (!known) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y.e[j] = 0.f;
      }
    }
    if (i >= n || !write) continue;
    if (side == 0 || KV == 0) {
      uint16_t* dst = static_cast<uint16_t*>(side == 0 ? a.q_out : a.k_out) +
                      ((size_t)t * (side == 0 ? a.hq : a.hkv) + h0 + i) * kHeadDim;
      *reinterpret_cast<uint2*>(dst + at.o0) = pack4<F16>(y.e);
      *reinterpret_cast<uint2*>(dst + at.o1) = pack4<F16>(y.e + 4);
    } else {
      const size_t row = ((size_t)page * a.hkv + h0 + i) * kBlk + crow;
      void* pool = side == 1 ? a.k_pool : a.v_pool;
      if (KV == 2) {
        uint8_t* dst = static_cast<uint8_t*>(pool) + row * kHeadDim;
        *reinterpret_cast<uint32_t*>(dst + at.o0) = pack4_e4m3(y.e);
        *reinterpret_cast<uint32_t*>(dst + at.o1) = pack4_e4m3(y.e + 4);
      } else {
        uint16_t* dst = static_cast<uint16_t*>(pool) + row * kHeadDim;
        *reinterpret_cast<uint2*>(dst + at.o0) = side == 2 ? raw[i][0] : pack4<F16>(y.e);
        *reinterpret_cast<uint2*>(dst + at.o1) = side == 2 ? raw[i][1] : pack4<F16>(y.e + 4);
      }
    }
  }
}

// Backward. Blocks [0, q_blocks) take Q rows, the others K rows, so that a
// thread's eight weight sums belong to one weight. Units are R heads of one
// token; a block strides over its side's units and leaves one row of 128
// partial sums, summed over its teams in a fixed order.
template <bool F16, int R>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const __grid_constant__ RopeBwdArgs a) {
  const int l = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
  const bool kside = (int)blockIdx.x >= a.q_blocks;
  const int heads = kside ? a.hkv : a.hq;
  const int chunks = (heads + R - 1) / R;
  const long long units = (long long)a.tokens * chunks;
  const int blk = kside ? (int)blockIdx.x - a.q_blocks : (int)blockIdx.x;
  const int blocks = kside ? (int)gridDim.x - a.q_blocks : a.q_blocks;
  const uint16_t* x = static_cast<const uint16_t*>(kside ? a.k : a.q);
  const uint16_t* dy = static_cast<const uint16_t*>(kside ? a.dk_out : a.dq_out);
  uint16_t* dx = static_cast<uint16_t*>(kside ? a.dk : a.dq);
  const long long xs = kside ? a.k_stride : a.q_stride, ds = kside ? a.dk_stride : a.dq_stride;
  const Place at = place_of(l, a.rotary, a.interleaved);
  float w[8], dw[8];
  {
    const float* wp = kside ? a.wk : a.wq;
    const float4 w0 = __ldg(reinterpret_cast<const float4*>(wp + at.o0));
    const float4 w1 = __ldg(reinterpret_cast<const float4*>(wp + at.o1));
    w[0] = w0.x, w[1] = w0.y, w[2] = w0.z, w[3] = w0.w;
    w[4] = w1.x, w[5] = w1.y, w[6] = w1.z, w[7] = w1.w;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = 0.f;
  // Both teams of a warp walk the same number of units (the sums over a row
  // are warp shuffles).
  for (long long u0 = (long long)blk * kTeams; u0 < units; u0 += (long long)blocks * kTeams) {
    const long long u = u0 + team;
    const bool live = u < units;
    const int t = live ? (int)(u / chunks) : 0;
    const int h0 = live ? (int)(u - (long long)t * chunks) * R : 0;
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
    float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
    if (at.turned && known) {
      const float* tab = a.cos_sin + (size_t)pos * a.rotary + 4 * l;
      cs = __ldg(reinterpret_cast<const float4*>(tab));
      sn = __ldg(reinterpret_cast<const float4*>(tab + a.rotary / 2));
      sn = make_float4(-sn.x, -sn.y, -sn.z, -sn.w);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      Row f, g;
      unpack4<F16>(rx[i][0], f.e);
      unpack4<F16>(rx[i][1], f.e + 4);
      unpack4<F16>(rd[i][0], g.e);
      unpack4<F16>(rd[i][1], g.e + 4);
      if (at.turned) turn(g, cs, sn, a.interleaved);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(f.e[j], f.e[j], ss);
        dot = fmaf(g.e[j] * w[j], f.e[j], dot);
      }
      ss = team_sum(ss);
      dot = team_sum(dot);
      const float r = rsqrtf(ss * (1.f / kHeadDim) + a.eps);
      const float k = r * r * dot * (1.f / kHeadDim);
      const bool counts = known && i < n;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (counts) dw[j] = fmaf(g.e[j] * r, f.e[j], dw[j]);
        g.e[j] = known ? r * (g.e[j] * w[j] - f.e[j] * k) : 0.f;
      }
      if (i >= n) continue;
      uint16_t* out = dx + t * ds + (h0 + i) * kHeadDim;
      *reinterpret_cast<uint2*>(out + at.o0) = pack4<F16>(g.e);
      *reinterpret_cast<uint2*>(out + at.o1) = pack4<F16>(g.e + 4);
    }
  }
  __shared__ float sums[kTeams][kHeadDim];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sums[team][at.o0 + j] = dw[j];
    sums[team][at.o1 + j] = dw[j + 4];
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
  const bool kside = blockIdx.x >= 4;
  const int col = (blockIdx.x & 3) * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  const int first = kside ? a.q_blocks : 0, last = kside ? blocks : a.q_blocks;
  float s = 0.f;
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

constexpr int kBwdRows = 2;  // heads of a token in flight per team

template <bool F16, int KV>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t s) {
  constexpr int R = 4;
  const long long per_token = (a.hq + R - 1) / R + (KV ? 2 : 1) * (long long)((a.hkv + R - 1) / R);
  const long long teams = (long long)a.tokens * per_token;
  rope_kernel<F16, KV, R><<<(unsigned)((teams + kTeams - 1) / kTeams), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  if (a.tokens == 0) return cudaSuccess;
  if (a.kv == 0) return a.f16 ? launch_rope_t<true, 0>(a, s) : launch_rope_t<false, 0>(a, s);
  if (a.kv == 2) return launch_rope_t<false, 2>(a, s);
  return a.f16 ? launch_rope_t<true, 1>(a, s) : launch_rope_t<false, 1>(a, s);
}

RopeBwdGrid rope_bwd_grid(long long tokens, int hq, int hkv) {
  // Enough blocks to fill the GPU (8 of 256 threads fit an SM), shared between the sides by their rows, but no
  // more than have a unit each.
  constexpr long long kMost = 152 * 8;
  const long long uq = tokens * ((hq + kBwdRows - 1) / kBwdRows), uk = tokens * ((hkv + kBwdRows - 1) / kBwdRows);
  const long long bq = (uq + kTeams - 1) / kTeams, bk = (uk + kTeams - 1) / kTeams;
  RopeBwdGrid g{(int)bq, (int)bk};
  if (bq + bk > kMost) {
    g.k_blocks = (int)((kMost * uk + uq + uk - 1) / (uq + uk));
    g.q_blocks = (int)(kMost - g.k_blocks);
  }
  return g;
}

cudaError_t launch_rope_bwd(const RopeBwdArgs& a, int k_blocks, cudaStream_t s) {
  const int blocks = a.q_blocks + k_blocks;
  if (blocks > 0) {
    if (a.f16) rope_bwd_kernel<true, kBwdRows><<<blocks, kThreads, 0, s>>>(a);
    else rope_bwd_kernel<false, kBwdRows><<<blocks, kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  rope_bwd_sum_kernel<<<8, 1024, 0, s>>>(a, blocks);
  return cudaGetLastError();
}

}  // namespace msa
