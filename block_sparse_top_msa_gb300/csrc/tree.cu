// Attention of drafted tokens in trees over a paged cache.
//
// A unit is up to 2 W consecutive query tokens of one request (W = 128 / G
// tokens fill the 128 rows of an MMA tile) with one KV head; it attends over
// the union of its tokens' listed blocks, each row to its own blocks and to
// the drafts its mask names. Drafts of one request choose much the same
// blocks, so a block is brought to shared memory once for both tiles: that
// halves the cache traffic and the E4M3 conversions (units of one tile: 78 us
// against 64 for 32 requests of 16 tokens with 64 query heads, 4 KV heads and
// 16 listed blocks, 376 against 305 for 128 E4M3 requests of 8 to 32 tokens;
// the figures below are of these two).
//
// The units' blocks, laid end to end, are cut into equal ranges, one per CTA
// (one CTA per SM): a CTA works through the segments its range cuts out of
// the units. A segment that is a whole unit writes its output, the others
// leave (m, l, O) partials that merge_tree_kernel joins. Where whole units
// load the CTAs nearly as evenly (within cut_cost blocks), a unit goes whole
// to the CTA whose range it begins in: the 32 requests take 64 us so, and 81
// with ranges cut. The unions' lengths are known on the device only: every CTA
// sums them (tree_union_kernel leaves one per unit), comes to the same choice
// and finds its own range.
//
// What bounds it: no unit, but the latency of a block's chain (S, its maxima,
// P, the products) by two streams of four warps, and what passes between two
// units. A block of two tiles takes 3500 clocks, its products 2350, and 11 to 17
// thousand pass between the last block of a unit and the next one's first; with
// E4M3 the tensor cores are busy 44% of the time, the issue slots 43%, memory
// 25%. The products of the unions would take 132 us of the 305, on the 32
// requests 27 of the 64, where random pages take 42. Waits are by
// mbar_wait_sleep (spinning: 302 and 65 us).
//
// Two streams of (QK^T, softmax, PV) keep the tensor cores busy: while one
// stream's softmax warps turn its S into P, the other's products run. With
// two tiles in the unit the streams are the tiles and share every block; with
// one tile they take the blocks in turn, each with its own O, m and l, and
// the epilogue joins the two. TMEM holds S (P over it) and O of each stream.
//
// Roles: warps 0-3 and 4-7 the softmax of stream 0 and 1 (a thread per row),
// warp 8 hands out the segments and loads Q, warp 10 brings K and V by TMA,
// warp 11 issues the products of Q and K, warp 9 those of P and V, and for E4M3
// caches warps 12-15 decode K and V into the swizzled layout the MMA reads. Two
// warps issue, as one that does both, waiting for each PV before the S that
// takes its P's place, spends 1050 clocks a product and is the slowest of all
// (128 E4M3 requests 393 us against 305, 32 bf16 requests 83 against 64).
// Keys past a sequence's end are masked in S, and their V rows zeroed in
// shared memory, as P = 0 times what a page may hold there need not be 0.
//
// E4M3 is decoded to f16, exactly, NaN codes included, by one conversion a
// pair (moving the bits by integer instructions took 6% longer). Q then
// is f16 too, each bf16 row scaled by the power of two that puts its largest
// value just below f16's largest (what falls below f16's range is under 2^-39
// of that); the power of two comes back with the softmax scale.
//
// A tile's rows share the products, so a row also multiplies, by P = 0, what
// it must not see: values of another row's drafts or blocks, which may be
// infinite or NaN. Rows whose l or O is not finite are left to odd_row, which
// computes them anew from the row's own keys alone.
#include <cuda_fp16.h>
#include <math.h>

#include <climits>

#include "common.cuh"
#include "internal.h"
#include "mma_issue.cuh"
#include "softmax.cuh"
#include "tmem_wide.cuh"

namespace msa {
namespace {

constexpr int kHalf = 16384;      // 128 rows x 128 bytes, swizzled: half of an operand tile
constexpr int kKSlots = 2;        // K ring (a slot frees when its last QK^T completes)
constexpr int kRawSlots = 2;      // E4M3 blocks as they are, on their way
constexpr int kSegRing = 4;
constexpr uint32_t kColS = 0, kColO = 256;  // TMEM: S of stream s at 128 s, O at 256 + 128 s

template <bool FP8>
struct Roles {
  static constexpr int kSched = 8;  // segments and Q
  static constexpr int kMma = 9;    // issues the products of P and V
  static constexpr int kKv = 10;    // K and V by TMA
  static constexpr int kQk = 11;    // issues the products of Q and K
  static constexpr int kDecode = 12;  // E4M3: first of the decoding warps
  static constexpr int kDecodeWarps = FP8 ? 4 : 0;
  static constexpr int kThreads = (kDecode + kDecodeWarps) * 32;
  static constexpr int kReaders = 2 + 8 + 1;  // of the segment ring
  static constexpr int kVSlots = FP8 ? 2 : 3;  // V ring (a slot frees when its last PV completes)
};

// A range of one unit's union, or (n == 0) a unit whose rows see nothing.
struct Segment {
  int unit;      // -1: no more; u = tile * Hkv + h
  int h, t0, b, nw, lk, lq;
  int j0, n;     // union positions [j0, j0 + n)
  int slot;      // partial slot, or -1: the whole unit
  int dual;      // two tiles
};

// What a raw E4M3 slot holds; g == -1: no more.
struct RawTile {
  int g, is_v, rows;  // rows: keys of the block within the sequence (0: no page)
};

template <bool FP8>
struct __align__(1024) Smem {
  static constexpr int kVSlots = Roles<FP8>::kVSlots;
  uint8_t q[2][2][kHalf];  // [tile][64-column half]
  uint8_t k[kKSlots][2][kHalf];
  uint8_t v[kVSlots][2][kHalf];
  uint8_t raw[FP8 ? kRawSlots : 1][FP8 ? kHalf : 16];
  RawTile raw_tile[kRawSlots];
  uint64_t raw_full[kRawSlots], raw_empty[kRawSlots];
  Segment seg[kSegRing];
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  uint64_t q_full, q_empty;
  uint64_t k_full[kKSlots], k_empty[kKSlots];
  uint64_t v_full[kVSlots], v_empty[kVSlots];
  uint64_t qk_done[2][2];          // per stream and 64-key half of a block: S readable
  uint64_t p_full[2][2];           // P written
  uint64_t pv_done[2][2];          // the half's PV complete: its P read, O written
  uint64_t o_done[2], o_free[2];   // per stream: O complete at a segment's end, O read out
  uint64_t ml_full, ml_empty, drain[2];
  uint64_t q_ready;                // E4M3: Q converted
  float2 ml[128];                  // stream 1's (m, l) for the epilogue that joins the streams
  float q_scale[128];              // E4M3, one tile: the rows' softmax scales
  long long scan[32];
  long long first_p0, total;
  int first_unit, most;  // most: of the CTAs' loads with whole units
  uint32_t tmem_base;
  int abort;
};
// A CTA's shared memory, which begins on 1024 bytes (the kernel looks).
static_assert(sizeof(Smem<false>) <= 227 * 1024 && sizeof(Smem<true>) <= 227 * 1024, "too much shared memory");

// The partition of [0, total) into the CTAs' ranges.
struct Ranges {
  long long total;
  int n;
  MSA_DEV long long start(int i) const { return total * i / n; }
  // The range that position p < total is in: the last i with start(i) <= p.
  MSA_DEV int holder(long long p) const { return (int)((p * n + n - 1) / total); }
};
MSA_DEV Ranges ranges_of(const TreeArgs& a, long long total, int grid) {
  const long long most = total / a.min_range;
  return {total, (int)(most < 1 ? 1 : most < grid ? most : grid)};
}
// Union positions of a unit (at p0, `len` blocks of weight w) within [c0, c1).
MSA_DEV int first_block(long long p0, long long c, int w, int len) {
  const long long j = c <= p0 ? 0 : (c - p0 + w - 1) / w;
  return (int)(j < len ? j : len);
}

// What a block costs a CTA, by the unit's tiles: bringing and decoding it is
// the same, but two tiles multiply twice (128 E4M3 requests: 305 us with 3 to
// 4, 318 with equal weights, 320 with 2 to 4).
constexpr int kOneTileWeight = 3, kTwoTileWeight = 4;
MSA_DEV int unit_weight(const TreeArgs& a, int tokens) {
  return tokens > a.tile_tokens ? kTwoTileWeight : kOneTileWeight;
}

// Which of block columns 32 * k .. 32 * k + 31 a token of a tree sees, as bits.
// base: the block's first column as a node number (negative before the
// drafts); mask: the token's `words` words; columns past lim end the sequence.
MSA_DEV uint32_t tree_bits(const uint32_t* mask, int words, long long base, int k, int lim) {
  const long long j0 = base + 32 * k;
  uint32_t bits;
  if (j0 <= -32) {
    bits = ~0u;
  } else {
    const int i = j0 < 0 ? -1 : (int)min(j0 >> 5, (long long)words);
    const uint32_t lo = i < 0 ? ~0u : i < words ? __ldg(mask + i) : 0u;
    const uint32_t hi = i + 1 < words ? __ldg(mask + i + 1) : 0u;
    bits = __funnelshift_r(lo, hi, (int)(j0 & 31));
  }
  const int left = lim - 32 * k;  // last column of these within the sequence
  return left >= 31 ? bits : left < 0 ? 0u : bits & ((2u << left) - 1u);
}

// Inclusive sum over the warp.
template <class T>
MSA_DEV T warp_inclusive(T v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// One block per unit (tile, KV head): which tokens it has (tiles are numbered
// sequence by sequence), the union of their lists, ascending, and each
// token's membership bits over the union's positions. The union is a bitmap
// over the sequence's blocks in shared memory: ranks are the bits before.
constexpr int kUnionThreads = 256;
__global__ void __launch_bounds__(kUnionThreads) tree_union_kernel(const __grid_constant__ TreeArgs a) {
  extern __shared__ uint32_t dyn[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = blockIdx.x, h = blockIdx.y, unit = tile * a.num_kv_heads + h;
  __shared__ int s_warp[kUnionThreads / 32];
  __shared__ int s_b, s_t0;
  grid_dependency_wait();
  grid_dependents_launch();
  if (tid == 0) {
    s_b = -1;
    if (tile == 0 && h == 0) *a.odd = 0;
  }
  int carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kUnionThreads) {
    const int b = b0 + tid;
    int start = 0, count = 0;
    if (b < a.batch) {
      start = __ldg(a.cu_q + b);
      const int lq = __ldg(a.cu_q + b + 1) - start;
      count = lq > 0 ? (lq + a.unit_tokens - 1) / a.unit_tokens : 0;
    }
    const int inc = warp_inclusive(count, lane);
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int before = carry, all = 0;
#pragma unroll
    for (int w = 0; w < kUnionThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    before += inc - count;
    if (count > 0 && tile >= before && tile < before + count) {
      s_b = b;
      s_t0 = start + (tile - before) * a.unit_tokens;
    }
    carry += all;
    if (tile < carry) break;
  }
  __syncthreads();
  const int b = s_b;
  if (b < 0) {
    if (tid == 0) {
      a.unit_len[unit] = 0;
      a.unit_info[2 * unit] = make_int4(-1, 0, 0, 0);
    }
    return;
  }
  const int t0 = s_t0, end = __ldg(a.cu_q + b + 1), lq = end - __ldg(a.cu_q + b);
  const int lk = __ldg(a.seqused_k + b), nw = min(a.unit_tokens, end - t0);
  const int nblk = min((int)(((long long)lk + kBlk - 1) / kBlk), a.max_pages);
  const int maps = (a.max_pages + 31) >> 5;
  uint32_t* map = dyn;                       // a bit per block of the sequence
  int* rank = reinterpret_cast<int*>(dyn) + maps;  // bits before each word
  uint32_t* mem = dyn + 2 * maps;            // (tokens, words)
  const int n = nw * a.topk, used_maps = nblk > 0 ? (nblk + 31) >> 5 : 0;
  for (int i = tid; i < used_maps; i += kUnionThreads) map[i] = 0u;
  for (int i = tid; i < nw * a.words; i += kUnionThreads) mem[i] = 0u;
  __syncthreads();
  const int32_t* ids = a.q2k + ((size_t)h * a.total_q + t0) * a.topk;
  for (int i = tid; i < n; i += kUnionThreads) {
    const int id = __ldg(ids + i);
    if (id >= 0 && id < nblk) atomicOr(&map[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  int base = 0;
  int32_t* list = a.union_blocks + (size_t)unit * a.cap;
  for (int i0 = 0; i0 < used_maps; i0 += kUnionThreads) {
    const int i = i0 + tid;
    uint32_t bits = i < used_maps ? map[i] : 0u;
    const int count = __popc(bits), inc = warp_inclusive(count, lane);
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int w = 0; w < kUnionThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    before += inc - count;
    if (i < used_maps) rank[i] = before;
    while (bits != 0u) {
      list[before++] = i * 32 + __ffs(bits) - 1;
      bits &= bits - 1u;
    }
    base += all;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kUnionThreads) {
    const int id = __ldg(ids + i), w = i / a.topk;
    if (id < 0 || id >= nblk) continue;
    const int at = rank[id >> 5] + __popc(map[id >> 5] & ((1u << (id & 31)) - 1u));
    atomicOr(&mem[w * a.words + (at >> 5)], 1u << (at & 31));
  }
  __syncthreads();
  uint32_t* member = a.member + (size_t)unit * a.unit_tokens * a.words;
  const int words = (base + 31) >> 5;
  for (int i = tid; i < nw * words; i += kUnionThreads) {
    const int w = i / words, k = i - w * words;
    member[w * a.words + k] = mem[w * a.words + k];
  }
  if (tid == 0) {
    a.unit_len[unit] = base * unit_weight(a, nw);
    a.unit_info[2 * unit] = make_int4(t0, b, nw, base);
    a.unit_info[2 * unit + 1] = make_int4(lq, lk, 0, 0);
  }
}

template <bool FP8, bool F16>
__global__ void __launch_bounds__(Roles<FP8>::kThreads, 1)
    tree_kernel(const __grid_constant__ TreeArgs a) {
  static_assert(!(FP8 && F16), "E4M3 goes with bf16 q");
  constexpr bool kF16Ops = FP8 || F16;  // the MMAs' operands are f16, else bf16
  // Columns of S a softmax thread holds: 64 are read once; in the E4M3 kernel
  // they would spill, and the smaller code matters too (its roles share the
  // instruction cache): 32, read twice, are 5% faster there and 5% slower in
  // the others.
  constexpr int kCols = FP8 ? 32 : 64;
  using R = Roles<FP8>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  {
    uint32_t dyn;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn));
    if (pad + sizeof(Smem<FP8>) > dyn) {
      grid_dependency_wait();
      if (threadIdx.x == 0) {
        atomicOr(a.fault, (unsigned)kFaultCapacity);
        a.cut[blockIdx.x] = make_int2(-1, -1);  // nothing to join
      }
      return;
    }
  }
  Smem<FP8>& sm = *reinterpret_cast<Smem<FP8>*>(smem_raw + pad);
  constexpr int kVSlots = R::kVSlots;
  unsigned* fault = a.fault;
  volatile int* abort = &sm.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.num_qo_heads / a.num_kv_heads, W = a.tile_tokens;
  const int units = a.max_tiles * a.num_kv_heads;

  if (tid == 0) {
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(&sm.seg_full[s], 1);
      mbar_init(&sm.seg_empty[s], R::kReaders);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(&sm.k_full[s], FP8 ? R::kDecodeWarps : 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kVSlots; ++s) {
      mbar_init(&sm.v_full[s], FP8 ? R::kDecodeWarps : 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sm.qk_done[s][h], 1);
        mbar_init(&sm.p_full[s][h], 4);
        mbar_init(&sm.pv_done[s][h], 1);
      }
      mbar_init(&sm.o_done[s], 1);
      mbar_init(&sm.o_free[s], 4);
    }
    mbar_init(&sm.ml_full, 4);
    mbar_init(&sm.ml_empty, 4);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    mbar_init(&sm.q_ready, 8);
    for (int s = 0; s < kRawSlots; ++s) {
      mbar_init(&sm.raw_full[s], 1);
      mbar_init(&sm.raw_empty[s], FP8 ? R::kDecodeWarps : 1);
    }
    sm.abort = 0;
    sm.first_unit = INT_MAX;
    fence_mbar_init();
  }
  if (warp == R::kMma) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  grid_dependency_wait();  // the unions
  grid_dependents_launch();

  // The sum of the units' weighted lengths, and where this CTA's range begins.
  const int per = (units + R::kThreads - 1) / R::kThreads;
  const int u_lo = min(units, tid * per), u_hi = min(units, u_lo + per);
  long long mine = 0;
  for (int u = u_lo; u < u_hi; ++u) mine += __ldg(a.unit_len + u);
  const long long inc = warp_inclusive(mine, lane);
  if (lane == 31) sm.scan[warp] = inc;
  __syncthreads();
  if (tid == 0) {
    long long s = 0;
    for (int w = 0; w < R::kThreads / 32; ++w) {
      const long long x = sm.scan[w];
      sm.scan[w] = s;
      s += x;
    }
    sm.total = s;
  }
  __syncthreads();
  const Ranges ranges = ranges_of(a, sm.total, gridDim.x);
  const int cta = blockIdx.x;
  // The loads with whole units: each to the range it begins in.
  {
    int* load = reinterpret_cast<int*>(&sm.q[0][0][0]);
    for (int i = tid; i < ranges.n; i += R::kThreads) load[i] = 0;
    if (tid == 0) sm.most = 0;
    __syncthreads();
    long long p = sm.scan[warp] + inc - mine;
    for (int u = u_lo; u < u_hi; ++u) {
      const int len = __ldg(a.unit_len + u);
      if (len > 0) atomicAdd(&load[ranges.holder(p)], len);
      p += len;
    }
    __syncthreads();
    int most = 0;
    for (int i = tid; i < ranges.n; i += R::kThreads) most = max(most, load[i]);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&sm.most, most);
    fence_async_smem();  // the loads' memory is Q's
    __syncthreads();
  }
  const bool whole = sm.most <= ranges.total / ranges.n + a.cut_cost;
  const bool works = cta < ranges.n, last = cta == ranges.n - 1;
  const long long c0 = works ? ranges.start(cta) : 0, c1 = works ? ranges.start(cta + 1) : 0;
  // A unit without blocks goes to the CTA whose range holds its place (the
  // last CTA, at the end).
  auto holds = [&](long long p0) { return (p0 >= c0 && p0 < c1) || (last && p0 >= c1); };
  {
    long long p = sm.scan[warp] + inc - mine;
    int found = INT_MAX;
    long long found_p = 0;
    for (int u = u_lo; works && u < u_hi && found == INT_MAX; ++u) {
      const long long len = __ldg(a.unit_len + u);
      if (len == 0 || whole ? holds(p) : p + len > c0) {
        found = u;
        found_p = p;
      }
      p += len;
    }
    if (found != INT_MAX) atomicMin(&sm.first_unit, found);
    __syncthreads();
    if (found != INT_MAX && found == sm.first_unit) sm.first_p0 = found_p;
    __syncthreads();
  }

  // The n-th segment of this CTA; false at the end (or when a wait gave up).
  auto read_seg = [&](int n, Segment& s) -> bool {
    const int slot = n % kSegRing;
    if (!mbar_wait_sleep(&sm.seg_full[slot], (n / kSegRing) & 1, fault, kFaultWaitOther, abort)) {
      s.unit = -2;
      return false;
    }
    s = sm.seg[slot];
    return s.unit >= 0;
  };
  auto release_seg = [&](int n) { mbar_arrive(&sm.seg_empty[n % kSegRing]); };

  if (warp == R::kSched) {
    // ------------------------------------------------------- segments and Q
    // The warp reads 32 units at a time, then walks them one by one, one
    // segment ahead of the Q tile it loads.
    int cut_unit = -1, head_unit = -1;
    if (lane == 0) tma_prefetch_desc(&a.tmap_q);
    bool ok = true;
    int n_pub = 0, n_q = 0;   // segments published, Q tiles loaded
    Segment pend{};           // published, its Q not loaded yet
    pend.unit = -1;
    bool q_flight = false;
    auto publish = [&](const Segment& s) {
      const int slot = n_pub % kSegRing;
      if (n_pub >= kSegRing &&
          !mbar_wait_sleep(&sm.seg_empty[slot], ((n_pub / kSegRing) - 1) & 1, fault, kFaultWaitOther, abort)) {
        ok = false;
        return;
      }
      sm.seg[slot] = s;
      mbar_arrive(&sm.seg_full[slot]);
      ++n_pub;
    };
    auto load_q = [&]() {
      if (!ok || pend.unit < 0) return;
      if (n_q > 0 && !mbar_wait_sleep(&sm.q_empty, (n_q - 1) & 1, fault, kFaultWaitMma, abort)) {
        ok = false;
        return;
      }
      const int tiles = pend.dual ? 2 : 1;
      mbar_expect_tx(&sm.q_full, (uint32_t)tiles * 2u * 128u * (uint32_t)(G * W));
      for (int t = 0; t < tiles; ++t)
        for (int c = 0; c < 2; ++c)
          tma_load_3d(sm.q[t][c], &a.tmap_q, &sm.q_full, c * 64, pend.h * G, pend.t0 + t * W);
      q_flight = true;
      ++n_q;
      pend.unit = -1;
    };
    if (works && sm.first_unit != INT_MAX) {
      long long p0 = sm.first_p0;
      bool more = true;
      for (int u0 = sm.first_unit; more && u0 < units; u0 += 32) {
        int4 info = make_int4(-1, 0, 0, 0);  // t0, sequence, tokens, union length
        int2 lens = make_int2(0, 0);         // Lq, Lk
        if (u0 + lane < units) {
          info = __ldg(a.unit_info + 2 * (u0 + lane));
          lens = __ldg(reinterpret_cast<const int2*>(a.unit_info + 2 * (u0 + lane) + 1));
        }
        for (int i = 0; i < 32 && more; ++i) {
          Segment s{};
          s.unit = u0 + i;
          s.t0 = __shfl_sync(0xffffffffu, info.x, i);
          s.b = __shfl_sync(0xffffffffu, info.y, i);
          s.nw = __shfl_sync(0xffffffffu, info.z, i);
          s.lq = __shfl_sync(0xffffffffu, lens.x, i);
          s.lk = __shfl_sync(0xffffffffu, lens.y, i);
          const int ulen = __shfl_sync(0xffffffffu, info.w, i);
          if (s.t0 < 0) {  // the tiles' end
            more = false;
            break;
          }
          s.h = s.unit % a.num_kv_heads;
          s.dual = s.nw > W;
          const int w = unit_weight(a, s.nw);
          bool mine_too;
          if (ulen == 0) {
            mine_too = holds(p0);
            more = p0 < c1 || last;
            s.slot = -1;
          } else {
            s.j0 = whole ? 0 : first_block(p0, c0, w, ulen);
            const int j1 = !whole ? first_block(p0, c1, w, ulen) : holds(p0) ? ulen : 0;
            s.n = j1 - s.j0;
            mine_too = s.n > 0;
            more = p0 < c1 || last;
            s.slot = s.j0 > 0 ? 2 * cta : j1 < ulen ? 2 * cta + 1 : -1;
            if (mine_too && s.j0 > 0) head_unit = s.unit;
            else if (mine_too && j1 < ulen) cut_unit = s.unit;
            p0 += (long long)ulen * w;
          }
          if (mine_too && lane == 0 && ok) {
            publish(s);
            load_q();  // of the segment before
            if (s.n > 0) pend = s;
          }
          if (!__shfl_sync(0xffffffffu, (int)ok, 0)) {
            ok = false;
            more = false;
          }
        }
      }
    }
    if (lane == 0) {
      load_q();
      if (ok) {
        Segment s{};
        s.unit = -1;
        publish(s);
      }
      a.cut[cta] = make_int2(cut_unit, head_unit);
      // A copy in flight lands before the CTA's shared memory is given back.
      if (!ok && q_flight) mbar_wait_sleep(&sm.q_full, (n_q - 1) & 1, fault, kFaultWaitTma);
    }
  } else if (warp == R::kQk || warp == R::kMma) {
    // -------------------------------------------------------------- MMA issue
    // One warp issues the products of Q and K, another those of P and V: a wait
    // takes about 100 clocks even where it has nothing to wait for. A whole warp
    // runs this, so that what an MMA needs stays in uniform registers; one
    // elected lane issues. (A single lane's branch spent about 100 clocks on
    // each MMA, which takes 73.)
    // Two tiles: both streams take every block. One tile: block j is stream
    // j & 1's. Either way the products go by halves of a block's keys, under
    // the softmax of the other half. (By whole blocks a stream's softmax and
    // products ran one after the other, and neither hid the other.)
    const bool is_qk = warp == R::kQk;
    const uint32_t el = elect_one();
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    constexpr uint32_t kTile16 = (2 * kHalf) >> 4, kHalf16 = kHalf >> 4;
    int nseg = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t phase, unsigned code) {
      ok = ok && mbar_wait_sleep(bar, phase, fault, code, abort);
    };
    auto commit = [&](uint64_t* bar) { commit_if(el, bar); };
    Segment s;
    // The next segment with blocks; false at the end.
    int ni = 0, n = 0;
    bool dual = false;
    auto next_seg = [&]() -> bool {
      n = 0;
      while (ok && n == 0) {
        const bool more = read_seg(ni, s);
        __syncwarp();
        if (!more) return false;
        if (lane == 0) release_seg(ni);
        ++ni;
        n = __shfl_sync(0xffffffffu, s.n, 0);
        dual = __shfl_sync(0xffffffffu, s.dual, 0) != 0;
      }
      return ok;
    };
    if (is_qk) {
      // S of a half takes the place of the P of the stream's half before, once
      // the PV that reads it is complete. (MMAs run in the order of their issue
      // where shape and accumulator are the same; these differ in both.)
      constexpr uint32_t idS = idesc_16bit_f32(128, 64, false, false, kF16Ops);
      // Descriptors differ in the start address, in their low words.
      const uint64_t dq = sdesc_sw128(smem_u32(&sm.q[0][0][0]), 16, 1024);
      const uint32_t hi = (uint32_t)(dq >> 32), q0 = (uint32_t)dq;
      const uint32_t k0 = (uint32_t)sdesc_sw128(smem_u32(&sm.k[0][0][0]), 16, 1024);
      Ring<kKSlots> rk;
      uint32_t used = 0u, pv_phase = 0u;  // a bit per stream and half: whether it held a P, and its PV's phase
      while (next_seg()) {
        if (FP8) wait(&sm.q_ready, nseg & 1, kFaultWaitSoftmax);
        else wait(&sm.q_full, nseg & 1, kFaultWaitTma);
#pragma unroll 1
        for (int b = 0; ok && b < n; ++b) {
          wait(&sm.k_full[rk.idx], rk.phase, kFaultWaitTma);
          const int x_end = dual ? 4 : 2;
#pragma unroll 1
          for (int x = 0; ok && x < x_end; ++x) {
            const int st = dual ? x & 1 : b & 1, h = dual ? x >> 1 : x;
            const uint32_t bit = 1u << (2 * st + h);
            if (used & bit) {
              wait(&sm.pv_done[st][h], (pv_phase & bit) != 0u, kFaultWaitMma);
              if (!ok) break;
              pv_phase ^= bit;
            }
            used |= bit;
            tc_fence_after();
            const uint32_t q = q0 + (dual ? st : 0) * kTile16, k = k0 + rk.idx * kTile16 + h * 512;
            const uint32_t d = tb + kColS + st * 128 + h * 64;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = (kk >> 2) * kHalf16 + (kk & 3) * 2;
              mma_ss_if(el, d, q + off, k + off, hi, idS, kk > 0);
            }
            commit(&sm.qk_done[st][h]);
          }
          if (!ok) break;
          commit(&sm.k_empty[rk.idx]);
          rk.next();
        }
        if (ok) commit(&sm.q_empty);
        ++nseg;
      }
    } else {
      constexpr uint32_t idO = idesc_16bit_f32(128, 128, false, true, kF16Ops);
      const uint64_t dv = sdesc_sw128(smem_u32(&sm.v[0][0][0]), kHalf, 1024);
      const uint32_t hi = (uint32_t)(dv >> 32), v0 = (uint32_t)dv;
      Ring<kVSlots> rv;
      uint32_t p_phase = 0u;  // a bit per stream
      while (next_seg()) {
        const int ahead = dual ? 1 : 2;  // blocks that are the streams' first, and last
#pragma unroll 1
        for (int t = 0; ok && t < n; ++t) {
          if (t < ahead && nseg > 0) {
            // O has been read: of both streams, every phase of each.
            if (dual || t == 0) wait(&sm.o_free[0], (nseg - 1) & 1, kFaultWaitSoftmax);
            if (dual || t == 1 || n == 1) wait(&sm.o_free[1], (nseg - 1) & 1, kFaultWaitSoftmax);
          }
          wait(&sm.v_full[rv.idx], rv.phase, kFaultWaitTma);
          const int x_end = dual ? 4 : 2;
#pragma unroll 1
          for (int x = 0; ok && x < x_end; ++x) {
            const int st = dual ? x & 1 : t & 1, h = dual ? x >> 1 : x;
            wait(&sm.p_full[st][h], (p_phase >> st) & 1u, kFaultWaitSoftmax);
            if (!ok) break;
            tc_fence_after();
            // O of the stream = (+=) P V for the half.
            const uint32_t v = v0 + rv.idx * kTile16 + h * 512;
            const uint32_t tp = tb + kColS + st * 128 + h * 64, d = tb + kColO + st * 128;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts_if(el, d, tp + kk * 8, v + kk * 128, hi, idO, kk > 0 || h > 0 || t >= ahead);
            commit(&sm.pv_done[st][h]);
            if (h == 1) {
              p_phase ^= 1u << st;
              if (t + ahead >= n) commit(&sm.o_done[st]);
            }
          }
          if (!ok) break;
          commit(&sm.v_empty[rv.idx]);
          rv.next();
        }
        ++nseg;
      }
    }
    commit(&sm.drain[is_qk]);
    mbar_wait_sleep(&sm.drain[is_qk], 0, fault, kFaultWaitMma);
    __syncwarp();
  } else if (warp == R::kKv) {
    // ---------------------------------------------------------------- K and V
    if (!FP8 && lane == 0) {
      tma_prefetch_desc(&a.tmap_k);
      tma_prefetch_desc(&a.tmap_v);
    }
    // The tiles of all segments, one after the other.
    Segment s;
    s.n = 0;
    int ni = 0, x = 0, g0 = 0;  // segments read, tiles taken of this one, blocks before it
    bool ok = true, more = true;
    // Pages of 32 blocks at a time, for K and for V apart (a page outside the
    // pool reads as zeros and is masked).
    const int32_t *list = nullptr, *prow = nullptr;
    int page_k = -1, page_v = -1, blk_k = 0, blk_v = 0;
    struct Tile {
      int g, page, blk, is_v, h, lk;
    };
    // The next tile, warp-wide; false at the end.
    auto take = [&](Tile& t) -> bool {
      while (more && x == 2 * s.n) {
        g0 += s.n;
        x = 0;
        s.n = 0;
        more = read_seg(ni, s);
        __syncwarp();
        if (!more) {
          ok = s.unit == -1;
          break;
        }
        if (lane == 0) release_seg(ni);
        ++ni;
        list = a.union_blocks + (size_t)s.unit * a.cap + s.j0;
        prow = a.page_table + (size_t)s.b * a.max_pages;
      }
      if (!more) return false;
      bool is_v;
      const int j = tile_order(x, s.n, is_v);
      ++x;
      auto fetch = [&](int& page, int& blk) {
        if ((j & 31) == 0) {
          blk = j + lane < s.n ? __ldg(list + j + lane) : 0;
          page = j + lane < s.n ? __ldg(prow + blk) : -1;
          if (page < 0 || page >= a.num_pages) page = a.num_pages;
        }
      };
      if (is_v) fetch(page_v, blk_v);
      else fetch(page_k, blk_k);
      t.page = __shfl_sync(0xffffffffu, is_v ? page_v : page_k, j & 31);
      t.blk = __shfl_sync(0xffffffffu, is_v ? blk_v : blk_k, j & 31);
      t.g = g0 + j;
      t.is_v = is_v;
      t.h = s.h;
      t.lk = s.lk;
      return true;
    };
    if constexpr (!FP8) {
      // Waits until the tile's slot may be written.
      auto slot_free = [&](const Tile& t) -> bool {
        const int ring = t.is_v ? kVSlots : kKSlots, slot = t.g % ring, round = t.g / ring;
        return round == 0 || mbar_wait_sleep(t.is_v ? &sm.v_empty[slot] : &sm.k_empty[slot], (round - 1) & 1, fault,
                                     kFaultWaitMma, abort);
      };
      int last_k[kKSlots], last_v[kVSlots];  // last block issued into each slot
      for (int i = 0; i < kKSlots; ++i) last_k[i] = -1;
      for (int i = 0; i < kVSlots; ++i) last_v[i] = -1;
      Tile t;
      while (ok && take(t)) {
        if (lane == 0 && slot_free(t)) {
          if (t.is_v) {
            const int vs = t.g % kVSlots;
            mbar_expect_tx(&sm.v_full[vs], 2 * kHalf);
            for (int c = 0; c < 2; ++c)
              tma_load_4d(sm.v[vs][c], &a.tmap_v, &sm.v_full[vs], c * 64, 0, t.h, t.page);
            last_v[vs] = t.g;
          } else {
            const int ks = t.g % kKSlots;
            mbar_expect_tx(&sm.k_full[ks], 2 * kHalf);
            for (int c = 0; c < 2; ++c)
              tma_load_4d(sm.k[ks][c], &a.tmap_k, &sm.k_full[ks], c * 64, 0, t.h, t.page);
            last_k[ks] = t.g;
          }
        } else if (lane == 0) {
          ok = false;
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      }
      if (!ok && lane == 0) {
        for (int i = 0; i < kKSlots; ++i)
          if (last_k[i] >= 0) mbar_wait_sleep(&sm.k_full[i], (last_k[i] / kKSlots) & 1, fault, kFaultWaitTma);
        for (int i = 0; i < kVSlots; ++i)
          if (last_v[i] >= 0) mbar_wait_sleep(&sm.v_full[i], (last_v[i] / kVSlots) & 1, fault, kFaultWaitTma);
      }
    } else {
      // E4M3: the blocks as they are into the raw ring, 16 KB of contiguous
      // memory each.
      int y = 0;
      auto put = [&](const RawTile& r, const uint8_t* src) -> bool {
        const int slot = y % kRawSlots;
        if (y >= kRawSlots &&
            !mbar_wait_sleep(&sm.raw_empty[slot], ((y / kRawSlots) - 1) & 1, fault, kFaultWaitOther, abort))
          return false;
        sm.raw_tile[slot] = r;
        if (r.rows > 0) {
          mbar_expect_tx(&sm.raw_full[slot], kHalf);
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  smem_u32(sm.raw[slot])),
              "l"(src), "r"(kHalf), "r"(smem_u32(&sm.raw_full[slot]))
              : "memory");
        } else {
          mbar_arrive(&sm.raw_full[slot]);
        }
        ++y;
        return true;
      };
      Tile t;
      while (ok && take(t)) {
        if (lane == 0) {
          const long long left = (long long)t.lk - (long long)t.blk * kBlk;
          const int rows = t.page >= a.num_pages || left <= 0 ? 0 : left < kBlk ? (int)left : kBlk;
          ok = put(RawTile{t.g, t.is_v, rows},
                   (t.is_v ? a.v_pool : a.k_pool) + ((size_t)(rows > 0 ? t.page : 0) * a.num_kv_heads + t.h) * kHalf);
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      }
      if (lane == 0) {
        if (ok) ok = put(RawTile{-1, 0, 0}, nullptr);
        // Copies in flight land before the CTA's shared memory is given back.
        if (!ok)
          for (int i = y < kRawSlots ? 0 : y - kRawSlots; i < y; ++i)
            mbar_wait_sleep(&sm.raw_full[i % kRawSlots], (i / kRawSlots) & 1, fault, kFaultWaitTma);
      }
    }
  } else if (FP8 && warp >= R::kDecode) {
    // ------------------------------------------------------------ E4M3 decode
    // 128 threads take a block's 128 rows of 128 bytes as eight 16-byte groups
    // each, give the raw slot back, and write f16. Rows past the sequence's end
    // become zeros.
    // Of eight threads four take the first half of a row and four the second
    // half of its neighbour, which keeps reads and writes off each other's
    // banks.
    const int ct = tid - R::kDecode * 32;
    const int q = ct & 7, r0 = (ct >> 3) ^ (q >> 2);
    bool ok = true;
    for (int y = 0;; ++y) {
      const int rs = y % kRawSlots;
      ok = mbar_wait_sleep(&sm.raw_full[rs], (y / kRawSlots) & 1, fault, kFaultWaitTma, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const RawTile t = sm.raw_tile[rs];
      uint4 raw[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int r = r0 + c * 16;
        raw[c] = r < t.rows ? *reinterpret_cast<const uint4*>(&sm.raw[rs][r * 128 + q * 16]) : make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.raw_empty[rs]);
      if (t.g < 0) break;
      const int ring = t.is_v ? kVSlots : kKSlots, slot = t.g % ring, round = t.g / ring;
      ok = round == 0 || mbar_wait_sleep(t.is_v ? &sm.v_empty[slot] : &sm.k_empty[slot], (round - 1) & 1, fault,
                                 kFaultWaitMma, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint8_t* dst = t.is_v ? &sm.v[slot][0][0] : &sm.k[slot][0][0];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int r = r0 + c * 16;
        uint32_t o[8];
        e4m3x4_to_f16(raw[c].x, o[0], o[1]);
        e4m3x4_to_f16(raw[c].y, o[2], o[3]);
        e4m3x4_to_f16(raw[c].z, o[4], o[5]);
        e4m3x4_to_f16(raw[c].w, o[6], o[7]);
        uint8_t* half = dst + (q >> 2) * kHalf;
        const int c16 = (q & 3) * 2;
        *reinterpret_cast<uint4*>(half + sw128_offset(r, c16)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(half + sw128_offset(r, c16 + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(t.is_v ? &sm.v_full[slot] : &sm.k_full[slot]);
    }
  } else {
    // ------------------------------------------------------ softmax, epilogue
    const int st = warp >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;  // TMEM lane
    const int wr = row / G, gh = row - wr * G;
    const uint32_t lanes = tbase + ((uint32_t)(q4 * 32) << 16);
    const uint32_t scol = lanes + kColS + st * 128;
    bool ok = true;
    int g0 = 0, nseg = 0;    // blocks, and segments with blocks, before this segment
    uint32_t nqk = 0;        // S tiles consumed by this stream
    uint32_t no[2] = {0, 0};  // O completions so far, per stream
    uint32_t nml = 0;        // segments whose streams were joined
    Segment s;
    for (int ni = 0; ok; ++ni) {
      const bool more = read_seg(ni, s);
      __syncwarp();
      if (!more) break;
      if (lane == 0) release_seg(ni);
      const int w = s.dual ? st * W + wr : wr;  // token of the unit
      const bool active = row < W * G && w < s.nw;
      const size_t orow = (size_t)(s.t0 + w) * a.num_qo_heads + (size_t)s.h * G + gh;
      if (s.n == 0) {
        // A unit that sees nothing: out = 0, lse = -inf.
        if (active && (s.dual || st == 0)) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * kHeadDim);
#pragma unroll
          for (int c = 0; c < 16; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
          if (a.lse != nullptr) a.lse[orow] = -INFINITY;
        }
        continue;
      }
      const int n = s.n, own = s.dual ? n : (n + 1 - st) / 2, step = s.dual ? 1 : 2;
      const int32_t* list = a.union_blocks + (size_t)s.unit * a.cap + s.j0;
      const uint32_t* mrow = a.member + ((size_t)s.unit * a.unit_tokens + (active ? w : 0)) * a.words;
      const uint32_t* mask = a.tree_mask + (size_t)(s.t0 + (active ? w : 0)) * a.mask_words;
      const int32_t* prow = a.page_table + (size_t)s.b * a.max_pages;
      float scale = a.scale_log2;  // of the row's S, to log2 units
      if constexpr (FP8) {
        if (s.dual || st == 0) {
          // The row of Q, in place: bf16 to f16 times 2^k.
          ok = mbar_wait_sleep(&sm.q_full, nseg & 1, fault, kFaultWaitTma, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* qt = &sm.q[s.dual ? st : 0][0][0];
          uint32_t big = 0u;
#pragma unroll 4
          for (int c = 0; c < 16; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(qt + (c >> 3) * kHalf + sw128_offset(row, c & 7));
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) big = max(big, max(xs[i] & 0x7f80u, (xs[i] >> 16) & 0x7f80u));
          }
          const int e = (int)(big >> 7);  // exponent field of the row's largest value
          const int k = e == 255 ? 0 : min(120, 142 - e);
          const float up = __uint_as_float((uint32_t)(127 + k) << 23);
          scale = a.scale_log2 * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll 4
          for (int c = 0; c < 16; ++c) {
            uint4* at = reinterpret_cast<uint4*>(qt + (c >> 3) * kHalf + sw128_offset(row, c & 7));
            const uint4 x = *at;
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[i] = pack_f16x2(__uint_as_float(xs[i] << 16) * up, __uint_as_float(xs[i] & 0xffff0000u) * up);
            *at = make_uint4(o[0], o[1], o[2], o[3]);
          }
          if (!s.dual) sm.q_scale[row] = scale;
          fence_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&sm.q_ready);
        if (!s.dual && st == 1) {
          ok = mbar_wait_sleep(&sm.q_ready, nseg & 1, fault, kFaultWaitSoftmax, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          scale = sm.q_scale[row];
        }
        ++nseg;
      }
      float m_ref = -INFINITY, l = 0.f;
      // Block ids two steps ahead, pages one step ahead.
      int j = s.dual ? 0 : st;
      int id1 = own > 0 ? __ldg(list + j) : 0, id2 = own > 1 ? __ldg(list + j + step) : 0;
      int pg1 = own > 0 ? __ldg(prow + id1) : 0;
      uint32_t word1 = own > 0 && active ? __ldg(mrow + ((s.j0 + j) >> 5)) : 0u;
      for (int t = 0; t < own; ++t, j += step) {
        const int blk = id1, pg = pg1, upos = s.j0 + j;
        const uint32_t word = word1;
        id1 = id2;
        if (t + 2 < own) id2 = __ldg(list + j + 2 * step);
        if (t + 1 < own) {
          pg1 = __ldg(prow + id1);
          if (active) word1 = __ldg(mrow + ((upos + step) >> 5));
        }
        bool mem = active && ((word >> (upos & 31)) & 1u) && pg >= 0 && pg < a.num_pages;
        // The row's visible columns, and the block's keys within the sequence.
        uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
        const long long left = (long long)s.lk - (long long)blk * kBlk;
        const long long base = (long long)blk * kBlk - ((long long)s.lk - s.lq);
        const int tail = left < 128 ? (left < 0 ? 0 : (int)left) : 128;
        bool hides = false;
        if (base + 127 >= 0 || tail < 128) {
          uint32_t any = 0u, all = ~0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            vis[k] = mem ? tree_bits(mask, a.mask_words, base, k, tail - 1) : 0u;
            any |= vis[k];
            all &= vis[k];
          }
          mem = any != 0u;
          // Rows that see nothing here are masked too where columns may hold anything.
          hides = all != ~0u && (mem || tail < 128);
        }
        const bool warp_mem = __any_sync(0xffffffffu, mem);
        const bool warp_hides = __any_sync(0xffffffffu, hides);
        if (!FP8 && tail < 128 && (st == 0 || !s.dual)) {
          // V rows past the end, before the first PV that reads the block (in
          // a unit of two tiles stream 0's, which is issued first). The wait
          // for the slot's phase needs the phase before it complete: V of the
          // block kVSlots earlier is there once this block's S is, as S of a
          // stream waits for the PV of its block before: one of the last three.
          const int g = g0 + j, vs = g % kVSlots;
          ok = mbar_wait_sleep(&sm.qk_done[st][0], nqk & 1, fault, kFaultWaitMma, abort) &&
               mbar_wait_sleep(&sm.v_full[vs], (g / kVSlots) & 1, fault, kFaultWaitTma, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          for (int i = tail * 16 + row; i < 128 * 16; i += 128)
            *reinterpret_cast<uint4*>(&sm.v[vs][(i >> 3) & 1][(i >> 4) * 128 + (i & 7) * 16]) =
                make_uint4(0u, 0u, 0u, 0u);
          fence_async_smem();
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint32_t vis0 = half == 0 ? vis[0] : vis[2], vis1 = half == 0 ? vis[1] : vis[3];
          const uint32_t hcol = scol + half * 64;  // P over the first half of its own S
          ok = mbar_wait_sleep(&sm.qk_done[st][half], nqk & 1, fault, kFaultWaitMma, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (warp_mem) {
            if (warp_hides) {
              // Few blocks: eight columns at a time, written back to S.
#pragma unroll 1
              for (int c = 0; c < 64; c += 8) {
                uint32_t x[8];
                tmem_ld8_nowait(hcol + c, x);
                tmem_wait_ld();
                const uint32_t see = (c < 32 ? vis0 : vis1) >> (c & 31);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = (see >> i) & 1u ? x[i] : 0xff800000u;
                tmem_st8_nowait(hcol + c, x);
                tmem_wait_st();
              }
            }
            float sv[kCols];
            float mx = -INFINITY;
#pragma unroll 1
            for (int c0q = 0; c0q < 64; c0q += kCols) {
              if constexpr (kCols == 64) tmem_ld64(hcol, sv);
              else tmem_ld32(hcol + c0q, sv);
              mx = max3_nan(mx, mx, row_max<kCols>(sv));
            }
            const bool on = mem && mx != -INFINITY;
            float alpha = 1.f;
            bool rescale = false;
            update_max(on, mx, scale, m_ref, l, alpha, rescale);
            if (__any_sync(0xffffffffu, rescale)) {
              // O has to hold the half before: this block's first or the last
              // block's second (in a unit's first half no row has a maximum yet).
              // The half before that is complete, as this S was issued after it.
              ok = mbar_wait_sleep(&sm.pv_done[st][half ^ 1], (nqk - (half ^ 1)) & 1, fault, kFaultWaitMma, abort);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                const uint32_t ocol = lanes + kColO + st * 128 + q * 32;
                float o[32];
                tmem_ld32(ocol, o);
                uint32_t ow[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) ow[c] = __float_as_uint(o[c] * alpha);
                tmem_st32(ocol, ow);
              }
            }
            float2 acc = make_float2(0.f, 0.f);
            const float neg_m = on ? -m_ref : -INFINITY;
#pragma unroll 1
            for (int c0q = 0; c0q < 64; c0q += kCols) {
              if constexpr (kCols == 32) tmem_ld32(hcol + c0q, sv);
              uint32_t pk[kCols / 2];
#pragma unroll
              for (int c = 0; c < kCols; c += 2) {
                const float2 x = __ffma2_rn(make_float2(sv[c], sv[c + 1]), make_float2(scale, scale),
                                            make_float2(neg_m, neg_m));
                const float2 p = make_float2(ex2(x.x), ex2(x.y));
                acc = __fadd2_rn(acc, p);
                pk[c >> 1] = pack_x2<kF16Ops>(p.x, p.y);
              }
              // Over columns that have been read.
              if constexpr (kCols == 64) tmem_st32(hcol, pk);
              else tmem_st16(hcol + (c0q >> 1), pk);
            }
            if (on) l += acc.x + acc.y;
          } else {
            uint32_t zero[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) zero[c] = 0u;
            tmem_st32(hcol, zero);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[st][half]);
        }
        if (!ok) break;
        ++nqk;
      }
      if (!ok) break;
      g0 += n;
      // ------------------------------------------------------------ epilogue
      float f[2] = {1.f, 0.f};
      uint32_t from[2] = {lanes + kColO + st * 128, 0u};
      if (!s.dual) {
        if (st == 1) {
          // Stream 0's warps join the two.
          if (nml > 0)
            ok = mbar_wait_sleep(&sm.ml_empty, (nml - 1) & 1, fault, kFaultWaitSoftmax, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++nml;
          ++no[0];
          if (n > 1) ++no[1];
          sm.ml[row] = make_float2(m_ref, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.ml_full);
          continue;
        }
        ok = mbar_wait_sleep(&sm.ml_full, nml & 1, fault, kFaultWaitSoftmax, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++nml;
        const float2 other = sm.ml[row];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ml_empty);
        const float m = fmaxf(m_ref, other.x);
        f[0] = m_ref == -INFINITY ? 0.f : ex2(m_ref - m);
        f[1] = other.x == -INFINITY ? 0.f : ex2(other.x - m);
        l = f[0] * l + f[1] * other.y;
        m_ref = m;
        from[1] = lanes + kColO + 128;
        ok = mbar_wait_sleep(&sm.o_done[0], no[0] & 1, fault, kFaultWaitMma, abort);
        ++no[0];
        if (ok && n > 1) {
          ok = mbar_wait_sleep(&sm.o_done[1], no[1] & 1, fault, kFaultWaitMma, abort);
          ++no[1];
        }
      } else {
        ok = mbar_wait_sleep(&sm.o_done[st], no[st] & 1, fault, kFaultWaitMma, abort);
        ++no[0];
        ++no[1];
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const bool joins = !s.dual && n > 1;
      const bool has = l > 0.f;
      const float inv = has ? 1.f / l : 0.f;
      const size_t slot = s.slot < 0 ? 0 : s.slot;
      const int prow_out = (s.dual ? st * W * G : 0) + row;
      float2 odd = make_float2(0.f, 0.f);  // NaN once an element of O is not finite
#pragma unroll 1
      for (int c0q = 0; c0q < 128; c0q += 32) {
        float o[32];
        tmem_ld32(from[0] + c0q, o);
        if (joins) {
          float o1[32];
          tmem_ld32(from[1] + c0q, o1);
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = f[0] * o[c] + f[1] * o1[c];
        }
        if (c0q == 96) {
          // O is read: the next segment's first PV may overwrite it.
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.o_free[st]);
            if (!s.dual) mbar_arrive(&sm.o_free[1]);
          }
        }
        if (active && s.slot < 0) {
#pragma unroll
          for (int c = 0; c < 32; c += 2)
            odd = __ffma2_rn(make_float2(o[c], o[c + 1]), make_float2(0.f, 0.f), odd);
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * kHeadDim + c0q);
#pragma unroll
          for (int c = 0; c < 32; c += 8)
            dst[c >> 3] = has ? make_uint4(pack_x2<F16>(o[c] * inv, o[c + 1] * inv),
                                           pack_x2<F16>(o[c + 2] * inv, o[c + 3] * inv),
                                           pack_x2<F16>(o[c + 4] * inv, o[c + 5] * inv),
                                           pack_x2<F16>(o[c + 6] * inv, o[c + 7] * inv))
                              : make_uint4(0u, 0u, 0u, 0u);
        } else if (active) {
          // Column by column, so that a warp's rows are one piece of memory.
          float* dst = a.part_o + (slot * kHeadDim + c0q) * a.rows_part + prow_out;
#pragma unroll
          for (int c = 0; c < 32; ++c) dst[(size_t)c * a.rows_part] = o[c];
        }
        __syncwarp();
      }
      if (active) {
        if (s.slot >= 0) {
          a.part_m[slot * a.rows_part + prow_out] = m_ref;
          a.part_l[slot * a.rows_part + prow_out] = l;
        } else {
          if (a.lse != nullptr) a.lse[orow] = has ? (m_ref + log2f(l)) * 0.69314718055994531f : -INFINITY;
          if (l != 0.f && !(odd.x + odd.y == 0.f && l < INFINITY)) a.odd[1 + atomicAdd(a.odd, 1)] = (int)orow;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kMma) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Output row (token, query head) from its own visible keys, in fp32, by a
// warp: a lane takes a key of 32, and then four columns of their V. For rows
// that are not finite above; as slow as it is short.
__device__ __noinline__ void odd_row(const TreeArgs& a, size_t orow, int lane) {
  const int t = (int)(orow / a.num_qo_heads), hq = (int)(orow - (size_t)t * a.num_qo_heads);
  const int h = hq / (a.num_qo_heads / a.num_kv_heads);
  int b = 0;  // the last sequence that begins at or before t
  for (int hi = a.batch; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (__ldg(a.cu_q + mid) <= t) b = mid; else hi = mid;
  }
  const int lq = __ldg(a.cu_q + b + 1) - __ldg(a.cu_q + b), lk = __ldg(a.seqused_k + b);
  const int nblk = min((int)(((long long)lk + kBlk - 1) / kBlk), a.max_pages);
  auto value = [&](const uint8_t* rows, int i, bool e4m3) {
    if (e4m3) {
      uint32_t lo, hi;
      e4m3x4_to_f16(__ldg(rows + i), lo, hi);
      return __low2float(*reinterpret_cast<const __half2*>(&lo));
    }
    const uint16_t w = __ldg(reinterpret_cast<const uint16_t*>(rows) + i);
    return a.f16 ? __half2float(__ushort_as_half(w)) : __uint_as_float((uint32_t)w << 16);
  };
  const uint8_t* q = static_cast<const uint8_t*>(a.q) + orow * kHeadDim * 2;
  const int32_t* ids = a.q2k + ((size_t)h * a.total_q + t) * a.topk;
  const int id0 = lane < a.topk ? __ldg(ids + lane) : -1, id1 = lane + 32 < a.topk ? __ldg(ids + lane + 32) : -1;
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < a.topk; ++i) {
    const int id = __shfl_sync(0xffffffffu, i < 32 ? id0 : id1, i & 31);
    // A block listed twice counts once.
    const bool again = (lane < i && id0 == id) || (lane + 32 < i && id1 == id);
    if (__any_sync(0xffffffffu, again) || id < 0 || id >= nblk) continue;
    const int page = __ldg(a.page_table + (size_t)b * a.max_pages + id);
    if (page < 0 || page >= a.num_pages) continue;
    const size_t at = ((size_t)page * a.num_kv_heads + h) * kBlk * kHeadDim * (a.e4m3 ? 1 : 2);
    const long long left = (long long)lk - (long long)id * kBlk;
    const int tail = left < kBlk ? (int)left : kBlk;
    for (int k = 0; k < 4; ++k) {
      const uint32_t see = tree_bits(a.tree_mask + (size_t)t * a.mask_words, a.mask_words,
                                     (long long)id * kBlk - ((long long)lk - lq), k, tail - 1);
      if (see == 0u) continue;
      float s = -INFINITY;
      if ((see >> lane) & 1u) {
        s = 0.f;
#pragma unroll 8
        for (int c = 0; c < kHeadDim; ++c)
          s = fmaf(value(q, c, false), value(a.k_pool + at, (32 * k + lane) * kHeadDim + c, a.e4m3), s);
        s *= a.scale_log2;
      }
      float top = s;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      top = fmaxf(top, m);
      const bool nan = __any_sync(0xffffffffu, s != s);
      if (top == -INFINITY && !nan) continue;
      const float alpha = m == -INFINITY ? 0.f : ex2(m - top);
      const float p = s == -INFINITY ? 0.f : ex2(s - top);
      m = top;
      l *= alpha;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] *= alpha;
      for (int x = 0; x < 32; ++x) {
        const float px = __shfl_sync(0xffffffffu, p, x);
        if (!((see >> x) & 1u)) continue;
        l += px;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[c] = fmaf(px, value(a.v_pool + at, (32 * k + x) * kHeadDim + 4 * lane + c, a.e4m3), acc[c]);
      }
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  auto pack = [&](float x, float y) { return a.f16 ? pack_f16x2(x, y) : pack_bf16x2(x, y); };
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * kHeadDim)[lane] =
      make_uint2(pack(acc[0] * inv, acc[1] * inv), pack(acc[2] * inv, acc[3] * inv));
  if (lane == 0 && a.lse != nullptr) a.lse[orow] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Joins the partials of the unit that is cut at the end of CTA k's range and
// begins within it (the CTAs after it whose first segment is of that unit hold
// the others): with M = max m_i and L = sum 2^(m_i - M) l_i, out = sum
// 2^(m_i - M) O_i / L and lse = (M + log2 L) ln 2, the sums in the order of
// the ranges. A block takes kMergeRows of the unit's rows, a thread four rows
// of four columns; kMergeChunk partials at a time, whose weights go through
// shared memory while their O are on the way. Odd rows are computed here too:
// those that whole units listed, and those that joining finds. Two blocks an
// SM, two partials ahead: 305, 63.5 and 21.8 us for 128 E4M3 requests, 32 and
// one, against 310, 65.2 and 22.3 with blocks of 64 rows, one an SM, and four
// partials ahead.
constexpr int kMergeRows = 32, kMergeThreads = 8 * kMergeRows, kMergeAhead = 2, kMergeChunk = 16;
__global__ void __launch_bounds__(kMergeThreads, 2)
    merge_tree_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ uint32_t s_out[kMergeRows][kHeadDim / 2 + 1];
  __shared__ float s_m[kMergeChunk][kMergeRows], s_l[kMergeChunk][kMergeRows];
  __shared__ int s_end;
  __shared__ uint32_t s_odd[kMergeRows / 32];
  const int k = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grid = gridDim.x;
  if (tid == 0) s_end = grid;
  if (tid < kMergeRows / 32) s_odd[tid] = 0u;
  __syncthreads();
  grid_dependency_wait();
  const int unit = __ldcg(a.cut + k).x, odd = __ldcg(a.odd);
  for (int i = (blockIdx.y * grid + k) * (kMergeThreads / 32) + warp; i < odd;
       i += gridDim.y * grid * (kMergeThreads / 32))
    odd_row(a, (size_t)__ldcg(a.odd + 1 + i), lane);
  if (unit < 0) return;
  for (int i = k + 1 + tid; i < grid; i += kMergeThreads)
    if (__ldcg(a.cut + i).y != unit) atomicMin(&s_end, i);
  const int4 info = __ldg(a.unit_info + 2 * unit);
  const int G = a.num_qo_heads / a.num_kv_heads, h = unit % a.num_kv_heads;
  const int row0 = blockIdx.y * kMergeRows, rows = min(kMergeRows, info.z * G - row0);
  __syncthreads();
  if (rows <= 0) return;
  const int count = s_end - k;
  auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * k + 1 : 2 * (k + i)); };
  const int q = tid % (kMergeRows / 4) * 4, c4 = tid / (kMergeRows / 4);  // first row of four, group of four columns
  const int left = rows - q;                    // rows of the thread's four that exist
  const bool quad = left >= 4 && (a.rows_part & 3) == 0;
  const float* part = a.part_o + (size_t)c4 * 4 * a.rows_part + row0 + q;
  auto load = [&](int i, float4 (&v)[4]) {
    const float* p = part + slot(i) * kHeadDim * a.rows_part;
#pragma unroll
    for (int c = 0; c < 4; ++c, p += a.rows_part)
      v[c] = quad ? __ldcg(reinterpret_cast<const float4*>(p))
                  : make_float4(left > 0 ? __ldcg(p) : 0.f, left > 1 ? __ldcg(p + 1) : 0.f,
                                left > 2 ? __ldcg(p + 2) : 0.f, left > 3 ? __ldcg(p + 3) : 0.f);
  };
  float M[4], L[4], acc[4][4];  // acc: [column][row]
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    M[r] = -INFINITY, L[r] = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c][r] = 0.f;
  }
  for (int i0 = 0; i0 < count; i0 += kMergeChunk) {
    const int n = min(kMergeChunk, count - i0);
    float4 v[kMergeAhead][4];
#pragma unroll
    for (int i = 0; i < kMergeAhead; ++i)
      if (i < n) load(i0 + i, v[i]);
    for (int x = tid; x < n * kMergeRows; x += kMergeThreads) {
      const int i = x / kMergeRows, r = x - i * kMergeRows;
      const size_t at = slot(i0 + i) * a.rows_part + row0 + r;
      s_m[i][r] = r < rows ? __ldcg(a.part_m + at) : -INFINITY;
      s_l[i][r] = r < rows ? __ldcg(a.part_l + at) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float m = M[r];
      for (int i = 0; i < n; ++i) m = fmaxf(m, s_m[i][q + r]);
      const float f = M[r] == -INFINITY ? 0.f : ex2(M[r] - m);
      M[r] = m;
      L[r] *= f;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c][r] *= f;
    }
    for (int j = 0; j < n; j += kMergeAhead) {
#pragma unroll
      for (int i = 0; i < kMergeAhead; ++i) {
        if (j + i >= n) break;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float m = s_m[j + i][q + r];
          const float f = m == -INFINITY ? 0.f : ex2(m - M[r]);
          L[r] += f * s_l[j + i][q + r];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float o = r == 0 ? v[i][c].x : r == 1 ? v[i][c].y : r == 2 ? v[i][c].z : v[i][c].w;
            // A partial without a visible key may hold anything.
            acc[c][r] = f > 0.f ? fmaf(f, o, acc[c][r]) : acc[c][r];
          }
        }
        if (j + i + kMergeAhead < n) load(i0 + j + i + kMergeAhead, v[i]);
      }
    }
    __syncthreads();
  }
  // Through shared memory to whole rows.
  auto pack = [&](float x, float y) { return a.f16 ? pack_f16x2(x, y) : pack_bf16x2(x, y); };
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float inv = L[r] > 0.f ? 1.f / L[r] : 0.f;
    float sum = 0.f;  // NaN where an element is not finite
#pragma unroll
    for (int c = 0; c < 4; ++c) sum = fmaf(acc[c][r], 0.f, sum);
    if (L[r] != 0.f && !(sum == 0.f && L[r] < INFINITY)) atomicOr(&s_odd[(q + r) >> 5], 1u << ((q + r) & 31));
    s_out[q + r][c4 * 2] = pack(acc[0][r] * inv, acc[1][r] * inv);
    s_out[q + r][c4 * 2 + 1] = pack(acc[2][r] * inv, acc[3][r] * inv);
    const int row = row0 + q + r, token = row / G;
    if (c4 == 0 && r < left && a.lse != nullptr)
      a.lse[(size_t)(info.x + token) * a.num_qo_heads + (size_t)h * G + (row - token * G)] =
          L[r] > 0.f ? (M[r] + log2f(L[r])) * 0.69314718055994531f : -INFINITY;
  }
  __syncthreads();
  for (int r = warp; r < rows; r += kMergeThreads / 32) {
    const int row = row0 + r, token = row / G;
    const size_t orow = (size_t)(info.x + token) * a.num_qo_heads + (size_t)h * G + (row - token * G);
    if ((s_odd[r >> 5] >> (r & 31)) & 1u)
      odd_row(a, orow, lane);
    else
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * kHeadDim)[lane] =
          make_uint2(s_out[r][2 * lane], s_out[r][2 * lane + 1]);
  }
}

template <bool FP8, bool F16>
cudaError_t launch_t(const TreeArgs& a, cudaStream_t s) {
  const int optin = device_smem_optin();
  if (optin <= 0) return cudaErrorInvalidDevice;
  size_t smem = sizeof(Smem<FP8>) + 1024;
  if (smem > (size_t)optin) smem = (size_t)optin;
  cudaError_t e = set_smem_limit((const void*)tree_kernel<FP8, F16>, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(tree_kernel<FP8, F16>, dim3(a.grid), Roles<FP8>::kThreads, smem, s, a);
  if (e != cudaSuccess) return e;
  const int rows = a.unit_tokens * (a.num_qo_heads / a.num_kv_heads);
  return launch_dependent(merge_tree_kernel, dim3(a.grid, (rows + kMergeRows - 1) / kMergeRows), kMergeThreads,
                          0, s, a);
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
  const int maps = (a.max_pages + 31) / 32;
  const int smem = (int)sizeof(uint32_t) * (2 * maps + a.unit_tokens * a.words);
  cudaError_t e = set_smem_limit((const void*)tree_union_kernel, smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(tree_union_kernel, dim3(a.max_tiles, a.num_kv_heads), kUnionThreads, smem, s, a);
  if (e != cudaSuccess) return e;
  if (a.e4m3) return launch_t<true, false>(a, s);
  return a.f16 ? launch_t<false, true>(a, s) : launch_t<false, false>(a, s);
}

}  // namespace msa
