// Attention over shared prefixes: units of many rows.
//
// A unit is up to 256 rows (two tiles of 128, a row per TMEM lane) with one KV
// head, over a run of blocks that all of its rows see, or see the beginning
// of. Two streams of (QK^T, softmax, PV) keep the tensor cores busy: while one
// stream's softmax warps turn its S into P, the other's products run. With two
// tiles in the unit the streams are the tiles and share every block; with one
// tile they take the blocks in turn, each with its own O, m and l, and the
// epilogue joins the two. TMEM holds S (P over it) and O of each stream.
//
// S of a block is one product of 128 keys; P of it goes back by halves, in 16 bits
// as the products take it (bf16, or f16 for f16 and E4M3 caches: half a step of it,
// what the output's own rounding is; l adds P before that in 32 bits), so that
// the product of P and V begins while the second half is still exponentials. S
// of the next block takes the place of P once that product is complete.
//
// Roles: warps 0-3 and 4-7 the softmax of stream 0 and 1 (a thread per row),
// warp 8 hands out the pieces, warp 10 brings K and V by TMA, warp 11 issues
// the products of Q and K, warp 9 those of P and V, and for E4M3 caches warps
// 12-15 decode K and V to f16 into the swizzled layout the MMA reads. A unit's
// rows lie anywhere in q, so each softmax thread brings its own row of Q; it
// does so for the next piece before it reads O of this one, so that the next
// piece's first products run under this one's epilogue.
//
// With E4M3 keys Q is f16 too, each row scaled by the power of two that puts
// its largest value just below f16's largest; it comes back with the softmax
// scale. P = 0 times what a page may hold need not be 0: V rows that no row of the
// unit sees are zeroed in shared memory, and of those that some see (a causal
// unit's last tokens) what is not finite; the rows that see it get it in the
// epilogue (add_not_finite).
//
// 64 requests of 4 to 12 drafts over 32000 shared tokens, 64/4 heads: 462 us,
// 1.18 PFLOP/s, the tensor cores 52% busy, issue slots 34%. What bounds it is a
// stream's chain: of the 3770 clocks from one S of it to the next its products
// take 1140, the softmax of both halves 1960, the rest lies between the roles.
// Eight warps a stream, two threads a row that read S twice, took 511 us.
// A unit of one block takes 8700 clocks: its masked block's softmax 3000, its Q
// 1900 (a token's place, then the row), its epilogue 2300, and 1700 until its
// first S. Of 4 prompts' 32 samples (E4M3, 181 us) 112 are left with prompts of
// one block. 4 x 512 tokens over 8192 shared ones: 660 us, 0.88 PFLOP/s, E4M3 674.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "mma_issue.cuh"
#include "prefix_work.cuh"
#include "softmax.cuh"
#include "tmem_wide.cuh"

namespace msa {
namespace {

constexpr int kHalf = 16384;  // 128 rows x 128 bytes, swizzled: half of an operand tile
constexpr int kKSlots = 2;    // K ring (a slot frees when its last QK^T completes)
constexpr int kRawSlots = 2;  // E4M3 blocks as they are, on their way
constexpr int kSegRing = 4;
constexpr uint32_t kColS = 0, kColO = 256;  // TMEM: S of stream s at 128 s, O at 256 + 128 s

template <bool FP8>
struct Roles {
  static constexpr int kSched = 8;    // pieces
  static constexpr int kPv = 9;       // issues the products of P and V
  static constexpr int kKv = 10;      // K and V by TMA
  static constexpr int kQk = 11;      // issues the products of Q and K
  static constexpr int kDecode = 12;  // E4M3: first of the decoding warps
  static constexpr int kDecodeWarps = FP8 ? 4 : 0;
  static constexpr int kThreads = (kDecode + kDecodeWarps) * 32;
  static constexpr int kReaders = 2 + 8 + 1;   // of the piece ring
  static constexpr int kVSlots = FP8 ? 2 : 3;  // V ring (a slot frees when its last PV completes)
};

// What a raw E4M3 slot holds; g == -1: no more.
struct RawTile {
  int g, is_v, rows;  // rows: keys of the block that some row of the unit sees (0: no page)
  int open;           // V: of those, that all rows see
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
  Piece piece[kSegRing];
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  uint64_t q_ready, q_empty;
  uint64_t k_full[kKSlots], k_empty[kKSlots];
  uint64_t v_full[kVSlots], v_empty[kVSlots];
  uint64_t qk_done[2];            // per stream: S readable
  uint64_t p_full[2][2];          // per stream and 64-key half: P written
  uint64_t pv_done[2][2];         // the half's PV complete: its P read, O written
  uint64_t o_done[2], o_free[2];  // per stream: O complete at a piece's end, O read out
  uint64_t ml_full, ml_empty, drain[2];
  float2 ml[128];                 // stream 1's (m, l) for the epilogue that joins the streams
  float q_scale[2][128];          // E4M3, one tile: the rows' softmax scales, of this piece and the next
  uint32_t tmem_base;
  int abort;
  int cleaned;                    // values that are not finite were zeroed in some unit of this CTA
};
// A CTA's shared memory, which begins on 1024 bytes (the kernel looks).
static_assert(sizeof(Smem<false>) <= 227 * 1024 && sizeof(Smem<true>) <= 227 * 1024, "too much shared memory");

// Eight values to 32 aligned bytes.
MSA_DEV void store8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Keys from a piece's first block on that all rows of it see: those of its first row.
MSA_DEV int open_keys(const PrefixArgs& a, const Piece& s) {
  const int G = a.num_qo_heads / a.num_kv_heads;
  const long long lim = min((long long)s.lk, (long long)s.hidden + s.row0 / G + 1) - (long long)s.j0 * kBlk;
  return (int)max(0ll, min(lim, (long long)s.keys));
}
// Of four E4M3 values: all bits of those that are NaN.
MSA_DEV uint32_t not_finite_e4m3(uint32_t x) { return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu); }
// Adds to a row, which its thread has written to `out` or `part`, the values that
// are not finite of the keys [from, to) of its page row: infinite or NaN times any
// probability is that.
template <bool FP8, bool F16>
__device__ __noinline__ void add_not_finite(const PrefixArgs& a, const int32_t* pages, int h, int from, int to, uint16_t* out,
                                            float* part) {
  constexpr int kSize = FP8 ? 1 : 2, kChunk = 16 / kSize, kAhead = 8;
  auto load = [](const uint8_t* at) { return __ldg(reinterpret_cast<const uint4*>(at)); };
  for (int key = from; key < to; ++key) {
    const int page = __ldg(pages + key / kBlk);
    if (page < 0 || page >= a.num_pages) continue;
    const uint8_t* at = a.v_pool + (((size_t)page * a.num_kv_heads + h) * kBlk + key % kBlk) * kHeadDim * kSize;
    uint32_t chunks = 0u;  // a bit for each with such a value
#pragma unroll 1
    for (int b0 = 0; b0 < kHeadDim / kChunk; b0 += kAhead) {
      uint4 x[kAhead];
#pragma unroll
      for (int b = 0; b < kAhead; ++b) x[b] = load(at + (b0 + b) * 16);
#pragma unroll
      for (int b = 0; b < kAhead; ++b) {
        const uint32_t any = FP8 ? not_finite_e4m3(x[b].x) | not_finite_e4m3(x[b].y) | not_finite_e4m3(x[b].z) | not_finite_e4m3(x[b].w)
                                 : not_finite2<F16>(x[b].x) | not_finite2<F16>(x[b].y) | not_finite2<F16>(x[b].z) | not_finite2<F16>(x[b].w);
        chunks |= (any != 0u ? 1u : 0u) << (b0 + b);
      }
    }
    for (; chunks != 0u; chunks &= chunks - 1) {
      const int c0 = (__ffs(chunks) - 1) * kChunk;
#pragma unroll 1
      for (int c = c0; c < c0 + kChunk; ++c) {
        float v;
        if constexpr (FP8) {
          if ((__ldg(at + c) & 0x7f) != 0x7f) continue;
          v = NAN;
        } else {
          const uint16_t w = __ldg(reinterpret_cast<const uint16_t*>(at) + c);
          if (not_finite2<F16>(w) == 0u) continue;
          v = F16 ? __half2float(__ushort_as_half(w)) : __uint_as_float((uint32_t)w << 16);
        }
        if (part != nullptr) {
          part[c] += v;
        } else {
          const float o = F16 ? __half2float(__ushort_as_half(out[c])) : __uint_as_float((uint32_t)out[c] << 16);
          out[c] = (uint16_t)pack_x2<F16>(o + v, 0.f);
        }
      }
    }
  }
}

template <bool FP8, bool F16>
__global__ void __launch_bounds__(Roles<FP8>::kThreads, 1)
    prefix_big_kernel(const __grid_constant__ PrefixArgs a) {
  static_assert(!(FP8 && F16), "E4M3 goes with bf16 q");
  constexpr bool kF16Ops = FP8 || F16;  // the MMAs' operands are f16, else bf16
  constexpr int kCols = FP8 ? 32 : 64;  // columns of S a softmax thread holds (64 would spill with E4M3's roles)
  using R = Roles<FP8>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  {
    uint32_t dyn;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn));
    if (pad + sizeof(Smem<FP8>) > dyn) {
      grid_dependency_wait();
      if (threadIdx.x == 0) atomicOr(a.fault, (unsigned)kFaultCapacity);
      return;
    }
  }
  Smem<FP8>& sm = *reinterpret_cast<Smem<FP8>*>(smem_raw + pad);
  constexpr int kVSlots = R::kVSlots;
  unsigned* fault = a.fault;
  volatile int* abort = &sm.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.num_qo_heads / a.num_kv_heads;

  if (tid == 0) {
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(&sm.seg_full[s], 1);
      mbar_init(&sm.seg_empty[s], R::kReaders);
    }
    mbar_init(&sm.q_ready, 8);
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
      mbar_init(&sm.qk_done[s], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sm.p_full[s][h], 4);
        mbar_init(&sm.pv_done[s][h], 1);
      }
      mbar_init(&sm.o_done[s], 2);
      mbar_init(&sm.o_free[s], 4);
    }
    mbar_init(&sm.ml_full, 4);
    mbar_init(&sm.ml_empty, 4);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    for (int s = 0; s < kRawSlots; ++s) {
      mbar_init(&sm.raw_full[s], 1);
      mbar_init(&sm.raw_empty[s], FP8 ? R::kDecodeWarps : 1);
    }
    sm.abort = 0;
    sm.cleaned = 0;
    fence_mbar_init();
  }
  if (warp == R::kPv) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  grid_dependency_wait();  // the work list
  grid_dependents_launch();

  // The n-th piece of this CTA; false at the end (or when a wait gave up).
  auto read_seg = [&](int n, Piece& s) -> bool {
    const int slot = n % kSegRing;
    if (!mbar_wait_sleep(&sm.seg_full[slot], (n / kSegRing) & 1, fault, kFaultWaitOther, abort)) {
      s.n = -1;
      return false;
    }
    s = sm.piece[slot];
    return s.n >= 0;
  };
  auto release_seg = [&](int n) { mbar_arrive(&sm.seg_empty[n % kSegRing]); };
  auto blocks_of = [](const Piece& s) { return (s.keys + kBlk - 1) / kBlk; };

  if (warp == R::kSched) {
    // ------------------------------------------------------------------ pieces
    Walk walk(a, blockIdx.x);
    Piece s{};
    int4 cut = make_int4(-1, 0, 0, 0);
    for (int n = 0;; ++n) {
      const bool more = walk.next(s);
      const int slot = n % kSegRing;
      bool ok = n < kSegRing ||
                mbar_wait_sleep(&sm.seg_empty[slot], ((n / kSegRing) - 1) & 1, fault, kFaultWaitOther, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        sm.piece[slot] = s;
        mbar_arrive(&sm.seg_full[slot]);
      }
      if (!more) break;
      if (s.alone && !s.whole && s.place >= 0) cut = make_int4(s.e, s.tile_head, 0, 0);
    }
    if (lane == 0) a.cut[blockIdx.x] = cut;
  } else if (warp == R::kQk || warp == R::kPv) {
    // -------------------------------------------------------------- MMA issue
    // A whole warp runs this, so that what an MMA needs stays in uniform
    // registers; one elected lane issues.
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
    Piece s;
    // The next piece with blocks; false at the end.
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
        n = __shfl_sync(0xffffffffu, blocks_of(s), 0);
        dual = __shfl_sync(0xffffffffu, s.rows > 128 ? 1 : 0, 0) != 0;
      }
      return ok;
    };
    if (is_qk) {
      // S takes the place of the stream's P, once the PV that reads it is
      // complete. (MMAs run in the order of their issue where shape and
      // accumulator are the same; these differ in the accumulator.)
      constexpr uint32_t idS = idesc_16bit_f32(128, 128, false, false, kF16Ops);
      const uint64_t dq = sdesc_sw128(smem_u32(&sm.q[0][0][0]), 16, 1024);
      const uint32_t hi = (uint32_t)(dq >> 32), q0 = (uint32_t)dq;
      const uint32_t k0 = (uint32_t)sdesc_sw128(smem_u32(&sm.k[0][0][0]), 16, 1024);
      Ring<kKSlots> rk;
      uint32_t used = 0u, pv_phase = 0u;  // a bit per stream: whether it held a P, and its PV's phase
      while (next_seg()) {
        wait(&sm.q_ready, nseg & 1, kFaultWaitSoftmax);
#pragma unroll 1
        for (int b = 0; ok && b < n; ++b) {
          wait(&sm.k_full[rk.idx], rk.phase, kFaultWaitTma);
          const int x_end = dual ? 2 : 1;
#pragma unroll 1
          for (int x = 0; ok && x < x_end; ++x) {
            const int st = dual ? x : b & 1;
            const uint32_t bit = 1u << st;
            if (used & bit) {
              wait(&sm.pv_done[st][1], (pv_phase & bit) != 0u, kFaultWaitMma);
              if (!ok) break;
              pv_phase ^= bit;
            }
            used |= bit;
            tc_fence_after();
            const uint32_t q = q0 + (dual ? st : 0) * kTile16, k = k0 + rk.idx * kTile16;
            const uint32_t d = tb + kColS + st * 128;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = (kk >> 2) * kHalf16 + (kk & 3) * 2;
              mma_ss_if(el, d, q + off, k + off, hi, idS, kk > 0);
            }
            commit(&sm.qk_done[st]);
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
            const int st = dual ? x >> 1 : t & 1, h = x & 1;
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
              if (t + ahead >= n) {
                commit(&sm.o_done[st]);
                // And what this warp waited for: sm.cleaned of this piece.
                if (lane == 0) mbar_arrive(&sm.o_done[st]);
              }
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
    // The tiles of all pieces, one after the other.
    Piece s{};
    int ni = 0, x = 0, n = 0, g0 = 0;  // pieces read, tiles taken of this one, its blocks, blocks before it
    bool ok = true, more = true;
    // Pages of 32 blocks at a time, for K and for V apart (a page outside the
    // pool reads as zeros and is masked).
    const int32_t* prow = nullptr;
    int page_k = -1, page_v = -1;
    struct Tile {
      int g, page, is_v, h, rows, open;  // rows, open: as of a raw tile
    };
    int open = 0;
    // The next tile, warp-wide; false at the end.
    auto take = [&](Tile& t) -> bool {
      while (more && x == 2 * n) {
        g0 += n;
        x = n = 0;
        more = read_seg(ni, s);
        __syncwarp();
        if (!more) {
          ok = *abort == 0;
          break;
        }
        if (lane == 0) release_seg(ni);
        ++ni;
        n = blocks_of(s);
        open = open_keys(a, s);
        prow = a.page_table + (size_t)s.b * a.max_pages + s.j0;
      }
      if (!more) return false;
      bool is_v;
      const int j = tile_order(x, n, is_v);
      ++x;
      auto fetch = [&](int& page) {
        if ((j & 31) == 0) {
          page = j + lane < n ? __ldg(prow + j + lane) : -1;
          if (page < 0 || page >= a.num_pages) page = a.num_pages;
        }
      };
      if (is_v) fetch(page_v);
      else fetch(page_k);
      t.page = __shfl_sync(0xffffffffu, is_v ? page_v : page_k, j & 31);
      t.g = g0 + j;
      t.is_v = is_v;
      t.h = s.h;
      t.rows = min(s.keys - j * kBlk, kBlk);
      t.open = open - j * kBlk;
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
          const int rows = t.page >= a.num_pages ? 0 : t.rows;
          ok = put(RawTile{t.g, t.is_v, rows, t.is_v ? t.open : kBlk},
                   (t.is_v ? a.v_pool : a.k_pool) + ((size_t)(rows > 0 ? t.page : 0) * a.num_kv_heads + t.h) * kHalf);
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      }
      if (lane == 0) {
        if (ok) ok = put(RawTile{-1, 0, 0, kBlk}, nullptr);
        // Copies in flight land before the CTA's shared memory is given back.
        if (!ok)
          for (int i = y < kRawSlots ? 0 : y - kRawSlots; i < y; ++i)
            mbar_wait_sleep(&sm.raw_full[i % kRawSlots], (i / kRawSlots) & 1, fault, kFaultWaitTma);
      }
    }
  } else if (FP8 && warp >= R::kDecode) {
    // ------------------------------------------------------------- E4M3 to f16
    // 128 threads take a block's 128 rows of 128 bytes as eight 16-byte groups
    // each, give the raw slot back, and write f16. Rows that no row of the unit sees
    // become zeros, NaN of those that not all see too.
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
      if (t.open < t.rows) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (r0 + c * 16 < t.open) continue;
          const uint4 x = raw[c], m = make_uint4(not_finite_e4m3(x.x), not_finite_e4m3(x.y), not_finite_e4m3(x.z), not_finite_e4m3(x.w));
          if (m.x | m.y | m.z | m.w) {
            raw[c] = make_uint4(x.x & ~m.x, x.y & ~m.y, x.z & ~m.z, x.w & ~m.w);
            *const_cast<volatile int*>(&sm.cleaned) = 1;
          }
        }
      }
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
    const uint32_t lanes = tbase + ((uint32_t)(q4 * 32) << 16);
    const uint32_t scol = lanes + kColS + st * 128;
    bool ok = true;
    int g0 = 0;               // blocks before this piece
    uint32_t nqk = 0;         // S tiles consumed by this stream
    uint32_t no[2] = {0, 0};  // O completions so far, per stream
    uint32_t nml = 0;         // pieces whose streams were joined
    int loaded = 0;           // pieces whose Q was brought
    float own_scale = a.scale_log2;  // of the row whose Q this thread brought last

    // Brings this thread's row of Q of a piece, once the products that read
    // the Q before are complete.
    auto load_q = [&](const Piece& s) -> bool {
      const bool dual = s.rows > 128;
      if (loaded > 0) {
        bool free = mbar_wait_sleep(&sm.q_empty, (loaded - 1) & 1, fault, kFaultWaitMma, abort);
        if (!__all_sync(0xffffffffu, free)) return false;
      }
      if (dual || st == 0) {
        const int r = (dual ? st * 128 : 0) + row, er = s.row0 + r;
        uint4 x[16];
        if (r < s.rows) {
          const int token = __ldcg(&a.token[s.tau + er / G].x);
          const uint4* q = static_cast<const uint4*>(a.q) +
                           ((size_t)token * a.num_qo_heads + (size_t)s.h * G + er % G) * (kHeadDim / 8);
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] = __ldg(q + c);
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        uint8_t* qt = &sm.q[dual ? st : 0][0][0];
        if constexpr (FP8) {
          // bf16 to f16 times 2^k.
          uint32_t big = 0u;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint32_t xs[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) big = max(big, max(xs[i] & 0x7f80u, (xs[i] >> 16) & 0x7f80u));
          }
          const int e = (int)(big >> 7);  // exponent field of the row's largest value
          const int k = e == 255 ? 0 : min(120, 142 - e);
          const float up = __uint_as_float((uint32_t)(127 + k) << 23);
          own_scale = scale_down(a.scale_log2, k);
          if (!dual) sm.q_scale[loaded & 1][row] = own_scale;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint32_t xs[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[i] = pack_f16x2(__uint_as_float(xs[i] << 16) * up, __uint_as_float(xs[i] & 0xffff0000u) * up);
            x[c] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<uint4*>(qt + (c >> 3) * kHalf + sw128_offset(row, c & 7)) = x[c];
        fence_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&sm.q_ready);
      ++loaded;
      return true;
    };
    // Where a row's parts of a piece go.
    auto place_of = [&](const Piece& s, int r) -> size_t {
      const int er = s.row0 + r;
      return s.place >= 0 ? first_part(a, (size_t)(s.place + er / G) * a.num_qo_heads + (size_t)s.h * G + er % G, blockIdx.x, r)
                          : a.part_rows + (size_t)blockIdx.x * kBigRows + r;
    };

    auto out_row = [&](const Piece& s, int r) -> size_t {
      const int er = s.row0 + r;
      return (size_t)__ldcg(&a.token[s.tau + er / G].x) * a.num_qo_heads + (size_t)s.h * G + er % G;
    };

    // The next piece with blocks; what rows of pieces without any get is here
    // too: nothing seen.
    Piece s, next;
    int ni = 0;
    auto next_piece = [&](Piece& p) -> bool {
      while (true) {
        const bool more = read_seg(ni, p);
        __syncwarp();
        if (!more) return false;
        if (lane == 0) release_seg(ni);
        ++ni;
        if (blocks_of(p) > 0) return true;
        const int r = st * 128 + row;
        if (r >= p.rows) continue;
        if (p.alone && p.whole) {
          const size_t orow = out_row(p, r);
          uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * kHeadDim);
#pragma unroll
          for (int c = 0; c < 16; ++c) to[c] = make_uint4(0u, 0u, 0u, 0u);
          if (a.lse != nullptr) a.lse[orow] = -INFINITY;
        } else {
          a.part_ml[place_of(p, r)] = make_float2(-INFINITY, 0.f);
        }
      }
    };
    bool more = next_piece(next) && load_q(next);
    for (int nseg = 0; more; ++nseg) {
      s = next;
      const bool dual = s.rows > 128;
      const int r = (dual ? st * 128 : 0) + row;  // of the unit
      const bool active = r < s.rows;
      float scale = FP8 ? own_scale : a.scale_log2;  // of the row's S, to log2 units
      if (FP8 && !dual && st == 1) {
        ok = mbar_wait_sleep(&sm.q_ready, nseg & 1, fault, kFaultWaitSoftmax, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        scale = sm.q_scale[nseg & 1][row];
      }
      const int n = blocks_of(s), own = dual ? n : (n + 1 - st) / 2, step = dual ? 1 : 2;
      const int32_t* prow = a.page_table + (size_t)s.b * a.max_pages + s.j0;
      // Keys that the row sees, and that all rows see, from the piece's first on.
      int sees;
      {
        const long long lim = min((long long)s.lk, (long long)s.hidden + (s.row0 + r) / G + 1) - (long long)s.j0 * kBlk;
        sees = active ? (int)max(0ll, min(lim, (long long)n * kBlk)) : 0;
      }
      const int open = open_keys(a, s);
      float m_ref = -INFINITY, l = 0.f;
      int j = dual ? 0 : st;
      int pg1 = own > 0 ? __ldg(prow + j) : 0;
      for (int t = 0; t < own; ++t, j += step) {
        const int pg = pg1;
        if (t + 1 < own) pg1 = __ldg(prow + j + step);
        const int cols = pg >= 0 && pg < a.num_pages ? min(sees - j * kBlk, kBlk) : 0;  // that the row sees
        const bool mem = cols > 0;
        const bool warp_mem = __any_sync(0xffffffffu, mem);
        const bool warp_hides = __any_sync(0xffffffffu, active && cols < kBlk);
        if (!FP8 && open - j * kBlk < kBlk && (st == 0 || !dual)) {
          // V rows that not all rows see, before the first PV that reads the block
          // (in a unit of two tiles stream 0's, which is issued first). The wait
          // for the slot's phase needs the phase before it complete: V of the
          // block kVSlots earlier is there once this block's S is, as S of a
          // stream waits for the PV of its block before, and PVs are issued in
          // the order of the blocks: one of the last two.
          const int g = g0 + j, vs = g % kVSlots;
          ok = mbar_wait_sleep(&sm.qk_done[st], nqk & 1, fault, kFaultWaitMma, abort) &&
               mbar_wait_sleep(&sm.v_full[vs], (g / kVSlots) & 1, fault, kFaultWaitTma, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int seen = s.keys - j * kBlk;  // by some row
          for (int i = max(open - j * kBlk, 0) * 16 + row; i < 128 * 16; i += 128) {
            uint4* at = reinterpret_cast<uint4*>(&sm.v[vs][(i >> 3) & 1][(i >> 4) * 128 + (i & 7) * 16]);
            if ((i >> 4) >= seen) {
              *at = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            const uint4 x = *at, m = make_uint4(not_finite2<F16>(x.x), not_finite2<F16>(x.y), not_finite2<F16>(x.z), not_finite2<F16>(x.w));
            if (m.x | m.y | m.z | m.w) {
              *at = make_uint4(x.x & ~m.x, x.y & ~m.y, x.z & ~m.z, x.w & ~m.w);
              *const_cast<volatile int*>(&sm.cleaned) = 1;
            }
          }
          fence_async_smem();
        }
        ok = mbar_wait_sleep(&sm.qk_done[st], nqk & 1, fault, kFaultWaitMma, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint32_t hcol = scol + half * 64;  // P over the first half of its own S
          if (warp_mem) {
            if (warp_hides) {
              // Few blocks: eight columns at a time, written back to S.
              const int seen = cols - half * 64;
#pragma unroll 1
              for (int c = 0; c < 64; c += 8) {
                uint32_t x[8];
                tmem_ld8_nowait(hcol + c, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = c + i < seen ? x[i] : 0xff800000u;
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
              // O has to hold the half before: this block's first. (That of the
              // block before is complete, as this S was issued after it.)
              if (half == 1) {
                ok = mbar_wait_sleep(&sm.pv_done[st][0], nqk & 1, fault, kFaultWaitMma, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
              }
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
      // The next piece's Q, then this one's epilogue.
      more = next_piece(next);
      if (more && !load_q(next)) break;
      // ------------------------------------------------------------ epilogue
      float f[2] = {1.f, 0.f};
      uint32_t from[2] = {lanes + kColO + st * 128, 0u};
      if (!dual) {
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
      const bool joins = !dual && n > 1;
      // A unit that is all of its rows' is written, others leave their parts.
      const bool writes = s.alone && s.whole;
      const size_t at = !active ? 0 : writes ? out_row(s, r) : place_of(s, r);
      const bool has = l != 0.f;
      const float inv = has ? 1.f / l : 0.f;
#pragma unroll 1
      for (int c0q = 0; c0q < 128; c0q += 32) {
        float o[32];
        tmem_ld32(from[0] + c0q, o);
        if (joins) {
          float o1[32];
          tmem_ld32(from[1] + c0q, o1);
          // A stream that saw nothing may hold anything.
#pragma unroll
          for (int c = 0; c < 32; ++c)
            o[c] = (f[0] > 0.f ? f[0] * o[c] : 0.f) + (f[1] > 0.f ? f[1] * o1[c] : 0.f);
        }
        if (c0q == 96) {
          // O is read: the next piece's first PV may overwrite it.
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.o_free[st]);
            if (!dual) mbar_arrive(&sm.o_free[1]);
          }
        }
        if (active && writes) {
          uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * kHeadDim + c0q);
#pragma unroll
          for (int c = 0; c < 32; c += 8)
            to[c >> 3] = has ? make_uint4(pack_x2<F16>(o[c] * inv, o[c + 1] * inv), pack_x2<F16>(o[c + 2] * inv, o[c + 3] * inv),
                                          pack_x2<F16>(o[c + 4] * inv, o[c + 5] * inv), pack_x2<F16>(o[c + 6] * inv, o[c + 7] * inv))
                             : make_uint4(0u, 0u, 0u, 0u);
        } else if (active) {
          float* to = a.part_o + at * kHeadDim + c0q;
#pragma unroll
          for (int c = 0; c < 32; c += 8) store8(to + c, o + c);
        }
        __syncwarp();
      }
      if (active && writes) {
        if (a.lse != nullptr) a.lse[at] = has ? (m_ref + log2f(l)) * 0.69314718055994531f : -INFINITY;
      } else if (active) {
        a.part_ml[at] = part_of_sum(m_ref, l);
      }
      if (active && has && open < sees && *const_cast<volatile int*>(&sm.cleaned))
        add_not_finite<FP8, F16>(a, prow, s.h, open, sees, writes ? static_cast<uint16_t*>(a.out) + at * kHeadDim : nullptr,
                                 writes ? nullptr : a.part_o + at * kHeadDim);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kPv) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <bool FP8, bool F16>
cudaError_t launch_t(const PrefixArgs& a, cudaStream_t s) {
  const int optin = device_smem_optin();
  if (optin <= 0) return cudaErrorInvalidDevice;
  size_t smem = sizeof(Smem<FP8>) + 1024;
  if (smem > (size_t)optin) smem = (size_t)optin;
  const cudaError_t e = set_smem_limit((const void*)prefix_big_kernel<FP8, F16>, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(prefix_big_kernel<FP8, F16>, dim3(a.grid), Roles<FP8>::kThreads, smem, s, a);
}

}  // namespace

cudaError_t launch_prefix_big(const PrefixArgs& a, cudaStream_t s) {
  if (a.e4m3) return launch_t<true, false>(a, s);
  return a.f16 ? launch_t<false, true>(a, s) : launch_t<false, false>(a, s);
}

}  // namespace msa
