// Attention over a paged cache in which groups of requests share their first
// pages: those are attended once for all tokens of a group.
//
// Each request's tokens attend to all of its keys, so a row (token, query head)
// is the softmax over two runs of blocks: its group's and its own. Both are
// entries of a work list, with the rows that attend them (a group's, all of its
// tokens' rows), and a row's parts (m, l, O) of each run are joined at the end:
// with M = max m_i and L = sum 2^(m_i - M) l_i, out = sum 2^(m_i - M) O_i / L.
//
// An entry's rows are cut into tiles and, with each KV head, units; the units'
// blocks, laid end to end, are cut into equal ranges, one per CTA, wherever
// they end: a long run is split over many CTAs, short ones share one. The first
// piece of a unit leaves its parts at the rows' own places, the others (a CTA
// has one at most, its first) at the CTA's. Without groups only units that are
// cut leave parts, so that a CTA has at most one first piece that does (its last):
// where rows are many, those lie at the CTA's too.
//
// Where the call names no groups and bounds every request's rows by 16 for each
// KV head, the units are of 16 rows and this file's kernel takes them; else they
// are of 256, prefix_big.cu's (the host does not read the arrays: with groups that
// share nothing, 32 requests of 4096 to 65536 keys take 338 us by the one and the
// other, with E4M3 keys 284 by this and 298 by that). A unit that is a request's
// alone and that one CTA has whole is written there and then; what is left is
// joined by the last kernel.
#include <cuda_fp16.h>
#include <math.h>

#include <climits>

#include "common.cuh"
#include "internal.h"
#include "prefix_work.cuh"
#include "softmax.cuh"

namespace msa {
namespace {

template <class T>
MSA_DEV T warp_upto(T v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}
constexpr int kPlanThreads = 1024;
// Running sums that stop at kMany, above any number of tokens there is: those of
// requests that are listed over and over would pass 32 bits. Every thread has to
// come to the block's.
constexpr unsigned kMany = 1u << 30;
MSA_DEV unsigned warp_tokens_upto(unsigned v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v = min(v + o, kMany);
  }
  return v;
}
MSA_DEV unsigned block_tokens_upto(unsigned v, unsigned* s_warp, unsigned& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned inc = warp_tokens_upto(v, lane);
  __syncthreads();
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  const unsigned w = warp_tokens_upto(s_warp[lane], lane);
  all = __shfl_sync(0xffffffffu, w, 31);
  const unsigned before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return min(inc + (warp > 0 ? before : 0u), kMany);
}

// Two running sums over a block; every thread has to come.
struct Sums {
  long long cost, counts;
};
MSA_DEV Sums block_sums(Sums x, Sums* s_warp, Sums& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = {warp_upto(x.cost, lane), warp_upto(x.counts, lane)};
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  Sums w = s_warp[lane];
  w = {warp_upto(w.cost, lane), warp_upto(w.counts, lane)};
  all = {__shfl_sync(0xffffffffu, w.cost, 31), __shfl_sync(0xffffffffu, w.counts, 31)};
  const int from = warp > 0 ? warp - 1 : 0;
  const Sums before{__shfl_sync(0xffffffffu, w.cost, from), __shfl_sync(0xffffffffu, w.counts, from)};
  if (warp > 0) x.cost += before.cost, x.counts += before.counts;
  return x;
}

// The work, by one block: the requests in the order of their groups, where
// their tokens begin in that order, the blocks that each group attends for
// all, the entries and the running sums of what they cost. Bound by the latency
// of its loads and sums: 7 us for 8 requests, 10 for 128 of 4 prompts.
__global__ void __launch_bounds__(kPlanThreads)
    prefix_plan_kernel(const __grid_constant__ PrefixArgs a) {
  extern __shared__ int dyn[];
  __shared__ Sums s_sums[32];
  __shared__ unsigned s_int[32];
  int* least = dyn;           // (batch): blocks that a group attends for all
  int* upto = dyn + a.batch;  // (batch): a group's tokens end before this one
  uint32_t* several = reinterpret_cast<uint32_t*>(dyn + 2 * a.batch);             // a bit per group: more than one request has some
  uint16_t* begins = reinterpret_cast<uint16_t*>(several + (a.batch + 31) / 32);  // (batch): cu_groups
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.num_qo_heads / a.num_kv_heads;
  grid_dependency_wait();
  grid_dependents_launch();
  const bool groups = a.group_rows != nullptr;
  // Up to a thread each the requests stay in registers from the first pass to
  // the second.
  int b = -1, t0 = 0, t1 = 0, lk = 0;
  auto request = [&](int i) {
    b = groups ? __ldg(a.group_rows + i) : i;
    t0 = t1 = lk = 0;
    if (b >= 0 && b < a.batch) {
      t0 = __ldg(a.cu_q + b), t1 = __ldg(a.cu_q + b + 1);
      lk = max(0, __ldg(a.seqused_k + b));
    }
  };
  if (tid < a.batch) request(tid);
  for (int g = tid; g < a.batch; g += kPlanThreads) {
    least[g] = groups ? max(0, min(__ldg(a.group_blocks + g), a.max_pages)) : 0;
    upto[g] = 0;
    begins[g] = (uint16_t)(groups ? max(0, min(__ldg(a.cu_groups + g), 65535)) : g);
    if ((g & 31) == 0) several[g >> 5] = 0u;
  }
  for (int i = tid; i < a.grid; i += kPlanThreads) a.cut[i] = make_int4(-1, 0, 0, 0);
  __syncthreads();
  unsigned before = 0u;
  int tau = 0, lq = 0, g = 0;
  for (int i0 = 0; i0 < a.batch; i0 += kPlanThreads) {
    const int i = i0 + tid;
    lq = 0;
    if (i < a.batch) {
      if (i0 > 0) request(i);
      if (t0 >= 0 && t1 <= a.total_q && t1 > t0) lq = t1 - t0;
      g = i;
      if (groups) {
        int lo = 0;  // the last group that begins at or before i
        for (int hi = a.batch; hi - lo > 1;) {
          const int mid = (lo + hi) >> 1;
          if (begins[mid] <= i) lo = mid; else hi = mid;
        }
        // Requests listed before any group begins are in none. (Groups that do
        // not ascend break the contract, but every place that is read lies among
        // the tokens there are: a group's run goes from its first request's on to
        // the last that is found to be in it.)
        g = begins[lo] <= i ? lo : -1;
      }
    }
    unsigned all;
    tau = (int)min(before + block_tokens_upto((unsigned)lq, s_int, all), kMany) - lq;
    before = min(before + all, kMany);
    if (i < a.batch) {
      // With requests listed twice the sums may pass the tokens there are: the
      // rest is left out.
      if (lq > a.total_q - tau) lq = 0;
      a.entry[2 * i] = make_int4(tau, lq, b, g);
      a.entry[2 * i + 1] = make_int4(t0, lk - lq, lk, -1);
      if (lq > 0 && g >= 0) {
        atomicMin(&least[g], max(0, lk - lq) / kBlk);
        if (atomicMax(&upto[g], tau + lq) > 0) atomicOr(&several[g >> 5], 1u << (g & 31));
      }
    }
  }
  __syncthreads();
  Sums base{};  // cost; entries, and chunks from bit 32
  const int tile = tile_rows_of(a);
  for (int e0 = 0; e0 < 2 * a.batch; e0 += kPlanThreads) {
    const int e = e0 + tid, eg = e - a.batch;
    int4 x = make_int4(0, 0, 0, 0), y = make_int4(0, 0, 0, 0);
    bool there = false, joined = false;
    if (e < a.batch) {
      int4 r, s;
      if (e0 == 0 && a.batch <= kPlanThreads) r = make_int4(tau, lq, b, g), s = make_int4(t0, lk - lq, lk, -1);
      else r = a.entry[2 * e], s = a.entry[2 * e + 1];
      const bool shares = r.w >= 0 && ((several[r.w >> 5] >> (r.w & 31)) & 1u);
      const int from = shares ? least[r.w] : 0;
      const int blocks = (int)min((long long)a.max_pages, ((long long)s.z + kBlk - 1) / kBlk);
      x = make_int4(r.x, r.y * G, r.z, from);
      y = make_int4(max(0, blocks - from), a.causal ? s.y : s.z, s.z, from > 0 ? r.w : -1);
      there = r.y > 0;
      joined = there && from > 0;
    } else if (e < 2 * a.batch && groups && ((several[eg >> 5] >> (eg & 31)) & 1u) && least[eg] > 0) {
      const int first = min((int)begins[eg], a.batch - 1), lead = __ldg(a.group_rows + first);
      const int tau0 = a.entry[2 * first].x;
      x = make_int4(tau0, (upto[eg] - tau0) * G, max(0, min(lead, a.batch - 1)), kGroupRun);
      y = make_int4(least[eg], least[eg] * kBlk, least[eg] * kBlk, -1);
      there = true;
    }
    Sums mine{};
    if (there) {
      mine.cost = (long long)((x.y + tile - 1) / tile) * a.num_kv_heads * (unit_cost(a) + (long long)y.x * block_cost(a, x.y));
      mine.counts = 1 + (joined ? (long long)((x.y + a.chunk_rows - 1) / a.chunk_rows) * a.num_kv_heads << 32 : 0);
    }
    Sums all;
    const Sums sums = block_sums(mine, s_sums, all);
    const long long counts = base.counts + sums.counts - mine.counts;
    const int at = (int)counts;
    if (there) {
      a.start[at] = base.cost + sums.cost - mine.cost;
      a.chunk[at] = (int)(counts >> 32);
      a.work[2 * at] = x;
      a.work[2 * at + 1] = y;
    }
    if (e < a.batch) a.entry[2 * e + 1].w = there ? at : -1;
    else if (e < 2 * a.batch) a.group[eg] = there ? at : -1;
    base = {base.cost + all.cost, base.counts + all.counts};
  }
  if (tid == 0) {
    const int n = (int)base.counts;
    a.start[n] = base.cost;
    a.chunk[n] = (int)(base.counts >> 32);
    a.meta[0] = n;
  }
  // Each token's place in the groups' order, a warp for each request.
  for (int i = warp; i < a.batch; i += kPlanThreads / 32) {
    const int4 x = a.entry[2 * i];
    const int first = a.entry[2 * i + 1].x;
    for (int j = lane; j < x.y; j += 32) a.token[x.x + j] = make_int2(first + j, i);
  }
}

// ------------------------------------------------------- few rows: 16 a tile
// Eight warps take 16 keys each of a block, all 16 rows: S by warp-level MMAs
// (the rows are too few for a tile of 128), its own softmax (m, l) and its own
// O, so a warp waits for no other until the piece ends, where the eight are
// joined. Bound by memory: a block of 64 KB takes an SM's share of the
// bandwidth 3000 clocks. P is rounded to the products' type (bf16, or f16 for f16
// and E4M3 caches: below 2^-25 of a part's largest it is 0 there), l is a sum in 32
// bits of P before that: half a step of the type on each, which the output's own
// rounding equals. One warp hands out the pieces with their Q, another
// brings K and V by TMA through a ring of blocks; the join borrows the next
// free slots of that ring. 32 requests of 4096 to 65536 keys, 4 KV heads,
// 16 bits: 338 to 345 us, 6.6 to 6.75 TB/s, what a copy reaches. E4M3 caches have half the
// bytes and the same MMAs, 256 a block, which bound them then (2000 clocks): 284
// us, 4.0 TB/s.
constexpr int kWarps = 8;
template <int KV>  // 0 bf16, 1 f16, 2 E4M3 with bf16 q
struct Small {
  static constexpr int kSize = KV == 2 ? 1 : 2;
  static constexpr int kTile = 128 * 128 * kSize;  // K or V of a block
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = KV == 2 ? 6 : 3;
  static constexpr int kJoin = kWarps * 16 * 128 * 4 / kStage;  // slots that eight O fill
  static constexpr int kThreads = (kWarps + 2) * 32;
};
constexpr int kPieces = 4;  // of the ring that hands them out
constexpr int kQStride = 272;  // bytes of a row of Q in shared memory
template <int KV>
struct __align__(1024) SmallSmem {
  uint8_t stage[Small<KV>::kStages][Small<KV>::kStage];
  uint8_t q[kPieces][16 * kQStride];
  Piece piece[kPieces];
  float2 ml[2][kWarps][16];
  int page_ok[Small<KV>::kStages];
  uint64_t piece_full[kPieces], piece_empty[kPieces], full[Small<KV>::kStages], empty[Small<KV>::kStages], join;
  int abort;
};
static_assert(sizeof(SmallSmem<0>) <= 226 * 1024 && sizeof(SmallSmem<2>) <= 226 * 1024, "too much shared memory");

MSA_DEV void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
MSA_DEV void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
MSA_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
MSA_DEV uint32_t e4m3x2_to_f16(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return h;
}
// Of two keys' 16 bits each: those below `n` kept.
MSA_DEV uint32_t keep_keys(int first, int n) { return (first < n ? 0xffffu : 0u) | (first + 1 < n ? 0xffff0000u : 0u); }

template <int KV>
__global__ void __launch_bounds__(Small<KV>::kThreads, 1)
    prefix_small_kernel(const __grid_constant__ PrefixArgs a) {
  using C = Small<KV>;
  constexpr bool kF16 = KV != 0;  // the MMAs' operands
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  SmallSmem<KV>& sm = *reinterpret_cast<SmallSmem<KV>*>(smem_raw + pad);
  unsigned* fault = a.fault;
  volatile int* abort = &sm.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.num_qo_heads / a.num_kv_heads;
  if (tid == 0) {
    for (int s = 0; s < kPieces; ++s) {
      mbar_init(&sm.piece_full[s], 33);
      mbar_init(&sm.piece_empty[s], kWarps + 1);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], kWarps);
    }
    mbar_init(&sm.join, kWarps);
    sm.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_launch();

  if (warp == kWarps) {
    // ------------------------------------------------------------ pieces and Q
    Walk walk(a, blockIdx.x);
    Piece p{};
    int e = -1, row0 = -1;
    uint32_t from[8];  // a lane's eight of the tile's sixteen-byte groups: token of the row, times heads
    int4 cut = make_int4(-1, 0, 0, 0);
    for (int np = 0;; ++np) {
      const bool more = walk.next(p);
      const int slot = np % kPieces;
      bool ok = np < kPieces ||
                mbar_wait_sleep(&sm.piece_empty[slot], ((np / kPieces) - 1) & 1, fault, kFaultWaitSoftmax, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (more) {
        // Q's rows of the tile, zeros behind them. A lane has 16 bytes of each
        // second row.
        const int c = lane & 15;
        if (p.e != e || p.row0 != row0) {
          e = p.e, row0 = p.row0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 2 * i + (lane >> 4), row = row0 + r;
            from[i] = r < p.rows ? (uint32_t)__ldcg(&a.token[p.tau + row / G].x) * a.num_qo_heads + row % G : 0u;
          }
        }
        const uint8_t* q = static_cast<const uint8_t*>(a.q) + c * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 2 * i + (lane >> 4);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(sm.q[slot] + r * kQStride + c * 16)),
                       "l"(q + ((size_t)from[i] + (r < p.rows ? p.h * G : 0)) * 256), "r"(r < p.rows ? 16 : 0)
                       : "memory");
        }
        if (!p.whole && p.place >= 0) cut = make_int4(p.e, p.tile_head, 0, 0);
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sm.piece_full[slot])) : "memory");
      if (lane == 0) {
        sm.piece[slot] = p;
        mbar_arrive(&sm.piece_full[slot]);
      }
      __syncwarp();
      if (!more) break;
    }
    if (lane == 0) a.cut[blockIdx.x] = cut;
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  if (warp == kWarps + 1) {
    // ---------------------------------------------------------------- K and V
    if (lane == 0) {
      tma_prefetch_desc(&a.tmap_k);
      tma_prefetch_desc(&a.tmap_v);
    }
    bool ok = true;
    int stage = 0;
    uint32_t turn = 0;  // of the ring: how often it has gone round
    auto acquire = [&]() -> bool {  // the next slot, free
      bool free = turn == 0 || mbar_wait_sleep(&sm.empty[stage], (turn - 1) & 1, fault, kFaultWaitSoftmax, abort);
      return __all_sync(0xffffffffu, free);
    };
    auto advance = [&]() {
      if (++stage == C::kStages) stage = 0, ++turn;
    };
    for (int np = 0; ok; ++np) {
      const int slot = np % kPieces;
      ok = mbar_wait_sleep(&sm.piece_full[slot], (np / kPieces) & 1, fault, kFaultWaitOther, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const Piece p = sm.piece[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.piece_empty[slot]);
      if (p.n < 0) break;
      const int blocks = (p.keys + kBlk - 1) / kBlk;
      const int32_t* pages = a.page_table + (size_t)p.b * a.max_pages + p.j0;
      int page32 = -1;
      for (int j = 0; ok && j < blocks; ++j) {
        if ((j & 31) == 0) page32 = j + lane < blocks ? __ldg(pages + j + lane) : -1;
        const int page = __shfl_sync(0xffffffffu, page32, j & 31);
        ok = acquire();
        if (!ok) break;
        if (lane == 0) {
          const bool there = page >= 0 && page < a.num_pages;
          sm.page_ok[stage] = there;
          if (there) {
            uint8_t* at = sm.stage[stage];
            mbar_expect_tx(&sm.full[stage], C::kStage);
            if constexpr (KV == 2) {
              tma_load_4d(at, &a.tmap_k, &sm.full[stage], 0, 0, p.h, page);
              tma_load_4d(at + C::kTile, &a.tmap_v, &sm.full[stage], 0, 0, p.h, page);
            } else {
              for (int c = 0; c < 2; ++c) {
                tma_load_4d(at + c * 16384, &a.tmap_k, &sm.full[stage], c * 64, 0, p.h, page);
                tma_load_4d(at + C::kTile + c * 16384, &a.tmap_v, &sm.full[stage], c * 64, 0, p.h, page);
              }
            }
          } else {
            mbar_arrive(&sm.full[stage]);
          }
        }
        __syncwarp();
        advance();
      }
      // The slots that the join uses.
      for (int j = 0; ok && j < C::kJoin; ++j) {
        ok = acquire();
        if (!ok) break;
        if (lane == 0) mbar_arrive(&sm.full[stage]);
        advance();
      }
    }
    // Copies in flight land before the CTA's shared memory is given back.
    if (!ok) {
      for (int s = 0; s < C::kStages; ++s) {
        // The slot's last phase: the one of this turn for slots before `stage`.
        const uint32_t t = s < stage ? turn : turn - 1;
        if (s < stage || turn > 0) mbar_wait_sleep(&sm.full[s], t & 1, fault, kFaultWaitTma);
      }
    }
    return;
  }

  // ---------------------------------------------------------------- the warps
  const int g = lane >> 2, t = lane & 3;
  int stage = 0, np = 0;
  uint32_t turn = 0, joins = 0;
  bool ok = true;
  auto advance = [&]() {
    if (++stage == C::kStages) stage = 0, ++turn;
  };
  while (true) {
    const int slot = np % kPieces, ms = np & 1;
    ok = mbar_wait_sleep(&sm.piece_full[slot], (np / kPieces) & 1, fault, kFaultWaitOther, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    ++np;
    const Piece p = sm.piece[slot];
    if (p.n < 0) break;
    // Of the row that this thread writes at the end.
    const int out_row = tid >> 4, er = p.row0 + out_row;
    const int token = out_row < p.rows ? __ldcg(&a.token[p.tau + er / G].x) : 0;
    // Q as the products want it; with E4M3 keys as f16, each row scaled by a
    // power of two that puts its largest value just below f16's largest, and
    // with the dims in the order in which a thread reads K: its 32 of them.
    uint32_t q[8][4];
    float scale[2] = {a.scale_log2, a.scale_log2};
    if constexpr (KV == 2) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t w[16];
        uint32_t big = 0u;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(sm.q[slot] + (g + 8 * r) * kQStride + t * 64 + c * 16);
          w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) big = max(big, max(w[i] & 0x7f80u, (w[i] >> 16) & 0x7f80u));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int e = (int)(big >> 7), k = e == 255 ? 0 : min(120, 142 - e);
        const float up = __uint_as_float((uint32_t)(127 + k) << 23);
        scale[r] = scale_down(a.scale_log2, k);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          q[i >> 1][r + 2 * (i & 1)] = pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        ldmatrix4(q[ks], smem_u32(sm.q[slot] + ((lane & 7) + ((lane >> 3) & 1) * 8) * kQStride + (ks * 2 + (lane >> 4)) * 16));
    }
    // Keys that rows g and g + 8 see, counted from the piece's first.
    int sees[2];
    const long long base = (long long)p.j0 * kBlk;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const long long lim = min((long long)p.lk, (long long)p.hidden + (p.row0 + g + 8 * r) / G + 1) - base;
      sees[r] = (int)max(0ll, min(lim, (long long)p.keys));
    }
    const int all_see = (int)max(0ll, min(min((long long)p.lk, (long long)p.hidden + p.row0 / G + 1) - base, (long long)p.keys));
    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
    const int blocks = (p.keys + kBlk - 1) / kBlk;
    for (int j = 0; j < blocks; ++j) {
      ok = mbar_wait_sleep(&sm.full[stage], turn & 1, fault, kFaultWaitTma, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int k0 = j * kBlk + warp * 16;  // the warp's first key
      if (k0 < p.keys && sm.page_ok[stage]) {
        const uint32_t ks0 = smem_u32(sm.stage[stage]), vs0 = ks0 + C::kTile;
        float s[2][4] = {};
        if constexpr (KV == 2) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int row = warp * 16 + nt * 8 + g;
            const uint8_t* at = sm.stage[stage] + row * 128;
            const uint4 x = *reinterpret_cast<const uint4*>(at + (((2 * t) ^ (row & 7)) << 4));
            const uint4 y = *reinterpret_cast<const uint4*>(at + (((2 * t + 1) ^ (row & 7)) << 4));
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma16816<kF16>(s[nt], q[ks], e4m3x2_to_f16(w[ks] & 0xffffu), e4m3x2_to_f16(w[ks] >> 16));
          }
        } else {
          const int row = warp * 16 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const int c = ks * 2 + ((lane >> 3) & 1);
            uint32_t b[4];
            ldmatrix4(b, ks0 + (c >> 3) * 16384 + sw128_offset(row, c & 7));
            mma16816<kF16>(s[0], q[ks], b[0], b[1]);
            mma16816<kF16>(s[1], q[ks], b[2], b[3]);
          }
        }
        if (k0 + 16 > all_see) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (k0 + nt * 8 + 2 * t + (c & 1) >= sees[c >> 1]) s[nt][c] = -INFINITY;
        }
        // The rows' maxima over the four threads that hold a row.
        bool grows = false;
        float alpha[2] = {1.f, 1.f}, ref[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          update_max(mx != -INFINITY, mx, scale[r], m[r], l[r], alpha[r], grows);
          ref[r] = m[r] == -INFINITY ? 0.f : m[r];
        }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[i][c] *= alpha[c >> 1];
        }
        uint32_t pa[4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = ex2(fmaf(s[nt][2 * r], scale[r], -ref[r])), p1 = ex2(fmaf(s[nt][2 * r + 1], scale[r], -ref[r]));
            l[r] += p0 + p1;
            pa[2 * nt + r] = pack_x2<kF16>(p0, p1);
          }
        // P = 0 times what a page may hold need not be 0. Values that no row sees
        // are zeroed, and of those that some see what is not finite: the rows that
        // see it get it below.
        const bool edge = k0 + 16 > all_see;
        const uint32_t keep0 = keep_keys(k0 + 2 * t, p.keys), keep1 = keep_keys(k0 + 8 + 2 * t, p.keys);
        const uint32_t some0 = ~keep_keys(k0 + 2 * t, all_see), some1 = ~keep_keys(k0 + 8 + 2 * t, all_see);
        uint32_t cleaned = 0u;
        auto clean = [&](uint32_t& x, uint32_t keep, uint32_t some) {
          x &= keep;
          const uint32_t m = not_finite2<kF16>(x) & some;
          cleaned |= m;
          x &= ~m;
        };
        const int vrow = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
        if constexpr (KV == 2) {
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t v[4];
            ldmatrix4_trans(v, vs0 + sw128_offset(vrow, cc * 2 + (lane >> 4)));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t b[2][2];  // [dim parity][keys 0-7, 8-15]
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                b[0][k] = e4m3x2_to_f16(__byte_perm(v[2 * h + k], 0u, 0x4420));
                b[1][k] = e4m3x2_to_f16(__byte_perm(v[2 * h + k], 0u, 0x4431));
                if (edge) clean(b[0][k], k ? keep1 : keep0, k ? some1 : some0), clean(b[1][k], k ? keep1 : keep0, k ? some1 : some0);
              }
              mma16816<kF16>(o[4 * cc + 2 * h], pa, b[0][0], b[0][1]);
              mma16816<kF16>(o[4 * cc + 2 * h + 1], pa, b[1][0], b[1][1]);
            }
          }
        } else {
#pragma unroll
          for (int dn = 0; dn < 8; ++dn) {
            const int c = dn * 2 + (lane >> 4);
            uint32_t v[4];
            ldmatrix4_trans(v, vs0 + (c >> 3) * 16384 + sw128_offset(vrow, c & 7));
            if (edge) clean(v[0], keep0, some0), clean(v[1], keep1, some1), clean(v[2], keep0, some0), clean(v[3], keep1, some1);
            mma16816<kF16>(o[2 * dn], pa, v[0], v[1]);
            mma16816<kF16>(o[2 * dn + 1], pa, v[2], v[3]);
          }
        }
        if (__any_sync(0xffffffffu, cleaned != 0u)) {
          // Infinite or NaN times any probability is that.
#pragma unroll 1
          for (int k = max(k0, all_see); k < min(k0 + 16, p.keys); ++k) {
            const int row = k - j * kBlk;
            const uint8_t* at = sm.stage[stage] + C::kTile;
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // A thread's columns of o[i]: values e and 2 + e are of rows g and g + 8.
                float x;
                if constexpr (KV == 2) {
                  const int col = 16 * (i >> 1) + 4 * t + (i & 1) + 2 * e;
                  x = (at[row * 128 + ((((col >> 4) ^ (row & 7)) << 4) | (col & 15))] & 0x7f) == 0x7f ? NAN : 0.f;
                } else {
                  const int col = 8 * i + 2 * t + e;
                  const uint16_t w = *reinterpret_cast<const uint16_t*>(at + (col >> 6) * 16384 + sw128_offset(row, (col >> 3) & 7) + (col & 7) * 2);
                  x = not_finite2<kF16>(w) == 0u ? 0.f : kF16 ? __half2float(__ushort_as_half(w)) : __uint_as_float((uint32_t)w << 16);
                }
                if (k < sees[0]) o[i][e] += x;
                if (k < sees[1]) o[i][2 + e] += x;
              }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[stage]);
      advance();
    }
    if (!ok) break;
    // ------------------------------------------------------------------ joined
    const int js = stage;
    for (int j = 0; ok && j < C::kJoin; ++j) {
      ok = mbar_wait_sleep(&sm.full[stage], turn & 1, fault, kFaultWaitOther, abort);
      ok = __all_sync(0xffffffffu, ok);
      advance();
    }
    if (!ok) break;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t == 0) sm.ml[ms][warp][g + 8 * r] = part_of_sum(m[r], l[r]);
    }
    // Warp w's O: row r, column c at r * 128 + (c ^ 8 (r & 3)) of its 8 KB.
    auto o_of = [&](int w) -> float* {
      const int byte = w * 8192, s = js + byte / C::kStage;
      return reinterpret_cast<float*>(sm.stage[s >= C::kStages ? s - C::kStages : s] + byte % C::kStage);
    };
    float* mine = o_of(warp);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = g + 8 * r, x = (row & 3) << 3;
      if constexpr (KV == 2) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<float4*>(mine + row * 128 + ((16 * c + 4 * t) ^ x)) =
              make_float4(o[2 * c][2 * r], o[2 * c + 1][2 * r], o[2 * c][2 * r + 1], o[2 * c + 1][2 * r + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          *reinterpret_cast<float2*>(mine + row * 128 + ((8 * i + 2 * t) ^ x)) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.join);
    ok = mbar_wait_sleep(&sm.join, joins & 1, fault, kFaultWaitOther, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    ++joins;
    const int col = (tid & 15) * 8;
    float M = -INFINITY;
    Joined own;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.ml[ms][w][out_row].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sm.ml[ms][w][out_row];
      if (ml.x == -INFINITY) continue;
      const float f = ex2(ml.x - M);
      own.l += f * ml.y;
      const float* from = o_of(w) + out_row * 128 + (col ^ ((out_row & 3) << 3));
      const float4 x = *reinterpret_cast<const float4*>(from), y = *reinterpret_cast<const float4*>(from + 4);
      const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int c = 0; c < 8; ++c) own.o[c] = fmaf(f, v[c], own.o[c]);
    }
    own.m = M;
    fence_async_smem();  // the slots are TMA's again
    __syncwarp();
    if (lane == 0) {
      for (int j = 0, s = js; j < C::kJoin; ++j, s = s + 1 == C::kStages ? 0 : s + 1) mbar_arrive(&sm.empty[s]);
      mbar_arrive(&sm.piece_empty[slot]);
    }
    // The row: written where the unit is whole, else its parts.
    const bool live = out_row < p.rows;
    const size_t hq = (size_t)p.h * G + er % G, own_row = (size_t)(p.tau + er / G) * a.num_qo_heads + hq;
    if (live && p.whole) {
      own.write(a, (size_t)token * a.num_qo_heads + hq, col);
    } else if (live) {
      const size_t at = p.place >= 0 ? first_part(a, own_row, blockIdx.x, out_row) : a.part_rows + (size_t)blockIdx.x * kSmallRows + out_row;
      float4* to = reinterpret_cast<float4*>(a.part_o + at * kHeadDim + col);
      to[0] = make_float4(own.o[0], own.o[1], own.o[2], own.o[3]);
      to[1] = make_float4(own.o[4], own.o[5], own.o[6], own.o[7]);
      if (col == 0) a.part_ml[at] = make_float2(own.m, own.l);
    }
  }
}

// ------------------------------------------------------------------ the join
// Joins what is left: of the requests with a group's run before their own, and
// of the other units that ranges cut. A block takes chunk_rows rows of one KV
// head at a time; each of its warps finds their parts for itself (ten loads one
// after the other: what a chunk of 16 rows mostly takes) and has two of each 16
// rows, 16 lanes each, of eight columns: first the parts of the group's run,
// then those of the own one, in the order of the pieces. In a chunk of fewer rows
// several half-warps take a row's parts by turns, where it has eight or more (8
// samples of 32768 tokens, 38 parts a row: the call 48 -> 41 us; split like that, rows
// of few parts cost the pair of 1300 tokens 1 us). Alone 7 to 18 us for up to 8192
// rows, bound by that search; 32 for 32768.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads)
    prefix_join_kernel(const __grid_constant__ PrefixArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.num_qo_heads / a.num_kv_heads;
  __shared__ Joined s_joined[kJoinThreads / 16][16];
  grid_dependency_wait();
  grid_dependents_launch();
  const int entries = __ldcg(a.meta);
  const Ranges ranges = ranges_of(a, entries);
  const int chunks = __ldcg(a.chunk + entries);
  for (int i = blockIdx.x; i < a.grid + chunks; i += gridDim.x) {
    int e, tile_head, row0, many;
    if (i < a.grid) {
      const int4 cut = __ldcg(a.cut + i);
      e = cut.x, tile_head = cut.y;
      if (e < 0) continue;
      row0 = tile_head / a.num_kv_heads * tile_rows_of(a), many = tile_rows_of(a);
    } else {
      e = last_upto(a.chunk, entries, i - a.grid);
      const int c = i - a.grid - __ldcg(a.chunk + e), r = c / a.num_kv_heads;
      row0 = r * a.chunk_rows, many = a.chunk_rows;
      tile_head = row0 / tile_rows_of(a) * a.num_kv_heads + c - r * a.num_kv_heads;
    }
    const int4* w = a.work + 2 * e;
    const int4 x = __ldcg(w), y = __ldcg(w + 1);
    const int h = tile_head % a.num_kv_heads, rows = min(many, x.y - row0), col = (lane & 15) * 8;
    const Parts parts = parts_of(a, ranges, e, x.y, y.x, tile_head);
    const Before f = before_of(a, ranges, y.w, x.x, row0, rows, h);
    if (i >= a.grid && a.chunk_rows < kJoinThreads / 16 && max(parts.n, max(f.parts[0].n, f.parts[1].n)) >= 8) {
      // Few rows of many parts: several half-warps to a row, whose first joins
      // what the others have.
      const int chunk = a.chunk_rows, step = kJoinThreads / 16 / chunk;
      const int half = 2 * warp + (lane >> 4), from = half / chunk, r = half % chunk, er = row0 + r;
      const size_t hq = (size_t)h * G + er % G, own_row = (size_t)(x.x + er / G) * a.num_qo_heads + hq;
      Joined all;
      if (r < rows) {
        all.add_before(a, f, r, own_row, col, from, step);
        all.add_parts(a, own_row, er % tile_rows_of(a), parts, col, from, step);
      }
      __syncthreads();  // the chunk before is done with
      s_joined[half][lane & 15] = all;
      __syncthreads();
      if (r < rows && from == 0) {
        for (int k = 1; k < step; ++k) {
          const Joined& other = s_joined[half + k * chunk][lane & 15];
          all.add(make_float2(other.m, other.l), other.o);
        }
        all.write(a, (size_t)__ldcg(&a.token[x.x + er / G].x) * a.num_qo_heads + hq, col);
      }
      continue;
    }
#pragma unroll 1
    for (int r0 = 2 * warp; r0 < rows; r0 += kJoinThreads / 16) {
      const int r = r0 + (lane >> 4), er = row0 + r;
      const size_t hq = (size_t)h * G + er % G, own_row = (size_t)(x.x + er / G) * a.num_qo_heads + hq;
      if (r < rows) {
        const int token = __ldcg(&a.token[x.x + er / G].x);
        Joined all;
        all.add_before(a, f, r, own_row, col);
        const int row = er % tile_rows_of(a);
        all.add_parts(a, first_part(a, own_row, parts.c0, row), row, parts, col);
        all.write(a, (size_t)token * a.num_qo_heads + hq, col);
      }
    }
  }
}

template <int KV>
cudaError_t launch_small(const PrefixArgs& a, cudaStream_t s) {
  const int smem = (int)sizeof(SmallSmem<KV>) + 1024;
  cudaError_t e = set_smem_limit((const void*)prefix_small_kernel<KV>, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(prefix_small_kernel<KV>, dim3(a.grid), Small<KV>::kThreads, smem, s, a);
}

}  // namespace

cudaError_t launch_prefix(const PrefixArgs& a, cudaStream_t s) {
  const int smem = (2 * a.batch + (a.batch + 31) / 32) * 4 + (a.batch * 2 + 3) / 4 * 4;
  cudaError_t e = set_smem_limit((const void*)prefix_plan_kernel, smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(prefix_plan_kernel, dim3(1), kPlanThreads, smem, s, a);
  if (e != cudaSuccess) return e;
  e = !a.small ? launch_prefix_big(a, s) : a.e4m3 ? launch_small<2>(a, s) : a.f16 ? launch_small<1>(a, s) : launch_small<0>(a, s);
  if (e != cudaSuccess) return e;
  // Cut units, and as many chunks as there can be: a block each, up to eight an
  // SM.
  const long long chunks = ((long long)a.total_q * a.num_qo_heads + a.chunk_rows - 1) / a.chunk_rows + (long long)a.batch * a.num_kv_heads;
  const long long items = a.grid + (a.group_rows != nullptr ? chunks : 0);
  const long long blocks = items < 8 * a.grid ? items : 8 * a.grid;
  return launch_dependent(prefix_join_kernel, dim3((unsigned)blocks), kJoinThreads, 0, s, a);
}

}  // namespace msa
