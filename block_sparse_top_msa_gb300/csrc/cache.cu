// Pages of a paged cache: accepted drafts moved up, pages copied, sequences
// forked, extended and freed. All of it runs on the device from device
// tables, so a serving loop needs no host copy of them.
//
// Sequences are rows of a page table (an entry of -1 names no page) with
// their lengths, and page_refs counts the entries that name each page; a page
// whose count is 0 is free. Free pages are handed out lowest first, in the
// order of the requests, so the tables that result do not depend on how the
// kernels are scheduled.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace msa {
namespace {

// ------------------------------------------------------------------ accept
// Request b's drafts lie at cache positions first .. first + Lq - 1 (first =
// Lk - Lq). Row first + path[j] moves to first + j. As path ascends, path[j]
// >= j: no destination is a later move's source. A thread owns one 16-byte
// column of a (pool, head) and makes its moves in order, up to kBatch of them
// loaded before the first is stored, so the moves need no buffer.
constexpr int kAcceptThreads = 128;
constexpr int kAcceptBatch = 8;
constexpr int kAcceptChunk = 64;  // moves whose addresses are held at a time

__global__ void __launch_bounds__(kAcceptThreads)
    cache_accept_kernel(const __grid_constant__ CachePools pools,
                        const __grid_constant__ CacheAcceptArgs a) {
  __shared__ long long s_src[kAcceptChunk], s_dst[kAcceptChunk];  // row offsets; -1: no move
  __shared__ int s_len;
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.y;
  const int lq = __ldg(a.cu_q + b + 1) - __ldg(a.cu_q + b);
  const int lk = __ldg(a.seqused_k + b);
  const int first = lk - lq;
  const int32_t* path = a.path + (size_t)b * a.max_path;
  // The path ends before its first entry that does not ascend or names no
  // draft.
  const int said = max(0, min(a.max_path, __ldg(a.path_len + b)));
  if (threadIdx.x == 0) s_len = said;
  __syncthreads();
  for (int j = threadIdx.x; j < said; j += kAcceptThreads) {
    const int p = __ldg(path + j);
    if (p >= lq || p < 0 || (j > 0 && p <= __ldg(path + j - 1))) atomicMin(&s_len, j);
  }
  __syncthreads();
  const int len = s_len;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.seqused_out[b] = max(0, first + len);
  const int chunks16 = a.row_bytes / 16;
  const int columns = a.num_pools * a.hkv * chunks16;
  const int col = blockIdx.x * kAcceptThreads + threadIdx.x;
  const int c = col % chunks16, ph = col / chunks16;
  const int h = ph % a.hkv, pool = ph / a.hkv;
  uint8_t* base = col < columns ? static_cast<uint8_t*>(pools.base[pool]) + c * 16 : nullptr;
  for (int j0 = 0; j0 < len; j0 += kAcceptChunk) {
    const int n = min(kAcceptChunk, len - j0);
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kAcceptThreads) {
      const int p = __ldg(path + j0 + j);
      const long long src = (long long)first + p, dst = (long long)first + j0 + j;
      long long so = -1, dof = -1;
      if (src != dst && dst >= 0 && src < (long long)a.max_pages * kBlk) {
        const int sp = __ldg(a.page_table + (size_t)b * a.max_pages + src / kBlk);
        const int dp = __ldg(a.page_table + (size_t)b * a.max_pages + dst / kBlk);
        if (sp >= 0 && sp < a.num_pages && dp >= 0 && dp < a.num_pages) {
          so = (long long)sp * a.hkv * kBlk + src % kBlk;
          dof = (long long)dp * a.hkv * kBlk + dst % kBlk;
        }
      }
      s_src[j] = so;
      s_dst[j] = dof;
    }
    __syncthreads();
    if (base == nullptr) continue;
    for (int j = 0; j < n; j += kAcceptBatch) {
      uint4 v[kAcceptBatch];
#pragma unroll
      for (int i = 0; i < kAcceptBatch; ++i)
        if (j + i < n && s_src[j + i] >= 0)
          v[i] = *reinterpret_cast<const uint4*>(base + (s_src[j + i] + (long long)h * kBlk) * a.row_bytes);
#pragma unroll
      for (int i = 0; i < kAcceptBatch; ++i)
        if (j + i < n && s_src[j + i] >= 0)
          *reinterpret_cast<uint4*>(base + (s_dst[j + i] + (long long)h * kBlk) * a.row_bytes) = v[i];
    }
  }
}

// -------------------------------------------------------------------- free
constexpr int kFreeThreads = 256;

__global__ void __launch_bounds__(kFreeThreads) cache_free_kernel(const __grid_constant__ CacheTableArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int i = blockIdx.x;
  const int r = __ldg(a.rows + i);
  if (r < 0 || r >= a.num_rows) return;
  // A row listed twice is freed by its first mention.
  bool again = false;
  for (int j = threadIdx.x; j < i; j += kFreeThreads) again |= __ldg(a.rows + j) == r;
  if (__syncthreads_or(again)) return;
  int32_t* row = a.page_table + (size_t)r * a.max_pages;
  for (int t = threadIdx.x; t < a.max_pages; t += kFreeThreads) {
    const int p = row[t];
    if (p >= 0 && p < a.num_pages) atomicAdd(a.page_refs + p, -1);
    if (p != -1) row[t] = -1;
  }
  if (threadIdx.x == 0) a.seqused_k[r] = 0;
}

// ----------------------------------------------------------- fork and extend
constexpr int kPlanThreads = 1024;
constexpr int kScanPerThread = 16;  // page counts a thread reads per step of the free-page search

enum { kDone = 0, kRefused = 1, kNoPage = 2 };

// Exclusive sum over the block's threads and the total; s holds 33.
template <class T>
MSA_DEV T block_exclusive(T v, T* s, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();  // s may still be read from an earlier call
  if (lane == 31) s[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const T w = s[lane];
    T wi = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T o = __shfl_up_sync(0xffffffffu, wi, d);
      if (lane >= d) wi += o;
    }
    s[lane] = wi - w;
    if (lane == 31) s[32] = wi;
  }
  __syncthreads();
  total = s[32];
  return s[warp] + inc - v;
}

// One block. Checks the requests, counts the pages each needs (a fork: one if
// the source ends inside a page; an extension: one for each block below the
// new length without a page, from the block the row ends in on), finds that
// many free pages and grants them in the order of the requests: a request is
// served when it and all before it fit. Extensions are entered into the
// tables here, forks by the kernel after this one.
template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const __grid_constant__ CacheTableArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  extern __shared__ int smem[];
  int* claim = smem;                   // num_rows: the first request for the row
  int* need = claim + a.num_rows;      // n: pages wanted, or -1 refused
  int* offset = need + a.n;            // n: pages wanted before, INT_MAX at most
  int* scan = offset + a.n;            // 33
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int r = tid; r < a.num_rows; r += kPlanThreads) claim[r] = INT_MAX;
  __syncthreads();
  for (int i = tid; i < a.n; i += kPlanThreads) {
    const int r = a.rows[i];
    if (r >= 0 && r < a.num_rows) atomicMin(&claim[r], i);
  }
  __syncthreads();
  // What can be told without reading whole rows, a thread per request.
  for (int i = tid; i < a.n; i += kPlanThreads) {
    const int r = a.rows[i], src = FORK ? a.src_rows[i] : 0, len = FORK ? 0 : a.lengths[i];
    bool ok = r >= 0 && r < a.num_rows && claim[r] == i;
    int want = 0;
    if (FORK) {
      ok = ok && src >= 0 && src < a.num_rows && claim[src] == INT_MAX;
      const int n = ok ? a.seqused_k[src] : 0, own = ok ? a.seqused_k[r] : 0;
      ok = ok && n >= 0 && (long long)n <= (long long)a.max_pages * kBlk && own == 0;
      if (ok && n % kBlk != 0) {
        const int p = a.page_table[(size_t)src * a.max_pages + n / kBlk];
        want = p >= 0 && p < a.num_pages;
      }
    } else {
      const int own = ok ? a.seqused_k[r] : 0;
      ok = ok && len >= own && (long long)len <= (long long)a.max_pages * kBlk;
      // Room for up to four more blocks is counted here, for more below.
      const int first = max(0, own) / kBlk, last = (int)(((long long)len + kBlk - 1) / kBlk);
      if (ok && last - first > 4) {
        want = INT_MAX;
      } else if (ok) {
        const int32_t* row = a.page_table + (size_t)r * a.max_pages;
#pragma unroll
        for (int t = 0; t < 4; ++t) want += first + t < last && row[first + t] < 0;
      }
    }
    need[i] = ok ? want : -1;
  }
  __syncthreads();
  // Whole rows, a warp per request: a row forked to holds no page; the pages
  // that a long extension lacks.
  for (int i = warp; i < a.n; i += kPlanThreads / 32) {
    if (FORK ? need[i] < 0 : need[i] != INT_MAX) continue;
    const int r = a.rows[i];
    const int32_t* row = a.page_table + (size_t)r * a.max_pages;
    int t0 = 0, last = a.max_pages;
    if (!FORK) {
      t0 = max(0, a.seqused_k[r]) / kBlk;
      last = (int)(((long long)a.lengths[i] + kBlk - 1) / kBlk);
    }
    int count = 0;
#pragma unroll 8
    for (int t = t0 + lane; t < last; t += 32) count += FORK ? row[t] >= 0 : row[t] < 0;
    count = __reduce_add_sync(0xffffffffu, count);
    __syncwarp();
    if (lane == 0) {
      if (!FORK) need[i] = count;
      else if (count > 0) need[i] = -1;
    }
  }
  __syncthreads();
  // Pages wanted before each request, in 64 bits: a table's rows together may
  // lack more than 2^31.
  __shared__ long long scan64[33];
  long long sum = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    long long total;
    const long long before = block_exclusive(i < a.n ? (long long)max(0, need[i]) : 0ll, scan64, total);
    if (i < a.n) offset[i] = (int)min(sum + before, (long long)INT_MAX);
    sum += total;
  }
  // The first `sum` free pages, ascending: the next step's counts are on their
  // way while this one's free pages are numbered.
  int found = 0;
  const int wanted = (int)min(sum, (long long)a.num_pages);
  const bool quads = (reinterpret_cast<uintptr_t>(a.page_refs) & 15) == 0;
  int4 held[kScanPerThread / 4];
  const unsigned pages = (unsigned)a.num_pages;
  auto fetch = [&](unsigned p) {
#pragma unroll
    for (int q = 0; q < kScanPerThread; q += 4) {
      int4& v = held[q / 4];
      if (quads && p + q + 4 <= pages) {
        v = *reinterpret_cast<const int4*>(a.page_refs + p + q);
      } else {
        v.x = p + q < pages ? a.page_refs[p + q] : 1;
        v.y = p + q + 1 < pages ? a.page_refs[p + q + 1] : 1;
        v.z = p + q + 2 < pages ? a.page_refs[p + q + 2] : 1;
        v.w = p + q + 3 < pages ? a.page_refs[p + q + 3] : 1;
      }
    }
  };
  constexpr unsigned step = kPlanThreads * kScanPerThread;
  if (wanted > 0) fetch(tid * kScanPerThread);
  for (unsigned p0 = 0; p0 < pages && found < wanted; p0 += step) {
    const unsigned p = p0 + tid * kScanPerThread;
    unsigned freed = 0;
#pragma unroll
    for (int q = 0; q < kScanPerThread; q += 4) {
      const int4 v = held[q / 4];
      freed |= (unsigned)((v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3) << q;
    }
    if (p0 + step < pages) fetch(p + step);
    int total;
    int at = found + block_exclusive(__popc(freed), scan, total);
    while (freed != 0u && at < wanted) {
      a.list[at++] = (int)p + __ffs(freed) - 1;
      freed &= freed - 1;
    }
    found += total;
  }
  found = min(found, wanted);
  __syncthreads();
  for (int i = warp; i < a.n; i += kPlanThreads / 32) {
    const int want = need[i], o = offset[i];
    const int st = want < 0 ? kRefused : (want > 0 && (long long)o + want > found) ? kNoPage : kDone;
    if (lane == 0) a.status[i] = st;
    if (FORK) {
      const int page = st == kDone && want > 0 ? a.list[o] : -1;
      if (lane == 0) {
        a.plan[i] = st != kDone ? -2 : page;
        if (page >= 0) a.page_refs[page] = 1;
      }
    } else if (st == kDone) {
      const int r = a.rows[i], len = a.lengths[i];
      int32_t* row = a.page_table + (size_t)r * a.max_pages;
      const int last = (int)(((long long)len + kBlk - 1) / kBlk);
      int k = o;
      for (int t0 = max(0, a.seqused_k[r]) / kBlk; t0 < last; t0 += 32) {
        const bool take = t0 + lane < last && row[min(t0 + lane, last - 1)] < 0;
        const unsigned m = __ballot_sync(0xffffffffu, take);
        if (take) {
          const int page = a.list[k + __popc(m & ((1u << lane) - 1))];
          row[t0 + lane] = page;
          a.page_refs[page] = 1;
        }
        k += __popc(m);
      }
      __syncwarp();
      if (lane == 0) a.seqused_k[r] = len;
    }
  }
}

// -------------------------------------------------------------------- copies
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyChunk = kCopyThreads * kCopyUnroll * 16;  // bytes per block

// One block's chunk of a page, 16 bytes per thread and access, every load
// issued before the first store.
MSA_DEV void copy_chunk(const uint8_t* src, uint8_t* dst, long long bytes) {
  uint4 v[kCopyUnroll];
  const long long o = (long long)threadIdx.x * 16;
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i)
    if (o + i * kCopyThreads * 16ll < bytes)
      v[i] = __ldcs(reinterpret_cast<const uint4*>(src + o + i * kCopyThreads * 16ll));
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i)
    if (o + i * kCopyThreads * 16ll < bytes)
      *reinterpret_cast<uint4*>(dst + o + i * kCopyThreads * 16ll) = v[i];
}

// A granted fork: in block (.., num_pools, i), if there is one, the table row:
// the source's whole pages, each with one more holder, then the fresh page,
// then nothing; in the others the begun page, a chunk of a pool each.
__global__ void __launch_bounds__(kCopyThreads)
    cache_fork_kernel(const __grid_constant__ CachePools pools, int num_pools, long long page_bytes,
                      const __grid_constant__ CacheTableArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int i = blockIdx.z;
  const int page = a.plan[i];
  const int src = a.src_rows[i];
  if (page == -2) return;
  const int len = a.seqused_k[src], whole = len / kBlk;
  const int32_t* from = a.page_table + (size_t)src * a.max_pages;
  if ((int)blockIdx.y == num_pools) {
    const int dst = a.rows[i];
    int32_t* to = a.page_table + (size_t)dst * a.max_pages;
    for (int t = blockIdx.x * kCopyThreads + threadIdx.x; t < a.max_pages; t += gridDim.x * kCopyThreads) {
      int p = -1;
      if (t < whole) {
        p = from[t];
        if (p >= 0 && p < a.num_pages) atomicAdd(a.page_refs + p, 1);
        else p = -1;
      } else if (t == whole) {
        p = page;
      }
      to[t] = p;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.seqused_k[dst] = len;
    return;
  }
  if (page < 0) return;
  uint8_t* base = static_cast<uint8_t*>(pools.base[blockIdx.y]);
  const long long o = (long long)blockIdx.x * kCopyChunk;
  copy_chunk(base + (long long)from[whole] * page_bytes + o, base + (long long)page * page_bytes + o,
             min((long long)kCopyChunk, page_bytes - o));
}

// Pair i is left out when its pages are not both in the pool, when a later
// pair has its destination, or when its source is any other pair's
// destination: what remains reads no page that is written.
__global__ void __launch_bounds__(kCopyThreads)
    cache_copy_kernel(const __grid_constant__ CachePools pools, long long page_bytes, int num_pages,
                      const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int i = blockIdx.z;
  const int from = __ldg(src + i), to = __ldg(dst + i);
  if (from < 0 || from >= num_pages || to < 0 || to >= num_pages || from == to) return;
  bool out = false;
  for (int j = threadIdx.x; j < n; j += kCopyThreads) {
    const int d = __ldg(dst + j);
    out |= j != i && ((d == to && j > i) || d == from);
  }
  if (__syncthreads_or(out)) return;
  uint8_t* base = static_cast<uint8_t*>(pools.base[blockIdx.y]);
  const long long o = (long long)blockIdx.x * kCopyChunk;
  copy_chunk(base + (long long)from * page_bytes + o, base + (long long)to * page_bytes + o,
             min((long long)kCopyChunk, page_bytes - o));
}

dim3 copy_grid(int num_pools, long long page_bytes, int n) {
  return dim3((unsigned)((page_bytes + kCopyChunk - 1) / kCopyChunk), (unsigned)num_pools, (unsigned)n);
}

template <bool FORK>
cudaError_t launch_plan(const CacheTableArgs& a, cudaStream_t s) {
  const int bytes = (a.num_rows + 2 * a.n + 33) * (int)sizeof(int);
  const cudaError_t e = set_smem_limit((const void*)cache_plan_kernel<FORK>, bytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(cache_plan_kernel<FORK>, dim3(1), kPlanThreads, bytes, s, a);
}

}  // namespace

cudaError_t launch_cache_accept(const CachePools& p, const CacheAcceptArgs& a, cudaStream_t s) {
  const int columns = a.num_pools * a.hkv * (a.row_bytes / 16);
  return launch_dependent(cache_accept_kernel, dim3((columns + kAcceptThreads - 1) / kAcceptThreads, a.batch),
                          kAcceptThreads, 0, s, p, a);
}

cudaError_t launch_cache_free(const CacheTableArgs& a, cudaStream_t s) {
  return launch_dependent(cache_free_kernel, dim3(a.n), kFreeThreads, 0, s, a);
}

cudaError_t launch_cache_extend(const CacheTableArgs& a, cudaStream_t s) { return launch_plan<false>(a, s); }

cudaError_t launch_cache_fork(const CacheTableArgs& a, cudaStream_t s) { return launch_plan<true>(a, s); }

cudaError_t launch_cache_fork_copy(const CachePools& p, int num_pools, long long page_bytes, bool tables,
                                   const CacheTableArgs& a, cudaStream_t s) {
  return launch_dependent(cache_fork_kernel, copy_grid(num_pools + (tables ? 1 : 0), page_bytes, a.n), kCopyThreads, 0,
                          s, p, num_pools, page_bytes, a);
}

cudaError_t launch_cache_copy_pages(const CachePools& p, int num_pools, long long page_bytes,
                                    int num_pages, const int32_t* src, const int32_t* dst, int n,
                                    cudaStream_t s) {
  return launch_dependent(cache_copy_kernel, copy_grid(num_pools, page_bytes, n), kCopyThreads, 0, s, p, page_bytes,
                          num_pages, src, dst, n);
}

}  // namespace msa
