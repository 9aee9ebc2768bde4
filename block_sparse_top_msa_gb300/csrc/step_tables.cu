// A step's tables from the requests' lengths, and the path that samples take
// through a tree of drafts: both read and write small integers that a serving
// loop would else copy to the host and back.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace msa {
namespace {

// Inclusive sum over the warp.
template <class T>
MSA_DEV T warp_sum_upto(T v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Inclusive sum over a block of kPlanThreads; every thread has to come.
constexpr int kPlanThreads = 1024;
template <class T>
MSA_DEV T block_sum_upto(T v, T* s_warp, T& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T inc = warp_sum_upto(v, lane);
  __syncthreads();  // the sums before have been read
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  T w = s_warp[lane];
  w = warp_sum_upto(w, lane);
  all = __shfl_sync(0xffffffffu, w, 31);
  const T before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return inc + (warp > 0 ? before : T(0));
}

MSA_DEV unsigned page_hash(int page) { return (unsigned)page * 2654435761u; }

// What a step's requests are, by one block: lengths, running sums of their
// tokens, and the groups of those that begin with the same page. A table in
// shared memory (open addressing, at most half full) holds for each first page
// the lowest request that has it: all that ever stands in a place are requests
// with one page, so which one is there while others look does not matter, and
// the lowest one is what is left. The members of a group are put in their order
// by one warp, 32 requests at a time, for which all warps have counted what
// stands before each among its 32. Bound by the latency of its steps: 2048
// requests take 17 us (28 where the one warp counts too, 480 clocks for each 32
// requests), 16 take 7.
__global__ void __launch_bounds__(kPlanThreads)
    step_plan_kernel(const __grid_constant__ StepTablesArgs a) {
  extern __shared__ int dyn[];
  __shared__ long long s_sum[32];
  __shared__ int s_int[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int slots = a.hash_slots;
  int* hash = dyn;          // (slots), while the groups are looked for
  int* first = dyn + slots;  // (batch): first page of each request that may share, else -1
  int* start = dyn;                // (batch) each, after that: where a group's members go,
  int* least = dyn + a.batch;      // the whole blocks before any new token of it,
  int* group = dyn + 2 * a.batch;  // its members' count, then each request's group
  int32_t* leader = a.plan + a.batch;
  int32_t* group_of = a.plan + 2 * a.batch;  // at a leader, then at every request
  int32_t* limit = a.plan + 3 * a.batch;     // whole blocks before a request's new tokens
  grid_dependency_wait();
  grid_dependents_launch();
  for (int i = tid; i < slots; i += kPlanThreads) hash[i] = -1;
  long long carry = 0;
  int fit = 0;  // the last sum within total_q
  if (tid == 0) a.cu_q[0] = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int len = 0, n = 0, page = -1;
    if (b < a.batch) {
      const int r = __ldg(a.rows + b), want = __ldg(a.new_lens + b);
      if (r >= 0 && r < a.num_rows) {
        page = __ldg(a.page_table + (size_t)r * a.max_pages);
        len = max(0, __ldg(a.seqused_k + r));
        n = min(max(0, want), len);
        if (n == 0 || page >= a.num_pages) page = -1;
      }
    }
    long long all;
    const long long upto = carry + block_sum_upto<long long>(n, s_sum, all);
    carry += all;
    // Requests whose tokens do not all fit get none, and neither does any after
    // them, as sums only grow: cu stays at the last sum that fits.
    const bool fits = upto <= a.total_q;
    const int last = __reduce_max_sync(0xffffffffu, fits ? (int)upto : 0);
    __syncthreads();
    if (lane == 0) s_int[tid >> 5] = last;
    __syncthreads();
    const int top = __reduce_max_sync(0xffffffffu, s_int[lane]);
    if (top > fit) fit = top;
    if (b < a.batch) {
      a.cu_q[b + 1] = fits ? (int)upto : fit;
      a.seqused_out[b] = len;
      first[b] = fits && page >= 0 ? page : -1;
      limit[b] = (len - n) / kBlk;
    }
  }
  __syncthreads();
  for (int b = tid; b < a.batch; b += kPlanThreads) {
    const int page = first[b];
    if (page < 0) continue;
    for (unsigned s = page_hash(page);; ++s) {
      int* at = hash + (s & (slots - 1));
      const int old = atomicCAS(at, -1, b);
      if (old == -1) break;
      if (first[old] == page) {
        atomicMin(at, b);
        break;
      }
    }
  }
  __syncthreads();
  // Leaders, numbered in their order.
  int groups = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int l = b;
    if (b < a.batch && first[b] >= 0)
      for (unsigned s = page_hash(first[b]);; ++s) {
        l = hash[s & (slots - 1)];
        if (first[l] == first[b]) break;
      }
    const bool leads = b < a.batch && l == b;
    int all;
    const int upto = block_sum_upto<int>(leads, s_int, all);
    if (b < a.batch) leader[b] = l;
    if (leads) group_of[b] = groups + upto - 1;
    groups += all;
  }
  __syncthreads();  // the table is done with
  for (int g = tid; g < a.batch; g += kPlanThreads) group[g] = 0, least[g] = a.max_pages;
  __syncthreads();
  for (int b = tid; b < a.batch; b += kPlanThreads) {
    const int l = leader[b], g = group_of[l];
    atomicAdd(&group[g], 1);
    atomicMin(&least[g], limit[b]);
  }
  __syncthreads();
  int placed = 0;
  for (int g0 = 0; g0 <= a.batch; g0 += kPlanThreads) {
    const int g = g0 + tid;
    const int n = g < a.batch ? group[g] : 0;
    int all;
    const int upto = block_sum_upto<int>(n, s_int, all);
    if (g <= a.batch) a.cu_groups[g] = placed + upto - n;
    if (g < a.batch) {
      start[g] = placed + upto - n;
      a.group_blocks[g] = n > 1 ? least[g] : 0;
    }
    placed += all;
  }
  __syncthreads();
  // Of 32 requests each: its group, how many of them stand before it there, and
  // at the first of a group how many there are.
  static_assert(kMaxCacheRows <= 1 << 14, "a group's number has 14 bits");
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int g = -1;
    if (b < a.batch) {
      const int l = leader[b];
      g = group_of[l];
      if (l != b) group_of[b] = g;
    }
    const unsigned same = __match_any_sync(0xffffffffu, g);
    const int before = __popc(same & ((1u << lane) - 1u));
    if (b < a.batch) group[b] = g | before << 14 | (before == 0 ? __popc(same) : 0) << 19;
  }
  __syncthreads();
  if (tid >= 32) return;
  int x = lane < a.batch ? group[lane] : -1;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int b = b0 + lane, next = b + 32 < a.batch ? group[b + 32] : -1, g = x & 0x3fff;
    const int at = x >= 0 ? start[g] : 0;
    __syncwarp();
    if (x >= 0) {
      a.group_rows[at + ((x >> 14) & 31)] = b;
      if (x >> 19) start[g] = at + (x >> 19);
    }
    __syncwarp();
    x = next;
  }
}

// A block per request: its row of the page table, its tokens' places, and how
// many of its blocks are its leader's too. 2048 requests with 1024 places each:
// 8.8 us; they begin under the plan's end. Counters are unsigned, as counts go up
// to 2^31 - 1 and a step past the last one has to stay above it.
constexpr int kRowThreads = 256;
__global__ void __launch_bounds__(kRowThreads)
    step_rows_kernel(const __grid_constant__ StepTablesArgs a) {
  const int b = blockIdx.x, tid = threadIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  const int r = __ldg(a.rows + b);
  const bool real = r >= 0 && r < a.num_rows;
  const int len = __ldcg(a.seqused_out + b), t0 = __ldcg(a.cu_q + b), n = __ldcg(a.cu_q + b + 1) - t0;
  const int used = (int)min((long long)a.max_pages, ((long long)len + kBlk - 1) / kBlk);
  const int32_t* row = a.page_table + (size_t)(real ? r : 0) * a.max_pages;
  int32_t* out = a.table_out + (size_t)b * a.max_pages;
  const int lead = __ldcg(a.plan + a.batch + b), g = __ldcg(a.plan + 2 * a.batch + b);
  const int32_t* other = a.page_table + (size_t)(lead != b ? __ldg(a.rows + lead) : 0) * a.max_pages;
  const int most = lead != b ? __ldcg(a.group_blocks + g) : 0;
  // A leader's own holes end what the others may share with it: each of them
  // sees those too.
  unsigned differs = UINT_MAX;
  for (unsigned j = tid; j < (unsigned)a.max_pages; j += kRowThreads) {
    int page = j < (unsigned)used ? __ldg(row + j) : -1;
    if (page < 0 || page >= a.num_pages) page = -1;
    out[j] = page;
    if (j < (unsigned)most && differs == UINT_MAX && (page < 0 || page != __ldg(other + j))) differs = j;
  }
  if (differs < (unsigned)most) atomicMin(a.group_blocks + g, (int)differs);
  for (unsigned i = tid; i < (unsigned)n; i += kRowThreads) {
    const int pos = len - n + (int)i;
    int page = pos / kBlk < a.max_pages ? __ldg(row + pos / kBlk) : -1;
    if (page >= a.num_pages) page = -1;
    a.token_rows[t0 + i] = b;
    a.positions[t0 + i] = pos;
    a.slots[t0 + i] = page < 0 ? -1 : (long long)page * kBlk + pos % kBlk;
  }
  for (unsigned t = __ldcg(a.cu_q + a.batch) + b * kRowThreads + tid; t < (unsigned)a.total_q; t += gridDim.x * kRowThreads) {
    a.token_rows[t] = -1;
    a.positions[t] = -1;
    a.slots[t] = -1;
  }
}

// The accepted path of each request, a warp for each. Nodes follow their
// parents, so one pass over a request's nodes finds the path: of the nodes not
// passed yet, the lowest child of the path's last node that the sample there
// names. A lane holds a node; its parent is its highest ancestor below it. Bound by
// the latency of its loads: 7 us a call for 8 requests and for 256.
constexpr int kPathWarps = 4;
__global__ void __launch_bounds__(kPathWarps * 32)
    draft_path_kernel(const __grid_constant__ DraftPathArgs a) {
  const int b = blockIdx.x * kPathWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  if (b >= a.batch) return;
  const int t0 = max(0, __ldg(a.cu_q + b)), n = min(__ldg(a.cu_q + b + 1), a.total_q) - t0;
  int32_t* path = a.path + (size_t)b * a.max_path;
  int len = 0, at = 0, want = -1;
  if (n > 0) {
    want = __ldg(a.sampled + t0);
    if (lane == 0) path[0] = 0;
    len = 1;
  }
  const unsigned nodes = max(n, 0);
  for (unsigned c0 = 0; c0 < nodes && len < a.max_path; c0 += 32) {
    const int c = (int)(c0 + lane);
    int parent = -1, draft = 0;
    if (c0 + lane < nodes) {
      draft = __ldg(a.drafts + t0 + c);
      const uint32_t* row = a.mask + (size_t)(t0 + c) * a.mask_words;
      int w = min(c >> 5, a.mask_words - 1);
      uint32_t bits = __ldg(row + w) & ((c >> 5) == w ? (1u << (c & 31)) - 1u : ~0u);
      while (bits == 0u && w > 0) bits = __ldg(row + --w);
      if (bits != 0u) parent = w * 32 + 31 - __clz(bits);
    }
    while (len < a.max_path) {
      const unsigned m = __ballot_sync(0xffffffffu, parent == at && c > at && draft == want);
      if (m == 0u) break;
      at = (int)c0 + __ffs(m) - 1;
      want = __ldg(a.sampled + t0 + at);
      if (lane == 0) path[len] = at;
      ++len;
    }
  }
  for (unsigned i = len + lane; i < (unsigned)a.max_path; i += 32) path[i] = -1;
  if (lane == 0) {
    a.path_len[b] = len;
    a.next[b] = want;
  }
}

}  // namespace

cudaError_t launch_step_tables(const StepTablesArgs& args, cudaStream_t s) {
  StepTablesArgs a = args;
  a.hash_slots = 64;
  while (a.hash_slots < 2 * a.batch) a.hash_slots *= 2;
  const int smem = (int)sizeof(int) * (a.hash_slots + a.batch);  // three numbers a request at least
  cudaError_t e = set_smem_limit((const void*)step_plan_kernel, smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(step_plan_kernel, dim3(1), kPlanThreads, smem, s, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(step_rows_kernel, dim3(a.batch), kRowThreads, 0, s, a);
}

cudaError_t launch_draft_path(const DraftPathArgs& a, cudaStream_t s) {
  return launch_dependent(draft_path_kernel, dim3((a.batch + kPathWarps - 1) / kPathWarps), kPathWarps * 32, 0, s, a);
}

}  // namespace msa
