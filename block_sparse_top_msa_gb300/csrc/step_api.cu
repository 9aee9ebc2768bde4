// C ABI of the operators around the attention of a serving step: host-side
// validation and launches of the norm and rotation (rope.cu), of the cache's
// pages (cache.cu), of a step's tables and drafted paths (step_tables.cu) and
// of sampling (sample.cu).
#include <cmath>

#include "../../include/msa.h"
#include "internal.h"

using namespace msa;

namespace {

bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
msa_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_CUDA_ERROR; }

// A pointer to `tokens` tokens' values: of none of them it may be NULL.
bool token_data(const void* p, uintptr_t a, int tokens) { return aligned(p, a) || (p == nullptr && tokens == 0); }

// A token stride in elements: whole 16-byte groups, no overlap of tokens.
bool stride_ok(long long stride, int heads) { return stride % 8 == 0 && stride >= 128ll * heads; }

// The checks that the forms of the norm and rotation share.
msa_status_t check_rope(const void* q, long long q_stride, const void* k, long long k_stride, msa_dtype_t dtype,
                        const float* wq, const float* wk, float eps, const float* cos_sin, int max_position,
                        int rotary_dim, const int32_t* positions, int total_q, int hq, int hkv, int head_dim) {
  if (total_q < 0 || hq < 1 || hkv < 1) return MSA_INVALID_ARG;
  if (!token_data(q, 16, total_q) || !token_data(k, 16, total_q) || !aligned(wq, 16) || !aligned(wk, 16) ||
      !token_data(positions, 4, total_q))
    return MSA_INVALID_ARG;
  if (!(eps > 0.f) || !std::isfinite(eps)) return MSA_INVALID_ARG;
  if (head_dim != 128 || (dtype != MSA_BF16 && dtype != MSA_FP16)) return MSA_UNSUPPORTED;
  if (rotary_dim < 0 || rotary_dim > 128 || rotary_dim % 16 != 0) return MSA_UNSUPPORTED;
  if (max_position < 1 || (rotary_dim > 0 && !aligned(cos_sin, 16))) return MSA_INVALID_ARG;
  if (!stride_ok(q_stride, hq) || !stride_ok(k_stride, hkv)) return MSA_INVALID_ARG;
  if ((long long)total_q * ((long long)hq + 2ll * hkv) >= (1ll << 31)) return MSA_UNSUPPORTED;
  return MSA_OK;
}

msa_status_t check_pools(void* const* pools, int num_pools, long long bytes, int num_pages) {
  if (pools == nullptr || num_pools < 1 || num_pages < 1 || bytes < 16 || bytes % 16 != 0) return MSA_INVALID_ARG;
  for (int i = 0; i < num_pools; ++i)
    if (!aligned(pools[i], 16)) return MSA_INVALID_ARG;
  return MSA_OK;
}

// What two of the pools have in common, of kApart (nothing), kSame (two are one
// pool) and kOverlap (two share a part) the last that is found.
enum PoolsShare { kApart, kSame, kOverlap };
PoolsShare pools_share(void* const* pools, int num_pools, uint64_t pool_bytes) {
  auto gap = [&](int i, int j) { return (uint64_t)(static_cast<uint8_t*>(pools[i]) - static_cast<uint8_t*>(pools[j])); };
  int i = 1;  // ascending pools, as slices of one allocation are, need one comparison each
  while (i < num_pools && pools[i] > pools[i - 1] && gap(i, i - 1) >= pool_bytes) ++i;
  PoolsShare found = kApart;
  for (; i < num_pools; ++i)
    for (int j = 0; j < i; ++j) {
      if (pools[i] == pools[j]) found = found == kOverlap ? kOverlap : kSame;
      else if ((pools[i] > pools[j] ? gap(i, j) : gap(j, i)) < pool_bytes) found = kOverlap;
    }
  return found;
}

// Calls launch(pools, count) for the pools in groups of what one launch takes.
template <class F>
cudaError_t for_pools(void* const* pools, int num_pools, F launch) {
  for (int i = 0; i < num_pools; i += kMaxCachePools) {
    CachePools p{};
    const int n = num_pools - i < kMaxCachePools ? num_pools - i : kMaxCachePools;
    for (int j = 0; j < n; ++j) p.base[j] = pools[i + j];
    const cudaError_t e = launch(p, n);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

msa_status_t check_tables(const int32_t* page_table, int max_pages, int num_rows, const int32_t* seqused_k,
                          const int32_t* page_refs, int num_pages, int n) {
  if (max_pages < 1 || num_rows < 1 || num_pages < 1 || n < 0) return MSA_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(seqused_k, 4) || !aligned(page_refs, 4)) return MSA_INVALID_ARG;
  if (num_rows > kMaxCacheRows || n > kMaxCacheRows) return MSA_UNSUPPORTED;
  return MSA_OK;
}

// The workspace of fork and extend: the requests' plan, then the free list.
msa_status_t place_plan(CacheTableArgs* a, void* workspace, size_t bytes) {
  if (workspace == nullptr || bytes < msa_cache_workspace_size(a->n, a->num_pages)) return MSA_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return MSA_INVALID_ARG;
  a->plan = static_cast<int32_t*>(workspace);
  a->list = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + up256((size_t)a->n * 4));
  return MSA_OK;
}

}  // namespace

extern "C" {

msa_status_t msa_qk_norm_rope(const void* q, long long q_stride, const void* k, long long k_stride,
                              msa_dtype_t dtype, const float* q_weight, const float* k_weight,
                              float eps, const float* cos_sin, int max_position, int rotary_dim,
                              int interleaved, const int32_t* positions, int total_q,
                              int num_qo_heads, int num_kv_heads, int head_dim, void* q_out,
                              void* k_out, cudaStream_t stream) {
  const msa_status_t st = check_rope(q, q_stride, k, k_stride, dtype, q_weight, k_weight, eps, cos_sin, max_position,
                                     rotary_dim, positions, total_q, num_qo_heads, num_kv_heads, head_dim);
  if (st != MSA_OK) return st;
  if (!token_data(q_out, 16, total_q) || !token_data(k_out, 16, total_q)) return MSA_INVALID_ARG;
  RopeArgs a{};
  a.q = q, a.k = k, a.q_stride = q_stride, a.k_stride = k_stride;
  a.f16 = dtype == MSA_FP16;
  a.wq = q_weight, a.wk = k_weight, a.eps = eps;
  a.cos_sin = cos_sin, a.max_position = max_position, a.rotary = rotary_dim, a.interleaved = interleaved != 0;
  a.positions = positions;
  a.tokens = total_q, a.hq = num_qo_heads, a.hkv = num_kv_heads;
  a.q_out = q_out, a.k_out = k_out;
  return from_cuda(launch_rope(a, stream));
}

msa_status_t msa_qk_norm_rope_append(
    const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
    long long v_stride, msa_dtype_t dtype, const float* q_weight, const float* k_weight, float eps,
    const float* cos_sin, int max_position, int rotary_dim, int interleaved,
    const int32_t* positions, const int32_t* cu_seqlens_q, int batch, const int32_t* page_table,
    int max_pages, int num_pages, const int32_t* seqused_k, int total_q, int num_qo_heads,
    int num_kv_heads, int head_dim, void* q_out, void* k_pool, void* v_pool,
    msa_dtype_t kv_dtype, cudaStream_t stream) {
  const msa_status_t st = check_rope(q, q_stride, k, k_stride, dtype, q_weight, k_weight, eps, cos_sin, max_position,
                                     rotary_dim, positions, total_q, num_qo_heads, num_kv_heads, head_dim);
  if (st != MSA_OK) return st;
  if (!token_data(v, 16, total_q) || !stride_ok(v_stride, num_kv_heads) || !token_data(q_out, 16, total_q) ||
      !aligned(k_pool, 16) ||
      !aligned(v_pool, 16) || !aligned(cu_seqlens_q, 4) || !aligned(page_table, 4) || !aligned(seqused_k, 4))
    return MSA_INVALID_ARG;
  if (batch < 1 || max_pages < 1 || num_pages < 1) return MSA_INVALID_ARG;
  if (kv_dtype != dtype && !(dtype == MSA_BF16 && kv_dtype == MSA_FP8_E4M3)) return MSA_UNSUPPORTED;
  RopeArgs a{};
  a.q = q, a.k = k, a.v = v, a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.f16 = dtype == MSA_FP16;
  a.kv = kv_dtype == MSA_FP8_E4M3 ? 2 : 1;
  a.wq = q_weight, a.wk = k_weight, a.eps = eps;
  a.cos_sin = cos_sin, a.max_position = max_position, a.rotary = rotary_dim, a.interleaved = interleaved != 0;
  a.positions = positions;
  a.tokens = total_q, a.hq = num_qo_heads, a.hkv = num_kv_heads;
  a.q_out = q_out;
  a.cu_q = cu_seqlens_q, a.batch = batch, a.page_table = page_table, a.max_pages = max_pages;
  a.num_pages = num_pages, a.seqused_k = seqused_k, a.k_pool = k_pool, a.v_pool = v_pool;
  return from_cuda(launch_rope(a, stream));
}

size_t msa_qk_norm_rope_bwd_workspace_size(int total_q, int num_qo_heads, int num_kv_heads) {
  if (total_q < 0 || num_qo_heads < 1 || num_kv_heads < 1) return 0;
  const RopeBwdGrid g = rope_bwd_grid(total_q, num_qo_heads, num_kv_heads);
  return up256(((size_t)g.q_blocks + g.k_blocks) * 128 * sizeof(float)) + 256;
}

msa_status_t msa_qk_norm_rope_bwd(
    const void* dq_out, const void* dk_out, const void* q, long long q_stride, const void* k,
    long long k_stride, msa_dtype_t dtype, const float* q_weight, const float* k_weight, float eps,
    const float* cos_sin, int max_position, int rotary_dim, int interleaved,
    const int32_t* positions, int total_q, int num_qo_heads, int num_kv_heads, int head_dim,
    void* dq, long long dq_stride, void* dk, long long dk_stride, float* dq_weight,
    float* dk_weight, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const msa_status_t st = check_rope(q, q_stride, k, k_stride, dtype, q_weight, k_weight, eps, cos_sin, max_position,
                                     rotary_dim, positions, total_q, num_qo_heads, num_kv_heads, head_dim);
  if (st != MSA_OK) return st;
  if (!token_data(dq_out, 16, total_q) || !token_data(dk_out, 16, total_q) || !token_data(dq, 16, total_q) ||
      !token_data(dk, 16, total_q) ||
      !aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !stride_ok(dq_stride, num_qo_heads) ||
      !stride_ok(dk_stride, num_kv_heads))
    return MSA_INVALID_ARG;
  if (workspace == nullptr ||
      workspace_bytes < msa_qk_norm_rope_bwd_workspace_size(total_q, num_qo_heads, num_kv_heads))
    return MSA_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return MSA_INVALID_ARG;
  const RopeBwdGrid g = rope_bwd_grid(total_q, num_qo_heads, num_kv_heads);
  RopeBwdArgs a{};
  a.dq_out = dq_out, a.dk_out = dk_out, a.q = q, a.k = k, a.q_stride = q_stride, a.k_stride = k_stride;
  a.f16 = dtype == MSA_FP16;
  a.wq = q_weight, a.wk = k_weight, a.eps = eps;
  a.cos_sin = cos_sin, a.max_position = max_position, a.rotary = rotary_dim, a.interleaved = interleaved != 0;
  a.positions = positions;
  a.tokens = total_q, a.hq = num_qo_heads, a.hkv = num_kv_heads;
  a.dq = dq, a.dk = dk, a.dq_stride = dq_stride, a.dk_stride = dk_stride;
  a.dwq = dq_weight, a.dwk = dk_weight;
  a.partials = static_cast<float*>(workspace);
  a.q_blocks = g.q_blocks;
  return from_cuda(launch_rope_bwd(a, g.k_blocks, stream));
}

size_t msa_cache_workspace_size(int n, int num_pages) {
  if (n < 0 || num_pages < 1) return 0;
  return up256((size_t)n * 4) + up256((size_t)num_pages * 4);
}

msa_status_t msa_cache_extend(int32_t* page_table, int max_pages, int num_rows, int32_t* seqused_k,
                              int32_t* page_refs, int num_pages, const int32_t* rows,
                              const int32_t* lengths, int n, int32_t* status, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  msa_status_t st = check_tables(page_table, max_pages, num_rows, seqused_k, page_refs, num_pages, n);
  if (st != MSA_OK) return st;
  if (n == 0) return MSA_OK;
  if (!aligned(rows, 4) || !aligned(lengths, 4) || !aligned(status, 4)) return MSA_INVALID_ARG;
  CacheTableArgs a{};
  a.page_table = page_table, a.max_pages = max_pages, a.num_rows = num_rows, a.num_pages = num_pages;
  a.seqused_k = seqused_k, a.page_refs = page_refs, a.rows = rows, a.lengths = lengths, a.n = n, a.status = status;
  st = place_plan(&a, workspace, workspace_bytes);
  if (st != MSA_OK) return st;
  if (status == rows || status == lengths) return MSA_INVALID_ARG;  // written while others are read
  return from_cuda(launch_cache_extend(a, stream));
}

msa_status_t msa_cache_fork(void* const* pools, int num_pools, long long page_bytes,
                            int32_t* page_table, int max_pages, int num_rows, int32_t* seqused_k,
                            int32_t* page_refs, int num_pages, const int32_t* src_rows,
                            const int32_t* dst_rows, int n, int32_t* status, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  msa_status_t st = check_pools(pools, num_pools, page_bytes, num_pages);
  if (st != MSA_OK) return st;
  st = check_tables(page_table, max_pages, num_rows, seqused_k, page_refs, num_pages, n);
  if (st != MSA_OK) return st;
  if (n == 0) return MSA_OK;
  if (!aligned(src_rows, 4) || !aligned(dst_rows, 4) || !aligned(status, 4)) return MSA_INVALID_ARG;
  CacheTableArgs a{};
  a.page_table = page_table, a.max_pages = max_pages, a.num_rows = num_rows, a.num_pages = num_pages;
  a.seqused_k = seqused_k, a.page_refs = page_refs, a.rows = dst_rows, a.src_rows = src_rows, a.n = n;
  a.status = status;
  st = place_plan(&a, workspace, workspace_bytes);
  if (st != MSA_OK) return st;
  if (status == src_rows || status == dst_rows) return MSA_INVALID_ARG;  // written while others are read
  if (pools_share(pools, num_pools, (uint64_t)page_bytes * num_pages) == kOverlap) return MSA_INVALID_ARG;
  cudaError_t e = launch_cache_fork(a, stream);
  bool tables = true;
  if (e == cudaSuccess)
    e = for_pools(pools, num_pools, [&](const CachePools& p, int count) {
      const cudaError_t r = launch_cache_fork_copy(p, count, page_bytes, tables, a, stream);
      tables = false;
      return r;
    });
  return from_cuda(e);
}

msa_status_t msa_cache_free(int32_t* page_table, int max_pages, int num_rows, int32_t* seqused_k,
                            int32_t* page_refs, int num_pages, const int32_t* rows, int n,
                            cudaStream_t stream) {
  const msa_status_t st = check_tables(page_table, max_pages, num_rows, seqused_k, page_refs, num_pages, n);
  if (st != MSA_OK) return st;
  if (n == 0) return MSA_OK;
  if (!aligned(rows, 4)) return MSA_INVALID_ARG;
  CacheTableArgs a{};
  a.page_table = page_table, a.max_pages = max_pages, a.num_rows = num_rows, a.num_pages = num_pages;
  a.seqused_k = seqused_k, a.page_refs = page_refs, a.rows = rows, a.n = n;
  return from_cuda(launch_cache_free(a, stream));
}

msa_status_t msa_cache_copy_pages(void* const* pools, int num_pools, long long page_bytes,
                                  int num_pages, const int32_t* src_pages,
                                  const int32_t* dst_pages, int n, cudaStream_t stream) {
  const msa_status_t st = check_pools(pools, num_pools, page_bytes, num_pages);
  if (st != MSA_OK) return st;
  if (n < 0) return MSA_INVALID_ARG;
  if (n > kMaxCopyPairs) return MSA_UNSUPPORTED;
  if (n == 0) return MSA_OK;
  if (!aligned(src_pages, 4) || !aligned(dst_pages, 4)) return MSA_INVALID_ARG;
  if (pools_share(pools, num_pools, (uint64_t)page_bytes * num_pages) == kOverlap) return MSA_INVALID_ARG;
  return from_cuda(for_pools(pools, num_pools, [&](const CachePools& p, int count) {
    return launch_cache_copy_pages(p, count, page_bytes, num_pages, src_pages, dst_pages, n, stream);
  }));
}

msa_status_t msa_cache_accept(void* const* pools, int num_pools, int row_bytes, int num_kv_heads,
                              const int32_t* page_table, int max_pages, int num_pages, int batch,
                              const int32_t* seqused_k, const int32_t* cu_seqlens_q,
                              const int32_t* path, const int32_t* path_len, int max_path,
                              int32_t* seqused_out, cudaStream_t stream) {
  const msa_status_t st = check_pools(pools, num_pools, row_bytes, num_pages);
  if (st != MSA_OK) return st;
  if (num_kv_heads < 1 || max_pages < 1 || batch < 1 || max_path < 1) return MSA_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(seqused_k, 4) || !aligned(cu_seqlens_q, 4) || !aligned(path, 4) ||
      !aligned(path_len, 4) || !aligned(seqused_out, 4) || seqused_out == seqused_k || seqused_out == path_len)
    return MSA_INVALID_ARG;
  if (batch > kMaxCacheRows || num_kv_heads > 1024 || row_bytes > 4096) return MSA_UNSUPPORTED;
  // A pool's rows move once: a pool given twice would read moved rows.
  if (pools_share(pools, num_pools, (uint64_t)row_bytes * num_kv_heads * 128 * num_pages) != kApart)
    return MSA_INVALID_ARG;
  CacheAcceptArgs a{};
  a.row_bytes = row_bytes, a.hkv = num_kv_heads;
  a.page_table = page_table, a.max_pages = max_pages, a.num_pages = num_pages, a.batch = batch;
  a.seqused_k = seqused_k, a.cu_q = cu_seqlens_q, a.path = path, a.path_len = path_len, a.max_path = max_path;
  a.seqused_out = seqused_out;
  return from_cuda(for_pools(pools, num_pools, [&](const CachePools& p, int count) {
    a.num_pools = count;
    return launch_cache_accept(p, a, stream);
  }));
}

size_t msa_step_tables_workspace_size(int batch) {
  if (batch < 1 || batch > kMaxCacheRows) return 0;
  return up256(4 * (size_t)batch * sizeof(int32_t));
}

msa_status_t msa_step_tables(const int32_t* page_table, int max_pages, int num_rows,
                             const int32_t* seqused_k, int num_pages, const int32_t* rows,
                             const int32_t* new_lens, int batch, int total_q,
                             int32_t* cu_seqlens_q, int32_t* seqused_out, int32_t* table_out,
                             int32_t* token_rows, int32_t* positions, long long* slots,
                             int32_t* group_rows, int32_t* cu_groups, int32_t* group_blocks,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (max_pages < 1 || num_rows < 1 || num_pages < 1 || batch < 1 || total_q < 0) return MSA_INVALID_ARG;
  for (const void* p : {(const void*)page_table, (const void*)seqused_k, (const void*)rows, (const void*)new_lens,
                        (const void*)cu_seqlens_q, (const void*)seqused_out, (const void*)table_out,
                        (const void*)group_rows, (const void*)cu_groups, (const void*)group_blocks})
    if (!aligned(p, 4)) return MSA_INVALID_ARG;
  if (!token_data(token_rows, 4, total_q) || !token_data(positions, 4, total_q) || !token_data(slots, 8, total_q))
    return MSA_INVALID_ARG;
  if (batch > kMaxCacheRows) return MSA_UNSUPPORTED;
  const size_t b = batch, t = total_q, width = max_pages;
  if (spans_clash({{cu_seqlens_q, 4 * (b + 1)}, {seqused_out, 4 * b}, {table_out, 4 * b * width}, {token_rows, 4 * t}, {positions, 4 * t}, {slots, 8 * t},
                   {group_rows, 4 * b}, {cu_groups, 4 * (b + 1)}, {group_blocks, 4 * b}, {workspace, msa_step_tables_workspace_size(batch)}},
                  {{page_table, 4 * (size_t)num_rows * width}, {seqused_k, 4 * (size_t)num_rows}, {rows, 4 * b}, {new_lens, 4 * b}}))
    return MSA_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < msa_step_tables_workspace_size(batch)) return MSA_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return MSA_INVALID_ARG;
  StepTablesArgs a{};
  a.page_table = page_table, a.max_pages = max_pages, a.num_rows = num_rows, a.num_pages = num_pages;
  a.seqused_k = seqused_k, a.rows = rows, a.new_lens = new_lens, a.batch = batch, a.total_q = total_q;
  a.cu_q = cu_seqlens_q, a.seqused_out = seqused_out, a.table_out = table_out;
  a.token_rows = token_rows, a.positions = positions, a.slots = slots;
  a.group_rows = group_rows, a.cu_groups = cu_groups, a.group_blocks = group_blocks;
  a.plan = static_cast<int32_t*>(workspace);
  return from_cuda(launch_step_tables(a, stream));
}

size_t msa_sample_workspace_size(int rows, int vocab, msa_dtype_t dtype) {
  if (rows < 0 || vocab < 1 || rows > (1 << 24) || vocab > kMaxVocab) return 0;
  if (dtype != MSA_BF16 && dtype != MSA_FP16 && dtype != MSA_FP32) return 0;
  const SampleSlices c = sample_slices(rows, vocab, dtype == MSA_FP32, false);
  const size_t n = (size_t)rows * c.slices;
  if (rows == 0) return 0;
  if (c.slices == 0) return 256;  // 16-bit logits need none
  return up256(n * 8) + up256((size_t)rows * kSampleParts * 4) + up256((size_t)rows * kSampleParts * 8) +
         up256(n * c.slice * 2) + up256(n * kSampleStarts * 2);
}

msa_status_t msa_sample(const void* logits, msa_dtype_t dtype, long long stride, int rows,
                        int vocab, const float* uniforms, const float* temperature,
                        const int32_t* top_k, const float* top_p, const float* min_p,
                        int32_t* tokens, float* logprobs, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  if (rows < 0 || vocab < 1 || stride < vocab) return MSA_INVALID_ARG;
  if (dtype != MSA_BF16 && dtype != MSA_FP16 && dtype != MSA_FP32) return MSA_UNSUPPORTED;
  if (!token_data(logits, dtype == MSA_FP32 ? 4 : 2, rows) || !token_data(uniforms, 4, rows) ||
      !token_data(tokens, 4, rows))
    return MSA_INVALID_ARG;
  for (const void* p : {(const void*)temperature, (const void*)top_k, (const void*)top_p, (const void*)min_p,
                        (const void*)logprobs})
    if (p != nullptr && !aligned(p, 4)) return MSA_INVALID_ARG;
  if (vocab > kMaxVocab || rows > (1 << 24)) return MSA_UNSUPPORTED;
  const size_t size = dtype == MSA_FP32 ? 4 : 2, r4 = 4 * (size_t)rows;
  if (spans_clash({{tokens, r4}, {logprobs, r4}, {workspace, msa_sample_workspace_size(rows, vocab, dtype)}},
                  {{logits, size * vocab, (size_t)rows, size * (size_t)stride}, {uniforms, r4}, {temperature, r4}, {top_k, r4}, {top_p, r4}, {min_p, r4}}))
    return MSA_INVALID_ARG;
  if (rows == 0) return MSA_OK;
  if (workspace == nullptr || workspace_bytes < msa_sample_workspace_size(rows, vocab, dtype)) return MSA_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return MSA_INVALID_ARG;
  const bool row_aligned = aligned(logits, 16) && (rows == 1 || stride % 4 == 0);
  const SampleSlices c = sample_slices(rows, vocab, dtype == MSA_FP32, row_aligned);
  SampleArgs a{};
  a.logits = logits, a.stride = stride, a.type = dtype == MSA_BF16 ? 0 : dtype == MSA_FP16 ? 1 : 2;
  a.rows = rows, a.vocab = vocab;
  a.uniforms = uniforms, a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p;
  a.tokens = tokens, a.logprobs = logprobs;
  a.slice = c.slice, a.slices = c.slices;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  auto place = [&](size_t bytes) {
    uint8_t* at = w;
    w += up256(bytes);
    return at;
  };
  const size_t n = (size_t)rows * c.slices;
  a.best = reinterpret_cast<unsigned long long*>(place(n * 8));
  a.parts_count = reinterpret_cast<uint32_t*>(place((size_t)rows * kSampleParts * 4));
  a.parts_mass = reinterpret_cast<unsigned long long*>(place((size_t)rows * kSampleParts * 8));
  a.order = reinterpret_cast<uint16_t*>(place(n * c.slice * 2));
  a.starts = reinterpret_cast<uint16_t*>(place(n * kSampleStarts * 2));
  return from_cuda(launch_sample(a, stream));
}

msa_status_t msa_draft_path(const int32_t* sampled, const int32_t* drafts,
                            const uint32_t* tree_mask, int mask_words,
                            const int32_t* cu_seqlens_q, int batch, int total_q, int max_path,
                            int32_t* path, int32_t* path_len, int32_t* next_tokens,
                            cudaStream_t stream) {
  if (mask_words < 1 || batch < 1 || total_q < 0 || max_path < 1) return MSA_INVALID_ARG;
  if (!token_data(sampled, 4, total_q) || !token_data(drafts, 4, total_q) || !token_data(tree_mask, 4, total_q) ||
      !aligned(cu_seqlens_q, 4) || !aligned(path, 4) || !aligned(path_len, 4) || !aligned(next_tokens, 4))
    return MSA_INVALID_ARG;
  const size_t b = batch, t = total_q;
  if (spans_clash({{path, 4 * b * max_path}, {path_len, 4 * b}, {next_tokens, 4 * b}},
                  {{sampled, 4 * t}, {drafts, 4 * t}, {tree_mask, 4 * t * mask_words}, {cu_seqlens_q, 4 * (b + 1)}}))
    return MSA_INVALID_ARG;
  DraftPathArgs a{};
  a.sampled = sampled, a.drafts = drafts, a.mask = tree_mask, a.mask_words = mask_words;
  a.cu_q = cu_seqlens_q, a.batch = batch, a.total_q = total_q, a.max_path = max_path;
  a.path = path, a.path_len = path_len, a.next = next_tokens;
  return from_cuda(launch_draft_path(a, stream));
}

}  // extern "C"
