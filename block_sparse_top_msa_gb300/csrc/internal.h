// Internal launch interface between the C-ABI layer (api.cu) and the kernels.
// Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace msa {

// Memory that an argument of a call covers: `rows` rows of `bytes`, `pitch` bytes
// from one to the next. NULL is none.
struct Span {
  const void* at;
  size_t bytes;
  size_t rows = 1, pitch = 0;
};
// Whether two of them meet, the first of which is one row.
inline bool spans_meet(const Span& a, const Span& b) {
  if (a.at == nullptr || b.at == nullptr) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.at), b0 = reinterpret_cast<uintptr_t>(b.at);
  const uintptr_t a1 = a0 + (a.bytes > 0 ? a.bytes : 1), row = b.bytes > 0 ? b.bytes : 1;
  if (b.rows <= 1 || b.pitch == 0) return a0 < b0 + row && b0 < a1;
  const uintptr_t first = a0 < b0 + row ? 0 : (a0 - b0 - row) / b.pitch + 1;  // row that ends behind a0
  return first < b.rows && b0 + first * b.pitch < a1;
}
// Whether what a call writes meets what it reads, or is given twice.
inline bool spans_clash(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (const Span* w = written.begin(); w != written.end(); ++w) {
    for (const Span& r : read)
      if (spans_meet(*w, r)) return true;
    for (const Span* o = written.begin(); o != w; ++o)
      if (spans_meet(*w, *o)) return true;
  }
  return false;
}

// Device address of the library's fault word on the current device (host).
unsigned* fault_word();

struct UnionArgs {
  const int32_t* q2k;
  int topk;
  const int32_t* cu_q;
  const int32_t* cu_k;       // flat lengths, or NULL
  const int32_t* seqused_k;  // paged lengths, or NULL
  int max_pages;
  int batch;
  int total_q;
  int num_kv_heads;
  int causal;
  int tile_tokens;  // W
  int max_tiles;
  int cap;          // W * topk
  int words;        // ceil(cap / 32)
  int32_t* union_len;
  int32_t* union_blocks;
  uint32_t* member;
  int32_t* tile_info;  // may be NULL
  int32_t* item_counter;  // may be NULL: set to 0 (the attention kernel's work counter)
  // May be NULL (only for tile_tokens <= 32): per union position, a mask of
  // the tile's tokens that selected it (bit w = token w of the tile), i.e.
  // the membership bits transposed; (num_kv_heads, max_tiles, cap) uint32.
  uint32_t* block_members;
};
cudaError_t launch_build_union(const UnionArgs& a, cudaStream_t s);
// Zeroes the attention kernel's work counter in a one-thread kernel that
// lets its programmatic dependent start at once.
cudaError_t launch_reset_counter(int32_t* counter, cudaStream_t s);

struct TopkArgs {
  const float* scores;
  int num_score_heads;
  int max_k_tiles;
  int total_q;
  int topk;
  int num_kv_heads_out;
  int32_t* q2k;
};
cudaError_t launch_topk(const TopkArgs& a, cudaStream_t s);


struct PrefillArgs {
  unsigned* fault;      // device fault word (bounded-wait expiry, capacity)
  CUtensorMap tmap_q;   // (d, Hq, Tq) bf16, box (64, G, W)
  CUtensorMap tmap_k;   // flat (d or d bytes, Hkv, Tk) / paged (.., 128, Hkv, pages)
  CUtensorMap tmap_v;
  int paged;
  int kv_fp8;           // E4M3 K/V, or packed NVFP4 K/V (kv_fp4), converted in the kernel
  int f16;              // q, k, v and out are fp16 (else bf16; E4M3 K/V only with bf16)
  // Packed NVFP4 paged K/V: per page (fp4_page_stride bytes apart) and KV
  // head, 128 x 64 bytes of E2M1 pairs and 128 x 8 E4M3 block scales for K
  // (scales token-major) and for V (scales in 4 x 4 tiles, scale-index major).
  int kv_fp4;
  const uint8_t* fp4_k;
  const uint8_t* fp4_k_scale;
  const uint8_t* fp4_v;
  const uint8_t* fp4_v_scale;
  long long fp4_page_stride;
  float out_scale;      // multiplies every output (the NVFP4 V global scale; else 1)
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* page_table;
  int max_pages;
  int num_pages;
  const int32_t* seqused_k;
  int batch;
  int total_q;
  int num_qo_heads;
  int num_kv_heads;
  int causal;
  float scale_log2;
  int tile_tokens;
  int max_tiles;
  int cap;
  int words;
  // Union metadata (written by the union kernel, or in direct mode by this
  // kernel's item setup).
  int32_t* union_len;
  int32_t* union_blocks;
  const uint32_t* member;
  int32_t* tile_info;
  void* out;
  float* lse;
  // Work items, handed out dynamically to a persistent grid. Units are (query tile, KV head)
  // pairs, head-major with the heaviest tiles first within a head. The first whole_units units are one item each and
  // write out/lse directly. Each remaining ("tail") unit is split into
  // `splits` items, item s taking union entries [s*pps, (s+1)*pps); a tail
  // unit whose union needs more than one split writes fp32 partials
  // (rows_part rows per item), combined by a second kernel.
  // Splitting only the tail evens out the last round of work across the SMs.
  int whole_units;
  int tail_units;
  int splits;
  int pps;
  int rows_part;
  int num_items;
  float* part_o;        // (tail_units*splits, rows_part, 128)
  float* part_ml;       // (tail_units*splits, rows_part, 2)
  int* item_counter;    // items handed out beyond the first round; 0 at launch
  // Swapped-orientation prefill kernel only: per union position, the mask of
  // the tile's tokens that selected it (bit w = token w), and a q map whose
  // box is one token's G query heads, (64, G, 1).
  const uint32_t* block_members;
  CUtensorMap tmap_q1;
  // One-token tiles (tile_tokens == 1, topk <= 32) may skip the union
  // kernel: with `direct` set, the attention kernel's item setup filters,
  // sorts and deduplicates the token's own q2k row (every union entry is
  // then a member) and writes union_len, union_blocks and tile_info itself.
  const int32_t* q2k;
  int topk;
  int direct;
  // The preceding kernel only zeroes item_counter (launch_reset_counter, an
  // ordinary launch, so every other input was complete before it began): the
  // attention kernel waits for it only before its first claim from the
  // counter.
  int wait_late;
};
cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t s);
// The swapped-orientation prefill kernel (bf16 / fp16 K/V, G a multiple of 8
// and at most 64, tile_tokens * G <= 256, tile_tokens <= 32, no splits).
cudaError_t launch_prefill_swapped(const PrefillArgs& a, cudaStream_t s);
int device_sm_count();
// Raises `kernel`'s dynamic shared-memory limit to at least `bytes` on the
// current device; the driver call is made once per (kernel, device, size).
cudaError_t set_smem_limit(const void* kernel, int bytes);
// The current device's per-block shared-memory limit (opt-in), cached.
int device_smem_optin();

// Attention of drafted trees (tree.cu).
struct TreeArgs {
  unsigned* fault;
  CUtensorMap tmap_q;  // (d, Hq, Tq) 16-bit, box (64, G, tile_tokens)
  CUtensorMap tmap_k;  // (.., 128, Hkv, pages), 16-bit caches
  CUtensorMap tmap_v;
  const void* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  int e4m3, f16;       // the cache's type, else bf16
  const int32_t* cu_q;
  const int32_t* page_table;
  int max_pages, num_pages;
  const int32_t* seqused_k;
  int num_qo_heads, num_kv_heads;
  float scale_log2;
  const uint32_t* tree_mask;  // (Tq, mask_words)
  int mask_words;
  int tile_tokens, unit_tokens;  // per MMA tile; per unit, at most two tiles
  int max_tiles;                 // bound on the groups of unit_tokens tokens
  const int32_t* q2k;            // (Hkv, Tq, topk)
  int topk, total_q, batch;
  int cap, words;                // unit_tokens * topk, and its bits in words
  // Per unit (tile * Hkv + h), written by the union kernel: weighted union
  // length; (t0, sequence, tokens, union length), t0 = -1 past the last tile,
  // and (Lq, Lk, 0, 0); the union (cap); each token's membership (words).
  int32_t* unit_len;
  int4* unit_info;
  int32_t* union_blocks;
  uint32_t* member;
  int min_range;    // least weighted length of a CTA's range, at least a block's
  int cut_cost;     // what ranges cut out of units cost, in weighted blocks of a CTA's time
  int grid, rows_part;
  float* part_o;    // (2 * grid, 128, rows_part): unnormalised O of a range's first and last segment
  float* part_m;    // (2 * grid, rows_part)
  float* part_l;
  int2* cut;        // (grid): the unit that begins in the CTA's range and goes on after it, and the
                    // one that began before it (of the CTA's first segment); -1: none
  int32_t* odd;     // (1 + Tq * Hq): how many rows were not finite, and which
  void* out;
  float* lse;
};
cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s);

// Attention over shared prefixes (prefix.cu, prefix_big.cu, prefix_work.cuh). A
// call's units are all of few rows (prefix.cu's kernel) or all of many
// (prefix_big.cu). Costs of a unit besides its blocks, and the least cost of a
// CTA's range, at least a unit's with one block.
constexpr int kSmallRows = 16, kBigRows = 256;
constexpr int kSmallUnitCost = 5, kBigUnitCost = 12, kSmallRange = 7, kBigRange = 16;
constexpr int kGroupRun = 1 << 30;  // of an entry's first block: the entry is a group's
struct PrefixArgs {
  unsigned* fault = nullptr;
  CUtensorMap tmap_k;  // (.., 128, Hkv, pages)
  CUtensorMap tmap_v;
  const void* q = nullptr;
  const uint8_t* k_pool = nullptr;
  const uint8_t* v_pool = nullptr;
  int e4m3 = 0, f16 = 0;  // the cache's type, else bf16
  const int32_t* cu_q = nullptr;
  const int32_t* page_table = nullptr;
  int max_pages = 0, num_pages = 0;
  const int32_t* seqused_k = nullptr;
  const int32_t* group_rows = nullptr;  // NULL: each request by itself
  const int32_t* cu_groups = nullptr;
  const int32_t* group_blocks = nullptr;
  int batch = 0, total_q = 0, num_qo_heads = 0, num_kv_heads = 0, causal = 0;
  float scale_log2 = 0.f;
  void* out = nullptr;
  float* lse = nullptr;
  int small = 0;  // units of kSmallRows rows (no groups then), else of kBigRows
  int grid = 0;   // CTAs
  int chunk_rows = 0;  // of the join's chunks: 4 to 64, a power of two
  // Workspace. Positions: the requests in the order of the groups. Entries: the
  // positions' own runs, then the groups', those that there are.
  int4* entry = nullptr;       // (batch, 2): first token in that order, tokens, request, group; first row of q, Lk - Lq, Lk, entry or -1
  int* group = nullptr;        // (batch): a group's entry or -1
  int4* work = nullptr;        // (2 batch, 2): first token, rows, page row, first block (| kGroupRun); blocks, keys that all rows see, Lk, group before or -1
  long long* start = nullptr;  // (2 batch + 1): running sums of the entries' costs
  int* chunk = nullptr;        // (2 batch + 1): running count of what the join does for entries with a group before: chunk_rows rows of one KV head each
  int2* token = nullptr;       // (total_q): each token's row of q, and its position
  int* meta = nullptr;         // entries
  int4* cut = nullptr;         // (grid): the unit without a group before that begins in the CTA's range and goes on after it: entry, tile and head; entry -1: none
  int at_cta = 0;              // units' first pieces leave their parts at the CTA's too, not at the rows' own places
  size_t part_rows = 0;        // rows of parts before those of the CTAs' later pieces
  float2* part_ml = nullptr;   // (part_rows + grid * kBigRows)
  float* part_o = nullptr;     // the same, 128 each
};
cudaError_t launch_prefix(const PrefixArgs& a, cudaStream_t s);
cudaError_t launch_prefix_big(const PrefixArgs& a, cudaStream_t s);  // the units, where they are of many rows

struct ProxyArgs {
  unsigned* fault;      // device fault word (bounded-wait expiry, capacity)
  CUtensorMap tmap_q;   // (d, Hq, Tq) 16-bit, box (64, G, Wm)
  CUtensorMap tmap_k;   // flat (d, Hkv, Tk) / paged (d, 128, Hkv, pages), 128-key box of
                        // 128 bytes (64 16-bit values, or 128 E4M3 codes)
  const int32_t* cu_q;
  const int32_t* cu_k;        // flat lengths, or NULL when paged
  int paged;
  const int32_t* page_table;  // (B, max_pages), paged only
  int max_pages;
  int num_pages;
  const int32_t* seqused_k;   // (B), paged only
  int batch;
  int total_q;
  int num_qo_heads;
  int num_kv_heads;
  int max_k_tiles;
  int causal;
  int reduce_heads;
  int tile_tokens;      // tokens per M-tile (128 / G)
  int max_tiles;        // upper bound on query tiles of 2 M-tiles each
  int one_m;            // query tiles of tile_tokens tokens (one M tile), else 2 * tile_tokens
  int slice_cols;       // block columns per CTA: CTA (tile, s) takes [s, s + 1) * slice_cols
  int slices;           // column slices per tile
  float* out;
  int f16;              // q (and 16-bit K) are fp16, else bf16
  int k_fp8;            // K is E4M3, upconverted in the kernel to q's type
};
cudaError_t launch_proxy(const ProxyArgs& a, cudaStream_t s);

// Flat E4M3 K and V (n16 16-byte groups each) decoded to bf16 copies.
struct KvDecodeArgs {
  const void* k8 = nullptr;
  const void* v8 = nullptr;
  void* k16 = nullptr;
  void* v16 = nullptr;
  size_t n16 = 0;
};
cudaError_t launch_kv_decode(const KvDecodeArgs& a, cudaStream_t s);

// Paged E4M3 (mode 1: (pages, Hkv, 128, 128) bytes) or packed NVFP4 (mode 2:
// planar pages) K/V decoded into a bf16 pool of batch * max_pages pages, with
// the renumbered page table written to pt_out (batch, max_pages).
struct PageDecodeArgs {
  int mode = 0;  // 0: nothing to do
  const int32_t* page_table = nullptr;
  const int32_t* seqused_k = nullptr;
  int max_pages = 0, num_pages = 0, batch = 0, hkv = 0;
  const uint8_t* k8 = nullptr;
  const uint8_t* v8 = nullptr;
  const uint8_t* fp4_k = nullptr;
  const uint8_t* fp4_k_scale = nullptr;
  const uint8_t* fp4_v = nullptr;
  const uint8_t* fp4_v_scale = nullptr;
  long long fp4_page_stride = 0;
  uint16_t* k16 = nullptr;
  uint16_t* v16 = nullptr;
  int32_t* pt_out = nullptr;
};
cudaError_t launch_page_decode(const PageDecodeArgs& a, cudaStream_t s);

// Packed-NVFP4 paged decode: one work unit per (query token, KV head) whose
// G <= 16 query heads form the 16 rows of warp-level MMAs; each unit attends
// over its token's own selected blocks. A list launch writes the units' block
// lists; the decode launch splits the list positions evenly over its CTAs.
constexpr int kFp4DecodeMaxCtas = 1024;  // partial slots in the workspace
struct Fp4DecodeArgs {
  unsigned* fault = nullptr;
  CUtensorMap tmap_kc;  // K codes (64 bytes, 128, Hkv, pages), 64-byte swizzle, box (64, 128, 1, 1)
  CUtensorMap tmap_vc;  // V codes, the same
  const uint16_t* q = nullptr;  // bf16 (total_q, Hq, 128)
  const int32_t* q2k = nullptr;  // (Hkv, total_q, topk)
  int topk = 0;
  const int32_t* cu_q = nullptr;
  const int32_t* page_table = nullptr;
  int max_pages = 0, num_pages = 0;
  const int32_t* seqused_k = nullptr;
  const uint8_t* k_scale = nullptr;  // (page, head) slice at p * page_stride + h * 1024
  const uint8_t* v_scale = nullptr;
  long long page_stride = 0;
  int batch = 0, total_q = 0, num_qo_heads = 0, num_kv_heads = 0, G = 0;
  float scale_log2 = 0.f;  // softmax scale * log2(e) * K global scale
  float out_scale = 1.f;   // V global scale
  uint16_t* out = nullptr;  // bf16 (total_q, Hq, 128)
  float* lse = nullptr;     // (total_q, Hq) or NULL
  // workspace (place_fp4_decode_workspace)
  int2* list = nullptr;      // (units, topk) of (page, visible keys); page -1: none
  int32_t* arrive = nullptr;  // (units): segments of the unit finished
  float* part_ml = nullptr;  // (max CTAs, 2, 16, 2): a segment's (m, l) per row
  float* part_o = nullptr;   // (max CTAs, 2, 16, 128): a segment's unnormalised O
};
size_t fp4_decode_workspace_bytes(long long units, int topk);
void place_fp4_decode_workspace(Fp4DecodeArgs* a, uint8_t* ws, long long units, int topk);
cudaError_t launch_fp4_decode(const Fp4DecodeArgs& a, cudaStream_t s);

// Per-head norm and rotation of q and k (rope.cu).
struct RopeArgs {
  const void* q = nullptr;  // (tokens, hq, 128) with token stride q_stride (elements); k, v alike
  const void* k = nullptr;
  const void* v = nullptr;
  long long q_stride = 0, k_stride = 0, v_stride = 0;
  int f16 = 0;  // else bf16
  int kv = 0;   // 0: K to k_out; 1: K and V to 16-bit pools; 2: to E4M3 pools
  const float* wq = nullptr;  // (128)
  const float* wk = nullptr;
  const float* cos_sin = nullptr;  // (max_position, rotary): cosines, then sines
  int max_position = 0, rotary = 0, interleaved = 0;
  const int32_t* positions = nullptr;  // (tokens)
  float eps = 0.f;
  int tokens = 0, hq = 0, hkv = 0;
  void* q_out = nullptr;  // (tokens, hq, 128)
  void* k_out = nullptr;
  const int32_t* cu_q = nullptr;
  int batch = 0;
  const int32_t* page_table = nullptr;  // (batch, max_pages)
  int max_pages = 0, num_pages = 0;
  const int32_t* seqused_k = nullptr;
  void* k_pool = nullptr;  // (num_pages, hkv, 128, 128)
  void* v_pool = nullptr;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);

struct RopeBwdArgs {
  const void* dq_out = nullptr;  // (tokens, hq, 128)
  const void* dk_out = nullptr;
  const void* q = nullptr;  // token strides in elements
  const void* k = nullptr;
  long long q_stride = 0, k_stride = 0;
  int f16 = 0;
  const float* wq = nullptr;
  const float* wk = nullptr;
  const float* cos_sin = nullptr;
  int max_position = 0, rotary = 0, interleaved = 0;
  const int32_t* positions = nullptr;
  float eps = 0.f;
  int tokens = 0, hq = 0, hkv = 0;
  void* dq = nullptr;
  void* dk = nullptr;
  long long dq_stride = 0, dk_stride = 0;
  float* dwq = nullptr;  // (128)
  float* dwk = nullptr;
  float* partials = nullptr;  // (blocks, 128): Q's blocks, then K's
  int q_blocks = 0;
};
struct RopeBwdGrid {
  int q_blocks, k_blocks;
};
RopeBwdGrid rope_bwd_grid(long long tokens, int hq, int hkv);
cudaError_t launch_rope_bwd(const RopeBwdArgs& a, int k_blocks, cudaStream_t s);

// Pages of a cache (cache.cu). Pools are (num_pages, ...) arrays of
// page_bytes per page that share one page numbering: K and V of every layer.
constexpr int kMaxCachePools = 256;    // pools per launch (longer lists take several)
constexpr int kMaxCacheRows = 16384;   // page table rows, and requests per call
constexpr int kMaxCopyPairs = 4096;    // page pairs per copy call
struct CachePools {
  void* base[kMaxCachePools];
};

struct CacheAcceptArgs {
  int num_pools = 0;
  int row_bytes = 0;   // one token's row of one KV head
  int hkv = 0;
  const int32_t* page_table = nullptr;
  int max_pages = 0, num_pages = 0, batch = 0;
  const int32_t* seqused_k = nullptr;
  const int32_t* cu_q = nullptr;
  const int32_t* path = nullptr;      // (batch, max_path)
  const int32_t* path_len = nullptr;  // (batch)
  int max_path = 0;
  int32_t* seqused_out = nullptr;
};
cudaError_t launch_cache_accept(const CachePools& p, const CacheAcceptArgs& a, cudaStream_t s);

struct CacheTableArgs {
  int32_t* page_table = nullptr;  // (num_rows, max_pages), -1 where a row has no page
  int max_pages = 0, num_rows = 0, num_pages = 0;
  int32_t* seqused_k = nullptr;   // (num_rows)
  int32_t* page_refs = nullptr;   // (num_pages): table entries naming the page
  const int32_t* rows = nullptr;  // (n): the rows freed, extended, or forked to
  const int32_t* src_rows = nullptr;  // (n): fork only
  const int32_t* lengths = nullptr;   // (n): extend only, the new lengths
  int n = 0;
  int32_t* status = nullptr;  // (n)
  int32_t* plan = nullptr;    // fork: (n) the fresh page, -1 none, -2 refused; then the list
  int32_t* list = nullptr;    // (num_pages): free pages, ascending
};
cudaError_t launch_cache_free(const CacheTableArgs& a, cudaStream_t s);
cudaError_t launch_cache_extend(const CacheTableArgs& a, cudaStream_t s);
// The plan; then, for each group of pools, the begun pages' copies, with the
// first group (tables) the rows too.
cudaError_t launch_cache_fork(const CacheTableArgs& a, cudaStream_t s);
cudaError_t launch_cache_fork_copy(const CachePools& p, int num_pools, long long page_bytes, bool tables,
                                   const CacheTableArgs& a, cudaStream_t s);
cudaError_t launch_cache_copy_pages(const CachePools& p, int num_pools, long long page_bytes,
                                    int num_pages, const int32_t* src, const int32_t* dst, int n,
                                    cudaStream_t s);

// A step's tables from its requests' lengths (step_tables.cu).
struct StepTablesArgs {
  const int32_t* page_table = nullptr;  // (num_rows, max_pages)
  int max_pages = 0, num_rows = 0, num_pages = 0;
  const int32_t* seqused_k = nullptr;  // (num_rows), the new tokens counted
  const int32_t* rows = nullptr;       // (batch)
  const int32_t* new_lens = nullptr;   // (batch)
  int batch = 0, total_q = 0;
  int32_t* cu_q = nullptr;         // (batch + 1)
  int32_t* seqused_out = nullptr;  // (batch)
  int32_t* table_out = nullptr;    // (batch, max_pages)
  int32_t* token_rows = nullptr;   // (total_q)
  int32_t* positions = nullptr;    // (total_q)
  long long* slots = nullptr;      // (total_q)
  int32_t* group_rows = nullptr;   // (batch)
  int32_t* cu_groups = nullptr;    // (batch + 1)
  int32_t* group_blocks = nullptr;  // (batch)
  int32_t* plan = nullptr;         // workspace (4, batch): nothing, leader, group, whole blocks before the new tokens
  int hash_slots = 0;
};
cudaError_t launch_step_tables(const StepTablesArgs& a, cudaStream_t s);

// The path of sampled tokens through trees of drafts (step_tables.cu).
struct DraftPathArgs {
  const int32_t* sampled = nullptr;  // (total_q)
  const int32_t* drafts = nullptr;   // (total_q)
  const uint32_t* mask = nullptr;    // (total_q, mask_words)
  int mask_words = 0;
  const int32_t* cu_q = nullptr;  // (batch + 1)
  int batch = 0, total_q = 0, max_path = 0;
  int32_t* path = nullptr;      // (batch, max_path)
  int32_t* path_len = nullptr;  // (batch)
  int32_t* next = nullptr;      // (batch)
};
cudaError_t launch_draft_path(const DraftPathArgs& a, cudaStream_t s);

// Tokens from logits (sample.cu).
constexpr int kMaxVocab = 1 << 19;
constexpr int kSampleParts = 1025;   // of a row's histogram
constexpr int kSampleStarts = 1032;  // where they begin in a slice's order, and its end; whole 16 bytes
struct SampleArgs {
  const void* logits = nullptr;  // (rows, vocab), `stride` values from row to row
  long long stride = 0;
  int type = 0;  // 0 bf16, 1 fp16, 2 fp32
  int rows = 0, vocab = 0;
  const float* uniforms = nullptr;     // (rows)
  const float* temperature = nullptr;  // (rows) or NULL, as the cuts
  const int32_t* top_k = nullptr;
  const float* top_p = nullptr;
  const float* min_p = nullptr;
  int32_t* tokens = nullptr;  // (rows)
  float* logprobs = nullptr;  // (rows) or NULL
  // Workspace.
  int slice = 0, slices = 0;             // values of a slice; slices of a row
  unsigned long long* best = nullptr;    // (rows, slices)
  uint32_t* parts_count = nullptr;       // (rows, kSampleParts)
  unsigned long long* parts_mass = nullptr;
  uint16_t* order = nullptr;             // (rows, slices, slice): a slice's tokens by parts
  uint16_t* starts = nullptr;            // (rows, slices, kSampleStarts): where the parts begin in it
};
struct SampleSlices {
  int slice, slices;  // (no slices of 16-bit logits)
};
SampleSlices sample_slices(int rows, int vocab, bool wide, bool aligned);
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s);
cudaError_t launch_sample_16(const SampleArgs& a, cudaStream_t s);

}  // namespace msa
