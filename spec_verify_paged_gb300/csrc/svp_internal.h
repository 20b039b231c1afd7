// svp_internal.h -- parameter blocks and launchers shared between the C-ABI
// host layer (api.cu) and the kernel translation units.  Not installed.
#pragma once
#include <cuda_runtime_api.h>
#include <cstddef>
#include <cstdint>

namespace svp {

struct SplitDesc;

constexpr int kBlockSize = 16;     // tokens per KV page
constexpr int kMaxQLen = 16;
constexpr int kMaxBatch = 65535;
constexpr int kMaxDraft = 15;
constexpr int kMaxPages = 1 << 26; // listed pages, pages to choose from
constexpr int kMaxNodes = 16;    // draft-tree nodes (= the verify rows)

// One paged_decode_attention launch.
struct AttnParams {
  const void *q;
  const void *k_cache;
  const void *v_cache;
  const int32_t *block_table;
  const int32_t *seq_lens;
  void *out;
  float *lse;
  // workspace pieces
  struct SplitDesc *desc;  // [grid] split group whose first page a CTA owns
  int2 *split;         // 4-bit kernel: [groups] first and last slice
  int merge_rows;      // 4-bit kernel: query rows the merge walks per group
  int whole;           // 4-bit kernel: one slice per group, no merge
  int parts;           // ... by this many warps of a CTA (1 unless whole)
  int slices;          // 4-bit kernel: set by its launcher, the partials' bound
  float *part_o;       // [2 * grid][RB][D] normalised partials: each CTA's
                       // first- and last-segment slot
  float *part_lse;     // [2 * grid][RB] log2-domain LSE of the partials
  int batch, num_q_heads, num_kv_heads, head_dim, group;
  int q_len, n_sink, window;
  int max_blocks, num_blocks;
  int rows;            // group * q_len query rows per (sequence, kv head)
  int rb;              // rows per work unit (row-group size)
  int n_rg;            // ceil(rows / rb)
  int min_pages;       // fewest items a CTA's slice may hold
  int seg_items;       // items that stand for a segment's fixed cost
  int ppi;             // pages per item: 1, or the tcgen05 kernel's tile
                       // (slices then split groups at tile boundaries)
  float qscale;        // scale * log2(e)
  const uint32_t *tree_mask;  // [batch, q_len] ancestor bits, or null
  float v_scale;       // FP8 caches: V value = code * v_scale (else 1)
  // 1: the previous kernel on the stream appended the q_len newest
  // positions of these sequences and wrote nothing else this call reads,
  // and every other input was written before it started.  The kernel then
  // reads everything but the pages holding those positions before its
  // grid-dependency wait, and waits before the first such page and before
  // its first write.  0: it waits before touching global memory.
  int early;
};

struct AttnPlan {
  int rb, n_rg, min_pages, seg_items, grid, ctas_per_sm;
  bool mma;            // warp-level mma.sync path
  bool tc;             // tcgen05 path (tensor-memory accumulators)
  bool fp4;            // 4-bit cache kernel
  bool whole;          // its slices are whole groups: no workspace, no merge
  int parts;           // and this many warps take one
  int batch_cap;       // sequences per launch
  size_t ws_head, ws_desc, ws_part_o, ws_part_lse, ws_total;
};

// paged_decode_attention (tree_mask null) or paged_tree_attention launched
// right after kv_append of the q_len newest positions on the same stream
// (the fused step): the prefix pages are read while the append runs.
int attention_after_append(const svp_dims *dims, const void *q,
                           const void *k_cache, const void *v_cache,
                           const int32_t *block_table, const int32_t *seq_lens,
                           int q_len, int n_sink, int window,
                           const uint32_t *tree_mask, float scale, void *out,
                           float *lse, cudaStream_t stream);

// Fills the plan (no CUDA launches).  dtype 0 = f32, 1 = bf16.  Returns 0 or
// a negative svp_status.
int plan_attention(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                   int dtype, int max_blocks, int q_len, int n_sink,
                   int window, int split_pages, int kernel_path, int num_sms,
                   long long num_blocks, AttnPlan *plan);

// The tcgen05 kernel's stream-K items are 8-page tiles; a segment's fixed
// cost (the masked last tile, epilogue, next Q) takes about two tiles'
// time: the split counts it.
constexpr int kTilePagesTc = 8;
constexpr int kSegItemsTc = 2;
// The CUDA-core kernel's items are pages; a segment's epilogue (the four
// warps' states merged through shared memory, the rows written out) is
// counted as this many pages.
constexpr int kSegItemsCc = 12;

// The 4-bit kernel's items are the four pages of a stage; a segment's fixed
// cost (Q, the result) counts as one.  At most kBatchFp4 sequences per
// launch: their prefix shares shared memory with the page ring.
constexpr int kTilePagesFp4 = 4;
constexpr int kSegItemsFp4 = 1;
constexpr int kBatchFp4 = 512;

// Query rows per kv head (GQA group x q_len) from which the automatic path
// choice uses tensor cores (bf16 only): tcgen05 for head_dim 128, warp-level
// mma.sync for head_dim 64.
constexpr int kMmaMinRows = 3;

// The same for 4-bit caches at head_dim 128: below, the mma.sync kernel, whose
// units convert the cache once per 16 or 24 rows (98 MB of cache, 8 heads: 4
// rows 35 us against 66 on tcgen05, 16 47 against 66, 24 61 against 76, 32 74
// against 76; 36 97 against 89, 48 99 against 90, 60 126 against 90).
constexpr int kFp4TcMinRows = 33;

// Occupancy-derived CTAs per SM for the attention kernel of this shape
// (queried once per device and shape, cached).
int attention_ctas_per_sm(int dtype, int head_dim, int rb, bool mma,
                          int batch);

cudaError_t launch_attention(const AttnParams &p, int dtype, bool mma,
                             int grid, cudaStream_t stream);

// The merge of split groups after either attention kernel (same grid).
cudaError_t launch_merge(const AttnParams &p, int dtype, int grid,
                         cudaStream_t stream);

// True when the driver provides cuTensorMapEncodeTiled.
bool tensor_maps_available();

// The tcgen05 kernel (attention_tc.cu): bf16, head_dim 128, 16 or 32 rows
// per group, at most tc_batch_cap() sequences per launch.
int tc_batch_cap();
int attention_tc_ctas_per_sm(int rb, int batch);
cudaError_t launch_attention_tc(const AttnParams &p, int grid,
                                cudaStream_t stream);

// The 4-bit cache kernels (attention_fp4.cu): the unit's row count (8, 16 or
// 24) for this many query rows per kv head and pages of the launch, the warps
// (slices) of a CTA, of which an SM holds one, and the launch of attention
// and merge.
// Calls whose sequences span at most kWholePages pages take whole groups,
// shared by up to kMaxParts warps, if a warp then has kPartPages at most (call
// times, one query row, 8 heads, 31 pages: 1 sequence 10.1 us against 14.1 in
// slices, 32 13.5 against 16.8, 128 27.6 against 33.2; 300, where warps take
// turns, 64.6 against 59.9.  63 pages: 1 sequence 12.7 against 14.0, 32 19.5
// against 23.1).
constexpr int kWholePages = 64;
constexpr int kPartPages = 32;
constexpr int kMaxParts = 8;
int attention_fp4_rows(int rows, long long pages, int sms);
int attention_fp4_warps(int rb);
cudaError_t launch_attention_fp4(const AttnParams &p, int grid,
                                 cudaStream_t stream);

// The tcgen05 kernel over 4-bit caches (attention_fp4_tc.cu): head_dim 128,
// units of 16, 32 or 64 rows; plan, batch cap and merge as attention_tc.cu.
int attention_fp4_tc_ctas_per_sm(int rb, int batch);
cudaError_t launch_attention_fp4_tc(const AttnParams &p, int grid,
                                    cudaStream_t stream);

struct AppendParams {
  const void *k_new;
  const void *v_new;
  void *k_cache;
  void *v_cache;
  const int32_t *block_table;
  const int32_t *seq_lens;
  int batch, num_kv_heads, head_dim, n_new, max_blocks, num_blocks;
  int elem_bytes;
  int fp8;                   // bf16 rows quantised into E4M3 caches
  int fp4;                   // bf16 rows quantised into 4-bit caches
  float k_scale, v_scale;
};
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream);

struct GatherParams {
  const void *k_cache;
  const void *v_cache;
  const int32_t *block_table;
  const int32_t *seq_lens;
  const int32_t *starts;     // or null: the newest n_rows positions
  void *k_out;
  void *v_out;
  int batch, num_kv_heads, head_dim, n_rows, max_blocks, num_blocks;
  int dtype;                 // svp_dtype of the caches
  float k_scale, v_scale;
};
cudaError_t launch_kv_gather(const GatherParams &p, cudaStream_t stream);

// One paged_score_update launch: query rows [row0, row0 + rows) of every kv
// head's group * q_len.
struct ScoreParams {
  const void *q;
  const void *k_cache;
  const float *lse;
  const int32_t *block_table;
  const int32_t *seq_lens;
  const uint32_t *tree_mask;  // [batch, q_len] ancestor bits, or null
  float *scores;
  int batch, num_q_heads, num_kv_heads, head_dim, group;
  int q_len, n_sink, window, n_fresh;
  int row0, rows;
  int max_blocks, num_blocks;
  int max_pages;              // bound of a sequence's visible pages
  int dtype;
  float qscale;               // scale * k_scale * log2(e)
};
constexpr int kScoreRows = 128;  // query rows of one launch
cudaError_t launch_score_update(const ScoreParams &p, int sms,
                                cudaStream_t stream);

// kv_append of packed rows: row i of k_new / v_new [n_rows, Hkv, D] to slot
// slots[i] (page * 16 + row; negative: nowhere).
struct AppendSlotsParams {
  const void *k_new;
  const void *v_new;
  void *k_cache;
  void *v_cache;
  const long long *slots;
  long long n_rows;
  int num_kv_heads, head_dim, num_blocks;
  int dtype;                 // svp_dtype of the caches
  float k_scale, v_scale;
};
cudaError_t launch_append_slots(const AppendSlotsParams &p, cudaStream_t stream);

// Page bounds, scores and selection (page_select.cu).
struct BoundsParams {
  const void *k_cache;
  void *bounds;               // bf16 [num_blocks, Hkv, 2, D]
  const int32_t *block_table;
  const int32_t *seq_lens;
  int batch, num_kv_heads, head_dim, n_new, max_blocks, num_blocks;
  int max_pages;              // bound of the pages that n_new positions touch
  int dtype;
  int heads;                  // set by the launcher: heads that a warp takes
};
cudaError_t launch_page_bounds(BoundsParams p, int sms, cudaStream_t stream);

struct PageScoreParams {
  const void *q;
  const void *bounds;
  const int32_t *block_table;
  const int32_t *seq_lens;
  float *scores;              // [batch, Hkv, max_blocks]
  int batch, num_q_heads, num_kv_heads, head_dim, group, q_len;
  int max_blocks, num_blocks;
  int row0, rows;             // query rows of this launch
  int more;                   // not the first launch: add to what is there
  int f32;                    // q is fp32
  int negate;                 // the scale is negative
  float scale;                // its magnitude
  int tiles_per_cta, chunks;  // set by the launcher
};
constexpr int kPageScoreRows = 128;  // query rows of one launch
constexpr int kPageScoreRowsF32 = 64;
cudaError_t launch_page_scores(PageScoreParams p, int sms, cudaStream_t stream);

struct PickParams {
  const float *scores;        // [batch, heads, max_blocks]
  const int32_t *seq_lens;
  int32_t *pages;             // [batch, heads, n_select]
  int batch, heads, max_blocks, n_select, n_sink, n_recent;
};
cudaError_t launch_pick_pages(const PickParams &p, cudaStream_t stream);

// One paged_sparse_attention call (attention_sparse.cu).
struct SparseParams {
  const void *q;
  const void *k_cache;
  const void *v_cache;
  const int32_t *block_table;
  const int32_t *seq_lens;
  const int32_t *pages;       // [batch, Hkv, n_select]
  const uint32_t *tree_mask;  // [batch, q_len] ancestor bits, or null
  void *out;
  float *lse;
  int batch, num_q_heads, num_kv_heads, head_dim, group, q_len;
  int n_select, max_blocks, num_blocks;
  int rows;                   // group * q_len
  int n_rb;                   // set by the launcher: units of these rows
  int split_pages;            // fewest list entries of a CTA, 0 = automatic
  float qscale;               // scale * log2(e) (* k_scale)
  float v_scale;
};
cudaError_t launch_sparse_attention(const SparseParams &p, int dtype, int sms,
                                    cudaStream_t stream);

constexpr int kSpCluster = 16;  // most CTAs of a unit; above 8 by leave

// CTAs that share a unit's list.  per_sm: CTAs that an SM holds; sixteen_fit():
// whether the device can place a cluster of sixteen, only asked where one is
// wanted.
template <class Fit>
int sparse_splits(long long units, int n_select, int split_pages, int sms, int per_sm,
                  bool f32, Fit sixteen_fit) {
  // split a list while the CTAs all find room and keep eight pages, or to the
  // caller's pages per CTA: 256 units of 128 bf16 pages take 44 us whole, 48 in
  // halves and 56 in quarters; 64 units of 256 FP8 pages 22 in quarters, 28 in
  // halves; 32 units of 128 fp32 pages, one CTA to an SM, 14 in quarters, 26 in
  // eighths
  const long long least = split_pages > 0 ? split_pages : 8;
  int splits = 1;
  while (splits < 8 && 2LL * splits * least <= n_select &&
         (split_pages > 0 || units * splits * 2 <= (long long)per_sm * sms))
    splits *= 2;
  // Sixteen where the CTAs leave room to spare, as larger clusters are placed
  // less evenly, which fp32's bytes feel first.  2048 pages of one sequence, 4
  // rows, eighths and sixteenths: one head bf16 28 us and 17, fp32 76 and 41; 8
  // heads bf16 34 and 29, FP8 31 and 30, fp32 77 and 83 (six units: 122 and 65).
  // (8 heads of 512 pages: bf16 11.0 and 10.3, but FP8 11.7 and 12.2; the rule
  // does not tell these types apart.)
  if (splits == 8 && 2LL * splits * least <= n_select &&
      units * kSpCluster <= (f32 ? sms * 2 / 3 : sms) && sixteen_fit())
    splits = kSpCluster;
  return splits;
}

struct AssignParams {
  int32_t *block_table;
  int32_t *seq_lens;
  const int32_t *new_lens;
  int32_t *free_pages;        // [capacity] stack
  int32_t *free_count;
  long long *slots;           // [n_slots] or null
  int32_t *offsets;           // [batch + 1] or null
  int batch, max_blocks, num_blocks, capacity, n_slots;
};
cudaError_t launch_assign_pages(const AssignParams &p, cudaStream_t stream);

struct LogprobParams {
  const void *logits;         // [rows, vocab]
  const int32_t *tokens;
  const uint32_t *allowed;    // [rows, words] or null
  float *logprobs;
  float *entropy;             // or null
  int32_t *ranks;             // or null
  float *top_logprobs;        // [rows, n_top]
  int32_t *top_tokens;
  int rows, vocab, words, n_top;
  float inv_t;                // 1 / temperature
  float sc;                   // log2(e) / temperature
};
constexpr int kMaxTop = 64;
constexpr int kMaxVocab = 320000;
cudaError_t launch_token_logprobs(const LogprobParams &p, int dtype, int sms,
                                  cudaStream_t stream);

struct EvictParams {
  void *k_cache;
  void *v_cache;
  float *scores;
  const int32_t *block_table;
  const int32_t *dst_table;   // the destination's block table
  const int32_t *seq_lens;
  int32_t *kept;
  int32_t *new_lens;
  int batch, num_kv_heads, row_bytes, max_blocks, dst_blocks, num_blocks;
  int budget, n_sink, n_recent;
};
cudaError_t launch_kv_evict(const EvictParams &p, int sms, cudaStream_t stream);

struct AcceptParams {
  const float *target_logits;
  const float *draft_logits;
  const int32_t *draft_tokens;
  const float *uniforms;
  int32_t *out_tokens;
  int32_t *n_accepted;
  int batch, num_draft, vocab;
  float sc;                  // log2(e) / temperature
  const uint32_t *allowed;   // [batch, K+1, words] token masks, or null
  int words;                 // (vocab + 31) / 32
  int greedy;                // argmax verification
  cudaStream_t stream;       // set by the launcher
};
cudaError_t launch_spec_accept(const AcceptParams &p, cudaStream_t stream);

struct AcceptTreeParams {
  const float *target_logits;  // [batch, N, vocab]
  const float *draft_logits;   // [batch, N, vocab]
  const int32_t *parents;      // [batch, N]
  const int32_t *node_tokens;  // [batch, N]
  const float *uniforms;       // [batch, N]
  int32_t *out_tokens;         // [batch, N]
  int32_t *out_nodes;          // [batch, N]
  int32_t *n_accepted;         // [batch]
  int batch, num_nodes, vocab;
};
cudaError_t launch_spec_accept_tree(const AcceptTreeParams &p,
                                    cudaStream_t stream);

// Device status words (one per translation unit), on the current device.
cudaError_t status_word_attention(unsigned **word);
cudaError_t status_word_attention_tc(unsigned **word);
cudaError_t status_word_attention_fp4(unsigned **word);
cudaError_t status_word_attention_fp4_tc(unsigned **word);
cudaError_t status_word_append(unsigned **word);
cudaError_t status_word_score(unsigned **word);
cudaError_t status_word_evict(unsigned **word);
cudaError_t status_word_accept(unsigned **word);
cudaError_t status_word_pages(unsigned **word);
cudaError_t status_word_sparse(unsigned **word);
cudaError_t status_word_assign(unsigned **word);
cudaError_t status_word_logprobs(unsigned **word);

#ifdef __CUDACC__
// A launch that may start while the previous kernel on the stream is still
// running (programmatic dependent launch); the kernel itself waits for that
// kernel's results (pdl_wait) before it reads anything it could have
// written.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), unsigned grid, unsigned block,
                       size_t smem, cudaStream_t stream, Args &&...args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args &&>(args)...);
}
#endif

}  // namespace svp
