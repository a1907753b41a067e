// Internal host/device interfaces shared by the translation units of libwise.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace wise {

// The paged-cache kernels are launched as programmatic dependents of whatever
// precedes them in the stream: a kernel that has triggered (grid_trigger) lets
// the next one's blocks start and set themselves up while it still runs. Every
// block calls grid_wait before its first access to global memory, which waits
// until the kernels before it are complete and their writes visible, and before
// it triggers: when a launch's blocks start, the launch two before it is complete.
// One launch runs beside the one before it instead (the own parts of
// wise_attn_prefix): it calls grid_wait at its end, and what it reads was ordered
// by a word that the plan, two launches before it, released and it acquires
// (TreeLaunch::go). What earlier kernels may have written is loaded plainly, never
// with __ldg: that names data which nothing writes while the kernel runs, so the
// compiler may move it above the wait.
template <class... P, class... A>
inline cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                  const A&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

struct AttnParams {
  int32_t bh_count;     // batch * heads
  int32_t heads;        // query heads per batch element
  int32_t kv_group;     // query heads per key/value head (1 without grouped-query attention)
  int32_t n;            // sequence length
  int32_t nb;           // n / BN key (and query) blocks
  int32_t n_qtiles;     // ceil(n / 128): work units (query tiles) per (batch, head)
  int32_t group_heads;  // (batch, head) slices per L2 group in the default order
  float scale_log2;     // softmax scale * log2(e)
  int32_t out_f32;      // O dtype: 0 bf16, 1 f32
  void* o;
  float* lse;           // optional
  float* mass;          // optional [bh, nb, nb] (discover only)
  float* lam;           // per-row, per-entry, per-half log2-sum-exp scratch (mass only)
  const int32_t* row_ptr;
  const int32_t* col_idx;
  int64_t col_cap;
  const int32_t* tile_order;  // optional unit order (reuse only)
  int64_t n_units;
  uint32_t* err;
  uint32_t sched_slot;  // work-counter slot of this launch
  // Selection fused into discovery with masses (one step of the window):
  // each completed mass row's Eq 6 step support is written (first step) or
  // OR-ed into sel_bits; the last step adds the sink / diagonal blocks and
  // writes the row counts. Off when sel_bits is null.
  uint32_t* sel_bits;   // [bh * nb, sel_nwords]
  int32_t* sel_counts;  // [bh * nb]
  int64_t sel_target_fx, sel_tol_fx;
  int32_t sel_nwords;
  int32_t sel_first, sel_last;
  uint32_t sel_flags;
  // Sparse steps with blocks of 32: the tiles' gathered entries, built once
  // per support (gather_plan.cu). Without them (null) the scheduler forms
  // each claimed tile's entries from its four CSR rows.
  const int32_t* plan_counts;    // [n_units] entries per tile
  const uint32_t* plan_entries;  // 4 words per entry, at plan_entry_index(bh, t, n_qtiles)
};

// Gathered-entry plan of sparse steps with blocks of 32: per work unit (one
// 128-row tile of one (batch, head) slice) its entry count, then, 16-byte
// aligned, the entries of each slice as a triangle: tile t has at most t + 1
// (its query blocks admit key blocks 0 .. 4t + 3, four per entry). An entry
// is four words: key blocks of slots 0 | 1 << 16, of slots 2 | 3 << 16, the
// slot mask (bit 4j + c: query block j of the tile lists slot c's block), 0.
__host__ __device__ inline int64_t plan_entry_index(int64_t bh, int64_t t, int64_t n_qtiles) {
  return bh * (n_qtiles * (n_qtiles + 1) / 2) + t * (t + 1) / 2;
}
__host__ __device__ inline int64_t plan_counts_bytes(int64_t n_units) { return (n_units * 4 + 15) / 16 * 16; }
__host__ __device__ inline int64_t plan_bytes(int64_t bh, int64_t n_qtiles) {
  return plan_counts_bytes(bh * n_qtiles) + plan_entry_index(bh, 0, n_qtiles) * 16;
}

struct GatherPlanLaunch {
  const int32_t* row_ptr;
  const int32_t* col_idx;
  int64_t col_cap;
  int32_t bh_count, nb, n_qtiles;
  int32_t* counts;
  uint32_t* entries;
  uint32_t* err;
};
cudaError_t launch_gather_plan(const GatherPlanLaunch& g, cudaStream_t stream);

struct SelectLaunch {
  const float* mass;
  int32_t window, bh_count, nb;
  int64_t target_fx, tol_fx;
  uint32_t flags;
  uint32_t* bits;
  int32_t* counts;
  int32_t* row_ptr;
  int32_t* col_idx;
  int64_t col_cap;
  int32_t* nnz;
  int32_t* tile_order;
  int32_t units_per_bh, qb_per_unit;
  int32_t mode;                // 0: Eq 6; 1: MassMatched; 2: SizeMatched (window 1)
  int32_t finalize_only;       // bits and counts are already built (fused selection)
  const int32_t* ref_row_ptr;  // reference working set of the controls
  const int32_t* ref_col_idx;
  int64_t ref_cap;
  uint32_t* err;
};

// Launch the attention kernel for one head dimension (defined in
// attn_d{64,96,128}.cu). maps = {Q, K, V, K128, V128} tensor maps (the last
// two with 128-row boxes, for consecutive gathered blocks of 32).
cudaError_t launch_attn_d64(int block, bool sparse, const CUtensorMap* maps, const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_d96(int block, bool sparse, const CUtensorMap* maps, const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_d128(int block, bool sparse, const CUtensorMap* maps, const AttnParams& p, cudaStream_t st);

cudaError_t launch_select(const SelectLaunch& s, cudaStream_t stream);

// Selection workspace layout: the row bitmasks [rows][nwords] and counts
// [rows] (int32), then, 16-byte aligned, the look-back state of the row_ptr
// scan (one 64-bit word per chunk of kSelectChunkRows rows plus a ticket).
constexpr int kSelectChunkRows = 256;
__host__ __device__ inline int64_t select_lookback_offset(int64_t rows, int64_t nwords) {
  return ((rows * nwords + rows) * 4 + 15) / 16 * 16;
}
__host__ __device__ inline int64_t select_lookback_bytes(int64_t rows) {
  return ((rows + kSelectChunkRows - 1) / kSelectChunkRows) * 8 + 16;
}

// Support diagnostics (diag_kernel.cu): retained future attention mass and
// the Jaccard index of two supports.
struct DiagLaunch {
  int64_t rows;  // batch * heads * nb CSR rows
  int32_t nb, batch;
  int64_t col_cap;           // col_idx entries of support A that may be read
  int64_t col_cap_b;         // ... of support B
  const float* mass;         // [rows, nb] (retained mass)
  const int32_t* row_ptr_a;  // support A (the only one for retained mass)
  const int32_t* col_idx_a;
  const int32_t* row_ptr_b;  // support B (Jaccard)
  const int32_t* col_idx_b;
  float* row_value;          // [rows] retained mass per row
  int32_t* row_counts;       // [rows][2] |A intersect B|, |A union B| per row
  double* batch_value;       // [batch] mean retained mass or Jaccard index (optional)
  long long* batch_counts;   // [batch][2] summed counts (optional)
  uint32_t* err;
};
cudaError_t launch_retained_mass(const DiagLaunch& d, cudaStream_t stream);
cudaError_t launch_jaccard(const DiagLaunch& d, cudaStream_t stream);

// A paged cache as the kernels see it (wise_paged_cache).
struct CacheView {
  int32_t batch, kv_heads, page_shift, max_pages;
  int64_t n_pages;
  uint16_t* k_pages;
  uint16_t* v_pages;
  const int32_t* page_table;
  const int32_t* lengths;
};
// Rows [batch, heads, n, d] with strides in elements (wise_rows).
struct RowsView {
  const uint16_t* data;
  int64_t sb, sh, sn;
};

// Cache maintenance (cache_kernel.cu).
struct AppendLaunch {
  CacheView cache;
  int32_t head_dim, n;
  RowsView k, v, q;
  int32_t heads;  // query heads; 0 without q
  uint16_t* q_out;
  const int32_t* new_len;
  const int32_t* positions;
  const int64_t* rope;
  int32_t rotary_dim;
  int32_t pairs;  // rotate neighbouring values instead of halves
  uint32_t* err;
};
cudaError_t launch_cache_append(const AppendLaunch& a, cudaStream_t stream);

struct AcceptLaunch {
  CacheView cache;
  int32_t head_dim, path_tokens;
  const int32_t* path;
  const int32_t* n_accepted;
  int32_t* new_lengths;
  uint32_t* err;
};
cudaError_t launch_cache_accept(const AcceptLaunch& a, cudaStream_t stream);

// Attention of new tokens over a paged cache (tree_wide.cuh, tree_narrow.cuh). The key
// tiles and kTreeOverhead places of each unit must number at most 2^31 - 1.
constexpr int kTreeMaxTokens = 128;
constexpr uint64_t kPlanTag = 0x706c616eull << 32;  // upper half of TreeLaunch::go
constexpr int kTreeOverhead = 8;  // at most this many places of the line of work per unit, besides its key tiles
struct TreeLaunch {
  CacheView cache;
  int32_t head_dim, heads, n;
  RowsView q;
  const int32_t* new_len;
  const int32_t* tree_mask;
  float scale;
  int32_t out_f32;
  void* o;
  float* lse;
  void* workspace;
  uint32_t* err;
  // For wise_attn_prefix's two launches (null and 0 elsewhere):
  const int32_t* skip;    // [batch]: tokens at the front of each sequence that are left out
  const int32_t* limit;   // the shared part's: blocks that have a share in it (the others leave at once)
  // Set: runs beside the launch before it, which it waits for at its end. The plan's
  // word: kPlanTag, and the blocks that share the work below it; taken back by the join.
  const uint64_t* go;
  int32_t rows_apart;     // records of all units, and no join
  // for groups of sequences over what they share: cache.batch counts groups, cache.lengths
  // are their shared tokens, cache.page_table and the rest are the sequences'
  const int32_t* starts;  // [groups + 1]: each group's first sequence
  const int32_t* leader;  // [groups]: the sequence whose page table is read
  int32_t sequences;      // of all groups
  int32_t members;        // of a group, at most
};
int64_t tree_workspace_bytes(int32_t batch, int32_t kv_heads, int32_t heads, int32_t n, int32_t head_dim);
// maps = {K, V}: 3-D tensor maps [n_pages, kv_heads * page, d] with boxes of one
// page of one head.
cudaError_t launch_tree(const TreeLaunch& t, const CUtensorMap* maps, cudaStream_t stream);

// Rows normed per head and rotated (norm_kernel.cu): into a paged cache, or
// dense ones.
constexpr int64_t kMaxNormHeads = 1ll << 18;  // of queries, keys and values together
struct NormLaunch {
  CacheView cache;  // paged
  int32_t paged;
  int32_t batch, n, head_dim, heads, kv_heads;  // heads: 0 without q
  RowsView q, k, v;                             // k, v: data null without them
  uint16_t* q_out;
  uint16_t* k_out;  // pool, or dense rows
  uint16_t* v_out;  // pool
  const int32_t* new_len;
  const int32_t* positions;  // [n_axes, batch, n]
  const int64_t* rope;
  const int32_t* axes;  // [rotary_dim / 2] or null: axis 0
  int32_t n_axes, rotary_dim, pairs;
  const void* q_weight;  // null: not normed
  const void* k_weight;
  int64_t q_weight_stride, k_weight_stride;  // elements from head to head (0: shared)
  int32_t weight_f32;
  float eps;
  int32_t part_heads, parts[2];  // set by launch_norm: heads of a block, blocks of q's and of k's
  uint32_t* err;
};
cudaError_t launch_norm(const NormLaunch& a, cudaStream_t stream);

// Eviction by weight (evict_kernel.cu).
struct EvictLaunch {
  CacheView cache;
  int32_t head_dim;
  int32_t budget, recent, sink;
  const float* weights;  // [batch, kv_heads, width]
  int64_t width;
  const int32_t* to_table;  // [batch, to_pages]
  int32_t to_pages;
  int32_t chunks;  // blocks of the move per key head
  int32_t* new_lengths;
  float* weights_out;  // [batch, kv_heads, width_out]
  int64_t width_out;
  int32_t* list;  // [batch, kv_heads, list_width]: kept places
  int64_t list_width;
  uint32_t* err;
};
int64_t evict_move_chunks(int64_t budget, int64_t width_out);
cudaError_t launch_evict(const EvictLaunch& e, cudaStream_t stream);

// Attention of a batch whose sequences share prefixes (prefix_kernel.cu): t as for
// launch_tree, with the whole call's workspace.
struct PrefixLaunch {
  TreeLaunch t;
  int32_t groups;
  const int32_t* group_starts;  // [groups + 1] or null: one group of all sequences
  const int32_t* prefix_lengths;  // [groups]
  int32_t members;                // sequences of a group, at most
};
int64_t prefix_workspace_bytes(int32_t batch, int32_t kv_heads, int32_t heads, int32_t n, int32_t head_dim, int32_t groups);
cudaError_t launch_prefix(const PrefixLaunch& p, const CUtensorMap* maps, cudaStream_t stream);

// Attention weight of new tokens, summed per cached token (weights_kernel.cu).
struct WeightsLaunch {
  CacheView cache;
  int32_t head_dim, heads, n;
  RowsView q;
  const float* lse;  // [batch, heads, n]
  const int32_t* new_len;
  const int32_t* tree_mask;
  float scale;
  float* weights;  // [batch, kv_heads, width]
  int64_t width;
  uint32_t* err;
};
// map = K's tensor map, as for launch_tree
cudaError_t launch_weights(const WeightsLaunch& w, const CUtensorMap* map, cudaStream_t stream);

}  // namespace wise
