// C ABI of libwise (declared in include/wise.h): argument validation, TMA
// descriptor encoding, workspace sizing, dispatch to the kernels, and the
// device error word.
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <mutex>
#include <vector>

#include "internal.h"
#include "ptx.cuh"
#include "wise.h"

// The one piece of library state: a per-device word that kernels OR error
// bits into (bounded-wait timeouts, malformed supports).
__device__ uint32_t g_wise_error_word;

namespace wise {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxBlocks = 1024;
constexpr size_t kL2GroupBytes = 32ull << 20;  // K/V bytes kept hot per group of heads

std::mutex g_mu;
uint32_t* g_err_ptr[kMaxDevices] = {};
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

int current_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  return dev;
}

// Device address of g_wise_error_word on the current device (looked up once).
uint32_t* error_word() {
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_err_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_wise_error_word) != cudaSuccess) return nullptr;
    g_err_ptr[dev] = static_cast<uint32_t*>(p);
  }
  return g_err_ptr[dev];
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  return g_encode;
}

// 2D view [rows = batch*heads*seq_len, head_dim] of a bf16 tensor; boxes of
// `box_rows` rows and 64 (128B swizzle) or 32 (64B swizzle, head_dim 96)
// columns.
int encode_map(CUtensorMap* m, const void* ptr, int64_t rows, int d, int box_rows) {
  auto enc = encoder();
  if (!enc) return WISE_ERR_CUDA;
  const int ch = (d == 96) ? 32 : 64;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {(cuuint32_t)ch, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, ch == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? WISE_OK : WISE_ERR_UNSUPPORTED;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_desc(const wise_attn_desc* d) {
  if (!d) return WISE_ERR_INVALID_ARGUMENT;
  if (d->batch < 1 || d->heads < 1 || d->seq_len < 1 || d->block < 1) return WISE_ERR_INVALID_ARGUMENT;
  if (d->kv_heads < 0 || (d->kv_heads > 0 && d->heads % d->kv_heads != 0)) return WISE_ERR_INVALID_ARGUMENT;
  if (d->out_dtype != WISE_BF16 && d->out_dtype != WISE_F32) return WISE_ERR_INVALID_ARGUMENT;
  if (!(d->softmax_scale >= 0.f) || isinf(d->softmax_scale)) return WISE_ERR_INVALID_ARGUMENT;
  if (d->seq_len % d->block != 0) return WISE_ERR_INVALID_ARGUMENT;
  if (d->head_dim != 64 && d->head_dim != 96 && d->head_dim != 128) return WISE_ERR_UNSUPPORTED;
  if (d->block != 32 && d->block != 64 && d->block != 128) return WISE_ERR_UNSUPPORTED;
  if (d->seq_len / d->block > kMaxBlocks) return WISE_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)d->batch * d->heads * d->seq_len;
  if (rows + 256 > INT32_MAX) return WISE_ERR_UNSUPPORTED;
  return WISE_OK;
}

struct Shape {
  int64_t bh;
  int n, d, bn, nb, n_qtiles, group_heads;
  int heads, kv_heads;  // kv_heads divides heads (grouped-query attention)
  int64_t n_units;
};

Shape shape_of(const wise_attn_desc* d) {
  Shape s;
  s.bh = (int64_t)d->batch * d->heads;
  s.n = d->seq_len;
  s.d = d->head_dim;
  s.bn = d->block;
  s.nb = d->seq_len / d->block;
  s.n_qtiles = (d->seq_len + 127) / 128;
  s.heads = d->heads;
  s.kv_heads = d->kv_heads > 0 ? d->kv_heads : d->heads;
  // K/V bytes per query head (query heads that share a key/value head share it)
  const size_t kv_per_head = (size_t)2 * d->seq_len * d->head_dim * 2 * s.kv_heads / s.heads;
  int64_t g = (int64_t)(kL2GroupBytes / (kv_per_head > 0 ? kv_per_head : 1));
  if (g < 1) g = 1;
  if (g > s.bh) g = s.bh;
  s.group_heads = (int)g;
  s.n_units = s.bh * s.n_qtiles;
  return s;
}

size_t lam_bytes(const Shape& s) {
  const int64_t ept = 128 / s.bn;
  const int64_t per_bh = ept * (int64_t)s.n_qtiles * (s.n_qtiles + 1) / 2;
  return (size_t)(s.bh * per_bh * 128 * sizeof(float));
}

int64_t fixed_point(double x);

// One step of a selection window fused into discovery (see AttnParams).
struct FusedSelect {
  uint32_t* bits;
  int32_t* counts;
  int64_t target_fx, tol_fx;
  int32_t nwords, first, last;
  uint32_t flags;
};

int launch_attention(const wise_attn_desc* desc, const void* q, const void* k, const void* v, void* o, float* lse,
                     float* mass, void* ws, const int32_t* row_ptr, const int32_t* col_idx, int64_t col_cap,
                     const int32_t* tile_order, bool sparse, cudaStream_t stream,
                     const FusedSelect* fs = nullptr, const void* plan = nullptr) {
  const Shape s = shape_of(desc);
  uint32_t* err = error_word();
  if (!err) return WISE_ERR_CUDA;
  // Q, K, V, and K, V with 128-row boxes (consecutive gathered blocks; the
  // same maps as K, V for the other variants)
  CUtensorMap maps[5];
  const int64_t rows = s.bh * s.n;
  const int64_t kv_rows = (int64_t)desc->batch * s.kv_heads * s.n;
  // K/V boxes: one key block (64 or 128 rows); blocks of 32 use 128-row
  // boxes in discovery and one 32-row box per gathered block in sparse steps
  const int kv_box = (s.bn == 32) ? (sparse ? 32 : 128) : s.bn;
  int st = encode_map(&maps[0], q, rows, s.d, 128);
  if (st == WISE_OK) st = encode_map(&maps[1], k, kv_rows, s.d, kv_box);
  if (st == WISE_OK) st = encode_map(&maps[2], v, kv_rows, s.d, kv_box);
  if (st == WISE_OK) st = encode_map(&maps[3], k, kv_rows, s.d, kv_box == 32 ? 128 : kv_box);
  if (st == WISE_OK) st = encode_map(&maps[4], v, kv_rows, s.d, kv_box == 32 ? 128 : kv_box);
  if (st != WISE_OK) return st;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.bh_count = (int32_t)s.bh;
  p.heads = s.heads;
  p.kv_group = s.heads / s.kv_heads;
  p.n = s.n;
  p.nb = s.nb;
  p.n_qtiles = s.n_qtiles;
  p.group_heads = s.group_heads;
  const float scale = desc->softmax_scale > 0.f ? desc->softmax_scale : 1.0f / sqrtf((float)s.d);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out_f32 = desc->out_dtype == WISE_F32;
  p.o = o;
  p.lse = lse;
  p.mass = mass;
  p.lam = static_cast<float*>(ws);
  p.row_ptr = row_ptr;
  p.col_idx = col_idx;
  p.col_cap = col_cap;
  p.tile_order = tile_order;
  p.n_units = s.n_units;
  p.err = err;
  if (plan) {
    p.plan_counts = static_cast<const int32_t*>(plan);
    p.plan_entries = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(plan) +
                                                        plan_counts_bytes(s.n_units));
  }
  if (fs) {
    p.sel_bits = fs->bits;
    p.sel_counts = fs->counts;
    p.sel_target_fx = fs->target_fx;
    p.sel_tol_fx = fs->tol_fx;
    p.sel_nwords = fs->nwords;
    p.sel_first = fs->first;
    p.sel_last = fs->last;
    p.sel_flags = fs->flags;
  }
  // The launch's work-counter ticket, one sequence shared by every attention
  // kernel (launches on different streams may run at the same time, so each
  // must hold its own slot); bit 31 marks a launch recorded into a CUDA graph
  static std::atomic<uint32_t> eager_tickets{0}, graph_tickets{0};
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) return WISE_ERR_CUDA;
  p.sched_slot = (cap == cudaStreamCaptureStatusActive) ? (0x80000000u | (graph_tickets.fetch_add(1u) & 0x7fffffffu))
                                                        : (eager_tickets.fetch_add(1u) & 0x7fffffffu);
  cudaError_t e;
  switch (s.d) {
    case 64: e = launch_attn_d64(s.bn, sparse, maps, p, stream); break;
    case 96: e = launch_attn_d96(s.bn, sparse, maps, p, stream); break;
    default: e = launch_attn_d128(s.bn, sparse, maps, p, stream); break;
  }
  return e == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int64_t fixed_point(double x) { return llrint(x * 4503599627370496.0); }  // x * 2^52, nearest even

// Fixed scratch of wise_select_support_noalloc: the per-row support bitmasks
// and counts that wise_select_support keeps in its caller's workspace. It is
// part of the library image, so every GPU that loads the library holds these
// bytes until the process exits; calls share it.
constexpr size_t kNoAllocScratchBytes = 2u << 20;
static __device__ __align__(256) uint8_t g_select_scratch[kNoAllocScratchBytes];
uint8_t* g_scratch_ptr[kMaxDevices] = {};

// Device address of g_select_scratch on the current device. The name is only
// a host-side stand-in, so the address is looked up once per device (with that
// device current) and cached.
uint8_t* select_scratch() {
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_select_scratch) != cudaSuccess || p == nullptr) return nullptr;
    g_scratch_ptr[dev] = static_cast<uint8_t*>(p);
  }
  return g_scratch_ptr[dev];
}

// ------------------------------------------------------------- paged cache

constexpr int64_t kMaxCacheTokens = 1ll << 30;  // per sequence

// The shape of a cache; with `pointers`, its buffers too.
int check_cache(const wise_paged_cache* c, bool pointers) {
  if (!c) return WISE_ERR_INVALID_ARGUMENT;
  if (c->batch < 1 || c->kv_heads < 1 || c->max_pages < 1 || c->n_pages < 1) return WISE_ERR_INVALID_ARGUMENT;
  if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128) return WISE_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return WISE_ERR_UNSUPPORTED;
  if (c->batch > 65535 || (int64_t)c->max_pages * c->page > kMaxCacheTokens || c->n_pages > INT32_MAX ||
      (int64_t)c->kv_heads * c->page > INT32_MAX)
    return WISE_ERR_UNSUPPORTED;
  if (!pointers) return WISE_OK;
  if (!c->k_pages || !c->v_pages || !c->page_table || !c->lengths) return WISE_ERR_INVALID_ARGUMENT;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || (reinterpret_cast<uintptr_t>(c->page_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(c->lengths) & 3u))
    return WISE_ERR_ALIGNMENT;
  return WISE_OK;
}

int check_rows(const wise_rows* r) {
  if (!r || !r->data) return WISE_ERR_INVALID_ARGUMENT;
  for (int64_t s : r->stride) {
    if (s < 0) return WISE_ERR_INVALID_ARGUMENT;
    if (s % 8 != 0) return WISE_ERR_ALIGNMENT;  // 16-byte loads
  }
  return aligned16(r->data) ? WISE_OK : WISE_ERR_ALIGNMENT;
}

// Whether [a, a + bytes_a) and [b, b + bytes_b) share memory (a null or empty one: no).
bool overlap(const void* a, int64_t bytes_a, const void* b, int64_t bytes_b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && bytes_a > 0 && bytes_b > 0 && x < y + (uintptr_t)bytes_b && y < x + (uintptr_t)bytes_a;
}

// Whether a dense array shares memory with any of the rows [batch, heads, n, d].
// Rows may lie around it (a slice of a larger buffer), so only where it falls
// between their first and last byte is each run of tokens looked at.
bool overlap_rows(const wise_rows* r, int64_t batch, int64_t heads, int64_t n, int64_t d, const void* out, int64_t bytes) {
  if (!r || !out) return false;
  const uintptr_t first = reinterpret_cast<uintptr_t>(r->data), row = (uintptr_t)d * 2;
  const uintptr_t sb = (uintptr_t)r->stride[0] * 2, sh = (uintptr_t)r->stride[1] * 2, sn = (uintptr_t)r->stride[2] * 2;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(out), hi = lo + (uintptr_t)bytes;
  auto meets = [&](uintptr_t from, uintptr_t last) { return from < hi && lo < last + row; };
  if (!meets(first, first + (batch - 1) * sb + (heads - 1) * sh + (n - 1) * sn)) return false;
  for (int64_t b = 0; b < batch; ++b)
    for (int64_t h = 0; h < heads; ++h) {
      const uintptr_t from = first + b * sb + h * sh;
      if (!meets(from, from + (n - 1) * sn)) continue;
      // the first row that ends past the array's beginning
      const uintptr_t at = sn == 0 || from + row > lo ? from : from + (lo - from - row) / sn * sn + sn;
      if (at < hi) return true;
    }
  return false;
}

int64_t pool_bytes(const wise_paged_cache* c) { return c->n_pages * c->kv_heads * c->page * c->head_dim * 2; }

// Whether a cache's keys and values share memory: calls that write them hand both
// to different threads.
bool pools_meet(const wise_paged_cache* c) { return overlap(c->k_pages, pool_bytes(c), c->v_pages, pool_bytes(c)); }

// Whether an array lies over any part of a cache.
bool overlap_cache(const wise_paged_cache* c, const void* out, int64_t bytes) {
  return overlap(out, bytes, c->k_pages, pool_bytes(c)) || overlap(out, bytes, c->v_pages, pool_bytes(c)) ||
         overlap(out, bytes, c->page_table, (int64_t)c->batch * c->max_pages * 4) ||
         overlap(out, bytes, c->lengths, (int64_t)c->batch * 4);
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

CacheView cache_view(const wise_paged_cache* c) {
  CacheView v;
  v.batch = c->batch;
  v.kv_heads = c->kv_heads;
  v.page_shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  v.max_pages = c->max_pages;
  v.n_pages = c->n_pages;
  v.k_pages = static_cast<uint16_t*>(c->k_pages);
  v.v_pages = static_cast<uint16_t*>(c->v_pages);
  v.page_table = c->page_table;
  v.lengths = c->lengths;
  return v;
}

RowsView rows_view(const wise_rows* r) {
  return RowsView{static_cast<const uint16_t*>(r->data), r->stride[0], r->stride[1], r->stride[2]};
}

// View [n_pages, kv_heads * page, head_dim] of a pool; boxes of one page of one
// head and 64 columns (of 96, the second box lies half outside and is filled
// with zeros there).
int encode_pages(CUtensorMap* m, const void* ptr, const wise_paged_cache* c) {
  auto enc = encoder();
  if (!enc) return WISE_ERR_CUDA;
  const cuuint64_t rows = (cuuint64_t)c->kv_heads * c->page;
  cuuint64_t dims[3] = {(cuuint64_t)c->head_dim, rows, (cuuint64_t)c->n_pages};
  cuuint64_t strides[2] = {(cuuint64_t)c->head_dim * 2, rows * c->head_dim * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)c->page, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? WISE_OK : WISE_ERR_UNSUPPORTED;
}

int check_tree(const wise_paged_cache* c, int32_t heads, int32_t new_tokens) {
  if (heads < 1 || heads % c->kv_heads != 0 || new_tokens < 1) return WISE_ERR_INVALID_ARGUMENT;
  if (new_tokens > kTreeMaxTokens || heads / c->kv_heads > 4096) return WISE_ERR_UNSUPPORTED;
  if ((int64_t)c->batch * heads * new_tokens > INT32_MAX / 2) return WISE_ERR_UNSUPPORTED;
  // key tiles of all units
  const int64_t pairs = ((int64_t)(heads / c->kv_heads) * new_tokens + 255) / 256;
  const int64_t tiles = ((int64_t)c->max_pages * c->page + 127) / 128 + kTreeOverhead;
  if (c->kv_heads > INT32_MAX / c->batch || (int64_t)c->batch * c->kv_heads * pairs > INT32_MAX / tiles)
    return WISE_ERR_UNSUPPORTED;
  return WISE_OK;
}

// Self-check of the bounded wait: one thread waits on an mbarrier that
// nothing arrives on, through the same wait routine as the attention kernels
// but with a 20 ms limit. The wait expires, kErrTimeout is recorded, and the
// kernel returns (no copy or MMA is in flight, so nothing needs draining).
constexpr uint64_t kSelfCheckWaitNs = 20000000ull;
__global__ void wait_expiry_kernel(uint32_t* err) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x != 0) return;
  mbar_init(&bar, 1);
  abort_flag = 0;
  fence_mbar_init();
  mbar_wait<6, kSelfCheckWaitNs>(&bar, 0, &abort_flag, err);
}

}  // namespace
}  // namespace wise

using namespace wise;

extern "C" {

int wise_abi_version(void) { return WISE_ABI_VERSION; }

const char* wise_status_str(int status) {
  switch (status) {
    case WISE_OK: return "ok";
    case WISE_ERR_INVALID_ARGUMENT: return "invalid argument";
    case WISE_ERR_UNSUPPORTED: return "unsupported shape or configuration";
    case WISE_ERR_ALIGNMENT: return "tensor base address not 16-byte aligned";
    case WISE_ERR_WORKSPACE: return "workspace missing or too small";
    case WISE_ERR_BAD_SUPPORT: return "malformed support (CSR) or schedule";
    case WISE_ERR_CUDA: return "CUDA error";
    case WISE_ERR_DEVICE_TIMEOUT: return "device wait timed out";
    case WISE_ERR_BAD_CACHE: return "invalid entries in a paged cache or an accepted path";
    default: return "unknown status";
  }
}

size_t wise_attn_discover_workspace(const wise_attn_desc* desc) {
  if (check_desc(desc) != WISE_OK) return 0;
  return lam_bytes(shape_of(desc));
}

int64_t wise_schedule_units(const wise_attn_desc* desc) {
  if (check_desc(desc) != WISE_OK) return 0;
  return shape_of(desc).n_units;
}

int64_t wise_support_capacity(const wise_attn_desc* desc) {
  if (check_desc(desc) != WISE_OK) return 0;
  const Shape s = shape_of(desc);
  return s.bh * (int64_t)s.nb * (s.nb + 1) / 2;
}

size_t wise_select_workspace(const wise_attn_desc* desc, int32_t window) {
  if (check_desc(desc) != WISE_OK || window < 1 || window > 8) return 0;
  const Shape s = shape_of(desc);
  const int64_t rows = s.bh * s.nb;
  const int64_t words = (s.nb + 31) / 32;
  return (size_t)(select_lookback_offset(rows, words) + select_lookback_bytes(rows) + 256);
}

int wise_attn_discover(const wise_attn_desc* desc, const void* q, const void* k, const void* v, void* o, float* lse,
                       float* block_mass, void* workspace, size_t workspace_bytes, wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!q || !k || !v || !o) return WISE_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return WISE_ERR_ALIGNMENT;
  if ((lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) || (block_mass && (reinterpret_cast<uintptr_t>(block_mass) & 3u)))
    return WISE_ERR_ALIGNMENT;
  if (block_mass) {
    const size_t need = lam_bytes(shape_of(desc));
    if (!workspace || workspace_bytes < need) return WISE_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return WISE_ERR_ALIGNMENT;
  }
  return launch_attention(desc, q, k, v, o, lse, block_mass, workspace, nullptr, nullptr, 0, nullptr, false,
                          reinterpret_cast<cudaStream_t>(stream));
}

int wise_attn_sparse(const wise_attn_desc* desc, const void* q, const void* k, const void* v, const int32_t* row_ptr,
                     const int32_t* col_idx, int64_t col_capacity, const int32_t* tile_order, void* o, float* lse,
                     wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!q || !k || !v || !o || !row_ptr || !col_idx || col_capacity < 0) return WISE_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return WISE_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(row_ptr) & 3u) || (reinterpret_cast<uintptr_t>(col_idx) & 3u) ||
      (tile_order && (reinterpret_cast<uintptr_t>(tile_order) & 3u)) ||
      (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return WISE_ERR_ALIGNMENT;
  return launch_attention(desc, q, k, v, o, lse, nullptr, nullptr, row_ptr, col_idx, col_capacity, tile_order, true,
                          reinterpret_cast<cudaStream_t>(stream));
}

int wise_attn_sparse_planned(const wise_attn_desc* desc, const void* q, const void* k, const void* v,
                             const int32_t* row_ptr, const int32_t* col_idx, int64_t col_capacity,
                             const int32_t* tile_order, const void* plan, void* o, float* lse,
                             wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!q || !k || !v || !o || !row_ptr || !col_idx || col_capacity < 0) return WISE_ERR_INVALID_ARGUMENT;
  if (plan && desc->block != 32) return WISE_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || (plan && !aligned16(plan)))
    return WISE_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(row_ptr) & 3u) || (reinterpret_cast<uintptr_t>(col_idx) & 3u) ||
      (tile_order && (reinterpret_cast<uintptr_t>(tile_order) & 3u)) ||
      (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return WISE_ERR_ALIGNMENT;
  return launch_attention(desc, q, k, v, o, lse, nullptr, nullptr, row_ptr, col_idx, col_capacity, tile_order, true,
                          reinterpret_cast<cudaStream_t>(stream), nullptr, plan);
}

size_t wise_gather_plan_bytes(const wise_attn_desc* desc) {
  if (check_desc(desc) != WISE_OK || desc->block != 32) return 0;
  const Shape s = shape_of(desc);
  return (size_t)plan_bytes(s.bh, s.n_qtiles);
}

int wise_gather_plan(const wise_attn_desc* desc, const int32_t* row_ptr, const int32_t* col_idx,
                     int64_t col_capacity, void* plan, size_t plan_bytes_given, wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (desc->block != 32) return WISE_ERR_UNSUPPORTED;
  if (!row_ptr || !col_idx || !plan || col_capacity < 0) return WISE_ERR_INVALID_ARGUMENT;
  if (plan_bytes_given < wise_gather_plan_bytes(desc)) return WISE_ERR_WORKSPACE;
  if (!aligned16(plan) || (reinterpret_cast<uintptr_t>(row_ptr) & 3u) || (reinterpret_cast<uintptr_t>(col_idx) & 3u))
    return WISE_ERR_ALIGNMENT;
  uint32_t* err = error_word();
  if (!err) return WISE_ERR_CUDA;
  const Shape s = shape_of(desc);
  GatherPlanLaunch g;
  g.row_ptr = row_ptr;
  g.col_idx = col_idx;
  g.col_cap = col_capacity;
  g.bh_count = (int32_t)s.bh;
  g.nb = s.nb;
  g.n_qtiles = s.n_qtiles;
  g.counts = static_cast<int32_t*>(plan);
  g.entries = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(plan) + plan_counts_bytes(s.n_units));
  g.err = err;
  return launch_gather_plan(g, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int wise_select_support(const wise_attn_desc* desc, const float* block_mass, int32_t window, double eta,
                        uint32_t flags, int32_t* row_ptr, int32_t* col_idx, int64_t col_capacity, int32_t* tile_order,
                        int32_t* nnz, void* workspace, size_t workspace_bytes, wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!block_mass || !row_ptr || !col_idx) return WISE_ERR_INVALID_ARGUMENT;
  if (window < 1 || window > 8 || !(eta > 0.0 && eta < 1.0) || (flags & ~3u)) return WISE_ERR_INVALID_ARGUMENT;
  if (col_capacity < wise_support_capacity(desc)) return WISE_ERR_BAD_SUPPORT;
  const size_t need = wise_select_workspace(desc, window);
  if (!workspace || workspace_bytes < need) return WISE_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 15u) || (reinterpret_cast<uintptr_t>(block_mass) & 3u) ||
      (reinterpret_cast<uintptr_t>(row_ptr) & 3u) || (reinterpret_cast<uintptr_t>(col_idx) & 3u))
    return WISE_ERR_ALIGNMENT;
  uint32_t* err = error_word();
  if (!err) return WISE_ERR_CUDA;
  const Shape s = shape_of(desc);
  const int64_t rows = s.bh * s.nb;
  const int64_t words = (s.nb + 31) / 32;
  SelectLaunch sl;
  memset(&sl, 0, sizeof(sl));
  sl.mass = block_mass;
  sl.window = window;
  sl.bh_count = (int32_t)s.bh;
  sl.nb = s.nb;
  sl.target_fx = fixed_point(eta);
  sl.tol_fx = fixed_point(1e-6);
  sl.flags = flags;
  sl.bits = static_cast<uint32_t*>(workspace);
  sl.counts = reinterpret_cast<int32_t*>(static_cast<uint32_t*>(workspace) + rows * words);
  sl.row_ptr = row_ptr;
  sl.col_idx = col_idx;
  sl.col_cap = col_capacity;
  sl.nnz = nnz;
  sl.tile_order = tile_order;
  sl.units_per_bh = s.n_qtiles;
  sl.qb_per_unit = 128 / s.bn;
  sl.err = err;
  cudaError_t e = launch_select(sl, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

// Largest nb of the fused selection (eight 32-block rounds per row in the
// epilogue warps' registers).
constexpr int kFusedSelectMaxBlocks = 256;

int wise_attn_discover_select(const wise_attn_desc* desc, const void* q, const void* k, const void* v, void* o,
                              float* lse, float* block_mass, void* workspace, size_t workspace_bytes, double eta,
                              uint32_t flags, int32_t step, int32_t window, void* select_state,
                              size_t select_state_bytes, wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!q || !k || !v || !o || !block_mass || !select_state) return WISE_ERR_INVALID_ARGUMENT;
  if (window < 1 || window > 8 || step < 0 || step >= window || !(eta > 0.0 && eta < 1.0) || (flags & ~3u))
    return WISE_ERR_INVALID_ARGUMENT;
  const Shape s = shape_of(desc);
  if (s.nb > kFusedSelectMaxBlocks) return WISE_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return WISE_ERR_ALIGNMENT;
  if ((lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) || (reinterpret_cast<uintptr_t>(block_mass) & 3u) ||
      (reinterpret_cast<uintptr_t>(select_state) & 15u))
    return WISE_ERR_ALIGNMENT;
  const size_t need = lam_bytes(s);
  if (!workspace || workspace_bytes < need) return WISE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return WISE_ERR_ALIGNMENT;
  if (select_state_bytes < wise_select_workspace(desc, window)) return WISE_ERR_WORKSPACE;
  const int64_t rows = s.bh * s.nb;
  const int64_t words = (s.nb + 31) / 32;
  FusedSelect fs;
  fs.bits = static_cast<uint32_t*>(select_state);
  fs.counts = reinterpret_cast<int32_t*>(static_cast<uint32_t*>(select_state) + rows * words);
  fs.target_fx = fixed_point(eta);
  fs.tol_fx = fixed_point(1e-6);
  fs.nwords = (int32_t)words;
  fs.first = step == 0;
  fs.last = step == window - 1;
  fs.flags = flags;
  return launch_attention(desc, q, k, v, o, lse, block_mass, workspace, nullptr, nullptr, 0, nullptr, false,
                          reinterpret_cast<cudaStream_t>(stream), &fs);
}

int wise_select_finalize(const wise_attn_desc* desc, const void* select_state, size_t select_state_bytes,
                         int32_t* row_ptr, int32_t* col_idx, int64_t col_capacity, int32_t* tile_order, int32_t* nnz,
                         wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!select_state || !row_ptr || !col_idx) return WISE_ERR_INVALID_ARGUMENT;
  if (col_capacity < wise_support_capacity(desc)) return WISE_ERR_BAD_SUPPORT;
  if (select_state_bytes < wise_select_workspace(desc, 1)) return WISE_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(select_state) & 15u) || (reinterpret_cast<uintptr_t>(row_ptr) & 3u) ||
      (reinterpret_cast<uintptr_t>(col_idx) & 3u) || (tile_order && (reinterpret_cast<uintptr_t>(tile_order) & 3u)) ||
      (nnz && (reinterpret_cast<uintptr_t>(nnz) & 3u)))
    return WISE_ERR_ALIGNMENT;
  uint32_t* err = error_word();
  if (!err) return WISE_ERR_CUDA;
  const Shape s = shape_of(desc);
  const int64_t rows = s.bh * s.nb;
  const int64_t words = (s.nb + 31) / 32;
  SelectLaunch sl;
  memset(&sl, 0, sizeof(sl));
  sl.window = 1;
  sl.bh_count = (int32_t)s.bh;
  sl.nb = s.nb;
  sl.bits = const_cast<uint32_t*>(static_cast<const uint32_t*>(select_state));
  sl.counts = reinterpret_cast<int32_t*>(sl.bits + rows * words);
  sl.row_ptr = row_ptr;
  sl.col_idx = col_idx;
  sl.col_cap = col_capacity;
  sl.nnz = nnz;
  sl.tile_order = tile_order;
  sl.units_per_bh = s.n_qtiles;
  sl.qb_per_unit = 128 / s.bn;
  sl.finalize_only = 1;
  sl.err = err;
  cudaError_t e = launch_select(sl, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int wise_select_support_noalloc(const wise_attn_desc* desc, const float* block_mass, int32_t window, double eta,
                                uint32_t flags, int32_t* row_ptr, int32_t* col_idx, int64_t col_capacity,
                                int32_t* tile_order, int32_t* nnz, wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!block_mass || !row_ptr || !col_idx) return WISE_ERR_INVALID_ARGUMENT;
  if (window < 1 || window > 8 || !(eta > 0.0 && eta < 1.0) || (flags & ~3u)) return WISE_ERR_INVALID_ARGUMENT;
  if (col_capacity < wise_support_capacity(desc)) return WISE_ERR_BAD_SUPPORT;
  if (wise_select_workspace(desc, window) > kNoAllocScratchBytes) return WISE_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(block_mass) & 3u) || (reinterpret_cast<uintptr_t>(row_ptr) & 3u) ||
      (reinterpret_cast<uintptr_t>(col_idx) & 3u))
    return WISE_ERR_ALIGNMENT;
  uint32_t* err = error_word();
  uint8_t* scratch = select_scratch();
  if (!err || !scratch) return WISE_ERR_CUDA;
  const Shape s = shape_of(desc);
  const int64_t rows = s.bh * s.nb;
  const int64_t words = (s.nb + 31) / 32;
  SelectLaunch sl;
  memset(&sl, 0, sizeof(sl));
  sl.mass = block_mass;
  sl.window = window;
  sl.bh_count = (int32_t)s.bh;
  sl.nb = s.nb;
  sl.target_fx = fixed_point(eta);
  sl.tol_fx = fixed_point(1e-6);
  sl.flags = flags;
  // every row writes its bitmask words and its count before they are read,
  // so the shared scratch needs no clearing between calls
  sl.bits = reinterpret_cast<uint32_t*>(scratch);
  sl.counts = reinterpret_cast<int32_t*>(scratch + rows * words * 4);
  sl.row_ptr = row_ptr;
  sl.col_idx = col_idx;
  sl.col_cap = col_capacity;
  sl.nnz = nnz;
  sl.tile_order = tile_order;
  sl.units_per_bh = s.n_qtiles;
  sl.qb_per_unit = 128 / s.bn;
  sl.err = err;
  cudaError_t e = launch_select(sl, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int wise_support_retained_mass(const wise_attn_desc* desc, const float* block_mass, const int32_t* row_ptr,
                                const int32_t* col_idx, int64_t col_capacity, float* row_retained, double* batch_mean,
                                wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!block_mass || !row_ptr || !col_idx || !row_retained || col_capacity < 0) return WISE_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(block_mass) & 3u) || (reinterpret_cast<uintptr_t>(row_ptr) & 3u) ||
      (reinterpret_cast<uintptr_t>(col_idx) & 3u) || (reinterpret_cast<uintptr_t>(row_retained) & 3u) ||
      (batch_mean && (reinterpret_cast<uintptr_t>(batch_mean) & 7u)))
    return WISE_ERR_ALIGNMENT;
  uint32_t* err = error_word();
  if (!err) return WISE_ERR_CUDA;
  const Shape s = shape_of(desc);
  DiagLaunch d;
  memset(&d, 0, sizeof(d));
  d.rows = s.bh * s.nb;
  d.nb = s.nb;
  d.batch = desc->batch;
  d.col_cap = col_capacity;
  d.mass = block_mass;
  d.row_ptr_a = row_ptr;
  d.col_idx_a = col_idx;
  d.row_value = row_retained;
  d.batch_value = batch_mean;
  d.err = err;
  return launch_retained_mass(d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int wise_support_jaccard(const wise_attn_desc* desc, const int32_t* row_ptr_a, const int32_t* col_idx_a,
                         int64_t col_capacity_a, const int32_t* row_ptr_b, const int32_t* col_idx_b,
                         int64_t col_capacity_b, int32_t* row_counts, int64_t* batch_counts, double* batch_jaccard,
                         wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!row_ptr_a || !col_idx_a || !row_ptr_b || !col_idx_b || !row_counts || col_capacity_a < 0 ||
      col_capacity_b < 0)
    return WISE_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(row_ptr_a) & 3u) || (reinterpret_cast<uintptr_t>(col_idx_a) & 3u) ||
      (reinterpret_cast<uintptr_t>(row_ptr_b) & 3u) || (reinterpret_cast<uintptr_t>(col_idx_b) & 3u) ||
      (reinterpret_cast<uintptr_t>(row_counts) & 3u) || (batch_counts && (reinterpret_cast<uintptr_t>(batch_counts) & 7u)) ||
      (batch_jaccard && (reinterpret_cast<uintptr_t>(batch_jaccard) & 7u)))
    return WISE_ERR_ALIGNMENT;
  uint32_t* err = error_word();
  if (!err) return WISE_ERR_CUDA;
  const Shape s = shape_of(desc);
  DiagLaunch d;
  memset(&d, 0, sizeof(d));
  d.rows = s.bh * s.nb;
  d.nb = s.nb;
  d.batch = desc->batch;
  d.col_cap = col_capacity_a;
  d.col_cap_b = col_capacity_b;
  d.row_ptr_a = row_ptr_a;
  d.col_idx_a = col_idx_a;
  d.row_ptr_b = row_ptr_b;
  d.col_idx_b = col_idx_b;
  d.row_counts = row_counts;
  d.batch_counts = reinterpret_cast<long long*>(batch_counts);
  d.batch_value = batch_jaccard;
  d.err = err;
  return launch_jaccard(d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int wise_select_control(const wise_attn_desc* desc, const float* block_mass, int32_t mode,
                        const int32_t* ref_row_ptr, const int32_t* ref_col_idx, int64_t ref_capacity, uint32_t flags,
                        int32_t* row_ptr, int32_t* col_idx, int64_t col_capacity, int32_t* tile_order, int32_t* nnz,
                        void* workspace, size_t workspace_bytes, wise_stream_t stream) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (mode != WISE_CONTROL_MASS_MATCHED && mode != WISE_CONTROL_SIZE_MATCHED) return WISE_ERR_INVALID_ARGUMENT;
  if (!block_mass || !ref_row_ptr || !ref_col_idx || !row_ptr || !col_idx || ref_capacity < 0 || (flags & ~3u))
    return WISE_ERR_INVALID_ARGUMENT;
  if (col_capacity < wise_support_capacity(desc)) return WISE_ERR_BAD_SUPPORT;
  const size_t need = wise_select_workspace(desc, 1);
  if (!workspace || workspace_bytes < need) return WISE_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 15u) || (reinterpret_cast<uintptr_t>(block_mass) & 3u) ||
      (reinterpret_cast<uintptr_t>(row_ptr) & 3u) || (reinterpret_cast<uintptr_t>(col_idx) & 3u) ||
      (reinterpret_cast<uintptr_t>(ref_row_ptr) & 3u) || (reinterpret_cast<uintptr_t>(ref_col_idx) & 3u))
    return WISE_ERR_ALIGNMENT;
  uint32_t* err = error_word();
  if (!err) return WISE_ERR_CUDA;
  const Shape s = shape_of(desc);
  const int64_t rows = s.bh * s.nb;
  const int64_t words = (s.nb + 31) / 32;
  SelectLaunch sl;
  memset(&sl, 0, sizeof(sl));
  sl.mass = block_mass;
  sl.window = 1;
  sl.bh_count = (int32_t)s.bh;
  sl.nb = s.nb;
  sl.target_fx = 0;
  sl.tol_fx = fixed_point(1e-6);
  sl.flags = flags;
  sl.bits = static_cast<uint32_t*>(workspace);
  sl.counts = reinterpret_cast<int32_t*>(static_cast<uint32_t*>(workspace) + rows * words);
  sl.row_ptr = row_ptr;
  sl.col_idx = col_idx;
  sl.col_cap = col_capacity;
  sl.nnz = nnz;
  sl.tile_order = tile_order;
  sl.units_per_bh = s.n_qtiles;
  sl.qb_per_unit = 128 / s.bn;
  sl.mode = mode;
  sl.ref_row_ptr = ref_row_ptr;
  sl.ref_col_idx = ref_col_idx;
  sl.ref_cap = ref_capacity;
  sl.err = err;
  cudaError_t e = launch_select(sl, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int wise_cache_append(const wise_paged_cache* cache, int32_t new_tokens, const wise_rows* k, const wise_rows* v,
                      int32_t heads, const wise_rows* q, void* q_out, const int32_t* new_len,
                      const int32_t* positions, const int64_t* rope, int32_t rotary_dim, uint32_t flags,
                      wise_stream_t stream) {
  int st = check_cache(cache, true);
  if (st != WISE_OK) return st;
  if (new_tokens < 1 || (q && (heads < 1 || !q_out)) || (flags & ~WISE_ROPE_PAIRS)) return WISE_ERR_INVALID_ARGUMENT;
  if (rotary_dim < 0 || rotary_dim > cache->head_dim || rotary_dim % 16 != 0) return WISE_ERR_INVALID_ARGUMENT;
  if (rotary_dim > 0 && !rope) return WISE_ERR_INVALID_ARGUMENT;
  if (new_tokens > kMaxCacheTokens || (int64_t)cache->batch * new_tokens > INT32_MAX ||
      2 * (int64_t)cache->kv_heads + (q ? heads : 0) > INT32_MAX)
    return WISE_ERR_UNSUPPORTED;
  if ((st = check_rows(k)) != WISE_OK || (st = check_rows(v)) != WISE_OK) return st;
  if (q && (st = check_rows(q)) != WISE_OK) return st;
  if ((q && !aligned16(q_out)) || misaligned4(new_len) || misaligned4(positions) ||
      (reinterpret_cast<uintptr_t>(rope) & 7u))
    return WISE_ERR_ALIGNMENT;
  if (pools_meet(cache)) return WISE_ERR_INVALID_ARGUMENT;
  if (q) {
    // threads write rows of q_out while others still read
    const int64_t batch = cache->batch, d = cache->head_dim, bytes = batch * heads * new_tokens * d * 2;
    if (overlap_cache(cache, q_out, bytes) || overlap_rows(q, batch, heads, new_tokens, d, q_out, bytes) ||
        overlap_rows(k, batch, cache->kv_heads, new_tokens, d, q_out, bytes) ||
        overlap_rows(v, batch, cache->kv_heads, new_tokens, d, q_out, bytes) ||
        overlap(q_out, bytes, new_len, batch * 4) || overlap(q_out, bytes, positions, batch * new_tokens * 4) ||
        overlap(q_out, bytes, rope, (int64_t)rotary_dim / 2 * 8))
      return WISE_ERR_INVALID_ARGUMENT;
  }
  AppendLaunch a;
  memset(&a, 0, sizeof(a));
  a.err = error_word();
  if (!a.err) return WISE_ERR_CUDA;
  a.cache = cache_view(cache);
  a.head_dim = cache->head_dim;
  a.n = new_tokens;
  a.k = rows_view(k);
  a.v = rows_view(v);
  if (q) {
    a.q = rows_view(q);
    a.heads = heads;
    a.q_out = static_cast<uint16_t*>(q_out);
  }
  a.new_len = new_len;
  a.positions = positions;
  a.rope = rope;
  a.rotary_dim = rotary_dim;
  a.pairs = (flags & WISE_ROPE_PAIRS) != 0;
  return launch_cache_append(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

size_t wise_attn_tree_workspace(const wise_paged_cache* cache, int32_t heads, int32_t new_tokens) {
  if (check_cache(cache, false) != WISE_OK || check_tree(cache, heads, new_tokens) != WISE_OK) return 0;
  return (size_t)tree_workspace_bytes(cache->batch, cache->kv_heads, heads, new_tokens, cache->head_dim);
}

int wise_attn_tree(const wise_paged_cache* cache, int32_t heads, int32_t new_tokens, const wise_rows* q,
                   const int32_t* new_len, const int32_t* tree_mask, float scale, int32_t out_dtype, void* o,
                   float* lse, void* workspace, size_t workspace_bytes, wise_stream_t stream) {
  int st = check_cache(cache, true);
  if (st != WISE_OK) return st;
  if ((st = check_tree(cache, heads, new_tokens)) != WISE_OK) return st;
  if (!o || (out_dtype != WISE_BF16 && out_dtype != WISE_F32) || !(scale >= 0.f) || isinf(scale))
    return WISE_ERR_INVALID_ARGUMENT;
  if ((st = check_rows(q)) != WISE_OK) return st;
  if (!aligned16(o) || misaligned4(lse) || misaligned4(new_len) || misaligned4(tree_mask)) return WISE_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < wise_attn_tree_workspace(cache, heads, new_tokens)) return WISE_ERR_WORKSPACE;
  if (!aligned16(workspace)) return WISE_ERR_ALIGNMENT;
  {
    // results and partial results are written while other blocks still read
    const int64_t batch = cache->batch, d = cache->head_dim, n = new_tokens, rows = batch * heads * n;
    const struct {
      const void* at;
      int64_t bytes;
    } outs[3] = {{o, rows * d * (out_dtype == WISE_F32 ? 4 : 2)},
                 {lse, rows * 4},
                 {workspace, (int64_t)wise_attn_tree_workspace(cache, heads, new_tokens)}};
    for (int i = 0; i < 3; ++i) {
      const void* at = outs[i].at;
      const int64_t bytes = outs[i].bytes;
      if (overlap_cache(cache, at, bytes) || overlap_rows(q, batch, heads, n, d, at, bytes) ||
          overlap(at, bytes, new_len, batch * 4) || overlap(at, bytes, tree_mask, batch * n * ((n + 31) / 32) * 4) ||
          overlap(at, bytes, outs[(i + 1) % 3].at, outs[(i + 1) % 3].bytes))
        return WISE_ERR_INVALID_ARGUMENT;
    }
  }
  TreeLaunch t;
  memset(&t, 0, sizeof(t));
  t.err = error_word();
  if (!t.err) return WISE_ERR_CUDA;
  t.cache = cache_view(cache);
  t.head_dim = cache->head_dim;
  t.heads = heads;
  t.n = new_tokens;
  t.q = rows_view(q);
  t.new_len = new_len;
  t.tree_mask = tree_mask;
  t.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)cache->head_dim);
  t.out_f32 = out_dtype == WISE_F32;
  t.o = o;
  t.lse = lse;
  t.workspace = workspace;
  CUtensorMap maps[2];
  st = encode_pages(&maps[0], cache->k_pages, cache);
  if (st == WISE_OK) st = encode_pages(&maps[1], cache->v_pages, cache);
  if (st != WISE_OK) return st;
  return launch_tree(t, maps, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int wise_cache_accept(const wise_paged_cache* cache, int32_t path_tokens, const int32_t* path,
                      const int32_t* n_accepted, int32_t* new_lengths, wise_stream_t stream) {
  int st = check_cache(cache, true);
  if (st != WISE_OK) return st;
  if (!n_accepted || !new_lengths || path_tokens < 1 || path_tokens > kMaxCacheTokens) return WISE_ERR_INVALID_ARGUMENT;
  if (misaligned4(path) || misaligned4(n_accepted) || misaligned4(new_lengths)) return WISE_ERR_ALIGNMENT;
  // a block may read its inputs after another has written new_lengths[b]
  const int64_t batch = cache->batch;
  if (overlap_cache(cache, new_lengths, batch * 4) || overlap(new_lengths, batch * 4, n_accepted, batch * 4) ||
      overlap(new_lengths, batch * 4, path, batch * path_tokens * 4) || (path && pools_meet(cache)))
    return WISE_ERR_INVALID_ARGUMENT;
  AcceptLaunch a;
  memset(&a, 0, sizeof(a));
  a.err = error_word();
  if (!a.err) return WISE_ERR_CUDA;
  a.cache = cache_view(cache);
  a.head_dim = cache->head_dim;
  a.path_tokens = path_tokens;
  a.path = path;
  a.n_accepted = n_accepted;
  a.new_lengths = new_lengths;
  return launch_cache_accept(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int wise_validate_support(const wise_attn_desc* desc, const int32_t* row_ptr, const int32_t* col_idx,
                          uint32_t flags) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!row_ptr || (!col_idx && row_ptr[0] != 0)) return WISE_ERR_INVALID_ARGUMENT;
  const Shape s = shape_of(desc);
  const int64_t rows = s.bh * s.nb;
  if (row_ptr[0] != 0) return WISE_ERR_BAD_SUPPORT;
  for (int64_t r = 0; r < rows; ++r) {
    const int32_t a = row_ptr[r], b = row_ptr[r + 1];
    if (b < a) return WISE_ERR_BAD_SUPPORT;
    const int q = (int)(r % s.nb);
    int prev = -1;
    bool has0 = false, hasq = false;
    for (int32_t j = a; j < b; ++j) {
      const int32_t c = col_idx[j];
      if (c <= prev || c > q) return WISE_ERR_BAD_SUPPORT;
      has0 |= (c == 0);
      hasq |= (c == q);
      prev = c;
    }
    if (((flags & WISE_SUPPORT_SINK) && !has0) || ((flags & WISE_SUPPORT_DIAG) && !hasq)) return WISE_ERR_BAD_SUPPORT;
  }
  return WISE_OK;
}

int wise_validate_schedule(const wise_attn_desc* desc, const int32_t* tile_order) {
  int st = check_desc(desc);
  if (st != WISE_OK) return st;
  if (!tile_order) return WISE_ERR_INVALID_ARGUMENT;
  const int64_t units = shape_of(desc).n_units;
  std::vector<uint8_t> seen((size_t)units, 0);
  for (int64_t x = 0; x < units; ++x) {
    const int32_t u = tile_order[x];
    if (u < 0 || u >= units || seen[(size_t)u]) return WISE_ERR_BAD_SUPPORT;
    seen[(size_t)u] = 1;
  }
  return WISE_OK;
}

int wise_wait_expiry_check(wise_stream_t stream) {
  uint32_t* err = error_word();
  if (!err) return WISE_ERR_CUDA;
  wait_expiry_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(err);
  return cudaGetLastError() == cudaSuccess ? WISE_OK : WISE_ERR_CUDA;
}

int wise_device_status(wise_stream_t stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return WISE_ERR_CUDA;
  uint32_t word = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&word, g_wise_error_word, sizeof(word)) != cudaSuccess) return WISE_ERR_CUDA;
  if (word && cudaMemcpyToSymbol(g_wise_error_word, &zero, sizeof(zero)) != cudaSuccess) return WISE_ERR_CUDA;
  if (word & kErrTimeout) return WISE_ERR_DEVICE_TIMEOUT;
  if (word & kErrInternal) return WISE_ERR_CUDA;
  if (word & kErrBadSupport) return WISE_ERR_BAD_SUPPORT;
  if (word & kErrBadCache) return WISE_ERR_BAD_CACHE;
  return WISE_OK;
}

}  // extern "C"
