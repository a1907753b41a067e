// Eviction from a paged cache: of a sequence longer than `budget` each key head
// keeps its first `sink` tokens, its last `recent` ones and, of those between,
// the heaviest (ties: the lowest place); kept tokens go, in their order, to the
// slots 0, 1, ... of other pages.
//
// Two launches: the selection writes each head's list of kept places, the move
// copies their rows. Measured (one GB300): 16 sequences of up to 8K, 8 key heads of
// 128, cut to 4K (474 MB): 86.8 us, 14 of them the selection and 70 the move, which
// runs at a copy's rate; one of 32K cut to 2K: 17.4 us, 12 the selection (eight blocks
// a head; 21.3 us when each block summed all 2048 counts of all eight). Weights that are
// mostly equal count into few words of shared memory, which costs little: a prompt of
// 32K with all weights 0 or all 1 17.9 us, with nine of ten 0 15.6, spread 15.6 to
// 17.9; 40 sequences of 32K cut to 2K (one block a head) 208, 202, 204 us.
#include <cooperative_groups.h>

#include "internal.h"
#include "ptx.cuh"

namespace wise {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 16;  // weights a thread keeps in registers

// Weights as whole numbers in the same order; NaN below everything, -0 = 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

// Committed tokens of sequence b, clamped to what the page table and the row of
// weights hold.
__device__ __forceinline__ int evict_length(const EvictLaunch& e, int b, bool flag) {
  const int64_t cap = (int64_t)e.cache.max_pages << e.cache.page_shift;
  const int64_t most = cap < e.width ? cap : e.width;
  const int64_t l = e.cache.lengths[b];
  if ((l < 0 || l > most) && flag) atomicOr(e.err, kErrBadCache);
  return (int)(l < 0 ? 0 : l > most ? most : l);
}

__device__ __forceinline__ uint32_t inclusive_sum(uint32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += v;
  }
  return x;
}

// A cluster of C blocks per (sequence, key head); block r holds the r-th part of
// the places that compete, each of its warps consecutive ones. The weight that
// the last kept place has is found from the top, 11, 11 and 10 bits at a time:
// each block counts its weights by those bits in shared memory, and one warp of each
// sums the counts of all, first of 64 bins together, then of the 64 that matter.
template <int C>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictLaunch e) {
  __shared__ uint32_t hist[3][2048], coarse[3][kSelWarps];
  __shared__ uint32_t found[3];
  __shared__ uint32_t greater[kSelWarps], equal[kSelWarps];
  __shared__ uint2 totals[C];  // of each block of the cluster: weights above the cut, weights at it
  grid_wait();
  grid_trigger();
  auto cluster = cg::this_cluster();
  const int rank = C == 1 ? 0 : (int)cluster.block_rank();
  const int64_t unit = blockIdx.x / C;
  const int b = (int)(unit / e.cache.kv_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = evict_length(e, b, tid == 0);
  const int keep = min(len, e.budget);
  if (unit % e.cache.kv_heads == 0 && rank == 0 && tid == 0) e.new_lengths[b] = keep;
  int32_t* list = e.list + unit * e.list_width;
  const float* w = e.weights + unit * e.width;
  if (len <= e.budget) {  // everything stays (the whole cluster leaves)
    for (int i = rank * kSelThreads + tid; i < len; i += C * kSelThreads) list[i] = i;
    return;
  }
  const int lo = e.sink, hi = len - e.recent, want = e.budget - e.sink - e.recent;
  for (int i = rank * kSelThreads + tid; i < e.sink; i += C * kSelThreads) list[i] = i;
  for (int i = rank * kSelThreads + tid; i < e.recent; i += C * kSelThreads) list[e.budget - e.recent + i] = hi + i;
  if (want == 0) return;
  // this warp's places: [at, at + seg), those below hi
  const int seg = (int)(((int64_t)hi - lo + C * kSelThreads - 1) / (C * kSelThreads)) * 32;
  const int64_t at = lo + (int64_t)(rank * kSelWarps + warp) * seg;
  const int count = (int)max((int64_t)0, min((int64_t)seg, hi - at));
  uint32_t keys[kSelKeys];
#pragma unroll
  for (int j = 0; j < kSelKeys; ++j) keys[j] = j * 32 + lane < count ? order_key(w[at + j * 32 + lane]) : 0u;
  // f(key, whether there is one) for 32 places at a time, in order
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < kSelKeys; ++j)
      if (j * 32 < count) f(j, keys[j], j * 32 + lane < count);
    for (int j = kSelKeys; j * 32 < count; ++j) {
      const bool in = j * 32 + lane < count;
      f(j, in ? order_key(w[at + j * 32 + lane]) : 0u, in);
    }
  };
  for (int i = tid; i < 3 * 2048; i += kSelThreads) (&hist[0][0])[i] = 0u;
  __syncthreads();
  uint32_t cut = 0u;           // the bits found so far
  uint32_t left = (uint32_t)want;  // places to take among the weights that begin with them
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int above = pass == 0 ? 32 : pass == 1 ? 21 : 10;  // bits from here on are found
    uint32_t* h = hist[pass];
    each([&](int, uint32_t key, bool in) {
      if (in && (pass == 0 || (key >> above) == (cut >> above))) atomicAdd(&h[(key >> shift) & 2047u], 1u);
    });
    // sums of 64 bins, a warp each; then, by one warp, the 64 bins in which the last
    // place lies, and the bin among them, both over the counts of all blocks
    __syncthreads();
    const uint2 x = *reinterpret_cast<const uint2*>(h + 64 * warp + 2 * lane);
    const uint32_t x64 = __reduce_add_sync(0xffffffffu, x.x + x.y);
    if (lane == 0) coarse[pass][warp] = x64;
    if (C == 1) __syncthreads();
    else cluster.sync();
    if (warp == 0) {
      // from the highest on: lane l has sums 31 - l, then bins 63 - 2l and 62 - 2l
      uint32_t n = 0u;
#pragma unroll
      for (int r = 0; r < C; ++r) n += (C == 1 ? coarse[pass] : cluster.map_shared_rank(coarse[pass], r))[31 - lane];
      uint32_t before = inclusive_sum(n, lane) - n;
      const uint32_t at = __ballot_sync(0xffffffffu, before < left && left <= before + n);
      const int c = 31 - (__ffs(at) - 1);  // (there is one: `left` places are left)
      const uint32_t rest = left - __shfl_sync(0xffffffffu, before, 31 - c);
      const int bin = 64 * c + 63 - 2 * lane;
      uint32_t n1 = 0u, n0 = 0u;
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const uint2 y = *reinterpret_cast<const uint2*>((C == 1 ? h : cluster.map_shared_rank(h, r)) + bin - 1);
        n0 += y.x;
        n1 += y.y;
      }
      before = inclusive_sum(n0 + n1, lane) - n0 - n1;
      if (before < rest && rest <= before + n1) {
        found[0] = (uint32_t)bin;
        found[1] = rest - before;
        found[2] = n1;
      } else if (before + n1 < rest && rest <= before + n1 + n0) {
        found[0] = (uint32_t)bin - 1u;
        found[1] = rest - before - n1;
        found[2] = n0;
      }
    }
    __syncthreads();
    cut |= found[0] << shift;
    left = found[1];
    const bool all = left == found[2];  // every weight that begins with these bits is taken
    __syncthreads();
    if (all) {
      // (a cut of 0 only where the least of all keys, NaN's, are taken: all of them)
      left = cut == 0u ? left : 0u;
      cut -= cut == 0u ? 0u : 1u;
      break;
    }
  }
  // all weights above the cut, and the first `left` of those at it
  uint32_t gt = 0u, eq = 0u;
  each([&](int, uint32_t key, bool in) {
    gt += in && key > cut;
    eq += in && key == cut;
  });
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    greater[warp] = gt;
    equal[warp] = eq;
  }
  __syncthreads();
  uint32_t gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? greater[lane] : 0u);
  uint32_t eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? equal[lane] : 0u);
  if constexpr (C > 1) {
    // this block's totals to every block
    if (warp == kSelWarps - 1 && lane < C)
      *cluster.map_shared_rank(&totals[rank], lane) = make_uint2(gt_before + gt, eq_before + eq);
    cluster.sync();
#pragma unroll
    for (int r = 0; r < C; ++r) {
      gt_before += r < rank ? totals[r].x : 0u;
      eq_before += r < rank ? totals[r].y : 0u;
    }
  }
  const uint32_t below = (1u << lane) - 1u;
  int32_t* out = list + e.sink;
  each([&](int j, uint32_t key, bool in) {
    const uint32_t mg = __ballot_sync(0xffffffffu, in && key > cut), me = __ballot_sync(0xffffffffu, in && key == cut);
    const uint32_t g = gt_before + __popc(mg & below), q = eq_before + __popc(me & below);
    if (in && (key > cut || (key == cut && q < left))) out[g + min(q, left)] = (int32_t)(at + j * 32 + lane);
    gt_before += __popc(mg);
    eq_before += __popc(me);
  });
}

// Element offset of place `slot` of a sequence whose page table row this is, or
// -1 (flagged).
__device__ __forceinline__ int64_t row_offset(const CacheView& c, const int32_t* table, int32_t pages, int64_t slot, int hk,
                                              int d, uint32_t* err) {
  const int64_t col = slot >> c.page_shift;
  const int32_t pg = col < pages ? table[col] : -1;
  if (pg < 0 || (int64_t)pg >= c.n_pages) {
    atomicOr(err, kErrBadCache);
    return -1;
  }
  return (((((int64_t)pg * c.kv_heads) + hk) << c.page_shift) + (slot & ((1 << c.page_shift) - 1))) * d;
}

// A block copies up to kMoveTokens kept tokens of one key head, keys and values.
constexpr int kMoveThreads = 128;
constexpr int kMoveTokens = 64;
template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictLaunch e) {
  constexpr int UNITS = D / 8, BATCH = 8;
  __shared__ int64_t from[kMoveTokens], to[kMoveTokens];
  grid_wait();
  grid_trigger();
  const int64_t unit = blockIdx.x / e.chunks;
  const int64_t i0 = (int64_t)(blockIdx.x - unit * e.chunks) * kMoveTokens;
  const int b = (int)(unit / e.cache.kv_heads), hk = (int)(unit % e.cache.kv_heads);
  const int len = evict_length(e, b, false), keep = min(len, e.budget);
  const int some = (int)max((int64_t)0, min((int64_t)kMoveTokens, keep - i0));
  if (threadIdx.x < kMoveTokens) {
    const int64_t i = i0 + threadIdx.x;
    float weight = 0.f;
    if (i < keep) {
      const int32_t src = e.list[unit * e.list_width + i];
      int64_t f = -1, t = -1;
      if (src >= 0 && src < len) {  // (else the workspace was written by another call meanwhile)
        weight = e.weights[unit * e.width + src];
        f = row_offset(e.cache, e.cache.page_table + (int64_t)b * e.cache.max_pages, e.cache.max_pages, src, hk, D, e.err);
        t = row_offset(e.cache, e.to_table + (int64_t)b * e.to_pages, e.to_pages, i, hk, D, e.err);
      }
      if (t < 0 || f == t) f = -1;  // (in its place already)
      from[threadIdx.x] = f;
      to[threadIdx.x] = t;
    }
    if (i < e.width_out) e.weights_out[unit * e.width_out + i] = weight;
  }
  __syncthreads();
  const int total = some * UNITS * 2;
  for (int x0 = threadIdx.x; x0 < total; x0 += kMoveThreads * BATCH) {
    uint4 v[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int x = x0 + k * kMoveThreads, row = x / (2 * UNITS), u = x % (2 * UNITS);
      if (x >= total || from[row] < 0) continue;
      const uint16_t* pool = u < UNITS ? e.cache.k_pages : e.cache.v_pages;
      v[k] = __ldcg(reinterpret_cast<const uint4*>(pool + from[row] + (u % UNITS) * 8));
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int x = x0 + k * kMoveThreads, row = x / (2 * UNITS), u = x % (2 * UNITS);
      if (x >= total || from[row] < 0) continue;
      uint16_t* pool = u < UNITS ? e.cache.k_pages : e.cache.v_pages;
      *reinterpret_cast<uint4*>(pool + to[row] + (u % UNITS) * 8) = v[k];
    }
  }
}

template <int C>
cudaError_t launch_selection(const EvictLaunch& e, int64_t units, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t r = cudaLaunchKernelEx(&cfg, select_kernel<C>, e);
  return r != cudaSuccess ? r : cudaGetLastError();
}

}  // namespace

int64_t evict_move_chunks(int64_t budget, int64_t width_out) {
  const int64_t most = budget > width_out ? budget : width_out;
  return (most + kMoveTokens - 1) / kMoveTokens;
}

cudaError_t launch_evict(const EvictLaunch& a, cudaStream_t stream) {
  EvictLaunch e = a;
  const int64_t units = (int64_t)e.cache.batch * e.cache.kv_heads;
  e.chunks = (int32_t)evict_move_chunks(e.budget, e.width_out);
  // one block where a sequence's weights fit its registers (or the heads fill
  // the GPU as they are), else eight
  const int64_t most = (int64_t)e.cache.max_pages << e.cache.page_shift;
  const bool one = most <= kSelThreads * kSelKeys || units >= 304;
  cudaError_t r = one ? launch_selection<1>(e, units, stream) : launch_selection<8>(e, units, stream);
  if (r != cudaSuccess) return r;
  auto move = e.head_dim == 64 ? move_kernel<64> : e.head_dim == 96 ? move_kernel<96> : move_kernel<128>;
  return launch_chained(move, dim3((unsigned)(units * e.chunks)), dim3(kMoveThreads), 0, stream, e);
}

}  // namespace wise
