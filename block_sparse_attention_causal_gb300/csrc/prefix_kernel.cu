// Attention of a batch whose sequences share prefixes: what a group of sequences
// shares is read once, for all of their rows together.
//
// The softmax over a row's tokens splits into the shared ones and its own:
//   O = (2^(L_p - L) O_p + 2^(L_s - L) O_s),   2^L = 2^L_p + 2^L_s,
// each part with its own maximum and sum. The shared part is a unit of all the
// group's rows over whole tiles of 128 tokens (a prefix that ends inside a tile
// leaves the rest of it to the sequences' own parts, so that no tile needs a mask),
// read through the page table of one of them; the own part is the attention of
// tree.cuh with those tiles left out.
#include "tree_wide.cuh"

namespace wise {

template cudaError_t launch_tree_rows<true>(const TreeLaunch&, const CUtensorMap*, cudaStream_t);

namespace {

struct PlanParams {
  CacheView cache;
  int32_t groups;
  const int32_t* group_starts;
  const int32_t* prefix_lengths;
  int32_t* starts;  // [groups + 1]
  int32_t* length;  // [groups] shared tokens, whole tiles
  int32_t* leader;  // [groups]
  int32_t* skip;    // [batch]
  uint32_t* err;
};

// One block, a warp per group. A sequence shorter than its group's prefix (an
// empty place of a padded batch, for instance) shares nothing; nor does a group
// of fewer than two that are long enough.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  grid_wait();
  grid_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto start = [&](int g) -> int32_t {
    return p.group_starts ? p.group_starts[g] : g == 0 ? 0 : p.cache.batch;
  };
  bool bad = false;
  for (int g = threadIdx.x; g <= p.groups; g += kPlanThreads) {
    const int32_t s = start(g);
    bad |= s < 0 || s > p.cache.batch || (g > 0 && s < start(g - 1));
  }
  const bool none = __syncthreads_or(bad);  // no groups then
  if (none && threadIdx.x == 0) atomicOr(p.err, kErrBadCache);
  for (int g = threadIdx.x; g <= p.groups; g += kPlanThreads) p.starts[g] = none ? 0 : start(g);
  for (int b = threadIdx.x; b < p.cache.batch; b += kPlanThreads)
    if (none || b < start(0) || b >= start(p.groups)) p.skip[b] = 0;
  const int64_t cap = (int64_t)p.cache.max_pages << p.cache.page_shift;
  for (int g = warp; g < p.groups; g += kPlanThreads / 32) {
    const int b0 = none ? 0 : start(g), b1 = none ? 0 : start(g + 1);
    const int32_t prefix = p.prefix_lengths[g];
    if ((prefix < 0 || prefix > cap) && lane == 0) atomicOr(p.err, kErrBadCache);
    // whole tiles; lengths past the page table are held to what it holds elsewhere
    int len = prefix < 0 || prefix > cap ? 0 : prefix / kTile * kTile;
    int sharing = 0, leader = 0;
    for (int b = b0; b < b1; b += 32) {
      const uint32_t m = __ballot_sync(0xffffffffu, b + lane < b1 && p.cache.lengths[b + lane] >= prefix);
      if (sharing == 0 && m != 0u) leader = b + __ffs(m) - 1;
      sharing += __popc(m);
    }
    if (sharing < 2) len = 0;
    for (int b = b0 + lane; b < b1; b += 32) p.skip[b] = p.cache.lengths[b] >= prefix ? len : 0;
    if (lane == 0) {
      p.length[g] = len;
      p.leader[g] = leader;
    }
  }
}

struct MergeParams {
  int64_t rows;
  int32_t per_sequence;  // rows of a sequence
  const int32_t* skip;
  const float* o_own;
  const float* o_shared;
  const float* lse_own;
  const float* lse_shared;
  void* o;
  float* lse;
  int32_t out_f32;
};

// A warp per row.
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const MergeParams p) {
  constexpr int E = D / 32;
  grid_wait();
  grid_trigger();
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= p.rows) return;
  const bool shared = p.skip[row / p.per_sequence] > 0;
  const float a = p.lse_own[row];
  float x[E], lse = a;
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = p.o_own[row * D + lane * E + e];
  if (shared) {
    const float b = p.lse_shared[row];
    const float top = fmaxf(a, b) == -INFINITY ? 0.f : fmaxf(a, b);
    const float wa = fast_exp2((a - top) * 1.4426950408889634f), wb = fast_exp2((b - top) * 1.4426950408889634f);
    const float sum = wa + wb;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float y = p.o_shared[row * D + lane * E + e];
      // (a part that saw nothing has no say, whatever its O)
      x[e] = (a == -INFINITY ? 0.f : x[e] * (wa * inv)) + (b == -INFINITY ? 0.f : y * (wb * inv));
    }
    lse = sum == 0.f ? -INFINITY : top + fast_log2(sum) * 0.69314718055994531f;
  }
  if (p.out_f32) {
#pragma unroll
    for (int e = 0; e < E; ++e) static_cast<float*>(p.o)[row * D + lane * E + e] = x[e];
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) static_cast<uint16_t*>(p.o)[row * D + lane * E + e] = (uint16_t)pack_bf16x2(x[e], 0.f);
  }
  if (lane == 0 && p.lse) p.lse[row] = lse;
}

struct PrefixLayout {
  int64_t tree, o_own, o_shared, lse_own, lse_shared, bytes;  // offsets in bytes; the plan's words at 0
};
PrefixLayout prefix_layout(int64_t batch, int64_t kv_heads, int64_t heads, int64_t n, int64_t d, int64_t groups) {
  PrefixLayout w;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  const int64_t per = heads / kv_heads * n, rows = batch * heads * n;
  const int64_t own = workspace_layout(batch, kv_heads, per, d, false).bytes;
  const int64_t shared = workspace_layout(groups, kv_heads, per * batch, d, true).bytes;
  w.tree = up((3 * groups + 1 + batch) * 4);
  w.o_own = w.tree + up(own > shared ? own : shared);
  w.o_shared = w.o_own + up(rows * d * 4);
  w.lse_own = w.o_shared + up(rows * d * 4);
  w.lse_shared = w.lse_own + up(rows * 4);
  w.bytes = w.lse_shared + up(rows * 4) + 256;  // the base is rounded up to 256 bytes
  return w;
}

}  // namespace

int64_t prefix_workspace_bytes(int32_t batch, int32_t kv_heads, int32_t heads, int32_t n, int32_t head_dim, int32_t groups) {
  return prefix_layout(batch, kv_heads, heads, n, head_dim, groups).bytes;
}

cudaError_t launch_prefix(const PrefixLaunch& l, const CUtensorMap* maps, cudaStream_t stream) {
  const CacheView& c = l.t.cache;
  const int32_t batch = c.batch;
  const PrefixLayout w = prefix_layout(batch, c.kv_heads, l.t.heads, l.t.n, l.t.head_dim, l.groups);
  uint8_t* ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(l.t.workspace) + 255) / 256 * 256);
  int32_t* words = reinterpret_cast<int32_t*>(ws);
  PlanParams plan{c, l.groups, l.group_starts, l.prefix_lengths, words, words + l.groups + 1, words + 2 * l.groups + 1,
                  words + 3 * l.groups + 1, l.t.err};
  cudaError_t e = launch_chained(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, plan);
  if (e != cudaSuccess) return e;
  // what is shared
  TreeLaunch t = l.t;
  t.cache.batch = l.groups;
  t.cache.lengths = plan.length;
  t.tree_mask = nullptr;
  t.starts = plan.starts;
  t.leader = plan.leader;
  t.sequences = batch;
  t.workspace = ws + w.tree;
  t.out_f32 = 1;
  t.o = ws + w.o_shared;
  t.lse = reinterpret_cast<float*>(ws + w.lse_shared);
  e = launch_tree_rows<true>(t, maps, stream);
  if (e != cudaSuccess) return e;
  // each sequence's own
  t = l.t;
  t.skip = plan.skip;
  t.workspace = ws + w.tree;
  t.out_f32 = 1;
  t.o = ws + w.o_own;
  t.lse = reinterpret_cast<float*>(ws + w.lse_own);
  e = launch_tree_rows<false>(t, maps, stream);
  if (e != cudaSuccess) return e;
  const MergeParams m{(int64_t)batch * l.t.heads * l.t.n,
                      l.t.heads * l.t.n,
                      plan.skip,
                      reinterpret_cast<const float*>(ws + w.o_own),
                      reinterpret_cast<const float*>(ws + w.o_shared),
                      reinterpret_cast<const float*>(ws + w.lse_own),
                      reinterpret_cast<const float*>(ws + w.lse_shared),
                      l.t.o,
                      l.t.lse,
                      l.t.out_f32};
  auto merge = l.t.head_dim == 64 ? merge_kernel<64> : l.t.head_dim == 96 ? merge_kernel<96> : merge_kernel<128>;
  return launch_chained(merge, dim3((unsigned)((m.rows + 7) / 8)), dim3(256), 0, stream, m);
}

}  // namespace wise
