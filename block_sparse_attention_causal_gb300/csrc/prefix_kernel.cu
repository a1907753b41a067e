// Attention of a batch whose sequences share prefixes: what a group of sequences
// shares is read once, for all of their rows together.
//
// The softmax over a row's tokens splits into the shared ones and its own:
//   O = 2^(L_p - L) O_p + 2^(L_s - L) O_s,   2^L = 2^L_p + 2^L_s,
// each part with its own maximum and sum. The shared part is a unit of all the
// group's rows over whole tiles of 128 tokens (a prefix that ends inside a tile
// leaves the rest of it to the sequences' own parts, so that no tile needs a mask),
// read through the page table of one of them; the own part is the attention of
// tree.cuh with those tiles left out.
//
// Four launches: a plan of one block; the shared part and the own parts, side by
// side on shares of the SMs that the plan sets by their work (the shared part is
// bound by the tensor core and the softmax, the own parts by the cache's bytes); and
// the join of everything that belongs to a row.
//
// Both parts round a softmax weight to bf16 (2^-8) before it meets V, as the attention
// without sharing does; its sum, the maxima and all partial results are fp32, and O is
// rounded once more where it is bf16. (Root mean square error of bf16 results against
// 64 bits 2.3e-3 of their size, 1.7e-3 of it the last rounding.)
//
// Measured (one GB300): next tokens of 64 sequences, 32/8 heads of 128, behind 32K shared
// and up to 1K of their own (299 MB, 35 GFLOP): 78 us, 97 when the parts ran one after
// the other, each with its own join. The plan takes 4 us, the parts start 1 and 3 us
// later, the first tiles are 6 us on, and the join ends 8 us behind the last of them.
#include "tree_wide.cuh"

namespace wise {

template cudaError_t launch_tree_rows<true>(const TreeLaunch&, const CUtensorMap*, cudaStream_t);

namespace {

struct Plan {
  uint64_t* go;     // kPlanTag and, below it, the blocks of the own parts: written last
  int32_t* starts;  // [groups + 1]
  int32_t* length;  // [groups] shared tokens, whole tiles
  int32_t* leader;  // [groups]
  int32_t* skip;    // [batch] the sequence's shared tokens
  int32_t* group;   // [batch] its group, where it shares any
  int32_t* live;    // [batch] its new tokens, as far as the page table holds them
  int32_t* limit;   // blocks of the shared part
};
struct PlanParams {
  TreeParams shared, own;
  int32_t groups, members;
  const int32_t* group_starts;
  const int32_t* prefix_lengths;
  Plan plan;
  float shared_cost, own_cost;  // of a place of the line
};

// One block, a warp per group. A sequence shorter than its group's prefix (an
// empty place of a padded batch, for instance) shares nothing; nor does a group
// of fewer than two that are long enough.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  __shared__ unsigned long long places[2];  // of the shared part and of the own parts
  prefetch_tables(p.own);
  grid_wait();
  grid_trigger();
  const CacheView& c = p.own.t.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < 2) places[threadIdx.x] = 0ull;
  auto start = [&](int g) -> int32_t { return p.group_starts ? p.group_starts[g] : g == 0 ? 0 : c.batch; };
  bool bad = false;
  for (int g = threadIdx.x; g <= p.groups; g += kPlanThreads) {
    const int32_t s = start(g);
    bad |= s < 0 || s > c.batch || (g > 0 && s < start(g - 1));
  }
  const bool none = __syncthreads_or(bad);  // no groups then
  if (none && threadIdx.x == 0) atomicOr(p.own.t.err, kErrBadCache);
  for (int g = threadIdx.x; g <= p.groups; g += kPlanThreads) p.plan.starts[g] = none ? 0 : start(g);
  for (int b = threadIdx.x; b < c.batch; b += kPlanThreads)
    if (none || b < start(0) || b >= start(p.groups)) p.plan.skip[b] = 0;
  const int64_t cap = (int64_t)c.max_pages << c.page_shift;
  unsigned long long sum = 0ull;
  for (int g = warp; g < p.groups; g += kPlanThreads / 32) {
    const int b0 = none ? 0 : start(g), b1 = none ? 0 : start(g + 1);
    const int32_t prefix = p.prefix_lengths[g];
    if ((prefix < 0 || prefix > cap) && lane == 0) atomicOr(p.own.t.err, kErrBadCache);
    // whole tiles; lengths past the page table are held to what it holds elsewhere
    int len = prefix < 0 || prefix > cap ? 0 : prefix / kTile * kTile;
    int sharing = 0, leader = 0;
    for (int b = b0; b < b1; b += 32) {
      const uint32_t m = __ballot_sync(0xffffffffu, b + lane < b1 && c.lengths[b + lane] >= prefix);
      if (sharing == 0 && m != 0u) leader = b + __ffs(m) - 1;
      sharing += __popc(m);
    }
    if (b1 - b0 > p.members) {  // more rows than the launch is made for
      if (lane == 0) atomicOr(p.own.t.err, kErrBadCache);
      len = 0;
    }
    if (sharing < 2) len = 0;
    for (int b = b0 + lane; b < b1; b += 32) {
      p.plan.skip[b] = c.lengths[b] >= prefix ? len : 0;
      p.plan.group[b] = g;
    }
    if (lane == 0) {
      p.plan.length[g] = len;
      p.plan.leader[g] = leader;
      int full, active;
      const int nl = len > 0 ? (b1 - b0) * p.own.t.n : 0;
      seq_tiles<true>(p.shared, len, nl, full, active);
      sum += (unsigned long long)seq_line<true>(p.shared, full, active);
    }
  }
  if (sum != 0ull) atomicAdd(&places[0], sum);
  __syncthreads();
  sum = 0ull;
  for (int b = threadIdx.x; b < c.batch; b += kPlanThreads) {
    int len, nl, full, active;
    seq_counts<false>(p.own.t, b, len, nl);
    p.plan.live[b] = nl;
    seq_tiles<false>(p.own, len, nl, full, active);
    sum += (unsigned long long)seq_line<false>(p.own, full, active);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) atomicAdd(&places[1], sum);
  __syncthreads();
  if (threadIdx.x == 0) {
    const float a = (float)places[0] * p.shared_cost, b = (float)places[1] * p.own_cost;
    int blocks = a == 0.f ? 0 : (int)((float)kTreeCtas * a / (a + b) + 0.5f);
    if (a != 0.f) blocks = min(max(blocks, 1), kTreeCtas - 1);
    p.plan.limit[0] = blocks;
    st_release_gpu(p.plan.go, kPlanTag | (uint32_t)(kTreeCtas - blocks));
  }
}

struct SharedJoin {
  TreeParams shared, own;
  Plan plan;
  void* o;
  float* lse;
  int32_t out_f32;
};

// What a unit left of one row, added to the row's sums: the whole row, or its parts
// in the line's order (BATCH of them asked for at a time).
template <int D>
__device__ __forceinline__ void add_unit(const TreeParams& p, int64_t unit, int r, int64_t out_row, int c4, float& m, float& l,
                                         float4& acc) {
  constexpr int BATCH = 8;
  const int4 ra = *reinterpret_cast<const int4*>(&p.rec[unit]);
  const int4 rb = *(reinterpret_cast<const int4*>(&p.rec[unit]) + 1);
  const bool whole = ra.x == 1;
  const int parts = whole ? 1 : rec_ok(p, ra, rb) ? ra.x : 0;
  const float* o_row = static_cast<const float*>(p.t.o) + out_row * D + c4 * 4;
  const bool wide = p.rows > 64;
  for (int k0 = 0; k0 < parts; k0 += BATCH) {
    float pm[BATCH], pl[BATCH];
    float4 x[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      pl[i] = 0.f;
      const int k = k0 + i;
      if (k >= parts) continue;
      const int64_t at = (k == 0 ? ra.y : 2 * (ra.z + k)) * (int64_t)p.row_slots;
      const float* st = whole ? p.t.lse + out_row : p.part_s + 2 * at + r;
      const float* o = whole  ? o_row
                       : wide ? p.part_o + at * D + ((int64_t)(r >> 5) * (D / 4) + c4) * 128 + (r & 31) * 4
                              : p.part_o + (at + r) * D + c4 * 4;
      x[i] = *reinterpret_cast<const float4*>(o);
      pm[i] = st[0];
      pl[i] = whole ? 1.f : st[p.row_slots];
    }
    if (whole) {
      pl[0] = pm[0] == -INFINITY ? 0.f : 1.f;
      pm[0] *= 1.4426950408889634f;
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (pl[i] != 0.f) top = fmaxf(top, pm[i]);
    const float f = l == 0.f ? 0.f : fast_exp2(m - top);
    m = top;
    l *= f;
    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (pl[i] == 0.f) continue;  // saw nothing
      const float g = fast_exp2(pm[i] - m);
      l += pl[i] * g;
      acc.x += x[i].x * g, acc.y += x[i].y * g, acc.z += x[i].z * g, acc.w += x[i].w * g;
    }
  }
}

// A lane per row of a key head (32 consecutive ones of the batch), a warp per four
// columns, so that partial results of consecutive rows are whole lines.
template <int D>
__global__ void __launch_bounds__(128) shared_join_kernel(const SharedJoin j) {
  grid_wait();
  grid_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *j.plan.go = 0ull;  // a later call's own parts must not take it for theirs
  const TreeParams& own = j.own;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kv_heads = own.t.cache.kv_heads, per = kv_heads * (D / 16);
  const int hk = blockIdx.x % per / (D / 16), c4 = blockIdx.x % (D / 16) * 4 + warp;
  const int64_t at = (int64_t)(blockIdx.x / per) * 32 + lane;
  const int b = (int)(at / own.rows), r = (int)(at - (int64_t)b * own.rows);
  if (b >= own.t.cache.batch) return;
  const int tok = row_token(own, r), h = hk * own.group + (r - tok * own.group);
  const int64_t out_row = ((int64_t)b * own.t.heads + h) * own.t.n + tok;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (j.plan.skip[b] > 0) {
    const int g = j.plan.group[b];
    const int row = (b - j.plan.starts[g]) * own.rows + r;
    add_unit<D>(j.shared, unit_rec<true>(j.shared, g, hk, row >> 8), row & 255, out_row, c4, m, l, acc);
  }
  add_unit<D>(own, unit_rec<false>(own, b, hk, r >> 8), r & 255, out_row, c4, m, l, acc);
  const bool zero = l == 0.f;
  const float inv = zero ? 0.f : 1.f / l;
  const float4 o = make_float4(zero ? 0.f : acc.x * inv, zero ? 0.f : acc.y * inv, zero ? 0.f : acc.z * inv,
                               zero ? 0.f : acc.w * inv);
  if (j.out_f32) reinterpret_cast<float4*>(static_cast<float*>(j.o) + out_row * D)[c4] = o;
  else
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(j.o) + out_row * D)[c4] =
        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  if (c4 == 0 && j.lse) j.lse[out_row] = zero ? -INFINITY : (m + fast_log2(l)) * 0.69314718055994531f;
}

struct PrefixLayout {
  int64_t shared, own, o_own, o_shared, lse_own, lse_shared, bytes;  // offsets in bytes; the plan's words at 0
};
PrefixLayout prefix_layout(int64_t batch, int64_t kv_heads, int64_t heads, int64_t n, int64_t d, int64_t groups,
                           int64_t members) {
  PrefixLayout w;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  const int64_t per = heads / kv_heads * n, rows = batch * heads * n;
  w.shared = up(8 + (3 * groups + 1 + 3 * batch + 1) * 4);
  w.own = w.shared + up(workspace_layout(shared_units(groups, kv_heads, per * batch), per * members, d, true).bytes);
  w.o_own = w.own + up(workspace_layout(tree_units(batch, kv_heads, per), per, d, true).bytes);
  w.o_shared = w.o_own + up(rows * d * 4);
  w.lse_own = w.o_shared + up(rows * d * 4);
  w.lse_shared = w.lse_own + up(rows * 4);
  w.bytes = w.lse_shared + up(rows * 4) + 256;  // the base is rounded up to 256 bytes
  return w;
}

// Time of a place of the line, in microseconds, by the rows of a unit: what decides
// how the SMs are shared out. (64 next tokens behind 32K and up to 1K of their own:
// 80.8, 77.3, 76.1, 83.0, 88.2 us with 0.6, 0.8, 0.85, 1.0, 1.2 for up to 16 rows; trees
// of 5 with 25 rows 51.5, 47.1, 45.9, 47.1 us with 0.8, 1.0, 1.2, 1.5.) Each constant
// swept with the others as they are, 32/8 heads of 64, 96 and 128 behind 8K and 32K,
// 256, 1K and 4K tokens of their own; how far the one taken is behind the sweep's best:
//   24 shared rows, 1.2 (of 0.8, 1.0, 1.2, 1.5)         0 to 12 % (best 1.0 to 1.5)
//   48 shared rows, 1.6 (of 0.8, 1.0, 1.2, 1.6, 2.0)    0 to 9 %  (0.8 to 1.6)
//   40 own rows, 1.6 (of the same)                      0 to 10 % (1.2 with 4K, else 1.6)
//   96 shared rows, 1.0 (of 0.6, 0.8, 1.0, 1.25, 1.6)   0 to 10 % (0.8 to 1.6)
//   192 shared rows, 1.65 (of 1.1, 1.35, 1.65, 2, 2.4)  0 to 8 %  (1.65 to 2.4)
//   256 shared rows, 1.65 (of the same)                 0 to 17 % (1.65 to 2.4; 17 % with 64
//                                                       dimensions and 4K of their own)
// A constant half as large as the best costs up to 1.6 times the time.
float place_cost(const TreeParams& p) {
  return p.rows > 128 ? 1.65f : p.rows > 64 ? 1.f : p.rows > 32 ? 1.6f : p.rows > 16 ? 1.2f : 0.85f;
}

}  // namespace

int64_t prefix_workspace_bytes(int32_t batch, int32_t kv_heads, int32_t heads, int32_t n, int32_t head_dim, int32_t groups) {
  return prefix_layout(batch, kv_heads, heads, n, head_dim, groups, batch).bytes;
}

cudaError_t launch_prefix(const PrefixLaunch& x, const CUtensorMap* maps, cudaStream_t stream) {
  const CacheView& c = x.t.cache;
  const PrefixLayout w = prefix_layout(c.batch, c.kv_heads, x.t.heads, x.t.n, x.t.head_dim, x.groups, x.members);
  uint8_t* ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(x.t.workspace) + 255) / 256 * 256);
  Plan plan;
  plan.go = reinterpret_cast<uint64_t*>(ws);
  plan.starts = reinterpret_cast<int32_t*>(ws + 8);
  plan.length = plan.starts + x.groups + 1;
  plan.leader = plan.length + x.groups;
  plan.skip = plan.leader + x.groups;
  plan.group = plan.skip + c.batch;
  plan.live = plan.group + c.batch;
  plan.limit = plan.live + c.batch;
  // what is shared: a cache of the groups
  TreeLaunch shared = x.t;
  shared.cache.batch = x.groups;
  shared.cache.lengths = plan.length;
  shared.tree_mask = nullptr;
  shared.new_len = plan.live;
  shared.starts = plan.starts;
  shared.leader = plan.leader;
  shared.sequences = c.batch;
  shared.members = x.members;
  shared.limit = plan.limit;
  shared.rows_apart = 1;
  shared.workspace = ws + w.shared;
  shared.out_f32 = 1;
  shared.o = ws + w.o_shared;
  shared.lse = reinterpret_cast<float*>(ws + w.lse_shared);
  // each sequence's own
  TreeLaunch own = x.t;
  own.skip = plan.skip;
  own.go = plan.go;
  own.rows_apart = 1;
  own.workspace = ws + w.own;
  own.out_f32 = 1;
  own.o = ws + w.o_own;
  own.lse = reinterpret_cast<float*>(ws + w.lse_own);
  const TreeParams ps = tree_params<true>(shared), po = tree_params<false>(own);
  const PlanParams pp{ps, po, x.groups, x.members, x.group_starts, x.prefix_lengths, plan, place_cost(ps), place_cost(po)};
  cudaError_t e = launch_chained(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, pp);
  if (e == cudaSuccess) e = launch_tree_rows<true>(shared, maps, stream);
  if (e == cudaSuccess) e = launch_tree_rows<false>(own, maps, stream);
  if (e != cudaSuccess) return e;
  const SharedJoin j{ps, po, plan, x.t.o, x.t.lse, x.t.out_f32};
  auto join = x.t.head_dim == 64 ? shared_join_kernel<64> : x.t.head_dim == 96 ? shared_join_kernel<96> : shared_join_kernel<128>;
  const int64_t rows = (int64_t)c.batch * po.rows;
  const int64_t blocks = (rows + 31) / 32 * c.kv_heads * (x.t.head_dim / 16);
  return launch_chained(join, dim3((unsigned)blocks), dim3(128), 0, stream, j);
}

}  // namespace wise
