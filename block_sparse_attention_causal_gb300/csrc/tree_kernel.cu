// Attention of new tokens over a paged cache: WISE §3 Eq 2 for the rows behind
// the prompt (a next token, a run of tokens, a tree of drafted tokens).
#include "internal.h"
#include "ptx.cuh"

namespace wise {
namespace {

constexpr int kWarps = 8;

// One block per (sequence, query head, new token). Each warp takes every
// eighth seen token with an online softmax (running maximum m, sum l and
// weighted values, all fp32; lane x holds dimensions x, x + 32, ...), and the
// eight partial results are joined at the end.
template <int D>
__global__ void __launch_bounds__(32 * kWarps) tree_kernel(const TreeLaunch p) {
  constexpr int E = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int i = blockIdx.x % p.n, bh = blockIdx.x / p.n;
  const int h = bh % p.heads, b = bh / p.heads;
  const int hk = h / (p.heads / p.cache.kv_heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t cap = (int64_t)p.cache.max_pages << p.cache.page_shift;
  int64_t len = __ldg(p.cache.lengths + b);
  int nl = p.new_len ? __ldg(p.new_len + b) : p.n;
  if (len < 0 || nl < 0 || nl > p.n || len + nl > cap) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrBadCache);
    nl = max(0, min(nl, p.n));
    len = max((int64_t)0, min(len, cap));
    nl = (int)min((int64_t)nl, cap - len);
  }
  float q[E];
  const uint16_t* qp = p.q.data + (int64_t)b * p.q.sb + (int64_t)h * p.q.sh + (int64_t)i * p.q.sn;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = __uint_as_float((uint32_t)qp[e * 32 + lane] << 16);
  const int words = (p.n + 31) / 32;
  const int32_t* mask = p.tree_mask ? p.tree_mask + ((int64_t)b * p.n + i) * words : nullptr;
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const int64_t keys = (i < nl) ? len + nl : 0;
  for (int64_t t = warp; t < keys; t += kWarps) {
    if (t >= len) {
      const int j = (int)(t - len);
      const bool sees = mask ? (__ldg(mask + j / 32) >> (j % 32)) & 1 : j <= i;
      if (!sees) continue;
    }
    const int32_t pg = __ldg(p.cache.page_table + (int64_t)b * p.cache.max_pages + (t >> p.cache.page_shift));
    if (pg < 0 || (int64_t)pg >= p.cache.n_pages) {
      if (lane == 0) atomicOr(p.err, kErrBadCache);
      continue;
    }
    const int64_t row = ((((int64_t)pg * p.cache.kv_heads + hk) << p.cache.page_shift) +
                         (t & ((1 << p.cache.page_shift) - 1))) * D;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * __uint_as_float((uint32_t)p.cache.k_pages[row + e * 32 + lane] << 16);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale;
    const float mn = fmaxf(m, s);
    const float f = (mn == -INFINITY) ? 1.f : expf(m - mn), w = (s == -INFINITY) ? 0.f : expf(s - mn);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * f + w * __uint_as_float((uint32_t)p.cache.v_pages[row + e * 32 + lane] << 16);
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][e * 32 + lane] = o[e];
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  float sum = 0.f, val = 0.f;
  const int x = threadIdx.x;
  for (int w = 0; w < kWarps; ++w) {
    if (sl[w] == 0.f) continue;
    const float f = expf(sm[w] - top);
    sum += sl[w] * f;
    if (x < D) val += so[w][x] * f;
  }
  const int64_t grow = (int64_t)bh * p.n + i;
  if (x < D) {
    const float r = sum == 0.f ? 0.f : val / sum;
    if (p.out_f32) static_cast<float*>(p.o)[grow * D + x] = r;
    else static_cast<uint16_t*>(p.o)[grow * D + x] = (uint16_t)pack_bf16x2(r, 0.f);
  }
  if (x == 0 && p.lse) p.lse[grow] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

int64_t tree_workspace_bytes(int32_t, int32_t, int32_t, int32_t, int32_t) { return 16; }

cudaError_t launch_tree(const TreeLaunch& t, cudaStream_t stream) {
  const unsigned grid = (unsigned)(t.cache.batch * t.heads * t.n);
  switch (t.head_dim) {
    case 64: tree_kernel<64><<<grid, 32 * kWarps, 0, stream>>>(t); break;
    case 96: tree_kernel<96><<<grid, 32 * kWarps, 0, stream>>>(t); break;
    default: tree_kernel<128><<<grid, 32 * kWarps, 0, stream>>>(t); break;
  }
  return cudaGetLastError();
}

}  // namespace wise
