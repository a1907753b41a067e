// Queries and keys normed per head and rotated by their positions in one pass:
//   y = x / sqrt(mean(x^2) + eps) * w          over a head's values,
//   (y1, y2) -> (y1 cos a - y2 sin a, y2 cos a + y1 sin a), a = 2 pi frac(position step / 2^64),
// into a paged cache (keys; values are copied) or into dense rows before a
// prompt's attention. A position may have several axes (time, row and column of
// an image), each pair of values turning with one of them.
#include "rotate.cuh"

namespace wise {
namespace {

// Sum over the lanes of one token, the same bits in each of them.
template <int G>
__device__ __forceinline__ float token_sum(float x, int lane) {
  if constexpr (G == 6) {
    const int first = lane / 6 * 6, c = lane - first;
    x += __shfl_sync(0xffffffffu, x, (first + (c + 3) % 6) & 31);
    const float x0 = __shfl_sync(0xffffffffu, x, first & 31), x1 = __shfl_sync(0xffffffffu, x, (first + 1) & 31),
                x2 = __shfl_sync(0xffffffffu, x, (first + 2) & 31);
    return (x0 + x1) + x2;
  } else {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  }
}

__device__ __forceinline__ void widen8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 narrow8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
// Eight weights from element `at` on.
__device__ __forceinline__ void weights8(const NormLaunch& p, const void* w, int64_t at, float* x) {
  if (p.weight_f32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 a = f[0], b = f[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + at), x);
  }
}

// One thread per (token, pair of 16-byte chunks), walking the query heads, the
// key heads and the values of its token, so that the sines and cosines of its
// eight pairs are taken once per token. A token's D / 16 threads are lanes of
// one warp (heads of 96: five tokens a warp, two lanes idle) and sum the squares
// among themselves. With few tokens the heads are spread over gridDim.y.
// AHEAD heads are loaded before the first is worked on.
template <int D, bool PAIRS, int AHEAD>
__global__ void __launch_bounds__(256, AHEAD == 4 ? 2 : 3) norm_kernel(const NormLaunch p) {
  constexpr int G = D / 16, TOKENS = 32 / G;  // lanes of a token, tokens of a warp
  grid_wait();
  grid_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t tok = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * TOKENS + lane / G;
  const bool on = lane < TOKENS * G && tok < (int64_t)p.batch * p.n;
  const int c = lane % G;
  const int b = on ? (int)(tok / p.n) : 0, i = on ? (int)(tok % p.n) : 0;
  // element offsets of the thread's two chunks within a head: halves rotation
  // pairs chunk c with chunk c + rotary_dim / 16; everything else takes
  // neighbouring chunks
  const int nrot = p.rotary_dim / 16;
  const bool rot = c < nrot;
  const int ca = (rot && !PAIRS) ? c * 8 : 2 * c * 8;
  const int cb = (rot && !PAIRS) ? (c + nrot) * 8 : ca + 8;
  int32_t len = 0;
  int64_t dst = -1;  // the token's key row of head 0
  if (p.paged) {
    len = p.cache.lengths[b];
    const int32_t nl = p.new_len ? p.new_len[b] : p.n;
    if (on && (len < 0 || nl < 0 || nl > p.n)) atomicOr(p.err, kErrBadCache);
    if (on && len >= 0 && i < nl) dst = slot_offset(p.cache, b, (int64_t)len + i, D, p.err);
  } else if (on) {
    dst = ((int64_t)b * p.kv_heads * p.n + i) * D;
  }
  const int64_t head_step = p.paged ? (int64_t)D << p.cache.page_shift : (int64_t)p.n * D;
  float cs[8], sn[8];
  bool turned = false;
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {  // queries, keys, values
    const RowsView& src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    const int heads = kind == 0 ? p.heads : src.data ? p.kv_heads : 0;
    const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
    const int64_t weight_step = kind == 0 ? p.q_weight_stride : p.k_weight_stride;
    uint16_t* out = kind == 0   ? p.q_out + ((int64_t)b * p.heads * p.n + i) * D
                    : kind == 1 ? p.k_out + dst
                                : p.v_out + dst;
    const int64_t out_step = kind == 0 ? (int64_t)p.n * D : head_step;
    const bool live = on && (kind == 0 || dst >= 0);
    const uint16_t* from = src.data + (int64_t)b * src.sb + (int64_t)i * src.sn;
    float w[16];
    if (weight && weight_step == 0 && (int)blockIdx.y < heads) {
      weights8(p, weight, ca, w);
      weights8(p, weight, cb, w + 8);
    }
#pragma unroll 1
    for (int u0 = blockIdx.y; u0 < heads; u0 += AHEAD * gridDim.y) {
      uint4 xa[AHEAD], xb[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int u = u0 + k * gridDim.y;
        xa[k] = xb[k] = make_uint4(0u, 0u, 0u, 0u);
        if (live && u < heads) {
          // past the L1 cache: each value is read once
          xa[k] = __ldcg(reinterpret_cast<const uint4*>(from + (int64_t)u * src.sh + ca));
          xb[k] = __ldcg(reinterpret_cast<const uint4*>(from + (int64_t)u * src.sh + cb));
        }
      }
      if (!turned && rot && on) {
        // after the first loads are on their way
        turned = true;
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          int64_t pos = (int64_t)len + i;
          if (p.positions) {
            const int axis = p.axes ? p.axes[8 * c + f] : 0;
            const bool known = axis >= 0 && axis < p.n_axes;
            if (!known) atomicOr(p.err, kErrBadCache);
            pos = known ? p.positions[((int64_t)axis * p.batch + b) * p.n + i] : 0;
          }
          sine_cosine((uint64_t)pos * (uint64_t)p.rope[8 * c + f], sn[f], cs[f]);
        }
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int u = u0 + k * gridDim.y;
        if (u >= heads) break;  // (the same for the whole block)
        if (kind < 2) {
          float x[16];
          widen8(xa[k], x);
          widen8(xb[k], x + 8);
          if (weight) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
            const float inv = rsqrtf(token_sum<G>(ss, lane) * (1.f / D) + p.eps);
            if (weight_step != 0 && live) {
              weights8(p, weight, u * weight_step + ca, w);
              weights8(p, weight, u * weight_step + cb, w + 8);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = x[e] * inv * w[e];
          }
          if (rot) {
#pragma unroll
            for (int f = 0; f < 8; ++f) {
              float& y1 = PAIRS ? x[2 * f] : x[f];
              float& y2 = PAIRS ? x[2 * f + 1] : x[8 + f];
              const float t = y1;
              y1 = t * cs[f] - y2 * sn[f];
              y2 = y2 * cs[f] + t * sn[f];
            }
          }
          xa[k] = narrow8(x);
          xb[k] = narrow8(x + 8);
        }
        if (live) {
          *reinterpret_cast<uint4*>(out + u * out_step + ca) = xa[k];
          *reinterpret_cast<uint4*>(out + u * out_step + cb) = xb[k];
        }
      }
    }
  }
}

template <int D>
cudaError_t launch_norm_d(const NormLaunch& a, cudaStream_t stream) {
  constexpr int TOKENS = 32 / (D / 16) * 8;  // of a block
  const int64_t blocks = ((int64_t)a.batch * a.n + TOKENS - 1) / TOKENS;
  const int units = a.heads + (a.k.data ? a.kv_heads : 0) + (a.v.data ? a.kv_heads : 0);
  // heads spread until the grid fills the GPU, and on, as long as a thread keeps
  // four of them, to 24 blocks per SM (cache_kernel.cu has the measurements)
  constexpr int64_t kFull = 152 * 8, kMany = 152 * 24;
  int64_t ny = kMany / blocks < units / 4 ? kMany / blocks : units / 4;
  if (ny < kFull / blocks) ny = kFull / blocks;
  ny = ny < 1 ? 1 : (ny > units ? units : ny);
  const int most = a.heads > a.kv_heads ? a.heads : a.kv_heads;
  if (ny > most) ny = most;
  const dim3 grid((unsigned)blocks, (unsigned)ny);
  auto kernel = ny * 4 <= units ? (a.pairs ? norm_kernel<D, true, 4> : norm_kernel<D, false, 4>)
                                : (a.pairs ? norm_kernel<D, true, 1> : norm_kernel<D, false, 1>);
  return launch_chained(kernel, grid, dim3(256), 0, stream, a);
}

}  // namespace

cudaError_t launch_norm(const NormLaunch& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_norm_d<64>(a, stream);
    case 96: return launch_norm_d<96>(a, stream);
    default: return launch_norm_d<128>(a, stream);
  }
}

}  // namespace wise
