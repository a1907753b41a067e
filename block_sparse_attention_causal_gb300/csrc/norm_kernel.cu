// Queries and keys normed per head and rotated by their positions in one pass:
//   y = x / sqrt(mean(x^2) + eps) * w          over a head's values,
//   (y1, y2) -> (y1 cos a - y2 sin a, y2 cos a + y1 sin a), a = 2 pi frac(position step / 2^64),
// into a paged cache (keys; values are copied) or into dense rows before a
// prompt's attention. A position may have several axes (time, row and column of
// an image), each pair of values turning with one of them.
#include "rotate.cuh"

namespace wise {
namespace {

constexpr int kStages = 4;   // heads under way in shared memory (2: 126 us for a prompt of 32K, 4: 121, 6 and 8 the same)
constexpr int kHeads = 16;   // heads of a block at most (8, 16, 32: 121.9, 121.2, 121.0 us; an image's 71, 64, 66)
static_assert(kMaxNormHeads / kHeads + 3 <= 65535, "the grid's second axis");

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

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

// Eight bf16 values as four pairs of fp32.
__device__ __forceinline__ void widen8(const uint4& v, uint64_t (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 narrow8(const uint64_t (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(x[i], lo, hi);
    w[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t swap2(uint64_t a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return f2_pack(hi, lo);
}
// Eight weights from element `at` on.
__device__ __forceinline__ void weights8(const NormLaunch& p, const void* w, int64_t at, uint64_t (&x)[4]) {
  if (p.weight_f32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 a = f[0], b = f[1];
    x[0] = f2_pack(a.x, a.y), x[1] = f2_pack(a.z, a.w), x[2] = f2_pack(b.x, b.y), x[3] = f2_pack(b.z, b.w);
  } else {
    widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + at), x);
  }
}

// One thread per (token, two 16-byte chunks of a head), walking some of the heads
// of one kind (queries, keys or values) of its token, so that sines, cosines and
// weights are taken once: they are multiplied into each other beforehand, and a
// pair costs four products, the root's factor comes last. A token's D / 16 threads
// are lanes of one warp (heads of 96: five tokens a warp, two lanes idle) and sum
// the squares among themselves. Arithmetic is on pairs of fp32.
// STAGES heads are under way at a time, each thread's own chunks in its own slots of
// shared memory (nothing to synchronise, and registers for three blocks per SM: with
// four heads ahead in registers, two blocks, a prompt of 32K took 127 us); STAGES 1:
// one, in registers.
//
// Bound by memory: a prompt of 32K tokens, 32/8 heads of 128, 805 MB, takes 121.2 us
// (6.64 TB/s, 98 % of a copy's rate; without norms cache_kernel.cu's 121); 16K tokens of
// 32/32 heads, dense, 84.6 us (94 %); 2 x 4K of an image, 40 heads of 96 with weights of
// their own and three axes, 64 us (79 %). 64 tokens: 3.6 us, latency.
template <int D, bool PAIRS, int STAGES>
__global__ void __launch_bounds__(256, 3) norm_kernel(const NormLaunch p) {
  constexpr int G = D / 16, TOKENS = 32 / G;  // lanes of a token, tokens of a warp
  grid_wait();
  grid_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t tok = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * TOKENS + lane / G;
  const bool on = lane < TOKENS * G && tok < (int64_t)p.batch * p.n;
  const int c = lane % G;
  const int b = on ? (int)(tok / p.n) : 0, i = on ? (int)(tok % p.n) : 0;
  // queries, keys, values: the block's kind, and its heads
  const int part = blockIdx.y;
  const int kind = part < p.parts[0] ? 0 : part < p.parts[0] + p.parts[1] ? 1 : 2;
  const int heads = kind == 0 ? p.heads : p.kv_heads;
  const int h0 = (part - (kind > 0 ? p.parts[0] : 0) - (kind > 1 ? p.parts[1] : 0)) * p.part_heads;
  const int h1 = min(h0 + p.part_heads, heads);
  // element offsets of the thread's two chunks within a head, a half apart (lanes
  // next to each other read next to each other); rotation by halves pairs chunk c
  // with chunk c + rotary_dim / 16, and chunks behind those with their neighbours
  const int nrot = p.rotary_dim / 16;
  const bool apart = PAIRS || 2 * nrot == D / 8 || nrot == 0;
  const int ca = apart || c < nrot ? c * 8 : 2 * c * 8;
  const int cb = apart ? ca + D / 2 : c < nrot ? (c + nrot) * 8 : ca + 8;
  const bool rot_a = kind < 2 && ca < p.rotary_dim, rot_b = kind < 2 && cb < p.rotary_dim;  // (the same for halves)
  int32_t len = 0;
  int64_t dst = -1;  // the token's row of head 0
  if (kind == 0) {
    dst = ((int64_t)b * p.heads * p.n + i) * D;
  } else if (!p.paged) {
    dst = ((int64_t)b * p.kv_heads * p.n + i) * D;
  }
  if (p.paged) {
    len = p.cache.lengths[b];
    const int32_t nl = p.new_len ? p.new_len[b] : p.n;
    if (on && (len < 0 || nl < 0 || nl > p.n)) atomicOr(p.err, kErrBadCache);
    if (kind > 0 && on && len >= 0 && i < nl) dst = slot_offset(p.cache, b, (int64_t)len + i, D, p.err);
  }
  const bool live = on && dst >= 0;
  const int64_t out_step = kind > 0 && p.paged ? (int64_t)D << p.cache.page_shift : (int64_t)p.n * D;
  const RowsView& src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
  uint16_t* out = (kind == 0 ? p.q_out : kind == 1 ? p.k_out : p.v_out) + dst;
  const uint16_t* from = src.data + (int64_t)b * src.sb + (int64_t)i * src.sn;
  const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  const int64_t weight_step = kind == 0 ? p.q_weight_stride : p.k_weight_stride;
  extern __shared__ uint4 slots[];  // [STAGES][2][256]
  float* head_weights = reinterpret_cast<float*>(slots + (STAGES > 1 ? STAGES * 512 : 0));  // [the block's heads][D]
  uint4* mine = slots + threadIdx.x;
  uint4 ra = make_uint4(0u, 0u, 0u, 0u), rb = ra;
  auto load = [&](int u) {
    // past the L1 cache: each value is read once
    const uint16_t* at = from + (int64_t)u * src.sh;
    if constexpr (STAGES > 1) {
      uint4* to = mine + (u - h0) % STAGES * 512;
      if (live && u < h1) {
        copy16(to, at + ca);
        copy16(to + 256, at + cb);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else if (live && u < h1) {
      ra = __ldcg(reinterpret_cast<const uint4*>(at + ca));
      rb = __ldcg(reinterpret_cast<const uint4*>(at + cb));
    }
  };
#pragma unroll
  for (int k = 0; k < STAGES; ++k) load(h0 + k);
  // after the first loads are on their way: for chunk a (b) the factors of its own
  // values and, where it is rotated, of those they are turned with
  uint64_t fa[4], ga[4], fb[4], gb[4];
  const uint64_t one = f2_pack(1.f, 1.f);
#pragma unroll
  for (int f = 0; f < 4; ++f) fa[f] = fb[f] = one, ga[f] = gb[f] = 0ull;
  if (on && weight && weight_step == 0) {
    weights8(p, weight, ca, fa);
    weights8(p, weight, cb, fb);
  }
  if (weight && weight_step != 0) {
    // the weights of the block's heads, in fp32
    for (int x = threadIdx.x; x < (h1 - h0) * (D / 8); x += 256) {
      const int h = x / (D / 8), e = x % (D / 8) * 8;
      uint64_t w[4];
      weights8(p, weight, (h0 + h) * weight_step + e, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) *reinterpret_cast<uint64_t*>(head_weights + h * D + e + 2 * k) = w[k];
    }
    __syncthreads();
  }
  if (on && (rot_a || rot_b)) {
    // the thread's eight pairs: the first four of chunk a and of chunk b
    // (neighbouring pairs), or the eight of chunk a (halves)
    int pair[8];
    int64_t pos[8];
    uint64_t step[8];
    float s[8], co[8];
    bool known = true;
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      pair[f] = PAIRS ? (f < 4 ? ca : cb) / 2 + (f & 3) : ca + f;
      if (PAIRS && !(f < 4 ? rot_a : rot_b)) pair[f] = 0;  // (not used)
      pos[f] = (int64_t)len + i;
    }
    // loads of one kind together, so that they are under way at the same time
    if (p.axes) {
      int axis[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) axis[f] = p.axes[pair[f]];
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        const bool in = axis[f] >= 0 && axis[f] < p.n_axes;
        known &= in;
        pos[f] = in ? p.positions[((int64_t)axis[f] * p.batch + b) * p.n + i] : 0;
      }
    } else if (p.positions) {
      const int32_t at = p.positions[(int64_t)b * p.n + i];
#pragma unroll
      for (int f = 0; f < 8; ++f) pos[f] = at;
    }
#pragma unroll
    for (int f = 0; f < 8; ++f) step[f] = (uint64_t)p.rope[pair[f]];
    if (!known) atomicOr(p.err, kErrBadCache);
#pragma unroll
    for (int f = 0; f < 8; ++f) sine_cosine((uint64_t)pos[f] * step[f], s[f], co[f]);
    if constexpr (PAIRS) {
      auto chunk = [&](int f0, uint64_t (&own)[4], uint64_t (&other)[4]) {
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          float w1, w2;
          f2_unpack(own[f], w1, w2);
          own[f] = f2_pack(w1 * co[f0 + f], w2 * co[f0 + f]);
          other[f] = f2_pack(-(w2 * s[f0 + f]), w1 * s[f0 + f]);
        }
      };
      if (rot_a) chunk(0, fa, ga);
      if (rot_b) chunk(4, fb, gb);
    } else {
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        float w0, w1, v0, v1;
        f2_unpack(fa[f], w0, w1);
        f2_unpack(fb[f], v0, v1);
        fa[f] = f2_pack(w0 * co[2 * f], w1 * co[2 * f + 1]);
        ga[f] = f2_pack(-(v0 * s[2 * f]), -(v1 * s[2 * f + 1]));
        fb[f] = f2_pack(v0 * co[2 * f], v1 * co[2 * f + 1]);
        gb[f] = f2_pack(w0 * s[2 * f], w1 * s[2 * f + 1]);
      }
    }
  }
#pragma unroll 1
  for (int u = h0; u < h1; ++u) {
    if constexpr (STAGES > 1) {
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      const uint4* at = mine + (u - h0) % STAGES * 512;
      if (live) {
        ra = at[0];
        rb = at[256];
      }
    } else if (u > h0) {
      load(u);
    }
    if (kind < 2) {
      uint64_t x[4], y[4];
      widen8(ra, x);
      widen8(rb, y);
      if constexpr (STAGES > 1) load(u + STAGES);
      uint64_t inv2 = one;
      if (weight) {
        uint64_t ss = 0ull;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = ffma2(x[e], x[e], ss);
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = ffma2(y[e], y[e], ss);
        float s0, s1;
        f2_unpack(ss, s0, s1);
        const float inv = rsqrtf(token_sum<G>(s0 + s1, lane) * (1.f / D) + p.eps);
        inv2 = f2_pack(inv, inv);
        if (weight_step != 0) {
          const float* w = head_weights + (u - h0) * D;
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const ulonglong2 wa = *reinterpret_cast<const ulonglong2*>(w + ca + 2 * e);
            const ulonglong2 wb = *reinterpret_cast<const ulonglong2*>(w + cb + 2 * e);
            x[e] = fmul2(x[e], wa.x), x[e + 1] = fmul2(x[e + 1], wa.y);
            y[e] = fmul2(y[e], wb.x), y[e + 1] = fmul2(y[e + 1], wb.y);
          }
        }
      }
      uint64_t ox[4], oy[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ox[e] = fmul2(x[e], fa[e]);
        oy[e] = fmul2(y[e], fb[e]);
      }
      // (values that do not turn are not added 0 times others: those may be infinite)
      if (rot_a) {
#pragma unroll
        for (int e = 0; e < 4; ++e) ox[e] = ffma2(PAIRS ? swap2(x[e]) : y[e], ga[e], ox[e]);
      }
      if (rot_b) {
#pragma unroll
        for (int e = 0; e < 4; ++e) oy[e] = ffma2(PAIRS ? swap2(y[e]) : x[e], gb[e], oy[e]);
      }
      if (weight) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ox[e] = fmul2(ox[e], inv2);
          oy[e] = fmul2(oy[e], inv2);
        }
      }
      ra = narrow8(ox);
      rb = narrow8(oy);
    }
    if (live) {
      *reinterpret_cast<uint4*>(out + u * out_step + ca) = ra;
      *reinterpret_cast<uint4*>(out + u * out_step + cb) = rb;
    }
    if constexpr (STAGES > 1)
      if (kind == 2) load(u + STAGES);
  }
}

template <int D>
cudaError_t launch_norm_d(NormLaunch a, cudaStream_t stream) {
  constexpr int TOKENS = 32 / (D / 16) * 8;  // of a block
  const int64_t blocks = ((int64_t)a.batch * a.n + TOKENS - 1) / TOKENS;
  const int q = a.heads, k = a.k.data ? a.kv_heads : 0, v = a.v.data ? a.kv_heads : 0;
  auto parts = [&](int each) {
    a.part_heads = each;
    a.parts[0] = (q + each - 1) / each;
    a.parts[1] = (k + each - 1) / each;
    return a.parts[0] + a.parts[1] + (v + each - 1) / each;
  };
  // Fewer heads a block (each takes its sines and cosines again) only until there
  // are two blocks per SM: 2K tokens take 12.3 us so, 14.4 with one or four per SM.
  int each = kHeads;
  while (each > 1 && blocks * parts(each) < 152 * 2) each /= 2;
  const dim3 grid((unsigned)blocks, (unsigned)parts(each));
  const bool staged = each >= 4;
  auto kernel = staged ? (a.pairs ? norm_kernel<D, true, kStages> : norm_kernel<D, false, kStages>)
                       : (a.pairs ? norm_kernel<D, true, 1> : norm_kernel<D, false, 1>);
  const size_t smem = (staged ? kStages * 2 * 256 * sizeof(uint4) : 0) +
                      (a.q_weight_stride != 0 || a.k_weight_stride != 0 ? (size_t)each * D * sizeof(float) : 0);
  return launch_chained(kernel, grid, dim3(256), smem, stream, a);
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
