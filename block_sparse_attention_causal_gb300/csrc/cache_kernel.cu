// Maintenance of a paged key/value cache: new tokens' keys and values appended
// with the position rotation applied on the way, and the drafted tokens that
// are kept moved up behind the committed ones. (No counterpart in the WISE
// paper: a served model's cache behind its prompt.)
#include "internal.h"
#include "ptx.cuh"

namespace wise {
namespace {

// Element offset in a pool of the row that holds token `slot` of sequence b
// (head 0), or -1 (flagged) when the token does not fit the page table or its
// page is not in the pool.
__device__ __forceinline__ int64_t slot_offset(const CacheView& c, int b, int64_t slot, int d, uint32_t* err) {
  const int64_t col = slot >> c.page_shift;
  if (slot < 0 || col >= c.max_pages) {
    atomicOr(err, kErrBadCache);
    return -1;
  }
  const int32_t pg = c.page_table[(int64_t)b * c.max_pages + col];
  if (pg < 0 || (int64_t)pg >= c.n_pages) {
    atomicOr(err, kErrBadCache);
    return -1;
  }
  const int64_t row = slot & ((1 << c.page_shift) - 1);
  return ((((int64_t)pg * c.kv_heads) << c.page_shift) + row) * d;
}

// Sine and cosine of `turn` / 2^64 turns, each to 2^-22 of its own value. The
// angle is split in whole numbers into quarter turns and a rest of at most an
// eighth of a turn, so that small sines and cosines keep their bits: a pair
// (x, 0) is rotated to bf16's own rounding wherever its angle lies. (The
// hardware's sine is off by 2^-21 whatever its size, 1 % of that of an angle of
// 5e-5, and 32 bits of the angle are too few for the slow pairs of a long
// context.) The rest in fp32 (2.5 roundings) goes into Taylor's series, whose
// next terms are below 2^-25 of the value there: t^11 / 11! and t^12 / 12!.
// Against the hardware's functions, a prompt of 32K takes 121.1 us instead of
// 120.9, 64 tokens 2.8 us instead of 2.7; sincospif after the same split took
// 122.1 and 3.4 us.
__device__ __forceinline__ void sine_cosine(uint64_t turn, float& s, float& c) {
  // the rest as its nearest multiple of 2^32 and a signed remainder, which
  // never cancel by more than half
  const uint32_t hi = (uint32_t)(turn >> 32) + 0x20000000u;
  const int32_t lo = (int32_t)(uint32_t)turn;
  const int32_t top = (int32_t)(hi & 0x3fffffffu) - 0x20000000 + (int32_t)((uint32_t)lo >> 31);
  constexpr float kTurn = 6.28318530717958648f;
  const float t = fmaf((float)top, kTurn * 0x1p-32f, (float)lo * (kTurn * 0x1p-64f));
  const float t2 = t * t;
  const float s0 = fmaf(t * t2, fmaf(t2, fmaf(t2, fmaf(t2, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), t);
  const float c0 =
      fmaf(t2, fmaf(t2, fmaf(t2, fmaf(t2, fmaf(t2, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  // quarters: (s, c), (c, -s), (-s, -c), (-c, s)
  const bool odd = (hi >> 30) & 1u;
  s = __uint_as_float(__float_as_uint(odd ? c0 : s0) ^ (hi & 0x80000000u));
  c = __uint_as_float(__float_as_uint(odd ? s0 : c0) ^ ((hi ^ (hi << 1)) & 0x80000000u));
}

// The two 16-byte chunks of a head that one thread rotates together.
struct ChunkPair {
  uint4 a, b;
};

// (x, y) -> (x c - y s, y c + x s) in fp32, rounded once to bf16. HALVES: x and
// y are the same places of the two chunks (halves rotation); else neighbouring
// values of one chunk, four pairs per chunk.
template <bool PAIRS>
__device__ __forceinline__ void rotate(ChunkPair& p, const float (&c)[8], const float (&s)[8]) {
  uint32_t* a = &p.a.x;
  uint32_t* b = &p.b.x;
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (PAIRS) {
      const float x0 = lo(a[i]), y0 = hi(a[i]), x1 = lo(b[i]), y1 = hi(b[i]);
      a[i] = pack_bf16x2(x0 * c[i] - y0 * s[i], y0 * c[i] + x0 * s[i]);
      b[i] = pack_bf16x2(x1 * c[4 + i] - y1 * s[4 + i], y1 * c[4 + i] + x1 * s[4 + i]);
    } else {
      const int f = 2 * i;
      const float x0 = lo(a[i]), y0 = lo(b[i]), x1 = hi(a[i]), y1 = hi(b[i]);
      a[i] = pack_bf16x2(x0 * c[f] - y0 * s[f], x1 * c[f + 1] - y1 * s[f + 1]);
      b[i] = pack_bf16x2(y0 * c[f] + x0 * s[f], y1 * c[f + 1] + x1 * s[f + 1]);
    }
  }
}

// Bound by memory: each value is read and written once (a prompt of 32K tokens,
// 32/8 heads of 128, 805 MB: 121 us = 6.63 TB/s, 98 % of a copy's rate).
//
// One thread per (token, pair of chunks), walking the heads of q, k and v of
// its token: the sines and cosines of its eight frequencies are computed once
// per token. With few tokens the heads are spread over gridDim.y.
// AHEAD heads are loaded before the first is stored (four where a thread has
// that many: a prompt of 32K took 134 us with one, 128 us with four, 140 us with
// eight; with few tokens the longer code costs more than it gives, 3.4 us
// against 3.1 us). The form with four is held to three blocks per SM: heads of 96
// would otherwise take 92 registers and run two (2 x 4K tokens of 40 heads: 72.5 us
// instead of 64.5). The other form fits four.
template <int D, bool PAIRS, int AHEAD>
__global__ void __launch_bounds__(256, AHEAD == 4 ? 3 : 4) append_kernel(const AppendLaunch p) {
  constexpr int NP = D / 16;  // chunk pairs of a head
  grid_wait();
  grid_trigger();
  const int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t tok = item / NP;
  if (tok >= (int64_t)p.cache.batch * p.n) return;
  const int c = (int)(item % NP);
  const int b = (int)(tok / p.n), i = (int)(tok % p.n);
  const int units = p.heads + 2 * p.cache.kv_heads;
  // element offsets of the thread's two chunks within a head: halves rotation
  // pairs chunk c with chunk c + rotary_dim / 16; everything else takes
  // neighbouring chunks
  const int nrot = p.rotary_dim / 16;
  const bool rot = c < nrot;
  const int ca = (rot && !PAIRS) ? c * 8 : 2 * c * 8;
  const int cb = (rot && !PAIRS) ? (c + nrot) * 8 : ca + 8;
  const int32_t len = p.cache.lengths[b];
  const int32_t nl = p.new_len ? p.new_len[b] : p.n;
  if (len < 0 || nl < 0 || nl > p.n) atomicOr(p.err, kErrBadCache);
  const bool store = len >= 0 && i < nl;
  const int64_t dst = store ? slot_offset(p.cache, b, (int64_t)len + i, D, p.err) : -1;
  const int64_t head_step = (int64_t)D << p.cache.page_shift;
  float cs[8], sn[8];
  const uint16_t* kb = p.k.data + (int64_t)b * p.k.sb + (int64_t)i * p.k.sn;
  const uint16_t* vb = p.v.data + (int64_t)b * p.v.sb + (int64_t)i * p.v.sn;
  for (int u0 = blockIdx.y; u0 < units; u0 += AHEAD * gridDim.y) {
    ChunkPair x[AHEAD];
    uint16_t* out[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int u = u0 + k * gridDim.y;
      const uint16_t* src;
      out[k] = nullptr;
      if (u < p.heads) {
        src = p.q.data + (int64_t)b * p.q.sb + (int64_t)u * p.q.sh + (int64_t)i * p.q.sn;
        out[k] = p.q_out + (((int64_t)b * p.heads + u) * p.n + i) * D;
      } else if (dst >= 0 && u < units) {
        const int h = u - p.heads;
        const bool key = h < p.cache.kv_heads;
        const int hv = key ? h : h - p.cache.kv_heads;
        src = (key ? kb : vb) + (int64_t)hv * (key ? p.k.sh : p.v.sh);
        out[k] = (key ? p.cache.k_pages : p.cache.v_pages) + dst + hv * head_step;
      }
      if (out[k]) {
        // past the L1 cache: each value is read once (through it a prompt of 32K takes 127 us)
        x[k].a = __ldcg(reinterpret_cast<const uint4*>(src + ca));
        x[k].b = __ldcg(reinterpret_cast<const uint4*>(src + cb));
      }
    }
    if (u0 == (int)blockIdx.y && rot) {
      // after the first loads are on their way
      const int64_t pos = p.positions ? (int64_t)p.positions[tok] : (int64_t)len + i;
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        // the angle in units of 2^-64 turn, exact: the low 64 bits of the product
        sine_cosine((uint64_t)pos * (uint64_t)p.rope[8 * c + f], sn[f], cs[f]);
      }
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (!out[k]) continue;
      if (rot && u0 + k * (int)gridDim.y < p.heads + p.cache.kv_heads) rotate<PAIRS>(x[k], cs, sn);
      *reinterpret_cast<uint4*>(out[k] + ca) = x[k].a;
      *reinterpret_cast<uint4*>(out[k] + cb) = x[k].b;
    }
  }
}

// One thread per (sequence, pool, head, 16-byte chunk). The block first looks up
// where the path's tokens lie (up to 128 at a time), then each thread moves its
// chunk of them in order. An entry that is kept ascends and is at least its
// place i: a batch's loads all come before its stores, and the stores of
// earlier entries (slots below i) are never a later entry's source.
// 64 paths of up to 12 tokens: 3.4 us (5.1 us when every thread looked up the
// page table for itself); bound by three loads in a row.
constexpr int kAcceptThreads = 128;
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptLaunch p) {
  constexpr int BATCH = 8;
  __shared__ int64_t from[kAcceptThreads], to[kAcceptThreads];
  grid_wait();
  grid_trigger();
  const int chunks = p.head_dim / 8;
  const int per_seq = 2 * p.cache.kv_heads * chunks;
  const int b = blockIdx.y;
  const int x = blockIdx.x * blockDim.x + threadIdx.x;
  const int32_t len = p.cache.lengths[b];
  int32_t na = p.n_accepted[b];
  const int64_t room = ((int64_t)p.cache.max_pages << p.cache.page_shift) - len;
  if (len < 0 || na < 0 || na > p.path_tokens || na > room) {
    if (x == 0) atomicOr(p.err, kErrBadCache);
    na = len < 0 ? 0 : max(0, (int32_t)min((int64_t)min(na, p.path_tokens), max(room, (int64_t)0)));
  }
  if (x == 0) p.new_lengths[b] = len + na;
  if (p.path == nullptr || len < 0) return;
  const int chunk = x % chunks, hp = x / chunks;
  const int h = hp % p.cache.kv_heads;
  uint16_t* pool = (hp < p.cache.kv_heads ? p.cache.k_pages : p.cache.v_pages) +
                   (((int64_t)h * p.head_dim) << p.cache.page_shift) + chunk * 8;
  const int32_t* path = p.path + (int64_t)b * p.path_tokens;
  for (int i0 = 0; i0 < na; i0 += kAcceptThreads) {
    const int mine = i0 + threadIdx.x;
    int64_t f = -1, t = -1;
    if (mine < na) {
      const int32_t src = path[mine], prev = mine > 0 ? path[mine - 1] : -1;
      if (src <= prev || src < mine) {
        atomicOr(p.err, kErrBadCache);
      } else if (src != mine) {  // else already in its place
        f = slot_offset(p.cache, b, (int64_t)len + src, p.head_dim, p.err);
        t = slot_offset(p.cache, b, (int64_t)len + mine, p.head_dim, p.err);
      }
    }
    from[threadIdx.x] = f;
    to[threadIdx.x] = f < 0 ? -1 : t;
    __syncthreads();
    const int some = min(na - i0, kAcceptThreads);
    if (x < per_seq) {
      for (int i = 0; i < some; i += BATCH) {
        uint4 v[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
          if (i + k < some && to[i + k] >= 0) v[k] = *reinterpret_cast<const uint4*>(pool + from[i + k]);
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
          if (i + k < some && to[i + k] >= 0) *reinterpret_cast<uint4*>(pool + to[i + k]) = v[k];
      }
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t launch_append_d(const AppendLaunch& a, cudaStream_t stream) {
  const int64_t items = (int64_t)a.cache.batch * a.n * (D / 16);
  const int units = a.heads + 2 * a.cache.kv_heads;
  const int64_t blocks = (items + 255) / 256;
  // Heads are spread until the grid holds a full GPU of threads, and on, as long
  // as a thread keeps four of them, to 24 blocks per SM: three run at a time, and
  // the fewer rounds they make the more of the last one is empty (a prompt of 32K:
  // 128 us with 7 blocks per SM, 121 us with 20).
  constexpr int64_t kFull = 152 * 8, kMany = 152 * 24;
  int64_t ny = kMany / blocks < units / 4 ? kMany / blocks : units / 4;
  if (ny < kFull / blocks) ny = kFull / blocks;
  ny = ny < 1 ? 1 : (ny > units ? units : ny);
  const dim3 grid((unsigned)blocks, (unsigned)ny);
  auto kernel = ny * 4 <= units ? (a.pairs ? append_kernel<D, true, 4> : append_kernel<D, false, 4>)
                                : (a.pairs ? append_kernel<D, true, 1> : append_kernel<D, false, 1>);
  return launch_chained(kernel, grid, dim3(256), 0, stream, a);
}

}  // namespace

cudaError_t launch_cache_append(const AppendLaunch& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_append_d<64>(a, stream);
    case 96: return launch_append_d<96>(a, stream);
    default: return launch_append_d<128>(a, stream);
  }
}

cudaError_t launch_cache_accept(const AcceptLaunch& a, cudaStream_t stream) {
  const int per_seq = 2 * a.cache.kv_heads * (a.head_dim / 8);
  const dim3 grid((unsigned)((per_seq + kAcceptThreads - 1) / kAcceptThreads), (unsigned)a.cache.batch);
  return launch_chained(accept_kernel, grid, dim3(kAcceptThreads), 0, stream, a);
}

}  // namespace wise
