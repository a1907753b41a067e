// Shared parts of the kernels that write new tokens' rows: slots of the paged
// cache, and the position rotation.
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace wise {

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

}  // namespace wise
