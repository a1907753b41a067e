// Attention of new tokens over a paged cache (tree.cuh) for units of up to 64
// rows: next tokens and small trees, whose bound is the cache's bytes.
//
// The tiles are turned round, so that the few rows are the MMAs' narrow side
// and the 128 keys fill the tensor core's rows and the softmax's threads:
//   S^T[key, row] = K Q^T     A = K tile (128 keys), B = Q (N rows)
//   O^T[dim, row] += V^T P^T  A = V tile read along its keys, B = P (N rows)
// with N = 16, 32 or 64. A tile then costs the tensor core 2 D / 16 + 16 MMAs
// of N columns and each softmax thread (one key) N exponentials, a fraction of
// the time in which its bytes arrive; rows-as-lanes tiles of 128 took longer
// than the bytes (one warp worked, 128 scores in each of its lanes).
//
// Measured (one GB300): next tokens of 32 sequences of up to 8K, 32/8 heads of
// 128, 657 MB: 105 us = 6.25 TB/s, 92 % of a copy's rate; one of 128K, 537 MB:
// 84 us, 94 %. A short prompt's next token takes 9.8 us, latency throughout.
//
// The row maximum goes over threads here. It need not be exact: a row's
// reference only moves when a score passes it by 2^8, so per tile a vote over
// the block of four warps is enough, and only a segment's first tile and the
// rare jumps reduce a maximum. The sums stay per thread until the segment ends.
//
// Warp roles (256 threads): 0 TMA, 1 guard of V, 2 MMA issue, 3 Q, 4-7 softmax
// (one key per thread) and results (one dimension per thread).
// TMEM: S^T_0 | S^T_1 | O^T, N columns each.
#pragma once
#include "tree.cuh"

namespace wise {
namespace {

constexpr int kNarrowThreads = 256;
// Leaves room for a waiting block of the join kernel (N of 16 and 32; with 64 the
// registers leave none).
constexpr uint32_t kSmemLimit = 232448u - 6144u;

template <int D, int N>
struct NarrowCfg {
  static constexpr int NP = (N == 64) ? 1 : 2;  // P buffers
  static constexpr uint32_t Q_BYTES = tile_bytes<D>(N);
  static constexpr uint32_t P_BYTES = (uint32_t)N * kTile * 2u;
  static constexpr uint32_t KV_BYTES = tile_bytes<D>(kTile);
  static constexpr int NS_MAX = 12;
  static constexpr int NBAR = 12 + 3 * NS_MAX;
  // thr[N], ref[N], fac[N], res[N], offs[N], wmax[4][N], wsum[4][N]; seen[2][64][2]; words[128]; nf; barriers; words
  static constexpr uint32_t SMALL = 14u * N * 4u + 2u * 64u * 8u + 128u * 4u + kNfRing * 16u + NBAR * 8u + (NS_MAX + kTileFlags) * 4u + 40u * 4u;
  static constexpr uint32_t FIXED = 2u * Q_BYTES + NP * P_BYTES + SMALL;
  static constexpr int NS_FIT = (int)((kSmemLimit - FIXED) / KV_BYTES);
  static constexpr int NS = NS_FIT < NS_MAX ? NS_FIT : NS_MAX;
  static_assert(NS >= 4, "ring");
  static constexpr uint32_t OFF_Q = NS * KV_BYTES;
  static constexpr uint32_t OFF_P = OFF_Q + 2u * Q_BYTES;
  static constexpr uint32_t OFF_SMALL = OFF_P + NP * P_BYTES;
  // the MMA's 128 rows of V^T read on past a tile of fewer dimensions; what
  // they find only reaches rows of O^T that nobody reads
  static constexpr uint32_t OVER = (D == 64) ? KV_BYTES : 0u;
  static constexpr uint32_t USED = OFF_SMALL + SMALL;
  static constexpr uint32_t SMEM_BYTES = USED > OFF_Q + OVER ? USED : OFF_Q + OVER;
  static_assert(SMEM_BYTES <= kSmemLimit, "shared memory");
  static_assert(Q_BYTES % 1024 == 0 && P_BYTES % 1024 == 0 && OFF_SMALL % 16 == 0, "swizzle atoms");
  static constexpr uint32_t TMEM_COLS = (N == 16) ? 64u : (N == 32) ? 128u : 256u;
};

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// N consecutive 32-bit columns of this thread's TMEM lane.
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t t, uint32_t (&r)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += 16) tmem_ld_x16(t + c, *reinterpret_cast<uint32_t(*)[16]>(&r[c]));
#pragma unroll
  for (int c = 0; c < N; c += 16) tmem_wait_ld16(*reinterpret_cast<uint32_t(*)[16]>(&r[c]));
}

// 8 columns, loaded and waited for.
__device__ __forceinline__ void tmem_ld_x8(uint32_t t, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(t)
      : "memory");
}

// Sums of N values over the warp's lanes by halving: each step sends half of
// the values away and adds what comes back. Afterwards lane x holds the sums
// of rows row_of(x) (N = 64: two of them).
template <int N>
__device__ __forceinline__ void warp_sums(const float (&x)[N], float* out, int lane) {
  constexpr int OFF = (N == 64) ? 16 : (N == 32) ? 16 : 8;
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = x[i];
  if (N == 16) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
  }
  int row = 0;
  int have = N;
#pragma unroll
  for (int o = OFF; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
    have >>= 1;
    if (up) row += have;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if (i < have) {
        const float send = up ? v[i] : v[i + have];
        const float keep = up ? v[i + have] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
  }
  if (N == 16 && lane >= 16) return;
  out[row] = v[0];
  if (N == 64) out[row + 1] = v[1];
}

template <int D, int N, bool PREFIX>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    tree_narrow_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const TreeParams p) {
  using C = NarrowCfg<D, N>;
  using R = RingCfg<D, C::NS>;
  constexpr int NS = C::NS, NP = C::NP;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* thr = reinterpret_cast<float*>(smem + C::OFF_SMALL);  // [N] scores above it move the row's reference
  float* ref = thr + N;                                        // [N] the row's reference (log2 domain)
  float* fac = ref + N;                                        // [N] factor of a moved reference
  float* res = fac + N;                                        // [N] factor of the results (< 0: the row sees nothing)
  int64_t* offs = reinterpret_cast<int64_t*>(res + N);         // [N] the row's place in the outputs
  float* wmax = reinterpret_cast<float*>(offs + N);                                       // [4][N]
  float* wsum = wmax + 4 * N;                                  // [4][N]
  uint32_t* seen = reinterpret_cast<uint32_t*>(wsum + 4 * N);  // [2][64][2] rows that see drafted token j (of even and odd segments)
  uint32_t* words = seen + 256;                                // [128] mask words of the segment
  uint32_t* nf = words + 128;                                   // [kNfRing][4]
  uint64_t* bars = reinterpret_cast<uint64_t*>(nf + kNfRing * 4);
  uint64_t* q_full = bars;         // [2] Q of a segment loaded
  uint64_t* q_empty = bars + 2;    // [2] its last S MMA done
  uint64_t* s_full = bars + 4;     // [2] S^T computed
  uint64_t* s_empty = bars + 6;    // [2] S^T read (4 warps)
  uint64_t* p_full = bars + 8;     // [NP] P written (4 warps)
  uint64_t* p_empty = bars + 10;   // [NP] PV MMA done
  Ring ring;
  ring.tiles = smem;
  ring.full = bars + 12;
  ring.empty = ring.full + C::NS_MAX;
  ring.guarded = ring.empty + C::NS_MAX;
  ring.uses = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  ring.flags = ring.uses + C::NS_MAX;
  uint32_t* misc = ring.flags + kTileFlags;
  uint32_t* tmem_base_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  int* scratch = reinterpret_cast<int*>(misc + 4);  // [8 + 12]
  uint32_t* err = p.t.err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if ((smem_u32(smem) & 1023u) != 0u) {  // swizzled tiles
    grid_wait();
    clear_recs(p);
    if (threadIdx.x == 0) atomicOr(err, kErrInternal);
    return;
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_empty[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&ring.full[i], 1);
      mbar_init(&ring.empty[i], 1);
      mbar_init(&ring.guarded[i], 1);
      ring.uses[i] = 0u;
    }
    for (int i = 0; i < kTileFlags; ++i) ring.flags[i] = 0u;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  prefetch_tables(p);
  const int blocks = wait_at_start<PREFIX>(p.t, misc + 2);
  if (!PREFIX && blocks < 0) {
    clear_recs(p);
    if (threadIdx.x == 0) atomicOr(err, kErrInternal);
  }
  if ((int)blockIdx.x >= blocks) {
    grid_trigger();
    wait_at_end<PREFIX>(p.t);
    return;
  }
  // tensor memory only now: a kernel before this one that still runs could wait
  // for what this one holds
  if (warp == 2) {
    tmem_alloc(tmem_base_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  grid_trigger();
  LinePart part;
  find_part<kNarrowThreads, PREFIX>(p, scratch, part, blocks);
  const uint32_t tbase = *tmem_base_slot;
  if (threadIdx.x == 128) clear_rec(p);
  WalkOf<PREFIX> w;
  if (part.left > 0) {
    w.start(p, part);
    if (warp == 0) {
      ring_producer<D, NS, 1>(p, w, ring, &tm_k, &tm_v, abort_flag, lane);
    } else if (warp == 1) {
      ring_guard<D, NS, 1>(p, w, ring, nf, abort_flag, lane);
    } else if (warp == 2) {
      // ------------------------------------------------------------ MMA issue
      // One thread; whichever is ready next: S^T of the next tile (up to two
      // tiles ahead of PV, so that it is there when the softmax comes to it),
      // or PV of the oldest tile.
      if (elect_one()) {
        constexpr uint32_t IDESC_S = idesc_bf16_f32(128, N, 0, 0);
        constexpr uint32_t IDESC_O = idesc_bf16_f32(128, N, 1, 0);
        const uint64_t ring_k = smem_desc(smem_u32(smem), 16, 8 * kRowBytes, kSwizzle128);
        const uint64_t ring_v = smem_desc(smem_u32(smem), kTile * kRowBytes, 8 * kRowBytes, kSwizzle128);
        const uint64_t q_desc = smem_desc(smem_u32(smem + C::OFF_Q), 16, 8 * kRowBytes, kSwizzle128);
        const uint64_t p_desc = smem_desc(smem_u32(smem + C::OFF_P), 16, 8 * kRowBytes, kSwizzle128);
        const uint32_t dO = tbase + 2 * N;
        uint32_t ts = 0, tp = 0;  // tiles whose S and PV are issued
        bool more = true;         // tiles whose S is not
        WalkOf<PREFIX> ws = w, wp = w;
        int s_at = w.t0, p_at = w.t0;  // tiles within the segments
        uint64_t t0 = 0;
        uint32_t idle = 0;  // rounds without work
        bool ok = true;
        while ((more || tp < ts) && ok) {
          bool moved = false;
          if (more && ts < tp + 2u) {
            const uint32_t pos = 2u * ts;
            const int slot = (int)(pos % NS);
            const bool head = s_at == ws.t0;
            if ((ts < 2u || mbar_test_wait(&s_empty[ts & 1], ((ts >> 1) - 1) & 1)) &&
                (!head || mbar_test_wait(&q_full[ws.seg & 1], (ws.seg >> 1) & 1)) &&
                mbar_test_wait(&ring.full[slot], (pos / NS) & 1)) {
              tc_fence_after();
              const uint64_t kd = ring_k + (uint64_t)((slot * C::KV_BYTES) >> 4);
              const uint64_t qd = q_desc + (uint64_t)(((ws.seg & 1) * C::Q_BYTES) >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const int c = kk / 4, wd = kk % 4;
                umma_ss(tbase + (ts & 1) * N, kd + (uint64_t)((c * kTile * kRowBytes + wd * 32) >> 4),
                        qd + (uint64_t)((c * N * kRowBytes + wd * 32) >> 4), IDESC_S, kk > 0);
              }
              umma_commit(&s_full[ts & 1]);
              umma_commit(&ring.empty[slot]);
              ++ts;
              if (++s_at == ws.t1) {
                umma_commit(&q_empty[ws.seg & 1]);
                more = ws.next(p);
                s_at = ws.t0;
              }
              moved = true;
            }
          }
          if (tp < ts) {
            const uint32_t pos = 2u * tp + 1u;
            const int slot = (int)(pos % NS);
            if (mbar_test_wait(&p_full[tp % NP], (tp / NP) & 1) && mbar_test_wait(&ring.full[slot], (pos / NS) & 1) &&
                mbar_test_wait(&ring.guarded[slot], R::guard_phase(pos) & 1)) {
              tc_fence_after();
              const uint64_t vd = ring_v + (uint64_t)((slot * C::KV_BYTES) >> 4);
              const uint64_t pd = p_desc + (uint64_t)(((tp % NP) * C::P_BYTES) >> 4);
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                umma_ss(dO, vd + (uint64_t)((kk * 16 * kRowBytes) >> 4),
                        pd + (uint64_t)(((kk / 4) * N * 128 + (kk % 4) * 32) >> 4), IDESC_O,
                        (p_at == wp.t0 && kk == 0) ? 0u : 1u);
              umma_commit(&ring.empty[slot]);
              umma_commit(&p_empty[tp % NP]);
              ++tp;
              if (++p_at == wp.t1) {
                wp.next(p);
                p_at = wp.t0;
              }
              moved = true;
            }
          }
          if (moved) {
            idle = 0;
          } else if ((++idle & 63u) == 0u) {
            if (idle == 64u) t0 = global_timer_ns();
            if (*abort_flag) {
              ok = false;
            } else if (global_timer_ns() - t0 > kWaitLimitNs) {
              *abort_flag = 1;
              atomicOr(err, kErrTimeout);
              ok = false;
            }
          }
        }
        // every MMA of this thread done before TMEM and shared memory go
        int none = 0;
        if (ts > 0) mbar_wait<1>(&s_full[(ts - 1) & 1], ((ts - 1) >> 1) & 1, &none, err);
        if (tp > 0) mbar_wait<1>(&p_empty[(tp - 1) % NP], ((tp - 1) / NP) & 1, &none, err);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ------------------------------------------------------------------- Q
      // Rows of the segment's unit, swizzled as TMA would write them; rows past
      // the last are zero (what lay there could be read as large scores).
      bool ok = true;
      do {
        const int buf = w.seg & 1;
        if (w.seg >= 2) ok = __all_sync(0xffffffffu, mbar_wait<1>(&q_empty[buf], ((w.seg >> 1) - 1) & 1, abort_flag, err));
        if (!ok) break;
        uint8_t* sq = smem + C::OFF_Q + buf * C::Q_BYTES;
        // each lane copies one row, or the lanes of a half-warp half of it
        constexpr int HALVES = N == 16 ? 2 : 1, ROWS = 32 / HALVES, UNITS = D / 8 / HALVES;
#pragma unroll 1
        for (int r = lane % ROWS; r < N; r += ROWS) {
          const int tok = row_token(p, r), g = r - tok * p.group, u0 = lane / ROWS * UNITS;
          const RowPlace at = row_place<PREFIX>(p.t, w.b, tok);
          const uint16_t* src = p.t.q.data + (int64_t)at.b * p.t.q.sb + ((int64_t)w.hk * p.group + g) * p.t.q.sh +
                                (int64_t)at.i * p.t.q.sn + u0 * 8;
#pragma unroll
          for (int i = 0; i < UNITS; ++i) {
            uint8_t* dst = sq + unit_offset(N, r, u0 + i);
            if (r < w.rows(p)) copy16(dst, src + i * 8);
            else *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        copy16_wait();
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[buf]);
      } while (w.next(p));
      __syncwarp();
    } else {
      // ----------------------------------------------------- softmax, results
      const int quarter = warp & 3;
      const int key = quarter * 32 + lane;  // key of the tile, dimension of the results
      const int tid = key;
      const uint32_t trow = tbase + (static_cast<uint32_t>(quarter * 32) << 16);
      const uint32_t tO = trow + 2 * N;
      const float sl2 = p.scale_log2;
      const int page_shift = p.t.cache.page_shift;
      // P[row][key] as the B operand: 64 keys per 128-byte swizzled row
      uint8_t* p_key = smem + C::OFF_P + (key >> 6) * N * 128;
      const uint32_t p_col = (uint32_t)(key & 63) * 2u;
      uint32_t tau = 0;
      bool ok = true;
      do {
        const bool tail = w.t1 * kTile > w.len;
        uint32_t* sees = seen + (w.seg & 1) * 128;
        // the mask's words, one per thread (at most 64 tokens of two words)
        if (tail && p.t.tree_mask && tid < w.nl * p.mask_words)
          words[tid] = (uint32_t)p.t.tree_mask[(int64_t)w.b * p.t.n * p.mask_words + tid];
        if (tail) {
          bar_or(1, 128, false);
          // turned round: the rows that see each drafted token
          if (tid < w.nl) {
            const int j = tid;
            uint64_t m = ~0ull << (j * p.group);
            if (p.t.tree_mask) {
              const uint64_t token = (p.group == 64) ? ~0ull : (1ull << p.group) - 1ull;
              m = 0ull;
#pragma unroll 1
              for (int i = 0; i < w.nl; ++i)
                if ((words[i * p.mask_words + (j >> 5)] >> (j & 31)) & 1u) m |= token << (i * p.group);
            }
            sees[2 * j] = (uint32_t)m;
            sees[2 * j + 1] = (uint32_t)(m >> 32);
          }
          bar_or(1, 128, false);
        }
        float l[N];
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = 0.f;
        for (int t = w.t0; t < w.t1; ++t, ++tau) {
          const int buf = (int)(tau & 1u);
          ok = __all_sync(0xffffffffu, mbar_wait<1>(&s_full[buf], (tau >> 1) & 1, abort_flag, err));
          uint32_t s[N];
          if (ok) {
            tc_fence_after();
            tmem_ld_n<N>(trow + buf * N, s);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[buf]);
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = 0u;
          }
          const int kb = t * kTile;
          const uint32_t bad = tile_bad<1>(ring, tau, abort_flag, err);
          if (kb + kTile > w.len || bad != 0u) {
            const int pos = kb + key;
            uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;
            if (pos >= w.len) {
              const int j = pos - w.len;
              m0 = (pos < w.keys) ? sees[2 * j] : 0u;
              m1 = (pos < w.keys) ? sees[2 * j + 1] : 0u;
            }
            if ((bad >> (key >> page_shift)) & 1u) m0 = m1 = 0u;  // a page outside the pool
#pragma unroll
            for (int i = 0; i < N; ++i)
              s[i] = (((i < 32 ? m0 : m1) >> (i & 31)) & 1u) ? s[i] : __float_as_uint(-INFINITY);
          }
          const bool head = t == w.t0;
          bool over = head || !ok;
          if (!head) {
#pragma unroll
            for (int c = 0; c < N; c += 4) {
              const float4 t4 = *reinterpret_cast<const float4*>(thr + c);
              over |= __uint_as_float(s[c]) * sl2 > t4.x || __uint_as_float(s[c + 1]) * sl2 > t4.y ||
                      __uint_as_float(s[c + 2]) * sl2 > t4.z || __uint_as_float(s[c + 3]) * sl2 > t4.w;
            }
          }
          // (also the barrier between the tiles' uses of the small arrays)
          if (bar_or(1, 128, over)) {
            // some row's reference moves
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float m = warp_max(__uint_as_float(s[i]));
              if (lane == (i & 31)) wmax[quarter * N + i] = m * sl2;
            }
            const bool failed = bar_or(1, 128, !ok);
            if (failed) {
              ok = false;
              break;
            }
            if (tid < N) {
              const float m = fmaxf(fmaxf(wmax[tid], wmax[N + tid]), fmaxf(wmax[2 * N + tid], wmax[3 * N + tid]));
              float f = 1.f;
              if (head) {
                thr[tid] = m + 8.f;
                ref[tid] = (m == -INFINITY) ? 0.f : m;
              } else if (m > thr[tid]) {
                // from "nothing seen yet" (its sum and O are 0) or from a lower one
                f = (thr[tid] == -INFINITY) ? 0.f : fast_exp2(ref[tid] - m);
                thr[tid] = m + 8.f;
                ref[tid] = m;
              }
              fac[tid] = f;
            }
            if (!head)  // O^T holds every PV so far once the last one is done
              ok = __all_sync(0xffffffffu, mbar_wait<1>(&p_empty[(tau - 1) % NP], ((tau - 1) / NP) & 1, abort_flag, err));
            if (bar_or(1, 128, !ok)) {
              ok = false;
              break;
            }
            if (!head) {
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < N; c += 16) {
                uint32_t o[16];
                tmem_ld_x16(tO + c, o);
                tmem_wait_ld16(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float f = fac[c + i];
                  o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  l[c + i] *= f;
                }
                tmem_st_x16(tO + c, o);
              }
              tmem_wait_st();
            }
          }
          // P = 2^(s scale log2e - ref), rounded to bf16 (2^-8) for the tensor core,
          // whose operands are both of V's type; the sum is of the fp32 values
          if (tau >= (uint32_t)NP)
            ok = __all_sync(0xffffffffu, mbar_wait<1>(&p_empty[tau % NP], (tau / NP - 1) & 1, abort_flag, err));
          uint8_t* pk = p_key + (tau % NP) * C::P_BYTES;
#pragma unroll
          for (int c = 0; c < N; c += 16) {
            // the references of 16 rows first: a load between the stores of P
            // would wait for the store before it
            float r[16];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 r4 = *reinterpret_cast<const float4*>(ref + c + i);
              r[i] = r4.x, r[i + 1] = r4.y, r[i + 2] = r4.z, r[i + 3] = r4.w;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = fast_exp2(fmaf(__uint_as_float(s[c + i]), sl2, -r[i]));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              l[c + i] += r[i];
              *reinterpret_cast<uint16_t*>(pk + (c + i) * 128 + (p_col ^ ((i & 7) << 4))) = (uint16_t)pack_bf16x2(r[i], 0.f);
            }
          }
          fence_proxy_async();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[tau % NP]);
        }
        // sums over the keys, and the factor of each row's results
        if (ok) {
          warp_sums<N>(l, wsum + quarter * N, lane);
          ok = __all_sync(0xffffffffu, mbar_wait<1>(&p_empty[(tau - 1) % NP], ((tau - 1) / NP) & 1, abort_flag, err));
          tc_fence_after();
        }
        if (bar_or(1, 128, !ok)) break;
        const bool whole = w.whole();
        const int rows = w.rows(p);
        float* po = p.part_o + (int64_t)w.part() * p.row_slots * D;
        if (tid < N) {
          const float sum = (wsum[tid] + wsum[N + tid]) + (wsum[2 * N + tid] + wsum[3 * N + tid]);
          const int tok = row_token(p, tid), g = tid - tok * p.group;
          const RowPlace at = row_place<PREFIX>(p.t, w.b, tok);
          const int64_t out_row = ((int64_t)at.b * p.t.heads + (int64_t)w.hk * p.group + g) * p.t.n + at.i;
          const bool zero = !row_live<PREFIX>(p.t, at, tok, w.nl) || sum == 0.f;  // sees nothing
          res[tid] = zero ? -1.f : whole ? 1.f / sum : 1.f;
          offs[tid] = whole ? out_row * D : (int64_t)tid * D;
          if (tid < rows) {
            if (!whole) {
              float* st = p.part_s + (int64_t)w.part() * 2 * p.row_slots + tid;
              st[0] = ref[tid];
              st[p.row_slots] = zero ? 0.f : sum;
            } else if (p.t.lse) {
              p.t.lse[out_row] = zero ? -INFINITY : (ref[tid] + fast_log2(sum)) * 0.69314718055994531f;
            }
          }
        }
        if (threadIdx.x == 128) write_rec(p, part, w);
        bar_or(1, 128, false);
        // O^T: one dimension per thread, a row's dimensions next to each other
        if (quarter * 32 < D) {
          const uint32_t* seg_nf = nf + (w.seg % kNfRing) * 4;
          const bool back = tail && (seg_nf[0] | seg_nf[1]) != 0u;
          float* of = whole ? static_cast<float*>(p.t.o) : po;
          uint16_t* oh = static_cast<uint16_t*>(p.t.o);
          auto rows8 = [&](int i0, auto put) {
            __syncwarp();
            uint32_t o[8];
            tmem_ld_x8(tO + i0, o);
            if (back) {
              // non-finite values of drafted tokens, for the rows that see them
#pragma unroll 1
              for (int j = 0; j < w.nl; ++j) {
                if (!((seg_nf[j >> 5] >> (j & 31)) & 1u)) continue;
                const uint16_t* v = draft_value(p.t, D, w.b, w.hk, w.len, j);
                const uint32_t x = v ? v[key] : 0u;
                if ((x & 0x7f80u) != 0x7f80u) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if ((sees[2 * j + (i0 >> 5)] >> ((i0 & 31) + i)) & 1u)
                    o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(x << 16));
              }
            }
            float x[8];
            int64_t at[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float f = res[i0 + i];
              x[i] = f < 0.f ? 0.f : __uint_as_float(o[i]) * f;
              at[i] = offs[i0 + i] + key;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i0 + i < rows) put(at[i], x[i]);
          };
          if (!whole || p.t.out_f32) {
#pragma unroll 1
            for (int i0 = 0; i0 < rows; i0 += 8) rows8(i0, [&](int64_t at, float x) { of[at] = x; });
          } else {
#pragma unroll 1
            for (int i0 = 0; i0 < rows; i0 += 8)
              rows8(i0, [&](int64_t at, float x) { oh[at] = (uint16_t)pack_bf16x2(x, 0.f); });
          }
        }
        tc_fence_before();
      } while (w.next(p));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
  wait_at_end<PREFIX>(p.t);
}

template <int D, int N, bool PREFIX>
cudaError_t launch_narrow(const TreeParams& p, const CUtensorMap* maps, cudaStream_t stream) {
  using C = NarrowCfg<D, N>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(tree_narrow_kernel<D, N, PREFIX>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  return launch_chained(tree_narrow_kernel<D, N, PREFIX>, dim3(kTreeCtas), dim3(kNarrowThreads), C::SMEM_BYTES, stream, maps[0], maps[1], p);
}

template <int D, bool PREFIX>
cudaError_t launch_narrow_d(const TreeParams& p, const CUtensorMap* maps, cudaStream_t stream) {
  if (p.rows <= 16) return launch_narrow<D, 16, PREFIX>(p, maps, stream);
  if (p.rows <= 32) return launch_narrow<D, 32, PREFIX>(p, maps, stream);
  return launch_narrow<D, 64, PREFIX>(p, maps, stream);
}

}  // namespace

template <bool PREFIX>
cudaError_t launch_tree_narrow(const TreeParams& p, const CUtensorMap* maps, cudaStream_t stream) {
  switch (p.t.head_dim) {
    case 64: return launch_narrow_d<64, PREFIX>(p, maps, stream);
    case 96: return launch_narrow_d<96, PREFIX>(p, maps, stream);
    default: return launch_narrow_d<128, PREFIX>(p, maps, stream);
  }
}

}  // namespace wise
