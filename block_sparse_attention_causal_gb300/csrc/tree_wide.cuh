// Attention of new tokens over a paged cache (tree.cuh) for units of more than
// 64 rows, the join of partial results, and the launch.
//
// Rows are the MMAs' 128 rows and the softmax's threads. Two streams of 128
// rows each work at the same time, so that one stream's softmax runs beside
// the other's MMAs: up to 128 rows, the streams take alternate key tiles of the
// same rows and are joined through TMEM at the end of a segment; more rows,
// each stream has rows of its own and both use every key tile.
//
// Measured (one GB300): 256 rows of each of 8 key heads over 32K tokens of 128
// (a drafted tree of 64, 34.4 GFLOP, 135 MB): 43.4 us. A key tile takes 1.63 us
// (1.33 at the rate of a large library product), bound by a stream's chain of S
// MMA (8 of 128 x 128 x 16 from shared memory), softmax and PV, the other
// stream's in between; the first one comes 6 us after the start, and the partial
// results take 12 us out and through the join. The compiler spills 250 to 370
// bytes a thread (a launch of 168 registers, 128 of them a softmax row's scores);
// sixteen softmax warps, half a row per thread, took 45.5 us (96 registers a
// thread are too few).
//
// Warp roles (384 threads): 0 TMA, 1 guard of V, 2 MMA issue for both streams,
// 4-7 softmax and results of stream 0 (one row per thread), 8-11 of stream 1.
// TMEM: S_0 | S_1 | O_0 | O_1, P (bf16) written over S.
#pragma once
#include "tree.cuh"

namespace wise {
namespace {

constexpr int kWideThreads = 384;
constexpr int kWideOverhead = 8, kNarrowOverhead = 2;
static_assert(kWideOverhead <= kTreeOverhead && kNarrowOverhead <= kTreeOverhead, "wise_attn_tree's bound on the line");

template <int D, int QROWS>
struct TreeCfg {
  static constexpr bool PAIR = QROWS == 256;
  static constexpr uint32_t Q_BYTES = tile_bytes<D>(128);
  static constexpr uint32_t KV_BYTES = tile_bytes<D>(kTile);
  static constexpr uint32_t LIMIT = 232448u;
  static constexpr int NS_MAX = 12;
  static constexpr int NBAR = 9 + 3 * NS_MAX;
  static constexpr uint32_t OFF_RING = (PAIR ? 2u : 1u) * Q_BYTES;
  static constexpr uint32_t STATS = PAIR ? 0u : 2u * 2u * 2u * 128u;
  // stats; nf; barriers; words
  static constexpr uint32_t SMALL = STATS * 4u + kNfRing * 16u + NBAR * 8u + (NS_MAX + kTileFlags) * 4u + 40u * 4u;
  static constexpr int NS_FIT = (int)((LIMIT - OFF_RING - SMALL) / KV_BYTES);
  static constexpr int NS = NS_FIT < NS_MAX ? NS_FIT : NS_MAX;
  static_assert(NS >= 4, "ring");
  static constexpr uint32_t OFF_SMALL = OFF_RING + NS * KV_BYTES;
  static constexpr uint32_t SMEM_BYTES = OFF_SMALL + SMALL;
  static_assert(SMEM_BYTES <= LIMIT && OFF_RING % 1024 == 0 && KV_BYTES % 1024 == 0, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;
  __device__ static constexpr uint32_t s_col(int s) { return 128u * (uint32_t)s; }
  __device__ static constexpr uint32_t o_col(int s) { return 256u + (uint32_t)(s * D); }
};

// 32 bits from bit `off` (0 .. 127) of a 128-bit mask.
__device__ __forceinline__ uint32_t bits32(const uint32_t (&m)[4], int off) {
  const int w = off >> 5;
  const uint32_t lo = w == 0 ? m[0] : w == 1 ? m[1] : w == 2 ? m[2] : m[3];
  const uint32_t hi = w == 0 ? m[1] : w == 1 ? m[2] : w == 2 ? m[3] : 0u;
  return __funnelshift_r(lo, hi, off & 31);
}
// Bits of the 32 tokens from token `pos` on that a row sees.
__device__ __forceinline__ uint32_t seen32(const uint32_t (&m)[4], int pos, int len) {
  const int off = pos - len;
  if (off <= -32) return 0xffffffffu;
  if (off < 0) return ((1u << -off) - 1u) | (m[0] << -off);
  return off < 128 ? bits32(m, off) : 0u;
}

// The non-finite values of drafted tokens in columns [col, col + 16), put back
// for a row that sees the tokens of w0 .. w3 (they were taken out of the MMA's V).
static __device__ __noinline__ void put_back(const TreeLaunch& t, int d, int b, int hk, int len, int col, uint32_t w0,
                                             uint32_t w1, uint32_t w2, uint32_t w3, uint32_t (&o)[16]) {
  const uint32_t ws[4] = {w0, w1, w2, w3};
#pragma unroll 1
  for (int w = 0; w < 4; ++w)
#pragma unroll 1
    for (uint32_t m = ws[w]; m != 0u; m &= m - 1u) {
      const uint16_t* v = draft_value(t, d, b, hk, len, 32 * w + __ffs(m) - 1);
      if (!v) continue;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint32_t x = v[col + c];
        if ((x & 0x7f80u) == 0x7f80u) o[c] = __float_as_uint(__uint_as_float(o[c]) + __uint_as_float(x << 16));
      }
    }
}

// O row segment [tO, tO + ncols) *= factor (the lazy rescale, rare).
static __device__ __noinline__ void rescale_row(uint32_t tO, int ncols, float factor) {
  for (int c = 0; c < ncols; c += 16) {
    uint32_t o[16];
    tmem_ld_x16(tO + c, o);
    tmem_wait_ld16(o);
#pragma unroll
    for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * factor);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            tO + c),
        "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]), "r"(o[8]), "r"(o[9]),
        "r"(o[10]), "r"(o[11]), "r"(o[12]), "r"(o[13]), "r"(o[14]), "r"(o[15])
        : "memory");
  }
}

template <int D, int QROWS, bool PREFIX>
__global__ void __launch_bounds__(kWideThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
  using C = TreeCfg<D, QROWS>;
  using R = RingCfg<D, C::NS>;
  constexpr bool PAIR = C::PAIR;
  constexpr int NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  // without PAIR: [2][2][2][128] of even and odd segments, each stream: references and sums of its rows
  float* stats = reinterpret_cast<float*>(smem + C::OFF_SMALL);
  uint32_t* nf = reinterpret_cast<uint32_t*>(stats + C::STATS);  // [kNfRing][4]
  uint64_t* bars = reinterpret_cast<uint64_t*>(nf + kNfRing * 4);
  uint64_t* q_full = bars;           // [2] Q of a segment in which stream s has tiles is in shared memory
  uint64_t* s_full = q_full + 2;     // [2] S_s computed
  uint64_t* p_full = s_full + 2;     // [2] P_s written (4 softmax warps)
  uint64_t* o_final = p_full + 2;    // [2] last PV MMA of the stream's segment done
  Ring ring;
  ring.tiles = smem + C::OFF_RING;
  uint64_t* drain = o_final + 2;     // all MMAs done
  ring.full = drain + 1;
  ring.empty = ring.full + C::NS_MAX;
  ring.guarded = ring.empty + C::NS_MAX;
  ring.uses = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  ring.flags = ring.uses + C::NS_MAX;
  uint32_t* misc = ring.flags + kTileFlags;
  uint32_t* tmem_base_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  int* scratch = reinterpret_cast<int*>(misc + 4);  // [12 + 12]
  uint32_t* err = p.t.err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if ((smem_u32(smem) & 1023u) != 0u) {  // swizzled tiles
    grid_wait();
    clear_recs(p);
    if (threadIdx.x == 0) atomicOr(err, kErrInternal);
    return;
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], PAIR ? 4 : 8);  // the warps that write it
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&o_final[s], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&ring.full[i], 1);
      mbar_init(&ring.empty[i], PAIR ? 2 : 1);
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
  find_part<kWideThreads, PREFIX>(p, scratch, part, blocks);
  const uint32_t tbase = *tmem_base_slot;
  const bool any = part.left > 0;
  if (threadIdx.x == 128) clear_rec(p);
  WalkOf<PREFIX> w;
  if (any) w.start(p, part);

  // Registers per thread: 80 (warps 0-3) and 208 (softmax), in sum below the
  // 384 x 168 of the launch.
  if (warp < 4) {
    setmaxnreg_dec<80>();
    if (any && warp == 0) {
      ring_producer<D, NS, 1>(p, w, ring, &tm_k, &tm_v, abort_flag, lane);
    } else if (any && warp == 1) {
      ring_guard<D, NS, 2>(p, w, ring, nf, abort_flag, lane);
    } else if (any && warp == 2) {
      // ---------------------------------------------------------- MMA issue
      // One thread for both streams: PV of a stream whose P is written and at
      // once S of its next tile (which may then overwrite P), as one block.
      // Issued from two threads, the streams' MMAs interleave, both wait twice
      // as long, and the tensor core idles while both are in their softmax
      // (measured: 3600 cycles per key tile of 256 rows).
      if (elect_one()) {
        constexpr uint32_t IDESC_S = idesc_bf16_f32(128, kTile, 0, 0);
        constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, 0, 1);
        const uint64_t q_desc = smem_desc(smem_u32(smem), 16, 8 * kRowBytes, kSwizzle128);
        const uint64_t kd_base = smem_desc(smem_u32(ring.tiles), 16, 8 * kRowBytes, kSwizzle128);
        const uint64_t vd_base = smem_desc(smem_u32(ring.tiles), kTile * kRowBytes, 8 * kRowBytes, kSwizzle128);
        constexpr int STEP = PAIR ? 1 : 2;
        struct Stream {
          WalkOf<PREFIX> w;
          uint32_t tau0;       // the CTA's tiles before the segment
          int i;               // the segment's tile that is next (S) or under way (PV)
          uint32_t nq, np;     // segments with tiles, P tiles so far
          bool want_s, done;
        };
        Stream s0, s1;
        auto enter = [&](Stream& st, int s) {  // the first segment from the present one on that has tiles
          while (st.w.t1 - st.w.t0 <= (PAIR ? 0 : s)) {
            st.tau0 += (uint32_t)(st.w.t1 - st.w.t0);
            if (!st.w.next(p)) {
              st.done = true;
              return;
            }
          }
          st.i = PAIR ? 0 : s;
          st.want_s = true;
        };
        auto init = [&](Stream& st, int s) {
          st.w = w;
          st.tau0 = st.nq = st.np = 0u;
          st.done = false;
          enter(st, s);
        };
        auto loaded = [&](uint32_t pos) -> bool {
          const uint32_t slot = pos % NS;
          return ld_acquire_smem(&ring.uses[slot]) == pos + 1u && mbar_test_wait(&ring.full[slot], (pos / NS) & 1);
        };
        // one step of stream s, if its operands are there
        auto advance = [&](Stream& st, int s) -> bool {
          const int nt = st.w.t1 - st.w.t0;
          const uint32_t dS = tbase + C::s_col(s);
          if (!st.want_s) {
            const uint32_t pos = 2u * (st.tau0 + (uint32_t)st.i) + 1u;
            const int slot = (int)(pos % NS);
            if (!mbar_test_wait(&p_full[s], st.np & 1) || !loaded(pos) ||
                !mbar_test_wait(&ring.guarded[slot], R::guard_phase(pos) & 1))
              return false;
            ++st.np;
            tc_fence_after();
            const uint64_t vd = vd_base + (uint64_t)((slot * C::KV_BYTES) >> 4);
            const bool head = st.i < STEP;
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_ts(tbase + C::o_col(s), dS + kk * 8, vd + (uint64_t)((kk * 16 * kRowBytes) >> 4), IDESC_O,
                      (head && kk == 0) ? 0u : 1u);
            umma_commit(&ring.empty[slot]);
            st.want_s = true;
            st.i += STEP;
            if (st.i >= nt) {
              umma_commit(&o_final[s]);
              st.tau0 += (uint32_t)nt;
              if (st.w.next(p)) enter(st, s);
              else st.done = true;
              return true;
            }
          }
          const bool head = st.i < STEP;
          const uint32_t pos = 2u * (st.tau0 + (uint32_t)st.i);
          const int slot = (int)(pos % NS);
          if ((head && !mbar_test_wait(&q_full[s], st.nq & 1)) || !loaded(pos)) return false;
          if (head) ++st.nq;
          tc_fence_after();
          const uint64_t qd = q_desc + (uint64_t)(((PAIR ? s : 0) * C::Q_BYTES) >> 4);
          const uint64_t kd = kd_base + (uint64_t)((slot * C::KV_BYTES) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int c = kk / 4, wd = kk % 4;
            umma_ss(dS, qd + (uint64_t)((c * 128 * kRowBytes + wd * 32) >> 4),
                    kd + (uint64_t)((c * kTile * kRowBytes + wd * 32) >> 4), IDESC_S, kk > 0);
          }
          umma_commit(&s_full[s]);
          umma_commit(&ring.empty[slot]);
          st.want_s = false;
          return true;
        };
        init(s0, 0);
        init(s1, 1);
        bool ok = true;
        uint32_t idle = 0;  // rounds without work
        uint64_t t0 = 0;
        while (ok && !(s0.done && s1.done)) {
          bool moved = !s0.done && advance(s0, 0);
          if (!s1.done && advance(s1, 1)) moved = true;
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
        umma_commit(drain);
        mbar_wait<3>(drain, 0, &none, err);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<208>();
    if (any) {
      // ---------------------------------------------------- softmax, results
      const int s = (warp - 4) >> 2;
      const int quarter = warp & 3;
      const int r = quarter * 32 + lane;  // row of the tile = TMEM lane
      const int wg_thread = (int)threadIdx.x - 128 - 128 * s;
      const uint32_t bar_id = PAIR ? 1u + (uint32_t)s : 1u;
      constexpr uint32_t bar_n = PAIR ? 128u : 256u;
      const uint32_t trow = tbase + (static_cast<uint32_t>(quarter * 32) << 16);
      const uint32_t tS = trow + C::s_col(s);
      const uint32_t tO = trow + C::o_col(s);
      const float sl2 = p.scale_log2;
      const int page_shift = p.t.cache.page_shift;
      uint32_t ne = 0, nfin = 0, tau0 = 0;
      bool ok = true;
      // Q of a segment, swizzled as TMA would write it. Neighbouring lanes copy
      // neighbouring 16-byte units, so that a warp asks for whole lines (a row
      // per lane took 5 us for the 128 rows of a cold Q).
      auto load_q = [&](const WalkOf<PREFIX>& x) {
        constexpr int UNITS = D / 8, GROUP = UNITS > 8 ? 16 : 8;  // lanes per row
        constexpr int STEP = (PAIR ? 128 : 256) / GROUP;          // rows per round
        const int row0 = x.pair * 256 + (PAIR ? 128 * s : 0), nrows = min(x.rows(p) - row0, 128);
        const int u = lane % GROUP;
        const uint16_t* src = p.t.q.data + (int64_t)x.hk * p.group * p.t.q.sh + u * 8;
        if constexpr (!PREFIX) src += (int64_t)x.b * p.t.q.sb;
        uint8_t* sq = smem + (PAIR ? s : 0) * C::Q_BYTES;
        const int qr0 = (PAIR ? wg_thread : (int)threadIdx.x - 128) / GROUP;
#pragma unroll 4
        for (int k = 0; k < 128 / STEP; ++k) {
          const int qr = qr0 + k * STEP;
          const int qt = row_token(p, row0 + qr), qg = (row0 + qr) - qt * p.group;
          if constexpr (PREFIX) {
            if (qr < nrows && u < UNITS) {
              const RowPlace at = row_place<true>(p.t, x.b, qt);
              copy16(sq + unit_offset(128, qr, u),
                     src + (int64_t)at.b * p.t.q.sb + (int64_t)qg * p.t.q.sh + (int64_t)at.i * p.t.q.sn);
            }
          } else if (qr < nrows && u < UNITS) {
            copy16(sq + unit_offset(128, qr, u), src + (int64_t)qg * p.t.q.sh + (int64_t)qt * p.t.q.sn);
          }
        }
      };
      auto publish_q = [&](const WalkOf<PREFIX>& x) {
        copy16_wait();
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) {
            mbar_arrive(&q_full[s]);
          } else {
            mbar_arrive(&q_full[0]);
            if (x.t1 - x.t0 > 1) mbar_arrive(&q_full[1]);
          }
        }
      };
      load_q(w);
      publish_q(w);
      for (;;) {
        WalkOf<PREFIX> wn = w;
        const bool more = wn.next(p);
        // rows of this tile: row = token * group + head of the group
        const int row0 = w.pair * 256 + (PAIR ? 128 * s : 0);
        const int nrows = max(0, min(w.rows(p) - row0, 128));
        const bool warp_on = quarter * 32 < nrows;
        const int row = row0 + r;
        const int tok = row_token(p, row), g = row - tok * p.group;
        const RowPlace place = row_place<PREFIX>(p.t, w.b, r < nrows ? tok : 0);
        const bool live = r < nrows && row_live<PREFIX>(p.t, place, tok, w.nl);
        // the row's mask words (drafted tokens it sees)
        uint32_t mrow[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mrow[i] = tok >= 32 * i + 31 ? 0xffffffffu : tok < 32 * i ? 0u : (2u << (tok - 32 * i)) - 1u;
          if (p.t.tree_mask) mrow[i] = 0u;
          if (p.t.tree_mask && live && i < p.mask_words)
            mrow[i] = (uint32_t)p.t.tree_mask[((int64_t)w.b * p.t.n + tok) * p.mask_words + i];
        }
        // word i of it without tokens past the sequence's new ones
        auto sees = [&](int i) -> uint32_t {
          return mrow[i] &
                 (!live || w.nl <= 32 * i ? 0u : w.nl < 32 * i + 32 ? (1u << (w.nl - 32 * i)) - 1u : 0xffffffffu);
        };
        float m_ref = -INFINITY, l = 0.f;
        int cnt = 0;
        const int nt = w.t1 - w.t0;
        for (int i = PAIR ? 0 : s; ok && i < nt; i += PAIR ? 1 : 2, ++cnt) {
          ok = __all_sync(0xffffffffu, mbar_wait<4>(&s_full[s], ne & 1, abort_flag, err));
          if (!ok) break;
          ++ne;
          if (!warp_on) {
            if (PAIR && more && i + 1 == nt) load_q(wn);
            if (lane == 0) mbar_arrive(&p_full[s]);
            continue;
          }
          tc_fence_after();
          // the stream's last S MMA of the segment has read Q: the next
          // segment's comes in while this tile is worked on
          if (PAIR && more && i + 1 == nt) load_q(wn);
          const uint32_t bad = tile_bad<4>(ring, tau0 + (uint32_t)i, abort_flag, err);
          uint32_t v[4][32];
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) tmem_ld_x32(tS + cc * 32, v[cc]);
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) tmem_wait_ld(v[cc]);
          const int kb = (w.t0 + i) * kTile;
          if (kb + kTile > w.len || bad != 0u) {
            const uint32_t m[4] = {sees(0), sees(1), sees(2), sees(3)};
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t see = seen32(m, kb + 32 * cc, w.len);
              // the pages of 32 tokens: one, or two of 16; those outside the
              // pool are not seen
              const int box = (32 * cc) >> page_shift;
              if ((bad >> box) & 1u) see &= page_shift == 4 ? 0xffff0000u : 0u;
              if (page_shift == 4 && ((bad >> (box + 1)) & 1u)) see &= 0xffffu;
#pragma unroll
              for (int q = 0; q < 32; ++q) v[cc][q] = ((see >> q) & 1u) ? v[cc][q] : __float_as_uint(-INFINITY);
            }
          }
          float mx8[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) mx8[q] = -INFINITY;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
#pragma unroll
            for (int q = 0; q < 16; ++q)
              mx8[q & 7] = fmax3(mx8[q & 7], __uint_as_float(v[cc][2 * q]), __uint_as_float(v[cc][2 * q + 1]));
          const float mx =
              fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])) * sl2;
          float factor = 1.f;
          bool resc = false;
          if (cnt == 0) {
            m_ref = mx;
          } else if (mx > m_ref + 8.f) {
            factor = fast_exp2(m_ref - mx);
            m_ref = mx;
            resc = true;
          }
          const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
          // P = 2^(s scale log2e - m), rounded to bf16 (2^-8) for the tensor core,
          // whose operands are both of V's type; the sum is of the fp32 values.
          // Against fp64, O is off by 0.0023 of its norm, 0.0017 of it from
          // O's own rounding; twice the MMAs would be needed for weights of 16 bits.
          const uint64_t sc2 = f2_pack(sl2, sl2), nm2 = f2_pack(-m_use, -m_use);
          uint64_t rs2[2] = {0ull, 0ull};
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              float e0, e1;
              f2_unpack(ffma2(f2_pack(__uint_as_float(v[cc][2 * q]), __uint_as_float(v[cc][2 * q + 1])), sc2, nm2), e0,
                        e1);
              const float p0 = fast_exp2(e0);
              const float p1 = fast_exp2(e1);
              pk[q] = pack_bf16x2(p0, p1);
              rs2[q & 1] = fadd2(rs2[q & 1], f2_pack(p0, p1));
            }
            tmem_st_x16(tS + cc * 16, pk);
          }
          float a0, a1;
          f2_unpack(fadd2(rs2[0], rs2[1]), a0, a1);
          l = l * factor + (a0 + a1);
          // O_s holds every PV MMA up to the previous tile (the S_s commit
          // covers them); rows whose maximum jumped are rescaled in place
          if (__any_sync(0xffffffffu, resc)) rescale_row(tO, D, factor);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[s]);
        }
        const bool has = cnt > 0;
        if (ok && has) {
          ok = __all_sync(0xffffffffu, mbar_wait<4>(&o_final[s], nfin & 1, abort_flag, err));
          ++nfin;
          tc_fence_after();
        }
        tau0 += (uint32_t)nt;
        // before the results: S of the next segment is then there after them
        if (PAIR && more) publish_q(wn);
        float w0 = 1.f, w1 = 0.f;  // weights of O_0 and O_1 (or of the stream's own O)
        if (!PAIR) {
          float* st = stats + (w.seg & 1) * 512 + s * 256;
          st[r] = m_ref;
          st[128 + r] = l;
          tc_fence_before();
        }
        if (bar_or(bar_id, bar_n, !ok)) break;
        if (!PAIR) {
          tc_fence_after();
          if (more) load_q(wn);  // (both streams are done with Q)
          const float* st = stats + (w.seg & 1) * 512;
          const float ma = st[r], mb = st[256 + r], la = st[128 + r], lb = st[256 + 128 + r];
          float top = fmaxf(ma, mb);
          if (top == -INFINITY) top = 0.f;
          w0 = la == 0.f ? 0.f : fast_exp2((ma == -INFINITY ? 0.f : ma) - top);
          w1 = lb == 0.f ? 0.f : fast_exp2((mb == -INFINITY ? 0.f : mb) - top);
          l = la * w0 + lb * w1;
          m_ref = top;
        } else if (m_ref == -INFINITY) {
          m_ref = 0.f;
        }
        if (warp_on) {
          const bool whole = w.whole();
          const int h = w.hk * p.group + g;
          const int64_t out_row = ((int64_t)place.b * p.t.heads + h) * p.t.n + place.i;
          const bool zero = !live || l == 0.f;  // sees nothing
          const float inv = (whole && !zero) ? 1.f / l : 1.f;
          const int pi = w.part();
          const uint32_t* seg_nf = nf + (w.seg % kNfRing) * 4;
          const uint32_t back[4] = {sees(0) & seg_nf[0], sees(1) & seg_nf[1], sees(2) & seg_nf[2], sees(3) & seg_nf[3]};
          const bool nonfin = (back[0] | back[1] | back[2] | back[3]) != 0u;
          // without PAIR each stream writes half of the columns
          constexpr int NCOL = PAIR ? D : D / 2;
          const int col0 = PAIR ? 0 : s * NCOL;
          const int pr = row - w.pair * 256;
          uint4* part_row = reinterpret_cast<uint4*>(p.part_o + (int64_t)pi * p.row_slots * D) + (pr >> 5) * (D / 4) * 32 + lane;
          auto load = [&](int c, uint32_t (&o)[16]) {
            __syncwarp();
            if (PAIR) {
              tmem_ld_x16(tO + c, o);
              tmem_wait_ld16(o);
            } else {
              uint32_t o1[16];
              tmem_ld_x16(trow + C::o_col(0) + c, o);
              tmem_ld_x16(trow + C::o_col(1) + c, o1);
              tmem_wait_ld16(o);
              tmem_wait_ld16(o1);
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                // a stream without tiles, or with nothing seen, has no O
                const float a = w0 == 0.f ? 0.f : __uint_as_float(o[q]) * w0;
                o[q] = __float_as_uint(w1 == 0.f ? a : a + __uint_as_float(o1[q]) * w1);
              }
            }
          };
          auto store = [&](int c, const uint32_t (&o)[16]) {
            float x[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) x[q] = zero ? 0.f : __uint_as_float(o[q]) * inv;
            if (r >= nrows) return;
            if (!whole) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                part_row[(c / 4 + q) * 32] = make_uint4(__float_as_uint(x[4 * q]), __float_as_uint(x[4 * q + 1]),
                                                        __float_as_uint(x[4 * q + 2]), __float_as_uint(x[4 * q + 3]));
            } else if (p.t.out_f32) {
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.t.o) + out_row * D + c);
#pragma unroll
              for (int q = 0; q < 4; ++q) dst[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.t.o) + out_row * D + c);
#pragma unroll
              for (int q = 0; q < 2; ++q)
                dst[q] = make_uint4(pack_bf16x2(x[8 * q], x[8 * q + 1]), pack_bf16x2(x[8 * q + 2], x[8 * q + 3]),
                                    pack_bf16x2(x[8 * q + 4], x[8 * q + 5]), pack_bf16x2(x[8 * q + 6], x[8 * q + 7]));
            }
          };
          if (__any_sync(0xffffffffu, nonfin)) {
#pragma unroll 1
            for (int c = col0; c < col0 + NCOL; c += 16) {
              uint32_t o[16];
              load(c, o);
              if (nonfin && !zero) put_back(p.t, D, w.b, w.hk, w.len, c, back[0], back[1], back[2], back[3], o);
              store(c, o);
            }
          } else {
#pragma unroll 1
            for (int c = col0; c < col0 + NCOL; c += 16) {
              uint32_t o[16];
              load(c, o);
              store(c, o);
            }
          }
          if (r < nrows && (PAIR || s == 0)) {
            if (whole) {
              if (p.t.lse) p.t.lse[out_row] = zero ? -INFINITY : (m_ref + fast_log2(l)) * 0.69314718055994531f;
            } else {
              float* st = p.part_s + (int64_t)pi * 2 * p.row_slots + (row - w.pair * 256);
              st[0] = m_ref;
              st[p.row_slots] = zero ? 0.f : l;
            }
          }
        }
        tc_fence_before();
        if (threadIdx.x == 128) write_rec(p, part, w);
        if (!more) break;
        if (!PAIR) publish_q(wn);
        w = wn;
      }
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

// Whether a record names parts that exist. After a wait that ran out a CTA
// leaves its records unwritten; what lies there must not be followed.
__device__ __forceinline__ bool rec_ok(const TreeParams& p, const int4& ra, const int4& rb) {
  return ra.x >= 2 && ra.y >= 0 && ra.z >= 0 && ra.x <= kTreeCtas - ra.z && ra.y < 2 * kTreeCtas && ra.w >= 0 &&
         ra.w < p.t.cache.batch && rb.x >= 0 && rb.x < p.t.cache.kv_heads && rb.y >= 0 && rb.y < p.pairs;
}

// Joins the partial results of a row whose unit was cut, in the line's order,
// whatever the order in which they were written. grid.x: join records, grid.y:
// rows (kJoinWarps of them per block, or one whose parts the warps share).
constexpr int kJoinWarps = 4;
template <int D, bool SHARE>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const TreeParams p) {
  constexpr int E = D / 32;
  constexpr int BATCH = 8;  // parts loaded at a time
  __shared__ float so[kJoinWarps][D], ss[kJoinWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = SHARE ? (int)blockIdx.y : (int)blockIdx.y * kJoinWarps + warp;  // row of the unit
  // every block waits: this grid must not end before the one it follows
  grid_wait();
  grid_trigger();
  const int4 ra = *reinterpret_cast<const int4*>(&p.rec[blockIdx.x]);
  const int4 rb = *(reinterpret_cast<const int4*>(&p.rec[blockIdx.x]) + 1);
  const int parts = ra.x, first_part = ra.y, first_cta = ra.z, b = ra.w, hk = rb.x;
  const int row = rb.y * 256 + r;
  if (!rec_ok(p, ra, rb) || r >= p.row_slots || row >= p.rows) return;
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int k0 = SHARE ? warp : 0; k0 < parts; k0 += BATCH * (SHARE ? kJoinWarps : 1)) {
    float pm[BATCH], pl[BATCH], v[BATCH][E];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int k = k0 + i * (SHARE ? kJoinWarps : 1);
      pl[i] = 0.f;
      if (k < parts) {
        const int64_t at = k == 0 ? first_part : 2 * (first_cta + k);
        const float* st = p.part_s + at * 2 * p.row_slots + r;
        pm[i] = st[0];
        pl[i] = st[p.row_slots];
        const float* o = p.part_o + (at * p.row_slots + r) * D + lane * E;
        if constexpr (E == 4) {
          const float4 x = *reinterpret_cast<const float4*>(o);
          v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = o[e];
        }
      }
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (pl[i] != 0.f) top = fmaxf(top, pm[i]);
    const float f = l == 0.f ? 0.f : fast_exp2(m - top);
    m = top;
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (pl[i] == 0.f) continue;  // saw nothing
      const float g = fast_exp2(pm[i] - m);
      l += pl[i] * g;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += v[i][e] * g;
    }
  }
  if constexpr (SHARE) {
    if (lane == 0) {
      ss[warp][0] = m;
      ss[warp][1] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k)
      if (ss[k][1] != 0.f) top = fmaxf(top, ss[k][0]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) {
      if (ss[k][1] == 0.f) continue;
      const float g = fast_exp2(ss[k][0] - top);
      l += ss[k][1] * g;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += so[k][lane * E + e] * g;
    }
    m = top;
  }
  const int tok = row_token(p, row), h = hk * p.group + (row - tok * p.group);
  const int64_t out_row = ((int64_t)b * p.t.heads + h) * p.t.n + tok;
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = l == 0.f ? 0.f : acc[e] * inv;
  if (p.t.out_f32) {
    float* o = static_cast<float*>(p.t.o) + out_row * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = acc[e];
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.t.o) + out_row * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = (uint16_t)pack_bf16x2(acc[e], 0.f);
  }
  if (lane == 0 && p.t.lse) p.t.lse[out_row] = l == 0.f ? -INFINITY : (m + fast_log2(l)) * 0.69314718055994531f;
}

// The same for wide units: a lane holds a row, a warp four columns of a block of
// 32 rows, the block's warps 16 columns. The first partial results are asked for
// before the maxima and sums that weigh them are known.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_wide_kernel(const TreeParams p) {
  constexpr int BATCH = 10;
  __shared__ float ss[kJoinWarps][2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rb = (int)blockIdx.y / (D / 16), c4 = (int)blockIdx.y % (D / 16) * kJoinWarps + warp;
  grid_wait();
  grid_trigger();
  const int4 ra = *reinterpret_cast<const int4*>(&p.rec[blockIdx.x]);
  const int4 rc = *(reinterpret_cast<const int4*>(&p.rec[blockIdx.x]) + 1);
  const int parts = ra.x, first_part = ra.y, first_cta = ra.z, b = ra.w, hk = rc.x;
  const int r = rb * 32 + lane, row = rc.y * 256 + r;
  if (!rec_ok(p, ra, rc) || rc.y * 256 + rb * 32 >= p.rows) return;
  auto part_at = [&](int k) -> int64_t { return k == 0 ? first_part : 2 * (first_cta + k); };
  const float* st = p.part_s + r;
  const float4* po = reinterpret_cast<const float4*>(p.part_o) + (rb * (D / 4) + c4) * 32 + lane;
  float pm[BATCH], pl[BATCH];
  float4 x[BATCH];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      pl[i] = 0.f;
      if (k0 + i < parts) {
        const int64_t at = part_at(k0 + i) * p.row_slots;
        x[i] = po[at * (D / 4)];
        pm[i] = st[at * 2];
        pl[i] = st[at * 2 + p.row_slots];
      }
    }
  };
  fetch(0);
  // the row's maximum and sum: every warp over its share of the parts
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int k = warp; k < parts; k += kJoinWarps) {
    const int64_t at = part_at(k) * p.row_slots;
    const float mk = st[at * 2], lk = st[at * 2 + p.row_slots];
    if (lk == 0.f) continue;  // saw nothing
    const float top = fmaxf(m, mk);
    l = (l == 0.f ? 0.f : l * fast_exp2(m - top)) + lk * fast_exp2(mk - top);
    m = top;
  }
  ss[warp][0][lane] = m;
  ss[warp][1][lane] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k)
    if (ss[k][1][lane] != 0.f) top = fmaxf(top, ss[k][0][lane]);
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k)
    if (ss[k][1][lane] != 0.f) sum += ss[k][1][lane] * fast_exp2(ss[k][0][lane] - top);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < parts; k0 += BATCH) {
    if (k0 > 0) fetch(k0);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (pl[i] == 0.f) continue;
      const float g = fast_exp2(pm[i] - top);
      acc.x += x[i].x * g, acc.y += x[i].y * g, acc.z += x[i].z * g, acc.w += x[i].w * g;
    }
  }
  if (row >= p.rows) return;
  const int tok = row_token(p, row), h = hk * p.group + (row - tok * p.group);
  const int64_t out_row = ((int64_t)b * p.t.heads + h) * p.t.n + tok;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const bool zero = sum == 0.f;
  const float4 o = make_float4(zero ? 0.f : acc.x * inv, zero ? 0.f : acc.y * inv, zero ? 0.f : acc.z * inv,
                               zero ? 0.f : acc.w * inv);
  if (p.t.out_f32) reinterpret_cast<float4*>(static_cast<float*>(p.t.o) + out_row * D)[c4] = o;
  else
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.t.o) + out_row * D)[c4] =
        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  if (c4 == 0 && p.t.lse) p.t.lse[out_row] = zero ? -INFINITY : (top + fast_log2(sum)) * 0.69314718055994531f;
}

struct WorkspaceLayout {
  int64_t recs, row_slots, part_o, part_s, bytes;  // offsets in bytes
};
// units: of `rows` rows at most; all_units: a record of each.
WorkspaceLayout workspace_layout(int64_t units, int64_t rows, int64_t d, bool all_units) {
  WorkspaceLayout w;
  w.recs = units < kTreeCtas || all_units ? units : kTreeCtas;
  w.row_slots = rows <= 64 ? rows : rows < 256 ? (rows + 31) / 32 * 32 : 256;
  w.part_o = w.recs * (int64_t)sizeof(JoinRec);
  w.part_s = w.part_o + 2 * kTreeCtas * w.row_slots * d * 4;
  w.bytes = w.part_s + 2 * kTreeCtas * 2 * w.row_slots * 4 + 16;  // the base is rounded up to 32 bytes
  return w;
}

template <int D, int QROWS, bool PREFIX>
cudaError_t launch_rows(const TreeParams& p, const CUtensorMap* maps, cudaStream_t stream) {
  using C = TreeCfg<D, QROWS>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(tree_kernel<D, QROWS, PREFIX>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  return launch_chained(tree_kernel<D, QROWS, PREFIX>, dim3(kTreeCtas), dim3(kWideThreads), C::SMEM_BYTES, stream, maps[0], maps[1], p);
}

template <int D, bool PREFIX>
cudaError_t launch_d(const TreeParams& p, const CUtensorMap* maps, cudaStream_t stream) {
  cudaError_t e = p.rows > 128  ? launch_rows<D, 256, PREFIX>(p, maps, stream)
                  : p.rows > 64 ? launch_rows<D, 128, PREFIX>(p, maps, stream)
                                : launch_tree_narrow<PREFIX>(p, maps, stream);
  if constexpr (PREFIX) {
    return e;  // (always rows_apart)
  } else {
    if (e != cudaSuccess || p.t.rows_apart) return e;
    // few rows: a row's parts are shared by a block's warps
    const bool wide = p.rows > 64;
    const bool share = (int64_t)p.recs * p.row_slots < kTreeCtas * 16;
    const int jobs = wide ? p.row_slots / 32 * (D / 4) : share ? p.row_slots * kJoinWarps : p.row_slots;
    const dim3 grid((unsigned)p.recs, (unsigned)((jobs + kJoinWarps - 1) / kJoinWarps));
    auto join = wide ? tree_join_wide_kernel<D> : share ? tree_join_kernel<D, true> : tree_join_kernel<D, false>;
    return launch_chained(join, grid, dim3(32 * kJoinWarps), 0, stream, p);
  }
}

}  // namespace

// Units of a cache whose (sequence, key head) has `rows` rows; of groups of
// sequences with `rows` rows in all (unit_rec's places).
inline int64_t tree_units(int64_t batch, int64_t kv_heads, int64_t rows) { return batch * kv_heads * ((rows + 255) / 256); }
inline int64_t shared_units(int64_t groups, int64_t kv_heads, int64_t rows) { return (rows / 256 + groups + 1) * kv_heads; }

// What a launch's kernels get.
template <bool PREFIX>
TreeParams tree_params(const TreeLaunch& t) {
  TreeParams p;
  p.t = t;
  p.group = t.heads / t.cache.kv_heads;
  p.group_mul = (uint32_t)((0x100000000ull + p.group - 1) / p.group);
  p.rows = p.group * t.n * (PREFIX ? t.members : 1);
  p.pairs = (p.rows + 255) / 256;
  p.mask_words = (t.n + 31) / 32;
  p.scale_log2 = t.scale * 1.4426950408889634f;
  // A change of units (results out, Q in, the pipeline filled again; 128 KB of
  // partial results for a wide unit) counts as so many key tiles in the line.
  // Measured: of 4, 6 and 8 places for wide units, and 0 to 3 for narrow ones, 8
  // and 2 gave the shortest times.
  p.overhead = p.rows > 64 ? kWideOverhead : kNarrowOverhead;
  const int64_t units = PREFIX ? shared_units(t.cache.batch, t.cache.kv_heads, (int64_t)p.group * t.n * t.sequences)
                               : tree_units(t.cache.batch, t.cache.kv_heads, p.rows);
  const WorkspaceLayout w = workspace_layout(units, p.rows, t.head_dim, t.rows_apart);
  uint8_t* ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(t.workspace) + 31) / 32 * 32);
  p.recs = (int32_t)w.recs;
  p.by_unit = t.rows_apart || units <= kTreeCtas;
  p.row_slots = (int32_t)w.row_slots;
  p.rec = reinterpret_cast<JoinRec*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  p.part_s = reinterpret_cast<float*>(ws + w.part_s);
  return p;
}

template <bool PREFIX>
cudaError_t launch_tree_rows(const TreeLaunch& t, const CUtensorMap* maps, cudaStream_t stream) {
  const TreeParams p = tree_params<PREFIX>(t);
  switch (t.head_dim) {
    case 64: return launch_d<64, PREFIX>(p, maps, stream);
    case 96: return launch_d<96, PREFIX>(p, maps, stream);
    default: return launch_d<128, PREFIX>(p, maps, stream);
  }
}

}  // namespace wise
