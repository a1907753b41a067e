// Attention weight gathered by the tokens of a paged cache: for each key head
//   w[t] += sum over the rows i of its group of heads that see t of exp(s_it - LSE_i),
// s_it = scale q_i k_t, with the LSE that the rows' attention returned.
//
// Tiles are turned round as in tree_narrow.cuh: 128 keys are the MMA's rows and
// up to 256 query rows its columns,
//   S^T[key, row] = K Q^T,
// so that a thread holds one key's scores of all rows and sums their weights in
// its registers, always in the same order; no value meets another key's, so what
// lies behind the last token, or in a key that a row does not see, has no way
// into a sum. More than 256 rows are further launches, one after the other.
//
// Warp roles (640 threads): 0 TMA (a ring of K tiles), 1 MMA issue, 2 and 3 Q
// and what belongs to it, then four groups of four warps that sum every fourth tile,
// one key per thread (with two groups the sums' latency took longer than the bytes
// of K: 128 rows over 131K tokens 57 us instead of 51).
// The key tiles of all (sequence, key head) units form the line of tree.cuh.
//
// Measured (one GB300): next tokens of 32 sequences of up to 8K, 32/8 heads of 128,
// 339 MB: 57.5 us, 87 % of a copy's rate (4 us before the first tile, 2 after the
// last); 128 rows of each key head over 32K tokens 18.6 us, 0.8 us a tile (its bytes
// 0.74); 256 rows over 131K 83 us: nothing is full (issue slots 52 %, DRAM 40 %,
// exponentials 34 %), the four groups wait for their one buffer of scores, its loads and
// the latency of their own sums; 1600 rows over 1000 62 us, seven launches of 9, each of
// which reads K again, whether its rows hold new tokens or not.
#include <type_traits>

#include "tree.cuh"

namespace wise {
namespace {

constexpr int kGroups = 4;  // of four warps that sum
constexpr int kThreads = 128 + 128 * kGroups;
constexpr int kMaxRows = 256;
constexpr int kMaxSlots = 6;
constexpr uint32_t kSmem = 232448u;

struct WeightsParams {
  TreeParams p;        // the line: units of one (sequence, key head)
  const float* lse;
  float* weights;
  int64_t width;
  int32_t row0, nrows;  // this launch's rows of a unit
  int32_t cols;         // nrows in whole blocks of 16, of 32 where there are more than 128
  int32_t half;         // columns of one MMA: cols, or half of them
  int32_t slots;        // ring
  int32_t q_bufs;       // buffers of Q
  uint32_t tmem_cols;
};

// Behind the ring and the Q buffers of `cols` rows:
struct Small {
  float neg_lse2[2][kMaxRows];            // of a segment (its Q's buffer): -LSE in powers of two, -inf: the row adds nothing
  uint32_t sees[2][kTreeMaxTokens][kMaxRows / 32];  // of each new token: the rows that see it
  uint32_t counts[2][kMaxRows / 32];                // the rows that add something
  int plain[2][2];                        // rows from 0 on that all count, as either of its warps found
  uint64_t q_full[2];   // Q and what belongs to it are there (2 warps)
  uint64_t seg_done[2];         // and no longer needed (all warps that sum)
  uint64_t s_full[kGroups];     // a group's scores computed
  uint64_t s_empty[kGroups];    // and read (4 warps)
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t drain;
  uint32_t flags[kTileFlags];
  uint32_t tmem_base;
  volatile int abort_flag;
  int scratch[kThreads / 32 + 12];
};
constexpr uint32_t kRoom = kSmem - (uint32_t)sizeof(Small);

__device__ __forceinline__ void add8(const float* neg_lse2, const uint32_t* s, float sl2, uint64_t (&sum)[2]) {
  const uint64_t sc = f2_pack(sl2, sl2);
#pragma unroll
  for (int c = 0; c < 8; c += 4) {
    const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(neg_lse2 + c);
    float e0, e1, e2, e3;
    f2_unpack(ffma2(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc, l.x), e0, e1);
    f2_unpack(ffma2(f2_pack(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sc, l.y), e2, e3);
    sum[0] = fadd2(sum[0], f2_pack(fast_exp2(e0), fast_exp2(e1)));
    sum[1] = fadd2(sum[1], f2_pack(fast_exp2(e2), fast_exp2(e3)));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tm_k, const WeightsParams a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const TreeParams& p = a.p;
  constexpr uint32_t KV_BYTES = tile_bytes<D>(kTile);
  const uint32_t q_bytes = tile_bytes<D>(a.cols);
  uint8_t* sq = smem + a.slots * KV_BYTES;
  Small& m = *reinterpret_cast<Small*>(sq + a.q_bufs * q_bytes);
  uint32_t* err = p.t.err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023u) != 0u) {  // swizzled tiles
    grid_wait();
    if (threadIdx.x == 0) atomicOr(err, kErrInternal);
    return;
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.q_full[i], 2);
      mbar_init(&m.seg_done[i], 4 * kGroups);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&m.s_full[i], 1);
      mbar_init(&m.s_empty[i], 4);
    }
    for (int i = 0; i < a.slots; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 1);
    }
    mbar_init(&m.drain, 1);
    for (int i = 0; i < kTileFlags; ++i) m.flags[i] = 0u;
    m.abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 0) tma_prefetch_desc(&tm_k);
  prefetch_tables(p);
  grid_wait();
  // tensor memory only now: a kernel before this one that still runs could wait
  // for what this one holds
  if (warp == 1) {
    tmem_alloc(&m.tmem_base, a.tmem_cols);
    tmem_relinquish();
  }
  grid_trigger();
  LinePart part;
  find_part<kThreads>(p, m.scratch, part, (int)gridDim.x);
  const uint32_t tbase = m.tmem_base;
  volatile int* abort_flag = &m.abort_flag;
  const int slots = a.slots;
  // the buffer of a segment's Q, and how often it was used before
  const int q_shift = a.q_bufs - 1;
  auto q_buf = [&](int seg) { return seg & q_shift; };
  auto q_turn = [&](int seg) { return (uint32_t)(seg >> q_shift); };
  Ring ring;
  ring.flags = m.flags;
  // rows of valid tokens, which come first
  auto live_rows = [&](const Walk& x) { return max(0, min(a.nrows, x.nl * p.group - a.row0)); };
  // Q of a segment by thread `th` of THREADS, swizzled as TMA would write it:
  // neighbouring lanes copy neighbouring 16-byte units of a row
  auto copy_q = [&](const Walk& x, int th, auto threads) {
    constexpr int THREADS = decltype(threads)::value, UNITS = D / 8, LANES = UNITS > 8 ? 16 : 8;
    const int u = th % LANES, live = live_rows(x);
    uint8_t* dst = sq + q_buf(x.seg) * q_bytes;
    const uint16_t* q = p.t.q.data + (int64_t)x.b * p.t.q.sb + (int64_t)x.hk * p.group * p.t.q.sh + u * 8;
#pragma unroll 4
    for (int r = th / LANES; r < a.cols; r += THREADS / LANES) {
      const int tok = row_token(p, a.row0 + r), g = a.row0 + r - tok * p.group;
      uint8_t* at = dst + unit_offset(a.cols, r, u);
      if (u >= UNITS) continue;
      if (r < live) copy16(at, q + (int64_t)g * p.t.q.sh + (int64_t)tok * p.t.q.sn);
      else *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
    }
  };
  // The rows that see each new token, turned round from the mask: 32 rows a word, a
  // token's rows next to each other.
  auto turn_mask = [&](const Walk& x, int th, auto threads) {
    if (x.t1 * kTile <= x.len) return;
    constexpr int THREADS = decltype(threads)::value;
    uint32_t* to = &m.sees[q_buf(x.seg)][0][0];
    const int words = (a.cols + 31) / 32;
    auto below = [](int k) -> uint32_t { return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u; };
    for (int y = th; y < x.nl * words; y += THREADS) {
      const int j = y / words, w = y - j * words, row = a.row0 + 32 * w;  // the word's first row
      uint32_t v = 0u;
      if (!p.t.tree_mask) {
        v = ~below(j * p.group - row);  // the rows of tokens j and later
      } else {
        const int last = min(row_token(p, row + 31), x.nl - 1);
        const int32_t* mask = p.t.tree_mask + (int64_t)x.b * p.t.n * p.mask_words + (j >> 5);
#pragma unroll 4
        for (int i = row_token(p, row); i <= last; ++i)
          if (((uint32_t)mask[(int64_t)i * p.mask_words] >> (j & 31)) & 1u)
            v |= below((i + 1) * p.group - row) & ~below(i * p.group - row);
      }
      to[j * (kMaxRows / 32) + w] = v;
    }
  };
  // the first segment's Q is copied by all but the first two warps (by the two that
  // copy the later ones, 128 rows took 2.4 us)
  constexpr int ALL = kThreads - 64;
  auto first_q = [&] {
    copy16_wait();
    fence_proxy_async();
    named_bar_sync(1, ALL);
  };
  if (part.left > 0) {
    Walk w;
    w.start(p, part);
    if (warp == 0) {
      // ----------------------------------------------------------------- TMA
      const int page = 1 << p.t.cache.page_shift;
      const int boxes = kTile >> p.t.cache.page_shift;  // pages per tile
      const uint32_t box_bytes = tile_bytes<D>(page);
      uint32_t tau = 0;
      int slot = 0;
      uint32_t turn = 0;  // uses of the present slot before
      bool ok = true, flagged = false;
      do {
        const int32_t* table = p.t.cache.page_table + (int64_t)w.b * p.t.cache.max_pages;
        const int last_page = (w.keys - 1) >> p.t.cache.page_shift;  // -1: none
        // the lanes hold 32 columns of the page table, and the 32 after them,
        // which are under way while these are used
        int have = w.t0 * boxes;
        auto columns = [&](int c) -> int32_t { return c + lane <= last_page ? table[c + lane] : -1; };
        int32_t held = columns(have), ahead = columns(have + 32);
        for (int t = w.t0; ok && t < w.t1; ++t, ++tau) {
          const int col = t * boxes;
          if (col >= have + 32) {  // (32 columns are whole tiles)
            have += 32;
            held = ahead;
            ahead = columns(have + 32);
          }
          const int32_t pg = __shfl_sync(0xffffffffu, held, (col - have + lane) & 31);
          const bool in = lane < boxes && col + lane <= last_page;
          const bool good = in && page_ok(p.t, pg);
          const uint32_t bad = __ballot_sync(0xffffffffu, in && !good);
          const uint32_t loads = __ballot_sync(0xffffffffu, good);
          if (bad != 0u && !flagged) {
            flagged = true;
            if (lane == 0) atomicOr(err, kErrBadCache);
          }
          if (turn > 0) ok = __all_sync(0xffffffffu, mbar_wait<1>(&m.empty[slot], (turn - 1) & 1, abort_flag, err));
          if (!ok) break;
          if (lane == 0) {
            *reinterpret_cast<volatile uint32_t*>(&m.flags[tau % kTileFlags]) = tile_word(tau, bad);
            mbar_arrive_expect_tx(&m.full[slot], (uint32_t)__popc(loads) * box_bytes);
          }
          __syncwarp();
          if (good) {
            uint8_t* dst = smem + slot * KV_BYTES + (uint32_t)(lane * page) * kRowBytes;
#pragma unroll
            for (int c = 0; c < row_chunks<D>(); ++c)
              tma_load_3d(dst + c * kTile * kRowBytes, &tm_k, &m.full[slot], c * 64, w.hk * page, pg);
          }
          __syncwarp();
          if (++slot == slots) slot = 0, ++turn;
        }
      } while (ok && w.next(p));
      // no copy into this CTA's shared memory may outlive the CTA
      if (lane == 0) {
        int none = 0;
        for (uint32_t i = (tau > (uint32_t)slots ? tau - slots : 0u); i < tau; ++i)
          mbar_wait<1>(&m.full[i % slots], (i / slots) & 1, &none, err);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ----------------------------------------------------------- MMA issue
      if (elect_one()) {
        const uint32_t idesc = idesc_bf16_f32(128, a.half, 0, 0);
        const uint64_t k_desc = smem_desc(smem_u32(smem), 16, 8 * kRowBytes, kSwizzle128);
        const uint64_t q_desc = smem_desc(smem_u32(sq), 16, 8 * kRowBytes, kSwizzle128);
        uint32_t tau = 0, turn = 0;
        int slot = 0;
        bool ok = true;
        const uint32_t halves = (uint32_t)(a.cols / a.half);
        // scores of half h of tile `tile`, whose K is in `at`
        auto issue = [&](uint32_t tile, uint32_t h, int at, uint64_t qd) -> bool {
          const int buf = (int)(tile % kGroups);
          const uint32_t u = tile / kGroups * halves + h;  // uses of the buffer before
          if (u > 0u && !mbar_wait<1>(&m.s_empty[buf], (u - 1) & 1, abort_flag, err)) return false;
          tc_fence_after();
          const uint64_t kd = k_desc + (uint64_t)((at * KV_BYTES) >> 4);
          const uint32_t c0 = h * (uint32_t)a.half;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int c = kk / 4, wd = kk % 4;
            umma_ss(tbase + buf * a.half, kd + (uint64_t)((c * kTile * kRowBytes + wd * 32) >> 4),
                    qd + (uint64_t)(((c * a.cols + c0) * kRowBytes + wd * 32) >> 4), idesc, kk > 0);
          }
          umma_commit(&m.s_full[buf]);
          if (h + 1u == halves) umma_commit(&m.empty[at]);
          return true;
        };
        do {
          ok = mbar_wait<1>(&m.q_full[q_buf(w.seg)], q_turn(w.seg) & 1, abort_flag, err);
          const uint64_t qd = q_desc + (uint64_t)((q_buf(w.seg) * q_bytes) >> 4);
          // the second halves follow two tiles behind the first ones: a group has one
          // buffer, and the others' come in between while it works on the first
          const int n = w.t1 - w.t0, lag = halves > 1u ? 2 : 0;
          for (int i = 0; ok && i < n + lag; ++i) {
            if (i < n) {
              ok = mbar_wait<1>(&m.full[slot], turn & 1, abort_flag, err) && issue(tau, 0u, slot, qd);
              ++tau;
              if (++slot == slots) slot = 0, ++turn;
            }
            if (ok && lag > 0 && i >= lag) {
              const int back = min(i, n - 1) - (i - lag) + 1;  // the tile is so many slots back
              ok = issue(tau - (uint32_t)back, 1u, (slot - back + slots) % slots, qd);
            }
          }
        } while (ok && w.next(p));
        // every MMA of this thread done before TMEM and shared memory go
        int none = 0;
        umma_commit(&m.drain);
        mbar_wait<1>(&m.drain, 0, &none, err);
      }
      __syncwarp();
    } else if (warp < 4) {
      // ------------------------------------------------------------------- Q
      const int th = threadIdx.x - 64;  // 0 .. 63
      bool ok = true;
      do {
        const int buf = q_buf(w.seg);
        if (q_turn(w.seg) > 0)
          ok = __all_sync(0xffffffffu, mbar_wait<1>(&m.seg_done[buf], (q_turn(w.seg) - 1) & 1, abort_flag, err));
        if (!ok) break;
        const int live = live_rows(w);
        float l[kMaxRows / 64];
#pragma unroll
        for (int k = 0; k < kMaxRows / 64; ++k) {
          const int r = th + 64 * k, tok = row_token(p, a.row0 + r), g = a.row0 + r - tok * p.group;
          l[k] = -INFINITY;
          if (r < live) l[k] = a.lse[((int64_t)w.b * p.t.heads + w.hk * p.group + g) * p.t.n + tok];
        }
        if (w.seg == 0) copy_q(w, th, std::integral_constant<int, ALL>());
        else copy_q(w, th, std::integral_constant<int, 64>());
        if (w.seg == 0) turn_mask(w, th, std::integral_constant<int, ALL>());
        else turn_mask(w, th, std::integral_constant<int, 64>());
        int first = live;  // first row that adds nothing
#pragma unroll
        for (int k = 0; k < kMaxRows / 64; ++k) {
          const int r = th + 64 * k;
          const uint32_t some = __ballot_sync(0xffffffffu, l[k] != -INFINITY);
          if (lane == 0) m.counts[buf][r >> 5] = some;
          if (r >= a.cols) continue;
          if (l[k] == -INFINITY) first = min(first, r);
          m.neg_lse2[buf][r] = l[k] == -INFINITY ? -INFINITY : l[k] * -1.4426950408889634f;
        }
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) m.plain[buf][warp & 1] = first;
        if (w.seg == 0) {
          first_q();
        } else {
          copy16_wait();
          fence_proxy_async();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&m.q_full[buf]);
      } while (w.next(p));
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- sums
      const int s = (warp - 4) >> 2;  // every kGroups-th tile
      const int quarter = warp & 3, key = quarter * 32 + lane;
      const uint32_t tS = tbase + (static_cast<uint32_t>(quarter * 32) << 16) + s * a.half;
      const float sl2 = p.scale_log2;
      uint32_t tau = 0, used = 0;
      bool ok = true;
      copy_q(w, (int)threadIdx.x - 64, std::integral_constant<int, ALL>());
      turn_mask(w, (int)threadIdx.x - 64, std::integral_constant<int, ALL>());
      first_q();
      do {
        const int buf = q_buf(w.seg);
        ok = __all_sync(0xffffffffu, mbar_wait<1>(&m.q_full[buf], q_turn(w.seg) & 1, abort_flag, err));
        const float* neg_lse2 = m.neg_lse2[buf];
        const int plain = ok ? min(m.plain[buf][0], m.plain[buf][1]) : 0;
        const int live = live_rows(w);
        float* row = a.weights + ((int64_t)w.b * p.t.cache.kv_heads + w.hk) * a.width;
        for (int t = w.t0; ok && t < w.t1; ++t, ++tau) {
          if ((int)(tau % kGroups) != s) continue;
          const int pos = t * kTile + key;
          const bool in = pos < w.keys && pos < a.width;
          const bool fresh = pos >= w.len && a.row0 == 0;  // a new token's sum begins with the first launch
          float old = 0.f;
          if (in && !fresh) old = row[pos];
          // of the warp's keys: is one behind the committed tokens, is there one at all
          const bool tail = t * kTile + quarter * 32 + 32 > w.len;
          const bool some = t * kTile + quarter * 32 < w.keys;
          uint64_t sum[2] = {0ull, 0ull};
          const int j = pos - w.len;  // (negative: a committed token)
          // the words of rows that see the key
          const uint32_t* sees = m.sees[buf][min(max(j, 0), kTreeMaxTokens - 1)];
          auto block = [&](int c0, const uint32_t (&v)[16]) {
            if (!tail && c0 + 16 <= plain) {
              add8(neg_lse2 + c0, v, sl2, sum);
              add8(neg_lse2 + c0 + 8, v + 8, sl2, sum);
            } else {
              // rows that do not see the key, or add nothing, are left out, whatever
              // their scores are
              const uint32_t bits = ((j < 0 ? 0xffffffffu : j < w.nl ? sees[c0 >> 5] : 0u) & m.counts[buf][c0 >> 5]) >> (c0 & 16);
              float e[2] = {0.f, 0.f};
#pragma unroll
              for (int c = 0; c < 16; c += 4) {
                const float4 l = *reinterpret_cast<const float4*>(neg_lse2 + c0 + c);
                const float x0 = fast_exp2(fmaf(__uint_as_float(v[c]), sl2, l.x));
                const float x1 = fast_exp2(fmaf(__uint_as_float(v[c + 1]), sl2, l.y));
                const float x2 = fast_exp2(fmaf(__uint_as_float(v[c + 2]), sl2, l.z));
                const float x3 = fast_exp2(fmaf(__uint_as_float(v[c + 3]), sl2, l.w));
                e[0] += (bits >> c) & 1u ? x0 : 0.f;
                e[1] += (bits >> (c + 1)) & 1u ? x1 : 0.f;
                e[0] += (bits >> (c + 2)) & 1u ? x2 : 0.f;
                e[1] += (bits >> (c + 3)) & 1u ? x3 : 0.f;
              }
              sum[0] = fadd2(sum[0], f2_pack(e[0], e[1]));
            }
          };
          uint32_t bad = 0u;
          for (int h0 = 0; ok && h0 < a.cols; h0 += a.half, ++used) {
            ok = __all_sync(0xffffffffu, mbar_wait<1>(&m.s_full[s], used & 1, abort_flag, err));
            if (!ok) break;
            if (h0 == 0) bad = tile_bad<1>(ring, tau, abort_flag, err);
            tc_fence_after();
            const int cols = some ? min(a.half, live - h0) : 0;
            // the scores of 32 rows at a time (16, with the next 16 on their way: 256 rows
            // over 131K tokens 92 us instead of 85; 48 spill registers, 113 us)
            for (int c0 = 0; c0 < cols; c0 += 32) {
              uint32_t v0[16], v1[16];
              const bool both = c0 + 16 < cols;
              __syncwarp();
              tmem_ld_x16(tS + c0, v0);
              if (both) tmem_ld_x16(tS + c0 + 16, v1);
              tmem_wait_ld16(v0);
              if (both) tmem_wait_ld16(v1);
              block(h0 + c0, v0);
              if (both) block(h0 + c0 + 16, v1);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.s_empty[s]);
          }
          if (!ok) break;
          if (pos < w.keys && pos >= a.width) atomicOr(err, kErrBadCache);
          float x0, x1;
          f2_unpack(fadd2(sum[0], sum[1]), x0, x1);
          // (a page outside the pool: its tokens are not seen)
          if (in) row[pos] = ((bad >> (key >> p.t.cache.page_shift)) & 1u) ? old : old + (x0 + x1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.seg_done[buf]);
      } while (ok && w.next(p));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, a.tmem_cols);
  }
}

template <int D>
cudaError_t launch_d(const WeightsParams& a, const CUtensorMap* map, uint32_t bytes, cudaStream_t stream) {
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  return launch_chained(weights_kernel<D>, dim3(kTreeCtas), dim3(kThreads), bytes, stream, *map, a);
}

}  // namespace

cudaError_t launch_weights(const WeightsLaunch& w, const CUtensorMap* map, cudaStream_t stream) {
  WeightsParams a;
  TreeParams& p = a.p;
  p = TreeParams{};
  p.t.cache = w.cache;
  p.t.head_dim = w.head_dim;
  p.t.heads = w.heads;
  p.t.n = w.n;
  p.t.q = w.q;
  p.t.new_len = w.new_len;
  p.t.tree_mask = w.tree_mask;
  p.t.err = w.err;
  p.group = w.heads / w.cache.kv_heads;
  p.group_mul = (uint32_t)((0x100000000ull + p.group - 1) / p.group);
  p.rows = p.group * w.n;
  p.pairs = 1;
  p.mask_words = (w.n + 31) / 32;
  p.overhead = 1;
  p.scale_log2 = w.scale * 1.4426950408889634f;
  a.lse = w.lse;
  a.weights = w.weights;
  a.width = w.width;
  for (a.row0 = 0; a.row0 < p.rows; a.row0 += kMaxRows) {
    a.nrows = p.rows - a.row0 < kMaxRows ? p.rows - a.row0 : kMaxRows;
    const bool halves = a.nrows > 128;
    a.cols = halves ? (a.nrows + 31) / 32 * 32 : (a.nrows + 15) / 16 * 16;
    a.half = halves ? a.cols / 2 : a.cols;
    a.q_bufs = halves ? 1 : 2;  // (room for a deeper ring)
    a.tmem_cols = 32;
    while (a.tmem_cols < (uint32_t)kGroups * a.half) a.tmem_cols *= 2;
    const uint32_t chunks = w.head_dim > 64 ? 2 : 1, tile = kTile * chunks * kRowBytes, q = a.q_bufs * a.cols * chunks * kRowBytes;
    a.slots = (int32_t)((kRoom - q) / tile);
    if (a.slots > kMaxSlots) a.slots = kMaxSlots;
    static_assert(kRoom - 2u * 256u * kRowBytes >= 4u * kTile * 2u * kRowBytes, "four slots beside 256 rows");
    const uint32_t bytes = a.slots * tile + q + (uint32_t)sizeof(Small);
    const cudaError_t e = w.head_dim == 64   ? launch_d<64>(a, map, bytes, stream)
                          : w.head_dim == 96 ? launch_d<96>(a, map, bytes, stream)
                                             : launch_d<128>(a, map, bytes, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace wise
