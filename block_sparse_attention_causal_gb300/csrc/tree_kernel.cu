// Attention of new tokens over a paged cache: WISE ("Attention Routing
// Stabilizes Early: Working-Set Inference for Recurrent Language Models") §3
// Eq 2 for the rows behind the prompt -- a next token, a run of tokens, a tree
// of drafted tokens.
//
//   O_i = sum_j a_ij v_j,  a_ij = exp(s_ij - LSE_i),  s_ij = scale q_i k_j,
//   LSE_i = log sum_j exp(s_ij), over the committed tokens j and the drafted
//   tokens that row i's mask lists.
//
// Every key and value is read once for all rows that share it (the queries of
// a group of heads times the new tokens, packed into tiles of 128 rows), so
// the bound is the cache's bytes: 4 * head_dim per token and key head, until
// there are more than about 256 rows.
//
// One CTA per SM. The key tiles (128 tokens) of all (sequence, key head)
// units are one line of work that is cut into equal parts, so that lengths
// may differ and one long sequence fills the GPU; a unit that a cut divides
// leaves partial results (unnormalised O, running maximum, sums), which
// tree_join_kernel joins in order.
//
// Warp roles (384 threads):
//   warp 0      TMA of K and V tiles, page by page, into one ring of slots
//   warp 1      guards V: in tiles that hold drafted tokens or end past the
//               last token, rows that nobody may see are cleared, and
//               infinities and NaN of drafted tokens are taken out (0 times
//               them would reach rows that do not see them) and put back at
//               the end for the rows that do
//   warps 2, 3  MMA issue of streams 0 and 1 (S = Q K^T, then O += P V)
//   warps 4-7   softmax of stream 0, one row per thread, and its results
//   warps 8-11  softmax of stream 1
// Up to 128 rows: the streams take alternate key tiles of the same rows and
// are joined through TMEM at the end of a unit. More rows: each stream has a
// tile of 128 rows and both use every key tile.
// TMEM: S_0 | S_1 | O_0 | O_1, P (bf16) written over S.
#include <cudaTypedefs.h>

#include "internal.h"
#include "ptx.cuh"

namespace wise {
namespace {

constexpr int kTile = 128;     // keys per tile
constexpr int kMaxCtas = 152;  // SMs of a GB300
constexpr int kThreads = 384;
constexpr int kNfRing = 16;    // segments whose taken-out values are remembered

struct TreeParams {
  TreeLaunch t;
  int32_t group;        // query heads per key head
  int32_t rows;         // rows of a unit: group * n
  int32_t pairs;        // tiles of 256 rows (1 unless rows > 128)
  int32_t row_slots;    // rows of a partial result
  int32_t mask_words;   // words of a mask row
  float scale_log2;
  int32_t* starts;      // [batch + 1] first key tile of each sequence on the line
  float* part_o;        // [2 * kMaxCtas][row_slots][d]
  float* part_s;        // [2 * kMaxCtas][3][row_slots]: maximum, sum, sum of the rounded weights
};

template <int D, int QROWS>
struct TreeCfg {
  static constexpr bool PAIR = QROWS == 256;
  static constexpr int QT = PAIR ? 128 : QROWS;  // rows of a Q buffer; the MMA's 128 rows read on past a short one
  static constexpr int CH = (D == 96) ? 32 : 64;
  static constexpr int NCH = D / CH;
  static constexpr uint32_t SWZ = (CH == 64) ? 2u : 4u;
  static constexpr uint32_t ROWB = CH * 2;
  static constexpr uint32_t Q_BYTES = (uint32_t)QT * D * 2u;
  static constexpr uint32_t KV_BYTES = (uint32_t)kTile * D * 2u;
  static constexpr uint32_t LIMIT = 232448u;
  static constexpr int NS_MAX = 12;
  static constexpr uint32_t STATS_BYTES = 2u * 3u * 128u * 4u;
  static constexpr uint32_t NF_BYTES = kNfRing * 16u;
  static constexpr int NBAR_FIXED = 2 + 2 + 2 + 2 + 2;  // q_full, s_full, p_full, o_final, drain
  static constexpr uint32_t MISC_BYTES = 48u * 4u;
  static constexpr uint32_t OFF_RING = (PAIR ? 2u : 1u) * Q_BYTES;
  static constexpr uint32_t FIXED = OFF_RING + STATS_BYTES + NF_BYTES + MISC_BYTES + (NBAR_FIXED + 3 * NS_MAX) * 8u + 2 * NS_MAX * 4u;
  static constexpr int NS_FIT = (int)((LIMIT - FIXED) / KV_BYTES);
  static constexpr int NS = NS_FIT < NS_MAX ? NS_FIT : NS_MAX;
  static_assert(NS >= 4, "ring");
  static constexpr uint32_t OFF_STATS = OFF_RING + NS * KV_BYTES;
  static constexpr uint32_t OFF_NF = OFF_STATS + STATS_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_NF + NF_BYTES;
  static constexpr uint32_t OFF_MISC = OFF_BAR + (NBAR_FIXED + 3 * NS_MAX) * 8u;
  static constexpr uint32_t SMEM_BYTES = OFF_MISC + MISC_BYTES + 2 * NS_MAX * 4u;
  static_assert(SMEM_BYTES <= LIMIT && OFF_RING % 1024 == 0 && KV_BYTES % 1024 == 0 && OFF_NF % 16 == 0, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;
  // Ring position pos (odd: a V tile) is its slot's use number pos / NS; with
  // an odd number of slots every other use of a slot is a V tile.
  __device__ static constexpr uint32_t guard_phase(uint32_t pos) { return (NS & 1) ? (pos / NS) >> 1 : pos / NS; }
  __device__ static constexpr uint32_t s_col(int s) { return 128u * (uint32_t)s; }
  __device__ static constexpr uint32_t o_col(int s) { return 256u + (uint32_t)(s * D); }
};

// Committed and new tokens of sequence b, clamped to what the page table
// holds; true if nothing had to be clamped.
__device__ __forceinline__ bool seq_counts(const TreeLaunch& t, int b, int& len, int& nl) {
  const int64_t cap = (int64_t)t.cache.max_pages << t.cache.page_shift;
  const int64_t l0 = __ldg(t.cache.lengths + b);
  const int n0 = t.new_len ? __ldg(t.new_len + b) : t.n;
  const int64_t l = l0 < 0 ? 0 : (l0 > cap ? cap : l0);
  int n = n0 < 0 ? 0 : (n0 > t.n ? t.n : n0);
  if (l + n > cap) n = (int)(cap - l);
  len = (int)l;
  nl = n;
  return l == l0 && n == n0;
}
// Key tiles of a unit's pair of row tiles that holds a valid token (`full`),
// and how many pairs do; each other pair counts one empty tile.
__device__ __forceinline__ void seq_tiles(const TreeParams& p, int len, int nl, int& full, int& active) {
  const int keys = len + nl;
  full = keys > 0 ? (keys + kTile - 1) / kTile : 1;
  active = (nl * p.group + 255) / 256;
  if (active > p.pairs) active = p.pairs;
}
__device__ __forceinline__ int64_t seq_line(const TreeParams& p, int full, int active) {
  return (int64_t)p.t.cache.kv_heads * ((int64_t)active * full + (p.pairs - active));
}
// The CTA whose part of the line (tiles [c T / G, (c + 1) T / G)) holds tile x.
__device__ __forceinline__ int line_owner(int64_t x, int64_t total, int ctas) {
  return (int)(((x + 1) * ctas - 1) / total);
}

// One CTA's walk over its part of the line, a segment (consecutive key tiles
// of one unit) at a time. Every role keeps its own.
struct Walk {
  int b, hk, pair;
  int len, nl, full, active;
  int t0, t1, nt;  // tiles [t0, t1) of the unit's nt
  int keys;        // tokens that the unit's rows may see
  int left;        // tiles of the CTA's part from t0 on
  int seg;         // segments before this one

  __device__ __forceinline__ void unit(const TreeParams& p) {
    const bool on = pair < active;
    nt = on ? full : 1;
    keys = on ? len + nl : 0;
    t1 = min(nt, t0 + left);
  }
  __device__ __forceinline__ void load(const TreeParams& p) {
    seq_counts(p.t, b, len, nl);
    seq_tiles(p, len, nl, full, active);
  }
  __device__ __forceinline__ bool next(const TreeParams& p) {
    left -= t1 - t0;
    if (left <= 0) return false;
    ++seg;
    t0 = 0;
    if (++pair == p.pairs) {
      pair = 0;
      if (++hk == p.t.cache.kv_heads) {
        hk = 0;
        ++b;
        load(p);
      }
    }
    unit(p);
    return true;
  }
};

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Wait until ring position `pos` is loaded. A wait for a barrier's phase parity
// alone is not enough: the slot's use before may belong to the other stream,
// and while that copy is still under way the barrier reads as done for the use
// after it (copies may end in another order than they began). The producer
// names the use that a slot is in, which says that every earlier one is over.
template <int TAG>
static __device__ __noinline__ bool wait_use_slow(const uint32_t* use, uint32_t want, volatile int* abort_flag,
                                                  uint32_t* err) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire_smem(use) == want) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(err, kErrTimeout);
        return false;
      }
    }
  }
}
template <int TAG>
__device__ __forceinline__ bool wait_loaded(uint64_t* full, const uint32_t* uses, int ns, uint32_t pos,
                                            volatile int* abort_flag, uint32_t* err) {
  const uint32_t slot = pos % (uint32_t)ns;
  if (ld_acquire_smem(&uses[slot]) != pos + 1u && !wait_use_slow<TAG>(&uses[slot], pos + 1u, abort_flag, err)) return false;
  return mbar_wait<TAG>(&full[slot], (pos / (uint32_t)ns) & 1u, abort_flag, err);
}
__device__ __forceinline__ bool page_ok(const TreeLaunch& t, int32_t pg) { return pg >= 0 && (int64_t)pg < t.cache.n_pages; }

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

// A drafted token's non-finite values in columns [col, col + 16), put back for
// a row that sees it (they were taken out of the MMA's V).
static __device__ __noinline__ void put_back(const TreeLaunch& t, int d, int b, int hk, int len, int col, uint32_t w0, uint32_t w1,
                                             uint32_t w2, uint32_t w3, uint32_t (&o)[16]) {
  const uint32_t ws[4] = {w0, w1, w2, w3};
#pragma unroll 1
  for (int w = 0; w < 4; ++w)
#pragma unroll 1
    for (uint32_t m = ws[w]; m != 0u; m &= m - 1u) {
      const int64_t tok = (int64_t)len + 32 * w + __ffs(m) - 1;
      const int32_t pg = __ldg(t.cache.page_table + (int64_t)b * t.cache.max_pages + (tok >> t.cache.page_shift));
      if (!page_ok(t, pg)) continue;
      const uint16_t* v = t.cache.v_pages + ((((int64_t)pg * t.cache.kv_heads + hk) << t.cache.page_shift) +
                                             (tok & ((1 << t.cache.page_shift) - 1))) * d + col;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint32_t x = v[c];
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

template <int D, int QROWS>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
  using C = TreeCfg<D, QROWS>;
  constexpr bool PAIR = C::PAIR;
  constexpr int NS = C::NS;
  constexpr uint32_t ROWB = C::ROWB;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;           // [2] Q of a segment in which stream s has tiles is in shared memory
  uint64_t* s_full = q_full + 2;     // [2] S_s computed
  uint64_t* p_full = s_full + 2;     // [2] P_s written (4 softmax warps)
  uint64_t* o_final = p_full + 2;    // [2] last PV MMA of the stream's segment done
  uint64_t* drain = o_final + 2;     // [2] all MMAs of issuer s done
  uint64_t* full = drain + 2;        // [NS] tile loaded
  uint64_t* empty = full + NS;       // [NS] tile no longer needed
  uint64_t* guarded = empty + NS;    // [NS] V tile passed by warp 1
  float* stats = reinterpret_cast<float*>(smem + C::OFF_STATS);  // [2][3][128]
  uint32_t* nf = reinterpret_cast<uint32_t*>(smem + C::OFF_NF);  // [kNfRing][4] drafted tokens with taken-out values
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  uint32_t* tmem_base_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  int* first = reinterpret_cast<int*>(misc + 2);          // the CTA's first segment: b, hk, pair, t0, tiles
  int* warp_sum = reinterpret_cast<int*>(misc + 16);      // [12]
  uint32_t* bad_boxes = misc + 48;                        // [NS] pages of the V tile that are not in the pool
  uint32_t* uses = bad_boxes + C::NS_MAX;                 // [NS] one past the ring position that the slot is used for
  uint32_t* err = p.t.err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // 128B-swizzled TMA tiles need 1024-byte aligned destinations
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) atomicOr(err, kErrInternal);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], PAIR ? 4 : 8);  // the warps that write it
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&o_final[s], 1);
      mbar_init(&drain[s], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], PAIR ? 2 : 1);
      mbar_init(&guarded[i], 1);
      uses[i] = 0u;
    }
    *abort_flag = 0;
    first[4] = 0;
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc(tmem_base_slot, C::TMEM_COLS);
    tmem_relinquish();
  }

  // The line: every thread sums the tiles of consecutive sequences, the block
  // scans the sums, and the thread whose sequences hold the CTA's first tile
  // finds it there.
  const int batch = p.t.cache.batch;
  const int per = (batch + kThreads - 1) / kThreads;
  const int b_lo = min(batch, (int)threadIdx.x * per), b_hi = min(batch, b_lo + per);
  int mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    int len, nl, fl, ac;
    if (!seq_counts(p.t, b, len, nl) && blockIdx.x == 0) atomicOr(err, kErrBadCache);
    seq_tiles(p, len, nl, fl, ac);
    mine += (int)seq_line(p, fl, ac);
  }
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) warp_sum[warp] = before;
  before -= mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const int ctas = min((int)gridDim.x, total);
  const int cta = blockIdx.x;
  const int x0 = cta < ctas ? (int)((int64_t)cta * total / ctas) : total;
  const int x1 = cta < ctas ? (int)((int64_t)(cta + 1) * total / ctas) : total;
  if (mine > 0 && (cta == 0 || (x0 >= before && x0 < before + mine))) {
    int at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      int len, nl, fl, ac;
      seq_counts(p.t, b, len, nl);
      seq_tiles(p, len, nl, fl, ac);
      const int line = (int)seq_line(p, fl, ac);
      if (cta == 0) {
        p.starts[b] = at;
        if (b == batch - 1) p.starts[batch] = total;
      }
      if (x0 >= at && x0 < at + line) {
        const int per_head = ac * fl + (p.pairs - ac);
        const int r = (x0 - at) % per_head;
        first[0] = b;
        first[1] = (x0 - at) / per_head;
        first[2] = r < ac * fl ? r / fl : ac + (r - ac * fl);
        first[3] = r < ac * fl ? r % fl : 0;
        first[4] = x1 - x0;
      }
      at += line;
    }
  }
  __syncthreads();
  const uint32_t tbase = *tmem_base_slot;
  Walk w;
  w.left = first[4];
  const bool any = w.left > 0;
  if (any) {
    w.b = first[0];
    w.hk = first[1];
    w.pair = first[2];
    w.t0 = first[3];
    w.seg = 0;
    w.load(p);
    w.unit(p);
  }

  // Registers per thread: 80 (warps 0-3) and 208 (softmax), in sum below the
  // 384 x 168 of the launch.
  if (warp < 4) {
    setmaxnreg_dec<80>();
    if (any && warp == 0) {
      // ---------------------------------------------------------- TMA loads
      // Ring position 2 tau holds K of the CTA's tile tau, 2 tau + 1 its V.
      const int page = 1 << p.t.cache.page_shift;
      const int boxes = kTile >> p.t.cache.page_shift;  // pages per tile
      const uint32_t box_bytes = (uint32_t)page * D * 2u;
      if (lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      uint32_t pos = 0;
      bool ok = true, flagged = false;
      do {
        const int32_t* table = p.t.cache.page_table + (int64_t)w.b * p.t.cache.max_pages;
        const int last_page = (w.keys - 1) >> p.t.cache.page_shift;  // -1: none
        int have = -1;  // first page-table column that the lanes hold
        int32_t held = -1;
        for (int t = w.t0; ok && t < w.t1; ++t) {
          const int col = t * boxes;
          if (have < 0 || col + boxes > have + 32) {
            have = col;
            held = (col + lane <= last_page) ? __ldg(table + col + lane) : -1;
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
          for (int kv = 0; kv < 2 && ok; ++kv, ++pos) {
            const int slot = (int)(pos % NS);
            if (pos >= (uint32_t)NS)
              ok = __all_sync(0xffffffffu, mbar_wait<1>(&empty[slot], ((pos / NS) - 1) & 1, abort_flag, err));
            if (!ok) break;
            if (lane == 0) {
              if (kv) bad_boxes[slot] = bad;
              st_release_smem(&uses[slot], pos + 1u);
              mbar_arrive_expect_tx(&full[slot], (uint32_t)__popc(loads) * box_bytes);
            }
            __syncwarp();
            if (good) {
              uint8_t* dst = smem + C::OFF_RING + slot * C::KV_BYTES + (uint32_t)(lane * page) * ROWB;
#pragma unroll
              for (int c = 0; c < C::NCH; ++c)
                tma_load_3d(dst + c * kTile * ROWB, kv ? &tm_v : &tm_k, &full[slot], c * C::CH, w.hk * page, pg);
            }
            __syncwarp();
          }
        }
      } while (ok && w.next(p));
      // No copy into this CTA's shared memory may outlive the CTA.
      if (lane == 0) {
        int none = 0;
        for (uint32_t i = (pos > (uint32_t)NS ? pos - NS : 0u); i < pos; ++i)
          mbar_wait<1>(&full[i % NS], (i / NS) & 1, &none, err);
      }
      __syncwarp();
    } else if (any && warp == 1) {
      // ------------------------------------------------------------ guard V
      const int page = 1 << p.t.cache.page_shift;
      uint32_t pos = 1;
      bool ok = true;
      do {
        uint32_t* seg_nf = nf + (w.seg % kNfRing) * 4;
        if (lane < 4) seg_nf[lane] = 0u;
        __syncwarp();
        for (int t = w.t0; ok && t < w.t1; ++t, pos += 2) {
          const int slot = (int)(pos % NS);
          ok = __all_sync(0xffffffffu, wait_loaded<2>(full, uses, NS, pos, abort_flag, err));
          if (!ok) break;
          const uint32_t bad = bad_boxes[slot];
          const int kb = t * kTile;
          uint8_t* v = smem + C::OFF_RING + slot * C::KV_BYTES;
          if (bad != 0u || kb + kTile > w.len || w.keys == 0) {
            const int rows = max(0, min(w.keys - kb, kTile));
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            for (int c = 0; c < C::NCH; ++c) {
              uint8_t* vc = v + c * kTile * ROWB;
              for (uint32_t x = rows * ROWB + lane * 16; x < kTile * ROWB; x += 512) *reinterpret_cast<uint4*>(vc + x) = zero;
              for (uint32_t m = bad; m != 0u; m &= m - 1u) {
                const uint32_t at = (uint32_t)((__ffs(m) - 1) * page) * ROWB;
                for (uint32_t x = lane * 16; x < page * ROWB; x += 512) *reinterpret_cast<uint4*>(vc + at + x) = zero;
              }
            }
            __syncwarp();
            // drafted tokens' rows of the tile (the swizzle permutes 16-byte
            // units within a row, so a row's units are visited in any order)
            constexpr int U = ROWB / 16;
            for (int x = max(0, w.len - kb) * U + lane; x < rows * U; x += 32)
              for (int c = 0; c < C::NCH; ++c) {
                uint4* at = reinterpret_cast<uint4*>(v + c * kTile * ROWB) + x;
                uint4 q = *at;
                uint32_t* e = &q.x;
                bool hit = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if ((e[i] & 0x7f80u) == 0x7f80u) {
                    e[i] &= 0xffff0000u;
                    hit = true;
                  }
                  if ((e[i] & 0x7f800000u) == 0x7f800000u) {
                    e[i] &= 0xffffu;
                    hit = true;
                  }
                }
                if (hit) {
                  *at = q;
                  const int j = kb + x / U - w.len;
                  atomicOr(&seg_nf[j >> 5], 1u << (j & 31));
                }
              }
            fence_proxy_async();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&guarded[slot]);
        }
      } while (ok && w.next(p));
      __syncwarp();
    } else if (any) {
      // ---------------------------------------------------------- MMA issue
      const int s = warp - 2;
      const bool leader = elect_one();
      constexpr uint32_t IDESC_S = idesc_bf16_f32(128, kTile, 0, 0);
      constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t qd = smem_desc(smem_u32(smem + (PAIR ? s : 0) * C::Q_BYTES), 16, 8 * ROWB, C::SWZ);
      const uint64_t kd_base = smem_desc(smem_u32(smem + C::OFF_RING), 16, 8 * ROWB, C::SWZ);
      const uint64_t vd_base = smem_desc(smem_u32(smem + C::OFF_RING), kTile * ROWB, 8 * ROWB, C::SWZ);
      const uint32_t dS = tbase + C::s_col(s);
      const uint32_t dO = tbase + C::o_col(s);
      // the CTA's tiles before the segment; the stream's segments and P tiles so far
      uint32_t tau = 0, nq = 0, np = 0;
      bool ok = true;
      auto issue_s = [&](uint32_t tile) -> bool {  // S_s = Q K^T of the CTA's tile `tile`
        const uint32_t pos = 2u * tile;
        const int slot = (int)(pos % NS);
        if (!__all_sync(0xffffffffu, wait_loaded<3>(full, uses, NS, pos, abort_flag, err))) return false;
        tc_fence_after();
        const uint64_t kd = kd_base + (uint64_t)((slot * C::KV_BYTES) >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int c = kk / (C::CH / 16), wd = kk % (C::CH / 16);
            umma_ss(dS, qd + (uint64_t)((c * C::QT * ROWB + wd * 32) >> 4),
                    kd + (uint64_t)((c * kTile * ROWB + wd * 32) >> 4), IDESC_S, kk > 0);
          }
          umma_commit(&s_full[s]);
          umma_commit(&empty[slot]);
        }
        __syncwarp();
        return true;
      };
      do {
        const int nt = w.t1 - w.t0;
        const int step = PAIR ? 1 : 2;
        int i = PAIR ? 0 : s;
        if (i < nt) {
          ok = __all_sync(0xffffffffu, mbar_wait<3>(&q_full[s], nq & 1, abort_flag, err));
          ++nq;
          if (ok) ok = issue_s(tau + i);
          for (bool head = true; ok && i < nt; i += step, head = false) {
            const uint32_t pos = 2u * (tau + i) + 1u;
            const int slot = (int)(pos % NS);
            // V loaded (then every earlier use of the slot is over, and with
            // it every earlier phase of `guarded`), passed on by warp 1, P written
            ok = __all_sync(0xffffffffu, wait_loaded<3>(full, uses, NS, pos, abort_flag, err) &&
                                             mbar_wait<3>(&guarded[slot], C::guard_phase(pos) & 1, abort_flag, err) &&
                                             mbar_wait<3>(&p_full[s], np & 1, abort_flag, err));
            if (!ok) break;
            ++np;
            tc_fence_after();
            const uint64_t vd = vd_base + (uint64_t)((slot * C::KV_BYTES) >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                umma_ts(dO, dS + kk * 8, vd + (uint64_t)((kk * 16 * ROWB) >> 4), IDESC_O, (head && kk == 0) ? 0u : 1u);
              umma_commit(&empty[slot]);
              if (i + step >= nt) umma_commit(&o_final[s]);
            }
            __syncwarp();
            if (i + step < nt) ok = issue_s(tau + i + step);
          }
        }
        tau += (uint32_t)nt;
      } while (ok && w.next(p));
      if (leader) {
        int none = 0;
        umma_commit(&drain[s]);  // every MMA of this thread done before TMEM is released
        mbar_wait<3>(&drain[s], 0, &none, err);
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
      uint32_t ne = 0, nfin = 0;
      bool ok = true;
      bool lead_part = true;  // the CTA's first segment
      do {
        // rows of this tile: row = token * group + head of the group
        const int row0 = w.pair * 256 + (PAIR ? 128 * s : 0);
        const int nrows = max(0, min(p.rows - row0, 128));
        const bool warp_on = quarter * 32 < nrows;
        const int row = row0 + r;
        const int tok = row / p.group, g = row - tok * p.group;
        const bool live = r < nrows && tok < w.nl;
        const int32_t* table = p.t.cache.page_table + (int64_t)w.b * p.t.cache.max_pages;
        // Q of the segment (its previous readers, the S MMAs of the segment
        // before, are done), swizzled as TMA would write it
        {
          const int units = D / 8;
          const int first_unit = PAIR ? wg_thread : (int)threadIdx.x - 128;
          uint8_t* sq = smem + (PAIR ? s : 0) * C::Q_BYTES;
          for (int x = first_unit; x < nrows * units; x += PAIR ? 128 : 256) {
            const int qr = x / units, u = x - qr * units;
            const int qt = (row0 + qr) / p.group, qg = (row0 + qr) - qt * p.group;
            const uint16_t* src = p.t.q.data + (int64_t)w.b * p.t.q.sb + (int64_t)(w.hk * p.group + qg) * p.t.q.sh +
                                  (int64_t)qt * p.t.q.sn + u * 8;
            const int c = u / (C::CH / 8), uc = u % (C::CH / 8);
            const int sw = (C::CH == 64) ? (uc ^ (qr & 7)) : (uc ^ ((qr >> 1) & 3));
            *reinterpret_cast<uint4*>(sq + c * C::QT * ROWB + qr * ROWB + sw * 16) =
                __ldg(reinterpret_cast<const uint4*>(src));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) {
            mbar_arrive(&q_full[s]);
          } else {
            mbar_arrive(&q_full[0]);
            if (w.t1 - w.t0 > 1) mbar_arrive(&q_full[1]);
          }
        }
        // the row's mask words (drafted tokens it sees)
        uint32_t mrow[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t m = 0u;
          if (live && 32 * i < w.nl) {
            if (p.t.tree_mask)
              m = i < p.mask_words ? (uint32_t)__ldg(p.t.tree_mask + ((int64_t)w.b * p.t.n + tok) * p.mask_words + i) : 0u;
            else
              m = tok >= 32 * i + 31 ? 0xffffffffu : tok < 32 * i ? 0u : (2u << (tok - 32 * i)) - 1u;
            if (w.nl < 32 * i + 32) m &= (1u << (w.nl - 32 * i)) - 1u;
          }
          mrow[i] = m;
        }
        // pages outside the pool (their tokens are not seen): looked up here
        // once, and tile by tile only where there are any
        bool bad_page = false;
        {
          const int c0 = (w.t0 * kTile) >> page_shift;
          const int c1 = min((w.t1 * kTile) >> page_shift, (w.keys + (1 << page_shift) - 1) >> page_shift);
          for (int c = c0 + wg_thread; c < c1; c += 128) bad_page |= !page_ok(p.t, __ldg(table + c));
        }
        bad_page = bar_or(bar_id, bar_n, bad_page);
        float m_ref = -INFINITY, l = 0.f, lt = 0.f;
        int cnt = 0;
        const int nt = w.t1 - w.t0;
        for (int i = PAIR ? 0 : s; ok && i < nt; i += PAIR ? 1 : 2, ++cnt) {
          ok = __all_sync(0xffffffffu, mbar_wait<4>(&s_full[s], ne & 1, abort_flag, err));
          if (!ok) break;
          ++ne;
          if (!warp_on) {
            if (lane == 0) mbar_arrive(&p_full[s]);
            continue;
          }
          tc_fence_after();
          uint32_t v[4][32];
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) tmem_ld_x32(tS + cc * 32, v[cc]);
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) tmem_wait_ld(v[cc]);
          const int kb = (w.t0 + i) * kTile;
          if (kb + kTile > w.len || bad_page) {
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t see = seen32(mrow, kb + 32 * cc, w.len);
              if (bad_page) {
                // the pages of 32 tokens: one, or two of 16
                const int c = (kb + 32 * cc) >> page_shift;
                const int cols = (w.keys + (1 << page_shift) - 1) >> page_shift;
                if (c < cols && !page_ok(p.t, __ldg(table + c))) see &= page_shift == 4 ? 0xffff0000u : 0u;
                if (page_shift == 4 && c + 1 < cols && !page_ok(p.t, __ldg(table + c + 1))) see &= 0xffffu;
              }
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
          // P = 2^(s scale log2e - m), rounded to bf16 for the tensor core. O
          // is divided by the sum of the rounded weights (a row that sees one
          // token gets its value exactly); the LSE takes the fp32 sum.
          const uint64_t sc2 = f2_pack(sl2, sl2), nm2 = f2_pack(-m_use, -m_use);
          uint64_t rs2[2] = {0ull, 0ull}, rt2[2] = {0ull, 0ull};
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
              add_bf16x2_to(rt2[q & 1], pk[q]);
            }
            tmem_st_x16(tS + cc * 16, pk);
          }
          float a0, a1, b0, b1;
          f2_unpack(fadd2(rs2[0], rs2[1]), a0, a1);
          f2_unpack(fadd2(rt2[0], rt2[1]), b0, b1);
          l = l * factor + (a0 + a1);
          lt = lt * factor + (b0 + b1);
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
        float w0 = 1.f, w1 = 0.f;  // weights of O_0 and O_1 (or of the stream's own O)
        if (!PAIR) {
          float* st = stats + s * 384;
          st[r] = m_ref;
          st[128 + r] = l;
          st[256 + r] = lt;
          tc_fence_before();
        }
        if (bar_or(bar_id, bar_n, !ok)) break;
        if (!PAIR) {
          tc_fence_after();
          const float ma = stats[r], mb = stats[384 + r], la = stats[128 + r], lb = stats[384 + 128 + r];
          float top = fmaxf(ma, mb);
          if (top == -INFINITY) top = 0.f;
          w0 = la == 0.f ? 0.f : fast_exp2((ma == -INFINITY ? 0.f : ma) - top);
          w1 = lb == 0.f ? 0.f : fast_exp2((mb == -INFINITY ? 0.f : mb) - top);
          l = la * w0 + lb * w1;
          lt = stats[256 + r] * w0 + stats[384 + 256 + r] * w1;
          m_ref = top;
        } else if (m_ref == -INFINITY) {
          m_ref = 0.f;
        }
        if (warp_on) {
          const bool whole = w.t0 == 0 && w.t1 == w.nt;
          const int h = w.hk * p.group + g;
          const int64_t out_row = ((int64_t)w.b * p.t.heads + h) * p.t.n + tok;
          const bool zero = !live || l == 0.f;  // sees nothing
          const float inv = (whole && !zero) ? 1.f / lt : 1.f;
          const int part = 2 * cta + (lead_part ? 0 : 1);
          const uint32_t* seg_nf = nf + (w.seg % kNfRing) * 4;
          const uint32_t back[4] = {mrow[0] & seg_nf[0], mrow[1] & seg_nf[1], mrow[2] & seg_nf[2], mrow[3] & seg_nf[3]};
          const bool nonfin = (back[0] | back[1] | back[2] | back[3]) != 0u;
          // without PAIR each stream writes half of the columns
          constexpr int NCOL = PAIR ? D : D / 2;
          const int col0 = PAIR ? 0 : s * NCOL;
#pragma unroll 1
          for (int c = col0; c < col0 + NCOL; c += 16) {
            __syncwarp();
            uint32_t o[16];
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
            if (nonfin && !zero) put_back(p.t, D, w.b, w.hk, w.len, c, back[0], back[1], back[2], back[3], o);
            if (r < nrows) {
#pragma unroll
              for (int q = 0; q < 16; ++q) o[q] = zero ? 0u : __float_as_uint(__uint_as_float(o[q]) * inv);
              if (!whole || p.t.out_f32) {
                float* dst = whole ? static_cast<float*>(p.t.o) + out_row * D + c
                                   : p.part_o + ((int64_t)part * p.row_slots + (row - w.pair * 256)) * D + c;
#pragma unroll
                for (int q = 0; q < 4; ++q) reinterpret_cast<uint4*>(dst)[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
              } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.t.o) + out_row * D + c);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  uint4 x;
                  x.x = pack_bf16x2(__uint_as_float(o[8 * q + 0]), __uint_as_float(o[8 * q + 1]));
                  x.y = pack_bf16x2(__uint_as_float(o[8 * q + 2]), __uint_as_float(o[8 * q + 3]));
                  x.z = pack_bf16x2(__uint_as_float(o[8 * q + 4]), __uint_as_float(o[8 * q + 5]));
                  x.w = pack_bf16x2(__uint_as_float(o[8 * q + 6]), __uint_as_float(o[8 * q + 7]));
                  dst[q] = x;
                }
              }
            }
          }
          if (r < nrows && (PAIR || s == 0)) {
            if (whole) {
              if (p.t.lse) p.t.lse[out_row] = zero ? -INFINITY : (m_ref + fast_log2(l)) * 0.69314718055994531f;
            } else {
              float* st = p.part_s + (int64_t)part * 3 * p.row_slots + (row - w.pair * 256);
              st[0] = zero ? 0.f : m_ref;
              st[p.row_slots] = zero ? 0.f : l;
              st[2 * p.row_slots] = zero ? 0.f : lt;
            }
          }
        }
        tc_fence_before();
        lead_part = false;
      } while (w.next(p));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

// Joins the partial results of rows whose unit was cut: one block per row,
// its warps over the parts, then over each other. The parts are joined in the
// line's order, whatever the order in which they were written.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const TreeParams p, int ctas_launched) {
  constexpr int E = D / 32;
  __shared__ float so[kJoinWarps][D];
  __shared__ float sl[kJoinWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // every block waits: this grid must not end before the one it follows
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row = blockIdx.x % p.rows;
  const int unit = blockIdx.x / p.rows;
  const int hk = unit % p.t.cache.kv_heads, b = unit / p.t.cache.kv_heads;
  int len, nl, full, active;
  seq_counts(p.t, b, len, nl);
  seq_tiles(p, len, nl, full, active);
  const int pair = row / 256;
  if (pair >= active || full == 1) return;  // one tile: never cut
  const int64_t total = p.starts[p.t.cache.batch];
  const int ctas = (int)min((int64_t)ctas_launched, total);
  const int64_t start = (int64_t)p.starts[b] + seq_line(p, full, active) / p.t.cache.kv_heads * hk + (int64_t)pair * full;
  const int ca = line_owner(start, total, ctas), cb = line_owner(start + full - 1, total, ctas);
  if (ca == cb) return;
  // CTA ca's part is its first segment if its part of the line starts here
  const int first_part = 2 * ca + ((int64_t)ca * total / ctas == start ? 0 : 1);
  const int rr = row - 256 * pair;
  const int parts = cb - ca + 1;
  auto slot = [&](int k) -> int64_t { return k == 0 ? first_part : 2 * (ca + k); };
  float top = -INFINITY;
  for (int k = lane; k < parts; k += 32) {
    const float* st = p.part_s + slot(k) * 3 * p.row_slots + rr;
    if (st[p.row_slots] != 0.f) top = fmaxf(top, st[0]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (top == -INFINITY) top = 0.f;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float l = 0.f, lt = 0.f;
#pragma unroll 4
  for (int k = warp; k < parts; k += kJoinWarps) {
    const float* st = p.part_s + slot(k) * 3 * p.row_slots + rr;
    const float m = st[0], lk = st[p.row_slots], ltk = st[2 * p.row_slots];
    const float* o = p.part_o + (slot(k) * p.row_slots + rr) * D + lane * E;
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = o[e];
    const float f = lk == 0.f ? 0.f : fast_exp2(m - top);
    l += lk * f;
    lt += ltk * f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f == 0.f ? 0.f : v[e] * f;
  }
  if (lane == 0) {
    sl[warp][0] = l;
    sl[warp][1] = lt;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
  __syncthreads();
  if (threadIdx.x >= D) return;
  l = lt = 0.f;
  float val = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) {
    l += sl[k][0];
    lt += sl[k][1];
    val += so[k][threadIdx.x];
  }
  const int tok = row / p.group, h = hk * p.group + (row - tok * p.group);
  const int64_t out_row = ((int64_t)b * p.t.heads + h) * p.t.n + tok;
  const float x = l == 0.f ? 0.f : val / lt;
  if (p.t.out_f32) static_cast<float*>(p.t.o)[out_row * D + threadIdx.x] = x;
  else static_cast<uint16_t*>(p.t.o)[out_row * D + threadIdx.x] = (uint16_t)pack_bf16x2(x, 0.f);
  if (threadIdx.x == 0 && p.t.lse) p.t.lse[out_row] = l == 0.f ? -INFINITY : (top + fast_log2(l)) * 0.69314718055994531f;
}

struct WorkspaceLayout {
  int64_t row_slots, part_o, part_s, bytes;  // offsets in bytes
};
WorkspaceLayout workspace_layout(int64_t batch, int64_t rows, int64_t d) {
  WorkspaceLayout w;
  w.row_slots = rows < 256 ? rows : 256;
  w.part_o = ((batch + 1) * 4 + 15) / 16 * 16;
  w.part_s = w.part_o + 2 * kMaxCtas * w.row_slots * d * 4;
  w.bytes = w.part_s + 2 * kMaxCtas * 3 * w.row_slots * 4;
  return w;
}

template <int D, int QROWS>
cudaError_t launch_rows(const TreeParams& p, const CUtensorMap* maps, cudaStream_t stream) {
  using C = TreeCfg<D, QROWS>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(tree_kernel<D, QROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  tree_kernel<D, QROWS><<<kMaxCtas, kThreads, C::SMEM_BYTES, stream>>>(maps[0], maps[1], p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const TreeParams& p, const CUtensorMap* maps, cudaStream_t stream) {
  cudaError_t e = p.rows > 128  ? launch_rows<D, 256>(p, maps, stream)
                  : p.rows > 64 ? launch_rows<D, 128>(p, maps, stream)
                                : launch_rows<D, 64>(p, maps, stream);
  if (e != cudaSuccess) return e;
  // a programmatic dependent launch: its blocks are resident and wait when the
  // last part is written
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.t.cache.batch * p.t.cache.kv_heads * p.rows));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_join_kernel<D>, p, kMaxCtas);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

int64_t tree_workspace_bytes(int32_t batch, int32_t kv_heads, int32_t heads, int32_t n, int32_t head_dim) {
  return workspace_layout(batch, (int64_t)(heads / kv_heads) * n, head_dim).bytes;
}

cudaError_t launch_tree(const TreeLaunch& t, const CUtensorMap* maps, cudaStream_t stream) {
  TreeParams p;
  p.t = t;
  p.group = t.heads / t.cache.kv_heads;
  p.rows = p.group * t.n;
  p.pairs = (p.rows + 255) / 256;
  p.mask_words = (t.n + 31) / 32;
  p.scale_log2 = t.scale * 1.4426950408889634f;
  const WorkspaceLayout w = workspace_layout(t.cache.batch, p.rows, t.head_dim);
  uint8_t* ws = static_cast<uint8_t*>(t.workspace);
  p.row_slots = (int32_t)w.row_slots;
  p.starts = reinterpret_cast<int32_t*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  p.part_s = reinterpret_cast<float*>(ws + w.part_s);
  switch (t.head_dim) {
    case 64: return launch_d<64>(p, maps, stream);
    case 96: return launch_d<96>(p, maps, stream);
    default: return launch_d<128>(p, maps, stream);
  }
}

}  // namespace wise
