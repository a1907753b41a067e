// Shared parts of the kernels that attend new tokens over a paged cache: WISE
// ("Attention Routing Stabilizes Early: Working-Set Inference for Recurrent
// Language Models") §3 Eq 2 for the rows behind the prompt -- a next token, a
// run of tokens, a tree of drafted tokens.
//
//   O_i = sum_j a_ij v_j,  a_ij = exp(s_ij - LSE_i),  s_ij = scale q_i k_j,
//   LSE_i = log sum_j exp(s_ij), over the committed tokens j and the drafted
//   tokens that row i's mask lists.
//
// A unit is one (sequence, key head) and up to 256 of the rows that share its
// keys: the queries of a group of heads times the new tokens, row = token *
// group + head of the group. The key tiles (128 tokens) of all units form one
// line of work that is cut into equal parts, one per CTA, so that lengths may
// differ and one long sequence fills the GPU. A unit that a cut divides leaves
// partial results (unnormalised O, running maximum, sum), which the join
// kernel joins in the line's order. Each unit's tiles follow `overhead` places
// of the line that stand for the change from one unit to the next (results
// out, Q in, the pipeline filled again), so that a CTA whose part holds such a
// change has fewer tiles.
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace wise {

constexpr int kTile = 128;       // keys per tile
constexpr int kTreeCtas = 152;   // SMs of a GB300
constexpr int kNfRing = 16;      // segments whose taken-out values are remembered

// A unit's partial results: CTA `first_cta`'s part `first_part`, then part
// 2 c of each later CTA c. parts 1: the unit was not cut, its rows are in the
// launch's own outputs (only the join of shared prefixes reads those); less: no
// record.
struct JoinRec {
  int32_t parts, first_part, first_cta, b, hk, pair, pad0, pad1;
};

struct TreeParams {
  TreeLaunch t;
  int32_t group;        // query heads per key head
  uint32_t group_mul;   // ceil(2^32 / group), for rows / group
  int32_t rows;         // rows of a (sequence, key head): group * n; of a group of sequences: times its members, at most
  int32_t pairs;        // units per (sequence, key head): ceil(rows / 256)
  int32_t row_slots;    // rows of a partial result: min(rows, 256), in whole blocks of 32 for wide units
  int32_t mask_words;   // words of a mask row
  int32_t recs;         // join records: one per unit if there are at most kTreeCtas or a
  int32_t by_unit;      // join reads all units (TreeLaunch::rows_apart), else one per CTA
  int32_t overhead;     // places of the line before a unit's tiles
  float scale_log2;
  JoinRec* rec;
  // [2 * kTreeCtas][row_slots * d]: rows of d values for narrow units; for wide
  // ones, whose threads hold a row each, blocks of 32 rows with four values of
  // each row next to each other: [row / 32][d / 4][row % 32][4]
  float* part_o;
  float* part_s;        // [2 * kTreeCtas][2][row_slots]: maximum (log2), sum
};

// row / group; exact for row * group < 2^32 (wise_attn_tree admits groups of at
// most 4096 heads and 128 tokens).
__device__ __forceinline__ int row_token(const TreeParams& p, int row) {
  return p.group == 1 ? row : (int)__umulhi((uint32_t)row, p.group_mul);
}

// Asynchronous 16-byte copy into shared memory (no registers, nothing to wait
// for between copies, so the loop over them stays small: a kernel that runs
// for a few microseconds spends much of them on fetching its own code).
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Tokens at the front of sequence b that are left out (whole tiles).
__device__ __forceinline__ int seq_skip(const TreeLaunch& t, int b) { return t.skip ? t.skip[b] : 0; }

// Committed and new tokens of sequence b, clamped to what the page table
// holds; true if nothing had to be clamped. PREFIX: shared tokens and rows
// (tokens of all its sequences) of group b.
template <bool PREFIX>
__device__ __forceinline__ bool seq_counts(const TreeLaunch& t, int b, int& len, int& nl) {
  if constexpr (PREFIX) {
    len = t.cache.lengths[b];
    nl = len > 0 ? (t.starts[b + 1] - t.starts[b]) * t.n : 0;
    return true;
  } else {
    const int64_t cap = (int64_t)t.cache.max_pages << t.cache.page_shift;
    const int64_t l0 = t.cache.lengths[b];
    const int n0 = t.new_len ? t.new_len[b] : t.n;
    const int64_t l = l0 < 0 ? 0 : (l0 > cap ? cap : l0);
    int n = n0 < 0 ? 0 : (n0 > t.n ? t.n : n0);
    if (l + n > cap) n = (int)(cap - l);
    len = (int)l - seq_skip(t, b);
    nl = n;
    return l == l0 && n == n0;
  }
}
// The page table's entries of sequence b (of group b: of the sequence that stands for it) from
// the first token on that is not left out.
template <bool PREFIX>
__device__ __forceinline__ const int32_t* seq_table(const TreeLaunch& t, int b) {
  if constexpr (PREFIX) return t.cache.page_table + (int64_t)t.leader[b] * t.cache.max_pages;
  else return t.cache.page_table + (int64_t)b * t.cache.max_pages + (seq_skip(t, b) >> t.cache.page_shift);
}
// Key tiles (`full`) of a unit that holds a valid token's row, and how many
// units of a key head do (`active`); each other unit counts one empty tile
// (PREFIX: there are no others).
template <bool PREFIX>
__device__ __forceinline__ void seq_tiles(const TreeParams& p, int len, int nl, int& full, int& active) {
  const int keys = PREFIX ? len : len + nl;
  full = keys > 0 ? (keys + kTile - 1) / kTile : 1;
  active = (nl * p.group + 255) / 256;
  if (active > p.pairs) active = p.pairs;
}
template <bool PREFIX>
__device__ __forceinline__ int seq_line(const TreeParams& p, int full, int active) {
  if constexpr (PREFIX) return p.t.cache.kv_heads * active * (full + p.overhead);
  else return p.t.cache.kv_heads * (active * full + (p.pairs - active) + p.pairs * p.overhead);
}

// The line as one CTA sees it: CTA c's part begins at place c * per + c * more
// / ctas (= c * total / ctas); and the CTA's first segment.
struct LinePart {
  int per, more, ctas;
  int x1;    // end of the part
  int left;  // places from the first segment's first tile on (<= 0: nothing to do)
  int b, hk, pair, t0, len, nl;
  __device__ __forceinline__ int begin(int c) const { return c * per + c * more / ctas; }
  // the CTA whose part holds place x
  __device__ __forceinline__ int owner(int x) const {
    int c = min((int)((float)x / ((float)per + (float)more / (float)ctas)), ctas - 1);
    while (c > 0 && begin(c) > x) --c;
    while (c + 1 < ctas && begin(c + 1) <= x) ++c;
    return c;
  }
};

// The lengths and the page table into L2 while the kernel before this one may
// still run (nothing is read; a line that it writes is written there). The
// first tiles wait for three loads in a row -- lengths, page table, keys --
// each of which takes a microsecond or two from a cold memory.
__device__ __forceinline__ void prefetch_tables(const TreeParams& p) {
  auto prefetch = [](const void* a) { asm volatile("prefetch.global.L2 [%0];" ::"l"(a)); };
  const int64_t line = (int64_t)threadIdx.x * 32;  // 32 entries of 4 bytes
  if (line < p.t.cache.batch) {
    prefetch(p.t.cache.lengths + line);
    if (p.t.new_len) prefetch(p.t.new_len + line);
  }
  // the table: a line per thread of the grid
  const int64_t at = line * gridDim.x + (int64_t)blockIdx.x * 32;
  if (at < (int64_t)p.t.cache.batch * p.t.cache.max_pages) prefetch(p.t.cache.page_table + at);
}

// Every thread sums the tiles of consecutive sequences, the block scans the
// sums, and the thread whose sequences hold the part's first tile finds it
// there. `blocks` of the grid share the line. Two block barriers; `scratch` holds
// warps + 12 words.
template <int THREADS, bool PREFIX = false>
__device__ __forceinline__ void find_part(const TreeParams& p, int* scratch, LinePart& part, int blocks) {
  constexpr int WARPS = THREADS / 32;
  int* sums = scratch;
  int* found = scratch + WARPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int batch = p.t.cache.batch;
  const int per = (batch + THREADS - 1) / THREADS;
  const int b_lo = min(batch, (int)threadIdx.x * per), b_hi = min(batch, b_lo + per);
  int mine = 0;
  int last_len = 0, last_nl = 0;  // of sequence b_hi - 1 (most batches: the thread's only one)
  bool good = true;
  for (int b = b_lo; b < b_hi; ++b) {
    int fl, ac;
    good &= seq_counts<PREFIX>(p.t, b, last_len, last_nl);
    seq_tiles<PREFIX>(p, last_len, last_nl, fl, ac);
    mine += seq_line<PREFIX>(p, fl, ac);
  }
  if (!good && blockIdx.x == 0) atomicOr(p.t.err, kErrBadCache);
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) sums[warp] = before;
  before -= mine;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  const int cta = blockIdx.x;
  part.ctas = max(min(blocks, total), 1);  // (an empty line: a batch that shares nothing)
  part.per = total / part.ctas;
  part.more = total - part.per * part.ctas;
  const int x0 = cta < part.ctas ? part.begin(cta) : total;
  const int x1 = cta < part.ctas ? part.begin(cta + 1) : total;
  if (x0 >= before && x0 < before + mine) {  // (x0 is the line's end without a part)
    int at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      int len = last_len, nl = last_nl, fl, ac;
      if (b + 1 < b_hi) seq_counts<PREFIX>(p.t, b, len, nl);
      seq_tiles<PREFIX>(p, len, nl, fl, ac);
      const int line = seq_line<PREFIX>(p, fl, ac);
      if (x0 >= at && x0 < at + line) {
        const int ov = p.overhead, per_head = line / p.t.cache.kv_heads;
        const int hk = (x0 - at) / per_head;
        int r = x0 - at - hk * per_head, pair;
        if (r < ac * (fl + ov)) {
          pair = r / (fl + ov);
          r -= pair * (fl + ov);
        } else {
          pair = ac + (r - ac * (fl + ov)) / (1 + ov);
          r -= ac * (fl + ov) + (pair - ac) * (1 + ov);
        }
        found[0] = b;
        found[1] = hk;
        found[2] = pair;
        found[3] = max(r - ov, 0);               // first tile
        found[4] = x1 - x0 - max(ov - r, 0);     // places from there on
        found[5] = len;
        found[6] = nl;
        break;
      }
      at += line;
    }
  }
  __syncthreads();
  part.x1 = x1;
  part.left = x1 > x0 ? found[4] : 0;
  part.b = found[0];
  part.hk = found[1];
  part.pair = found[2];
  part.t0 = found[3];
  part.len = found[5];
  part.nl = found[6];
}

// A CTA's walk over its part, a segment (consecutive key tiles of one unit) at
// a time. Every role keeps its own.
template <bool PREFIX>
struct WalkOf {
  int b, hk, pair;  // PREFIX: b is a group
  int len, nl, full, active;
  int t0, t1, nt;  // tiles [t0, t1) of the unit's nt
  int keys;        // tokens that the unit's rows may see
  int left;        // places of the part from tile t0 on
  int seg;         // segments before this one

  __device__ __forceinline__ void unit() {
    const bool on = pair < active;
    nt = on ? full : 1;
    keys = on ? (PREFIX ? len : len + nl) : 0;
    t1 = min(nt, t0 + left);
  }
  __device__ __forceinline__ void start(const TreeParams& p, const LinePart& f) {
    b = f.b;
    hk = f.hk;
    pair = f.pair;
    len = f.len;
    nl = f.nl;
    t0 = f.t0;
    left = f.left;
    seg = 0;
    seq_tiles<PREFIX>(p, len, nl, full, active);
    unit();
  }
  __device__ __forceinline__ bool next(const TreeParams& p) {
    left -= t1 - t0 + p.overhead;
    if (left <= 0) return false;
    ++seg;
    t0 = 0;
    if (++pair == (PREFIX ? active : p.pairs)) {
      pair = 0;
      if (++hk == p.t.cache.kv_heads) {
        hk = 0;
        do {
          ++b;
          seq_counts<PREFIX>(p.t, b, len, nl);
          seq_tiles<PREFIX>(p, len, nl, full, active);
        } while (PREFIX && active == 0);  // (places are left, so a group with rows follows)
      }
    }
    unit();
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
  // partial result of this segment: 2 c for the part's first segment, 2 c + 1
  // for its last
  __device__ __forceinline__ int part() const { return 2 * (int)blockIdx.x + (seg == 0 ? 0 : 1); }
  // rows of the sequence (of the group) and key head
  __device__ __forceinline__ int rows(const TreeParams& p) const { return PREFIX ? nl * p.group : p.rows; }
};
using Walk = WalkOf<false>;

// A row's sequence and token: `tok` counts the tokens of all of a group's
// sequences with PREFIX (tok < nl: the group has such a row).
struct RowPlace {
  int b, i;
};
template <bool PREFIX>
__device__ __forceinline__ RowPlace row_place(const TreeLaunch& t, int b, int tok) {
  if constexpr (!PREFIX) return RowPlace{b, tok};
  const int m = tok / t.n;
  return RowPlace{t.starts[b] + m, tok - m * t.n};
}
// Whether the row's token is one of its sequence's new ones.
template <bool PREFIX>
__device__ __forceinline__ bool row_live(const TreeLaunch& t, const RowPlace& r, int tok, int nl) {
  if (tok >= nl) return false;
  return !PREFIX || r.i < t.new_len[r.b];
}

// The join record of the unit whose first tile lies in this segment (one
// thread calls it for every segment, and first clear_rec).
__device__ __forceinline__ void clear_rec(const TreeParams& p) {
  if (!p.by_unit) p.rec[blockIdx.x].parts = 0;
}
// No unit is joined (a CTA that cannot work).
__device__ __forceinline__ void clear_recs(const TreeParams& p) {
  for (int i = threadIdx.x; i < p.recs; i += blockDim.x) p.rec[i].parts = 0;
}
// Place of a unit's record where each has one. PREFIX: a group's units follow those
// of the rows before it, one place later for each group (its last unit may be part
// of 256 rows only).
template <bool PREFIX>
__device__ __forceinline__ int64_t unit_rec(const TreeParams& p, int b, int hk, int pair) {
  if constexpr (PREFIX)
    return ((int64_t)p.t.starts[b] * p.t.n * p.group / 256 + b + pair) * p.t.cache.kv_heads + hk;
  else return ((int64_t)b * p.t.cache.kv_heads + hk) * p.pairs + pair;
}
template <bool PREFIX>
__device__ __forceinline__ void write_rec(const TreeParams& p, const LinePart& f, const WalkOf<PREFIX>& w) {
  if (w.t0 != 0) return;
  const bool cut = w.t1 < w.nt;
  JoinRec r = {1, 0, (int)blockIdx.x, w.b, w.hk, w.pair, 0, 0};
  if (cut) {
    // up to the CTA that holds the unit's last tile, w.nt - w.t1 places past
    // the end of this part
    r.parts = f.owner(f.x1 + (w.nt - w.t1) - 1) - (int)blockIdx.x + 1;
    r.first_part = w.part();
  }
  if (p.by_unit) p.rec[unit_rec<PREFIX>(p, w.b, w.hk, w.pair)] = r;
  else if (cut) p.rec[blockIdx.x] = r;
}

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
__device__ __forceinline__ bool page_ok(const TreeLaunch& t, int32_t pg) { return pg >= 0 && (int64_t)pg < t.cache.n_pages; }

// Wait until ring position `pos` is loaded. A wait for a barrier's phase parity
// alone is not enough where a consumer skips uses of a slot: while the use
// before is still being copied the barrier reads as done for the use after it
// (copies may end in another order than they began). The producer names the
// use that a slot is in, which says that every earlier one is over.
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

// The ring of K and V tiles in shared memory: position 2 tau holds K of the
// CTA's tile tau, 2 tau + 1 its V, position x in slot x % NS.
// A tile's rows lie in chunks of 64 values (128 swizzled bytes). For 96
// dimensions the second chunk's upper half lies past the tensor and is filled
// with zeros: chunks of 32 values would need no room for them, but half as many
// copy requests again (rows of 64 bytes).
constexpr uint32_t kRowBytes = 128u;
constexpr uint32_t kSwizzle128 = 2u;  // descriptor code
template <int D>
__host__ __device__ constexpr int row_chunks() { return (D + 63) / 64; }
template <int D>
__host__ __device__ constexpr uint32_t tile_bytes(int rows) { return (uint32_t)rows * row_chunks<D>() * kRowBytes; }
// Byte offset of a row's 16-byte unit u in a tile of `rows` rows.
__device__ __forceinline__ uint32_t unit_offset(int rows, int row, int u) {
  return (uint32_t)((u >> 3) * rows + row) * kRowBytes + (uint32_t)((u & 7) ^ (row & 7)) * 16u;
}
template <int D, int NS>
struct RingCfg {
  static constexpr int NCH = row_chunks<D>();  // TMA boxes per page
  static constexpr uint32_t KV_BYTES = tile_bytes<D>(kTile);
  // Ring position pos (odd: a V tile) is its slot's use number pos / NS; with
  // an odd number of slots every other use of a slot is a V tile.
  __device__ static constexpr uint32_t guard_phase(uint32_t pos) { return (NS & 1) ? (pos / NS) >> 1 : pos / NS; }
};
struct Ring {
  uint8_t* tiles;
  uint64_t* full;       // [NS] tile loaded
  uint64_t* empty;      // [NS] tile no longer needed
  uint64_t* guarded;    // [NS] V tile passed by the guard
  uint32_t* uses;       // [NS] one past the ring position that the slot is used for
  uint32_t* flags;      // [kTileFlags] see tile_bad
};

// Pages of the CTA's tile `tile` that are not in the pool (bit i: page i of the
// tile), as the producer found them. Its word names the tile, so that a reader
// knows the word for its own (nothing else hangs on it, so it needs no acquire:
// that took 100 cycles a tile); the ring holds far fewer than kTileFlags tiles.
constexpr int kTileFlags = 16;
__device__ __forceinline__ uint32_t tile_word(uint32_t tile, uint32_t bad) { return ((tile + 1u) << 8) | bad; }
template <int TAG>
static __device__ __noinline__ uint32_t tile_bad_slow(const uint32_t* flag, uint32_t tile, volatile int* abort_flag,
                                                      uint32_t* err) {
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    const uint32_t v = *reinterpret_cast<const volatile uint32_t*>(flag);
    if ((v >> 8) == (tile_word(tile, 0u) >> 8)) return v & 0xffu;
    if (*abort_flag) return 0u;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      atomicOr(err, kErrTimeout);
    }
  }
}
// (called once the tile's copies or MMAs were seen done, so the word is there
// or a few cycles away)
template <int TAG>
__device__ __forceinline__ uint32_t tile_bad(const Ring& ring, uint32_t tile, volatile int* abort_flag, uint32_t* err) {
  const uint32_t* flag = &ring.flags[tile % kTileFlags];
  const uint32_t v = *reinterpret_cast<const volatile uint32_t*>(flag);
  if ((v >> 8) == (tile_word(tile, 0u) >> 8)) return v & 0xffu;
  return tile_bad_slow<TAG>(flag, tile, abort_flag, err);
}

// The warp that loads the ring, page by page (whole warp; lane i issues the
// tile's page i).
template <int D, int NS, int TAG, bool PREFIX>
__device__ __forceinline__ void ring_producer(const TreeParams& p, WalkOf<PREFIX> w, const Ring& ring, const CUtensorMap* tm_k,
                                              const CUtensorMap* tm_v, volatile int* abort_flag, int lane) {
  using C = RingCfg<D, NS>;
  uint32_t* err = p.t.err;
  const int page = 1 << p.t.cache.page_shift;
  const int boxes = kTile >> p.t.cache.page_shift;  // pages per tile
  const uint32_t box_bytes = tile_bytes<D>(page);
  uint32_t pos = 0;
  bool ok = true, flagged = false;
  do {
    const int32_t* table = seq_table<PREFIX>(p.t, w.b);
    const int last_page = (w.keys - 1) >> p.t.cache.page_shift;  // -1: none
    // the lanes hold 32 columns of the page table from `have` on, and the 32
    // after them, which are under way while these are used
    int have = w.t0 * boxes;
    auto columns = [&](int c) -> int32_t { return c + lane <= last_page ? table[c + lane] : -1; };
    int32_t held = columns(have), ahead = columns(have + 32);
    for (int t = w.t0; ok && t < w.t1; ++t) {
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
      if (lane == 0) *reinterpret_cast<volatile uint32_t*>(&ring.flags[(pos >> 1) % kTileFlags]) = tile_word(pos >> 1, bad);
      for (int kv = 0; kv < 2 && ok; ++kv, ++pos) {
        const int slot = (int)(pos % NS);
        if (pos >= (uint32_t)NS)
          ok = __all_sync(0xffffffffu, mbar_wait<TAG>(&ring.empty[slot], ((pos / NS) - 1) & 1, abort_flag, err));
        if (!ok) break;
        if (lane == 0) {
          st_release_smem(&ring.uses[slot], pos + 1u);
          mbar_arrive_expect_tx(&ring.full[slot], (uint32_t)__popc(loads) * box_bytes);
        }
        __syncwarp();
        if (good) {
          uint8_t* dst = ring.tiles + slot * C::KV_BYTES + (uint32_t)(lane * page) * kRowBytes;
#pragma unroll
          for (int c = 0; c < C::NCH; ++c)
            tma_load_3d(dst + c * kTile * kRowBytes, kv ? tm_v : tm_k, &ring.full[slot], c * 64, w.hk * page, pg);
        }
        __syncwarp();
      }
    }
  } while (ok && w.next(p));
  // No copy into this CTA's shared memory may outlive the CTA.
  if (lane == 0) {
    int none = 0;
    for (uint32_t i = (pos > (uint32_t)NS ? pos - NS : 0u); i < pos; ++i)
      mbar_wait<TAG>(&ring.full[i % NS], (i / NS) & 1, &none, err);
  }
  __syncwarp();
}

// The warp that guards V: in tiles that hold drafted tokens or end past the
// last token, rows that nobody may see are cleared (0 times what lies there
// could be NaN), and infinities and NaN of drafted tokens are taken out, since
// 0 times them would reach rows that do not see them. nf[seg % kNfRing][4]
// names those tokens; their values are put back at the end for the rows that
// see them. The ring holds fewer than kNfRing tiles, so a list is not reused
// before its segment's results are out.
template <int D, int NS, int TAG, bool PREFIX>
__device__ __forceinline__ void ring_guard(const TreeParams& p, WalkOf<PREFIX> w, const Ring& ring, uint32_t* nf,
                                           volatile int* abort_flag, int lane) {
  using C = RingCfg<D, NS>;
  static_assert(NS / 2 + 2 < kNfRing && NS / 2 + 4 < kTileFlags, "nf ring, tile flags");
  const int page = 1 << p.t.cache.page_shift;
  uint32_t pos = 1;
  bool ok = true;
  do {
    uint32_t* seg_nf = nf + (w.seg % kNfRing) * 4;
    if (lane < 4) seg_nf[lane] = 0u;
    __syncwarp();
    for (int t = w.t0; ok && t < w.t1; ++t, pos += 2) {
      const int slot = (int)(pos % NS);
      ok = __all_sync(0xffffffffu, wait_loaded<TAG>(ring.full, ring.uses, NS, pos, abort_flag, p.t.err));
      if (!ok) break;
      const uint32_t bad = tile_bad<TAG>(ring, pos >> 1, abort_flag, p.t.err);
      const int kb = t * kTile;
      uint8_t* v = ring.tiles + slot * C::KV_BYTES;
      if (bad != 0u || kb + kTile > w.len || w.keys == 0) {
        const int rows = max(0, min(w.keys - kb, kTile));
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int c = 0; c < C::NCH; ++c) {
          uint8_t* vc = v + c * kTile * kRowBytes;
          for (uint32_t x = rows * kRowBytes + lane * 16; x < kTile * kRowBytes; x += 512) *reinterpret_cast<uint4*>(vc + x) = zero;
          for (uint32_t m = bad; m != 0u; m &= m - 1u) {
            const uint32_t at = (uint32_t)((__ffs(m) - 1) * page) * kRowBytes;
            for (uint32_t x = lane * 16; x < page * kRowBytes; x += 512) *reinterpret_cast<uint4*>(vc + at + x) = zero;
          }
        }
        __syncwarp();
        // drafted tokens' rows of the tile (the swizzle permutes 16-byte
        // units within a row, so a row's units are visited in any order)
        constexpr int U = kRowBytes / 16;
        for (int x = max(0, w.len - kb) * U + lane; x < rows * U; x += 32)
          for (int c = 0; c < C::NCH; ++c) {
            uint4* at = reinterpret_cast<uint4*>(v + c * kTile * kRowBytes) + x;
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
      if (lane == 0) mbar_arrive(&ring.guarded[slot]);
    }
  } while (ok && w.next(p));
  __syncwarp();
}

// The wait for the launch before this one: at the start, or, for a launch that runs
// beside it, at the end, since a launch must not end before those it follows. A
// launch beside another starts when every block of that one has triggered, each
// after its own wait for the plan, so the plan is complete; but only a wait of its
// own would make what was written before visible here. Instead one thread acquires
// the word that the plan released last, whose tag shows that it is this call's (the
// join takes it back, so no earlier call with this workspace has left one). That
// orders everything that the plan's own wait had made visible, and the barrier hands
// it on to the block; the fence does so for copies by TMA. Returns the blocks that
// share the work (the others leave at once), or -1: the word is not there (it is not
// waited for). `blocks`: a word of shared memory. (In graphs, against a fence without
// the word: 64 next tokens behind 32K 78.0 instead of 77.4 us, trees of three groups
// 46.4 and 46.8.) PREFIX: the shared part, which waits, on a share of the SMs.
template <bool PREFIX>
__device__ __forceinline__ int wait_at_start(const TreeLaunch& t, volatile uint32_t* blocks) {
  if (PREFIX || !t.go) {
    grid_wait();
    return PREFIX ? *t.limit : (int)gridDim.x;
  }
  if (threadIdx.x == 0) {
    const uint64_t word = ld_acquire_gpu(t.go);
    *blocks = (word ^ kPlanTag) >> 32 == 0u ? (uint32_t)word : 0xffffffffu;
  }
  __syncthreads();
  asm volatile("fence.proxy.async.global;" ::: "memory");
  return (int)*blocks;
}
template <bool PREFIX>
__device__ __forceinline__ void wait_at_end(const TreeLaunch& t) {
  if (!PREFIX && t.go) grid_wait();
}

// Row pointer of drafted token j's values in the pool, or null.
__device__ __forceinline__ const uint16_t* draft_value(const TreeLaunch& t, int d, int b, int hk, int len, int j) {
  const int64_t tok = (int64_t)len + j;
  const int32_t pg = seq_table<false>(t, b)[tok >> t.cache.page_shift];
  if (!page_ok(t, pg)) return nullptr;
  return t.cache.v_pages + ((((int64_t)pg * t.cache.kv_heads + hk) << t.cache.page_shift) +
                            (tok & ((1 << t.cache.page_shift) - 1))) * d;
}

// Up to 64 rows per unit (tree_narrow.cuh), and more (tree_wide.cuh, with the
// join of either's partial results). PREFIX: the rows of a group of sequences
// over the tokens that they share.
template <bool PREFIX>
cudaError_t launch_tree_narrow(const TreeParams& p, const CUtensorMap* maps, cudaStream_t stream);
template <bool PREFIX>
cudaError_t launch_tree_rows(const TreeLaunch& t, const CUtensorMap* maps, cudaStream_t stream);
extern template cudaError_t launch_tree_narrow<false>(const TreeParams&, const CUtensorMap*, cudaStream_t);
extern template cudaError_t launch_tree_narrow<true>(const TreeParams&, const CUtensorMap*, cudaStream_t);
extern template cudaError_t launch_tree_rows<false>(const TreeLaunch&, const CUtensorMap*, cudaStream_t);
extern template cudaError_t launch_tree_rows<true>(const TreeLaunch&, const CUtensorMap*, cudaStream_t);

}  // namespace wise
