// lsa_window_attn and lsa_prefix_decode_attn: attention read in place from the
// paged KV pools, without a compact copy.
//
//   window:  the query at position p of its sequence sees the keys j <= p with
//            j > p - window or j < n_sink, for prompts, pieces of prompts and
//            single tokens of one batch;
//   prefix:  one decode step of a batch whose groups share a prefix: each
//            sequence sees its group's prefix, then its own tokens, and the
//            prefix is read once for the whole group.
//
//   out = sum_j softmax_j(scale q . k_j) v_j
//
// One kernel serves both.  The work is two lists of units; a unit is 64 tokens
// (one chunk) of K and V of one KV head, 32 KiB, against the queries of a tile:
//   wide tiles    9 to 32 queries (x 8 query heads): prompts, large groups;
//   narrow tiles  up to 8: single tokens, the tokens behind a shared prefix.
// The units of a list's tiles are laid end to end (a tile's also count kTileCost
// more, for its start and its end) and cut into equal contiguous shares: one per
// CTA for the wide list, two per CTA for the narrow one.  So one token over a long
// window, a ragged batch and a long prompt all fill the chip evenly.  A call with
// both gives each list its own CTAs, as many as its units cost (every CTA with a
// share of both, one after the other, takes 12% longer for 32 sequences over a prefix
// of 32768 tokens and up to 1024 of their own, 25% for 33 queries over 512 tokens).
// A tile that a cut splits leaves partials (normalised rows and their log-sum-exps),
// which are folded in the order of the shares, so that the result does not depend on
// timing: by the share that adds a tile's last one where that is little for one SM
// (single tokens: no second launch), else by a second kernel (32 sequences over a
// prefix of 32768 tokens leave 19 MB).
//
// A CTA (one per SM, 12 warps) has two pipelines w = 0, 1 of
//   warps 4w..4w+3  a softmax warpgroup, a thread per row: the scores of a unit
//                   come from TMEM, the probabilities go back in their place as
//                   bf16.  The running maximum is only raised when it grows by
//                   2^8 or more (the sums stay exact, the accumulator is rescaled
//                   rarely);
//   warp 8 + w      issues the tcgen05.mma: S = Q K^T (128 x 64 x 128) into one
//                   of two score buffers, O += P V (128 x 128 x 64) with P from
//                   TMEM;
//   warp 10 + w     plans and loads (TMA).
// In a wide share both pipelines use every unit, each with half of the tile's
// queries; warp 10 streams K and V through all 8 half-stages of 16 KiB, warp 11
// walks the list a few segments ahead and loads the queries.  Of the narrow shares
// each pipeline has one, with its own stream through 4 half-stages, so that one's
// start of a tile, its latencies and its end run beside the other's units; that
// carries single tokens at the rate of the memory although 8 of the 128 rows of a
// product are theirs.
//
// What bounds it.  Narrow shares: memory (one token over 100000: 70.6 us, 5.8 TB/s,
// 89% of the copy rate; 64 tokens over windows of 1024: 55.0 us, 4.9 TB/s, the rest is
// the start, 5 us, and the spread of the CTAs' ends).  Wide shares: the chain of a
// unit, 1450 cycles for 128 x 2 rows, of which the tensor core is busy 1350 (with
// 64 keys a product of scores is fed by shared memory: 48 KiB in 384 cycles for 256 of
// products); and what is no unit: of the 139.6 us of a prompt of 4096 queries over a
// window of 1024 (0.86 PFLOP/s) its 108 units a CTA are about 82, the ends of 7 tiles
// some 25, the merge 11, the start 5 to 7.  Without the softmax's arithmetic it would
// take 92%.  Single tokens over short contexts: latency, about 5 us until the first
// scores, 1.5 us a unit, 2 us for the fold.  (Times are of calls in a row; a single one
// after a flush of the L2 cache takes 5 to 25 us longer.)
//
// TMEM (512 columns): scores 2 pipelines x 2 buffers x 64, accumulators 2 x 128.
// Rows that no query of a tile sees are zeroed in V's stage before the product,
// so a page's unwritten tail may hold anything (0 times NaN is NaN); the scores
// there are masked by selection.
#include <math.h>
#include <math_constants.h>

#include <atomic>
#include <mutex>

#include "lsa_common.cuh"
#include "lsa_runtime.cuh"

namespace lsa {
namespace pool {

// Queries of a wide tile, of a narrow one.  Narrow up to 8, whose rows fill half of a
// product (up to 4): 8 queries each of 64 sequences over windows of 1024 57.4 (74.8)
// us, of 16 25.4 (29.2), of one over 4096 tokens 17.1 (17.6).
constexpr int kWideQ = 32, kNarrowQ = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 10;  // of pipeline 0; 9 and 11 are pipeline 1's
constexpr int kThreads = 12 * 32;
constexpr int kHalves = 8;                   // half-stages: a unit's K or V of one head
constexpr int kBoxBytes = 8192;              // 64 tokens x 64 dims
constexpr int kPartRows = 16, kPartBytes = kPartRows * 128;   // of a chunk that is not seen whole: 16 tokens x 64 dims
constexpr int kHalfBytes = 2 * kBoxBytes;
constexpr int kQBoxBytes = 16384;            // 128 rows x 64 dims
constexpr int kQTileBytes = 2 * kQBoxBytes;
constexpr int kQ2Bytes = 8192;               // a pipeline's second narrow query tile: rows 64.. of its region
constexpr int kTurnBytes = 4096;             // a warp's rows on their way out: 32 rows x 128 bytes
constexpr int kAhead = 4;                    // places for segments that a planner is ahead
constexpr int kMaxCtas = LSA_POOL_ATTN_MAX_CTAS;
constexpr int kTileCost = 3;                 // 2 to 5 measured alike
constexpr int kMinShare = 3;                 // smallest share of a list worth a pipeline (or a CTA) of its own: one token
                                             // over 4096 takes 14.9 us with 2, 14.2 with 3, 14.5 with 4
// What a wide unit costs on a CTA, in narrow ones (two pipelines, each with its own).
// Shared prefixes, groups x sequences over prefix + own tokens: 24 over 8000 + 100
// take 26.2 us (1.5: 27.0, 2.3: 26.2), 64 over 8000 + 2000 64 (70, 67), 5 x 26 over
// 16384 + 512 116 (121, 127); pieces of 30 over a window of 1024 64 (69, 67).
constexpr float kWideCost = 1.8f;
constexpr int kFmaEvery = 4;                 // of the pairs of powers of two, one in 4 on the FMA pipe
constexpr float kRaise = 8.f;                // growth of the maximum (log2) that rescales the accumulator
// The maximum of a row that has seen keys whose scores are all -inf, and the
// log-sum-exp of a partial of only such; -inf: it has seen none.  A row that ends
// so is 0 / 0, one without a key zeros.  (Below every maximum of finite scores, so
// that the first of them replaces it and weighs its partials 0.)
constexpr float kLowest = -3.402823466e38f;
constexpr int kSCols = 64, kOCol0 = 256;     // TMEM: S[w][b] at (2 w + b) * 64, O[w] at 256 + 128 w

struct Plan {
  int B, groups;             // groups: prefix mode only
  int64_t rows;              // queries in q
  const int32_t* cu;         // cu_q [B + 1], or cu_group [groups + 1]
  const int32_t* len;        // [B]: cached tokens, or own tokens
  const int32_t* group_len;  // [groups]
  const int32_t* table;      // [B][max_chunks] or null (identity)
  const int32_t* group_table;   // [groups][group_chunks]
  int max_chunks, group_chunks;
  int max_q, window, sinks;
  int64_t n_slots;
  unsigned long long wait_ns;   // limit of every wait
  int withheld;              // CTA whose planners write no segment (lsa_debug_withhold_share), or -1
};
// What a launch can meet: a window call whose sequences have one query each
// (narrow tiles only, folded in the kernel), any window call, a prefix call.  Each
// has only its own code: the softmax loop has no registers to spare.
enum Mode { kWindowToken, kWindow, kPrefixes };

// Partials.  A share can hold the end, or a middle, of a tile that began in an
// earlier one, and the start of a tile that goes on in the next: share c has a
// slot for each, 2c and 2c + 1, of as many rows as its kind of tile has.  In
// prefix mode the rows of a whole tile have places of their own, 64 per sequence
// for its prefix and 64 for its own tokens, since a sequence's output joins both.
// Place says how a query's rows lie there.
struct Work {
  float* o;          // 128 values a row, normalised: the places, the wide slots, the narrow slots
  float* lse;        // [rows], base 2
  int64_t slots[2];  // first row of the narrow slots, of the wide ones
  int rows[2];       // rows of a narrow slot, of a wide one
  int block_rows[2]; // rows of one of its blocks
  int* count;        // kWindowToken: [2 kMaxCtas], by a tile's first share: units that its partials
                     // hold so far, zero between calls
  int4* parts;       // kWindow: by slot (wide, then narrow), its tile: first query, KV head,
                     // first and last share, queries (0: no partial)
  int* ends;         // prefix mode: [4][8 B], by (sequence, KV head): first and last partial of the
                     // prefix, of the own tokens
  int* ok;           // [kMaxCtas], not kWindowToken: the CTA's partials are whole (valid offsets, no wait ran out)
};
// The first partial of a (sequence, KV head): its share, whether of the wide
// list, the query's block and number there, or that the rows are in their own
// place; kNone: no partial.
constexpr int kEndShare = 0x3ff, kEndWide = 1 << 11, kEndPlace = 16, kEndWhole = 1 << 24, kNone = -1;

// The queries and the keys of one list entry: a sequence, or a group over its prefix.
struct List {
  int q0, nq, len;
  const int32_t* table;
  int64_t ident;             // identity layout: slot of chunk 0 (table null)
};

__device__ __forceinline__ int chunks_of(int len) { return len > 0 ? (len + kChunkTokens - 1) / kChunkTokens : 0; }
// A length out of range counts as none (-1; the scan reports it).
__device__ __forceinline__ int checked_len(int len, int chunks) {
  return len < 0 || len > chunks * kChunkTokens ? -1 : len;
}

template <bool kPrefix>
__device__ __forceinline__ List load_list(const Plan& p, int v) {
  List s;
  int cap;
  if (kPrefix && v >= p.groups) {
    const int b = v - p.groups;
    s.q0 = b;
    s.nq = 1;
    s.len = ld_dep(p.len + b);
    cap = p.max_chunks;
    s.ident = static_cast<int64_t>(b) * p.max_chunks;
    s.table = p.table ? p.table + s.ident : nullptr;
  } else {
    s.q0 = ld_dep(p.cu + v);
    s.nq = ld_dep(p.cu + v + 1) - s.q0;
    s.len = ld_dep((kPrefix ? p.group_len : p.len) + v);
    cap = kPrefix ? p.group_chunks : p.max_chunks;
    s.ident = static_cast<int64_t>(v) * cap;
    const int32_t* t = kPrefix ? p.group_table : p.table;
    s.table = t ? t + s.ident : nullptr;
  }
  s.len = checked_len(s.len, cap);
  return s;
}

// Tiles are 32 queries long; the last one of an entry is narrow when it has at
// most 8.
__device__ __forceinline__ int tiles_of(const List& s, bool wide) {
  const int rest = s.nq % kWideQ;
  return wide ? s.nq / kWideQ + (rest > kNarrowQ) : (rest > 0 && rest <= kNarrowQ);
}

// sum over y < x of floor(y / 2)
__device__ __forceinline__ int64_t half_sum(int64_t x) { return x > 0 ? (x - 1) * (x - 1) / 4 : 0; }
// sum over i < t of min(cap, max(0, floor((a + 32 i) / 64)))
__device__ __forceinline__ int64_t chunk_sum(int a, int t, int64_t cap) {
  const int64_t c = a >> 5;
  const int64_t x0 = c > 0 ? c : 0;
  const int64_t x1 = c + t > x0 ? c + t : x0;
  const int64_t full = 2 * cap;   // from here on the term is cap
  const int64_t b0 = x0 < full ? x0 : full, b1 = x1 < full ? x1 : full;
  return half_sum(b1) - half_sum(b0) + cap * ((x1 - b1) - (x0 - b0));
}

// Window mode, a tile of `cnt` queries from position p0 on: the first chunk of
// its window and the sink chunks before it; returns the chunks that it sees.
__device__ __forceinline__ int tile_chunks(const Plan& p, int p0, int cnt, int& low, int& first) {
  const int p1 = p0 + cnt - 1;
  low = max(0, p0 - p.window + 1) >> 6;
  first = min(low, (p.sinks + kChunkTokens - 1) / kChunkTokens);
  return p1 < 0 ? 0 : (p1 >> 6) - low + 1 + first;
}

// Units, with kTileCost for each tile, of the first t wide tiles of an entry, or
// of its narrow tile (t = 1), for one KV head.  A tile without a key in sight
// still has one (empty) unit, so that its rows are written.
template <bool kPrefix>
__device__ __forceinline__ int64_t span(const Plan& p, const List& s, bool wide, int t) {
  if (t <= 0) return 0;
  if (kPrefix) return static_cast<int64_t>(t) * (max(1, chunks_of(s.len)) + kTileCost);
  const int pos0 = max(s.len, 0) - s.nq;
  if (!wide) {
    int low, first;
    const int rest = s.nq % kWideQ;
    return max(1, tile_chunks(p, pos0 + s.nq - rest, rest, low, first)) + kTileCost;
  }
  const int64_t none = int64_t{1} << 40;
  const int a_low = pos0 - p.window + 1;
  int64_t n = chunk_sum(pos0 + kWideQ - 1, t, none) - chunk_sum(a_low, t, none) +
              chunk_sum(a_low, t, (p.sinks + kChunkTokens - 1) / kChunkTokens) + static_cast<int64_t>(t) * (1 + kTileCost);
  if (t * kWideQ > s.nq) {   // the last tile ends before its 32nd query
    const int full = (pos0 + t * kWideQ - 1) >> 6, real = (pos0 + s.nq - 1) >> 6;
    n += (real > 0 ? real : 0) - (full > 0 ? full : 0);
  }
  return n;
}
template <bool kPrefix>
__device__ __forceinline__ int64_t span(const Plan& p, const List& s, bool wide) {
  return s.nq > 0 ? kNumKVHeads * span<kPrefix>(p, s, wide, tiles_of(s, wide)) : 0;
}

// A 64-bit quotient, in 32 bits where the operands allow it (five times faster).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}
// A list cut into equal shares: at most `most`, none smaller than kMinShare
// (unless it is the only one).
struct Partition {
  int64_t base, rem;
  int parts;
  __device__ Partition(int64_t total, int most) {
    const int64_t worth = quotient(total, kMinShare);
    parts = static_cast<int>(worth < 1 || most < 1 ? 1 : worth < most ? worth : most);
    base = quotient(total, parts);
    rem = total - base * parts;
  }
  __device__ int64_t start(int c) const {
    c = min(c, parts);
    return c * base + (c < rem ? c : rem);
  }
  __device__ int share_of(int64_t u) const {
    const int64_t big = rem * (base + 1);
    return static_cast<int>(u < big ? quotient(u, base + 1) : rem + quotient(u - big, base));
  }
};

// A walk over the tiles of one list, within a share [.., end).
template <bool kPrefix>
struct Cursor {
  int v, g, t, j;            // entry, KV head, tile, unit of the tile
  List s;
  int tiles;
  int cnt, n;                // queries of the tile, its units
  int p0;                    // window mode: position of its first query
  int low, first;            // window mode: first chunk of the window, sink chunks before it
  bool empty;                // no key in sight: the one unit is empty
  int64_t at, end;           // the tile's place in the list, the share's end

  __device__ void set_tile(const Plan& p, bool wide) {
    const int i = wide ? t * kWideQ : s.nq - s.nq % kWideQ;
    cnt = min(kWideQ, s.nq - i);
    p0 = low = first = 0;
    if (kPrefix) {
      n = chunks_of(s.len);
    } else {
      p0 = max(s.len, 0) - s.nq + i;
      n = tile_chunks(p, p0, cnt, low, first);
    }
    empty = n == 0;
    n = max(n, 1);
  }
  __device__ int row(bool wide) const { return s.q0 + (wide ? t * kWideQ : s.nq - s.nq % kWideQ); }
  // At place r of entry `entry`, whose KV heads have per_head places each; the
  // place in the list is u.  (The whole warp.)
  __device__ void start(const Plan& p, bool wide, int entry, const List& l, int64_t per_head, int64_t r, int64_t u, int lane) {
    v = entry;
    s = l;
    tiles = tiles_of(s, wide);
    g = static_cast<int>(quotient(r, per_head));
    r -= g * per_head;
    // The last tile that starts at or before r, 32 ways at a time.
    int lo = 0, n = tiles;
    int64_t before = 0;
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int64_t x = lane * step < n ? span<kPrefix>(p, s, wide, lo + lane * step) : r + 1;
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, x <= r));   // lane 0's is
      before = __shfl_sync(0xffffffffu, x, k);
      n = min(step, n - k * step);
      lo += k * step;
    }
    t = lo;
    r -= before;
    at = u - r;
    j = max(0, static_cast<int>(r) - kTileCost);
    set_tile(p, wide);
  }
  // To the first unit of the next tile, if the share has any of it.
  __device__ bool next(const Plan& p, bool wide) {
    at += n + kTileCost;
    if (at >= end) return false;
    j = 0;
    if (++t == tiles) {
      t = 0;
      if (++g == kNumKVHeads) {
        g = 0;
        do {
          ++v;
          s = load_list<kPrefix>(p, v);
          tiles = tiles_of(s, wide);
        } while (tiles == 0);
      }
    }
    set_tile(p, wide);
    return units() > 0;
  }
  // Units from j on that the share has.
  __device__ int units() const {
    const int64_t x = end - at - kTileCost;
    return static_cast<int>(x < n ? x : n) - j;
  }
};

// 64 bits: the lowest x.
__device__ __forceinline__ uint64_t lowest(int x) {
  return x <= 0 ? 0ull : x >= 64 ? ~0ull : (1ull << x) - 1;
}
// Window mode: tokens of the chunk that begins at token kb which some query of a
// tile sees.
__device__ __forceinline__ uint64_t tile_sees(const Plan& p, int kb, int p0, int cnt) {
  return lowest(p0 + cnt - kb) & (~lowest(p0 - p.window + 1 - kb) | lowest(p.sinks - kb));
}

// Barriers and copies by shared address: a generic pointer takes two registers
// and a conversion at every use.
__device__ __forceinline__ void bar_init(uint32_t bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Whether the phase has completed, at once: try_wait may sleep for a while first,
// which a caller that has something else to do must not.
__device__ __forceinline__ bool bar_test(uint32_t bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits, at most limit_ns, or until another role has given up; the same
// answer in every lane, so that the warp's collective instructions stay whole.
// `abort_flag`: 0, or 1 once a wait of the CTA ran out.
__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, unsigned parity, uint32_t abort_flag,
                                              unsigned long long limit_ns, unsigned* status) {
  const unsigned long long t0 = globaltimer_ns();
  for (unsigned it = 1;; ++it) {
    if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
    if ((it & 63u) == 0) {
      int given_up;
      asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(given_up) : "r"(abort_flag) : "memory");
      const bool late = globaltimer_ns() - t0 > limit_ns;
      if (__any_sync(0xffffffffu, given_up || late)) {
        if (!given_up) set_status(status, LSA_DEV_ERR_TIMEOUT);
        asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(abort_flag), "r"(1) : "memory");
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, unsigned parity, uint32_t abort_flag, unsigned long long limit_ns,
                                         unsigned* status) {
  if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
  return bar_wait_slow(bar, parity, abort_flag, limit_ns, status);
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// A query's 8 rows of 64 dims to the output, by the async proxy: issued by a lane,
// whose group it is.
__device__ __forceinline__ void store_box(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n\tcp.async.bulk.commit_group;" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(src)
      : "memory");
}
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// One lane of the warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Shared-memory descriptors as a constant upper word and a lower word that holds
// the address in 16-byte steps (and the leading offset), so that a tile's k-steps
// are additions.  Both operands use the 128-byte swizzle, with 8-row groups 1024
// bytes apart (stride offset).  K-major (Q, K): the leading offset is unused.
// V is the N x K operand (N = dims, K = tokens) stored token by token, N
// contiguous: its 64-dim boxes are 8192 bytes apart (leading offset).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo_kmajor(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_lo_v(uint32_t saddr) {
  return ((saddr >> 4) & 0x3FFFu) | (static_cast<uint32_t>(kBoxBytes >> 4) << 16);
}
// The warp runs these together and the lane with `leader` set issues: a branch
// around them would keep the operands out of the uniform registers that they
// are read from.
// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 e, %6, 0;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 e, %6, 0;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}
constexpr uint32_t kIdescS = umma_idesc_bf16_f32(128, kChunkTokens);
constexpr uint32_t kIdescO = umma_idesc_bf16_f32(128, kHeadDim) | (1u << 16);   // B with N contiguous

// 32 consecutive columns of this thread's TMEM lane; the caller waits.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// The waits tie the loaded registers to the instruction, so that no use of them
// is scheduled before it.
__device__ __forceinline__ void tmem_wait_ld(float* v, int n) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < n; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations in one instruction, and the maximum of three.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
// (NaN if any is: a query or a key that is not a number reaches the maximum, and
// with it every probability of the row.)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float v;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(v) : "f"(a), "f"(b), "f"(c));
  return v;
}
// 2^x of two values at most kRaise, by the FMA pipe: floor by an addition that
// rounds down, a polynomial of degree 4 for 2^f on [0, 1) with value 1 at 0
// (minimax for the relative error: 2.9e-6, against up to 2^-8 of the rounding to
// bf16 that follows), and the integer part added to the exponent.  From -127 down
// (masked scores among them) exactly 0.
__device__ __forceinline__ void exp2_fma(uint64_t x, float& a, float& b) {
  float lo, hi;
  unpack2(x, lo, hi);
  x = pack2(fmaxf(lo, -127.f), fmaxf(hi, -127.f));
  constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: an integer sits in the low bits of a sum with it
  uint64_t t;
  asm("add.rm.f32x2 %0, %1, %2;" : "=l"(t) : "l"(x), "l"(pack2(kMagic, kMagic)));
  const uint64_t n = add2(t, pack2(-kMagic, -kMagic));
  const uint64_t f = fma2(n, pack2(-1.f, -1.f), x);
  uint64_t p = fma2(f, pack2(0.013426689f, 0.013426689f), pack2(0.052242465f, 0.052242465f));
  p = fma2(p, f, pack2(0.24128021f, 0.24128021f));
  p = fma2(p, f, pack2(0.69304484f, 0.69304484f));
  p = fma2(p, f, pack2(1.f, 1.f));
  float p0, p1, t0, t1;
  unpack2(p, p0, p1);
  unpack2(t, t0, t1);
  a = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(t0) << 23));
  b = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(t1) << 23));
}

// Registers per thread from here on, for a warpgroup whose warps all say so: the
// block's 384 x 168 go 208 + 208 to the softmax warpgroups and 88 to the others.
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "the shares come out of the block's own registers");

// Exclusive prefix sums of x[0 .. kSums - 1] over the block (kWarps warps), and the totals.
template <int kWarps, int kSums>
__device__ __forceinline__ void block_scan(const int64_t* x, int64_t* before, int64_t* total, int64_t* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc[kSums];
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    inc[k] = x[k];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc[k], off);
      if (lane >= off) inc[k] += y;
    }
    if (lane == 31) sm[k * kWarps + warp] = inc[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    int64_t sum = 0;
    before[k] = inc[k] - x[k];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int64_t y = sm[k * kWarps + w];
      if (w < warp) before[k] += y;
      sum += y;
    }
    total[k] = sum;
  }
}

// ---- folding the partials -----------------------------------------------------
__device__ __forceinline__ uint4 ld_l2(const float4* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ float ld_l2(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
// Where the 8 rows (query heads of a KV head) of a query lie in a partial: dims 4 c
// .. 4 c + 3 of row h at work.o + o + c * stride + 4 h, the log-sum-exp at work.lse
// + lse + h.  A slot holds a block of up to 4 queries for each warp that writes
// it, so that a warp, a thread per row, stores 16 bytes a thread side by side.
struct Place {
  int64_t o, lse;
  int stride;
};
__device__ __forceinline__ Place slot_place(const Work& w, int wide, int slot, int block, int query) {
  // (Not by index: the structure would move to local memory.)
  const int rows = wide ? w.block_rows[1] : w.block_rows[0];
  const int64_t slot_rows = wide ? w.rows[1] : w.rows[0];
  const int64_t first = (wide ? w.slots[1] : w.slots[0]) + slot * slot_rows + block * rows;
  return {first * kHeadDim + query * (kGroup * 4), first + query * kGroup, rows * 4};
}
// Prefix mode, a whole tile's: of a sequence's prefix, or of its own tokens.
__device__ __forceinline__ Place own_place(const Work& w, int B, int b, int g, bool own) {
  const int64_t first = (static_cast<int64_t>(own ? B : 0) + b) * kNumQHeads + g * kGroup;
  return {first * kHeadDim, first, kGroup * 4};
}

// The 8 rows of a query: joins its n partials at place(0) .. place(n - 1), in
// that order, and writes part `part` of kParts of the output's dims.  A warp;
// lane i has row i % 8 and the dims 4 c .. 4 c + 3 with c % 4 = i / 8.  The loads
// of kBatch partials are in flight together.
template <int kParts, int kBatch, typename At>
__device__ __forceinline__ void fold_query(const Work& w, int n, int lane, At place, __nv_bfloat16* out, int part = 0) {
  constexpr int kPieces = kHeadDim / 16 / kParts;
  const int h = lane & 7, c0 = (lane >> 3) + 4 * kPieces * part;
  float m = -INFINITY, den = 0.f;
  float4 acc[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i = 0; i < n; i += kBatch) {
    float lse[kBatch];
    uint4 a[kBatch][kPieces];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      lse[x] = -INFINITY;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) a[x][k] = make_uint4(0, 0, 0, 0);
      if (i + x < n) {
        const Place p = place(i + x);
        lse[x] = ld_l2(w.lse + p.lse + h);
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
          a[x][k] = ld_l2(reinterpret_cast<const float4*>(w.o + p.o + h * 4 + (c0 + 4 * k) * p.stride));
      }
    }
    float top = m;
#pragma unroll
    for (int x = 0; x < kBatch; ++x) top = max3(top, lse[x], lse[x]);   // (a row that is not a number stays so)
    const float ref = top == -INFINITY ? 0.f : top;
    const float f = fast_exp2(m - ref);
    m = top;
    den *= f;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      acc[k].x *= f; acc[k].y *= f; acc[k].z *= f; acc[k].w *= f;
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const float wt = fast_exp2(lse[x] - ref);
      den += wt;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        acc[k].x = fmaf(wt, __uint_as_float(a[x][k].x), acc[k].x);
        acc[k].y = fmaf(wt, __uint_as_float(a[x][k].y), acc[k].y);
        acc[k].z = fmaf(wt, __uint_as_float(a[x][k].z), acc[k].z);
        acc[k].w = fmaf(wt, __uint_as_float(a[x][k].w), acc[k].w);
      }
    }
  }
  const float id = m == -INFINITY ? 0.f : m == kLowest ? CUDART_NAN_F : 1.f / den;
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
    *reinterpret_cast<uint2*>(out + h * kHeadDim + 4 * (c0 + 4 * k)) =
        make_uint2(pack_bf16(acc[k].x * id, acc[k].y * id), pack_bf16(acc[k].z * id, acc[k].w * id));
}

// A segment: the units of one tile that a share has.  The planners write them to
// shared memory a few ahead, so that no other role walks the list or waits for
// its loads.
struct Seg {
  int units;                 // 0: the share has ended
  int flags;                 // kSegEmpty ...
  int j0;                    // its first unit in the tile
  int cnt, row, head;        // the tile's queries, the first one's row of q, the first query head
  int first, low;            // chunk of unit j: j < first ? j : low + j - first
  int f0, f1, f2;            // units that every query sees whole: j < f0 and f1 <= j <= f2
  int p0, len;               // window mode: position of the first query; prefix mode: tokens
  int slot;                  // of its partial
  int lo, hi;                // window mode: first and last share of the tile
  int all;                   // units of the tile
  int g;
  const int32_t* table;
  int64_t ident;
};
constexpr int kSegEmpty = 1, kSegAgain = 2, kSegGroup = 4, kSegWhole = 8, kSegAlone = 16;

// Shared memory, from a 1024-byte boundary.
constexpr int kQAt = kHalves * kHalfBytes, kTurnAt = kQAt + 2 * kQTileBytes;
constexpr int kSegAt = kTurnAt + 8 * kTurnBytes;   // [3][kAhead]: the wide share's, each pipeline's narrow share's
// Barriers, 8 bytes each.
constexpr int kBarAt = kSegAt + 3 * kAhead * static_cast<int>(sizeof(Seg));
constexpr int kFull = kBarAt, kEmpty = kFull + 8 * kHalves;            // half-stages
constexpr int kSFull = kEmpty + 8 * kHalves;                           // [2 pipelines][2 buffers] scores are there
constexpr int kPFull = kSFull + 32, kODone = kPFull + 32;              // probabilities are; the product that read them is done
constexpr int kQFull = kODone + 32, kQEmpty = kQFull + 16;             // [2] query tiles of the wide share
constexpr int kNFull = kQEmpty + 16, kNEmpty = kNFull + 32;            // [2 pipelines][2] of the narrow ones
constexpr int kSegFull = kNEmpty + 32, kSegDone = kSegFull + 24 * kAhead;   // [3][kAhead]
constexpr int kDrain = kSegDone + 24 * kAhead, kMeet = kDrain + 16;            // [2], [2]: a warpgroup's warps
constexpr int kTmemAt = kMeet + 16, kAbortAt = kTmemAt + 4, kVerdictAt = kAbortAt + 4;   // (two verdicts)
// The entry at the start of the wide share, or of the two narrow ones.
struct Found {
  List s;
  int64_t r, per_head;       // the place in the entry, the entry's places per KV head
  int v;
};
constexpr int kFoundAt = kVerdictAt + 8;
constexpr int kSmemBytes = kFoundAt + 2 * static_cast<int>(sizeof(Found));
static_assert(kSmemBytes <= 232448 && sizeof(Seg) % 8 == 0 && kFoundAt % 8 == 0, "shared memory of one CTA");

// The place in the ring of the x-th half (K of unit i: 2 i, V: 2 i + 1) of a
// share, and the parity of its use.  A wide share goes around all 8, the narrow
// one of pipeline w around 4w .. 4w + 3.
struct Ring {
  unsigned first, mask, shift;
  __device__ unsigned half(unsigned x) const { return first + (x & mask); }
  __device__ unsigned parity(unsigned x) const { return (x >> shift) & 1; }
};
__device__ __forceinline__ Ring ring_of(bool wide, int w) { return wide ? Ring{0, 7, 3} : Ring{4u * w, 3, 2}; }

template <Mode kMode>
__global__ void __launch_bounds__(kThreads, 1)
pool_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CUtensorMap tm_k_part, const __grid_constant__ CUtensorMap tm_v_part,
                 const __grid_constant__ CUtensorMap tm_q16, const __grid_constant__ CUtensorMap tm_q8,
                 const __grid_constant__ CUtensorMap tm_q1, const __grid_constant__ CUtensorMap tm_out, const Plan plan,
                 const Work work, float scale_log2, __nv_bfloat16* __restrict__ out, unsigned* status) {
  constexpr bool kPrefix = kMode == kPrefixes, kFold = kMode == kWindowToken, kHasWide = !kFold;
  constexpr bool kParts = !kPrefix;   // chunks that are not seen whole are loaded by parts
  extern __shared__ __align__(1024) uint8_t smem[];
  // (The warp's index by a shuffle: the compiler has to know that it is the same in
  // every lane, or the products' operands are moved to uniform registers one by one.)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t sm = smem_u32(smem);
  const uint32_t abort_flag = sm + kAbortAt;

  // ---- before the previous kernel has ended: barriers and TMEM ---------------
  if (tid == 0) {
    for (int i = 0; i < kHalves; ++i) {
      bar_init(sm + kFull + 8 * i, 1);
      bar_init(sm + kEmpty + 8 * i, 2);   // both product warps (or one of them twice)
    }
    for (int i = 0; i < 4; ++i) {
      bar_init(sm + kSFull + 8 * i, 1);
      bar_init(sm + kPFull + 8 * i, 4);   // the warps of the warpgroup
      bar_init(sm + kODone + 8 * i, 1);
      bar_init(sm + kNFull + 8 * i, 1);
      bar_init(sm + kNEmpty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(sm + kQFull + 8 * i, 1);
      bar_init(sm + kQEmpty + 8 * i, 1);
      bar_init(sm + kDrain + 8 * i, 1);
      bar_init(sm + kMeet + 8 * i, 4);
    }
    for (int i = 0; i < 3 * kAhead; ++i) {
      bar_init(sm + kSegFull + 8 * i, 1);
      bar_init(sm + kSegDone + 8 * i, i < kAhead ? 11 : 5);   // softmax, product and (wide) load warps
    }
    *reinterpret_cast<volatile int*>(smem + kAbortAt) = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(reinterpret_cast<uint32_t*>(smem + kTmemAt), 512);
  if (tid == kLoadWarp * 32) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    if (kParts) {
      tma_prefetch_desc(&tm_k_part);
      tma_prefetch_desc(&tm_v_part);
    }
    if (kHasWide) {
      tma_prefetch_desc(&tm_q16);
      tma_prefetch_desc(&tm_q8);
    }
    tma_prefetch_desc(&tm_q1);
    tma_prefetch_desc(&tm_out);
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the lists: validity, totals, and the places where the shares start ----
  // (The scan's scratch lies where rows turn later.)
  int64_t* const scan = reinterpret_cast<int64_t*>(smem + kTurnAt);
  Found* const found = reinterpret_cast<Found*>(smem + kFoundAt);
  const int V = plan.B + (kPrefix ? plan.groups : 0);
  const int per = (V + kThreads - 1) / kThreads;
  const int v_lo = min(V, tid * per), v_hi = min(V, v_lo + per);
  int bad = 0;
  int64_t mine[2] = {0, 0};   // [narrow, wide]
  const int n_cu = kPrefix ? plan.groups : plan.B;
  if (tid == kThreads - 1 && n_cu > 0) {
    const int last = ld_dep(plan.cu + n_cu);
    bad |= ld_dep(plan.cu) != 0 || last < 0 || last > plan.rows;
  }
  List s_last = {};   // the thread's last entry: its only one for up to kThreads entries
  for (int v = v_lo; v < v_hi; ++v) {
    s_last = load_list<kPrefix>(plan, v);
    if (s_last.len < 0 && blockIdx.x == 0) set_status(status, LSA_DEV_ERR_BAD_COUNT);
    // (Each entry's rows by themselves: offsets may wrap around and still end in range.)
    bad |= s_last.nq < 0 || s_last.nq > plan.max_q || s_last.q0 < 0 || s_last.q0 > plan.rows - s_last.nq;
    mine[0] += span<kPrefix>(plan, s_last, false);
    if (kHasWide) mine[1] += span<kPrefix>(plan, s_last, true);
  }
  bad = __syncthreads_or(bad);
  if (bad) mine[0] = mine[1] = 0;
  int64_t total[2] = {0, 0};
  int64_t before[2] = {0, 0};
  block_scan<kThreads / 32, kHasWide ? 2 : 1>(mine, before, total, scan);
  // CTAs of the wide list, the others are the narrow one's: by what the lists cost,
  // or as many as the shorter one is worth.
  const int grid = gridDim.x;
  int grid_w = kHasWide && total[1] ? grid : 0;
  if (grid_w && total[0]) {
    const float cost = kWideCost * static_cast<float>(total[1]);
    grid_w = min(max(static_cast<int>(grid * (cost / (cost + static_cast<float>(total[0]))) + 0.5f), 1), grid - 1);
    const int64_t worth_w = quotient(total[1], kMinShare), worth_n = (quotient(total[0], kMinShare) + 1) / 2;
    if (worth_w < grid_w) grid_w = max(static_cast<int>(worth_w), 1);
    else if (worth_n < grid - grid_w) grid_w = grid - max(static_cast<int>(worth_n), 1);
  }
  const Partition part_n(total[0], 2 * (grid - grid_w)), part_w(total[1], grid_w);
  if (part_n.base >= (1 << 30) || part_w.base >= (1 << 30)) bad = 1;   // a share counts its units in 32 bits
  if (bad && blockIdx.x == 0 && tid == 0) set_status(status, LSA_DEV_ERR_CAPACITY);
  if (sm & 1023u) {                      // the 128-byte swizzle repeats every 1024 bytes
    if (tid == 0) set_status(status, LSA_DEV_ERR_INTERNAL);
    bad = 1;
  }
  const int me = blockIdx.x;
  // Prefix mode: sequences from `grouped` on belong to no group.
  const int grouped = plan.groups ? ld_dep(plan.cu + plan.groups) : 0;
  if (!kFold && tid == 0) work.ok[me] = bad ? 0 : 1;
#pragma unroll
  for (int x = 0; x < 2; ++x) {   // the entry at the start of the wide share, or the entries of the two narrow ones
    const bool k = me < grid_w;
    const int64_t u = k ? part_w.start(me) : part_n.start(2 * (me - grid_w) + x);
    int64_t at = k ? before[1] : before[0], n = k ? mine[1] : mine[0];
    if (!bad && !(k && x) && at <= u && u < at + n) {   // one thread, if u is in the list
      int v = v_lo;
      List s = s_last;
      if (per > 1) {
        for (;; ++v) {
          s = load_list<kPrefix>(plan, v);
          n = span<kPrefix>(plan, s, k);
          if (u < at + n) break;
          at += n;
        }
      }
      found[x] = {s, u - at, n / kNumKVHeads, v};
    }
  }
  const bool wide = kHasWide && me < grid_w;   // what the CTA does
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *reinterpret_cast<const volatile uint32_t*>(smem + kTmemAt);
  const Seg* const segs = reinterpret_cast<const Seg*>(smem + kSegAt);
  auto wait = [&](int bar, unsigned parity) { return bar_wait(sm + bar, parity, abort_flag, plan.wait_ns, status); };
  // Two at once: a barrier that is ready still costs its round trip.
  auto wait2 = [&](int a, unsigned parity_a, int b, unsigned parity_b) {
    const bool ready_a = bar_try(sm + a, parity_a), ready_b = bar_try(sm + b, parity_b);
    return __all_sync(0xffffffffu, ready_a && ready_b) || (wait(a, parity_a) && wait(b, parity_b));
  };
  // Segment k of share x (0: wide, 1 + w: narrow); its place is free again once
  // every role has said so.
  auto seg_get = [&](int x, unsigned k) { return wait(kSegFull + 8 * (x * kAhead + k % kAhead), (k / kAhead) & 1); };
  auto seg_done = [&](int x, unsigned k) {
    __syncwarp();
    if (lane == 0) bar_arrive(sm + kSegDone + 8 * (x * kAhead + k % kAhead));
  };

  if (warp >= kMmaWarp) {
    fewer_registers<kOtherRegs>();
    const int w = warp & 1;
    if (warp >= kLoadWarp) {
      // ============================ plan and load ============================
      Cursor<kPrefix> cur = {};
      unsigned put = 0;      // segments of the share written
      bool more = false;     // the cursor stands on one
      bool ended = false;    // the share's end is written
      auto begin = [&](int x, const Partition& part, int64_t all, int share) {
        const int64_t u = part.start(share);
        cur.end = part.start(share + 1);
        put = 0;
        ended = false;
        more = !bad && u < cur.end && u < all;
        if (more) {
          const Found& f = found[x == 0 ? 0 : x - 1];
          cur.start(plan, x == 0, f.v, f.s, f.per_head, f.r, u, lane);
          more = cur.units() > 0;
        }
      };
      // Writes the next segment of share x, or its end; `advance` follows.
      auto publish = [&](int x, const Partition& part, int share) {
        const int place = x * kAhead + put % kAhead;
        if (put >= kAhead && !wait(kSegDone + 8 * place, (put / kAhead - 1) & 1)) return false;
        Seg* const s = reinterpret_cast<Seg*>(smem + kSegAt) + place;
        if (!more) {
          if (lane == 0) s->units = 0;
          ended = true;
        } else {
          const bool own = kPrefix && cur.v >= plan.groups;
          const int units = cur.units();
          const bool begins = cur.j == 0, ends = cur.j + units == cur.n;
          const int flags = (cur.empty ? kSegEmpty : 0) | (cur.tiles > 1 ? kSegAgain : 0) |
                            (kPrefix && !own ? kSegGroup : 0) | (begins && ends ? kSegWhole : 0) |
                            (own && cur.v - plan.groups >= grouped ? kSegAlone : 0);
          if (lane == 0) {
            s->units = units;
            s->flags = flags;
            s->j0 = cur.j;
            s->cnt = cur.cnt;
            s->row = cur.row(wide);
            s->head = cur.g * kGroup;
            s->first = cur.first;
            s->low = cur.low;
            int f0 = 0, f1 = 0, f2 = -1;
            if (kPrefix) {
              f0 = cur.s.len / kChunkTokens;
            } else if (!cur.empty) {
              f0 = min(cur.first, plan.sinks / kChunkTokens);
              f1 = cur.first + (max(0, cur.p0 + cur.cnt - plan.window + kChunkTokens - 1) >> 6) - cur.low;
              f2 = cur.first + ((cur.p0 - (kChunkTokens - 1)) >> 6) - cur.low;
            }
            s->f0 = f0;
            s->f1 = f1;
            s->f2 = f2;
            s->p0 = cur.p0;
            s->len = cur.s.len;
            s->slot = 2 * share + (begins ? 1 : 0);
            s->all = cur.n;
            s->g = cur.g;
            s->table = cur.s.table;
            s->ident = cur.s.ident;
          }
          if (kFold && !(begins && ends)) {
            const int lo = begins ? share : part.share_of(cur.at + kTileCost);
            const int hi = ends ? share : part.share_of(cur.at + kTileCost + cur.n - 1);
            if (lane == 0) {
              s->lo = lo;
              s->hi = hi;
            }
          }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(sm + kSegFull + 8 * place);
        ++put;
        return true;
      };
      auto advance = [&](int x, const Partition& part, int share) {
        if (more) {
          if (kMode == kWindow) {   // what the merge has to know
            const bool begins = cur.j == 0, ends = cur.j + cur.units() == cur.n;
            if (!(begins && ends)) {
              const int lo = begins ? share : part.share_of(cur.at + kTileCost);
              const int hi = ends ? share : part.share_of(cur.at + kTileCost + cur.n - 1);
              if (lane == 0)
                work.parts[(wide ? 0 : 2 * kMaxCtas) + 2 * share + (begins ? 1 : 0)] =
                    make_int4(cur.row(wide), cur.g, lo | (hi << 16), cur.cnt);
            }
          }
          more = cur.next(plan, wide);
        }
      };
      const uint64_t policy_once = l2_policy_evict_first(), policy_again = l2_policy_evict_normal();
      const int beyond = static_cast<int>(plan.n_slots) * (kNumKVHeads * kChunkTokens);   // reads as zeros
      // The narrow shares are 2 turned and the next; every CTA has an index of that
      // kind too, so that each place of work.parts is written by one lane.
      const int turned = me - grid_w + (me < grid_w ? grid : 0);
      if (kMode == kWindow && lane == 0) {
        int4* const narrow = work.parts + 2 * kMaxCtas + 2 * (2 * turned + w);
        narrow[0] = narrow[1] = make_int4(0, 0, 0, 0);
        if (w) work.parts[2 * me] = work.parts[2 * me + 1] = make_int4(0, 0, 0, 0);
      }
      const Ring ring = ring_of(wide, w);
      unsigned halves = 0;   // loads so far
      // K and V of a segment's units, the next ones of the share.  In window mode only
      // the parts (16 tokens) of a chunk with a token in sight are loaded; what the
      // other rows hold is masked (K) and zeroed (V).  64 single tokens over windows of
      // 1024 take 4% less time so than with whole chunks (275 MB read, 300), a prompt of
      // 4096 2%.  A prefix call has only ends of sequences to save on, and takes longer by
      // more but smaller loads (128 sequences, 5 groups: 3%).
      auto load_units = [&](int units, int flags, int j0, int first, int low, int g, const int32_t* table, int64_t ident,
                            int p0, int cnt) {
        // Another tile of the entry reads the same chunks: they stay in L2.
        const uint64_t policy = (flags & kSegAgain) ? policy_again : policy_once;
        int row = 0;
        for (int i = 0; i < units; ++i) {
          if ((i & 31) == 0) {   // 32 units at a time, a lane each: the pool row (a multiple of 64) and 4 bits, the parts
            row = beyond;
            if (!(flags & kSegEmpty) && i + lane < units) {
              const int j = j0 + i + lane, c = j < first ? j : low + j - first;
              const int64_t slot = table ? ld_dep(table + c) : ident + c;
              if (slot >= 0 && slot < plan.n_slots)
                row = (static_cast<int>(slot) * kNumKVHeads + g) * kChunkTokens;
              else
                set_status(status, LSA_DEV_ERR_BAD_SLOT);
              const uint64_t seen = tile_sees(plan, c * kChunkTokens, p0, cnt);
              const uint32_t lo = static_cast<uint32_t>(seen), hi = static_cast<uint32_t>(seen >> 32);
              if (kParts) row |= ((lo & 0xffff) != 0) | (lo >> 16 != 0) << 1 | ((hi & 0xffff) != 0) << 2 | (hi >> 16 != 0) << 3;
            }
          }
          const int of_unit = __shfl_sync(0xffffffffu, row, i & 31);
          const int y = of_unit & ~63, parts = kParts ? of_unit & 15 : 15;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const unsigned h = ring.half(halves);
            // The use before this one has been read.
            if (halves > ring.mask && !wait(kEmpty + 8 * h, ring.parity(halves) ^ 1)) return false;
            if (lane == 0) {
              const uint32_t dst = sm + h * kHalfBytes, bar = sm + kFull + 8 * h;
              if (parts == 15) {
                const CUtensorMap* const map = kv ? &tm_v : &tm_k;
                bar_expect(bar, kHalfBytes);
                load_box(dst, map, 0, y, bar, policy);
                load_box(dst + kBoxBytes, map, 64, y, bar, policy);
              } else {
                const CUtensorMap* const map = kv ? &tm_v_part : &tm_k_part;
                bar_expect(bar, __popc(parts) * 2 * kPartBytes);
                for (int b = 0; b < 4; ++b) {
                  if (!((parts >> b) & 1)) continue;
                  load_box(dst + b * kPartBytes, map, 0, y + b * kPartRows, bar, policy);
                  load_box(dst + kBoxBytes + b * kPartBytes, map, 64, y + b * kPartRows, bar, policy);
                }
              }
            }
            __syncwarp();
            // A wide share's first K comes alone: every CTA starts at once, and with
            // the whole ring asked for together the first products would wait 4 us.
            if (wide && halves == 0 && !wait(kFull + 8 * h, 0)) {
              halves = 1;
              return false;
            }
            ++halves;
          }
        }
        return true;
      };
      // The loads of a share that was given up land before the CTA ends.
      auto land = [&]() {
        volatile int never = 0;
        for (unsigned i = halves > ring.mask ? halves - ring.mask - 1 : 0; i < halves; ++i)
          mbar_wait_bounded(reinterpret_cast<uint64_t*>(smem + kFull) + ring.half(i), ring.parity(i), &never);
      };
      // A planner that withholds its share: the others wait for its segments and it
      // for the end of their products, until the limit.
      bool ok = true;
      if (plan.withheld == me) {
        wait(kDrain + 8 * w, 0);
        ok = false;
      }
      if (wide && warp == kLoadWarp) {
        for (unsigned k = 0; ok; ++k) {
          ok = seg_get(0, k);
          if (!ok) break;
          const Seg& s = segs[k % kAhead];
          const int units = s.units, flags = s.flags, j0 = s.j0, first = s.first, low = s.low, g = s.g, p0 = s.p0, cnt = s.cnt;
          const int32_t* const table = s.table;
          const int64_t ident = s.ident;
          seg_done(0, k);
          if (units == 0) break;
          ok = load_units(units, flags, j0, first, low, g, table, ident, p0, cnt);
        }
        if (!ok && lane == 0) land();
      } else if (wide) {
        begin(0, part_w, total[1], me);
        // One place stays free: in segment k the planner writes segment k + 3
        // where k - 1 was, which does not hold back the query tiles of k + 1.
        ok = ok && publish(0, part_w, me);
        unsigned k = 0;
        for (; ok; ++k) {
          const Seg& s = segs[k % kAhead];
          const int units = s.units, cnt = s.cnt, row = s.row, head = s.head;
          if (units == 0) break;
          for (int t = 0; ok && t < 2; ++t) {   // a pipeline's half of the queries each
            if (k) ok = wait(kQEmpty + 8 * t, (k - 1) & 1);
            if (ok && lane == 0) {
              const uint32_t bar = sm + kQFull + 8 * t, q = sm + kQAt + t * kQTileBytes;
              const int at = row + (t ? (cnt + 1) >> 1 : 0);
              bar_expect(bar, kQTileBytes);
              load_box(q, &tm_q16, 0, head, at, bar);
              load_box(q + kQBoxBytes, &tm_q16, 64, head, at, bar);
            }
            __syncwarp();
          }
          while (ok && !ended && put < k + kAhead) {   // (after the first segment's query tiles)
            advance(0, part_w, me);
            ok = publish(0, part_w, me);
          }
        }
        if (!ok && lane == 0 && k) {   // tiles in flight land before the CTA ends
          volatile int never = 0;
          for (int t = 0; t < 2; ++t)
            mbar_wait_bounded(reinterpret_cast<uint64_t*>(smem + kQFull) + t, (k - 1) & 1, &never);
        }
      } else {
        unsigned loads = 0;
        begin(1 + w, part_n, total[0], 2 * turned + w);
        for (unsigned k = 0; ok; ++k) {
          const int units = more ? cur.units() : 0, cnt = cur.cnt, row = cur.row(false), j0 = cur.j, first = cur.first,
                    low = cur.low, g = cur.g, flags = cur.empty ? kSegEmpty : 0, p0 = cur.p0;
          const int32_t* const table = cur.s.table;
          const int64_t ident = cur.s.ident;
          ok = publish(1 + w, part_n, 2 * turned + w);
          if (!ok || units == 0) break;
          const int b = k & 1;
          if (k >= 2) ok = wait(kNEmpty + 16 * w + 8 * b, ((k >> 1) - 1) & 1);
          if (!ok) break;
          if (lane == 0) {
            const uint32_t bar = sm + kNFull + 16 * w + 8 * b, q = sm + kQAt + w * kQTileBytes + b * kQ2Bytes;
            const bool one = kFold || cnt == 1;       // (what other rows hold is not read back)
            const CUtensorMap* const map = one ? &tm_q1 : &tm_q8;
            bar_expect(bar, 2 * 128 * kGroup * (one ? 1 : kNarrowQ));
            load_box(q, map, 0, g * kGroup, row, bar);
            load_box(q + kQBoxBytes, map, 64, g * kGroup, row, bar);
          }
          __syncwarp();
          ++loads;
          ok = load_units(units, flags, j0, first, low, g, table, ident, p0, cnt);
          advance(1 + w, part_n, 2 * turned + w);
        }
        if (!ok && lane == 0) {   // copies in flight land before the CTA ends
          volatile int never = 0;
          uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + kNFull) + 2 * w;
          for (unsigned i = loads > 2 ? loads - 2 : 0; i < loads; ++i) mbar_wait_bounded(bars + (i & 1), (i >> 1) & 1, &never);
          land();
        }
      }
    } else {
      // =============================== products ==============================
      // The whole warp walks the segments (its values stay uniform) and one lane
      // issues.
      const uint32_t leader = elect_one() ? 1u : 0u;
      const uint32_t k_lo0 = desc_lo_kmajor(sm), v_lo0 = desc_lo_v(sm), q_lo0 = desc_lo_kmajor(sm + kQAt + w * kQTileBytes);
      const uint32_t o_acc = tmem + kOCol0 + w * kHeadDim, s_col0 = tmem + 2 * w * kSCols;
      const int s_bar = kSFull + 16 * w, p_bar = kPFull + 16 * w, o_bar = kODone + 16 * w;
      const Ring ring = ring_of(wide, w);
      const int x = wide ? 0 : 1 + w;   // the share
      unsigned job = 0;                 // units so far
      bool ok = true;
      for (unsigned k = 0; ok; ++k) {
        ok = seg_get(x, k);
        if (!ok) break;
        const int n = segs[x * kAhead + k % kAhead].units;
        seg_done(x, k);
        if (n == 0) break;
        const int q_full = x == 0 ? kQFull + 8 * w : kNFull + 16 * w + 8 * (k & 1);
        const int q_empty = x == 0 ? kQEmpty + 8 * w : kNEmpty + 16 * w + 8 * (k & 1);
        const uint32_t q_lo = q_lo0 + (x == 0 ? 0 : (k & 1) * (kQ2Bytes >> 4));
        ok = wait(q_full, (x == 0 ? k : k >> 1) & 1);
        // Scores run up to two units (both buffers) before the products: in the
        // narrow share as far as units have arrived, since waiting for one that
        // has not would hold back the product that frees a half-stage.
        int next = 0;
        for (int i = 0; ok && i < n; ++i) {
          for (; next < min(n, i + 2); ++next) {
            const unsigned kx = 2 * (job + next), h = ring.half(kx), jb = job + next, buf = jb & 1;
            if (x && next > i && !__all_sync(0xffffffffu, bar_test(sm + kFull + 8 * h, ring.parity(kx)))) break;
            // K is there, and the buffer's probabilities have been read.
            ok = jb < 2 ? wait(kFull + 8 * h, ring.parity(kx))
                        : wait2(kFull + 8 * h, ring.parity(kx), o_bar + 8 * buf, ((jb - 2) >> 1) & 1);
            if (!ok) break;
            tcgen05_fence_after();
            const uint32_t k_lo = k_lo0 + h * (kHalfBytes >> 4), d = s_col0 + buf * kSCols;
#pragma unroll
            for (int y = 0; y < 8; ++y)
              mma_ss(leader, d, q_lo + (y >> 2) * (kQBoxBytes >> 4) + (y & 3) * 2,
                     k_lo + (y >> 2) * (kBoxBytes >> 4) + (y & 3) * 2, kIdescS, y > 0);
            mma_commit(leader, sm + s_bar + 8 * buf);
            mma_commit(leader, sm + kEmpty + 8 * h);
            if (x) mma_commit(leader, sm + kEmpty + 8 * h);
            if (next == n - 1) mma_commit(leader, sm + q_empty);
          }
          if (!ok) break;
          const unsigned vx = 2 * (job + i) + 1, h = ring.half(vx), jb = job + i, buf = jb & 1;
          ok = wait2(kFull + 8 * h, ring.parity(vx), p_bar + 8 * buf, (jb >> 1) & 1);
          if (!ok) break;
          tcgen05_fence_after();
          const uint32_t v_lo = v_lo0 + h * (kHalfBytes >> 4), a = s_col0 + buf * kSCols;
#pragma unroll
          for (int y = 0; y < 4; ++y)
            mma_ts(leader, o_acc, a + 8 * y, v_lo + y * (2048 >> 4), kIdescO, y > 0 || i > 0);
          mma_commit(leader, sm + o_bar + 8 * buf);
          mma_commit(leader, sm + kEmpty + 8 * h);
          if (x) mma_commit(leader, sm + kEmpty + 8 * h);
        }
        job += n;
      }
      mma_commit(leader, sm + kDrain + 8 * w);   // every product has ended before TMEM is given back
      volatile int never = 0;
      mbar_wait_bounded(reinterpret_cast<uint64_t*>(smem + kDrain) + w, 0, &never);
    }
  } else {
    // ================================= softmax ================================
    more_registers<kSoftmaxRegs>();
    const int w = warp >> 2, wq = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_col0 = tmem + 2 * w * kSCols + lanes, o_col0 = tmem + kOCol0 + w * kHeadDim + lanes;
    const int s_bar = kSFull + 16 * w, p_bar = kPFull + 16 * w, o_bar = kODone + 16 * w;
    const uint64_t scale2 = pack2(scale_log2, scale_log2);
    const int share = wide ? 0 : 1 + w;
    unsigned job = 0, meets = 0;      // units so far
    bool ok = true;
    // The warps of the warpgroup.
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) bar_arrive(sm + kMeet + 8 * w);
      return wait(kMeet + 8 * w, meets++ & 1);
    };
    for (unsigned k = 0; ok; ++k) {
      ok = seg_get(share, k);
      if (!ok) break;
      const Seg& sg = segs[share * kAhead + k % kAhead];
      const int n = sg.units, j0 = sg.j0, f0 = sg.f0 - j0, f1 = sg.f1 - j0, f2 = sg.f2 - j0;
      if (n == 0) break;
      // The warp's queries: i_first .. of the tile, 4 at most.
      const int half = (sg.cnt + 1) >> 1;
      const int i_first = (wide && w ? half : 0) + 4 * wq;
      const int queries = min(4, (wide && !w ? half : sg.cnt) - i_first);
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const unsigned buf = (job + i) & 1;
        uint64_t see = ~0ull;                      // tokens of the unit that this row sees
        const bool edge = !(i < f0 || (i >= f1 && i <= f2));
        ok = wait(s_bar + 8 * buf, ((job + i) >> 1) & 1);
        if (!ok) break;
        tcgen05_fence_after();
        if (edge) {
          uint64_t any;                            // tokens that some query of the tile sees
          const int j = j0 + i, kb = (j < sg.first ? j : sg.low + j - sg.first) * kChunkTokens;
          if (sg.flags & kSegEmpty) {
            any = see = 0;
          } else if (kPrefix) {
            any = see = lowest(sg.len - kb);
          } else {
            const int pos = sg.p0 + i_first + (lane >> 3) - kb;   // of the row's query, in the unit
            any = tile_sees(plan, kb, sg.p0, sg.cnt);
            see = lowest(pos + 1) & (~lowest(pos - plan.window + 1) | lowest(plan.sinks - kb));
          }
          if (any != ~0ull) {
            // Unseen rows of V become zeros (their probabilities are zero, what
            // the page holds there may not be finite).  Both pipelines write the
            // same zeros to a wide tile's.
            const Ring ring = ring_of(wide, w);
            const unsigned vx = 2 * (job + i) + 1, h = ring.half(vx);
            ok = wait(kFull + 8 * h, ring.parity(vx));
            if (!ok) break;
            // (Thread t of the warpgroup: piece t % 16 of rows t / 16 + 8 x.)
            const int t = wq * 32 + lane;
            uint8_t* const vs = smem + h * kHalfBytes + ((t >> 3) & 1) * kBoxBytes + (t >> 4) * 128 + (t & 7) * 16;
            const uint64_t rows = any >> (t >> 4);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              if (!((rows >> (8 * x)) & 1)) *reinterpret_cast<uint4*>(vs + x * 1024) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
        }
        if (queries > 0) {
          const uint32_t sp = s_col0 + buf * kSCols;
          float s[64];
          tmem_ld32(sp, s);
          tmem_ld32(sp + 32, s + 32);
          tmem_wait_ld(s, 64);
          if (edge) {
            const uint32_t see0 = static_cast<uint32_t>(see), see1 = static_cast<uint32_t>(see >> 32);
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              if (!((see0 >> c) & 1)) s[c] = -INFINITY;
              if (!((see1 >> c) & 1)) s[c + 32] = -INFINITY;
            }
          }
          float mx[4] = {max3(s[0], s[1], s[2]), max3(s[3], s[4], s[5]), max3(s[6], s[7], s[8]), max3(s[9], s[10], s[11])};
#pragma unroll
          for (int c = 12; c < 60; c += 8) {
            mx[0] = max3(mx[0], s[c], s[c + 1]);
            mx[1] = max3(mx[1], s[c + 2], s[c + 3]);
            mx[2] = max3(mx[2], s[c + 4], s[c + 5]);
            mx[3] = max3(mx[3], s[c + 6], s[c + 7]);
          }
          mx[0] = max3(mx[0], s[60], s[61]);
          mx[1] = max3(mx[1], s[62], s[63]);
          const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]) * scale_log2;
          // (A row's first score that is not masked always does; until then every unit.)
          const bool raise = !(top < m + kRaise) && (lane >> 3) < queries;
          if (__any_sync(0xffffffffu, raise)) {
            // A maximum of +inf is no number from here on: inf - inf is none in the
            // formula either, and the powers on the FMA pipe would make zeros of it.
            float m_new = m, f = 1.f;
            if (raise) {
              m_new = top == INFINITY ? CUDART_NAN_F : top == -INFINITY && !(edge && see == 0) ? kLowest : top;
              f = top == -INFINITY ? 0.f : fast_exp2(m - m_new);
            }
            m = m_new;
            l *= f;
            if (i > 0) {                           // the accumulator of earlier units follows
              ok = wait(o_bar + 8 * (buf ^ 1), ((job + i - 1) >> 1) & 1);
              if (!ok) break;
              tcgen05_fence_after();
#pragma unroll 1
              for (int c = 0; c < kHeadDim; c += 32) {
                float o[32];
                tmem_ld32(o_col0 + c, o);
                tmem_wait_ld(o, 32);
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] *= f;
                tmem_st32(o_col0 + c, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;   // nothing seen yet: every probability is 0
          const uint64_t ref2 = pack2(-ref, -ref);
          uint64_t sum[4] = {0, 0, 0, 0};
          float pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            float a, b;
            const uint64_t x = fma2(pack2(s[2 * c], s[2 * c + 1]), scale2, ref2);
            if (c % kFmaEvery == kFmaEvery - 1) {
              exp2_fma(x, a, b);
            } else {
              unpack2(x, a, b);
              a = fast_exp2(a);
              b = fast_exp2(b);
            }
            sum[c & 3] = add2(sum[c & 3], pack2(a, b));
            // One rounding of the probabilities to bf16, half a step (2^-8 of the
            // value) at most: the output is rounded to the same type.
            pk[c] = __uint_as_float(pack_bf16(a, b));
          }
          tmem_st32(sp, pk);
          float sa, sb;
          unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), sa, sb);
          l += sa + sb;
          tmem_wait_st();
        }
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(sm + p_bar + 8 * buf);
      }
      if (!ok) break;

      // ---- the end of a segment: the output of a whole tile, or a partial ----
      job += n;
      ok = wait(o_bar + 8 * ((job - 1) & 1), ((job - 1) >> 1) & 1);   // its commit follows all earlier products
      if (!ok) break;
      tcgen05_fence_after();
      if (queries > 0) {
        const bool whole = sg.flags & kSegWhole, final = whole && (!kPrefix || (sg.flags & kSegAlone));
        // (No sum: no key, or scores of -inf only; a partial says which in its log-sum-exp.)
        const float inv = l == 0.f ? (final && m == kLowest ? CUDART_NAN_F : 0.f) : 1.f / l;
        const int row0 = sg.row + i_first, head = sg.head;   // the warp's first query, its first query head
        if (final) {
          // Output rows (query, head): 64 dims at a time through the warp's 4 KiB of
          // shared memory, 16-byte piece x of row y at x ^ (y % 8) (the map's 128-byte
          // swizzle), and from there by TMA, 8 rows of a query at once.  The next
          // tile does not wait for them.
          uint8_t* const row_at = smem + kTurnAt + warp * kTurnBytes + lane * 128;
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 64) {
            stores_read();                         // what lay here before has been read
            __syncwarp();
#pragma unroll
            for (int z = 0; z < 8; z += 4) {
              float o[32];
              tmem_ld32(o_col0 + c + 8 * z, o);
              tmem_wait_ld(o, 32);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] *= inv;
#pragma unroll
              for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4*>(row_at + (((z + x) ^ (lane & 7)) << 4)) =
                    make_uint4(pack_bf16(o[8 * x], o[8 * x + 1]), pack_bf16(o[8 * x + 2], o[8 * x + 3]),
                               pack_bf16(o[8 * x + 4], o[8 * x + 5]), pack_bf16(o[8 * x + 6], o[8 * x + 7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane < queries) store_box(&tm_out, c, head, row0 + lane, sm + kTurnAt + warp * kTurnBytes + lane * 1024);
          }
        } else {
          const Place at_o = whole ? own_place(work, plan.B, row0 + (lane >> 3), head >> 3, !(sg.flags & kSegGroup))
                                   : slot_place(work, wide, sg.slot, wide ? warp : wq, lane >> 3);
          float* const to = work.o + at_o.o + (lane & 7) * 4;
          const bool valid = (lane >> 3) < queries;
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 32) {
            float o[32];
            tmem_ld32(o_col0 + c, o);
            tmem_wait_ld(o, 32);
            if (valid) {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                *reinterpret_cast<float4*>(to + (c / 4 + x) * at_o.stride) =
                    make_float4(o[4 * x] * inv, o[4 * x + 1] * inv, o[4 * x + 2] * inv, o[4 * x + 3] * inv);
            }
          }
          if (valid) work.lse[at_o.lse + (lane & 7)] = l == 0.f ? m : m + __log2f(l);
        }
        tcgen05_fence_before();
        if (kPrefix && lane < queries) {   // where the merge finds the partials
          const int part = (sg.flags & kSegGroup) ? 0 : 2, pairs = plan.B * kNumKVHeads;
          int* const ends = work.ends + (row0 + lane) * kNumKVHeads + (head >> 3);
          if (j0 == 0)
            ends[part * pairs] = final ? kNone
                                       : (sg.slot >> 1) | (wide ? kEndWide : 0) |
                                             (((wide ? warp : wq) * 4 + lane) << kEndPlace) | (whole ? kEndWhole : 0);
          if (j0 + n == sg.all) ends[(part + 1) * pairs] = sg.slot >> 1;
          if (sg.flags & kSegAlone) ends[0] = kNone;
        }
      }
      if (kFold && !(sg.flags & kSegWhole)) {
        // One query a tile: the share that adds its last units folds the partials, a
        // quarter of the dims a warp.
        int* const verdict = reinterpret_cast<int*>(smem + kVerdictAt) + w;
        __threadfence();
        ok = meet();                               // the partial is written
        if (!ok) break;
        if (wq == 0 && lane == 0) {
          int* const count = work.count + sg.lo;
          __threadfence();
          const bool last = atomicAdd(count, n) + n == sg.all;
          if (last) *count = 0;
          *verdict = last;
        }
        ok = meet();
        if (!ok) break;
        if (*verdict) {
          __threadfence();
          const int lo = sg.lo;
          fold_query<4, 12>(work, sg.hi - lo + 1, lane,
                            [&](int x) { return slot_place(work, 0, 2 * (lo + x) + (x == 0), 0, 0); },
                            out + (static_cast<int64_t>(sg.row) * kNumQHeads + sg.head) * kHeadDim, wq);
        }
      }
      tcgen05_fence_before();
      seg_done(share, k);
    }
    stores_done();
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  // A wait ran out: what the merge would read may be a former call's.
  if (!kFold && tid == 0 && *reinterpret_cast<const volatile int*>(smem + kAbortAt)) work.ok[blockIdx.x] = 0;
  if (warp == kMmaWarp) {
    tcgen05_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- the merge kernels --------------------------------------------------------
// Whether no CTA of the call has given up: a tile's partials lie with several, and
// one that is missing would be a former call's.  (The whole warp.)
__device__ __forceinline__ bool call_is_whole(const Work& w, int grid, int lane) {
  int ok = 1;
#pragma unroll
  for (int i = 0; i < kMaxCtas; i += 32) ok &= ld_dep(w.ok + min(i + lane, grid - 1));
  return __all_sync(0xffffffffu, ok);
}

// Window mode.  The queries of a split tile are shared out over the slots that
// hold its partials.  The first kMergeY x 2 grid CTAs: kMergeY to a slot of the wide
// shares, 2 warps (half the dims each) to a query; the others: 2 slots of the
// narrow shares, 4 warps (a quarter of the dims each) to a query, since such a tile
// can have a partial for every few units.  Most CTAs find nothing to do, so it
// counts how many there are and how many an SM holds: over 1000 queries the call
// takes 37 us with 2 to a slot and 2 on an SM, 42 with 4 and 1 (149 registers, 12
// partials at a time instead of 8).
constexpr int kMergeWarps = 8, kMergeY = 2;
__global__ void __launch_bounds__(32 * kMergeWarps, 2)
window_merge_kernel(const Work work, int grid, __nv_bfloat16* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rest = static_cast<int>(blockIdx.x) - kMergeY * 2 * grid;
  const int wide = rest < 0;
  const int slot = wide ? blockIdx.x / kMergeY : rest * 2 + (warp >> 2);
  const uint4 a = ld_dep(reinterpret_cast<const uint4*>(work.parts + (wide ? 0 : 2 * kMaxCtas) + slot));
  const bool whole = call_is_whole(work, grid, lane);
  if (!a.w || !whole) return;
  const int lo = a.z & 0xffff, n = static_cast<int>(a.z >> 16) - lo + 1, cnt = static_cast<int>(a.w);
  const int half = wide ? (cnt + 1) >> 1 : cnt;   // pipeline 0's queries are in blocks 0 .., pipeline 1's in blocks 4 ..
  const int first = wide ? blockIdx.x % kMergeY * (kMergeWarps / 2) + (warp >> 1) : 0;
  const int step = wide ? kMergeY * kMergeWarps / 2 : 1;
  for (int q = (slot >> 1) - lo + n * first; q < cnt; q += n * step) {
    const int i = q < half ? q : q - half, block = (q < half ? 0 : 4) + (i >> 2);
    const auto at = [&](int k) { return slot_place(work, wide, 2 * (lo + k) + (k == 0), block, i & 3); };
    __nv_bfloat16* const to = out + ((static_cast<int64_t>(a.x) + q) * kNumQHeads + static_cast<int>(a.y) * kGroup) * kHeadDim;
    if (wide) fold_query<2, 4>(work, n, lane, at, to, warp & 1);
    else fold_query<4, 8>(work, n, lane, at, to, warp & 3);
  }
}

// Prefix mode: a CTA of 4 warps per (sequence, KV head), a quarter of the dims
// each: the partials of its group's tile, then those of its own tokens.
// kBatch partials at a time: 16 while the CTAs of 2 an SM are all that there are,
// 8 beyond.  16 (8): 9 sequences 19.6 (21.8) us, 128 under 16 prefixes of up to 1000
// 45.8 (42.7); 32 over a prefix of 32768 tokens 2% less than with 8.
constexpr int kFoldParts = 4;
template <int kBatch>
__global__ void __launch_bounds__(32 * kFoldParts, kBatch > 8 ? 2 : 4)
prefix_merge_kernel(const Work work, int grid, int B, __nv_bfloat16* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int pairs = B * kNumKVHeads, pair = blockIdx.x;
  int ends[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ends[i] = ld_dep(work.ends + i * static_cast<int64_t>(pairs) + pair);
  const bool whole = call_is_whole(work, grid, lane);
  if (!whole || ends[2] == kNone) return;   // (kNone: the output is written)
  auto many = [&](int first, int last) {
    return first == kNone ? 0 : first & kEndWhole ? 1 : last - (first & kEndShare) + 1;
  };
  const int n0 = many(ends[0], ends[1]), n1 = many(ends[2], ends[3]);
  fold_query<kFoldParts, kBatch>(work, n0 + n1, lane,
             [&](int i) {
               const bool own = i >= n0;
               const int first = own ? ends[2] : ends[0];
               if (own) i -= n0;
               if (first & kEndWhole) return own_place(work, B, pair / kNumKVHeads, pair % kNumKVHeads, own);
               return slot_place(work, first & kEndWide ? 1 : 0,
                                 2 * ((first & kEndShare) + i) + (i == 0),
                                 (first >> (kEndPlace + 2)) & 7, (first >> kEndPlace) & 3);
             },
             out + static_cast<int64_t>(pair) * kGroup * kHeadDim, threadIdx.x >> 5);
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// The workspace's parts: counts, rows and their log-sum-exps, parts, ends, the
// verdicts.  `queries`: the most queries of an entry; `pairs`: prefix mode's.
size_t layout(Work* w, void* at, int64_t places, int queries, int64_t pairs) {
  const int narrow = kGroup * (queries <= 4 ? queries : kNarrowQ);   // whole blocks of 4 queries, or one smaller block
  const int wide = queries <= kNarrowQ ? 0 : kGroup * kWideQ;
  const int64_t rows = places + 2ll * kMaxCtas * wide + 4ll * kMaxCtas * narrow;
  const size_t count = 2 * kMaxCtas * sizeof(int), parts = 6 * kMaxCtas * sizeof(int4);
  const size_t o = static_cast<size_t>(rows) * kHeadDim * 4, lse = round16(rows * 4);
  const size_t ends = round16(4 * pairs * 4), ok = kMaxCtas * sizeof(int);
  if (w) {
    char* p = static_cast<char*>(at);
    w->count = reinterpret_cast<int*>(p);
    w->o = reinterpret_cast<float*>(p += count);
    w->lse = reinterpret_cast<float*>(p += o);
    w->parts = reinterpret_cast<int4*>(p += lse);
    w->ends = reinterpret_cast<int*>(p += parts);
    w->ok = reinterpret_cast<int*>(p += ends);
    w->rows[0] = narrow;
    w->rows[1] = wide;
    w->block_rows[0] = narrow < 4 * kGroup ? narrow : 4 * kGroup;
    w->block_rows[1] = 4 * kGroup;
    w->slots[1] = places;
    w->slots[0] = places + 2ll * kMaxCtas * wide;
  }
  return count + o + lse + parts + ends + ok;
}
size_t window_layout(Work* w, void* at, int max_q) { return layout(w, at, 0, max_q, 0); }
size_t prefix_layout(Work* w, void* at, int B) {
  return layout(w, at, 2ll * kNumQHeads * B, B, static_cast<int64_t>(B) * kNumKVHeads);
}

std::mutex g_mu;
bool g_attr_set[3][64] = {};
// lsa_debug_withhold_share: the limit in microseconds and the CTA + 1 for the next
// call, 0: none.
std::atomic<uint64_t> g_withhold{0};

int encode_pool(CUtensorMap* map, const void* base, int64_t n_slots, int rows) {
  const cuuint64_t dims[2] = {kHeadDim, static_cast<cuuint64_t>(n_slots) * kNumKVHeads * kChunkTokens};
  const cuuint64_t strides[1] = {kHeadDim * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(rows)}, estr[2] = {1, 1};
  return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? LSA_OK
             : LSA_ERR_CUDA;
}
// The 8 query heads of a KV head for `queries` queries: rows (query, head).
int encode_q(CUtensorMap* map, const void* base, int64_t rows, int queries) {
  const cuuint64_t dims[3] = {kHeadDim, kNumQHeads, static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {kHeadDim * 2, kNumQHeads * kHeadDim * 2};
  const cuuint32_t box[3] = {64, kGroup, static_cast<cuuint32_t>(queries)}, estr[3] = {1, 1, 1};
  return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? LSA_OK
             : LSA_ERR_CUDA;
}

// Checks of the arguments that both calls share.
int check(const void* q, const void* k_pool, const void* v_pool, int64_t n_slots, const int32_t* len, int B, int max_chunks,
          int least_chunks, float scale, const void* out) {
  if (!q || !k_pool || !v_pool || !len || !out || n_slots <= 0 || B <= 0 || max_chunks < least_chunks)
    return LSA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return LSA_ERR_INVALID_ARG;
  if (B > LSA_MAX_BATCH) return LSA_ERR_UNSUPPORTED_SHAPE;
  // Positions and TMA rows (n_slots * 512) are 32-bit.
  if (max_chunks > (1 << 23) || n_slots >= (int64_t{1} << 22)) return LSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return LSA_ERR_MISALIGNED;
  return LSA_OK;
}

template <Mode kMode>
int launch(Plan& plan, const Work& work, const void* q, const void* k_pool, const void* v_pool, float scale, void* out,
           int64_t most_units, void* stream) {
  const int sms = device_sm_count();
  if (sms < 2 || !tensor_map_encoder()) return LSA_ERR_NO_DEVICE;   // (wide and narrow tiles have CTAs of their own)
  int dev = 0;
  cudaGetDevice(&dev);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (dev < 64 && !g_attr_set[kMode][dev]) {
      if (cudaFuncSetAttribute(pool_attn_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess) {
        cudaGetLastError();
        return LSA_ERR_CUDA;
      }
      g_attr_set[kMode][dev] = true;
    }
  }
  CUtensorMap tm_k, tm_v, tm_k_part = {}, tm_v_part = {}, tm_q16 = {}, tm_q8 = {}, tm_q1, tm_out;
  int st = encode_pool(&tm_k, k_pool, plan.n_slots, kChunkTokens);
  if (st == LSA_OK) st = encode_pool(&tm_v, v_pool, plan.n_slots, kChunkTokens);
  if (kMode != kPrefixes) {
    if (st == LSA_OK) st = encode_pool(&tm_k_part, k_pool, plan.n_slots, kPartRows);
    if (st == LSA_OK) st = encode_pool(&tm_v_part, v_pool, plan.n_slots, kPartRows);
  }
  if (kMode != kWindowToken) {   // single tokens have neither wide tiles nor others than of one query
    if (st == LSA_OK) st = encode_q(&tm_q16, q, plan.rows, kWideQ / 2);
    if (st == LSA_OK) st = encode_q(&tm_q8, q, plan.rows, kNarrowQ);
  }
  if (st == LSA_OK) st = encode_q(&tm_q1, q, plan.rows, 1);
  if (st == LSA_OK) st = encode_q(&tm_out, out, plan.rows, 1);
  if (st != LSA_OK) return st;
  // As many CTAs as the most that there can be to do is worth, one per SM.
  const int most = sms < kMaxCtas ? sms : kMaxCtas;
  const int64_t want = (most_units + kMinShare - 1) / kMinShare;
  const int grid = want < most ? (want < 2 ? 2 : static_cast<int>(want)) : most;
  const uint64_t withhold = g_withhold.exchange(0);
  plan.withheld = withhold ? static_cast<int>((withhold & 0xffffffffu) - 1) % grid : -1;
  plan.wait_ns = withhold ? (withhold >> 32) * 1000 : kWaitLimitNs;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  __nv_bfloat16* const o = static_cast<__nv_bfloat16*>(out);
  launch_pdl(true, pool_attn_kernel<kMode>, dim3(grid), dim3(kThreads), kSmemBytes, s, tm_k, tm_v, tm_k_part, tm_v_part,
             tm_q16, tm_q8, tm_q1, tm_out, plan, work,
             scale * 1.4426950408889634f, o, lsa_device_status_ptr());
  if (kMode == kPrefixes)
    launch_pdl(true, plan.B * kNumKVHeads > 2 * sms ? prefix_merge_kernel<8> : prefix_merge_kernel<16>,
               dim3(plan.B * kNumKVHeads), dim3(32 * kFoldParts), 0, s, work, grid, plan.B, o);
  else if (kMode == kWindow)
    launch_pdl(true, window_merge_kernel, dim3((2 * kMergeY + 2) * grid),
               dim3(32 * kMergeWarps), 0, s, work, grid, o);
  return launch_status();
}

}  // namespace pool
}  // namespace lsa

extern "C" {

int lsa_debug_withhold_share(int cta, unsigned int limit_us) {
  if (cta < -1 || limit_us == 0 || limit_us > 2000000u) return LSA_ERR_INVALID_ARG;
  lsa::pool::g_withhold.store(cta < 0 ? 0 : static_cast<uint64_t>(limit_us) << 32 | (static_cast<unsigned>(cta) + 1u));
  return LSA_OK;
}

size_t lsa_window_attn_workspace_size(int B, int max_q) {
  if (B <= 0 || B > LSA_MAX_BATCH || max_q <= 0) return 0;
  return lsa::pool::window_layout(nullptr, nullptr, max_q);
}

int lsa_window_attn(const void* q, int64_t T, const void* k_pool, const void* v_pool, int64_t n_slots,
                    const int32_t* chunk_table, const int32_t* cu_q, const int32_t* seq_len, int B, int max_chunks, int max_q,
                    int window, int n_sink, float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                    void* stream) {
  using namespace lsa;
  if (!cu_q || T <= 0 || max_q <= 0 || window <= 0 || n_sink < 0) return LSA_ERR_INVALID_ARG;
  const int st = pool::check(q, k_pool, v_pool, n_slots, seq_len, B, max_chunks, 1, softmax_scale, out);
  if (st != LSA_OK) return st;
  if (T > (int64_t{1} << 30)) return LSA_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || workspace_bytes < pool::window_layout(nullptr, nullptr, max_q)) return LSA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LSA_ERR_MISALIGNED;
  const int most = max_chunks * kChunkTokens;
  pool::Plan plan = {};
  plan.B = B;
  plan.rows = T;
  plan.cu = cu_q;
  plan.len = seq_len;
  plan.table = chunk_table;
  plan.max_chunks = max_chunks;
  plan.max_q = max_q;
  plan.window = window < most ? window : most;
  plan.sinks = n_sink < most ? n_sink : most;
  plan.n_slots = n_slots;
  pool::Work work;
  pool::window_layout(&work, workspace, max_q);
  // A bound of the units: every tile sees its window, its queries' span and the sinks.
  const int64_t seen = static_cast<int64_t>(plan.window) / kChunkTokens + 3 + plan.sinks / kChunkTokens + 1;
  const int64_t tiles = T / pool::kWideQ + B;
  const int64_t units = kNumKVHeads * tiles * ((seen < max_chunks ? seen : max_chunks) + pool::kTileCost);
  // Folded in the kernel (by a second one): 14.1 (15.7) us for one token over 4096,
  // 22.5 (23.8) over 20000; but 26.2 (24.2) for 2 queries over 20000, 21.6 (20.4) for
  // 4 of 4 sequences each, 36 (32) for 8 of 8.
  return max_q == 1
             ? pool::launch<pool::kWindowToken>(plan, work, q, k_pool, v_pool, softmax_scale, out, units, stream)
             : pool::launch<pool::kWindow>(plan, work, q, k_pool, v_pool, softmax_scale, out, units, stream);
}

size_t lsa_prefix_attn_workspace_size(int B, int n_groups) {
  if (B <= 0 || B > LSA_MAX_BATCH || n_groups < 0 || n_groups > B) return 0;
  return lsa::pool::prefix_layout(nullptr, nullptr, B);
}

int lsa_prefix_decode_attn(const void* q, const void* k_pool, const void* v_pool, int64_t n_slots,
                           const int32_t* prefix_table, const int32_t* cu_group, const int32_t* prefix_len, int n_groups,
                           int max_prefix_chunks, const int32_t* chunk_table, const int32_t* suffix_len, int B,
                           int max_chunks, float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                           void* stream) {
  using namespace lsa;
  if (n_groups < 0 || n_groups > B || (n_groups > 0 && (!prefix_table || !cu_group || !prefix_len || max_prefix_chunks <= 0)))
    return LSA_ERR_INVALID_ARG;
  // (Without a table there may be no own chunks at all: before the first own token.)
  const int st = pool::check(q, k_pool, v_pool, n_slots, suffix_len, B, max_chunks, chunk_table ? 1 : 0, softmax_scale, out);
  if (st != LSA_OK) return st;
  if (max_prefix_chunks > (1 << 23)) return LSA_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || workspace_bytes < pool::prefix_layout(nullptr, nullptr, B)) return LSA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LSA_ERR_MISALIGNED;
  pool::Plan plan = {};
  plan.B = B;
  plan.groups = n_groups;
  plan.rows = B;
  plan.cu = cu_group;
  plan.len = suffix_len;
  plan.group_len = prefix_len;
  plan.table = chunk_table;
  plan.group_table = prefix_table;
  plan.max_chunks = max_chunks;
  plan.group_chunks = max_prefix_chunks;
  plan.max_q = B;
  plan.n_slots = n_slots;
  pool::Work work;
  pool::prefix_layout(&work, workspace, B);
  const int64_t tiles = n_groups > 0 ? B / pool::kWideQ + n_groups : 0;
  const int64_t units = kNumKVHeads * (tiles * (static_cast<int64_t>(max_prefix_chunks) + pool::kTileCost) +
                                       static_cast<int64_t>(B) * (max_chunks + pool::kTileCost));
  return pool::launch<pool::kPrefixes>(plan, work, q, k_pool, v_pool, softmax_scale, out, units, stream);
}

}  // extern "C"
