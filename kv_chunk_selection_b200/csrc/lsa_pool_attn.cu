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
// One kernel serves both.  Its work is a list of units: a unit is 64 tokens
// (one chunk) of K and V of one KV head, 32 KiB, against a tile of up to 32
// queries (x 8 query heads = 256 rows).  The units of all tiles are laid end
// to end and the grid (one CTA per SM) cuts the list into equal contiguous
// ranges, so a single token over a long window and a long prompt both fill the
// chip; a tile that a cut splits leaves one partial per CTA (normalised rows
// and their log-sum-exps), which a second kernel folds in CTA order.
//
// Roles of a CTA (12 warps):
//   warps 0-3, 4-7  two softmax warpgroups, a thread per row: the scores of a
//                   unit come from TMEM, the probabilities go back to TMEM in
//                   the scores' place as bf16.  The running maximum is only
//                   raised when it grows by more than 2^8 (the sums stay
//                   exact, the accumulator is rescaled rarely);
//   warps 8, 9      issue the tcgen05.mma of a warpgroup each: S = Q K^T (128 x
//                   64 x 128), and O += P V (128 x 128 x 64) with P from TMEM;
//   warp 10         streams the units with TMA into a ring of 4 stages;
//   warp 11         walks the list, a few segments ahead of the others, and
//                   loads the query tiles.
// A tile of more than 16 queries is "wide": each warpgroup has 16 queries (128
// rows) and both use every unit.  A smaller tile is "narrow": both warpgroups
// have the same rows and take alternate units, so that the softmax of one unit
// runs beside the products of the next, and their two accumulators are joined
// at the end; that carries single tokens at the rate of the memory although 8
// of 128 rows of a product are theirs.
//
// TMEM (512 columns): scores 2 warpgroups x 2 buffers x 64, accumulators 2 x
// 128.  Rows that no query of a tile sees are zeroed in V's stage before the
// product, so a page's unwritten tail may hold anything (0 times NaN is NaN);
// the scores there are masked by selection.
#include <math.h>

#include <mutex>

#include "lsa_common.cuh"
#include "lsa_runtime.cuh"

namespace lsa {
namespace pool {

constexpr int kWideQ = 32;                   // queries of a tile
constexpr int kHalfQ = 16;                   // queries of a warpgroup: 16 x 8 heads = 128 rows
constexpr int kSoftmaxThreads = 256;
constexpr int kMmaWarp = 8;                  // and 9: one for each softmax warpgroup
constexpr int kLoadWarp = 10, kPlanWarp = 11;
constexpr int kThreads = 12 * 32;
constexpr int kStages = 4;
constexpr int kBoxBytes = 8192;              // 64 tokens x 64 dims
constexpr int kStageBytes = 4 * kBoxBytes;   // K dims 0-63, 64-127, V dims 0-63, 64-127
constexpr int kQBoxBytes = 16384;            // 128 rows x 64 dims
constexpr int kQTileBytes = 2 * kQBoxBytes;
constexpr int kTurnBytes = 4096;             // a warp's rows on their way out: 32 rows x 128 bytes
constexpr int kAhead = 8;                    // places for segments that the planner is ahead
constexpr int kMaxCtas = LSA_POOL_ATTN_MAX_CTAS;
#ifndef FMA_EVERY
#define FMA_EVERY 4
#endif
constexpr int kFmaEvery = FMA_EVERY;
constexpr float kRaise = 8.f;                // growth of the maximum (log2) that rescales the accumulator
constexpr int kSCols = 64, kOCol0 = 256;     // TMEM: S[w][b] at (2 w + b) * 64, O[w] at 256 + 128 w
constexpr int64_t kMinUnitsPerCta = 2;

struct Plan {
  int prefix_mode;
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
  __device__ int lists() const { return prefix_mode ? groups + B : B; }
};

// Partials.  A CTA's first and last segment can be part of a tile: they have a
// record each, slots 2c and 2c + 1, of rows_cap rows (query x head).  In window
// mode a whole tile goes straight to the output; in prefix mode its rows have
// places of their own, 64 per sequence for its prefix and 64 for its own tokens,
// after which the slots follow.
struct Work {
  float* o;          // [rows][128], normalised
  float* lse;        // [rows], base 2
  int4* seg;         // window mode: [2 * kMaxCtas], a slot's tile: first query, KV head and queries,
                     // first and last CTA, slot of the first CTA's record + 1 (0: nothing to fold)
  int* ends;         // prefix mode: [4][8 B], by (sequence, KV head): first and last partial of the
                     // prefix, of the own tokens
  int* ok;           // prefix mode: the offsets were valid
  int rows_cap;
};
// The first partial of a (sequence, KV head): CTA, slot 2c + bit, the query's
// place in the tile, or that the rows are in their own place; kNone: no partial.
constexpr int kEndSlot = 1 << 8, kEndPlace = 16, kEndWhole = 1 << 24, kNone = -1;

// The queries and the keys of one list: a sequence, or a group over its prefix.
struct List {
  int q0, nq, len;
  const int32_t* table;
  int64_t ident;             // identity layout: slot of chunk 0 (table null)
};

__device__ __forceinline__ List load_list(const Plan& p, int v) {
  List s;
  int cap;
  if (p.prefix_mode && v >= p.groups) {
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
    s.len = ld_dep((p.prefix_mode ? p.group_len : p.len) + v);
    cap = p.prefix_mode ? p.group_chunks : p.max_chunks;
    s.ident = static_cast<int64_t>(v) * cap;
    const int32_t* t = p.prefix_mode ? p.group_table : p.table;
    s.table = t ? t + s.ident : nullptr;
  }
  if (s.len < 0 || s.len > cap * kChunkTokens) s.len = -1;   // reported by the scan
  return s;
}

__device__ __forceinline__ int tiles_of(const List& s) { return (s.nq + kWideQ - 1) / kWideQ; }

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

// Units of the first t tiles of a list, for one KV head.  A tile without a key
// in sight still has one (empty) unit, so that its rows are written.
__device__ __forceinline__ int64_t units_before(const Plan& p, const List& s, int t) {
  if (p.prefix_mode) {
    const int n = s.len > 0 ? (s.len + kChunkTokens - 1) / kChunkTokens : 1;
    return static_cast<int64_t>(t) * n;
  }
  const int pos0 = (s.len < 0 ? 0 : s.len) - s.nq;
  const int64_t none = int64_t{1} << 40;
  const int a_low = pos0 - p.window + 1;
  int64_t n = chunk_sum(pos0 + kWideQ - 1, t, none) + t - chunk_sum(a_low, t, none) +
              chunk_sum(a_low, t, (p.sinks + kChunkTokens - 1) / kChunkTokens);
  if (t > 0 && t * kWideQ > s.nq) {   // the last tile ends before its 32nd query
    const int full = (pos0 + t * kWideQ - 1) >> 6, real = (pos0 + s.nq - 1) >> 6;
    n += (real > 0 ? real : 0) - (full > 0 ? full : 0);
  }
  return n;
}

// A 64-bit quotient, in 32 bits where the operands allow it (five times faster).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}
struct Partition {
  int64_t base, rem;
  __device__ Partition(int64_t total, int G) : base(quotient(total, G)), rem(total - base * G) {}
  __device__ int64_t start(int c) const { return c * base + (c < rem ? c : rem); }
  __device__ int cta_of(int64_t u) const {
    const int64_t big = rem * (base + 1);
    return static_cast<int>(u < big ? quotient(u, base + 1) : rem + quotient(u - big, base));
  }
};

// A walk over the tiles of the unit list.
struct Cursor {
  int v, g, t, j;            // list, KV head, tile, unit of the tile
  List s;
  int tiles;
  int cnt;                   // queries of the tile
  int n;                     // its units
  int p0;                    // window mode: position of its first query
  int low, first;            // window mode: first chunk of the window, sink chunks before it
  bool empty;                // no key in sight: the one unit is empty

  __device__ void set_tile(const Plan& p) {
    cnt = min(kWideQ, s.nq - t * kWideQ);
    if (p.prefix_mode) {
      n = s.len > 0 ? (s.len + kChunkTokens - 1) / kChunkTokens : 0;
      p0 = low = first = 0;
    } else {
      p0 = (s.len < 0 ? 0 : s.len) - s.nq + t * kWideQ;
      const int p1 = p0 + cnt - 1;
      low = max(0, p0 - p.window + 1) >> 6;
      first = min(low, (p.sinks + kChunkTokens - 1) / kChunkTokens);
      n = p1 < 0 ? 0 : (p1 >> 6) - low + 1 + first;
    }
    empty = n == 0;
    n = max(n, 1);
  }
  __device__ void set_list(const Plan& p) {
    s = load_list(p, v);
    tiles = tiles_of(s);
  }
  // At unit r of list `list`, whose KV heads have per_head units each.
  __device__ void start(const Plan& p, int list, const List& l, int64_t per_head, int64_t r) {
    v = list;
    s = l;
    tiles = tiles_of(s);
    g = static_cast<int>(quotient(r, per_head));
    r -= g * per_head;
    int lo = 0, hi = tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (units_before(p, s, mid) <= r) lo = mid; else hi = mid - 1;
    }
    t = lo;
    j = static_cast<int>(r - units_before(p, s, t));
    set_tile(p);
  }
  // To the first unit of the next tile; the caller knows that there is one.
  __device__ void next(const Plan& p) {
    j = 0;
    if (++t == tiles) {
      t = 0;
      if (++g == kNumKVHeads) {
        g = 0;
        do {
          ++v;
          set_list(p);
        } while (tiles == 0);
      }
    }
    set_tile(p);
  }
  __device__ int chunk(int u) const { return u < first ? u : low + u - first; }
  __device__ bool wide() const { return cnt > kHalfQ; }
};

// 64 bits: the lowest x.
__device__ __forceinline__ uint64_t lowest(int x) {
  return x <= 0 ? 0ull : x >= 64 ? ~0ull : (1ull << x) - 1;
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
// Waits, at most kWaitLimitNs, or until another role has given up; the same
// answer in every lane, so that the warp's collective instructions stay whole.
// `abort_flag`: 0, or 1 once a wait of the CTA ran out.
__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, unsigned parity, uint32_t abort_flag, unsigned* status) {
  const unsigned long long t0 = globaltimer_ns();
  for (unsigned it = 1;; ++it) {
    if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
    if ((it & 63u) == 0) {
      int given_up;
      asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(given_up) : "r"(abort_flag) : "memory");
      const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
      if (__any_sync(0xffffffffu, given_up || late)) {
        if (!given_up) set_status(status, LSA_DEV_ERR_TIMEOUT);
        asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(abort_flag), "r"(1) : "memory");
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, unsigned parity, uint32_t abort_flag, unsigned* status) {
  if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
  return bar_wait_slow(bar, parity, abort_flag, status);
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
// (minimax for the relative error: 2.9e-6, against 2^-9 of the rounding to bf16
// that follows), and the integer part added to the exponent.  From -127 down
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

// Exclusive prefix sum of `x` over the block (kWarps warps) and the total.
template <int kWarps>
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* sm, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += y;
  }
  if (lane == 31) sm[warp] = inc;
  __syncthreads();
  int64_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm[w];
    sum += sm[w];
  }
  *total = sum;
  return before + inc - x;
}

// A segment: the units of one tile that this CTA has.  The planner warp writes
// them to shared memory a few ahead, so that no other role walks the list or
// waits for its loads.
struct Seg {
  int units;                 // 0: the list has ended
  int flags;                 // kSegWide ...
  int j0;                    // its first unit in the tile
  int cnt, row, head;        // the tile's queries, the first one's row of q, the first query head
  int first, low;            // chunk of unit j: j < first ? j : low + j - first
  int f0, f1, f2;            // units that every query sees whole: j < f0 and f1 <= j <= f2
  int p0, len;               // window mode: position of the first query; prefix mode: tokens
  int g;
  const int32_t* table;
  int64_t ident;
};
constexpr int kSegWide = 1, kSegEmpty = 2, kSegAgain = 4, kSegGroup = 8, kSegWhole = 16;

// Shared memory, from a 1024-byte boundary.
constexpr int kQAt = kStages * kStageBytes, kTurnAt = kQAt + 2 * kQTileBytes, kMlAt = kTurnAt + 8 * kTurnBytes;
constexpr int kSegAt = kMlAt + 2 * 2 * 128 * 4, kBarAt = kSegAt + kAhead * static_cast<int>(sizeof(Seg));
// Barriers, 8 bytes each.
constexpr int kFull = kBarAt, kEmpty = kFull + 8 * kStages;            // ring stages
constexpr int kSFull = kEmpty + 8 * kStages;                            // [2 warpgroups][2 buffers] scores are there
constexpr int kPFull = kSFull + 32, kODone = kPFull + 32;               // probabilities are; the product that read them is done
constexpr int kQFull = kODone + 32, kQEmpty = kQFull + 8;
constexpr int kSegFull = kQEmpty + 8, kSegEmptied = kSegFull + 8 * kAhead;
constexpr int kMeet = kSegEmptied + 8 * kAhead, kReady = kMeet + 8;     // both warpgroups; the scratch has been read
constexpr int kDrain = kReady + 8;                                      // [2]
constexpr int kTmemAt = kDrain + 16, kAbortAt = kTmemAt + 4;
constexpr int kSmemBytes = kAbortAt + 4;
static_assert(kSmemBytes <= 232448 && sizeof(Seg) % 8 == 0, "shared memory of one CTA");

__global__ void __launch_bounds__(kThreads, 1)
pool_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q1, const Plan plan,
                 const Work work, float scale_log2, __nv_bfloat16* __restrict__ out, unsigned* status) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sm = smem_u32(smem);
  const uint32_t abort_flag = sm + kAbortAt;

  // ---- before the previous kernel has ended: barriers and TMEM ---------------
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(sm + kFull + 8 * i, 1);
      bar_init(sm + kEmpty + 8 * i, 2);   // both product warps (or one of them twice)
    }
    for (int i = 0; i < 4; ++i) {
      bar_init(sm + kSFull + 8 * i, 1);
      bar_init(sm + kPFull + 8 * i, 4);   // the warps of the warpgroup
      bar_init(sm + kODone + 8 * i, 1);
    }
    bar_init(sm + kQFull, 1);
    bar_init(sm + kQEmpty, 2);
    for (int i = 0; i < kAhead; ++i) {
      bar_init(sm + kSegFull + 8 * i, 1);
      bar_init(sm + kSegEmptied + 8 * i, 11);   // softmax, product and load warps
    }
    bar_init(sm + kMeet, kSoftmaxThreads / 32);
    bar_init(sm + kReady, 1);
    bar_init(sm + kDrain, 1);
    bar_init(sm + kDrain + 8, 1);
    *reinterpret_cast<volatile int*>(smem + kAbortAt) = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(reinterpret_cast<uint32_t*>(smem + kTmemAt), 512);
  if (tid == kLoadWarp * 32) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_q1);
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the unit list: validity, total, and the place where this CTA starts --
  // (The scratch lies in the ring, which is empty until the roles start.)
  int64_t* scan = reinterpret_cast<int64_t*>(smem);
  List* found = reinterpret_cast<List*>(scan + 40);
  const int V = plan.lists();
  const int per = (V + kThreads - 1) / kThreads;
  const int v_lo = min(V, tid * per), v_hi = min(V, v_lo + per);
  int bad = 0;
  int64_t mine = 0;
  const int n_cu = plan.prefix_mode ? plan.groups : plan.B;
  if (tid == kThreads - 1 && n_cu > 0) {
    bad |= ld_dep(plan.cu) != 0;
    const int last = ld_dep(plan.cu + n_cu);
    bad |= last < 0 || last > plan.rows;
  }
  auto units_of_list = [&](const List& s) {
    return s.nq > 0 ? kNumKVHeads * units_before(plan, s, tiles_of(s)) : 0;
  };
  List s_last = {};   // the thread's last list: its only one for up to kThreads lists
  for (int v = v_lo; v < v_hi; ++v) {
    s_last = load_list(plan, v);
    if (s_last.len < 0 && blockIdx.x == 0) set_status(status, LSA_DEV_ERR_BAD_COUNT);
    bad |= s_last.nq < 0 || (!plan.prefix_mode && s_last.nq > plan.max_q);
    mine += units_of_list(s_last);
  }
  int64_t total;
  bad = __syncthreads_or(bad);
  const int64_t before = block_scan<kThreads / 32>(bad ? 0 : mine, scan, &total);
  const Partition part(total, gridDim.x);
  const int64_t u0 = part.start(blockIdx.x), u1 = part.start(blockIdx.x + 1);
  if (part.base >= (1 << 30)) bad = 1;   // a CTA counts its units in 32 bits
  if (sm & 1023u) {                      // the 128-byte swizzle repeats every 1024 bytes
    if (tid == 0) set_status(status, LSA_DEV_ERR_INTERNAL);
    bad = 1;
  }
  if (blockIdx.x == 0) {
    if (tid == 0) {
      if (bad) set_status(status, LSA_DEV_ERR_CAPACITY);
      if (plan.prefix_mode) *work.ok = bad ? 0 : 1;
    }
    if (plan.prefix_mode && !bad)   // sequences behind the last group have no prefix
      for (int x = (n_cu ? ld_dep(plan.cu + n_cu) : 0) * kNumKVHeads + tid; x < plan.B * kNumKVHeads; x += kThreads)
        work.ends[x] = kNone;
  }
  const bool idle = bad || u0 >= u1;
  if (!idle && before <= u0 && u0 < before + mine) {   // one thread: the list of unit u0
    int64_t at = before, n = mine;
    int v = v_lo;
    if (per > 1) {
      for (;; ++v) {
        s_last = load_list(plan, v);
        n = units_of_list(s_last);
        if (u0 < at + n) break;
        at += n;
      }
    }
    *found = s_last;
    scan[32] = v;
    scan[33] = u0 - at;
    scan[34] = n / kNumKVHeads;
  }
  fence_proxy_async_smem();   // the scratch was written here; TMA writes it next
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *reinterpret_cast<const volatile uint32_t*>(smem + kTmemAt);
  const Seg* const segs = reinterpret_cast<const Seg*>(smem + kSegAt);
  auto wait = [&](int bar, unsigned parity) { return bar_wait(sm + bar, parity, abort_flag, status); };
  // Segment k of this CTA; its place is free again once every role has said so.
  auto seg_get = [&](unsigned k) { return wait(kSegFull + 8 * (k % kAhead), (k / kAhead) & 1); };
  auto seg_done = [&](unsigned k) {
    __syncwarp();
    if (lane == 0) bar_arrive(sm + kSegEmptied + 8 * (k % kAhead));
  };

  if (warp >= kMmaWarp) {
    fewer_registers<kOtherRegs>();
    if (warp == kPlanWarp) {
      // ===================== the list, and the query tiles ===================
      Cursor cur = {};
      int left = 0;
      if (!idle) {
        cur.start(plan, static_cast<int>(scan[32]), *found, scan[34], scan[33]);
        left = static_cast<int>(u1 - u0);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(sm + kReady);   // the scratch has been read: the ring may be filled
      const int me = blockIdx.x;
      int4 seg0 = make_int4(0, 0, 0, 0), seg1 = seg0;
      unsigned put = 0;      // segments written
      bool ended = false;    // the list's end is
      auto publish = [&]() {
        if (put >= kAhead && !wait(kSegEmptied + 8 * (put % kAhead), (put / kAhead - 1) & 1)) return false;
        Seg* const s = reinterpret_cast<Seg*>(smem + kSegAt) + put % kAhead;
        if (left <= 0) {
          if (lane == 0) s->units = 0;
          ended = true;
        } else {
          const int units = min(cur.n - cur.j, left), row = cur.s.q0 + cur.t * kWideQ;
          const bool begins = cur.j == 0, ends = cur.j + units == cur.n;
          if (lane == 0) {
            s->units = units;
            s->flags = (cur.cnt > kHalfQ ? kSegWide : 0) | (cur.empty ? kSegEmpty : 0) | (cur.tiles > 1 ? kSegAgain : 0) |
                       (plan.prefix_mode && cur.v < plan.groups ? kSegGroup : 0) | (begins && ends ? kSegWhole : 0);
            s->j0 = cur.j;
            s->cnt = cur.cnt;
            s->row = row;
            s->head = cur.g * kGroup;
            s->first = cur.first;
            s->low = cur.low;
            int f0 = 0, f1 = 0, f2 = -1;
            if (plan.prefix_mode) {
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
            s->g = cur.g;
            s->table = cur.s.table;
            s->ident = cur.s.ident;
          }
          // What the merge has to know.
          if (plan.prefix_mode) {
            if (lane < cur.cnt) {
              int* at = work.ends + (cur.v < plan.groups ? 0 : 2 * kNumKVHeads * plan.B) + (row + lane) * kNumKVHeads + cur.g;
              if (begins) at[0] = me | (put ? kEndSlot : 0) | (lane << kEndPlace) | (ends ? kEndWhole : 0);
              if (ends) at[kNumKVHeads * plan.B] = me;
            }
          } else if (!(begins && ends)) {
            const int64_t tile_u = u1 - left - cur.j;   // the tile's first unit
            const int lo = begins ? me : part.cta_of(tile_u), hi = ends ? me : part.cta_of(tile_u + cur.n - 1);
            const int4 a = make_int4(row, cur.g | (cur.cnt << 8), lo | (hi << 16), 2 * lo + (part.start(lo) == tile_u ? 0 : 1) + 1);
            if (put) seg1 = a;
            else seg0 = a;
          }
          left -= units;
          if (left > 0) cur.next(plan);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(sm + kSegFull + 8 * (put % kAhead));
        ++put;
        return true;
      };
      bool ok = true;
      unsigned loads = 0;
      // One place stays free: in segment k the planner writes segment k + 7 where
      // k - 1 was, which does not hold back the query tile of k + 1.
      for (int i = 0; ok && i < kAhead - 1 && !ended; ++i) ok = publish();
      for (unsigned k = 0; ok; ++k) {
        const Seg& s = segs[k % kAhead];
        const int units = s.units, cnt = s.cnt, row = s.row, head = s.head;
        if (units == 0) break;
        if (k) ok = wait(kQEmpty, (k - 1) & 1);
        if (!ok) break;
        ++loads;
        if (lane == 0) {
          const uint32_t bar = sm + kQFull, q = sm + kQAt;
          if (cnt == 1) {   // 8 rows; what the other rows of the tile hold is not read back
            bar_expect(bar, 2 * kGroup * 128);
            load_box(q, &tm_q1, 0, head, row, bar);
            load_box(q + kQBoxBytes, &tm_q1, 64, head, row, bar);
          } else {
            const int halves = cnt > kHalfQ ? 2 : 1;
            bar_expect(bar, halves * kQTileBytes);
            for (int w = 0; w < halves; ++w) {
              load_box(q + w * kQTileBytes, &tm_q, 0, head, row + w * kHalfQ, bar);
              load_box(q + w * kQTileBytes + kQBoxBytes, &tm_q, 64, head, row + w * kHalfQ, bar);
            }
          }
        }
        __syncwarp();
        if (!ended) ok = publish();
      }
      if (!plan.prefix_mode && lane < 2) work.seg[2 * me + lane] = lane ? seg1 : seg0;
      if (!ok && lane == 0 && loads) {   // a tile in flight lands before the CTA ends
        volatile int never = 0;
        mbar_wait_bounded(reinterpret_cast<uint64_t*>(smem + kQFull), (loads - 1) & 1, &never);
      }
    } else if (warp == kLoadWarp) {
      // ========================== K and V of the units =======================
      const uint64_t policy_once = l2_policy_evict_first(), policy_again = l2_policy_evict_normal();
      const int beyond = static_cast<int>(plan.n_slots) * (kNumKVHeads * kChunkTokens);   // reads as zeros
      unsigned it = 0;
      bool ok = wait(kReady, 0);
      for (unsigned k = 0; ok; ++k) {
        ok = seg_get(k);
        if (!ok) break;
        const Seg& s = segs[k % kAhead];
        const int units = s.units, flags = s.flags, j0 = s.j0, first = s.first, low = s.low, g = s.g;
        const int32_t* const table = s.table;
        const int64_t ident = s.ident;
        seg_done(k);
        if (units == 0) break;
        // Another tile of the list reads the same chunks: they stay in L2.
        const uint64_t policy = (flags & kSegAgain) ? policy_again : policy_once;
        int row = 0;
        for (int i = 0; i < units; ++i, ++it) {
          if ((i & 31) == 0) {   // the rows of 32 units at a time, a lane each
            row = beyond;
            if (!(flags & kSegEmpty) && i + lane < units) {
              const int j = j0 + i + lane, c = j < first ? j : low + j - first;
              const int64_t slot = table ? ld_dep(table + c) : ident + c;
              if (slot >= 0 && slot < plan.n_slots)
                row = (static_cast<int>(slot) * kNumKVHeads + g) * kChunkTokens;
              else
                set_status(status, LSA_DEV_ERR_BAD_SLOT);
            }
          }
          const int y = __shfl_sync(0xffffffffu, row, i & 31);
          const int st = it % kStages;
          if (it >= kStages) ok = wait(kEmpty + 8 * st, (it / kStages - 1) & 1);
          if (!ok) break;
          if (lane == 0) {
            const uint32_t dst = sm + st * kStageBytes, bar = sm + kFull + 8 * st;
            bar_expect(bar, kStageBytes);
            load_box(dst, &tm_k, 0, y, bar, policy);
            load_box(dst + kBoxBytes, &tm_k, 64, y, bar, policy);
            load_box(dst + 2 * kBoxBytes, &tm_v, 0, y, bar, policy);
            load_box(dst + 3 * kBoxBytes, &tm_v, 64, y, bar, policy);
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) {   // copies in flight land before the CTA ends
        volatile int never = 0;
        for (unsigned i = it > kStages ? it - kStages : 0; i < it; ++i)
          mbar_wait_bounded(reinterpret_cast<uint64_t*>(smem + kFull) + i % kStages, (i / kStages) & 1, &never);
      }
    } else {
      // =============================== products ==============================
      // A warp for each softmax warpgroup: the issue of one's products, and its
      // waits, run beside the other's.  The whole warp walks the segments (its
      // values stay uniform) and one lane issues.
      const int w = warp - kMmaWarp;
      const uint32_t leader = elect_one() ? 1u : 0u;
      const uint32_t k_lo0 = desc_lo_kmajor(sm), v_lo0 = desc_lo_v(sm + 2 * kBoxBytes), q_lo0 = desc_lo_kmajor(sm + kQAt);
      const uint32_t o_acc = tmem + kOCol0 + w * kHeadDim, s_col0 = tmem + 2 * w * kSCols;
      const int s_bar = kSFull + 16 * w, p_bar = kPFull + 16 * w, o_bar = kODone + 16 * w;
      unsigned it = 0, job = 0;   // units, and units of this warpgroup so far
      bool ok = true;
      for (unsigned k = 0; ok; ++k) {
        ok = seg_get(k);
        if (!ok) break;
        const int n = segs[k % kAhead].units;
        const bool wide = segs[k % kAhead].flags & kSegWide;
        seg_done(k);
        if (n == 0) break;
        const int mine = wide ? n : (n + 1 - w) >> 1;   // units of this warpgroup: all, or every other one
        const unsigned step = wide ? 1 : 2, at0 = it + (wide ? 0 : w);
        const uint32_t q_lo = q_lo0 + (wide ? w * (kQTileBytes >> 4) : 0);
        ok = wait(kQFull, k & 1);
        if (ok && !mine && lane == 0) bar_arrive(sm + kQEmpty);
        // Scores run up to two units (both buffers) before the products, as far
        // as units have arrived: waiting for one that has not would hold back the
        // product that frees a stage.
        int next = 0;
        for (int i = 0; ok && i < mine; ++i) {
          for (; next < min(mine, i + 2); ++next) {
            const unsigned at = at0 + next * step, st = at % kStages, x = job + next, buf = x & 1;
            if (next > i) {
              if (!__all_sync(0xffffffffu, bar_try(sm + kFull + 8 * st, (at / kStages) & 1))) break;
            } else {
              ok = wait(kFull + 8 * st, (at / kStages) & 1);
            }
            if (ok && x >= 2) ok = wait(o_bar + 8 * buf, ((x - 2) >> 1) & 1);   // the buffer's probabilities are read
            if (!ok) break;
            tcgen05_fence_after();
            const uint32_t k_lo = k_lo0 + st * (kStageBytes >> 4), d = s_col0 + buf * kSCols;
#pragma unroll
            for (int x8 = 0; x8 < 8; ++x8)
              mma_ss(leader, d, q_lo + (x8 >> 2) * (kQBoxBytes >> 4) + (x8 & 3) * 2,
                     k_lo + (x8 >> 2) * (kBoxBytes >> 4) + (x8 & 3) * 2, kIdescS, x8 > 0);
            mma_commit(leader, sm + s_bar + 8 * buf);
            if (next == mine - 1) mma_commit(leader, sm + kQEmpty);
          }
          if (!ok) break;
          const unsigned at = at0 + i * step, st = at % kStages, x = job + i, buf = x & 1;
          ok = wait(p_bar + 8 * buf, (x >> 1) & 1);
          if (!ok) break;
          tcgen05_fence_after();
          const uint32_t v_lo = v_lo0 + st * (kStageBytes >> 4), a = s_col0 + buf * kSCols;
#pragma unroll
          for (int x4 = 0; x4 < 4; ++x4)
            mma_ts(leader, o_acc, a + 8 * x4, v_lo + x4 * (2048 >> 4), kIdescO, x4 > 0 || i > 0);
          mma_commit(leader, sm + o_bar + 8 * buf);
          mma_commit(leader, sm + kEmpty + 8 * st);
          if (!wide) mma_commit(leader, sm + kEmpty + 8 * st);
        }
        job += mine;
        it += n;
      }
      mma_commit(leader, sm + kDrain + 8 * w);   // every product has ended before TMEM is given back
      volatile int never = 0;
      mbar_wait_bounded(reinterpret_cast<uint64_t*>(smem + kDrain) + w, 0, &never);
    }
  } else {
    // ================================= softmax ================================
    more_registers<kSoftmaxRegs>();
    const int w = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;                    // row of the tile
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_col0 = tmem + 2 * w * kSCols + lanes, o_mine = tmem + kOCol0 + w * kHeadDim + lanes;
    const int s_bar = kSFull + 16 * w, p_bar = kPFull + 16 * w, o_bar = kODone + 16 * w;
    const uint64_t scale2 = pack2(scale_log2, scale_log2);
    unsigned job0 = 0, job1 = 0, it = 0, joins = 0;
    bool ok = true;
    // Both warpgroups.
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) bar_arrive(sm + kMeet);
      return wait(kMeet, joins++ & 1);
    };
    for (unsigned k = 0; ok; ++k) {
      ok = seg_get(k);
      if (!ok) break;
      const Seg& sg = segs[k % kAhead];
      const int n = sg.units, j0 = sg.j0, f0 = sg.f0 - j0, f1 = sg.f1 - j0, f2 = sg.f2 - j0;
      if (n == 0) break;
      const bool wide = sg.flags & kSegWide;
      const int rows = kGroup * (wide ? (w == 0 ? kHalfQ : sg.cnt - kHalfQ) : sg.cnt);   // of this warpgroup
      const bool active = wq * 32 < rows;            // the warp has rows
      float m = -INFINITY, l = 0.f;
      const unsigned job_first = w ? job1 : job0;
      unsigned job = job_first;
      for (int i = wide ? 0 : w; i < n; i += wide ? 1 : 2, ++job) {
        const unsigned buf = job & 1;
        uint64_t see = ~0ull;                        // tokens of the unit that this row sees
        const bool edge = !(i < f0 || (i >= f1 && i <= f2));
        ok = wait(s_bar + 8 * buf, (job >> 1) & 1);
        if (!ok) break;
        tcgen05_fence_after();
        if (edge) {
          uint64_t any;                              // tokens that some query of the tile sees
          const int j = j0 + i, kb = (j < sg.first ? j : sg.low + j - sg.first) * kChunkTokens;
          if (sg.flags & kSegEmpty) {
            any = see = 0;
          } else if (plan.prefix_mode) {
            any = see = lowest(sg.len - kb);
          } else {
            const int pos = sg.p0 + (wide ? w * kHalfQ : 0) + (r >> 3) - kb;   // of the row's query, in the unit
            any = lowest(sg.p0 + sg.cnt - kb) & (~lowest(sg.p0 - plan.window + 1 - kb) | lowest(plan.sinks - kb));
            see = lowest(pos + 1) & (~lowest(pos - plan.window + 1) | lowest(plan.sinks - kb));
          }
          if (any != ~0ull) {
            // Unseen rows of V become zeros (their probabilities are zero, what
            // the page holds there may not be finite).  Both warpgroups of a wide
            // tile write the same zeros.
            const unsigned at = it + i, st = at % kStages;
            ok = wait(kFull + 8 * st, (at / kStages) & 1);
            if (!ok) break;
            uint8_t* vs = smem + st * kStageBytes + 2 * kBoxBytes;
            for (int x = wq * 32 + lane; x < kChunkTokens * 16; x += 128) {
              const int row = x >> 4;
              if (!((any >> row) & 1))
                *reinterpret_cast<uint4*>(vs + ((x >> 3) & 1) * kBoxBytes + row * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
        }
        if (active) {
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
          const bool raise = !(top <= m + kRaise) && r < rows;   // a row's first score that is not masked always does
          if (__any_sync(0xffffffffu, raise)) {
            const float m_new = raise ? top : m;
            const float f = raise ? fast_exp2(m - m_new) : 1.f;
            m = m_new;
            l *= f;
            if (job != job_first) {                  // the accumulator of earlier units follows
              ok = wait(o_bar + 8 * (buf ^ 1), ((job - 1) >> 1) & 1);
              if (!ok) break;
              tcgen05_fence_after();
#pragma unroll 1
              for (int c = 0; c < kHeadDim; c += 32) {
                float o[32];
                tmem_ld32(o_mine + c, o);
                tmem_wait_ld(o, 32);
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] *= f;
                tmem_st32(o_mine + c, o);
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
            // One rounding of the probabilities to bf16, half a step (2^-9) at
            // most: the output is rounded to the same type.
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

      // ---- the end of a segment: the tile's output, or this CTA's partial ----
      const unsigned n0 = wide ? n : (n + 1) >> 1, n1 = wide ? n : n >> 1;
      const unsigned last0 = job0 + n0 - 1, last1 = job1 + n1 - 1;
      float* const ml = reinterpret_cast<float*>(smem + kMlAt);   // [2 warpgroups][m, l][128 rows]
      if (!wide) {
        ml[2 * w * 128 + r] = m;
        ml[(2 * w + 1) * 128 + r] = l;
        ok = meet();   // both have their last scores: the waits below name each barrier's next phase
      }
      // The last product of a warpgroup (its commit follows all earlier ones).
      if (ok && (!wide || w == 0)) ok = wait(kODone + 8 * (last0 & 1), (last0 >> 1) & 1);
      if (ok && (wide ? w == 1 : n1 > 0)) ok = wait(kODone + 16 + 8 * (last1 & 1), (last1 >> 1) & 1);
      if (!ok) break;
      tcgen05_fence_after();
      float part0 = 1.f, part1 = 0.f;
      if (!wide) {
        const float m0 = ml[r], l0 = ml[128 + r], m1 = ml[256 + r], l1 = ml[384 + r];
        m = fmaxf(m0, m1);
        const float ref = m == -INFINITY ? 0.f : m;
        part0 = fast_exp2(m0 - ref);
        part1 = fast_exp2(m1 - ref);
        l = l0 * part0 + l1 * part1;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      part0 *= inv;
      part1 *= inv;
      // Where the rows go: 128 bytes of a row per 8 lanes.  A thread holds a row,
      // so the rows turn in the warp's 4 KiB of shared memory, 16-byte piece x of
      // row y at place x ^ (y % 8) (no bank conflicts either way).
      if (active) {
        const bool whole = sg.flags & kSegWhole, final = whole && !plan.prefix_mode;
        const int q_first = (wide ? w * kHalfQ : 0) + wq * 4;   // the warp's first query in the tile
        // Output rows: (query, head); a record's: the same, a tile at a time.
        const int64_t out_row = (static_cast<int64_t>(sg.row) + q_first) * kNumQHeads + sg.head;
        int64_t rec = out_row;
        int q_rows = kNumQHeads;                                // rows from a query to the next
        if (plan.prefix_mode && whole) {
          rec += (sg.flags & kSegGroup) ? 0 : static_cast<int64_t>(kNumQHeads) * plan.B;
        } else if (!final) {
          rec = (plan.prefix_mode ? 2ll * kNumQHeads * plan.B : 0) + (2ll * blockIdx.x + (k > 0)) * work.rows_cap +
                q_first * kGroup;
          q_rows = kGroup;
        }
        uint8_t* const mine = smem + kTurnAt + warp * kTurnBytes;
        uint8_t* const row_at = mine + lane * 128;
        // fp32 records go 32 columns at a time, bf16 outputs 64.
        const int c_lo = wide ? 0 : 64 * w, c_hi = wide ? kHeadDim : 64 * w + 64;
        uint8_t* to = final ? reinterpret_cast<uint8_t*>(out) + (out_row * kHeadDim + c_lo) * 2
                            : reinterpret_cast<uint8_t*>(work.o + rec * kHeadDim + c_lo);
        const int row_bytes = final ? 2 * kHeadDim : 4 * kHeadDim;
#pragma unroll 1
        for (int c = c_lo; c < c_hi; c += 32) {
          float o[32];
          tmem_ld32((wide ? o_mine : tmem + kOCol0 + lanes) + c, o);
          if (!wide && n1) {
            float o2[32];
            tmem_ld32(tmem + kOCol0 + kHeadDim + lanes + c, o2);
            tmem_wait_ld(o, 32);
            tmem_wait_ld(o2, 32);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = fmaf(o2[x], part1, o[x] * part0);
          } else {
            tmem_wait_ld(o, 32);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] *= part0;
          }
          if (final) {
            const int z = (c >> 3) & 4;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              *reinterpret_cast<uint4*>(row_at + (((z + x) ^ (lane & 7)) << 4)) =
                  make_uint4(pack_bf16(o[8 * x], o[8 * x + 1]), pack_bf16(o[8 * x + 2], o[8 * x + 3]),
                             pack_bf16(o[8 * x + 4], o[8 * x + 5]), pack_bf16(o[8 * x + 6], o[8 * x + 7]));
            if (!z) continue;
          } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              *reinterpret_cast<float4*>(row_at + ((x ^ (lane & 7)) << 4)) =
                  make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int y = 4 * x + (lane >> 3);   // row of the warp: query y / 8, head y % 8
            if (wq * 32 + y < rows)
              *reinterpret_cast<uint4*>(to + ((y >> 3) * q_rows + (y & 7)) * row_bytes + (lane & 7) * 16) =
                  *reinterpret_cast<const uint4*>(mine + y * 128 + (((lane & 7) ^ (y & 7)) << 4));
          }
          __syncwarp();
          to += 128;
        }
        if (!final && r < rows && (wide || w == 0))
          work.lse[rec + (lane >> 3) * q_rows + (lane & 7)] = l == 0.f ? -INFINITY : m + __log2f(l);
      }
      tcgen05_fence_before();
      // In a narrow tile each warpgroup reads the other's accumulator: neither
      // lets the next segment's products start before both have.
      if (!wide) ok = meet();
      seg_done(k);
      job0 += n0;
      job1 += n1;
      it += n;
    }
  }
  __syncwarp();
  tcgen05_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tcgen05_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- folding the partials -----------------------------------------------------
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;

// The partials of one row, joined in their order: `row(i)` for i < n.  The loads
// of 8 partials are issued together.
struct Fold {
  float m = -INFINITY, den = 0.f;
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  template <typename Row>
  __device__ void add(const Work& w, int n, int lane, Row row) {
    constexpr int kBatch = 8;
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      float lse[kBatch];
      uint4 raw[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        lse[i] = -INFINITY;
        if (i0 + i < n) {
          const int64_t at = row(i0 + i);
          lse[i] = ld_dep(w.lse + at);
          raw[i] = ld_dep(reinterpret_cast<const uint4*>(w.o + at * kHeadDim) + lane);
        }
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) top = fmaxf(top, lse[i]);
      const float ref = top == -INFINITY ? 0.f : top;
      const float f = fast_exp2(m - ref);
      m = top;
      den *= f;
      r.x *= f; r.y *= f; r.z *= f; r.w *= f;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (i0 + i < n) {
          const float wt = fast_exp2(lse[i] - ref);
          den += wt;
          r.x = fmaf(wt, __uint_as_float(raw[i].x), r.x);
          r.y = fmaf(wt, __uint_as_float(raw[i].y), r.y);
          r.z = fmaf(wt, __uint_as_float(raw[i].z), r.z);
          r.w = fmaf(wt, __uint_as_float(raw[i].w), r.w);
        }
      }
    }
  }
  __device__ void store(__nv_bfloat16* out, int64_t row, int lane) const {   // row: query * 64 + head
    const float id = den == 0.f ? 0.f : 1.f / den;
    *reinterpret_cast<uint2*>(out + row * kHeadDim + 4 * lane) =
        make_uint2(pack_bf16(r.x * id, r.y * id), pack_bf16(r.z * id, r.w * id));
  }
};

// Window mode: CTA c looks at the tiles that attention CTA c began or ended
// with; the rows of a split one are shared out over the CTAs it was split over.
__global__ void __launch_bounds__(kMergeThreads) window_merge_kernel(const Work work, __nv_bfloat16* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  const uint4 seg[2] = {ld_dep(reinterpret_cast<const uint4*>(work.seg + 2 * c)),
                        ld_dep(reinterpret_cast<const uint4*>(work.seg + 2 * c + 1))};
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const uint4 a = seg[side];
    if (!a.w) continue;
    const int lo = a.z & 0xffff, n = static_cast<int>(a.z >> 16) - lo + 1, rows = kGroup * static_cast<int>(a.y >> 8);
    for (int r = c - lo + n * warp; r < rows; r += n * kMergeWarps) {
      Fold f;
      f.add(work, n, lane, [&](int i) {
        return static_cast<int64_t>(i == 0 ? static_cast<int>(a.w) - 1 : 2 * (lo + i)) * work.rows_cap + r;
      });
      f.store(out, (static_cast<int64_t>(a.x) + (r >> 3)) * kNumQHeads + (a.y & 0xff) * kGroup + (r & 7), lane);
    }
  }
}

// Prefix mode: a CTA per (sequence, KV head), a warp per query head: the
// partials of its group's tile, then those of its own tokens.
__global__ void __launch_bounds__(kMergeThreads) prefix_merge_kernel(const Work work, int B, __nv_bfloat16* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x, pairs = B * kNumKVHeads;   // (sequence, KV head)
  const int ok = ld_dep(work.ok);
  int ends[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ends[i] = ld_dep(work.ends + i * static_cast<int64_t>(pairs) + pair);
  if (!ok) return;
  const int64_t row = static_cast<int64_t>(pair) * kGroup + h;   // query * 64 + head
  Fold f;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    const int first = ends[2 * part], last = ends[2 * part + 1];
    if (first == kNone) continue;
    const int c0 = first & 0xff;
    const int64_t slots = 2ll * kNumQHeads * B + ((first >> kEndPlace) & 0xff) * kGroup + h;
    const bool whole = first & kEndWhole;
    f.add(work, whole ? 1 : last - c0 + 1, lane, [&](int i) {
      return whole ? row + part * static_cast<int64_t>(kNumQHeads) * B
                   : slots + (2ll * (c0 + i) + (i == 0 && (first & kEndSlot) ? 1 : 0)) * work.rows_cap;
    });
  }
  f.store(out, row, lane);
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// Rows of a record: a tile's queries x 8 heads.
int rows_cap(int queries) { return kGroup * (queries < kWideQ ? queries : kWideQ); }
// The workspace's parts: rows and their log-sum-exps, the segments or the ends, the verdict.
size_t layout(Work* w, void* at, int64_t place_rows, int queries, int64_t pairs) {
  const int64_t rows = place_rows + 2ll * kMaxCtas * rows_cap(queries);
  const size_t o = static_cast<size_t>(rows) * kHeadDim * 4, lse = round16(rows * 4);
  const size_t seg = 2 * kMaxCtas * sizeof(int4), ends = round16(4 * pairs * 4), ok = 16;
  if (w) {
    char* p = static_cast<char*>(at);
    w->o = reinterpret_cast<float*>(p);
    w->lse = reinterpret_cast<float*>(p += o);
    w->seg = reinterpret_cast<int4*>(p += lse);
    w->ends = reinterpret_cast<int*>(p += seg);
    w->ok = reinterpret_cast<int*>(p += ends);
    w->rows_cap = rows_cap(queries);
  }
  return o + lse + seg + ends + ok;
}
size_t window_layout(Work* w, void* at, int max_q) { return layout(w, at, 0, max_q, 0); }
size_t prefix_layout(Work* w, void* at, int B) {
  return layout(w, at, 2ll * kNumQHeads * B, B, static_cast<int64_t>(B) * kNumKVHeads);
}

std::mutex g_mu;
bool g_attr_set[64] = {};

int encode_pool(CUtensorMap* map, const void* base, int64_t n_slots) {
  const cuuint64_t dims[2] = {kHeadDim, static_cast<cuuint64_t>(n_slots) * kNumKVHeads * kChunkTokens};
  const cuuint64_t strides[1] = {kHeadDim * 2};
  const cuuint32_t box[2] = {64, kChunkTokens}, estr[2] = {1, 1};
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
          float scale, const void* out) {
  if (!q || !k_pool || !v_pool || !len || !out || n_slots <= 0 || B <= 0 || max_chunks <= 0) return LSA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return LSA_ERR_INVALID_ARG;
  if (B > LSA_MAX_BATCH) return LSA_ERR_UNSUPPORTED_SHAPE;
  // Positions and TMA rows (n_slots * 512) are 32-bit.
  if (max_chunks > (1 << 23) || n_slots >= (int64_t{1} << 22)) return LSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return LSA_ERR_MISALIGNED;
  return LSA_OK;
}

int launch(const Plan& plan, const Work& work, const void* q, const void* k_pool, const void* v_pool, float scale, void* out,
           int64_t max_units, void* stream) {
  const int sms = device_sm_count();
  if (sms <= 0 || !tensor_map_encoder()) return LSA_ERR_NO_DEVICE;
  int dev = 0;
  cudaGetDevice(&dev);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (dev < 64 && !g_attr_set[dev]) {
      if (cudaFuncSetAttribute(pool_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess) {
        cudaGetLastError();
        return LSA_ERR_CUDA;
      }
      g_attr_set[dev] = true;
    }
  }
  CUtensorMap tm_k, tm_v, tm_q, tm_q1;
  int st = encode_pool(&tm_k, k_pool, plan.n_slots);
  if (st == LSA_OK) st = encode_pool(&tm_v, v_pool, plan.n_slots);
  if (st == LSA_OK) st = encode_q(&tm_q, q, plan.rows, kHalfQ);
  if (st == LSA_OK) st = encode_q(&tm_q1, q, plan.rows, 1);
  if (st != LSA_OK) return st;
  const int most = sms < kMaxCtas ? sms : kMaxCtas;
  const int64_t want = (max_units + kMinUnitsPerCta - 1) / kMinUnitsPerCta;
  const int grid = want < most ? static_cast<int>(want) : most;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  launch_pdl(true, pool_attn_kernel, dim3(grid), dim3(kThreads), kSmemBytes, s, tm_k, tm_v, tm_q, tm_q1, plan, work,
             scale * 1.4426950408889634f, o, lsa_device_status_ptr());
  if (plan.prefix_mode)
    launch_pdl(true, prefix_merge_kernel, dim3(plan.B * kNumKVHeads), dim3(kMergeThreads), 0, s, work, plan.B, o);
  else
    launch_pdl(true, window_merge_kernel, dim3(grid), dim3(kMergeThreads), 0, s, work, o);
  return launch_status();
}

}  // namespace pool
}  // namespace lsa

extern "C" {

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
  const int st = pool::check(q, k_pool, v_pool, n_slots, seq_len, B, max_chunks, softmax_scale, out);
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
  const int64_t units = kNumKVHeads * (T / pool::kWideQ + B) * (seen < max_chunks ? seen : max_chunks);
  return pool::launch(plan, work, q, k_pool, v_pool, softmax_scale, out, units, stream);
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
  const int st = pool::check(q, k_pool, v_pool, n_slots, suffix_len, B, max_chunks, softmax_scale, out);
  if (st != LSA_OK) return st;
  if (max_prefix_chunks > (1 << 23)) return LSA_ERR_UNSUPPORTED_SHAPE;
  if (!workspace || workspace_bytes < pool::prefix_layout(nullptr, nullptr, B)) return LSA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LSA_ERR_MISALIGNED;
  pool::Plan plan = {};
  plan.prefix_mode = 1;
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
  plan.n_slots = n_slots;
  pool::Work work;
  pool::prefix_layout(&work, workspace, B);
  const int64_t tiles = n_groups > 0 ? B / pool::kWideQ + n_groups : 0;
  const int64_t units = kNumKVHeads * (tiles * max_prefix_chunks + static_cast<int64_t>(B) * max_chunks);
  return pool::launch(plan, work, q, k_pool, v_pool, softmax_scale, out, units, stream);
}

}  // extern "C"
