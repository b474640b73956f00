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
// Roles of a CTA (11 warps):
//   warps 0-3, 4-7  two softmax warpgroups, a thread per row: the scores of a
//                   unit come from TMEM, the probabilities go back to TMEM in
//                   the scores' place as bf16.  The running maximum is only
//                   raised when it grows by more than 2^8 (the sums stay
//                   exact, the accumulator is rescaled rarely);
//   warp 8          issues the tcgen05.mma: S = Q K^T (128 x 64 x 128), and
//                   O += P V (128 x 128 x 64) with P read from TMEM;
//   warp 9          streams the units with TMA into a ring of 5 stages;
//   warp 10         loads the query tile of the next segment.
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
constexpr int kMmaWarp = 8, kLoadWarp = 9, kQueryWarp = 10;
constexpr int kThreads = 11 * 32;
constexpr int kStages = 5;
constexpr int kBoxBytes = 8192;              // 64 tokens x 64 dims
constexpr int kStageBytes = 4 * kBoxBytes;   // K dims 0-63, 64-127, V dims 0-63, 64-127
constexpr int kQBoxBytes = 16384;            // 128 rows x 64 dims
constexpr int kQTileBytes = 2 * kQBoxBytes;
constexpr int kSmemBytes = kStages * kStageBytes + 2 * kQTileBytes + 2 * 2 * 128 * 4 + 256;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
constexpr int kMaxCtas = LSA_POOL_ATTN_MAX_CTAS;
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

// Partials: `rows_cap` rows per record.
struct Work {
  float* o;          // [record rows][128]
  float* lse;        // [record rows]
  int64_t* base;     // prefix mode: first unit of each list, then the total; window mode: the total
  int4* seg;         // window mode: [2 * kMaxCtas][2] first and last segment of each CTA
  int* ok;           // [1]: the offsets were valid
  int rows_cap;
};

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

struct Partition {
  int64_t base, rem;
  __device__ Partition(int64_t total, int G) : base(total / G), rem(total % G) {}
  __device__ int64_t start(int c) const { return c * base + (c < rem ? c : rem); }
  __device__ int cta_of(int64_t u) const {
    const int64_t big = rem * (base + 1);
    return static_cast<int>(u < big ? u / (base + 1) : rem + (u - big) / base);
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
  // At unit r of list v.
  __device__ void start(const Plan& p, int list, int64_t r) {
    v = list;
    set_list(p);
    const int64_t per_head = units_before(p, s, tiles);
    g = static_cast<int>(r / per_head);
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

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// Shared-memory descriptor of V as the N x K operand (N = dims, K = tokens),
// stored token by token (N contiguous) with the 128-byte swizzle: 64-dim boxes
// 8192 bytes apart (leading offset), 8-token groups 1024 bytes apart (stride).
__device__ __forceinline__ uint64_t umma_desc_v(uint32_t saddr) {
  return (static_cast<uint64_t>((saddr >> 4) & 0x3FFFu)) | (static_cast<uint64_t>(kBoxBytes >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (static_cast<uint64_t>(1u) << 46) |
         (static_cast<uint64_t>(2u) << 61);
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

__global__ void __launch_bounds__(kThreads, 1)
pool_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q1, const Plan plan,
                 const Work work, float scale_log2, __nv_bfloat16* __restrict__ out, unsigned* status) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  griddep_launch_dependents();

  uint8_t* q_smem = smem + kStages * kStageBytes;
  float* ml = reinterpret_cast<float*>(q_smem + 2 * kQTileBytes);   // [2 warpgroups][m, l][128 rows]
  uint64_t* full = reinterpret_cast<uint64_t*>(ml + 2 * 2 * 128);
  uint64_t* empty = full + kStages;
  uint64_t* s_full = empty + kStages;   // [2][2]
  uint64_t* p_full = s_full + 4;        // [2][2]
  uint64_t* o_done = p_full + 4;        // [2][2], by the score buffer that the product read
  uint64_t* q_full = o_done + 4;
  uint64_t* q_empty = q_full + 1;
  uint64_t* drain = q_empty + 1;
  uint64_t* join = drain + 1;           // all 8 softmax warps
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(join + 1);
  int* flags = reinterpret_cast<int*>(tmem_ptr + 1);   // [0] abort

  // ---- the unit list: validity, total, and the place where this CTA starts --
  // (The scratch of the scan lies in the ring, which is empty until the roles start.)
  int64_t* scan = reinterpret_cast<int64_t*>(smem);
  const int V = plan.lists();
  const int per = (V + kThreads - 1) / kThreads;
  const int v_lo = min(V, tid * per), v_hi = min(V, v_lo + per);
  int bad = (smem_u32(smem) & 1023u) ? 1 : 0;
  int64_t mine = 0;
  const int n_cu = plan.prefix_mode ? plan.groups : plan.B;
  if (tid == 0 && n_cu > 0) {
    bad |= ld_dep(plan.cu) != 0;
    const int last = ld_dep(plan.cu + n_cu);
    bad |= last < 0 || last > plan.rows;
  }
  for (int v = v_lo; v < v_hi; ++v) {
    const List s = load_list(plan, v);
    if (s.len < 0 && blockIdx.x == 0) set_status(status, LSA_DEV_ERR_BAD_COUNT);
    bad |= s.nq < 0 || (!plan.prefix_mode && s.nq > plan.max_q);
    if (s.nq > 0) mine += kNumKVHeads * units_before(plan, s, tiles_of(s));
  }
  int64_t total;
  bad = __syncthreads_or(bad);
  const int64_t before = block_scan<kThreads / 32>(bad ? 0 : mine, scan, &total);
  const Partition part(total, gridDim.x);
  const int64_t u0 = part.start(blockIdx.x), u1 = part.start(blockIdx.x + 1);
  if (blockIdx.x == 0 && tid == 0) {
    if (bad) set_status(status, LSA_DEV_ERR_CAPACITY);
    *work.ok = bad ? 0 : 1;
    work.base[plan.prefix_mode ? V : 0] = total;
  }
  if (!bad) {
    int64_t at = before;
    const bool here = before <= u0 && u0 < before + mine && u0 < u1;
    const bool write = plan.prefix_mode && blockIdx.x == 0;
    if (here || write) {
      for (int v = v_lo; v < v_hi; ++v) {
        const List s = load_list(plan, v);
        const int64_t n = s.nq > 0 ? kNumKVHeads * units_before(plan, s, tiles_of(s)) : 0;
        if (write) work.base[v] = at;
        if (here && at <= u0 && u0 < at + n) {
          scan[32] = v;
          scan[33] = at;
        }
        at += n;
      }
    }
  }
  if (bad || u0 >= u1) {
    if (!plan.prefix_mode && tid < 4) work.seg[blockIdx.x * 4 + tid] = make_int4(0, 0, 0, 0);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);   // one arrival per warp of the warpgroup
      mbar_init(&o_done[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    mbar_init(join, kSoftmaxThreads / 32);
    flags[0] = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_ptr, 512);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *tmem_ptr;
  volatile int* abort_flag = flags;
  Cursor cur;
  cur.start(plan, static_cast<int>(scan[32]), u0 - scan[33]);
  fence_proxy_async_smem();   // the scan's scratch was written here; TMA writes it next
  __syncthreads();

  auto give_up = [&]() {
    if (!*abort_flag) set_status(status, LSA_DEV_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == kLoadWarp) {
    // ============================ K and V of the units =======================
    uint64_t policy_once = 0, policy_again = 0;
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      policy_once = l2_policy_evict_first();
      policy_again = l2_policy_evict_normal();
    }
    const int beyond = static_cast<int>(plan.n_slots) * (kNumKVHeads * kChunkTokens);   // reads as zeros
    int64_t it = 0;
    bool ok = true;
    for (int64_t u = u0; ok;) {
      const int j1 = static_cast<int>(min(static_cast<int64_t>(cur.n), cur.j + (u1 - u)));
      // Another tile of the list reads the same chunks: they stay in L2.
      const uint64_t policy = cur.tiles > 1 ? policy_again : policy_once;
      int row = 0;
      for (int j = cur.j; j < j1; ++j, ++it) {
        if (((j - cur.j) & 31) == 0) {   // the rows of 32 units at a time, a lane each
          row = beyond;
          if (!cur.empty && j + lane < j1) {
            const int c = cur.chunk(j + lane);
            const int64_t slot = cur.s.table ? ld_dep(cur.s.table + c) : cur.s.ident + c;
            if (slot >= 0 && slot < plan.n_slots)
              row = (static_cast<int>(slot) * kNumKVHeads + cur.g) * kChunkTokens;
            else
              set_status(status, LSA_DEV_ERR_BAD_SLOT);
          }
        }
        const int y = __shfl_sync(0xffffffffu, row, (j - cur.j) & 31);
        const int st = static_cast<int>(it % kStages);
        int good = 1;
        if (lane == 0) {
          if (it >= kStages) good = mbar_wait_bounded(&empty[st], static_cast<unsigned>((it / kStages - 1) & 1), abort_flag);
          if (good) {
            uint8_t* dst = smem + st * kStageBytes;
            mbar_arrive_expect_tx(&full[st], kStageBytes);
            tma_load_2d(dst, &tm_k, 0, y, &full[st], policy);
            tma_load_2d(dst + kBoxBytes, &tm_k, 64, y, &full[st], policy);
            tma_load_2d(dst + 2 * kBoxBytes, &tm_v, 0, y, &full[st], policy);
            tma_load_2d(dst + 3 * kBoxBytes, &tm_v, 64, y, &full[st], policy);
          } else {
            give_up();
          }
        }
        ok = __shfl_sync(0xffffffffu, good, 0) != 0;
        if (!ok) break;
      }
      u += j1 - cur.j;
      if (u >= u1) break;
      if (ok) cur.next(plan);
    }
    if (lane == 0 && *abort_flag) {   // copies in flight land before the CTA ends
      int never = 0;
      for (int64_t i = it > kStages ? it - kStages : 0; i < it; ++i)
        mbar_wait_bounded(&full[i % kStages], static_cast<unsigned>((i / kStages) & 1), &never);
    }
  } else if (warp == kQueryWarp) {
    // ================================ query tiles =============================
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_q1);
      unsigned segs = 0;
      for (int64_t u = u0;;) {
        const int j1 = static_cast<int>(min(static_cast<int64_t>(cur.n), cur.j + (u1 - u)));
        if (segs && !mbar_wait_bounded(q_empty, (segs - 1) & 1, abort_flag)) {
          give_up();
          break;
        }
        const int row = cur.s.q0 + cur.t * kWideQ, head = cur.g * kGroup;
        if (cur.cnt == 1) {   // 8 rows; what the other rows of the tile hold is not read back
          mbar_arrive_expect_tx(q_full, 2 * kGroup * 128);
          tma_load_3d(q_smem, &tm_q1, 0, head, row, q_full);
          tma_load_3d(q_smem + kQBoxBytes, &tm_q1, 64, head, row, q_full);
        } else {
          const int halves = cur.wide() ? 2 : 1;
          mbar_arrive_expect_tx(q_full, halves * kQTileBytes);
          for (int w = 0; w < halves; ++w) {
            tma_load_3d(q_smem + w * kQTileBytes, &tm_q, 0, head, row + w * kHalfQ, q_full);
            tma_load_3d(q_smem + w * kQTileBytes + kQBoxBytes, &tm_q, 64, head, row + w * kHalfQ, q_full);
          }
        }
        ++segs;
        u += j1 - cur.j;
        if (u >= u1) break;
        cur.next(plan);
      }
      if (*abort_flag && segs) {
        int never = 0;
        mbar_wait_bounded(q_full, (segs - 1) & 1, &never);
      }
    }
  } else if (warp == kMmaWarp) {
    // ================================= products ===============================
    if (lane == 0) {
      const uint32_t ring = smem_u32(smem), q_base = smem_u32(q_smem);
      int64_t it = 0;
      unsigned jobs[2] = {0, 0};   // units each warpgroup has had
      unsigned segs = 0;
      bool ok = true;
      for (int64_t u = u0; ok;) {
        const int j1 = static_cast<int>(min(static_cast<int64_t>(cur.n), cur.j + (u1 - u)));
        const int n = j1 - cur.j;
        const bool wide = cur.wide();
        const int ahead = wide ? 2 : 4;   // both score buffers of both warpgroups
        ok = mbar_wait_bounded(q_full, segs & 1, abort_flag);
        // S of unit i, into the score buffer that O(job - 2) has read.
        auto scores = [&](int i) {
          const int st = static_cast<int>((it + i) % kStages);
          if (!mbar_wait_bounded(&full[st], static_cast<unsigned>(((it + i) / kStages) & 1), abort_flag)) return false;
          tcgen05_fence_after();
          const uint32_t kb = ring + st * kStageBytes;
          for (int w = wide ? 0 : (i & 1); w < (wide ? 2 : (i & 1) + 1); ++w) {
            const unsigned job = jobs[w] + (wide ? i : i >> 1);
            const int buf = 2 * w + (job & 1);
            if (job >= 2 && !mbar_wait_bounded(&o_done[buf], ((job - 2) >> 1) & 1, abort_flag)) return false;
            const uint32_t qa = q_base + (wide ? w * kQTileBytes : 0);
            const uint32_t d = tmem + buf * kSCols;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              umma_bf16(d, umma_desc_kmajor_sw128(qa + (k >> 2) * kQBoxBytes + (k & 3) * 32),
                        umma_desc_kmajor_sw128(kb + (k >> 2) * kBoxBytes + (k & 3) * 32), kIdescS, k > 0);
            umma_commit(&s_full[buf]);
          }
          if (i == n - 1) umma_commit(q_empty);
          return true;
        };
        for (int i = 0; ok && i < min(ahead, n); ++i) ok = scores(i);
        for (int i = 0; ok && i < n; ++i) {
          const int st = static_cast<int>((it + i) % kStages);
          const uint32_t vb = ring + st * kStageBytes + 2 * kBoxBytes;
          for (int w = wide ? 0 : (i & 1); ok && w < (wide ? 2 : (i & 1) + 1); ++w) {
            const unsigned done = wide ? i : i >> 1;
            const unsigned job = jobs[w] + done;
            const int buf = 2 * w + (job & 1);
            ok = mbar_wait_bounded(&p_full[buf], (job >> 1) & 1, abort_flag);
            if (!ok) break;
            tcgen05_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_ts(tmem + kOCol0 + w * kHeadDim, tmem + buf * kSCols + 8 * k,
                           umma_desc_v(vb + k * 2048), kIdescO, done > 0 || k > 0);
            umma_commit(&o_done[buf]);
          }
          if (!ok) break;
          umma_commit(&empty[st]);
          if (i + ahead < n) ok = scores(i + ahead);
        }
        if (!ok) break;
        jobs[0] += wide ? n : (n + 1) >> 1;
        jobs[1] += wide ? n : n >> 1;
        it += n;
        ++segs;
        u += n;
        if (u >= u1) break;
        cur.next(plan);
      }
      if (!ok) give_up();
      umma_commit(drain);   // every product has ended before TMEM is given back
      int never = 0;
      mbar_wait_bounded(drain, 0, &never);
    }
  } else {
    // ================================= softmax ================================
    const int w = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;                    // row of the tile
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t o_mine = tmem + kOCol0 + w * kHeadDim + lanes;
    unsigned jobs[2] = {0, 0};
    int64_t it = 0;
    bool ok = true;
    int seg_no = 0;
    unsigned joins = 0;
    // The same answer in every lane: the warp's collective instructions stay whole.
    auto warp_wait = [&](uint64_t* bar, unsigned parity) {
      return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag)) != 0;
    };
    // Both warpgroups, with a bounded wait.
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(join);
      return warp_wait(join, joins++ & 1);
    };
    for (int64_t u = u0; ok; ++seg_no) {
      const int j0 = cur.j;
      const int j1 = static_cast<int>(min(static_cast<int64_t>(cur.n), j0 + (u1 - u)));
      const int n = j1 - j0;
      const bool wide = cur.wide();
      const int rows = kGroup * (wide ? (w == 0 ? kHalfQ : cur.cnt - kHalfQ) : cur.cnt);   // of this warpgroup
      const bool active = wq * 32 < rows;            // the warp has rows
      const int i_q = (wide ? w * kHalfQ : 0) + (r >> 3);   // query of the tile
      const int pos = cur.p0 + i_q;
      float m = -INFINITY, l = 0.f;
      unsigned job = jobs[w];
      for (int i = wide ? 0 : w; i < n; i += wide ? 1 : 2, ++job) {
        const int buf = 2 * w + (job & 1);
        if (!warp_wait(&s_full[buf], (job >> 1) & 1)) {
          give_up();
          ok = false;
          break;
        }
        tcgen05_fence_after();
        // Rows of this unit that some query of the tile sees.
        const int kb = (cur.empty ? 0 : cur.chunk(j0 + i)) * kChunkTokens;
        const int p1 = cur.p0 + cur.cnt - 1;
        int last, low;                               // seen by all: [low, last] relative to the unit
        uint64_t any;
        bool edge;
        if (plan.prefix_mode) {
          last = cur.s.len - 1 - kb;                 // len -1 (invalid) or 0: nothing
          low = 0;
          any = lowest(last + 1);
          edge = last < 63;
        } else {
          any = cur.empty ? 0ull
                          : lowest(p1 - kb + 1) & (~lowest(cur.p0 - plan.window + 1 - kb) | lowest(plan.sinks - kb));
          edge = cur.p0 - kb < 63 || (p1 - plan.window + 1 - kb > 0 && plan.sinks - kb < 64);
          last = pos - kb;
          low = pos - plan.window + 1 - kb;
        }
        if (any != ~0ull) {
          // Unseen rows of V become zeros (their probabilities are zero, what
          // the page holds there may not be finite).  Both warpgroups of a wide
          // tile write the same zeros.
          const int64_t unit = it + i;
          const int st = static_cast<int>(unit % kStages);
          if (!warp_wait(&full[st], static_cast<unsigned>((unit / kStages) & 1))) {
            give_up();
            ok = false;
            break;
          }
          uint8_t* vs = smem + st * kStageBytes + 2 * kBoxBytes;
          for (int x = wq * 32 + lane; x < kChunkTokens * 16; x += 128) {
            const int row = x >> 4;
            if (!((any >> row) & 1))
              *reinterpret_cast<uint4*>(vs + ((x >> 3) & 1) * kBoxBytes + row * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (active) {
          const uint32_t sp = tmem + buf * kSCols + lanes;
          float s[64];
          tmem_ld32(sp, s);
          tmem_ld32(sp + 32, s + 32);
          tmem_wait_ld(s, 64);
          if (edge) {
            const uint64_t see = plan.prefix_mode || cur.empty
                                     ? any
                                     : lowest(last + 1) & (~lowest(low) | lowest(plan.sinks - kb));
            const uint32_t s0 = static_cast<uint32_t>(see), s1 = static_cast<uint32_t>(see >> 32);
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              if (!((s0 >> c) & 1)) s[c] = -INFINITY;
              if (!((s1 >> c) & 1)) s[c + 32] = -INFINITY;
            }
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale_log2;
          const bool raise = top > m + kRaise;       // the first finite score always does
          if (__any_sync(0xffffffffu, raise)) {
            const float m_new = raise ? top : m;
            const float f = raise ? fast_exp2(m - m_new) : 1.f;
            m = m_new;
            l *= f;
            if (job != jobs[w]) {                    // the accumulator of earlier units follows
              if (!warp_wait(&o_done[2 * w + ((job - 1) & 1)], ((job - 1) >> 1) & 1)) {
                give_up();
                ok = false;
              }
              tcgen05_fence_after();
#pragma unroll
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
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          float pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float a = fast_exp2(fmaf(s[2 * c], scale_log2, -ref)), b = fast_exp2(fmaf(s[2 * c + 1], scale_log2, -ref));
            sum[c & 3] += a + b;
            // One rounding of the probabilities to bf16, half a step (2^-9) at
            // most: the output is rounded to the same type.
            pk[c] = __uint_as_float(pack_bf16(a, b));
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st32(sp, pk);
          tmem_wait_st();
        }
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
        if (!ok) break;
      }
      if (!ok) break;

      // ---- the end of a segment: the tile's output, or this CTA's partial ----
      const unsigned n0 = wide ? n : (n + 1) >> 1, n1 = wide ? n : n >> 1;
      const bool whole = !plan.prefix_mode && j0 == 0 && j1 == cur.n;
      const unsigned had = w == 0 ? n0 : n1;
      const unsigned last0 = jobs[0] + n0 - 1, last1 = jobs[1] + n1 - 1;
      if (!wide) {
        ml[(2 * w + 0) * 128 + r] = had ? m : -INFINITY;
        ml[(2 * w + 1) * 128 + r] = had ? l : 0.f;
        ok = meet();   // both have their last scores: the waits below name each barrier's next phase
      }
      // The last product of a warpgroup (its commit follows all earlier ones).
      if (ok && (!wide || w == 0)) ok = warp_wait(&o_done[last0 & 1], (last0 >> 1) & 1);
      if (ok && (wide ? w == 1 : n1 > 0)) ok = warp_wait(&o_done[2 + (last1 & 1)], (last1 >> 1) & 1);
      if (!ok) {
        give_up();
        break;
      }
      tcgen05_fence_after();
      float f0 = 1.f, f1 = 0.f;
      if (!wide) {
        const float m0 = ml[r], l0 = ml[128 + r], m1 = ml[256 + r], l1 = ml[384 + r];
        m = fmaxf(m0, m1);
        const float ref = m == -INFINITY ? 0.f : m;
        f0 = fast_exp2(m0 - ref);
        f1 = fast_exp2(m1 - ref);
        l = l0 * f0 + l1 * f1;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      f0 *= inv;
      f1 *= inv;
      // Where the row goes.
      const int64_t q_row = cur.s.q0 + cur.t * kWideQ + i_q;
      const int h = r & 7;
      const bool row_here = r < rows;
      int64_t rec = 0;
      if (plan.prefix_mode) {
        const int64_t tile_row = cur.v < plan.groups
                                     ? static_cast<int64_t>(kGroup) * (8ll * cur.s.q0 + cur.g * static_cast<int64_t>(cur.s.nq) + cur.t * kWideQ)
                                     : 64ll * plan.B + 64ll * cur.s.q0 + 8 * cur.g;
        rec = tile_row + static_cast<int64_t>(blockIdx.x) * work.rows_cap;
      } else {
        rec = (2ll * blockIdx.x + (seg_no > 0)) * work.rows_cap;
      }
      rec += i_q * kGroup + h;
      if (active) {
        const uint32_t o0 = tmem + kOCol0 + lanes, o1 = o0 + kHeadDim;
        const int c_lo = wide ? 0 : 64 * w, c_hi = wide ? kHeadDim : 64 * w + 64;
        for (int c = c_lo; c < c_hi; c += 32) {
          float o[32];
          tmem_ld32((wide ? o_mine : o0) + c, o);
          tmem_wait_ld(o, 32);
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] *= f0;
          if (!wide && n1) {
            float o2[32];
            tmem_ld32(o1 + c, o2);
            tmem_wait_ld(o2, 32);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = fmaf(o2[x], f1, o[x]);
          }
          if (row_here) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(out + (q_row * kNumQHeads + cur.g * kGroup + h) * kHeadDim + c);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                dst[x] = make_uint4(pack_bf16(o[8 * x], o[8 * x + 1]), pack_bf16(o[8 * x + 2], o[8 * x + 3]),
                                    pack_bf16(o[8 * x + 4], o[8 * x + 5]), pack_bf16(o[8 * x + 6], o[8 * x + 7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(work.o + rec * kHeadDim + c);
#pragma unroll
              for (int x = 0; x < 8; ++x) dst[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
            }
          }
        }
        if (row_here && !whole && (wide || w == 0)) work.lse[rec] = l == 0.f ? -INFINITY : m + __log2f(l);
      }
      // What the merge needs of the CTA's first and last segment.
      if (!plan.prefix_mode && tid == 0) {
        const int64_t tile_u = u - j0;   // first unit of the tile
        const int4 a = make_int4(static_cast<int>(tile_u & 0xffffffff), static_cast<int>(tile_u >> 32), cur.n, cur.cnt);
        const int4 b = make_int4(cur.s.q0 + cur.t * kWideQ, cur.g, 1, 0);
        int4* dst = work.seg + blockIdx.x * 4;
        if (seg_no == 0) {
          dst[0] = a;
          dst[1] = b;
          dst[2] = dst[3] = make_int4(0, 0, 0, 0);
        } else {
          dst[2] = a;
          dst[3] = b;
        }
      }
      tcgen05_fence_before();
      // In a narrow tile each warpgroup reads the other's accumulator: neither
      // lets the next segment's products start before both have.
      if (!wide && ok) ok = meet();
      if (!ok) {
        give_up();
        break;
      }
      jobs[0] += n0;
      jobs[1] += n1;
      it += n;
      u += n;
      if (u >= u1) break;
      cur.next(plan);
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

// The records of one row, in the order of its partials: `row(i)` for i < n.
struct Fold {
  float m = -INFINITY, den = 0.f;
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  template <typename Row>
  __device__ void add(const Work& w, int n, int lane, Row row) {
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int k = min(32, n - i0);
      const float lse = lane < k ? ld_dep(w.lse + row(i0 + lane)) : -INFINITY;
      float top = lse;
#pragma unroll
      for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float m_new = fmaxf(m, top);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float f = fast_exp2(m - ref);
      const float wt = fast_exp2(lse - ref);
      den *= f;
      r.x *= f; r.y *= f; r.z *= f; r.w *= f;
      m = m_new;
#pragma unroll 4
      for (int i = 0; i < k; ++i) {
        const float wi = __shfl_sync(0xffffffffu, wt, i);
        const uint4 raw = ld_dep(reinterpret_cast<const uint4*>(w.o + row(i0 + i) * kHeadDim) + lane);
        den += wi;
        r.x = fmaf(wi, __uint_as_float(raw.x), r.x);
        r.y = fmaf(wi, __uint_as_float(raw.y), r.y);
        r.z = fmaf(wi, __uint_as_float(raw.z), r.z);
        r.w = fmaf(wi, __uint_as_float(raw.w), r.w);
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
  if (!ld_dep(work.ok)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  const Partition part(*static_cast<const volatile int64_t*>(work.base), gridDim.x);
  int64_t prev = -1;
  for (int side = 0; side < 2; ++side) {
    const uint4 a = ld_dep(reinterpret_cast<const uint4*>(work.seg + c * 4 + side * 2));
    const uint4 b = ld_dep(reinterpret_cast<const uint4*>(work.seg + c * 4 + side * 2 + 1));
    if (!b.z) continue;
    const int64_t tile = static_cast<int64_t>(a.x) | (static_cast<int64_t>(a.y) << 32);
    if (tile == prev) continue;
    prev = tile;
    const int lo = part.cta_of(tile), hi = part.cta_of(tile + a.z - 1);
    if (lo == hi) continue;
    const int n = hi - lo + 1, rows = kGroup * static_cast<int>(a.w);
    const int lo_rec = 2 * lo + (part.start(lo) == tile ? 0 : 1);   // there it may come after other tiles
    for (int r = c - lo + n * warp; r < rows; r += n * kMergeWarps) {
      Fold f;
      f.add(work, n, lane, [&](int i) {
        return static_cast<int64_t>(i == 0 ? lo_rec : 2 * (lo + i)) * work.rows_cap + r;
      });
      f.store(out, (static_cast<int64_t>(b.x) + (r >> 3)) * kNumQHeads + b.y * kGroup + (r & 7), lane);
    }
  }
}

// Prefix mode: a CTA per (sequence, KV head), a warp per query head: the
// partials of its group's tile, then those of its own tokens.
__global__ void __launch_bounds__(kMergeThreads) prefix_merge_kernel(const Plan plan, const Work work, int grid,
                                                                     __nv_bfloat16* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  if (!ld_dep(work.ok)) return;
  const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / kNumKVHeads, g = blockIdx.x % kNumKVHeads;
  const int V = plan.groups + plan.B;
  const volatile int64_t* base = work.base;
  const Partition part(base[V], grid);
  Fold f;
  if (plan.groups > 0 && b < ld_dep(plan.cu + plan.groups)) {
    int lo = 0, hi = plan.groups - 1;   // the group: the last one that starts at or before b and is not empty
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (ld_dep(plan.cu + mid) <= b) lo = mid; else hi = mid - 1;
    }
    const List s = load_list(plan, lo);
    const int i = b - s.q0, t = i / kWideQ;
    const int n = s.len > 0 ? (s.len + kChunkTokens - 1) / kChunkTokens : 1;
    const int64_t first = base[lo] + (static_cast<int64_t>(g) * tiles_of(s) + t) * n;
    const int c0 = part.cta_of(first), c1 = part.cta_of(first + n - 1);
    const int64_t row = static_cast<int64_t>(kGroup) * (8ll * s.q0 + g * static_cast<int64_t>(s.nq) + i) + h;
    f.add(work, c1 - c0 + 1, lane, [&](int x) { return row + static_cast<int64_t>(c0 + x) * work.rows_cap; });
  }
  {
    const List s = load_list(plan, plan.groups + b);
    const int n = s.len > 0 ? (s.len + kChunkTokens - 1) / kChunkTokens : 1;
    const int64_t first = base[plan.groups + b] + static_cast<int64_t>(g) * n;
    const int c0 = part.cta_of(first), c1 = part.cta_of(first + n - 1);
    const int64_t row = 64ll * plan.B + 64ll * b + kGroup * g + h;
    f.add(work, c1 - c0 + 1, lane, [&](int x) { return row + static_cast<int64_t>(c0 + x) * work.rows_cap; });
  }
  f.store(out, static_cast<int64_t>(b) * kNumQHeads + g * kGroup + h, lane);
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// The workspace's parts: records, their log-sum-exps, the first units of the
// lists, the CTAs' segments, the verdict.
size_t layout(Work* w, void* at, int64_t record_rows, int64_t lists, int rows_cap) {
  const size_t o = static_cast<size_t>(record_rows) * kHeadDim * 4, lse = round16(record_rows * 4);
  const size_t base = round16((lists + 1) * 8), seg = kMaxCtas * 4 * sizeof(int4), ok = 16;
  if (w) {
    char* p = static_cast<char*>(at);
    w->o = reinterpret_cast<float*>(p);
    w->lse = reinterpret_cast<float*>(p += o);
    w->base = reinterpret_cast<int64_t*>(p += lse);
    w->seg = reinterpret_cast<int4*>(p += base);
    w->ok = reinterpret_cast<int*>(p += seg);
    w->rows_cap = rows_cap;
  }
  return o + lse + base + seg + ok;
}
// Rows of a record: a tile's queries x 8 heads.
int rows_cap(int queries) { return kGroup * (queries < kWideQ ? queries : kWideQ); }
size_t window_layout(Work* w, void* at, int max_q) {
  return layout(w, at, 2ll * kMaxCtas * rows_cap(max_q), 0, rows_cap(max_q));   // first and last segment of each CTA
}
// Each row of the batch has a place for its prefix and one for its own tokens,
// shifted by a record for each CTA, so that all partials of a tile fit in order.
size_t prefix_layout(Work* w, void* at, int B, int groups) {
  return layout(w, at, 2ll * kNumQHeads * B + static_cast<int64_t>(kMaxCtas) * rows_cap(B), groups + static_cast<int64_t>(B),
                rows_cap(B));
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
    launch_pdl(true, prefix_merge_kernel, dim3(plan.B * kNumKVHeads), dim3(kMergeThreads), 0, s, plan, work, grid, o);
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
  return lsa::pool::prefix_layout(nullptr, nullptr, B, n_groups);
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
  if (!workspace || workspace_bytes < pool::prefix_layout(nullptr, nullptr, B, n_groups)) return LSA_ERR_WORKSPACE;
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
  pool::prefix_layout(&work, workspace, B, n_groups);
  const int64_t tiles = n_groups > 0 ? B / pool::kWideQ + n_groups : 0;
  const int64_t units = kNumKVHeads * (tiles * max_prefix_chunks + static_cast<int64_t>(B) * max_chunks);
  return pool::launch(plan, work, q, k_pool, v_pool, softmax_scale, out, units, stream);
}

}  // extern "C"
