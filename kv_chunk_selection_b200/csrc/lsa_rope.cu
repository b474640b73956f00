// lsa_qk_norm_rope and lsa_qk_norm_rope_pool: what a serving step does to the
// row of the fused query/key/value projection before any attention call.
//
// Per token and per head of 128 dims (64 query heads, then 8 key heads; the 8
// value heads are copied):
//
//   y   = x * rsqrt(mean(x^2) + eps) * w                 (RMS norm; skipped without w)
//   a'  = s (a cos t - b sin t),  b' = s (b cos t + a sin t)   for each rotated pair
//
// with t = position * inv_freq[i] for pair i < rot_dim / 2, the pair being dims
// (i, i + rot_dim / 2) in the half layout and (2i, 2i + 1) in the interleaved
// one; dims rot_dim .. 127 keep y.  Everything is fp32 and rounded once to bf16,
// except the angle: a position near 2^20 times a frequency near 1 has no bits
// left for the fraction of a turn in fp32, so the turns are formed in fp64 (one
// multiply per pair), reduced to [-1/2, 1/2] and only then handed to sincospif.
//
// A block of 256 threads takes one token as 16 half-warps; half-warp w takes
// heads w, w + 16, ... (5 of the 80), so its 16 lanes hold a head as 8 dims
// each and the norm is 4 shuffles.  A lane's dims are chosen so that both
// members of its 4 pairs are its own: dims 4l .. 4l+3 and rot_dim/2 + 4l .. in
// the half layout, 8l .. 8l+7 in the interleaved one.  The lane's 4 (cos, sin)
// are then the same for all of its heads.  The block computes each of the token's
// once, while the loads of the heads are in flight, and passes them on in shared
// memory (58% of the issue slots; every half-warp its own: 68%, and 2% slower).
//
// The bytes bound it: 20 KiB read and 20 KiB written per token.  8191 tokens into
// the pool take 58.4 us in a row, 5.7 TB/s, 88% of the copy rate; one token 2.9 us,
// a launch and two rounds to memory.  5 blocks an SM (48 registers, 24 bytes of
// them spilled in the half layout): with 4 (60) 7% slower, with 6 (40) 19%.
#include <math.h>

#include "lsa_common.cuh"
#include "lsa_runtime.cuh"

namespace lsa {
namespace rope {

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;
constexpr int kHeadsIn = kNumQHeads + 2 * kNumKVHeads;   // 80 heads in a row of the projection
constexpr int kPerHalfWarp = kHeadsIn / kHalfWarps;      // 5: 4 query heads, then a key or a value head
static_assert(kPerHalfWarp * kHalfWarps == kHeadsIn && kNumQHeads % kHalfWarps == 0 && 2 * kNumKVHeads == kHalfWarps,
              "half-warps take whole rounds of query heads, then one key or value head");

struct Args {
  const __nv_bfloat16* qkv;
  int64_t row_stride;         // elements between the rows of the projection
  const float* w_q;           // [128] or nullptr: no norm
  const float* w_k;
  float eps;
  const int32_t* positions;   // [T]
  const float* inv_freq;      // [rot_dim / 2]
  int rot_dim;
  float scale;
  __nv_bfloat16* q_out;       // [T][64][128]
  __nv_bfloat16* k_out;       // [T][8][128], or the pool [slot][8][64][128]
  __nv_bfloat16* v_out;       // may be null in the dense form
  // The pool form (table_rows > 0): token t goes to position cache_pos[t] of
  // sequence seq_ids[t].
  const int32_t* chunk_table;
  const int32_t* seq_ids;
  const int32_t* cache_pos;
  int64_t n_slots;
  int table_rows, max_chunks;
};

__device__ __forceinline__ uint2 ld_dep2(const __nv_bfloat16* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_dep4(const float* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p)
               : "memory");
  return v;
}

// Row of the pool that token t's K and V go to, or -1 (not written).
__device__ __forceinline__ int64_t pool_row(const Args& a, int64_t t, unsigned* status, bool report) {
  const int pos = ld_dep(a.cache_pos + t);
  if (pos < 0) return -1;
  const int b = ld_dep(a.seq_ids + t);
  if (b < 0 || b >= a.table_rows) {
    if (report) set_status(status, LSA_DEV_ERR_BAD_COUNT);
    return -1;
  }
  if (pos / kChunkTokens >= a.max_chunks) {
    if (report) set_status(status, LSA_DEV_ERR_BAD_CHUNK);
    return -1;
  }
  const int64_t at = static_cast<int64_t>(b) * a.max_chunks + pos / kChunkTokens;
  const int64_t slot = a.chunk_table ? ld_dep(a.chunk_table + at) : at;
  if (slot < 0 || slot >= a.n_slots) {
    if (report) set_status(status, LSA_DEV_ERR_BAD_SLOT);
    return -1;
  }
  return slot * (kNumKVHeads * kChunkTokens) + pos % kChunkTokens;
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 5) qk_norm_rope_kernel(const Args a, unsigned* status) {
  // The wait first: the next kernel may be an attention call that reads what the one
  // before this wrote (the gather's chunks, under LSA_ATTN_KV_UNCHANGED) without a
  // wait of its own.
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int hw = threadIdx.x >> 4, lane = threadIdx.x & 15;
  // This lane's two runs of 4 dims.
  const int half = a.rot_dim >> 1;
  const bool turns = 8 * lane < a.rot_dim;   // rot_dim is a multiple of 8: a lane's dims all turn, or none
  int d0 = 8 * lane, d1 = 8 * lane + 4;
  if (!kInterleaved && turns) {
    d0 = 4 * lane;
    d1 = half + 4 * lane;
  }
  const __nv_bfloat16* row = a.qkv + t * a.row_stride;
  uint2 in[kPerHalfWarp][2];
#pragma unroll
  for (int i = 0; i < kPerHalfWarp; ++i) {
    const __nv_bfloat16* x = row + (hw + kHalfWarps * i) * kHeadDim;
    in[i][0] = ld_dep2(x + d0);
    in[i][1] = ld_dep2(x + d1);
  }
  // The token's (cos, sin), a pair per thread, while the loads are on their way.
  __shared__ float4 turn_of[kHeadDim / 4];
  if (static_cast<int>(threadIdx.x) < half) {
    const double pos = static_cast<double>(ld_dep(a.positions + t)) * 0.15915494309189533577;   // 1 / (2 pi)
    const double turn = pos * static_cast<double>(ld_dep(a.inv_freq + threadIdx.x));
    float c, s;
    sincospif(2.f * static_cast<float>(turn - rint(turn)), &s, &c);
    reinterpret_cast<float2*>(turn_of)[threadIdx.x] = make_float2(c * a.scale, s * a.scale);
  }
  float4 w0 = make_float4(1.f, 1.f, 1.f, 1.f), w1 = w0;
  if (a.w_q) {
    w0 = ld_dep4(a.w_q + d0);
    w1 = ld_dep4(a.w_q + d1);
  }
  __syncthreads();
  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (turns) {
    const float4 x = turn_of[2 * lane], y = turn_of[2 * lane + 1];
    cs[0] = x.x; sn[0] = x.y; cs[1] = x.z; sn[1] = x.w;
    cs[2] = y.x; sn[2] = y.y; cs[3] = y.z; sn[3] = y.w;
  }

  // One head: norm, rotation, and the two packed runs of dims.
  auto turn_head = [&](const uint2 lo, const uint2 hi, bool norm, uint2& out0, uint2& out1) {
    float x[8] = {bf16_lo(lo.x), bf16_hi(lo.x), bf16_lo(lo.y), bf16_hi(lo.y),
                  bf16_lo(hi.x), bf16_hi(hi.x), bf16_lo(hi.y), bf16_hi(hi.y)};
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
#pragma unroll
      for (int off = 8; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float r = rsqrtf(ss * (1.f / kHeadDim) + a.eps);
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
    }
    if (turns) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = kInterleaved ? 2 * j : j, q = kInterleaved ? 2 * j + 1 : 4 + j;
        const float u = x[p], v = x[q];
        x[p] = u * cs[j] - v * sn[j];
        x[q] = v * cs[j] + u * sn[j];
      }
    }
    out0 = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    out1 = make_uint2(pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  };

  __nv_bfloat16* q = a.q_out + t * (kNumQHeads * kHeadDim);
#pragma unroll
  for (int i = 0; i < kPerHalfWarp - 1; ++i) {
    uint2 o0, o1;
    turn_head(in[i][0], in[i][1], a.w_q != nullptr, o0, o1);
    __nv_bfloat16* dst = q + (hw + kHalfWarps * i) * kHeadDim;
    *reinterpret_cast<uint2*>(dst + d0) = o0;
    *reinterpret_cast<uint2*>(dst + d1) = o1;
  }

  // The last head of this half-warp: key head hw, or value head hw - 8 (whole
  // warps take either).
  const bool is_k = hw < kNumKVHeads;
  const int g = hw & (kNumKVHeads - 1);
  uint2 o0 = in[kPerHalfWarp - 1][0], o1 = in[kPerHalfWarp - 1][1];
  if (is_k) {
    if (a.w_k) {
      w0 = ld_dep4(a.w_k + d0);
      w1 = ld_dep4(a.w_k + d1);
    }
    turn_head(in[kPerHalfWarp - 1][0], in[kPerHalfWarp - 1][1], a.w_k != nullptr, o0, o1);
  }
  __nv_bfloat16* kv = is_k ? a.k_out : a.v_out;
  if (!kv) return;
  int64_t at;
  if (a.table_rows > 0) {
    const int64_t r = pool_row(a, t, status, threadIdx.x == 0);
    if (r < 0) return;
    at = r + g * kChunkTokens;
  } else {
    at = t * kNumKVHeads + g;
  }
  *reinterpret_cast<uint2*>(kv + at * kHeadDim + d0) = o0;
  *reinterpret_cast<uint2*>(kv + at * kHeadDim + d1) = o1;
}

// Checks and launch shared by both forms.
int launch(const Args& a, int64_t T, unsigned flags, void* stream) {
  if (!a.qkv || !a.q_out || !a.k_out || T <= 0) return LSA_ERR_INVALID_ARG;
  if (a.k_out == a.v_out || a.q_out == a.k_out || a.q_out == a.v_out) return LSA_ERR_INVALID_ARG;   // two heads, one place
  if (flags & ~static_cast<unsigned>(LSA_ROPE_INTERLEAVED)) return LSA_ERR_INVALID_ARG;
  if (a.rot_dim < 0 || a.rot_dim > kHeadDim || a.row_stride < kHeadsIn * kHeadDim) return LSA_ERR_INVALID_ARG;
  if (a.rot_dim > 0 && (!a.positions || !a.inv_freq)) return LSA_ERR_INVALID_ARG;
  if (!(a.eps >= 0.f) || !isfinite(a.eps) || !isfinite(a.scale)) return LSA_ERR_INVALID_ARG;
  if (a.rot_dim % 8 != 0 || T > 0x7fffffff) return LSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(a.qkv) || a.row_stride % 8 != 0 || !aligned16(a.q_out) || !aligned16(a.k_out) || !aligned16(a.v_out) ||
      !aligned16(a.w_q) || !aligned16(a.w_k))
    return LSA_ERR_MISALIGNED;
  if (device_sm_count() <= 0) return LSA_ERR_NO_DEVICE;
  const auto kernel = (flags & LSA_ROPE_INTERLEAVED) ? qk_norm_rope_kernel<true> : qk_norm_rope_kernel<false>;
  launch_pdl(true, kernel, dim3(static_cast<unsigned>(T)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a,
             lsa_device_status_ptr());
  return launch_status();
}

}  // namespace rope
}  // namespace lsa

extern "C" {

int lsa_qk_norm_rope(const void* qkv, int64_t row_stride, int64_t T, const float* q_weight, const float* k_weight,
                     float eps, const int32_t* positions, const float* inv_freq, int rot_dim, float rope_scale,
                     unsigned int flags, void* q_out, void* k_out, void* v_out, void* stream) {
  using namespace lsa;
  rope::Args a = {};
  a.qkv = static_cast<const __nv_bfloat16*>(qkv);
  a.row_stride = row_stride;
  a.w_q = q_weight;
  a.w_k = k_weight;
  a.eps = eps;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.rot_dim = rot_dim;
  a.scale = rope_scale;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  return rope::launch(a, T, flags, stream);
}

int lsa_qk_norm_rope_pool(const void* qkv, int64_t row_stride, int64_t T, const float* q_weight, const float* k_weight,
                          float eps, const int32_t* positions, const float* inv_freq, int rot_dim, float rope_scale,
                          unsigned int flags, void* q_out, void* k_pool, void* v_pool, int64_t n_slots,
                          const int32_t* chunk_table, const int32_t* seq_ids, const int32_t* cache_pos, int B,
                          int max_chunks, void* stream) {
  using namespace lsa;
  if (!v_pool || !seq_ids || !cache_pos || B <= 0 || max_chunks <= 0 || n_slots <= 0) return LSA_ERR_INVALID_ARG;
  rope::Args a = {};
  a.qkv = static_cast<const __nv_bfloat16*>(qkv);
  a.row_stride = row_stride;
  a.w_q = q_weight;
  a.w_k = k_weight;
  a.eps = eps;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.rot_dim = rot_dim;
  a.scale = rope_scale;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_pool);
  a.v_out = static_cast<__nv_bfloat16*>(v_pool);
  a.chunk_table = chunk_table;
  a.seq_ids = seq_ids;
  a.cache_pos = cache_pos;
  a.n_slots = n_slots;
  a.table_rows = B;
  a.max_chunks = max_chunks;
  return rope::launch(a, T, flags, stream);
}

}  // extern "C"
