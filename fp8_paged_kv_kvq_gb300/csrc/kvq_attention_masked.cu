// kvq_attention_masked.cu -- paged attention over the FP8 cache whose rows see a
// sliding window and the first tokens of their sequence, or the ancestors of a
// drafted token.
//
//   s_j = sm_scale k_scale_j (q . kc_j),  out = sum_j p_j v_scale_j vc_j / sum_j p_j,
//   p_j = exp(s_j - max_j s_j), j over the tokens the row sees
//
// A block per (query row, query head), a warp per eighth of the tokens, four dims
// a lane, one pass with a running maximum and sum.
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kMkWarps = 8;

struct MkParams {
  kvq_cache c;
  MaskedArgs a;
  int32_t ctx_limit, G, words;
};

__device__ __forceinline__ float mk_e4m3(uint32_t code) {
  const float x = __uint_as_float(((code & 0x80u) << 24) | ((code & 0x7Fu) << 20)) * 0x1p120f;
  return (code & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : x;
}

__global__ void __launch_bounds__(32 * kMkWarps) attn_masked_kernel(const MkParams p) {
  __shared__ float part[kMkWarps][kHeadDim + 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int R = p.a.rows_per_request, Hq = p.a.num_q_heads, H = p.c.num_kv_heads;
  const int hq = static_cast<int>(blockIdx.x % Hq);
  const int64_t row = blockIdx.x / Hq;
  const int r = static_cast<int>(row / R), i = static_cast<int>(row % R), h = hq / p.G;
  allow_dependents_launch();
  grid_dependency_wait();
  int L = p.a.context_lens[r];
  if (L < 0 || L > p.ctx_limit) {
    if (threadIdx.x == 0 && p.a.err_flags) atomicOr(p.a.err_flags, KVQ_ERRF_CONTEXT_RANGE);
    L = L < 0 ? 0 : p.ctx_limit;
  }
  const uint2 qw = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.a.q) +
                                                   (row * Hq + hq) * kHeadDim)[lane];
  const float q[4] = {bf16_lo(qw.x), bf16_hi(qw.x), bf16_lo(qw.y), bf16_hi(qw.y)};
  const int base = L - R, own = base + i;
  const int32_t *mask = p.a.tree_mask ? p.a.tree_mask + row * p.words : nullptr;
  float m = -INFINITY, sum = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = warp; j < L; j += kMkWarps) {
    bool seen;
    if (mask) {
      const int b = j - base;
      seen = b < 0 || ((mask[b >> 5] >> (b & 31)) & 1) != 0;
    } else {
      seen = j <= own && (j < p.a.num_sinks || j > own - static_cast<int64_t>(p.a.window));
    }
    if (!seen) continue;
    const int page = p.a.block_tables[static_cast<int64_t>(r) * p.a.max_blocks_per_req + (j >> p.a.log2_block)];
    if (page < 0 || page >= (p.c.num_slots >> p.a.log2_block)) {
      if (lane == 0 && p.a.err_flags) atomicOr(p.a.err_flags, KVQ_ERRF_BLOCK_RANGE);
      continue;
    }
    const int64_t at = ((static_cast<int64_t>(page) << p.a.log2_block) + (j & ((1 << p.a.log2_block) - 1))) * H + h;
    const uint32_t k = reinterpret_cast<const uint32_t *>(p.c.k_codes + at * kHeadDim)[lane];
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fmaf(q[e], mk_e4m3((k >> (8 * e)) & 0xFFu), s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    s *= p.c.k_scales[at] * p.a.sm_scale;
    const float top = fmaxf(m, s), f = m == -INFINITY ? 0.0f : expf(m - top), w = expf(s - top);
    const uint32_t v = reinterpret_cast<const uint32_t *>(p.c.v_codes + at * kHeadDim)[lane];
    const float wv = w * p.c.v_scales[at];
    m = top;
    sum = sum * f + w;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fmaf(wv, mk_e4m3((v >> (8 * e)) & 0xFFu), o[e] * f);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) part[warp][4 * lane + e] = o[e];
  if (lane == 0) {
    part[warp][kHeadDim] = m;
    part[warp][kHeadDim + 1] = sum;
  }
  __syncthreads();
  const int d = threadIdx.x;
  if (d < kHeadDim) {
    float top = -INFINITY, all = 0.0f, x = 0.0f;
    for (int w = 0; w < kMkWarps; ++w) top = fmaxf(top, part[w][kHeadDim]);
    for (int w = 0; w < kMkWarps; ++w) {
      const float f = part[w][kHeadDim] == -INFINITY ? 0.0f : expf(part[w][kHeadDim] - top);
      all += part[w][kHeadDim + 1] * f;
      x += part[w][d] * f;
    }
    static_cast<uint16_t *>(p.a.out)[(row * Hq + hq) * kHeadDim + d] =
        static_cast<uint16_t>(pack_bf16x2(all > 0.0f || all != all ? x / all : 0.0f, 0.0f));
  }
}

}  // namespace

size_t attn_masked_workspace_bytes(const MaskedArgs &, int32_t) { return 0; }

cudaError_t launch_attn_masked(const kvq_cache &c, const MaskedArgs &a, cudaStream_t stream) {
  const int64_t cap = static_cast<int64_t>(a.max_blocks_per_req) << a.log2_block;
  MkParams p{c, a, static_cast<int32_t>(cap < a.max_context_len ? cap : a.max_context_len),
             a.num_q_heads / c.num_kv_heads, (a.rows_per_request + 31) / 32};
  const int64_t blocks = static_cast<int64_t>(a.num_requests) * a.rows_per_request * a.num_q_heads;
  return launch_overlapped(attn_masked_kernel, dim3(static_cast<unsigned>(blocks)),
                           dim3(32 * kMkWarps), 0, stream, p);
}

}  // namespace kvq
