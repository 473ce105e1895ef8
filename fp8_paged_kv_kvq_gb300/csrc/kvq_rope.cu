// kvq_rope.cu -- the rotary position embedding and the store of a step's rows
// in one pass: query and key rows rotated by their tokens' positions, the
// rotated keys and the values quantised into the FP8 E4M3 paged cache.
//
// The rows' format is the store's (FreeToken PR #354 "feat(kvcache): store the
// KV cache as fp8 e4m3 codes"; ROCm/ATOM PR #2655, K/V bullet); the pages store
// keys that were rotated and rounded to bf16 by an earlier kernel.  Here the
// rotation happens between the load and the quantiser, in binary32, so a row
// crosses HBM once and loses one rounding.
//
// Each pair (a, b) of a row's first rotary_dim dims, at angle index i of its
// token's table row, becomes (a c_i - b s_i, b c_i + a s_i).  Products and sums
// round separately (no contraction): the codes and scales are then a function
// of the inputs alone and match an elementwise fp32 evaluation bit for bit.
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeLanes = 4;                       // lanes of a row
constexpr int kRopeRows = kRopeThreads / kRopeLanes;   // rows of a CTA
constexpr int kRopeChunks = kHeadDim / 8 / kRopeLanes;  // 16-byte pieces of a lane

struct RopeParams {
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int64_t num_tokens;
  const int64_t *positions;
  const float *table;
  int64_t num_positions;
  const int64_t *slot_ids;
  uint8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  int64_t num_slots;
  int32_t num_q_heads, num_kv_heads, rotary_dim;
  int32_t *err_flags;
  uint64_t rows_magic;      // row id / rows per token by a multiply
  int32_t rows_shift;
};

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x);
  x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z);
  x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void load8(const float *src, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(src));
  const float4 b = __ldg(reinterpret_cast<const float4 *>(src) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// a c - b s and b c + a s, each product and sum rounded once
__device__ __forceinline__ float turn_first(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_second(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Four codes of binary32 values: fl32(x / s) then e4m3 round-to-nearest-even,
// every code with its value's sign (a zero keeps its sign).
template <bool kFast>
__device__ __forceinline__ uint32_t encode4_f32(const float *x, float s, float y) {
  float q[4];
  if (kFast) {
    const uint64_t ns = pack_f32x2(-s, -s), yy = pack_f32x2(y, y);
    unpack_f32x2(div_markstein_x2(pack_f32x2(x[0], x[1]), ns, yy), q[0], q[1]);
    unpack_f32x2(div_markstein_x2(pack_f32x2(x[2], x[3]), ns, yy), q[2], q[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = __fdiv_rn(x[e], s);
  }
  const uint32_t s01 = prmt(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x0073u);
  const uint32_t s23 = prmt(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x0073u);
  const uint32_t signs = prmt(s01, s23, 0x5410u) & 0x80808080u;
  return e4m3x2_rn(q[0], q[1]) | (e4m3x2_rn(q[2], q[3]) << 16) | signs;
}

// One row per 4-lane group, rows ordered (token; query heads, key heads, value
// heads).  Lane `sub` holds the row's 16-byte pieces sub + 4 j, j < 4, so each
// of its loads and stores is part of a contiguous 64 bytes, and for a rotation
// of 128 or 64 dims in halves both dims of a pair lie in one lane (pieces 8 or
// 4 apart: j with j + 2 or j + 1).
template <int kLayout>
__global__ void __launch_bounds__(kRopeThreads)
rope_quantize_kernel(const RopeParams p) {
  const int sub = threadIdx.x & (kRopeLanes - 1);
  const unsigned gmask = ((1u << kRopeLanes) - 1u) << (threadIdx.x & 31 & ~(kRopeLanes - 1));
  const uint32_t rid = blockIdx.x * kRopeRows + threadIdx.x / kRopeLanes;
  const int Hq = p.num_q_heads, H = p.num_kv_heads;
  const uint32_t t32 =
      static_cast<uint32_t>((static_cast<uint64_t>(rid) * p.rows_magic) >> p.rows_shift);
  grid_dependency_wait();
  allow_dependents_launch();
  if (t32 >= p.num_tokens) return;
  const int64_t t = t32;
  int h = static_cast<int>(rid - t32 * static_cast<uint32_t>(Hq + 2 * H));
  const bool flagger = sub == 0 && h == 0 && p.err_flags != nullptr;
  const int kind = h < Hq ? 0 : (h < Hq + H ? 1 : 2);   // query, key, value
  h -= kind == 0 ? 0 : (kind == 1 ? Hq : Hq + H);
  const uint16_t *src = (kind == 0 ? p.q + t * p.q_stride
                                   : (kind == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride)) +
                        h * kHeadDim;
  // (plain loads: the rotation may be in place)
  uint4 w[kRopeChunks];
#pragma unroll
  for (int j = 0; j < kRopeChunks; ++j)
    w[j] = *reinterpret_cast<const uint4 *>(src + 8 * (sub + kRopeLanes * j));
  const int64_t slot = p.slot_ids[t];
  if (slot < 0) return;
  const int64_t pos = p.positions[t];
  if (slot >= p.num_slots || pos < 0 || pos >= p.num_positions) {
    if (flagger) {
      int32_t f = slot >= p.num_slots ? KVQ_ERRF_SLOT_RANGE : 0;
      if (pos < 0 || pos >= p.num_positions) f |= KVQ_ERRF_POSITION_RANGE;
      atomicOr(p.err_flags, f);
    }
    return;
  }
  float x[kRopeChunks][8];
#pragma unroll
  for (int j = 0; j < kRopeChunks; ++j) unpack8(w[j], x[j]);
  if (kind != 2) {
    const int r = p.rotary_dim, half = r >> 1;
    const float *cs = p.table + pos * r;
#pragma unroll
    for (int j = 0; j < kRopeChunks; ++j) {
      const int e0 = 8 * (sub + kRopeLanes * j);        // the piece's first dim
      if (e0 >= r) continue;
      if (kLayout == KVQ_ROPE_INTERLEAVED) {
        const float4 c = __ldg(reinterpret_cast<const float4 *>(cs + (e0 >> 1)));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + half + (e0 >> 1)));
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[j][2 * i], b = x[j][2 * i + 1];
          x[j][2 * i] = turn_first(a, b, cc[i], ss[i]);
          x[j][2 * i + 1] = turn_second(a, b, cc[i], ss[i]);
        }
      } else {
        // the piece of the pairs' other dims, half a rotation away
        const bool first = e0 < half;
        const int i0 = first ? e0 : e0 - half;
        float o[8], c[8], s[8];
        unpack8(*reinterpret_cast<const uint4 *>(src + (first ? e0 + half : i0)), o);
        load8(cs + i0, c);
        load8(cs + half + i0, s);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[j][i] = first ? turn_first(x[j][i], o[i], c[i], s[i])
                          : turn_second(o[i], x[j][i], c[i], s[i]);
      }
    }
    uint16_t *dst = kind == 0 ? p.q_out + t * p.q_out_stride
                              : (p.k_out ? p.k_out + t * p.k_out_stride : nullptr);
    // (every lane has read the row before any of it is overwritten in place)
    __syncwarp(gmask);
    if (dst != nullptr) {
#pragma unroll
      for (int j = 0; j < kRopeChunks; ++j)
        *reinterpret_cast<uint4 *>(dst + h * kHeadDim + 8 * (sub + kRopeLanes * j)) = pack8(x[j]);
    }
    if (kind == 0) return;
  }
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < kRopeChunks; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[j][i]));
#pragma unroll
  for (int off = 1; off < kRopeLanes; off <<= 1)
    amax = fmaxf(amax, __shfl_xor_sync(gmask, amax, off));
  uint2 codes[kRopeChunks];
#pragma unroll
  for (int j = 0; j < kRopeChunks; ++j) codes[j] = make_uint2(0u, 0u);
  float s = 0.0f;
  if (amax != 0.0f) {
    s = row_scale(amax);
    if (s >= kMarksteinMinScale) {
      const float y = __frcp_rn(s);
#pragma unroll
      for (int j = 0; j < kRopeChunks; ++j)
        codes[j] = make_uint2(encode4_f32<true>(&x[j][0], s, y), encode4_f32<true>(&x[j][4], s, y));
    } else {
#pragma unroll
      for (int j = 0; j < kRopeChunks; ++j)
        codes[j] = make_uint2(encode4_f32<false>(&x[j][0], s, 0.0f),
                              encode4_f32<false>(&x[j][4], s, 0.0f));
    }
  }
  const int64_t row = slot * H + h;
  uint8_t *dst = (kind == 2 ? p.v_codes : p.k_codes) + row * kHeadDim;
#pragma unroll
  for (int j = 0; j < kRopeChunks; ++j)
    *reinterpret_cast<uint2 *>(dst + 8 * (sub + kRopeLanes * j)) = codes[j];
  if (sub == 0) (kind == 2 ? p.v_scales : p.k_scales)[row] = s;
}

}  // namespace

cudaError_t launch_rope_quantize_scatter(const kvq_cache &c, const RopeArgs &a, int32_t *err_flags,
                                         cudaStream_t stream) {
  RopeParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.k = static_cast<const uint16_t *>(a.k);
  p.v = static_cast<const uint16_t *>(a.v);
  p.q_out = static_cast<uint16_t *>(a.q_out);
  p.k_out = static_cast<uint16_t *>(a.k_out);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_out_stride = a.q_out_stride;
  p.k_out_stride = a.k_out_stride;
  p.num_tokens = a.num_tokens;
  p.positions = a.positions;
  p.table = a.table;
  p.num_positions = a.num_positions;
  p.slot_ids = a.slot_ids;
  p.k_codes = c.k_codes;
  p.v_codes = c.v_codes;
  p.k_scales = c.k_scales;
  p.v_scales = c.v_scales;
  p.num_slots = c.num_slots;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = c.num_kv_heads;
  p.rotary_dim = a.rotary_dim;
  p.err_flags = err_flags;
  // n / d == (n * ceil(2^S / d)) >> S for every n < 2^31 when S = 32 + ceil(log2 d)
  const uint64_t d = static_cast<uint64_t>(a.num_q_heads) + 2u * static_cast<uint64_t>(c.num_kv_heads);
  int l = 0;
  while ((uint64_t(1) << l) < d) ++l;
  p.rows_shift = 32 + l;
  p.rows_magic = ((uint64_t(1) << (32 + l)) + d - 1) / d;
  const int64_t rows = a.num_tokens * static_cast<int64_t>(d);
  const dim3 grid(static_cast<unsigned>((rows + kRopeRows - 1) / kRopeRows));
  if (a.layout == KVQ_ROPE_INTERLEAVED)
    return launch_overlapped(rope_quantize_kernel<KVQ_ROPE_INTERLEAVED>, grid, dim3(kRopeThreads),
                             0, stream, p);
  return launch_overlapped(rope_quantize_kernel<KVQ_ROPE_HALVES>, grid, dim3(kRopeThreads), 0,
                           stream, p);
}

}  // namespace kvq
