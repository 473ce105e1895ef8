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
//
// What bounds it: HBM from some 2,000 tokens on -- 32 + 8 + 8 heads, k_out
// written: 16,384 tokens 71 us, 5.75 TB/s, 86% of a copy's rate; 65,536 tokens
// 272 us, 91%.  Below, a launch and the chain slot, position, angles, rows: one
// token 2.0 us, 1,021 tokens of 32 rows 3.8 us.  16,384 tokens take 65 us in halves
// of 32 dims, 70 in neighbours; other halves, which read a row's partner pieces
// and angles again, 70 us where 16 or 32 dims turn and 77 where 96 do (80% of a
// copy's rate).
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeLanes = 4;                       // lanes of a row
constexpr int kRopeGroups = 32 / kRopeLanes;        // rows of a warp at a time
constexpr int kRopeChunks = kHeadDim / 8 / kRopeLanes;  // 16-byte pieces of a lane

// Where a pair's dims lie: a lane holds the row's 16-byte pieces sub + 4 j.
constexpr int kRopeHalves128 = 0;   // halves of 64 dims: pieces j and j + 2 of the same lane
constexpr int kRopeHalves64 = 1;    // halves of 32 dims: pieces 0 and 1 of the same lane
constexpr int kRopePairs = 2;       // neighbours: within a piece
constexpr int kRopeHalvesAny = 3;   // other halves: the partner's piece is read as well

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
  int32_t warps_per_token;
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

// The largest, or NaN where one of them is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_or_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// The angles of a lane's pieces, in registers for all of a token's rows (for
// kRopeHalvesAny they are read again for each row).
template <int kMode>
struct RopeAngles {
  static constexpr int kN = kMode == kRopeHalves128 ? 16 : (kMode == kRopeHalves64 ? 8 : 16);
  float c[kN], s[kN];
  __device__ __forceinline__ void load(const float *cs, int r, int sub) {
    const int half = r >> 1;
    if (kMode == kRopeHalves128 || kMode == kRopeHalves64) {
#pragma unroll
      for (int j = 0; j < kN / 8; ++j) {
        load8(cs + 8 * (sub + kRopeLanes * j), *reinterpret_cast<float (*)[8]>(c + 8 * j));
        load8(cs + half + 8 * (sub + kRopeLanes * j), *reinterpret_cast<float (*)[8]>(s + 8 * j));
      }
    } else if (kMode == kRopePairs) {
#pragma unroll
      for (int j = 0; j < kRopeChunks; ++j) {
        const int i0 = 4 * (sub + kRopeLanes * j);      // the piece's first pair
        if (i0 < half) {
          const float4 a = __ldg(reinterpret_cast<const float4 *>(cs + i0));
          const float4 b = __ldg(reinterpret_cast<const float4 *>(cs + half + i0));
          c[4 * j] = a.x; c[4 * j + 1] = a.y; c[4 * j + 2] = a.z; c[4 * j + 3] = a.w;
          s[4 * j] = b.x; s[4 * j + 1] = b.y; s[4 * j + 2] = b.z; s[4 * j + 3] = b.w;
        }
      }
    }
  }
};

// A lane's pieces of one row, rotated in place (src: the row, for kRopeHalvesAny).
template <int kMode>
__device__ __forceinline__ void rotate_row(float (&x)[kRopeChunks][8], const RopeAngles<kMode> &ang,
                                           const uint16_t *src, const float *cs, int r, int sub) {
  if (kMode == kRopeHalves128 || kMode == kRopeHalves64) {
    constexpr int kFar = kMode == kRopeHalves128 ? 2 : 1;
#pragma unroll
    for (int j = 0; j < kFar; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = x[j][i], b = x[j + kFar][i];
        x[j][i] = turn_first(a, b, ang.c[8 * j + i], ang.s[8 * j + i]);
        x[j + kFar][i] = turn_second(a, b, ang.c[8 * j + i], ang.s[8 * j + i]);
      }
  } else if (kMode == kRopePairs) {
#pragma unroll
    for (int j = 0; j < kRopeChunks; ++j)
      if (8 * (sub + kRopeLanes * j) < r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[j][2 * i], b = x[j][2 * i + 1];
          x[j][2 * i] = turn_first(a, b, ang.c[4 * j + i], ang.s[4 * j + i]);
          x[j][2 * i + 1] = turn_second(a, b, ang.c[4 * j + i], ang.s[4 * j + i]);
        }
  } else {
    const int half = r >> 1;
#pragma unroll
    for (int j = 0; j < kRopeChunks; ++j) {
      const int e0 = 8 * (sub + kRopeLanes * j);        // the piece's first dim
      if (e0 >= r) continue;
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
}

// A warp, or warps_per_token of them, takes one token's rows, ordered (query
// heads, key heads, value heads), eight at a time, each on four lanes: the
// lane's loads and stores of a row are parts of contiguous 64 bytes, the
// token's angles stay in registers, and the next row is fetched while this one
// is worked on.  (16,384 tokens: blocks of 32 rows, whosever they are, with the
// angles read for each row 98.5 us; this 79.5; with streaming stores of the
// bf16 rows, 71.)
template <int kMode, bool kLoop>
__global__ void __launch_bounds__(kRopeWarps * 32)
rope_quantize_kernel(const RopeParams p) {
  const int sub = threadIdx.x & (kRopeLanes - 1);
  const unsigned gmask = ((1u << kRopeLanes) - 1u) << (threadIdx.x & 31 & ~(kRopeLanes - 1));
  const uint32_t warp = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);   // (below 2^31)
  const uint32_t token = warp / static_cast<uint32_t>(p.warps_per_token);
  const int part = static_cast<int>(warp - token * static_cast<uint32_t>(p.warps_per_token));
  const int64_t t = token;
  const int Hq = p.num_q_heads, H = p.num_kv_heads, rows = Hq + 2 * H;
  const int stride = kRopeGroups * p.warps_per_token;
  const int h0 = kRopeGroups * part + ((threadIdx.x & 31) / kRopeLanes);
  grid_dependency_wait();
  allow_dependents_launch();
  if (t >= p.num_tokens || h0 >= rows) return;
  auto row_at = [&](int h) -> const uint16_t * {
    return h < Hq ? p.q + t * p.q_stride + static_cast<int64_t>(h) * kHeadDim
                  : (h < Hq + H ? p.k + t * p.k_stride + static_cast<int64_t>(h - Hq) * kHeadDim
                                : p.v + t * p.v_stride + static_cast<int64_t>(h - Hq - H) * kHeadDim);
  };
  // (plain loads: the rotation may be in place)
  uint4 w[kRopeChunks];
  auto fetch = [&](int h) {
    const uint16_t *src = row_at(h);
#pragma unroll
    for (int j = 0; j < kRopeChunks; ++j)
      w[j] = *reinterpret_cast<const uint4 *>(src + 8 * (sub + kRopeLanes * j));
  };
  fetch(h0);
  const int64_t slot = p.slot_ids[t];
  if (slot < 0) return;
  const int64_t pos = p.positions[t];
  if (slot >= p.num_slots || pos < 0 || pos >= p.num_positions) {
    if (sub == 0 && h0 == 0 && p.err_flags) {
      int32_t f = slot >= p.num_slots ? KVQ_ERRF_SLOT_RANGE : 0;
      if (pos < 0 || pos >= p.num_positions) f |= KVQ_ERRF_POSITION_RANGE;
      atomicOr(p.err_flags, f);
    }
    return;
  }
  const float *cs = p.table + pos * p.rotary_dim;
  RopeAngles<kMode> ang;
  ang.load(cs, p.rotary_dim, sub);
  for (int hh = h0; hh < rows; hh += stride) {
    float x[kRopeChunks][8];
#pragma unroll
    for (int j = 0; j < kRopeChunks; ++j) unpack8(w[j], x[j]);
    if (kLoop && hh + stride < rows) fetch(hh + stride);
    const bool is_q = hh < Hq, is_v = hh >= Hq + H;
    const int h = is_q ? hh : (is_v ? hh - Hq - H : hh - Hq);
    if (!is_v) {
      rotate_row<kMode>(x, ang, row_at(hh), cs, p.rotary_dim, sub);
      uint16_t *dst = is_q ? p.q_out + t * p.q_out_stride
                           : (p.k_out ? p.k_out + t * p.k_out_stride : nullptr);
      // (every lane has read the row before any of it is overwritten in place)
      if (kMode == kRopeHalvesAny) __syncwarp(gmask);
      if (dst != nullptr) {
#pragma unroll
        for (int j = 0; j < kRopeChunks; ++j)
          __stcs(reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(h) * kHeadDim +
                                           8 * (sub + kRopeLanes * j)), pack8(x[j]));
      }
      if (is_q) {
        if (!kLoop) return;
        continue;
      }
    }
    // a NaN reaches the scale, as in the plain store (a chain per piece: one of all
    // 32 values takes 2.1 us for one token, not 1.9)
    float part[kRopeChunks];
#pragma unroll
    for (int j = 0; j < kRopeChunks; ++j) {
      part[j] = fabsf(x[j][0]);
#pragma unroll
      for (int i = 1; i < 7; i += 2)
        part[j] = max_or_nan(part[j], fabsf(x[j][i]), fabsf(x[j][i + 1]));
      part[j] = max_or_nan(part[j], fabsf(x[j][7]));
    }
    static_assert(kRopeChunks == 4, "the pieces' maxima");
    float amax = max_or_nan(max_or_nan(part[0], part[1], part[2]), part[3]);
#pragma unroll
    for (int off = 1; off < kRopeLanes; off <<= 1)
      amax = max_or_nan(amax, __shfl_xor_sync(gmask, amax, off));
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
    uint8_t *dst = (is_v ? p.v_codes : p.k_codes) + row * kHeadDim;
#pragma unroll
    for (int j = 0; j < kRopeChunks; ++j)
      *reinterpret_cast<uint2 *>(dst + 8 * (sub + kRopeLanes * j)) = codes[j];
    if (sub == 0) (is_v ? p.v_scales : p.k_scales)[row] = s;
    if (!kLoop) return;
  }
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
  // few tokens: their rows over more warps; many (8 an SM and up): one warp a
  // token, which reads its angles once and fetches ahead.  With 24 for 8, 1,021
  // tokens of 32 rows take 5.3 us instead of 3.6, 2,048 of 48 rows 9.3 instead
  // of 8.3; below 512 tokens the two differ by less than 0.2 us.
  const int64_t rows = static_cast<int64_t>(a.num_q_heads) + 2 * int64_t(c.num_kv_heads);
  const int64_t most = (rows + kRopeGroups - 1) / kRopeGroups;
  int64_t per_token = (8 * static_cast<int64_t>(a.sms) + a.num_tokens - 1) / a.num_tokens;
  per_token = per_token < 1 ? 1 : (per_token > most ? most : per_token);
  p.warps_per_token = static_cast<int32_t>(per_token);
  const int64_t warps = a.num_tokens * per_token;
  const dim3 grid(static_cast<unsigned>((warps + kRopeWarps - 1) / kRopeWarps));
  const dim3 block(kRopeWarps * 32);
  const int mode = a.layout == KVQ_ROPE_INTERLEAVED
                       ? kRopePairs
                       : (a.rotary_dim == 128 ? kRopeHalves128
                                              : (a.rotary_dim == 64 ? kRopeHalves64 : kRopeHalvesAny));
  const bool loop = per_token < most;
  using Kernel = void (*)(RopeParams);
  static constexpr Kernel kernels[4][2] = {
      {rope_quantize_kernel<kRopeHalves128, false>, rope_quantize_kernel<kRopeHalves128, true>},
      {rope_quantize_kernel<kRopeHalves64, false>, rope_quantize_kernel<kRopeHalves64, true>},
      {rope_quantize_kernel<kRopePairs, false>, rope_quantize_kernel<kRopePairs, true>},
      {rope_quantize_kernel<kRopeHalvesAny, false>, rope_quantize_kernel<kRopeHalvesAny, true>}};
  return launch_overlapped(kernels[mode][loop ? 1 : 0], grid, block, 0, stream, p);
}

}  // namespace kvq
