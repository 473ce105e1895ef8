// kvq_prompt.cu -- causal attention of packed prompts over their own bf16 keys
// and values (grouped query heads, sequences of different lengths in one token
// buffer), before anything is read from the cache.
//
// A unit of work is 64 of the stacked rows m = i G + g (token i, query head
// h G + g) of one sequence and KV head h: the G heads that share a KV head use
// the same keys, so a tile of few tokens fills the matrix product's rows.
// Sequence s may use the units floor(cu[s] G / 64) + s up to the next
// sequence's: at least as many as its rows need, and a unit finds its sequence
// by a search over cu_seqlens with no plan made beforehand.
#include <cuda_runtime.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kPrRows = 64;                  // stacked rows of a unit
constexpr int kPrKeys = 64;                  // keys of a tile
constexpr int kPrWarps = 4;                  // 16 rows each
constexpr int kPrPitch = kHeadDim + 8;       // elements: rows 16 bytes apart in the banks

struct PromptParams {
  const uint16_t *q, *k, *v;
  uint16_t *out;
  int64_t q_stride, k_stride, v_stride, out_stride;
  int32_t num_tokens;
  const int32_t *cu;
  int32_t N, max_seqlen, G, H;
  float scale2;                              // sm_scale log2(e)
  int32_t *err_flags;
};

__device__ __forceinline__ float pr_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// 16-bit lanes of w that hold an infinity or NaN become 0.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return w;
}

__global__ void __launch_bounds__(kPrWarps * 32)
prompt_attention_kernel(const PromptParams p) {
  __shared__ __align__(16) uint16_t ks[kPrKeys * kPrPitch];
  __shared__ __align__(16) uint16_t vs[kPrKeys * kPrPitch];
  __shared__ int dirty;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  allow_dependents_launch();
  grid_dependency_wait();
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.H));
  const int64_t x = blockIdx.x / static_cast<unsigned>(p.H);
  auto base = [&](int s) -> int64_t {
    return static_cast<int64_t>(p.cu[s]) * p.G / kPrRows + s;
  };
  if (p.err_flags) {
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * (kPrWarps * 32) + tid; s < p.N;
         s += static_cast<int64_t>(gridDim.x) * (kPrWarps * 32)) {
      const int a = p.cu[s], b = p.cu[s + 1];
      if (a < 0 || b < a || b > p.num_tokens || b - a > p.max_seqlen)
        atomicOr(p.err_flags, KVQ_ERRF_SEQUENCE_RANGE);
    }
  }
  int lo = 0, hi = p.N - 1;
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (base(mid) <= x) lo = mid;
    else hi = mid - 1;
  }
  const int start = p.cu[lo], end = p.cu[lo + 1];
  if (start < 0 || end < start || end > p.num_tokens || end - start > p.max_seqlen) return;
  const int len = end - start;
  const int64_t rows = static_cast<int64_t>(len) * p.G;
  const int64_t units = (rows + kPrRows - 1) / kPrRows;
  const int64_t u = units - 1 - (x - base(lo));          // heaviest first
  if (u < 0 || u >= units) return;
  const int64_t row0 = u * kPrRows;
  const int g4 = lane >> 2, c4 = lane & 3;

  // this thread's two rows (g4 and g4 + 8 of its warp's 16)
  int tok[2];
  const uint16_t *qp[2];
  uint16_t *op[2];
  bool ok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = row0 + 16 * warp + g4 + 8 * i;
    ok[i] = m < rows;
    const int64_t mm = ok[i] ? m : rows - 1;
    tok[i] = static_cast<int>(mm / p.G);
    const int64_t head = static_cast<int64_t>(h) * p.G + (mm - static_cast<int64_t>(tok[i]) * p.G);
    qp[i] = p.q + (start + tok[i]) * p.q_stride + head * kHeadDim;
    op[i] = p.out + (start + tok[i]) * p.out_stride + head * kHeadDim;
  }
  uint32_t qf[8][4];
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    qf[kk][0] = *reinterpret_cast<const uint32_t *>(qp[0] + 16 * kk + 2 * c4);
    qf[kk][1] = *reinterpret_cast<const uint32_t *>(qp[1] + 16 * kk + 2 * c4);
    qf[kk][2] = *reinterpret_cast<const uint32_t *>(qp[0] + 16 * kk + 8 + 2 * c4);
    qf[kk][3] = *reinterpret_cast<const uint32_t *>(qp[1] + 16 * kk + 8 + 2 * c4);
  }
  float o[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};

  const int first_tok = static_cast<int>(row0 / p.G);
  const int64_t last_row = (row0 + kPrRows < rows ? row0 + kPrRows : rows) - 1;
  const int keys = static_cast<int>(last_row / p.G) + 1;  // keys the unit's last row sees
  for (int j0 = 0; j0 < keys; j0 += kPrKeys) {
    // a tile some row does not see whole: its values with infinities and NaN
    // taken out (a zero probability would not), those are added at the end
    const bool edge = j0 + kPrKeys - 1 > first_tok;
    __syncthreads();
    if (tid == 0) dirty = 0;
    __syncthreads();
    for (int i = tid; i < kPrKeys * (kHeadDim / 8); i += kPrWarps * 32) {
      const int r = i / (kHeadDim / 8), c = i % (kHeadDim / 8);
      uint4 kw = make_uint4(0u, 0u, 0u, 0u), vw = kw;
      if (j0 + r < keys) {
        kw = *reinterpret_cast<const uint4 *>(p.k + (start + j0 + r) * p.k_stride + h * kHeadDim + 8 * c);
        vw = *reinterpret_cast<const uint4 *>(p.v + (start + j0 + r) * p.v_stride + h * kHeadDim + 8 * c);
      }
      if (edge) {
        const uint4 f = make_uint4(finite_or_zero(vw.x), finite_or_zero(vw.y),
                                   finite_or_zero(vw.z), finite_or_zero(vw.w));
        if (f.x != vw.x || f.y != vw.y || f.z != vw.z || f.w != vw.w) dirty = 1;
        vw = f;
      }
      *reinterpret_cast<uint4 *>(ks + r * kPrPitch + 8 * c) = kw;
      *reinterpret_cast<uint4 *>(vs + r * kPrPitch + 8 * c) = vw;
    }
    __syncthreads();
    float s[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < 8; kk += 2) {
        uint32_t b[4];
        ldsm_x4(smem_addr(ks + (8 * n + (lane & 7)) * kPrPitch + 16 * kk + 8 * (lane >> 3)), b);
        mma_bf16_16816(s[n], qf[kk], b[0], b[1]);
        mma_bf16_16816(s[n], qf[kk + 1], b[2], b[3]);
      }
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = j0 + 8 * n + 2 * c4 + (i & 1);
        if (key > tok[i >> 1]) s[n][i] = -INFINITY;
        mx[i >> 1] = fmaxf(mx[i >> 1], s[n][i]);
      }
    float shift[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 1));
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 2));
      const float m_new = fmaxf(m_run[i], mx[i]);
      const float f = m_run[i] == -INFINITY ? 0.0f : pr_ex2((m_run[i] - m_new) * p.scale2);
      m_run[i] = m_new;
      shift[i] = m_new == -INFINITY ? 0.0f : m_new * p.scale2;
      l_run[i] *= f;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        o[n][2 * i] *= f;
        o[n][2 * i + 1] *= f;
      }
    }
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[n][i] = pr_ex2(fmaf(s[n][i], p.scale2, -shift[i >> 1]));
        l_run[i >> 1] += s[n][i];
      }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint32_t a[4] = {pack_bf16x2(s[2 * kk][0], s[2 * kk][1]),
                             pack_bf16x2(s[2 * kk][2], s[2 * kk][3]),
                             pack_bf16x2(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                             pack_bf16x2(s[2 * kk + 1][2], s[2 * kk + 1][3])};
#pragma unroll
      for (int n = 0; n < 16; n += 2) {
        uint32_t b[4];
        ldsm_x4_trans(smem_addr(vs + (16 * kk + (lane & 15)) * kPrPitch + 8 * n + 8 * (lane >> 4)), b);
        mma_bf16_16816(o[n], a, b[0], b[1]);
        mma_bf16_16816(o[n + 1], a, b[2], b[3]);
      }
    }
    if (dirty) {
      // the infinities and NaN that a row does see, as the sum has them
      for (int r = 0; r < kPrKeys && j0 + r < keys; ++r)
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t e = p.v[(start + j0 + r) * p.v_stride + h * kHeadDim + 8 * n + 2 * c4 + (i & 1)];
            if ((e & 0x7F80u) == 0x7F80u && j0 + r <= tok[i >> 1]) o[n][i] += bf16_lo(e);
          }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l_run[i] += __shfl_xor_sync(0xFFFFFFFFu, l_run[i], 1);
    l_run[i] += __shfl_xor_sync(0xFFFFFFFFu, l_run[i], 2);
    const float inv = 1.0f / l_run[i];
    if (!ok[i]) continue;
#pragma unroll
    for (int n = 0; n < 16; ++n)
      *reinterpret_cast<uint32_t *>(op[i] + 8 * n + 2 * c4) =
          pack_bf16x2(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
  }
}

int64_t prompt_units(const PromptArgs &a) {
  const int64_t G = a.num_q_heads / a.num_kv_heads;
  return (a.num_tokens * G / kPrRows + a.num_seqs) * a.num_kv_heads;
}

}  // namespace

bool prompt_attention_supported(const PromptArgs &a) { return prompt_units(a) <= 0x7FFFFFFF; }

cudaError_t launch_prompt_attention(const PromptArgs &a, cudaStream_t stream) {
  PromptParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.k = static_cast<const uint16_t *>(a.k);
  p.v = static_cast<const uint16_t *>(a.v);
  p.out = static_cast<uint16_t *>(a.out);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.out_stride = a.out_stride;
  p.num_tokens = static_cast<int32_t>(a.num_tokens);
  p.cu = a.cu_seqlens;
  p.N = a.num_seqs;
  p.max_seqlen = a.max_seqlen;
  p.G = a.num_q_heads / a.num_kv_heads;
  p.H = a.num_kv_heads;
  p.scale2 = a.sm_scale * 1.4426950408889634f;
  p.err_flags = a.err_flags;
  return launch_overlapped(prompt_attention_kernel, dim3(static_cast<unsigned>(prompt_units(a))),
                           dim3(kPrWarps * 32), 0, stream, p);
}

}  // namespace kvq
