// kvq_prompt.cu -- causal attention of packed prompts over their own bf16 keys
// and values (grouped query heads, sequences of different lengths in one token
// buffer), before anything is read from the cache, on the 5th-generation
// tensor cores.
//
//   out_i = sum_{j <= i} p_j v_j / sum_{j <= i} p_j,  p_j = 2^(c (q_i . k_j - m_i) - 16),
//   c = sm_scale log2(e), m_i a running reference within 16 / c of the row's maximum
//
//  * A unit of work is two 128-row tiles of one sequence and KV head.  The G
//    query heads that share a KV head are stacked: row t G + g of a tile is
//    token t, head h G + g, with floor(128 / G) tokens per tile, so short
//    prompts fill the tensor core's rows and a key tile is read once for all G
//    heads.  The unit's key tiles (128 keys) go from its diagonal down to 0.
//    Two chains (QK^T -> softmax -> PV) work on it, one per row tile; where a
//    call has few units, on one row tile, each over every other key tile, their
//    sums and outputs joined at the end (launch_prompt_attention has the rule).
//  * Units are numbered through the sequences; every CTA sums their counts in
//    shared memory, so there is no plan launch and no workspace.  (Cutting the
//    packed tokens instead, with rows of several sequences in one tile, took 9 us
//    instead of 15 for 64 prompts of 16 tokens, but 348 us instead of the 322 of
//    the time for 8 of 355 to 4,096 and 64 heads: diagonals that no longer end with
//    a key tile.)  Of more than kPtSeqs sequences, whose counts would not fit, s
//    uses the numbers floor(cu[s] / TU) + s up to the next one's (TU tokens a
//    unit), at least ceil(len / TU) of them, and a number finds its sequence by a
//    search over cu_seqlens itself, with no bound on their count; the numbers left
//    over cost a look each.  (Searched so, 64 prompts of 16 tokens take 16.3 us,
//    not 14.1, and 2,048 of up to 64 tokens 105, not 79.)
//  * CTAs of 512 threads, one per SM, that go on with the units of blocks that
//    have not started (cluster launch control) until there are none, longest
//    rows of a sequence first.  Warps 0-3 and 4-7: softmax of chain 0 and 1 (a
//    thread owns a TMEM lane, a row); 8-11: the epilogue, which overlaps the next
//    unit; 12: work numbers and TMA; 13 and 14: the MMAs of chain 0 and 1; 15:
//    clears what the edge value tiles must not contribute.
//  * S = Q K^T (128 x 128 x 128, both operands from shared memory) into TMEM;
//    the softmax reads S, writes P as bf16 over S's own columns, and O += P V
//    takes P from TMEM.  The chains alternate on the tensor core: PV and the next
//    QK^T of one run while the other is in its softmax.  Each has an issuing warp
//    of its own, since the pipe takes an MMA about when it starts: whatever one
//    warp spends on barriers, the other's MMAs fill (one warp for both left the
//    tensor core idle for 60% of the time).
//  * A row's reference m moves only when a score passes it by 2^16 in the
//    exponent (with 2^8 the rows of the ragged batch moved often enough to take
//    328 us, not 323).  The exponents are 16 lower for it, so that P, as in the
//    formula under the maximum itself, is at most 1 and no sum passes
//    sum_j |v_j|.  (At the other end, probabilities below 2^-110 are 0, and products
//    with values below 2^-110 are subnormal, which the tensor cores keep.)  The
//    thread that moves it rescales its O row, with no PV in flight on it since
//    the QK^T that it waited for was issued after it.  P is rounded to bf16 for
//    the product (2^-8 of each term at most, the tensor core's operand type) and
//    not for the sum.
//  * 0 times an infinity is not 0, so zero probabilities do not hide unseen
//    values.  Of the value tiles that some row of the unit does not see whole
//    warp 15 clears the rows that none sees, and in the rows that some see every
//    infinity and NaN; the epilogue adds those a row does see back, whatever
//    their probability (rare, one flag per unit).
//  * What bounds it: the tensor core, and on large calls the card's 1.4 kW
//    (1.78-1.94 GHz in a loop), so that a few calls are faster than a loop:
//    16,381 tokens of 32 heads 1.32-1.36 ms and 1.36-1.40 (1,570-1,670 TFLOP/s, 82
//    to 87% of what a bf16 library product reaches in a burst); 4 x 8,192 tokens
//    1.33-1.38 and 1.40-1.44; the ragged batch of 64 heads 305 and 334 us (figures
//    of it here are of a few calls).  A step of two row tiles over a key tile takes
//    about 2,700 cycles: MMAs of 2,048, and at each of the two hand-overs some 300
//    of waiting for the turn and for the second half of P.  A change of units takes
//    some 5,000 more (queries from memory, a masked softmax, an epilogue of 2,500 a tile).
//    Short prompts are bound by latency, 2 us to the first MMA, 1.5 us a step, 1 us
//    for the rows (64 tokens take 6.4 us in a graph; calls one after the other from
//    Python wait for the binding, 8.4 us each).
//  * Code that runs once a unit is kept in one copy (one search for units, one
//    epilogue for both chains): the roles share an instruction cache, and with
//    two copies 8 x 1,024 tokens take 86 us instead of 83, the short ragged batch
//    28.5 instead of 27.7.
//  * Every wait is bounded; a role that gives up raises a shared abort flag,
//    copies and MMAs in flight complete, the CTA frees its tensor memory
//    (KVQ_ERRF_WAIT_TIMEOUT).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kPtKeys = 128;                          // keys of a tile
constexpr int kPtStages = 4;                          // ring: key tiles in even stages, values in odd
constexpr int kPtWarpEpi = 8, kPtWarpLoad = 12, kPtWarpMma = 13, kPtWarpClear = 15;
constexpr int kPtThreads = 512;
constexpr int kPtUnits = 4;                           // units ahead
constexpr int kPtSeqs = 2048;                         // sequences whose units are summed
constexpr float kPtLazy = 16.0f;                       // a row's maximum over its reference, log2

// shared memory, offsets from a 1024-byte aligned base
constexpr int kPtTileBytes = 128 * kHeadDim * 2;      // [2 halves of 64 dims][128 rows][128 B]
constexpr int kPtHalf = kPtTileBytes / 2;
constexpr int kPtOffQ = 0;
constexpr int kPtOffKv = 2 * kPtTileBytes;
constexpr int kPtOffSum = kPtOffKv + kPtStages * kPtTileBytes;   // [chain][128] denominators
constexpr int kPtOffRef = kPtOffSum + 2 * 128 * 4;               // [chain][128] references
constexpr int kPtOffUnit = kPtOffRef + 2 * 128 * 4;
constexpr int kPtOffDirty = kPtOffUnit + kPtUnits * 16;
constexpr int kPtOffSteal = kPtOffDirty + kPtUnits * 4;          // two answers of 16 bytes
constexpr int kPtOffMisc = kPtOffSteal + 32;                     // tmem base, abort
constexpr int kPtOffScan = kPtOffMisc + 16;                      // a warp's sum each
constexpr int kPtOffPre = kPtOffScan + 16 * 4;                   // units before each sequence
constexpr int kPtOffCu = kPtOffPre + (kPtSeqs + 1) * 4;          // cu_seqlens
constexpr int kPtOffBar = (kPtOffCu + (kPtSeqs + 1) * 4 + 7) / 8 * 8;
enum : int {
  kPtKvFull = 0,
  kPtKvEmpty = kPtKvFull + kPtStages,
  kPtQFull = kPtKvEmpty + kPtStages,                  // per chain, as the next six
  kPtQEmpty = kPtQFull + 2,
  kPtSFull = kPtQEmpty + 2,
  kPtPReady = kPtSFull + 2,
  kPtOFull = kPtPReady + 4,                           // (P: per chain and half of the keys)
  kPtOEmpty = kPtOFull + 2,
  kPtSumFull = kPtOEmpty + 2,
  kPtVClear = kPtSumFull + 2,                         // per ring stage
  kPtUnitFull = kPtVClear + kPtStages,
  kPtUnitEmpty = kPtUnitFull + kPtUnits,
  kPtDrain = kPtUnitEmpty + kPtUnits,                 // per chain
  kPtTurn = kPtDrain + 2,                             // per chain
  kPtSteal = kPtTurn + 2,                             // per answer
  kPtBars = kPtSteal + 2
};
constexpr int kPtSmem = kPtOffBar + 8 * kPtBars + 1024;
static_assert(kPtOffBar % 8 == 0 && kPtOffUnit % 16 == 0 && kPtOffSteal % 16 == 0, "alignment");
static_assert(kPtSmem <= 227 * 1024, "shared memory budget");
static_assert(kPtSeqs >= 32, "a warp counts the units of up to 32 sequences");

// TMEM: S of chain a at 128 a (its P over the first 64 columns), O at 256 + 128 a
constexpr uint32_t kPtTmemCols = 512;
__device__ __forceinline__ uint32_t pt_s(int a) { return 128u * a; }
__device__ __forceinline__ uint32_t pt_o(int a) { return 256u + 128u * a; }

constexpr uint32_t kPtBf16 = (1u << 7) | (1u << 10);   // A and B bf16
constexpr uint32_t kPtIdescQK = mma_idesc(128, kPtKeys, false, false) | kPtBf16;
constexpr uint32_t kPtIdescPV = mma_idesc(128, kHeadDim, false, true) | kPtBf16;

// The upper word of every operand's shared-memory descriptor (smem_desc:
// stride offset 1024, version 1, 128-byte swizzle) and the two leading offsets.
constexpr uint32_t kPtDescHi = (1024u >> 4) | (1u << 14) | (kSmemSwizzle128 << 29);
constexpr uint32_t kPtKMajor = 1u << 16, kPtMnMajor = (kPtHalf >> 4) << 16;

// S (+)= Q K^T and O (+)= P V, 16 dims or keys each: the descriptors' lower
// words vary, the rest is constant (an issuing warp's time goes by the
// instructions around each MMA).
__device__ __forceinline__ void pt_mma_qk(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n"
      :: "r"(d), "r"(a_lo), "r"(b_lo), "n"(kPtIdescQK), "r"(acc), "n"(kPtDescHi) : "memory");
}
__device__ __forceinline__ void pt_mma_pv(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n"
      :: "r"(d), "r"(a_tmem), "r"(b_lo), "n"(kPtIdescPV), "r"(acc), "n"(kPtDescHi) : "memory");
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool pt_elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(r));
  return r != 0;
}

struct PromptParams {
  const uint16_t *v;
  uint16_t *out;
  int64_t v_stride, out_stride;
  int32_t num_tokens;
  const int32_t *cu;
  int32_t N, max_seqlen, G, H;
  int32_t TQ;                                          // tokens of a row tile: 128 / G
  int32_t TU;                                          // of a unit: one or two tiles
  int32_t inv_g;                                       // ceil(65536 / G)
  uint64_t h_magic;                                    // ceil(2^h_shift / H): n / H for n < 2^31
  int32_t h_shift;                                     // 32 + ceil(log2(H))
  float scale2;                                        // sm_scale log2(e)
  int32_t out_by_32;                                   // out rows are 32-byte aligned
  int32_t *err_flags;
};

__device__ __forceinline__ float pt_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pt_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pt_fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint64_t pt_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Bounded wait that also gives up once another role raised the abort flag.
__device__ __forceinline__ bool pt_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort) {
#pragma unroll 1
  for (int i = 0; i < (1 << 19); ++i) {
    if (mbar_try_wait_sleep(bar, parity, 2000u)) return true;
    if ((i & 15) == 15 && *abort) return false;
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool pt_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
  return mbar_try_wait(bar, parity) || pt_wait_slow(bar, parity, abort);
}

// The whole warp's (every lane tries; one that gives up speaks for all).
__device__ __forceinline__ bool pt_wait_all(uint32_t bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xFFFFFFFFu, pt_wait(bar, parity, abort));
}

// A unit: sequence rows [start, start + len), KV head h, queries from token tok0
// (within the sequence) on; len = 0 ends the work.  `a` is one of the two chains
// (QK^T, softmax, PV, O): a row tile each over all the key tiles or, where the
// keys are split, the same row tile over every other key tile.
template <bool kSplit>
struct PtUnit {
  int start, len, h, tok0;
  int n0, n1;                                          // key tiles of row tile 0 and 1
  __device__ __forceinline__ void shape(const int4 e, int TQ) {
    start = e.x;
    len = e.y;
    h = e.z;
    tok0 = e.w;
    const int t0 = min(len, tok0 + TQ), t1 = min(len, tok0 + 2 * TQ);
    n0 = (t0 + kPtKeys - 1) / kPtKeys;
    n1 = !kSplit && t1 > t0 ? (t1 + kPtKeys - 1) / kPtKeys : 0;
  }
  __device__ __forceinline__ int tiles() const { return kSplit ? n0 : max(n0, n1); }
  // steps: key tiles, or pairs of them
  __device__ __forceinline__ int steps() const { return kSplit ? (n0 + 1) / 2 : max(n0, n1); }
  // chain a's key tiles, from the top: top(a) (-1: none), ..., bottom(a)
  __device__ __forceinline__ int top(int a) const {
    return kSplit ? n0 - 1 - a : (a == 0 ? n0 : n1) - 1;
  }
  __device__ __forceinline__ int bottom(int a) const { return kSplit ? (n0 - 1 - a) & 1 : 0; }
  __device__ __forceinline__ int row_tile(int a) const { return kSplit ? 0 : a; }
  // keys of key tile j that some row sees
  __device__ __forceinline__ int keys(int j, int TQ) const {
    return min(kPtKeys, min(len, tok0 + (kSplit ? 1 : 2) * TQ) - j * kPtKeys);
  }
  // key tile j has a key that the unit's first row does not see
  __device__ __forceinline__ bool edge(int j) const { return j * kPtKeys + kPtKeys - 1 > tok0; }
};

__device__ __forceinline__ bool pt_bounds_ok(const PromptParams &p, int begin, int end) {
  return begin >= 0 && end >= begin && end <= p.num_tokens && end - begin <= p.max_seqlen;
}

// The last i in [lo, hi) with below(i), which holds up to some i; -1 if none.
// All lanes of a warp.
template <typename F>
__device__ __forceinline__ int pt_last(int lo, int hi, int lane, F below) {
  for (;;) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + lane * step;
    const int c = __ffs(~__ballot_sync(0xFFFFFFFFu, i < hi && below(i))) - 1;
    const int cnt = c < 0 ? 32 : c;                    // leading lanes below
    if (cnt == 0) return -1;
    lo += (cnt - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) return lo;
  }
}

__device__ __forceinline__ int pt_units_of(int len, int TU) {
  return len / TU + (len % TU != 0 ? 1 : 0);
}

// Inclusive sums over a warp.
__device__ __forceinline__ int pt_scan(int n, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, n, off);
    if (lane >= off) n += v;
  }
  return n;
}

// Work number w as a unit (len 0: none there).  All lanes of a warp.
__device__ __forceinline__ int4 pt_find(const PromptParams &p, const int *pre, const int *cu_s,
                                        uint32_t w, int lane) {
  const int TU = p.TU;
  const uint32_t x = static_cast<uint32_t>((static_cast<uint64_t>(w) * p.h_magic) >> p.h_shift);
  const int h = static_cast<int>(w - x * static_cast<uint32_t>(p.H));      // w % H
  int s, a, b;
  int64_t u;                                           // within the sequence, longest rows first
  if (p.N <= kPtSeqs) {
    if (x >= static_cast<uint32_t>(pre[p.N])) return make_int4(0, 0, 0, 0);
    s = pt_last(0, p.N, lane, [&](int i) { return static_cast<uint32_t>(pre[i]) <= x; });
    a = cu_s[s];
    b = cu_s[s + 1];
    u = static_cast<int64_t>(pre[s + 1]) - 1 - x;
  } else {
    s = pt_last(0, p.N, lane, [&](int i) {
      return static_cast<int64_t>(__ldg(p.cu + i) / TU) + i <= x;
    });
    if (s < 0) return make_int4(0, 0, 0, 0);
    a = __ldg(p.cu + s);
    b = __ldg(p.cu + s + 1);
    if (!pt_bounds_ok(p, a, b)) return make_int4(0, 0, 0, 0);
    u = pt_units_of(b - a, TU) - 1 - (x - (static_cast<int64_t>(a / TU) + s));
  }
  if (u < 0 || u * TU >= b - a) return make_int4(0, 0, 0, 0);
  return make_int4(a, b - a, h, static_cast<int>(u) * TU);
}

__device__ __forceinline__ void pt_tma_4d(uint32_t dst, const void *tmap, int x, int y, int z,
                                          int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];\n"
      :: "r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar) : "memory");
}

__device__ __forceinline__ void pt_prefetch_map(const void *tmap) {
  asm volatile("prefetch.tensormap [%0];\n" :: "l"(tmap) : "memory");
}

// 64 bytes of an output row, in whole 32-byte sectors where it is aligned (in
// halves of them, the ragged batch of 64 heads takes 319 us, not 309).
__device__ __forceinline__ void pt_store64(uint16_t *dst, const uint32_t (&w)[16], bool by_32) {
  if (by_32) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n"
                   :: "l"(dst + 2 * i), "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]),
                      "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7]) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<uint4 *>(dst + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// Asks for the number of a block of this grid that has not started, which then
// never starts; the answer (16 bytes) completes on `bar`.
__device__ __forceinline__ void pt_steal(uint32_t answer, uint32_t bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
      " [%0], [%1];\n" :: "r"(answer), "r"(bar) : "memory");
}
// The answer: a block number, or -1 once every block has started.
__device__ __forceinline__ int pt_stolen(uint32_t answer) {
  uint32_t some, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      " selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
      : "=r"(some), "=r"(x) : "r"(answer) : "memory");
  return some != 0 ? static_cast<int>(x) : -1;
}

// The running statistics of one row.
struct PtRow {
  float m = -INFINITY;                                 // reference
  float sum = 0.0f;                                    // denominator under it

  // The reference moved to a tile's maximum `top` where that is far above it,
  // the denominator and (unless fresh) the O row brought under the new one;
  // returns the shift of the exponents.
  __device__ __forceinline__ float meet(float top, float scale2, bool fresh, uint32_t ocol) {
    const bool unset = m == -INFINITY;
    const bool move = unset ? top > -INFINITY : (top - m) * scale2 > kPtLazy;
    if (__any_sync(0xFFFFFFFFu, move && !unset)) {
      // (rows of the warp that stay multiply by 1)
      const float f = (move && !unset) ? pt_ex2((m - top) * scale2) : 1.0f;
      sum *= f;
      if (!fresh) {
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 16) {
          float o[16];
          tmem_ld16(ocol + c, o);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] *= f;
          tmem_st16(ocol + c, o);
        }
      }
    }
    if (move) m = top;
    return m == -INFINITY ? 0.0f : fmaf(-m, scale2, -kPtLazy);
  }
};

// P of 32 scores as bf16 in 16 columns, its sum added to `sum`.
__device__ __forceinline__ void pt_part(const uint32_t (&x)[32], uint32_t col, uint64_t scale,
                                        uint64_t shift, uint64_t (&sum)[2]) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a, b;
    unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                           scale, shift), a, b);
    a = pt_ex2(a);
    b = pt_ex2(b);
    sum[i & 1] = pt_add2(sum[i & 1], pack_f32x2(a, b));
    w[i] = pack_bf16x2(a, b);
  }
  tmem_st16u(col, w);
}

// 64 keys of P are in TMEM.
__device__ __forceinline__ void pt_announce(uint32_t bar, int lane) {
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// One key tile of one row whose warp sees all its keys: S from TMEM, the row's
// statistics brought up to date, P as bf16 over S's columns, its two halves
// announced one after the other.
__device__ __forceinline__ void pt_softmax(uint32_t scol, uint32_t ocol, float scale2, bool fresh,
                                           uint32_t ready, int lane, PtRow &row) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int c = 0; c < 128; c += 64) {
    float x[64];
    tmem_ld64(scol + c, x);
#pragma unroll
    for (int i = 0; i < 64; i += 8)
#pragma unroll
      for (int q = 0; q < 4; ++q) mx[q] = pt_max3(mx[q], x[i + q], x[i + q + 4]);
  }
  uint32_t x0[32], x1[32];
  tmem_ld32_start(scol, x0);
  const float top = fmaxf(pt_max3(mx[0], mx[1], mx[2]), mx[3]);
  const float shift = row.meet(top, scale2, fresh, ocol);
  const uint64_t sc = pack_f32x2(scale2, scale2), sh = pack_f32x2(shift, shift);
  uint64_t sum[2] = {pack_f32x2(0.0f, 0.0f), pack_f32x2(0.0f, 0.0f)};
  tmem_ld32_done(x0);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    tmem_ld32_start(scol + 64 * h + 32, x1);
    pt_part(x0, scol + 32 * h, sc, sh, sum);
    tmem_ld32_done(x1);
    if (h == 0) tmem_ld32_start(scol + 64, x0);
    pt_part(x1, scol + 32 * h + 16, sc, sh, sum);
    if (h == 0) tmem_ld32_done(x0);
    pt_announce(ready + 8 * h, lane);
  }
  float a, b;
  unpack_f32x2(pt_add2(sum[0], sum[1]), a, b);
  row.sum += a + b;
}

// The same for a tile whose keys some of the warp's rows do not see: the row
// sees the keys lo .. hi, counted within the tile, and both rise along the rows.
// 32 keys at a time; the scores of parts that no row sees are not read and
// their P is 0.
__device__ __forceinline__ void pt_softmax_edge(uint32_t scol, uint32_t ocol, int hi,
                                                float scale2, bool fresh, uint32_t ready, int lane,
                                                PtRow &row) {
  const int hi0 = __shfl_sync(0xFFFFFFFFu, hi, 0), hi31 = __shfl_sync(0xFFFFFFFFu, hi, 31);
  const int parts = hi31 < 0 ? 0 : min(4, hi31 / 32 + 1);
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int c = 0; c < 32 * parts; c += 32) {
    float x[32];
    tmem_ld32(scol + c, x);
    if (hi0 < c + 31) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = i <= hi - c ? x[i] : -INFINITY;
      tmem_st32(scol + c, x);
    }
#pragma unroll
    for (int i = 0; i < 32; i += 8)
#pragma unroll
      for (int q = 0; q < 4; ++q) mx[q] = pt_max3(mx[q], x[i + q], x[i + q + 4]);
  }
  tmem_wait_st();
  const float top = fmaxf(pt_max3(mx[0], mx[1], mx[2]), mx[3]);
  const float shift = row.meet(top, scale2, fresh, ocol);
  const uint64_t sc = pack_f32x2(scale2, scale2), sh = pack_f32x2(shift, shift);
  uint64_t sum[2] = {pack_f32x2(0.0f, 0.0f), pack_f32x2(0.0f, 0.0f)};
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    if (i < parts) {
      uint32_t x[32];
      tmem_ld32_start(scol + 32 * i, x);
      tmem_ld32_done(x);
      pt_part(x, scol + 16 * i, sc, sh, sum);
    } else {
      uint32_t w[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = 0u;
      tmem_st16u(scol + 16 * i, w);
    }
    if (i & 1) pt_announce(ready + 8 * (i >> 1), lane);
  }
  float a, b;
  unpack_f32x2(pt_add2(sum[0], sum[1]), a, b);
  row.sum += a + b;
}

template <bool kSplit>
__global__ void __launch_bounds__(kPtThreads, 1)
prompt_attention_kernel(const PromptParams p, const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bar0 = smem_addr(smem + kPtOffBar);
  auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kPtOffMisc);
  volatile int *abort_s = reinterpret_cast<volatile int *>(smem + kPtOffMisc + 4);
  volatile int *dirty_s = reinterpret_cast<volatile int *>(smem + kPtOffDirty);
  int4 *unit_s = reinterpret_cast<int4 *>(smem + kPtOffUnit);
  volatile float *ref_s = reinterpret_cast<volatile float *>(smem + kPtOffRef);
  volatile float *sum_s = reinterpret_cast<volatile float *>(smem + kPtOffSum);

  allow_dependents_launch();
  if (tid < kPtBars) {
    uint32_t count = 1;
    if (tid >= kPtKvEmpty && tid < kPtKvEmpty + kPtStages)
      count = (kSplit ? 1 : 2) + ((tid - kPtKvEmpty) & 1);   // the chains; value tiles: warp 15 too
    if ((tid >= kPtPReady && tid < kPtPReady + 4) || (tid >= kPtOEmpty && tid < kPtOEmpty + 2) ||
        (tid >= kPtSumFull && tid < kPtSumFull + 2))
      count = 4;                                       // a warp each of the softmax or epilogue
    if (tid >= kPtUnitEmpty && tid < kPtUnitEmpty + kPtUnits)
      count = 8 + 4 + 3;                               // softmax, epilogue, warps 13-15
    mbar_init(BAR(tid), count);
    fence_mbarrier_init();
  }
  if (tid == 0) *abort_s = 0;
  if (tid == 64) {
    pt_prefetch_map(&tm_q);
    pt_prefetch_map(&tm_k);
    pt_prefetch_map(&tm_v);
  }
  if (warp == kPtWarpLoad) {
    tmem_alloc(smem_addr(tmem_slot), kPtTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  int *pre = reinterpret_cast<int *>(smem + kPtOffPre);
  int *cu_s = reinterpret_cast<int *>(smem + kPtOffCu);
  // Units of sequence i, which is flagged if it is not to be computed.
  auto count_units = [&](int i) -> int {
    const int a = __ldg(p.cu + i), b = __ldg(p.cu + i + 1);
    cu_s[i] = a;
    cu_s[i + 1] = b;
    if (pt_bounds_ok(p, a, b)) return pt_units_of(b - a, p.TU);
    if (p.err_flags) atomicOr(p.err_flags, KVQ_ERRF_SEQUENCE_RANGE);
    return 0;
  };
  if (p.N <= 32) {
    // the loading warp alone, which is the one to use them (with every warp and
    // its barriers, one prompt of 64 tokens took 7.5 us, not 7.1)
    if (warp == kPtWarpLoad) {
      int n = lane < p.N ? count_units(lane) : 0;
      n = pt_scan(n, lane);
      if (lane < p.N) pre[lane + 1] = n;
      if (lane == 0) pre[0] = 0;
      __syncwarp();
    }
  } else if (p.N <= kPtSeqs) {
    int *warp_sum = reinterpret_cast<int *>(smem + kPtOffScan);
    int carry = 0;
    for (int s0 = 0; s0 < p.N; s0 += kPtThreads) {
      const int i = s0 + tid;
      const int n = pt_scan(i < p.N ? count_units(i) : 0, lane);
      if (lane == 31) warp_sum[warp] = n;
      __syncthreads();
      int before = carry;
#pragma unroll
      for (int k = 0; k < kPtThreads / 32; ++k) {
        const int v = warp_sum[k];
        if (k < warp) before += v;
        carry += v;
      }
      if (i < p.N) pre[i + 1] = before + n;
      __syncthreads();
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
  }

  // Unit `t` of this CTA; the caller's warp (or lone lane) releases its entry.
  using Unit = PtUnit<kSplit>;
  auto take_unit = [&](int t, Unit &u) -> bool {
    const int e = t % kPtUnits;
    if (!pt_wait(BAR(kPtUnitFull + e), (t / kPtUnits) & 1, abort_s)) return false;
    u.shape(unit_s[e], p.TQ);
    return true;
  };
  bool gave_up = false;

  if (warp < kPtWarpEpi) {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n");
    const int a = warp >> 2;
    const int m = tid & 127;                           // row of the tile, TMEM lane
    const int t_row = (m * p.inv_g) >> 16;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    uint32_t steps = 0, done = 0;                      // key tiles and units of tile a
    for (int t = 0;; ++t) {
      Unit u;
      const bool ok = take_unit(t, u);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        gave_up = true;
        break;
      }
      if (lane == 0) mbar_arrive(BAR(kPtUnitEmpty + t % kPtUnits));
      if (u.len == 0) break;
      const int top = u.top(a), bottom = u.bottom(a);
      if (top < 0) continue;
      const int tok = u.tok0 + u.row_tile(a) * p.TQ + t_row;
      // the key tiles that all of the warp's rows see whole (the first row sees least)
      const int whole = (__shfl_sync(0xFFFFFFFFu, tok, 0) + 1) / kPtKeys;
      PtRow row;
      for (int j = top; j >= bottom; j -= kSplit ? 2 : 1, ++steps) {
        if (__any_sync(0xFFFFFFFFu, !pt_wait(BAR(kPtSFull + a), steps & 1, abort_s))) {
          gave_up = true;
          break;
        }
        tc_fence_after();
        if (j < whole)
          pt_softmax(tl + pt_s(a), tl + pt_o(a), p.scale2, j == top, BAR(kPtPReady + 2 * a), lane,
                     row);
        else
          pt_softmax_edge(tl + pt_s(a), tl + pt_o(a), tok - j * kPtKeys, p.scale2, j == top,
                          BAR(kPtPReady + 2 * a), lane, row);
      }
      if (gave_up) break;
      // the row's statistics, once the epilogue has read the last unit's
      if (done > 0 &&
          __any_sync(0xFFFFFFFFu, !pt_wait(BAR(kPtOEmpty + a), (done - 1) & 1, abort_s))) {
        gave_up = true;
        break;
      }
      sum_s[128 * a + m] = row.sum;
      if (kSplit) ref_s[128 * a + m] = row.m;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(kPtSumFull + a));
      ++done;
    }
  } else if (warp < kPtWarpLoad) {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;\n");
    const int q4 = warp & 3;
    const int m = 32 * q4 + lane;
    const int t_row = (m * p.inv_g) >> 16;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    uint32_t par = 0;                                  // barrier parities, bit a
    for (int t = 0;; ++t) {
      Unit u;
      const bool ok = take_unit(t, u);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        gave_up = true;
        break;
      }
      if (u.len == 0) break;
#pragma unroll 1
      for (int a = 0; a < (kSplit ? 1 : 2); ++a) {
        if (u.top(a) < 0) continue;
        const bool both = kSplit && u.top(1) >= 0;
        bool got = pt_wait(BAR(kPtSumFull + a), (par >> a) & 1, abort_s) &&
                   pt_wait(BAR(kPtOFull + a), (par >> a) & 1, abort_s);
        if (both)
          got = got && pt_wait(BAR(kPtSumFull + 1), par >> 1, abort_s) &&
                pt_wait(BAR(kPtOFull + 1), par >> 1, abort_s);
        if (__any_sync(0xFFFFFFFFu, !got)) {
          gave_up = true;
          break;
        }
        tc_fence_after();
        par ^= 1u << a;
        float inv = sum_s[128 * a + m], inv_b = 0.0f;
        if (both) {
          // the two chains' sums and outputs under the larger reference (of a row
          // that saw no key of a chain, nothing)
          par ^= 2u;
          const float m0 = ref_s[m], m1 = ref_s[128 + m], top = fmaxf(m0, m1);
          const float f0 = m0 == -INFINITY ? 0.0f : pt_ex2((m0 - top) * p.scale2);
          const float f1 = m1 == -INFINITY ? 0.0f : pt_ex2((m1 - top) * p.scale2);
          const float all = 1.0f / (f0 * inv + f1 * sum_s[128 + m]);
          inv = f0 * all;
          inv_b = f1 * all;
        } else {
          inv = 1.0f / inv;
        }
        const int tok = u.tok0 + u.row_tile(a) * p.TQ + t_row;
        const bool dirty = dirty_s[t % kPtUnits] != 0;
        const bool mine = t_row < p.TQ && tok < u.len;
        uint16_t *dst = p.out + (static_cast<int64_t>(u.start) + tok) * p.out_stride +
                        (static_cast<int64_t>(u.h) * p.G + (m - t_row * p.G)) * kHeadDim;
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 32) {
          float o[32];
          tmem_ld32(tl + pt_o(a) + c, o);
          const uint64_t inv2 = pack_f32x2(inv, inv);
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            unpack_f32x2(mul_f32x2(pack_f32x2(o[i], o[i + 1]), inv2), o[i], o[i + 1]);
          if (both) {
            float o1[32];
            tmem_ld32(tl + pt_o(1) + c, o1);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(o1[i], inv_b, o[i]);
          }
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
          if (mine) pt_store64(dst + c, w, p.out_by_32);
        }
        if (dirty && mine) {
          // the infinities and NaN this row sees of the cleared rows, added to what
          // was stored (rare, and little code)
#pragma unroll 1
          for (int j = u.tok0 + 1; j <= tok; ++j) {
            const uint16_t *vr = p.v + (static_cast<int64_t>(u.start) + j) * p.v_stride + u.h * kHeadDim;
#pragma unroll 1
            for (int d = 0; d < kHeadDim; d += 8) {
              const uint4 x = __ldg(reinterpret_cast<const uint4 *>(vr + d));
              const uint32_t sum = pt_fma_bf16x2(x.x, 0u, 0u) | pt_fma_bf16x2(x.y, 0u, 0u) |
                                   pt_fma_bf16x2(x.z, 0u, 0u) | pt_fma_bf16x2(x.w, 0u, 0u);
              if ((sum & 0x7FFF7FFFu) == 0u) continue;
#pragma unroll 1
              for (int i = d; i < d + 8; ++i)
                if ((vr[i] & 0x7F80u) == 0x7F80u)
                  dst[i] = static_cast<uint16_t>(pack_bf16x2(bf16_lo(dst[i]) + bf16_lo(vr[i]), 0.0f));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(BAR(kPtOEmpty + a));
          if (both) mbar_arrive(BAR(kPtOEmpty + 1));
        }
      }
      if (gave_up) break;
      // (held to here: the entry's dirty flag is the unit's until it is taken again)
      if (lane == 0) mbar_arrive(BAR(kPtUnitEmpty + t % kPtUnits));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
    if (warp == kPtWarpLoad) {
      // ----------------------------------------------- work numbers and TMA
      uint32_t loads0 = 0, loads1 = 0;                 // query tiles of each chain
      // Units: the own block's first, then those of blocks that have not
      // started.  Answers are asked for before a unit's last two tiles are loaded
      // (any earlier, and the CTAs that ask first hold work back from those that
      // finish first: asked one unit earlier, 1,999 tokens take 33.1 us instead of
      // 31.6), two of them if it has no more.
      const uint32_t steal = smem_addr(smem + kPtOffSteal);
      uint32_t asked = 0, heard = 0;
      bool more = true;
      auto ask = [&](uint32_t ahead) {
        for (; more && asked - heard < ahead; ++asked)
          if (lane == 0) pt_steal(steal + 16 * (asked & 1), BAR(kPtSteal + (asked & 1)));
        __syncwarp();
      };
      // the unit of work number w (none: the next answer's), or none (length 0)
      auto next_unit = [&](int w, int4 &e) -> bool {
        e = make_int4(0, 0, 0, 0);
#pragma unroll 1
        for (;;) {
          if (w >= 0) {
            // (every work number is somebody's, and there are more than sequences)
            if (p.N > kPtSeqs && lane == 0 && w < p.N && p.err_flags &&
                !pt_bounds_ok(p, __ldg(p.cu + w), __ldg(p.cu + w + 1)))
              atomicOr(p.err_flags, KVQ_ERRF_SEQUENCE_RANGE);
            e = pt_find(p, pre, cu_s, static_cast<uint32_t>(w), lane);
            if (e.y > 0) return true;
          }
          ask(1);
          if (asked == heard) return true;
          if (!pt_wait_all(BAR(kPtSteal + (heard & 1)), (heard >> 1) & 1, abort_s)) return false;
          w = pt_stolen(steal + 16 * (heard & 1));
          ++heard;
          fence_proxy_async_smem();
          __syncwarp();
          if (w < 0) more = false;                     // (an answer may still be under way)
        }
      };
      auto announce = [&](int t, const int4 e) -> bool {
        const int b = t % kPtUnits;
        if (t >= kPtUnits &&
            !pt_wait_all(BAR(kPtUnitEmpty + b), (t / kPtUnits - 1) & 1, abort_s))
          return false;
        if (lane == 0) {
          unit_s[b] = e;
          mbar_arrive(BAR(kPtUnitFull + b));
        }
        return true;
      };
      // key (kv = 0) or value tile j of the unit into ring stage b, round by round
      auto load_tile = [&](const Unit &u, int j, int kv, uint32_t b, uint32_t round) -> bool {
        if (round > 0 && !pt_wait(BAR(kPtKvEmpty + b), (round - 1) & 1, abort_s)) return false;
        mbar_arrive_expect_tx(BAR(kPtKvFull + b), kPtTileBytes);
        pt_tma_4d(smem_addr(smem + kPtOffKv + b * kPtTileBytes), kv == 0 ? &tm_k : &tm_v, 0,
                  u.start + j * kPtKeys, 0, u.h, BAR(kPtKvFull + b));
        return true;
      };
      // ring entries issued (split: each chain's keys and values; no arrays: they
      // would be in local memory, a cold miss at the kernel's start)
      uint32_t idx = 0, k0 = 0, k1 = 0, v0 = 0, v1 = 0;
      // the tiles of the unit's step i (split: from -1 on, with the first keys)
      auto load_step = [&](const Unit &u, int i) -> bool {
        bool ok = true;
        if constexpr (kSplit) {
          // chain 0's values of this step, its keys of the next, the same of chain 1:
          // the order in which their places come free (all keys, then all values: 1 x
          // 4,096 tokens of 4 heads take 43.4 us instead of 30.0; in a loop, 31.6)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int a = x >> 1, keys = x & 1;
            const int step = i + keys, j = u.top(a) - 2 * step;
            uint32_t &n = a == 0 ? (keys ? k0 : v0) : (keys ? k1 : v1);
            if (!ok || step < 0 || j < 0) continue;
            ok = load_tile(u, j, 1 - keys, 2 * a + 1 - keys, n);
            n += ok;
          }
        } else {
#pragma unroll 1
          for (int kv = 0; kv < 2 && ok; ++kv) {
            ok = load_tile(u, u.tiles() - 1 - i, kv, idx % kPtStages, idx / kPtStages);
            idx += ok;
          }
        }
        return ok;
      };
      auto load_q = [&](const Unit &u) -> bool {
        // the chains' last products with the tiles are done
        if (loads0 > 0 && !pt_wait(BAR(kPtQEmpty), (loads0 - 1) & 1, abort_s)) return false;
        if ((kSplit || u.top(1) >= 0) && loads1 > 0 &&
            !pt_wait(BAR(kPtQEmpty + 1), (loads1 - 1) & 1, abort_s))
          return false;
        ++loads0;
        loads1 += u.top(1) >= 0;
#pragma unroll 1
        for (int a = 0; a < (kSplit ? 1 : 2); ++a) {
          if (u.top(a) < 0) continue;
          const uint32_t dst = smem_addr(smem + kPtOffQ + a * kPtTileBytes);
          mbar_arrive_expect_tx(BAR(kPtQFull + a), 2u * 128u * p.TQ * p.G);
          for (int half = 0; half < 2; ++half)
            pt_tma_4d(dst + half * kPtHalf, &tm_q, 0, u.h * p.G, u.start + u.tok0 + a * p.TQ, half,
                      BAR(kPtQFull + a));
        }
        return true;
      };
      bool ok = true;
      int w = static_cast<int>(blockIdx.x);
      for (int t = 0; ok; ++t, w = -1) {
        int4 e;
        ok = next_unit(w, e);
        if (!ok) break;
        Unit u;
        u.shape(e, p.TQ);
        const int steps = u.steps();                   // (0: no unit)
        // (where the keys are split there hardly is a unit before, nor anything to
        // wait for)
        if (kSplit || steps == 0) ok = announce(t, e);
        if (steps == 0) break;
        for (int i = kSplit ? -1 : 0; i < steps && ok; ++i) {
          if (kSplit && i < 0 && lane == 0) ok = load_q(u);
          if (ok && lane == 0) ok = load_step(u, i);
          if (!kSplit && i == 0) {
            // the first keys and values ahead of the queries, whose tiles are free
            // only once the last unit's products with them are done (values last,
            // the ragged batch takes 319 us instead of 309)
            ok = __all_sync(0xFFFFFFFFu, ok) && announce(t, e);
            if (ok && lane == 0) ok = load_q(u);
          }
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (ok && i == max(steps - 3, 0)) ask(steps > 2 ? 1 : 2);
        }
      }
      gave_up = !ok;
      // copies in flight land before the CTA leaves
      if (lane == 0) {
#pragma unroll
        for (uint32_t b = 0; b < kPtStages; ++b) {
          // rounds of this stage so far
          const uint32_t n = kSplit ? (b == 0 ? k0 : (b == 1 ? v0 : (b == 2 ? k1 : v1)))
                                    : (idx + kPtStages - 1 - b) / kPtStages;
          if (n > 0) mbar_wait_sleep_bounded(BAR(kPtKvFull + b), (n - 1) & 1);
        }
        if (loads0 > 0) mbar_wait_sleep_bounded(BAR(kPtQFull), (loads0 - 1) & 1);
        if (!kSplit && loads1 > 0) mbar_wait_sleep_bounded(BAR(kPtQFull + 1), (loads1 - 1) & 1);
        for (; asked > heard; ++heard)
          mbar_wait_sleep_bounded(BAR(kPtSteal + (heard & 1)), (heard >> 1) & 1);
      }
    } else if (warp < kPtWarpClear) {
      // ---------------------------------------------------- MMAs of a chain
      // Each turn: PV of one key tile and QK^T of the next (a unit's first turn
      // has no PV, its last no QK^T), chain 0's and chain 1's bursts one after the
      // other (free to interleave, the chains fell into step: both in the softmax,
      // then both at the tensor core; 4 x 8,192 tokens 1.98 ms instead of 1.66).
      // Everything but P is waited for before the turn.  The warp stays
      // converged and elects a lane for each group of MMAs: addresses stay
      // uniform, 8 instructions an MMA instead of 11 for a lone lane.
      const int a = warp - kPtWarpMma;
      const uint32_t q_lo = (smem_addr(smem + kPtOffQ + (kSplit ? 0 : a) * kPtTileBytes) >> 4) | kPtKMajor;
      const uint32_t kv0 = smem_addr(smem + kPtOffKv) >> 4;
      const uint32_t s_col = tmem + pt_s(a), o_col = tmem + pt_o(a);
      uint32_t base = 0;                               // ring entries (split: tiles) of earlier units
      uint32_t par_q = 0, par_p = 0, par_o = 1;        // barrier parities
      uint32_t par_clear = 0;                          // bit per ring stage
      uint32_t par_turn = a ^ 1;                       // chain 0 goes first
      bool ok = true;
      // The next unit is taken while this one's last softmax runs (after its last
      // product, the ragged batch of 64 heads takes 320 us instead of 312); where the
      // keys are split there hardly is one.
      auto take = [&](int t, Unit &u) -> bool {
        if (!__all_sync(0xFFFFFFFFu, take_unit(t, u))) return false;
        if (lane == 0) mbar_arrive(BAR(kPtUnitEmpty + t % kPtUnits));
        return true;
      };
      Unit u, next;
      ok = take(0, u);
      for (int t = 0; ok && u.len != 0; ++t, u = next) {
        const int steps = u.steps(), top = u.top(a);
        const bool turns = u.top(1) >= 0;              // (a lone chain 0 need not pass them)
        // turn j: PV of one of the chain's key tiles (jv, none in the first turn) and
        // QK^T of the next (none in the last)
        for (int j = steps; j >= 0; --j) {
          int jv = j;
          bool pv = j <= top, qk = j > 0 && j - 1 <= top;
          bool pv_first = j == top, pv_last = j == 0, qk_first = j - 1 == top, qk_last = j == 1;
          // (not split: tiles that are only the other chain's are waited for and
          // released too)
          bool use_v = j < steps, use_k = j > 0;
          uint32_t ek = base + 2 * (steps - j);        // its entry in the ring; the values' is before
          uint32_t bk = ek % kPtStages, bv = (ek - 1) % kPtStages;
          uint32_t pk = ek / kPtStages, pvv = (ek - 1) / kPtStages;
          if (kSplit) {
            jv = top - 2 * (steps - j) + 2;
            const int jk = jv - 2, bottom = u.bottom(a);
            pv = use_v = j < steps && jv >= 0;
            qk = use_k = j > 0 && jk >= 0;
            pv_first = jv == top;
            pv_last = jv == bottom;
            qk_first = jk == top;
            qk_last = jk == bottom;
            bk = 2 * a;
            bv = bk + 1;
            pk = base + (steps - j);
            pvv = pk - 1;
          }
          const uint32_t v_lo = (kv0 + bv * (kPtTileBytes >> 4)) | kPtMnMajor;
          const uint32_t k_lo = (kv0 + bk * (kPtTileBytes >> 4)) | kPtKMajor;
          if (use_v) {
            ok = pt_wait_all(BAR(kPtKvFull + bv), pvv & 1, abort_s);
            if (u.edge(jv)) {
              if (ok && pv) ok = pt_wait_all(BAR(kPtVClear + bv), (par_clear >> bv) & 1, abort_s);
              par_clear ^= 1u << bv;
            }
          }
          if (ok && use_k) ok = pt_wait_all(BAR(kPtKvFull + bk), pk & 1, abort_s);
          if (ok && qk && qk_first) {
            // (split: the one tile of every unit)
            ok = pt_wait_all(BAR(kPtQFull + (kSplit ? 0 : a)), kSplit ? t & 1 : par_q, abort_s);
            par_q ^= 1u;
          }
          if (!kSplit && ok && j == 0) ok = take(t + 1, next);
          if (ok && pv) {
            if (pv_first) {
              ok = pt_wait_all(BAR(kPtOEmpty + a), par_o, abort_s);
              par_o ^= 1u;
            }
            ok = ok && pt_wait_all(BAR(kPtPReady + 2 * a), par_p, abort_s);
          }
          if (turns) {
            ok = ok && pt_wait_all(BAR(kPtTurn + a), par_turn, abort_s);
            par_turn ^= 1u;
          }
          if (!ok) break;
          if (pv) {
            // 64 keys at a time, as the softmax has them ready
            tc_fence_after();
            if (pt_elect()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                pt_mma_pv(o_col, s_col + 8 * kk, v_lo + (2048 >> 4) * kk,
                          (pv_first && kk == 0) ? 0u : 1u);
            }
            ok = pt_wait_all(BAR(kPtPReady + 2 * a + 1), par_p, abort_s);
            if (!ok) break;
            par_p ^= 1u;
            tc_fence_after();
            if (pt_elect()) {
#pragma unroll
              for (int kk = 4; kk < 8; ++kk)
                pt_mma_pv(o_col, s_col + 8 * kk, v_lo + (2048 >> 4) * kk, 1u);
            }
          }
          if (qk && pt_elect()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = (kk & 3) * 2 + (kk >> 2) * (kPtHalf >> 4);
              pt_mma_qk(s_col, q_lo + off, k_lo + off, kk != 0);
            }
            tc_commit(BAR(kPtSFull + a));
          }
          __syncwarp();
          if (pt_elect()) {
            if (turns) mbar_arrive(BAR(kPtTurn + (a ^ 1)));
            if (pv && pv_last) tc_commit(BAR(kPtOFull + a));
            if (qk && qk_last) tc_commit(BAR(kPtQEmpty + a));
            if (use_v) tc_commit(BAR(kPtKvEmpty + bv));
            if (use_k) tc_commit(BAR(kPtKvEmpty + bk));
          }
          __syncwarp();
        }
        base += kSplit ? (top >= 0 ? top / 2 + 1 : 0) : 2 * steps;
        if (kSplit && ok) ok = take(t + 1, next);
      }
      gave_up = !ok;
      // every MMA issued has completed before the tensor memory is freed
      __syncwarp();
      if (pt_elect()) tc_commit(BAR(kPtDrain + a));
      mbar_wait_sleep_bounded(BAR(kPtDrain + a), 0);
    } else {
      // ------------------------------------------- edge value tiles cleared
      uint32_t tiles0 = 0, tiles1 = 0;                 // of each chain (not split: of both)
      for (int t = 0; !gave_up; ++t) {
        Unit u;
        const bool ok = take_unit(t, u);
        if (__any_sync(0xFFFFFFFFu, !ok)) {
          gave_up = true;
          break;
        }
        if (lane == 0) {
          dirty_s[t % kPtUnits] = 0;
          mbar_arrive(BAR(kPtUnitEmpty + t % kPtUnits));
        }
        __syncwarp();
        if (u.len == 0) break;
        // (every value tile is waited for and released, or this warp could be
        // phases ahead of the ring or behind it)
        for (int j = u.tiles() - 1; j >= 0; --j) {
          const uint32_t e = 2 * tiles0 + 1;
          uint32_t b = e % kPtStages, round = e / kPtStages;
          if (kSplit) {
            const int a = (u.tiles() - 1 - j) & 1;
            b = 2 * a + 1;
            round = a == 0 ? tiles0 : tiles1;
            tiles0 += a ^ 1;
            tiles1 += a;
          } else {
            ++tiles0;
          }
          if (__any_sync(0xFFFFFFFFu, !pt_wait(BAR(kPtKvFull + b), round & 1, abort_s))) {
            gave_up = true;
            break;
          }
          if (!u.edge(j)) {
            if (lane == 0) mbar_arrive(BAR(kPtKvEmpty + b));
            continue;
          }
          uint8_t *tile = smem + kPtOffKv + b * kPtTileBytes;
          // the rows that some rows of the unit see and some do not
          const int lo = max(0, u.tok0 + 1 - j * kPtKeys), rows = u.keys(j, p.TQ);
          // 0 times the values, summed: NaN where one of them is not finite
          uint32_t sum0 = 0u, sum1 = 0u;
#pragma unroll 1
          for (int half = 0; half < 2; ++half)
#pragma unroll 1
            for (int r0 = lo; r0 < rows; r0 += 32) {
              uint4 w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = min(r0 + 4 * i + (lane >> 3), rows - 1);
                w[i] = *reinterpret_cast<const uint4 *>(tile + half * kPtHalf + r * 128 +
                                                         16 * (lane & 7));
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                sum0 = pt_fma_bf16x2(w[i].x, 0u, sum0);
                sum1 = pt_fma_bf16x2(w[i].y, 0u, sum1);
                sum0 = pt_fma_bf16x2(w[i].z, 0u, sum0);
                sum1 = pt_fma_bf16x2(w[i].w, 0u, sum1);
              }
            }
          if (__any_sync(0xFFFFFFFFu, ((sum0 | sum1) & 0x7FFF7FFFu) != 0u)) {
            if (lane == 0) dirty_s[t % kPtUnits] = 1;
            for (int r = 2 * lo; r < 2 * rows; ++r) {
              uint32_t *w = reinterpret_cast<uint32_t *>(tile + (r & 1) * kPtHalf + (r >> 1) * 128) + lane;
              uint32_t x = *w;
              if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
              if ((x & 0x7F800000u) == 0x7F800000u) x &= 0x0000FFFFu;
              *w = x;
            }
          }
          // the rows after them
          for (int r = rows + (lane >> 3); r < 128; r += 4) {
            *reinterpret_cast<uint4 *>(tile + r * 128 + 16 * (lane & 7)) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(tile + kPtHalf + r * 128 + 16 * (lane & 7)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(BAR(kPtVClear + b));
            mbar_arrive(BAR(kPtKvEmpty + b));
          }
        }
      }
    }
  }
  if (gave_up) {
    *abort_s = 1;
    if (lane == 0 && p.err_flags) atomicOr(p.err_flags, KVQ_ERRF_WAIT_TIMEOUT);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kPtWarpLoad) {
    tc_fence_after();
    // (read again: kept over the roles, the base spills)
    tmem_dealloc(*tmem_slot, kPtTmemCols);
  }
}

// Work numbers of a call with units of `tiles` row tiles: at least those.
int64_t prompt_units(const PromptArgs &a, int tiles) {
  const int64_t TU = tiles * (128 / (a.num_q_heads / a.num_kv_heads));
  int64_t n = a.num_tokens / TU + a.num_seqs;
  if (a.num_seqs <= kPtSeqs) {
    const int64_t most = (static_cast<int64_t>(a.max_seqlen) + TU - 1) / TU;
    n = std::min(n, a.num_seqs * std::max<int64_t>(most, 1));
  }
  return n * a.num_kv_heads;
}

}  // namespace

bool prompt_attention_supported(const PromptArgs &a) {
  // (a tensor map's strides are below 2^40 bytes)
  const int64_t most = int64_t(1) << 39;
  if (a.q_stride >= most || a.k_stride >= most || a.v_stride >= most) return false;
  return a.num_seqs <= 0x7FFFFF00 && prompt_units(a, 1) <= 0x7FFFFFFF;
}

cudaError_t launch_prompt_attention(const PromptArgs &a, cudaStream_t stream) {
  const int G = a.num_q_heads / a.num_kv_heads;
  PromptParams p;
  p.v = static_cast<const uint16_t *>(a.v);
  p.out = static_cast<uint16_t *>(a.out);
  p.v_stride = a.v_stride;
  p.out_stride = a.out_stride;
  p.num_tokens = static_cast<int32_t>(a.num_tokens);
  p.cu = a.cu_seqlens;
  p.N = a.num_seqs;
  p.max_seqlen = a.max_seqlen;
  p.G = G;
  p.H = a.num_kv_heads;
  p.TQ = 128 / G;
  p.inv_g = (65536 + G - 1) / G;
  int l = 0;
  while ((int64_t(1) << l) < p.H) ++l;
  p.h_shift = 32 + l;
  p.h_magic = ((uint64_t(1) << p.h_shift) + p.H - 1) / p.H;
  // Units of one row tile, its keys split between the two chains: twice the units
  // of half the steps.  That pays where they all start at once (8 KV heads of 4
  // query heads, 512 tokens, 128 units: 9.7 us against 12.3) and, while a second
  // unit hides behind the longest, somewhat beyond: the room grows with the key
  // tiles of a sequence, and falls with their number (numbers go sequence by
  // sequence, so long units start late).  152 SMs, not split against split: 1 x
  // 4,800 tokens, 300 units, 58 and 40 us; 1 x 640, 160 units, 13.9 and 11.5; 1 x
  // 900, 232 units, 16.9 and 18.4; 2 x 1,500, 188 units, 23.1 and 19.2; 3 x 1,000,
  // 192 units, 18.0 and 19.4; 4 x 350, 176 units, 11.0 and 12.6.  (Padding behind
  // the sequences is not theirs: 1 x 900 tokens in a buffer of 16,000, counted as
  // 16,000 and split, took 18.4 us instead of 17.0.)
  const int64_t tokens =
      std::min(a.num_tokens, static_cast<int64_t>(a.num_seqs) * a.max_seqlen);
  const int64_t room = 8 * tokens / kPtKeys / a.num_seqs / a.num_seqs;
  const bool split = prompt_units(a, 1) <= a.sms + std::min<int64_t>(a.sms, room);
  p.TU = (split ? 1 : 2) * p.TQ;
  const int64_t units = prompt_units(a, split ? 1 : 2);
  p.scale2 = a.sm_scale * 1.4426950408889634f;
  p.out_by_32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride % 16 == 0;
  p.err_flags = a.err_flags;
  CUtensorMap mq, mk, mv;
  if (!encode_head_tensor_map(&mq, a.q, a.num_tokens, a.num_q_heads, a.q_stride, G, p.TQ) ||
      !encode_row_tensor_map(&mk, a.k, a.num_tokens, a.num_kv_heads, a.k_stride, kPtKeys) ||
      !encode_row_tensor_map(&mv, a.v, a.num_tokens, a.num_kv_heads, a.v_stride, kPtKeys))
    return cudaErrorInvalidValue;
  const auto kernel = split ? prompt_attention_kernel<true> : prompt_attention_kernel<false>;
  static std::atomic<uint64_t> configured[2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t(1) << dev) : 0;
  if (bit == 0 || !(configured[split].load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPtSmem);
    if (e != cudaSuccess) return e;
    configured[split].fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_overlapped(kernel, dim3(static_cast<unsigned>(units)), dim3(kPtThreads), kPtSmem,
                           stream, p, mq, mk, mv);
}

}  // namespace kvq
