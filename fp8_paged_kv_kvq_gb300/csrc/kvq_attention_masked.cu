// kvq_attention_masked.cu -- paged attention over the FP8 cache whose rows see a
// sliding window and the first tokens of their sequence, or the ancestors of a
// drafted token, on the 5th-generation tensor cores.
//
//   s_j = sm_scale k_scale_j (q . kc_j),  out = sum_j p_j v_scale_j vc_j / sum_j p_j,
//   p_j = exp(s_j - max_j s_j), j over the tokens the row sees
//
//  * Rows.  The R query rows of a request that share a KV head are stacked with
//    their G query heads: row m is query row m / G, head m % G.  A unit of work is
//    one (request, KV head, row tile) over the tokens that some row of the tile
//    sees, in chunks of 128.  Two chains (QK^T -> softmax -> PV) work on a unit: of
//    more than 128 rows each has a 128-row tile of its own over all chunks (kPair),
//    of fewer they take turns at the chunks, and their sums and outputs are joined
//    at the end.  Of at most 32 rows the tile is repeated four times on the tensor
//    core's 128 rows and copy c takes the tokens [32 c, 32 c + 32) of a chunk, so
//    that all four warps of a chain's softmax have work.
//  * Tokens.  A unit's tokens are numbered without the gap between sinks and
//    window: x < S16 is position x, the others x + shift (both parts start on a
//    multiple of 16 tokens), so that a few sinks cost no chunk of their own.
//  * Split.  The chunks of all units, in order, with a charge for each unit's start,
//    are cut into one equal range per SM; a unit that is cut leaves a piece per range
//    (normalised output, reference, denominator) in the workspace, and the block
//    whose piece comes last joins them (a counter per unit, tagged with the call).
//  * S = Q K^T: 128 x 128 x 128, kind::f8f6f4, the query as two e4m3 pieces (q = 2^e
//    (p1 + p2), exact for elements >= 2^-9 of the row's largest) on the key codes as
//    they are.  O += P V: kind::f16, P'' = p v_scale in f16 from tensor memory, the
//    value codes converted exactly to f16.
//  * References.  With u_j = s_j log2(e) the softmax holds a reference m for which
//    2^(u_j - m) v_scale_j is at most 2^14 (f16 ends at 2^16) and that some token
//    seen so far reaches: m moves only when max_j (u_j + log2 v_scale_j) passes it by
//    14.  A chunk whose largest score cannot do that under the chunk's largest scales
//    is not searched for it.  Value scales are held over 2^Eg, Eg the unit's largest
//    log2 so far but at most 30, so that no weight or sum leaves binary32: weights
//    reach 2^(14 - lg) for a scale of 2^(Eg + lg), with lg taken as at least -90 (sums
//    of tokens of value 0 stay finite) and at most 97.  A token that a row does not
//    see can raise Eg to 30, no more, so that it costs no precision to rows of values
//    above 2^-60.
//  * Unseen tokens take no part: their scores are -infinity, their weights are set
//    to 0 after the product with the scale (which may be NaN), and in chunks that
//    some row of the unit does not see whole, value rows with a NaN code are cleared
//    (0 times NaN is NaN) and noted; a row that does see one becomes NaN.
//  * Roles, 640 threads: warps 0-3 and 4-7 the softmax of chain 0 and 1 (a thread owns
//    a TMEM lane, a row), 8-11 the epilogue, 12-15 the value codes' conversion, 16 the
//    units and the copies of codes, 17 and 18 the MMAs of chain 0 and 1, 19 the
//    scales.  Every wait is bounded; a role that gives up raises a shared abort flag,
//    copies and MMAs in flight complete, the block frees its tensor memory
//    (KVQ_ERRF_WAIT_TIMEOUT).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kMkTok = 128;                           // tokens of a chunk
constexpr int kMkWarpEpi = 8, kMkWarpConv = 12, kMkWarpLoad = 16, kMkWarpMma = 17, kMkWarpScale = 19;
constexpr int kMkThreads = 640;
constexpr int kMkUnits = 8;                           // units announced ahead
constexpr int kMkIdAhead = 4;                         // chunks whose page ids are in flight
constexpr int kMkMaxBoxes = 8;                        // pages of a chunk (boxes of >= 16 tokens)
constexpr int kMkScales = 6;                          // chunks of scales in the ring
constexpr int kMkMaxRequests = 1024;                  // of a launch
constexpr int kMkCharge = 2;                          // chunks that a unit's start counts for
constexpr float kMkLazy = 14.0f;                      // log2 of the largest P''
constexpr float kMkFloor = -90.0f;                    // log2 of the smallest value scale, over 2^Eg
constexpr int kMkMaxEg = 30;                          // Eg at most

// Shapes: kPair (two row tiles, one per chain) or one row tile of kRows rows whose
// chunks the chains share.
template <bool kPair, int kRows>
struct MkShape {
  static constexpr int kTileRows = kPair ? 256 : kRows;      // rows of a unit
  static constexpr int kCopies = 128 / kRows;
  static constexpr int kQTiles = kPair ? 2 : 1;
  // shared memory, offsets from a 1024-byte aligned base
  static constexpr int kKStages = kPair || kRows == 32 ? 3 : 4;
  static constexpr int kVStages = kPair ? 2 : 3;
  static constexpr int kCode = kMkTok * kHeadDim;            // a chunk's codes
  static constexpr int kQPiece = 128 * kHeadDim;
  static constexpr int kOffQ = 0;                            // [tile][piece]
  static constexpr int kOffVf = kOffQ + kQTiles * 2 * kQPiece;   // f16 values, two chunks
  static constexpr int kVfBytes = 2 * kCode;
  static constexpr int kOffK = kOffVf + 2 * kVfBytes;
  static constexpr int kOffV = kOffK + kKStages * kCode;
  static constexpr int kOffSum = kOffV + kVStages * kCode;   // [chain][128] denominators
  static constexpr int kOffRef = kOffSum + 2 * 128 * 4;      // [chain][128] references
  static constexpr int kOffEg = kOffRef + 2 * 128 * 4;       // [chain]
  static constexpr int kOffSc = kOffEg + 16;                 // [stage][K | V][128]
  static constexpr int kOffMeta = kOffSc + kMkScales * 2 * kMkTok * 4;   // [stage] float4
  static constexpr int kOffUnit = kOffMeta + kMkScales * 16;
  static constexpr int kOffIds = kOffUnit + kMkUnits * 64;
  static constexpr int kOffBad = kOffIds + (kMkIdAhead + 1) * kMkMaxBoxes * 4;   // [Vf][4 words]
  static constexpr int kOffMisc = kOffBad + 32;              // tmem base, abort, ticket
  static constexpr int kOffScan = kOffMisc + 16;             // a warp's sum each
  static constexpr int kOffPre = kOffScan + kMkThreads / 32 * 4;
  static constexpr int kOffBar = (kOffPre + (kMkMaxRequests + 1) * 4 + 7) / 8 * 8;
  static constexpr int kKFull = 0;
  static constexpr int kKEmpty = kKFull + kKStages;
  static constexpr int kVcFull = kKEmpty + kKStages;
  static constexpr int kVcEmpty = kVcFull + kVStages;
  static constexpr int kVfFull = kVcEmpty + kVStages;
  static constexpr int kVfEmpty = kVfFull + 2;
  static constexpr int kScFull = kVfEmpty + 2;
  static constexpr int kScEmpty = kScFull + kMkScales;
  static constexpr int kQFull = kScEmpty + kMkScales;        // per chain from here on
  static constexpr int kQEmpty = kQFull + 2;
  static constexpr int kSFull = kQEmpty + 2;
  static constexpr int kPReady = kSFull + 2;                 // (per chain and half of the chunk)
  static constexpr int kOFull = kPReady + 4;
  static constexpr int kOEmpty = kOFull + 2;
  static constexpr int kSumFull = kOEmpty + 2;
  static constexpr int kTurn = kSumFull + 2;
  static constexpr int kDrain = kTurn + 2;
  static constexpr int kUnitFull = kDrain + 2;
  static constexpr int kUnitEmpty = kUnitFull + kMkUnits;
  static constexpr int kBars = kUnitEmpty + kMkUnits;
  // at most 32 rows: the copies' outputs, 32 dims at a time
  static constexpr int kOffX = (kOffBar + 8 * kBars + 127) / 128 * 128;
  static constexpr int kSmem = kOffX + (kRows == 32 ? 4 * 32 * 32 * 4 : 0) + 1024;
  static_assert(kOffK % 1024 == 0 && kOffVf % 1024 == 0 && kOffSc % 16 == 0 && kOffMeta % 16 == 0 &&
                    kOffUnit % 16 == 0 && kOffBad % 16 == 0 && kOffMisc % 16 == 0 && kOffBar % 8 == 0,
                "alignment");
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kBars <= kMkThreads, "a thread initialises each barrier");
};

// TMEM: S of chain a at 128 a (its P'' over the first 64 columns), O at 256 + 128 a
constexpr uint32_t kMkTmemCols = 512;
__device__ __forceinline__ uint32_t mk_s(int a) { return 128u * a; }
__device__ __forceinline__ uint32_t mk_o(int a) { return 256u + 128u * a; }

constexpr uint32_t kMkIdescQK = mma_idesc(128, kMkTok, false, false);        // e4m3
constexpr uint32_t kMkIdescPV = mma_idesc(128, kHeadDim, false, true);       // f16, B MN-major
// The operands' shared-memory descriptors (smem_desc: stride offset 1024, version 1,
// 128-byte swizzle), upper words and the two leading offsets.
constexpr uint32_t kMkDescHi = (1024u >> 4) | (1u << 14) | (kSmemSwizzle128 << 29);
constexpr uint32_t kMkKMajor = 1u << 16, kMkMnMajor = (16384u >> 4) << 16;

__device__ __forceinline__ void mk_mma_qk(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}\n"
      :: "r"(d), "r"(a_lo), "r"(b_lo), "n"(kMkIdescQK), "r"(acc), "n"(kMkDescHi) : "memory");
}
__device__ __forceinline__ void mk_mma_pv(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n"
      :: "r"(d), "r"(a_tmem), "r"(b_lo), "n"(kMkIdescPV), "r"(acc), "n"(kMkDescHi) : "memory");
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool mk_elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(r));
  return r != 0;
}

struct MkParams {
  const uint16_t *q;
  uint16_t *out;
  const int32_t *tables;
  const int32_t *lens;
  const float *k_scales, *v_scales;
  const int32_t *tree;                                 // mask words, null: a window
  int32_t N, R, Hq, H, G, M;
  int32_t T;                                           // units of a request and head
  int32_t width;                                       // max_blocks_per_req
  int32_t ctx_limit, num_blocks, log2_bs, box;
  int32_t window, sinks, words;
  float scale2;                                        // |sm_scale| log2(e)
  uint32_t flip;                                       // sign bits of a negative sm_scale
  float *o_part;                                       // [grid][2][rows of a unit][128]
  float2 *ml_part;                                     // [grid][2][rows of a unit]
  unsigned long long *tickets;                         // [N * H * T]
  uint32_t tag;
  int32_t *err_flags;
};

__device__ __forceinline__ float mk_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float mk_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t mk_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float mk_pow2(int e) {      // e in [-126, 127]
  return __int_as_float((127 + e) << 23);
}
__device__ __forceinline__ float mk_pow2_down(int e) { // 2^e for e <= 0, 0 below 2^-126
  return e < -126 ? 0.0f : mk_pow2(e);
}
// e with |x| < 2^e, at least -126 (infinity and NaN: 129).
__device__ __forceinline__ int mk_ceil_log2(float x) {
  return static_cast<int>((__float_as_uint(x) >> 23) & 0xFFu) - 126;
}
// The lowest n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t mk_low(int n) {
  return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// Bounded wait that also gives up once another role raised the abort flag.
__device__ __forceinline__ bool mk_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort) {
#pragma unroll 1
  for (int i = 0; i < (1 << 19); ++i) {
    if (mbar_try_wait_sleep(bar, parity, 2000u)) return true;
    if ((i & 15) == 15 && *abort) return false;
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool mk_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
  return mbar_try_wait(bar, parity) || mk_wait_slow(bar, parity, abort);
}
// The whole warp's (every lane tries; one that gives up speaks for all).
__device__ __forceinline__ bool mk_wait_all(uint32_t bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xFFFFFFFFu, mk_wait(bar, parity, abort));
}

// ---------------------------------------------------------------------------
// Units.

// The tokens of unit t (rows [t rows, (t + 1) rows)) of a request of L tokens.
struct MkSpan {
  int X;                                               // how many, without the gap
  int s16, shift;                                      // x < s16 is position x, others x + shift
};
template <int kTileRows>
__device__ __forceinline__ MkSpan mk_span(const MkParams &p, int L, int t) {
  MkSpan s{L, 0, 0};
  if (p.tree != nullptr) return s;
  const int first = t * kTileRows / p.G, last = (min(p.M, (t + 1) * kTileRows) - 1) / p.G;
  const int base = L - p.R;
  if (base + last < 0) return MkSpan{0, 0, 0};
  const int lo16 = max(0, base + first - p.window + 1) & ~15;
  s.s16 = min((p.sinks + 15) & ~15, lo16);
  s.shift = lo16 - s.s16;
  s.X = base + last + 1 - s.shift;
  return s;
}

__device__ __forceinline__ int mk_len(const MkParams &p, int r) {
  const int L = p.lens[r];
  return L < 0 ? 0 : min(L, p.ctx_limit);
}

__device__ __forceinline__ int mk_positions(int X) {   // of a unit in the work sequence
  return X > 0 ? (X + kMkTok - 1) / kMkTok + kMkCharge : 0;
}

// A unit as the loading warp announces it: the chunks [c0, c0 + n) of a unit, which is
// whole (direct) or one of the pieces of the blocks [b_first, b_last].  n = 0 ends the work.
struct __align__(16) MkUnit {
  int r, h, row0, n;
  int c0, X, s16, shift;
  int base, direct, slot, b_first;
  int b_last, index, pad0, pad1;

  __device__ __forceinline__ int pos(int x) const { return x < s16 ? x : x + shift; }
};

// What a query row sees, in a unit's token numbers: x < hi and (x < sinks or x >= lo),
// or x < base and the nodes of its mask row.
struct MkSeen {
  int lo, hi, base;
  const int32_t *words;
  __device__ __forceinline__ uint32_t bits(const MkParams &p, int x0, int X) const {
    if (p.tree == nullptr)
      return mk_low(hi - x0) & (mk_low(p.sinks - x0) | ~mk_low(lo - x0));
    const int o = x0 - base;                           // node of the first bit
    uint32_t node = 0u;
    if (o > -32 && o < p.R) {
      const int w = o >> 5;                            // (floor)
      const uint32_t a = w >= 0 ? static_cast<uint32_t>(__ldg(words + w)) : 0u;
      const uint32_t b = w + 1 < p.words ? static_cast<uint32_t>(__ldg(words + w + 1)) : 0u;
      node = __funnelshift_r(a, b, o & 31);
    }
    return (mk_low(-o) | (node & ~mk_low(-o))) & mk_low(X - x0);
  }
};
__device__ __forceinline__ MkSeen mk_seen(const MkParams &p, const MkUnit &u, int m) {
  MkSeen s;
  const int i = min(m, p.M - 1) / p.G;                 // (rows past the last see what it sees)
  const int own = u.base + i;
  s.hi = own + 1 - u.shift;
  s.lo = max(own - p.window + 1, u.s16 + u.shift) - u.shift;
  s.base = u.base;
  s.words = p.tree + (static_cast<int64_t>(u.r) * p.R + i) * p.words;
  return s;
}
// Whether the rows between a first and a last one see all of the tokens [x0, x0 + n).
__device__ __forceinline__ bool mk_whole(const MkParams &p, int hi_first, int lo_last, int base,
                                         int x0, int n) {
  if (p.tree != nullptr) return x0 + n <= base;
  return x0 + n <= hi_first && (x0 + n <= p.sinks || x0 >= lo_last);
}

// ---------------------------------------------------------------------------
// Softmax pieces.

struct MkRow {
  float m = -INFINITY;                                 // reference
  float sum = 0.0f;                                    // denominator under it
  int eg = 0;                                          // value scales are held over 2^eg
};

// max_j (u_j + log2 of the value scale) over the seen of 32 tokens.
__device__ __forceinline__ float mk_top32(const float (&x)[32], const float *ks, const float *vs,
                                          float rowf, uint32_t bits, float top) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 k4 = reinterpret_cast<const float4 *>(ks)[q];
    const float4 v4 = reinterpret_cast<const float4 *>(vs)[q];
    const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w = x[4 * q + i] * kk[i] * rowf +
                      fmaxf(static_cast<float>(mk_ceil_log2(vv[i])), kMkFloor);
      if ((bits >> (4 * q + i)) & 1u) top = fmaxf(top, w);
    }
  }
  return top;
}

// The reference moved where `top` is far above it, the denominator and (unless the
// chain has no earlier chunk of the unit) the O row brought under the new one; `de`:
// by how much 2^Eg grew, which the O rows are brought under as well.
__device__ __forceinline__ void mk_meet(MkRow &row, float top, int de, bool fresh, uint32_t ocol) {
  const bool unset = row.m == -INFINITY;
  const bool move = unset ? top > -INFINITY : top - row.m > kMkLazy;
  const float f = (move && !unset) ? mk_ex2(row.m - top) : 1.0f;
  if (!fresh && __any_sync(0xFFFFFFFFu, (move && !unset) || de != 0)) {
    const float fo = f * mk_pow2_down(-de);
    row.sum *= f;
#pragma unroll 1
    for (int c = 0; c < kHeadDim; c += 16) {
      float o[16];
      tmem_ld16(ocol + c, o);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] *= fo;
      tmem_st16(ocol + c, o);
    }
    tmem_wait_st();
  }
  if (move) row.m = top;
}

// P'' of 32 scores as f16 in w, the sum of the p added to `sum`.
template <bool kMasked>
__device__ __forceinline__ void mk_part(const uint32_t (&x)[32], const float *ks, const float *vs,
                                        uint64_t rowf, uint64_t shift, uint32_t bits,
                                        uint64_t (&sum)[2], uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 k4 = reinterpret_cast<const float4 *>(ks)[q];
    const float4 v4 = reinterpret_cast<const float4 *>(vs)[q];
    const uint64_t kk[2] = {pack_f32x2(k4.x, k4.y), pack_f32x2(k4.z, k4.w)};
    const uint64_t vv[2] = {pack_f32x2(v4.x, v4.y), pack_f32x2(v4.z, v4.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 4 * q + 2 * i;
      const uint64_t s = pack_f32x2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
      float a, b, wa, wb;
      unpack_f32x2(fma_f32x2(mul_f32x2(s, kk[i]), rowf, shift), a, b);
      if (kMasked) {
        a = (bits >> e) & 1u ? a : -INFINITY;
        b = (bits >> (e + 1)) & 1u ? b : -INFINITY;
      }
      const uint64_t p = pack_f32x2(mk_ex2(a), mk_ex2(b));
      sum[i] = mk_add2(sum[i], p);
      unpack_f32x2(mul_f32x2(p, vv[i]), wa, wb);
      if (kMasked) {
        wa = (bits >> e) & 1u ? wa : 0.0f;
        wb = (bits >> (e + 1)) & 1u ? wb : 0.0f;
      }
      w[2 * q + i] = pack_f16x2(wa, wb);
    }
  }
}

// Part of a chunk's P'' is in TMEM.
__device__ __forceinline__ void mk_announce(uint32_t bar, int lane) {
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// One chunk of one row: S from TMEM, the row's statistics brought up to date, P'' over
// S's columns, its halves announced one after the other.  ks, vs: the chunk's scales;
// meta: the largest key scale, the log2 of the largest value scale, Eg.  bits: what the
// row sees of the four groups of 32 tokens (kMasked).
template <bool kMasked>
__device__ __forceinline__ void mk_softmax128(uint32_t scol, uint32_t ocol, const float *ks,
                                              const float *vs, const float4 meta, float rowf,
                                              const uint32_t (&bits)[4], bool fresh,
                                              uint32_t ready, int lane, MkRow &row) {
  const int eg = __float_as_int(meta.z);
  const int de = fresh ? 0 : eg - row.eg;
  row.eg = eg;
  bool search = true;
  if (!kMasked) {
    float mx[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int c = 0; c < 128; c += 64) {
      float x[64];
      tmem_ld64(scol + c, x);
#pragma unroll
      for (int i = 0; i < 64; i += 8)
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = mk_max3(mx[q], x[i + q], x[i + q + 4]);
    }
    const float most = fmaxf(mk_max3(mx[0], mx[1], mx[2]), mx[3]) * meta.x * rowf + meta.y;
    search = __any_sync(0xFFFFFFFFu, !(most - row.m <= kMkLazy));
  }
  if (search || de != 0) {
    float top = -INFINITY;
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
      float x[32];
      tmem_ld32(scol + 32 * g, x);
      const uint32_t b = !kMasked ? 0xFFFFFFFFu : (g == 0 ? bits[0] : g == 1 ? bits[1] : g == 2 ? bits[2] : bits[3]);
      top = mk_top32(x, ks + 32 * g, vs + 32 * g, rowf, b, top);
    }
    mk_meet(row, top, de, fresh, ocol);
  }
  const float sh = row.m == -INFINITY ? 0.0f : -row.m;
  const uint64_t rf = pack_f32x2(rowf, rowf), s2 = pack_f32x2(sh, sh);
  uint64_t sum[2] = {pack_f32x2(0.0f, 0.0f), pack_f32x2(0.0f, 0.0f)};
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t x0[32], x1[32], w[16];
    tmem_ld32_start(scol + 64 * h, x0);
    tmem_ld32_done(x0);
    tmem_ld32_start(scol + 64 * h + 32, x1);
    mk_part<kMasked>(x0, ks + 64 * h, vs + 64 * h, rf, s2, h == 0 ? bits[0] : bits[2], sum, w);
    tmem_ld32_done(x1);
    tmem_st16u(scol + 32 * h, w);
    mk_part<kMasked>(x1, ks + 64 * h + 32, vs + 64 * h + 32, rf, s2, h == 0 ? bits[1] : bits[3], sum, w);
    tmem_st16u(scol + 32 * h + 16, w);
    mk_announce(ready + 8 * h, lane);
  }
  float a, b;
  unpack_f32x2(mk_add2(sum[0], sum[1]), a, b);
  row.sum += a + b;
}

// The same for a row of which each of four copies takes 32 tokens of the chunk: this
// thread's are those of `copy`; the other copies' columns are 0.
__device__ __forceinline__ void mk_softmax32(uint32_t scol, uint32_t ocol, const float *ks,
                                             const float *vs, const float4 meta, float rowf,
                                             uint32_t bits, int copy, bool fresh, uint32_t ready,
                                             int lane, MkRow &row) {
  const int eg = __float_as_int(meta.z);
  const int de = fresh ? 0 : eg - row.eg;
  row.eg = eg;
  float x[32];
  tmem_ld32(scol + 32 * copy, x);
  const float *kc = ks + 32 * copy, *vc = vs + 32 * copy;
  mk_meet(row, mk_top32(x, kc, vc, rowf, bits, -INFINITY), de, fresh, ocol);
  const float sh = row.m == -INFINITY ? 0.0f : -row.m;
  uint64_t sum[2] = {pack_f32x2(0.0f, 0.0f), pack_f32x2(0.0f, 0.0f)};
  uint32_t xu[32], w[16], z[16];
#pragma unroll
  for (int i = 0; i < 32; ++i) xu[i] = __float_as_uint(x[i]);
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0u;
  mk_part<true>(xu, kc, vc, pack_f32x2(rowf, rowf), pack_f32x2(sh, sh), bits, sum, w);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c == copy) tmem_st16u(scol + 16 * c, w);
    else tmem_st16u(scol + 16 * c, z);
  }
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(ready);
    mbar_arrive(ready + 8);
  }
  float a, b;
  unpack_f32x2(mk_add2(sum[0], sum[1]), a, b);
  row.sum += a + b;
}

// A query row as two e4m3 pieces into its place in a K-major, 128-byte swizzled tile;
// returns 2^e |sm_scale| log2(e), which takes its scores to log2 units.
__device__ __forceinline__ float mk_query_row(const uint4 (&v)[16], float scale2, uint32_t flip,
                                              uint8_t *tile, int row, bool store) {
  uint32_t mg = 0u;                                    // largest magnitude, as bf16 bits
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    mg = __vmaxu2(mg, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu));
    mg = __vmaxu2(mg, __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
  }
  const uint32_t top = max(mg & 0xFFFFu, mg >> 16);
  const int ex = static_cast<int>(top >> 7);
  int e = ex == 0 ? -126 : ex - 127 - 7;
  e = e < -126 ? -126 : e;
  // (a row with an infinity or a NaN has no scores)
  const float back = ex == 255 ? __uint_as_float(0x7FC00000u) : mk_pow2(e) * scale2;
  if (store) {
    const float inv = top == 0u ? 0.0f : mk_pow2(-e);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t p1[4], p2[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 &y = v[2 * c + (j >> 1)];
        const uint32_t w0 = (j & 1) ? y.z : y.x, w1 = (j & 1) ? y.w : y.y;
        const float xs[4] = {bf16_lo(w0) * inv, bf16_hi(w0) * inv, bf16_lo(w1) * inv, bf16_hi(w1) * inv};
        e4m3_pieces4(xs, p1[j], p2[j]);
        p1[j] ^= flip;
        p2[j] ^= flip;
      }
      const int off = row * kHeadDim + ((c ^ (row & 7)) << 4);
      *reinterpret_cast<uint4 *>(tile + off) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
      *reinterpret_cast<uint4 *>(tile + 128 * kHeadDim + off) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
    }
  }
  return back;
}

template <bool kPair, int kRows>
__global__ void __launch_bounds__(kMkThreads, 1)
attn_masked_kernel(const MkParams p, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
  using S = MkShape<kPair, kRows>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bar0 = smem_addr(smem + S::kOffBar);
  auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffMisc);
  volatile int *abort_s = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
  volatile int *ticket_s = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 8);
  MkUnit *unit_s = reinterpret_cast<MkUnit *>(smem + S::kOffUnit);
  volatile float *sum_s = reinterpret_cast<volatile float *>(smem + S::kOffSum);
  volatile float *ref_s = reinterpret_cast<volatile float *>(smem + S::kOffRef);
  volatile int *eg_s = reinterpret_cast<volatile int *>(smem + S::kOffEg);
  volatile uint32_t *bad_s = reinterpret_cast<volatile uint32_t *>(smem + S::kOffBad);
  int *pre = reinterpret_cast<int *>(smem + S::kOffPre);

  allow_dependents_launch();
  if (tid < S::kBars) {
    uint32_t count = 1;
    const int i = tid;
    if ((i >= S::kKEmpty && i < S::kKEmpty + S::kKStages) || (i >= S::kVfEmpty && i < S::kVfEmpty + 2))
      count = kPair ? 2 : 1;                           // a commit of each chain that reads it
    if ((i >= S::kVcEmpty && i < S::kVcEmpty + S::kVStages) || (i >= S::kVfFull && i < S::kVfFull + 2))
      count = 4;                                       // the converting warps
    if (i >= S::kScEmpty && i < S::kScEmpty + kMkScales) count = kPair ? 8 : 4;
    if ((i >= S::kQFull && i < S::kQFull + 2) || (i >= S::kPReady && i < S::kPReady + 4) ||
        (i >= S::kOEmpty && i < S::kOEmpty + 2) || (i >= S::kSumFull && i < S::kSumFull + 2))
      count = 4;                                       // a chain's softmax or the epilogue
    if (i >= S::kUnitEmpty && i < S::kUnitEmpty + kMkUnits)
      count = 8 + 4 + 4 + 2 + 1;                       // softmax, epilogue, conversion, MMAs, scales
    mbar_init(BAR(i), count);
    fence_mbarrier_init();
  }
  if (tid == 0) *abort_s = 0;
  if (warp == kMkWarpLoad) {
    tmem_alloc(smem_addr(tmem_slot), kMkTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();

  // positions of the requests in the work sequence, and the sums before each
  auto request_positions = [&](int r) -> int {
    const int L = p.lens[r];
    if ((L < 0 || L > p.ctx_limit) && blockIdx.x == 0 && p.err_flags)
      atomicOr(p.err_flags, KVQ_ERRF_CONTEXT_RANGE);
    const int Lc = L < 0 ? 0 : min(L, p.ctx_limit);
    int w = 0;
    for (int t = 0; t < p.T; ++t) w += mk_positions(mk_span<S::kTileRows>(p, Lc, t).X);
    return w * p.H;
  };
  int *warp_sum = reinterpret_cast<int *>(smem + S::kOffScan);
  int carry = 0;
  for (int r0 = 0; r0 < p.N; r0 += kMkThreads) {
    const int r = r0 + tid;
    int w = r < p.N ? request_positions(r) : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, w, off);
      if (lane >= off) w += v;
    }
    if (lane == 31) warp_sum[warp] = w;
    __syncthreads();
    int before = carry;
    for (int k = 0; k < kMkThreads / 32; ++k) {
      const int v = warp_sum[k];
      if (k < warp) before += v;
      carry += v;
    }
    if (r < p.N) pre[r + 1] = before + w;
    __syncthreads();
  }
  if (tid == 0) pre[0] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = carry;
  const int B = max(1, static_cast<int>((static_cast<int64_t>(total) + gridDim.x - 1) / gridDim.x));

  // Unit t of this block; the caller's warp (converged) releases its entry.
  auto take_unit = [&](int t, MkUnit &u) -> bool {
    const int e = t % kMkUnits;
    if (!mk_wait_all(BAR(S::kUnitFull + e), (t / kMkUnits) & 1, abort_s)) return false;
    const int4 *src = reinterpret_cast<const int4 *>(unit_s + e);
    int4 *dst = reinterpret_cast<int4 *>(&u);
    dst[0] = src[0];
    dst[1] = src[1];
    dst[2] = src[2];
    dst[3] = src[3];
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(S::kUnitEmpty + e));
    return true;
  };
  // chunks of chain a in a unit, and whether it has any
  auto chain_chunks = [&](const MkUnit &u, int a) -> int {
    if (kPair) return a == 0 || u.row0 + 128 < p.M ? u.n : 0;
    return (u.n + 1 - a) / 2;
  };
  bool gave_up = false;

  if (warp < kMkWarpEpi) {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;\n");
    const int a = warp >> 2, q4 = warp & 3;
    const int lane_row = 32 * q4 + lane;               // TMEM lane
    const int copy = kRows == 32 ? q4 : 0;
    const int trow = (kPair ? 128 * a : 0) + (kRows == 32 ? lane : lane_row);   // of the unit
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    uint32_t steps = 0, done = 0, seq = 0;             // chunks and units of this chain, chunks of all
    uint32_t q_units = 0, q_units1 = 0;                // units with rows of chain a (split: 0 and 1)
    for (int t = 0;; ++t) {
      MkUnit u;
      if (!take_unit(t, u)) {
        gave_up = true;
        break;
      }
      if (u.n == 0) break;
      const int n = chain_chunks(u, a);
      float rowf = 0.0f;
      if (n > 0) {
        // the row's query; the tile's space is free once the last unit's products
        // with it are done.  (Where the chains share a tile, chain 0 stores it.)
        const int m = u.row0 + trow;
        uint4 v[16];
        const int i = m / p.G;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + ((static_cast<int64_t>(u.r) * p.R + i) * p.Hq + u.h * p.G + (m - i * p.G)) * kHeadDim);
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = m < p.M ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        const bool store = kPair || a == 0;
        bool ok = true;
        if (kPair && q_units > 0) ok = mk_wait_all(BAR(S::kQEmpty + a), (q_units - 1) & 1, abort_s);
        if (!kPair && store) {
          if (q_units > 0) ok = mk_wait_all(BAR(S::kQEmpty), (q_units - 1) & 1, abort_s);
          if (ok && q_units1 > 0) ok = mk_wait_all(BAR(S::kQEmpty + 1), (q_units1 - 1) & 1, abort_s);
        }
        if (!ok) {
          gave_up = true;
          break;
        }
        rowf = mk_query_row(v, p.scale2, p.flip, smem + S::kOffQ + (kPair ? a : 0) * 2 * S::kQPiece,
                            kRows == 32 ? 32 * copy + lane : lane_row, store);
        if (store) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(S::kQFull + (kPair ? a : 0)));
        }
      }
      q_units += kPair ? n > 0 : 1;
      q_units1 += u.n >= 2;
      const MkSeen seen = mk_seen(p, u, u.row0 + trow);
      // the warp's first and last row
      const int hi0 = __shfl_sync(0xFFFFFFFFu, seen.hi, 0), lo31 = __shfl_sync(0xFFFFFFFFu, seen.lo, 31);
      const int hi_first = mk_seen(p, u, u.row0).hi, lo_last = mk_seen(p, u, u.row0 + S::kTileRows - 1).lo;
      MkRow row;
      bool nan_row = false, fresh = true;
      for (int k = 0; k < u.n; ++k, ++seq) {
        if (!kPair && (k & 1) != a) continue;
        const uint32_t sb = seq % kMkScales;
        bool ok = mk_wait_all(BAR(S::kScFull + sb), (seq / kMkScales) & 1, abort_s);
        if (ok && n > 0) ok = mk_wait_all(BAR(S::kSFull + a), steps & 1, abort_s);
        if (!ok) {
          gave_up = true;
          break;
        }
        if (n > 0) {
          tc_fence_after();
          const int x0 = (u.c0 + k) * kMkTok;
          const float *ks = reinterpret_cast<const float *>(smem + S::kOffSc) + sb * 2 * kMkTok;
          const float *vs = ks + kMkTok;
          const float4 meta = reinterpret_cast<const float4 *>(smem + S::kOffMeta)[sb];
          uint32_t bits[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
          // (edge: some row of the unit does not see all of the chunk)
          const bool edge = !mk_whole(p, hi_first, lo_last, u.base, x0, kMkTok);
          const bool whole = mk_whole(p, hi0, lo31, u.base, x0, kMkTok);
          if (!whole) {
            if (kRows == 32) {
              bits[0] = seen.bits(p, x0 + 32 * copy, u.X);
            } else {
#pragma unroll
              for (int g = 0; g < 4; ++g) bits[g] = seen.bits(p, x0 + 32 * g, u.X);
            }
          }
          if (edge) {
            // value rows with a NaN code, which the conversion has cleared
            if (!mk_wait_all(BAR(S::kVfFull + (seq & 1)), (seq >> 1) & 1, abort_s)) {
              gave_up = true;
              break;
            }
            const volatile uint32_t *bad = bad_s + 4 * (seq & 1);
            if (kRows == 32) {
              nan_row |= (bad[copy] & bits[0]) != 0u;
            } else {
#pragma unroll
              for (int g = 0; g < 4; ++g) nan_row |= (bad[g] & bits[g]) != 0u;
            }
          }
          const uint32_t ready = BAR(S::kPReady + 2 * a);
          if (kRows == 32)
            mk_softmax32(tl + mk_s(a), tl + mk_o(a), ks, vs, meta, rowf, bits[0], copy, fresh, ready,
                         lane, row);
          else if (whole)
            mk_softmax128<false>(tl + mk_s(a), tl + mk_o(a), ks, vs, meta, rowf, bits, fresh, ready,
                                 lane, row);
          else
            mk_softmax128<true>(tl + mk_s(a), tl + mk_o(a), ks, vs, meta, rowf, bits, fresh, ready,
                                lane, row);
          fresh = false;
          ++steps;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(S::kScEmpty + sb));
      }
      if (gave_up) break;
      if (n == 0) continue;
      // the row's statistics, once the epilogue has read the last unit's
      if (done > 0 && !mk_wait_all(BAR(S::kOEmpty + a), (done - 1) & 1, abort_s)) {
        gave_up = true;
        break;
      }
      sum_s[128 * a + lane_row] = nan_row ? __uint_as_float(0x7FC00000u) : row.sum;
      ref_s[128 * a + lane_row] = row.m;
      if (q4 == 0 && lane == 0) eg_s[a] = row.eg;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(S::kSumFull + a));
      ++done;
    }
  } else if (warp < kMkWarpConv) {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
    const int q4 = warp & 3;
    const int lane_row = 32 * q4 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    uint32_t par = 0;                                  // barrier parities, bit a
    auto out_row = [&](const MkUnit &u, int m) -> uint16_t * {
      const int i = m / p.G;
      return p.out + ((static_cast<int64_t>(u.r) * p.R + i) * p.Hq + u.h * p.G + (m - i * p.G)) * kHeadDim;
    };
    for (int t = 0;; ++t) {
      MkUnit u;
      if (!take_unit(t, u)) {
        gave_up = true;
        break;
      }
      if (u.n == 0) break;
      const int64_t piece = static_cast<int64_t>(u.slot) * S::kTileRows;
#pragma unroll 1
      for (int a = 0; a < (kPair ? 2 : 1); ++a) {
        if (chain_chunks(u, a) == 0) continue;
        const bool both = !kPair && u.n >= 2;
        bool got = mk_wait_all(BAR(S::kSumFull + a), (par >> a) & 1, abort_s) &&
                   mk_wait_all(BAR(S::kOFull + a), (par >> a) & 1, abort_s);
        if (both)
          got = got && mk_wait_all(BAR(S::kSumFull + 1), par >> 1, abort_s) &&
                mk_wait_all(BAR(S::kOFull + 1), par >> 1, abort_s);
        if (!got) {
          gave_up = true;
          break;
        }
        tc_fence_after();
        par ^= 1u << a;
        if (both) par ^= 2u;
        // the row's parts (chains, copies) under their largest reference
        const int row = kRows == 32 ? lane : lane_row;
        float top = -INFINITY, all = 0.0f;
        if (kPair) {
          top = ref_s[128 * a + lane_row];
          all = sum_s[128 * a + lane_row];
        } else {
#pragma unroll
          for (int c = 0; c < S::kCopies; ++c) {
            top = fmaxf(top, ref_s[32 * c + row]);
            if (both) top = fmaxf(top, ref_s[128 + 32 * c + row]);
          }
#pragma unroll
          for (int c = 0; c < S::kCopies; ++c) {
            const float m0 = ref_s[32 * c + row];
            if (m0 != -INFINITY) all += mk_ex2(m0 - top) * sum_s[32 * c + row];
            else all += sum_s[32 * c + row];           // (0, or NaN)
            if (both) {
              const float m1 = ref_s[128 + 32 * c + row];
              if (m1 != -INFINITY) all += mk_ex2(m1 - top) * sum_s[128 + 32 * c + row];
              else all += sum_s[128 + 32 * c + row];
            }
          }
        }
        const bool none = all == 0.0f;                 // (the row has seen nothing)
        auto factor = [&](int chain) -> float {
          const float m = ref_s[128 * chain + lane_row];
          if (none) return 0.0f;
          const float f = m == -INFINITY ? 0.0f : mk_ex2(m - top);
          return f / all * mk_pow2(eg_s[chain]);
        };
        const float f0 = factor(kPair ? a : 0), f1 = both ? factor(1) : 0.0f;
        const int m = u.row0 + (kPair ? 128 * a : 0) + row;
        const bool mine = m < p.M;
        // 32 dims of this lane's part of its row
        auto dims = [&](int c, float (&o)[32]) {
          tmem_ld32(tl + mk_o(kPair ? a : 0) + c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = none ? 0.0f : o[i] * f0;
          if (both) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float o1[16];
              tmem_ld16(tl + mk_o(1) + c + 16 * h, o1);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[16 * h + i] = none ? 0.0f : fmaf(o1[i], f1, o[16 * h + i]);
            }
          }
        };
        uint16_t *dst = out_row(u, mine ? m : 0);
        const int64_t prow = piece + (kPair ? 128 * a : 0) + row;
        if (kRows == 32) {
          float *xs = reinterpret_cast<float *>(smem + S::kOffX);   // [copy][32 dims][32 rows]
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 32) {
            float o[32];
            dims(c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) xs[(32 * q4 + i) * 32 + lane] = o[i];
            named_barrier(1, 128);
            float y[8];                                // dims c + 8 q4 .. + 7 of the row
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              y[j] = 0.0f;
#pragma unroll
              for (int k = 0; k < 4; ++k) y[j] += xs[(32 * k + 8 * q4 + j) * 32 + lane];
            }
            if (mine) {
              if (u.direct) {
                *reinterpret_cast<uint4 *>(dst + c + 8 * q4) =
                    make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                               pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
              } else {
                float4 *to = reinterpret_cast<float4 *>(p.o_part + prow * kHeadDim + c + 8 * q4);
                to[0] = make_float4(y[0], y[1], y[2], y[3]);
                to[1] = make_float4(y[4], y[5], y[6], y[7]);
              }
            }
            named_barrier(1, 128);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 32) {
            float o[32];
            dims(c, o);
            if (mine) {
              if (u.direct) {
                uint4 *to = reinterpret_cast<uint4 *>(dst + c);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  to[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                                     pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
              } else {
                float4 *to = reinterpret_cast<float4 *>(p.o_part + prow * kHeadDim + c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  to[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
              }
            }
          }
        }
        if (!u.direct && mine && (kRows != 32 || q4 == 0)) p.ml_part[prow] = make_float2(top, all);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(BAR(S::kOEmpty + a));
          if (both) mbar_arrive(BAR(S::kOEmpty + 1));
        }
      }
      if (gave_up) break;
      if (u.direct) continue;
      // the block whose piece comes last joins the unit's pieces
      __threadfence();
      named_barrier(1, 128);
      if (q4 == 0 && lane == 0) {
        const uint32_t landed = ticket_take(p.tickets + u.index, p.tag);
        const bool last = landed == static_cast<uint32_t>(u.b_last - u.b_first + 1);
        if (last) p.tickets[u.index] = 0ull;
        if (landed == 0u && p.err_flags) atomicOr(p.err_flags, KVQ_ERRF_WAIT_TIMEOUT);
        *ticket_s = last ? 1 : 0;
        __threadfence();
      }
      named_barrier(1, 128);
      if (*ticket_s) {
        const int rows = min(S::kTileRows, p.M - u.row0);
        for (int r = q4; r < rows; r += 4) {
          float top = -INFINITY, all = 0.0f;
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
          for (int b = u.b_first; b <= u.b_last; ++b) {
            const int64_t at = static_cast<int64_t>(2 * b + (b == u.b_first ? 1 : 0)) * S::kTileRows + r;
            const float2 ml = __ldcg(p.ml_part + at);
            const float4 o = __ldcg(reinterpret_cast<const float4 *>(p.o_part + at * kHeadDim) + lane);
            const float next = fmaxf(top, ml.x);
            const float f = top == -INFINITY ? 0.0f : mk_ex2(top - next);
            // (a part that saw nothing has no reference and a sum of 0, or NaN)
            const float w = ml.x == -INFINITY ? ml.y : mk_ex2(ml.x - next) * ml.y;
            all = all * f + w;
            y.x = y.x * f + o.x * w;
            y.y = y.y * f + o.y * w;
            y.z = y.z * f + o.z * w;
            y.w = y.w * f + o.w * w;
            top = next;
          }
          const float inv = all == 0.0f ? 0.0f : 1.0f / all;
          *reinterpret_cast<uint2 *>(out_row(u, u.row0 + r) + 4 * lane) =
              make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
        }
      }
    }
    // units whose rows see no token: zero rows, spread over the grid
    if (!gave_up) {
      const int units = p.N * p.H * p.T;
      for (int x = blockIdx.x * 4 + q4; x < units; x += gridDim.x * 4) {
        const int t = x % p.T, rh = x / p.T, h = rh % p.H, r = rh / p.H;
        if (mk_span<S::kTileRows>(p, mk_len(p, r), t).X > 0) continue;
        MkUnit u;
        u.r = r;
        u.h = h;
        for (int m = t * S::kTileRows; m < min(p.M, (t + 1) * S::kTileRows); ++m)
          *reinterpret_cast<uint2 *>(out_row(u, m) + 4 * lane) = make_uint2(0u, 0u);
      }
    }
  } else if (warp < kMkWarpLoad) {
    // ------------------------------------------- value codes to f16 values
    // Thread j converts token j: dims 64 b + 8 c .. in block b, MN-major and 128-byte
    // swizzled.  Tokens past the unit's are cleared.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;\n");
    const int q4 = warp & 3, j = 32 * q4 + lane;
    uint32_t seq = 0;
    for (int t = 0; !gave_up; ++t) {
      MkUnit u;
      if (!take_unit(t, u)) {
        gave_up = true;
        break;
      }
      if (u.n == 0) break;
      const int hi_first = mk_seen(p, u, u.row0).hi, lo_last = mk_seen(p, u, u.row0 + S::kTileRows - 1).lo;
      for (int k = 0; k < u.n; ++k, ++seq) {
        const uint32_t b = seq % S::kVStages;
        bool ok = mk_wait_all(BAR(S::kVcFull + b), (seq / S::kVStages) & 1, abort_s);
        if (ok && seq >= 2) ok = mk_wait_all(BAR(S::kVfEmpty + (seq & 1)), ((seq >> 1) - 1) & 1, abort_s);
        if (!ok) {
          gave_up = true;
          break;
        }
        const int x0 = (u.c0 + k) * kMkTok;
        const uint8_t *src = smem + S::kOffV + b * S::kCode + j * kHeadDim;
        uint8_t *dst = smem + S::kOffVf + (seq & 1) * S::kVfBytes + j * 128;
        bool keep = x0 + j < u.X;
        if (!mk_whole(p, hi_first, lo_last, u.base, x0, kMkTok)) {
          bool bad = false;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 w = *reinterpret_cast<const uint4 *>(src + ((c ^ (j & 7)) << 4));
            bad |= (__vcmpeq4(w.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(w.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                    __vcmpeq4(w.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(w.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu)) != 0u;
          }
          const uint32_t word = __ballot_sync(0xFFFFFFFFu, keep && bad);
          if (lane == 0) bad_s[4 * (seq & 1) + q4] = word;
          keep = keep && !bad;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4 w = *reinterpret_cast<const uint4 *>(src + ((c ^ (j & 7)) << 4));
          if (!keep) w = make_uint4(0u, 0u, 0u, 0u);
          const uint4 lo = make_uint4(e4m3x2_to_f16x2(w.x & 0xFFFFu), e4m3x2_to_f16x2(w.x >> 16),
                                      e4m3x2_to_f16x2(w.y & 0xFFFFu), e4m3x2_to_f16x2(w.y >> 16));
          const uint4 hi = make_uint4(e4m3x2_to_f16x2(w.z & 0xFFFFu), e4m3x2_to_f16x2(w.z >> 16),
                                      e4m3x2_to_f16x2(w.w & 0xFFFFu), e4m3x2_to_f16x2(w.w >> 16));
          uint8_t *blk = dst + (c >> 2) * (S::kVfBytes / 2);
          const int c0 = (2 * c) & 7;
          *reinterpret_cast<uint4 *>(blk + ((c0 ^ (j & 7)) << 4)) = lo;
          *reinterpret_cast<uint4 *>(blk + (((c0 + 1) ^ (j & 7)) << 4)) = hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(BAR(S::kVcEmpty + b));
          mbar_arrive(BAR(S::kVfFull + (seq & 1)));
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    if (warp == kMkWarpLoad) {
      // --------------------------------------------- units, copies of codes
      int x = static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * B, static_cast<int64_t>(total)));
      const int x_end = static_cast<int>(min(static_cast<int64_t>(x) + B, static_cast<int64_t>(total)));
      // the next piece of the block's range with chunks (n = 0: none left)
      auto next_unit = [&]() -> MkUnit {
        MkUnit u;
        u.n = 0;
        while (x < x_end) {
          int lo = 0, hi = p.N - 1;                    // the last request with pre[r] <= x
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= x) lo = mid;
            else hi = mid - 1;
          }
          const int L = mk_len(p, lo), W = (pre[lo + 1] - pre[lo]) / p.H;
          const int h = (x - pre[lo]) / W;
          int at = pre[lo] + h * W;                    // where unit t starts
          MkSpan s{0, 0, 0};
          int t = 0, V = 0;
          for (;; ++t) {
            s = mk_span<S::kTileRows>(p, L, t);
            V = mk_positions(s.X);
            if (x < at + V || t == p.T - 1) break;
            at += V;
          }
          const int first = at + kMkCharge, end = min(at + V, x_end), from = max(x, first);
          x = max(end, x + 1);
          if (from >= end) continue;
          u.r = lo;
          u.h = h;
          u.row0 = t * S::kTileRows;
          u.c0 = from - first;
          u.n = end - from;
          u.X = s.X;
          u.s16 = s.s16;
          u.shift = s.shift;
          u.base = L - p.R;
          u.direct = u.n == V - kMkCharge;
          u.b_first = first / B;
          u.b_last = (at + V - 1) / B;
          u.slot = 2 * static_cast<int>(blockIdx.x) + (static_cast<int>(blockIdx.x) == u.b_first ? 1 : 0);
          u.index = (lo * p.H + h) * p.T + t;
          break;
        }
        return u;
      };
      bool ok = true;
      int published = 0;
      auto publish = [&](const MkUnit &u) {
        const int e = published % kMkUnits;
        if (published >= kMkUnits &&
            !mk_wait_all(BAR(S::kUnitEmpty + e), (published / kMkUnits - 1) & 1, abort_s)) {
          ok = false;
          return;
        }
        if (lane == 0) {
          unit_s[e] = u;
          mbar_arrive(BAR(S::kUnitFull + e));
        }
        __syncwarp();
        ++published;
      };
      int32_t *ids = reinterpret_cast<int32_t *>(smem + S::kOffIds);
      const int boxes = kMkTok / p.box;
      MkUnit f = next_unit(), u = f;                   // of the page ids, of the copies
      publish(f);
      int fk = 0;
      // page ids of the next chunk of f (a commit group in any case)
      auto fetch = [&](uint32_t slot) {
        if (f.n != 0 && ok) {
          const int xt = (f.c0 + fk) * kMkTok + lane * p.box;
          if (lane < boxes) {
            const bool need = xt < f.X;
            const int32_t *src = p.tables + static_cast<int64_t>(f.r) * p.width +
                                 (need ? f.pos(xt) >> p.log2_bs : 0);
            cp_async_4(ids + slot * kMkMaxBoxes + lane, src, need ? 4u : 0u);
          }
          if (++fk == f.n) {
            f = next_unit();
            publish(f);
            fk = 0;
          }
        }
        cp_async_commit();
      };
#pragma unroll 1
      for (uint32_t i = 0; i < kMkIdAhead; ++i) fetch(i);
      const uint64_t pol = l2_policy_evict_normal();
      const int mask = (1 << p.log2_bs) - 1;
      uint32_t seq = 0, k_issued = 0, v_issued = 0;
      bool bad = false;
      int unit_no = 0;
      while (u.n != 0 && ok) {
        for (int k = 0; k < u.n && ok; ++k, ++seq) {
          fetch((seq + kMkIdAhead) % (kMkIdAhead + 1));
          cp_async_wait<kMkIdAhead>();
          __syncwarp();
          if (lane == 0) {
            const int32_t *cid = ids + (seq % (kMkIdAhead + 1)) * kMkMaxBoxes;
            const int x0 = (u.c0 + k) * kMkTok;
#pragma unroll 1
            for (int kv = 0; kv < 2 && ok; ++kv) {
              const uint32_t ring = kv == 0 ? S::kKStages : S::kVStages;
              const uint32_t b = seq % ring, round = seq / ring;
              const uint32_t full = BAR((kv == 0 ? S::kKFull : S::kVcFull) + b);
              if (round > 0)
                ok = mk_wait(BAR((kv == 0 ? S::kKEmpty : S::kVcEmpty) + b), (round - 1) & 1, abort_s);
              if (!ok) break;
              const uint32_t dst = smem_addr(smem + (kv == 0 ? S::kOffK : S::kOffV) + b * S::kCode);
              uint32_t bytes = 0;
#pragma unroll 1
              for (int i = 0; i < boxes; ++i) {
                const int xt = x0 + i * p.box;
                if (xt >= u.X) break;
                const uint32_t page = static_cast<uint32_t>(cid[i]);
                if (page >= static_cast<uint32_t>(p.num_blocks)) {
                  bad = true;
                  continue;
                }
                const int slot = static_cast<int>((page << p.log2_bs) | (u.pos(xt) & mask));
                tma_load_3d_hint(dst + i * p.box * kHeadDim, kv == 0 ? &tm_k : &tm_v, 0, u.h, slot, full, pol);
                bytes += p.box * kHeadDim;
              }
              mbar_arrive_expect_tx(full, bytes);
              if (kv == 0) ++k_issued;
              else ++v_issued;
            }
          }
          ok = __all_sync(0xFFFFFFFFu, ok);
        }
        // the next unit, announced by now
        ++unit_no;
        if (ok && unit_no < published) {
          const int4 *src = reinterpret_cast<const int4 *>(unit_s + unit_no % kMkUnits);
          int4 *dst = reinterpret_cast<int4 *>(&u);
          dst[0] = src[0];
          dst[1] = src[1];
          dst[2] = src[2];
          dst[3] = src[3];
        } else {
          u.n = 0;
        }
      }
      cp_async_wait<0>();
      gave_up = !ok;
      if (lane == 0) {
        if (bad && p.err_flags) atomicOr(p.err_flags, KVQ_ERRF_BLOCK_RANGE);
        // copies in flight land before the block leaves
        for (uint32_t v = k_issued > S::kKStages ? k_issued - S::kKStages : 0; v < k_issued; ++v)
          mbar_wait_sleep_bounded(BAR(S::kKFull + v % S::kKStages), (v / S::kKStages) & 1);
        for (uint32_t v = v_issued > S::kVStages ? v_issued - S::kVStages : 0; v < v_issued; ++v)
          mbar_wait_sleep_bounded(BAR(S::kVcFull + v % S::kVStages), (v / S::kVStages) & 1);
      }
    } else if (warp == kMkWarpScale) {
      // -------------------------------------------------------------- scales
      // Lane l has the tokens 4 l .. 4 l + 3 of a chunk.  Page ids are read two chunks
      // ahead and scales one.
      struct Walk {
        MkUnit u;
        int t = -1, k = 0;
        bool end = false;
      };
      bool ok = true;
      auto advance = [&](Walk &w) {                    // to the next chunk
        if (w.end || !ok) return;
        if (w.t >= 0 && ++w.k < w.u.n) return;
        ++w.t;
        w.k = 0;
        const int e = w.t % kMkUnits;
        ok = mk_wait_all(BAR(S::kUnitFull + e), (w.t / kMkUnits) & 1, abort_s);
        if (!ok) return;
        const int4 *src = reinterpret_cast<const int4 *>(unit_s + e);
        int4 *dst = reinterpret_cast<int4 *>(&w.u);
        dst[0] = src[0];
        dst[1] = src[1];
        w.end = w.u.n == 0;
      };
      auto read_id = [&](const Walk &w) -> int {
        const int x = (w.u.c0 + w.k) * kMkTok + 4 * lane;
        if (w.end || !ok || x >= w.u.X) return -1;
        return __ldg(p.tables + static_cast<int64_t>(w.u.r) * p.width + (w.u.pos(x) >> p.log2_bs));
      };
      auto read_scales = [&](const Walk &w, int page, float (&kk)[4], float (&vv)[4]) {
        const int x = (w.u.c0 + w.k) * kMkTok + 4 * lane;
        const bool in = !w.end && ok && static_cast<uint32_t>(page) < static_cast<uint32_t>(p.num_blocks);
        const int64_t slot = (static_cast<int64_t>(page) << p.log2_bs) + (w.u.pos(x) & ((1 << p.log2_bs) - 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool get = in && x + i < w.u.X;
          kk[i] = get ? __ldg(p.k_scales + (slot + i) * p.H + w.u.h) : 0.0f;
          vv[i] = get ? __ldg(p.v_scales + (slot + i) * p.H + w.u.h) : 0.0f;
        }
      };
      Walk wi, ws;                                     // of the ids, of the scales
      advance(wi);
      int id = read_id(wi);
      ws = wi;
      float kn[4], vn[4];
      read_scales(ws, id, kn, vn);
      advance(wi);
      id = read_id(wi);
      uint32_t seq = 0;
      int eg = 0;
      while (ok && !ws.end) {
        float kk[4], vv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          kk[i] = kn[i];
          vv[i] = vn[i];
        }
        const bool first = ws.k == 0, last = ws.k == ws.u.n - 1;
        const int t = ws.t;
        advance(ws);
        read_scales(ws, id, kn, vn);
        advance(wi);
        id = read_id(wi);
        if (!ok) break;
        const uint32_t b = seq % kMkScales;
        if (seq >= kMkScales &&
            !mk_wait_all(BAR(S::kScEmpty + b), (seq / kMkScales - 1) & 1, abort_s)) {
          ok = false;
          break;
        }
        // the largest scales (of non-negative numbers, as unsigned words; NaN aside)
        uint32_t km = 0u, vm = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kk[i] == kk[i]) km = max(km, __float_as_uint(fabsf(kk[i])));
          if (vv[i] == vv[i]) vm = max(vm, __float_as_uint(fabsf(vv[i])));
        }
        km = __reduce_max_sync(0xFFFFFFFFu, km);
        vm = __reduce_max_sync(0xFFFFFFFFu, vm);
        const int ev = min(mk_ceil_log2(__uint_as_float(vm)), 126);
        if (first) eg = min(ev, kMkMaxEg);
        else if (ev > eg) eg = min(ev + 2, kMkMaxEg);
        const float down = mk_pow2(-eg);
        float *ks = reinterpret_cast<float *>(smem + S::kOffSc) + b * 2 * kMkTok;
        reinterpret_cast<float4 *>(ks)[lane] = make_float4(kk[0], kk[1], kk[2], kk[3]);
        reinterpret_cast<float4 *>(ks + kMkTok)[lane] =
            make_float4(vv[0] * down, vv[1] * down, vv[2] * down, vv[3] * down);
        if (lane == 0)
          reinterpret_cast<float4 *>(smem + S::kOffMeta)[b] =
              make_float4(__uint_as_float(km), fmaxf(static_cast<float>(ev - eg), kMkFloor),
                          __int_as_float(eg), 0.0f);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(BAR(S::kScFull + b));
          // (held to here: the walks have read the unit)
          if (last) mbar_arrive(BAR(S::kUnitEmpty + t % kMkUnits));
        }
        ++seq;
      }
      gave_up = !ok;
    } else {
      // ---------------------------------------------------- MMAs of a chain
      // Each turn: PV of one of the chain's chunks and QK^T of its next, chain 0's and
      // chain 1's bursts one after the other; everything but P'' is waited for before
      // the turn.
      const int a = warp - kMkWarpMma;
      const uint32_t q1 = (smem_addr(smem + S::kOffQ + (kPair ? a : 0) * 2 * S::kQPiece) >> 4) | kMkKMajor;
      const uint32_t q2 = q1 + (S::kQPiece >> 4);
      const uint32_t k0 = (smem_addr(smem + S::kOffK) >> 4) | kMkKMajor;
      const uint32_t v0 = (smem_addr(smem + S::kOffVf) >> 4) | kMkMnMajor;
      const uint32_t s_col = tmem + mk_s(a), o_col = tmem + mk_o(a);
      uint32_t base = 0;                               // chunks of earlier units
      uint32_t par_q = 0, par_p = 0, par_o = 1, par_turn = a ^ 1;
      bool ok = true;
      for (int t = 0; ok; ++t) {
        MkUnit u;
        ok = take_unit(t, u);
        if (!ok || u.n == 0) break;
        const int mine = chain_chunks(u, a);           // chunks with products of this chain
        const int steps = kPair ? u.n : (u.n + 1) / 2;
        const bool turns = chain_chunks(u, 1) > 0;     // (a lone chain 0 need not pass them)
        const bool live = mine > 0;
        for (int j = 0; j <= steps; ++j) {
          const int cv = kPair ? j - 1 : 2 * (j - 1) + a, cq = kPair ? j : 2 * j + a;
          const bool use_v = j > 0 && cv < u.n, use_k = cq < u.n;
          const bool pv = use_v && live, qk = use_k && live;
          const uint32_t sv = base + cv, sq = base + cq;
          const uint32_t bk = sq % S::kKStages, bv = sv & 1;
          if (use_v) ok = mk_wait_all(BAR(S::kVfFull + bv), (sv >> 1) & 1, abort_s);
          if (ok && use_k) ok = mk_wait_all(BAR(S::kKFull + bk), (sq / S::kKStages) & 1, abort_s);
          if (ok && qk && j == 0) ok = mk_wait_all(BAR(S::kQFull + (kPair ? a : 0)), kPair ? par_q : t & 1, abort_s);
          if (ok && pv) {
            if (j == 1) {
              ok = mk_wait_all(BAR(S::kOEmpty + a), par_o, abort_s);
              par_o ^= 1u;
            }
            ok = ok && mk_wait_all(BAR(S::kPReady + 2 * a), par_p, abort_s);
          }
          if (turns) {
            ok = ok && mk_wait_all(BAR(S::kTurn + a), par_turn, abort_s);
            par_turn ^= 1u;
          }
          if (!ok) break;
          if (pv) {
            const uint32_t v_lo = v0 + bv * (S::kVfBytes >> 4);
            tc_fence_after();
            if (mk_elect()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mk_mma_pv(o_col, s_col + 8 * kk, v_lo + (2048 >> 4) * kk, (j == 1 && kk == 0) ? 0u : 1u);
            }
            ok = mk_wait_all(BAR(S::kPReady + 2 * a + 1), par_p, abort_s);
            if (!ok) break;
            par_p ^= 1u;
            tc_fence_after();
            if (mk_elect()) {
#pragma unroll
              for (int kk = 4; kk < 8; ++kk)
                mk_mma_pv(o_col, s_col + 8 * kk, v_lo + (2048 >> 4) * kk, 1u);
            }
          }
          if (qk) {
            const uint32_t k_lo = k0 + bk * (S::kCode >> 4);
            tc_fence_after();
            if (mk_elect()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mk_mma_qk(s_col, q1 + 2 * kk, k_lo + 2 * kk, kk != 0);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mk_mma_qk(s_col, q2 + 2 * kk, k_lo + 2 * kk, 1u);
              tc_commit(BAR(S::kSFull + a));
            }
          }
          __syncwarp();
          if (mk_elect()) {
            if (turns) mbar_arrive(BAR(S::kTurn + (a ^ 1)));
            if (pv && (kPair ? cv == u.n - 1 : cv + 2 >= u.n)) tc_commit(BAR(S::kOFull + a));
            if (qk && (kPair ? cq == u.n - 1 : cq + 2 >= u.n)) tc_commit(BAR(S::kQEmpty + a));
            if (use_v) tc_commit(BAR(S::kVfEmpty + bv));
            if (use_k) tc_commit(BAR(S::kKEmpty + bk));
          }
          __syncwarp();
        }
        if (live) par_q ^= 1u;
        base += u.n;
      }
      gave_up = !ok;
      // every MMA issued has completed before the tensor memory is freed
      __syncwarp();
      if (mk_elect()) tc_commit(BAR(S::kDrain + a));
      mbar_wait_sleep_bounded(BAR(S::kDrain + a), 0);
    }
  }
  if (gave_up) {
    *abort_s = 1;
    if (lane == 0 && p.err_flags) atomicOr(p.err_flags, KVQ_ERRF_WAIT_TIMEOUT);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMkWarpLoad) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, kMkTmemCols);
  }
}

int mk_tile_rows(int M) { return M <= 32 ? 32 : (M <= 128 ? 128 : 256); }

template <bool kPair, int kRows>
cudaError_t mk_launch(const MkParams &p, const CUtensorMap &mk, const CUtensorMap &mv, int grid,
                      cudaStream_t stream) {
  constexpr int kSmem = MkShape<kPair, kRows>::kSmem;
  const auto kernel = attn_masked_kernel<kPair, kRows>;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t(1) << dev) : 0;
  if (bit == 0 || !(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_overlapped(kernel, dim3(static_cast<unsigned>(grid)), dim3(kMkThreads), kSmem, stream,
                           p, mk, mv);
}

size_t mk_round(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t attn_masked_workspace_bytes(const MaskedArgs &a, int32_t num_kv_heads) {
  const int64_t M = static_cast<int64_t>(a.rows_per_request) * (a.num_q_heads / num_kv_heads);
  const int64_t rows = mk_tile_rows(static_cast<int>(M)), T = (M + rows - 1) / rows;
  const int64_t n = std::min(a.num_requests, kMkMaxRequests);
  const size_t slots = static_cast<size_t>(a.sms) * 2 * rows;
  return mk_round(static_cast<size_t>(n * num_kv_heads * T) * 8) +
         mk_round(slots * kHeadDim * sizeof(float)) + mk_round(slots * sizeof(float2));
}

cudaError_t launch_attn_masked(const kvq_cache &c, const MaskedArgs &a, cudaStream_t stream) {
  MkParams p;
  const int H = c.num_kv_heads;
  const int64_t cap = static_cast<int64_t>(a.max_blocks_per_req) << a.log2_block;
  p.ctx_limit = static_cast<int32_t>(std::min<int64_t>(cap, a.max_context_len));
  p.R = a.rows_per_request;
  p.Hq = a.num_q_heads;
  p.H = H;
  p.G = a.num_q_heads / H;
  p.M = p.R * p.G;
  const int rows = mk_tile_rows(p.M);
  p.T = (p.M + rows - 1) / rows;
  p.width = a.max_blocks_per_req;
  p.num_blocks = static_cast<int32_t>(c.num_slots >> a.log2_block);
  p.log2_bs = a.log2_block;
  // boxes of a copy: a window and its sinks start on any 16 tokens of a page
  p.box = a.tree_mask != nullptr ? std::min(1 << a.log2_block, kMkTok) : 16;
  // (beyond the longest context neither bound means anything)
  p.window = std::min(a.window, a.max_context_len + p.R);
  p.sinks = std::min(a.num_sinks, a.max_context_len);
  p.words = (p.R + 31) / 32;
  p.scale2 = (a.sm_scale < 0.0f ? -a.sm_scale : a.sm_scale) * 1.4426950408889634f;
  p.flip = a.sm_scale < 0.0f ? 0x80808080u : 0u;
  p.k_scales = c.k_scales;
  p.v_scales = c.v_scales;
  p.err_flags = a.err_flags;
  CUtensorMap mk, mv;
  if (!encode_code_tensor_map(&mk, c.k_codes, c.num_slots, H, p.box) ||
      !encode_code_tensor_map(&mv, c.v_codes, c.num_slots, H, p.box))
    return cudaErrorInvalidValue;
  const int grid = a.sms;
  for (int r0 = 0; r0 < a.num_requests; r0 += kMkMaxRequests) {
    p.N = std::min(a.num_requests - r0, kMkMaxRequests);
    const int64_t row = static_cast<int64_t>(r0) * p.R;
    p.q = static_cast<const uint16_t *>(a.q) + row * p.Hq * kHeadDim;
    p.out = static_cast<uint16_t *>(a.out) + row * p.Hq * kHeadDim;
    p.tables = a.block_tables + static_cast<int64_t>(r0) * p.width;
    p.lens = a.context_lens + r0;
    p.tree = a.tree_mask != nullptr ? a.tree_mask + row * p.words : nullptr;
    char *ws = static_cast<char *>(a.workspace);
    const size_t slots = static_cast<size_t>(grid) * 2 * rows;
    p.tickets = reinterpret_cast<unsigned long long *>(ws);
    ws += mk_round(static_cast<size_t>(std::min(a.num_requests, kMkMaxRequests)) * H * p.T * 8);
    p.o_part = reinterpret_cast<float *>(ws);
    ws += mk_round(slots * kHeadDim * sizeof(float));
    p.ml_part = reinterpret_cast<float2 *>(ws);
    p.tag = next_call_tag();
    const cudaError_t e = rows == 32    ? mk_launch<false, 32>(p, mk, mv, grid, stream)
                          : rows == 128 ? mk_launch<false, 128>(p, mk, mv, grid, stream)
                                        : mk_launch<true, 128>(p, mk, mv, grid, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kvq
