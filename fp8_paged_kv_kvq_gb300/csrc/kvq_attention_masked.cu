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
//    sees, in chunks.  Two chains (QK^T -> softmax -> PV) work on a unit: of more
//    than 128 rows each has a 128-row tile of its own over all chunks (kPair), of
//    fewer they share a tile, take the chunks in turn, and their sums and outputs are
//    joined at the end.  Of at most 32 (64) rows a unit is four (two) KV heads side by
//    side, 32 (64) of the tensor core's 128 rows each; its chunk is 32 (64) tokens of
//    each head, and a row's weights are 0 at the other heads' keys.  All four warps of
//    a softmax have work so, and one copy brings a page's tokens of four heads
//    (window of 64 requests, a unit per head: 172 us, per four heads 125).
//  * Tokens.  A unit's tokens are numbered without the gap between sinks and
//    window: x < S16 is position x, the others x + shift (both parts start on a
//    multiple of 16 tokens), so that a few sinks cost no chunk of their own.
//  * Split.  The chunks of all units, in order, with a charge for each unit's start,
//    are cut into one equal range per SM; a unit that is cut leaves a piece per range
//    (normalised output, reference, denominator) in the workspace, which a second
//    launch joins, with all SMs (joined by the block whose piece came last, 175 rows in
//    7 pieces took it 34 us).
//  * Stages.  A chunk's K and V codes are copied by TMA, 16 tokens (of a tree and one head
//    the whole page) and all the unit's heads a copy; of a last group of fewer heads the
//    boxes are those heads wide, so that every box lies within its plane.  kPair: two stages, values converted
//    into two f16 buffers of their own.  Else five stages, values converted in place,
//    over the chunk's own keys (once its scores are made) and codes: the copies in flight
//    are what bounds a step's time with few rows (with separate buffers and three stages
//    the window of 64 requests took 125 us, in place 115).
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
//    see, or one of another head of the unit, can raise Eg to 30, no more, so that it costs
//    no precision to rows of values above 2^-60 (it can move the roundings of others).
//  * Unseen tokens take no part: their scores become -infinity before the exponential,
//    value scales that are not finite become 0, and value rows with a NaN code are cleared
//    (0 times NaN is NaN) in chunks that some row of the unit does not see whole and, where
//    a unit has several heads, in all chunks, since the product runs over the other heads'
//    keys with weights of 0.  What was cleared is noted, and a row that sees it becomes NaN:
//    by its softmax warp, or, of a chunk that all rows see, by the epilogue for the head.
//  * Roles, 512 threads: warps 0-3 and 4-7 the softmax of chain 0 and 1 (a thread owns
//    a TMEM lane, a row), 8-11 the value codes' conversion and the epilogue, 12 the
//    units and the copies of codes, 13 and 14 the MMAs of chain 0 and 1, 15 the scales.
//    Every wait is bounded; a role that gives up raises a shared abort flag, copies and
//    MMAs in flight complete, the block frees its tensor memory (KVQ_ERRF_WAIT_TIMEOUT).
//  * What bounds it.  Few rows: memory, once the batch is large; a chunk of 32 KB costs
//    1,094 tensor cycles (two pieces of the query, all 128 rows), 1,460 at the measured
//    copy rate, and takes some 1,850: two chains in flight, whose score, softmax, product and
//    their hand-overs follow one another, and five stages.  Window of 4,096 over 64 requests
//    (421 MB): 87 us replayed in a graph, 72% of the measured copy rate, 89 us and 70% in calls
//    on other inputs each time; trees of 8 nodes over 128 requests (891 MB) 180 us and 73%, 190
//    us and 69%.  That is this form's limit, not the operator's: attn_stream_kernel copies the
//    same boxes for at most 8 stacked rows at 77%.  kPair: a step of both chains costs 2,190
//    tensor cycles and takes some 5,000; the softmax of a chain, 2,900 cycles of dependent
//    instructions in one warp per scheduler, is as long as its products and the other chain's
//    together, and no single part of it is the limit (taken out of a form of 582 us: loading
//    scales 554, exponentials 584, the search for the largest 569, three quarters of the
//    conversion's stores 571).  The nearest limit is instruction fetch (84% of its peak, 90% of
//    requests hit): layouts of the same code differ by several percent.  4 x 2,048 rows of 32 /
//    8 heads, window 4,096: 596 us in a graph, 48% of the measured bf16 product rate.  Small
//    calls are latency: one row over 1,028 tokens 16 us: set-up 1, unit 2.4, pages 3.3, keys
//    4.2, queries 5.3, then three chunks, epilogue, and 4 us of the join, a second launch that
//    every call makes.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kMkTok = 128;                           // keys of a chunk: (token, KV head) pairs
constexpr int kMkWarpConv = 8, kMkWarpLoad = 12, kMkWarpMma = 13, kMkWarpScale = 15;
constexpr int kMkThreads = 512;
constexpr int kMkUnits = 8;                           // units announced ahead
constexpr int kMkMaxRequests = 1024;                  // of a launch
constexpr float kMkLazy = 14.0f;                      // log2 of the largest P''
constexpr float kMkFloor = -90.0f;                    // log2 of the smallest value scale, over 2^Eg
constexpr int kMkMaxEg = 30;                          // Eg at most

// A unit as the loading warp announces it: the chunks [c0, c0 + n) of the rows from row0
// on of the heads from h on of request r, of X tokens (x < s16 is position x, others x +
// shift); all of them (direct) or a piece, for workspace slot `slot`.  base: the position
// of query row 0.  n = 0 ends the work.
struct __align__(16) MkUnit {
  int r, h, row0, n;
  int c0, X, s16, shift;
  int base, direct, slot, pad;
};

// Shapes: kPair (two row tiles of one head, one per chain), or one tile of kRows rows of
// each of 128 / kRows heads, whose chunks the chains share.
template <bool kPair, int kRows>
struct MkShape {
  static constexpr int kTileRows = kPair ? 256 : kRows;      // rows of a unit, per head
  static constexpr int kLanes = kPair ? 256 : 128;           // of all its heads
  static constexpr int kHeads = 128 / kRows;
  static constexpr int kTok = kMkTok / kHeads;               // tokens of a chunk
  // Chunks that a unit's start counts for: its queries are read and converted and the chains
  // run empty.  (Window of 64 requests: 98 us with 2, 89 with 6 and with 8, 91 with 13; tree
  // batch 198, 185, 184, 187.  Chunks of prompts: 589 with 1, 586 with 2, 584 with 3; 5 trees
  // of 25 nodes 44, 40, 42.)
  static constexpr int kCharge = kPair ? 2 : 8;
  static constexpr int kTokLog2 = kRows == 32 ? 5 : (kRows == 64 ? 6 : 7);
  static constexpr int kQTiles = kPair ? 2 : 1;
  // shared memory, offsets from a 1024-byte aligned base
  // Code stages of a chunk.  kPair: values are converted into two
  // buffers of their own.  Else in place, over the chunk's key codes (which S has been made
  // of) and its value codes, so that five chunks are on their way or at work.
  static constexpr int kStages = kPair ? 2 : 5;
  static constexpr int kVfs = kPair ? 2 : kStages;
  static constexpr int kScales = kPair ? 6 : kStages;        // chunks of scales in their ring
  static constexpr int kStage = 2 * kMkTok * kHeadDim;       // the chunk's K codes, then its V codes
  static constexpr int kVOff = kMkTok * kHeadDim;
  static constexpr int kGroup = 8 * kHeadDim;                // 8 rows
  static constexpr int kQPiece = 128 * kHeadDim;
  static constexpr int kOffQ = 0;                            // [tile][piece]
  static constexpr int kVfBytes = kMkTok * kHeadDim * 2;     // f16 values of a chunk
  static constexpr int kOffKv = kOffQ + kQTiles * 2 * kQPiece;
  static constexpr int kOffVf = kPair ? kOffKv + kStages * kStage : kOffKv;
  static constexpr int kOffSum = kOffKv + kStages * kStage + (kPair ? 2 * kVfBytes : 0);   // [chain][128] denominators
  static constexpr int kOffRef = kOffSum + 2 * 128 * 4;      // [chain][128] references
  static constexpr int kOffEg = kOffRef + 2 * 128 * 4;       // [chain]
  static constexpr int kOffSc = kOffEg + 16;                 // [stage][K | V | log2 V][128]
  static constexpr int kOffMeta = kOffSc + kScales * 3 * kMkTok * 4;   // [stage] float4
  static constexpr int kOffUnit = kOffMeta + kScales * 16;
  static constexpr int kOffBad = kOffUnit + kMkUnits * static_cast<int>(sizeof(MkUnit));   // [Vf][4 words], [scales][4 words]
  static constexpr int kOffMisc = kOffBad + (kVfs + kScales) * 16;              // tmem base, abort
  static constexpr int kOffNan = kOffMisc + 16;              // [unit, odd or even][warp] heads with a NaN
  static constexpr int kOffScan = kOffNan + 2 * 4 * 4;       // a warp's sum each
  static constexpr int kOffPre = kOffScan + kMkThreads / 32 * 4;
  static constexpr int kOffBar = (kOffPre + (kMkMaxRequests + 1) * 4 + 7) / 8 * 8;
  static constexpr int kKvFull = 0;
  static constexpr int kKvEmpty = kKvFull + kStages;
  static constexpr int kVfFull = kKvEmpty + kStages;
  // (kPair; else kVfFull: cleared values of a chunk noted, per chain, kVfEmpty: those of a
  // unit's whole chunks, odd and even units)
  static constexpr int kVfEmpty = kVfFull + 2;
  static constexpr int kScFull = kVfEmpty + 2;
  static constexpr int kScEmpty = kScFull + kScales;
  static constexpr int kQFull = kScEmpty + kScales;        // per chain from here on
  static constexpr int kQEmpty = kQFull + 2;
  static constexpr int kSFull = kQEmpty + 2;
  static constexpr int kPReady = kSFull + 2;                 // (per chain and half of the chunk)
  static constexpr int kOFull = kPReady + 4;
  static constexpr int kOEmpty = kOFull + 2;
  static constexpr int kSumFull = kOEmpty + 2;
  static constexpr int kTurn = kSumFull + 2;
  static constexpr int kDrain = kTurn + 2;
  static constexpr int kQRows = kDrain + 2;                  // (of a shared tile, per 32 rows)
  static constexpr int kUnitFull = kQRows + 4;
  static constexpr int kUnitEmpty = kUnitFull + kMkUnits;
  static constexpr int kBars = kUnitEmpty + kMkUnits;
  static constexpr int kSmem = kOffBar + 8 * kBars + 1024;
  static_assert(kStage == kVfBytes && kOffKv % 1024 == 0 && kOffVf % 1024 == 0 && kOffSc % 16 == 0 && kOffMeta % 16 == 0 &&
                    kOffUnit % 16 == 0 && kOffBad % 16 == 0 && kOffMisc % 16 == 0 && kOffBar % 8 == 0,
                "alignment");
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kBars <= kMkThreads, "a thread initialises each barrier");
};

// TMEM: S of chain a at 128 a (P'' of each half of its tokens over the first 32 columns
// of that half), O at 256 + 128 a
constexpr uint32_t kMkTmemCols = 512;
__device__ __forceinline__ uint32_t mk_s(int a) { return 128u * a; }
__device__ __forceinline__ uint32_t mk_o(int a) { return 256u + 128u * a; }

constexpr uint32_t kMkIdescQK = mma_idesc(128, kMkTok, false, false);        // e4m3
constexpr uint32_t kMkIdescPV = mma_idesc(128, kHeadDim, false, true);       // f16, B MN-major
// The operands' shared-memory descriptors (smem_desc: stride offset, version 1, 128-byte
// swizzle), upper words and the two leading offsets.
constexpr uint32_t kMkDescHi = (1024u >> 4) | (1u << 14) | (kSmemSwizzle128 << 29);
constexpr uint32_t kMkKMajor = 1u << 16;

__device__ __forceinline__ void mk_mma_qk(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t b_hi,
                                          uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %6};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}\n"
      :: "r"(d), "r"(a_lo), "r"(b_lo), "n"(kMkIdescQK), "r"(acc), "n"(kMkDescHi), "r"(b_hi)
      : "memory");
}
__device__ __forceinline__ void mk_mma_pv(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi,
                                          uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n"
      :: "r"(d), "r"(a_tmem), "r"(b_lo), "n"(kMkIdescPV), "r"(acc), "r"(b_hi) : "memory");
}

// One box of a copy: a plane's codes of some heads, from group z of 8 slots on.
__device__ __forceinline__ void mk_load_box(uint32_t dst, const void *tmap, int z, int head,
                                            uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %2, %3, %4}], [%5], %6;\n"
      :: "r"(dst), "l"(tmap), "r"(0), "r"(z), "r"(head), "r"(bar), "l"(policy) : "memory");
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
  uint32_t inv_g;                                      // ceil(2^32 / G), G > 1
  int32_t T, HG;                                       // units of a request and group of heads, groups
  int32_t width;                                       // max_blocks_per_req
  int32_t ctx_limit, num_blocks, log2_bs, box;
  int32_t tail;                                        // the first head of a last group of fewer heads, else H
  int32_t window, sinks, words;
  float scale2;                                        // |sm_scale| log2(e)
  uint32_t flip;                                       // sign bits of a negative sm_scale
  float *o_part;                                       // [grid][2][lanes of a unit][128]
  float2 *ml_part;                                     // [grid][2][lanes of a unit]
  int4 *cuts;                                          // [grid]: the unit that block b is the first of several to work on
  int32_t *err_flags;
  int32_t least;                                       // positions of a block's range
};

// The planes' maps: whole groups of heads, and the last group's where it has fewer.
struct MkMaps {
  CUtensorMap k, v, k_tail, v_tail;
};

// m / G, m < 2^13: exact, since m (inv_g G - 2^32) < 2^26
__device__ __forceinline__ int mk_query(const MkParams &p, int m) {
  return p.G == 1 ? m : static_cast<int>(__umulhi(static_cast<uint32_t>(m), p.inv_g));
}

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

// Bounded wait (about a second) that also gives up once another role raised the abort
// flag.  One small loop: it is at every wait, and the roles share an instruction cache.
__device__ __forceinline__ bool mk_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
#pragma unroll 1
  for (int i = 0; i < (1 << 19); ++i) {
    if (mbar_try_wait_sleep(bar, parity, 2000u)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  return false;
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
  const int first = mk_query(p, t * kTileRows), last = mk_query(p, min(p.M, (t + 1) * kTileRows) - 1);
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

template <typename S>
__device__ __forceinline__ int mk_positions(int X) {   // of a unit in the work sequence
  return X > 0 ? ((X + S::kTok - 1) >> S::kTokLog2) + S::kCharge : 0;
}

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
  const int i = mk_query(p, min(m, p.M - 1));          // (rows past the last see what it sees)
  const int own = u.base + i;
  s.hi = own + 1 - u.shift;
  s.lo = max(own - p.window + 1, u.s16 + u.shift) - u.shift;
  s.base = u.base;
  s.words = p.tree + (static_cast<int64_t>(u.r) * p.R + i) * p.words;
  return s;
}
// The chunks of a unit (numbered from its piece's first) that the rows from a first to a
// last one see whole: those below `hi` that are below `sink` or not below `lo`.
struct MkWhole {
  int hi, sink, lo;
  __device__ __forceinline__ bool at(int k) const { return k < hi && (k < sink || k >= lo); }
};
template <typename S>
__device__ __forceinline__ MkWhole mk_whole(const MkParams &p, const MkUnit &u, int hi_first,
                                            int lo_last) {
  constexpr int kLog2 = S::kTokLog2;
  if (p.tree != nullptr) return MkWhole{(u.base >> kLog2) - u.c0, 0, 0};
  return MkWhole{(hi_first >> kLog2) - u.c0, (p.sinks >> kLog2) - u.c0,
                 ((lo_last + S::kTok - 1) >> kLog2) - u.c0};
}
template <typename S>
__device__ __forceinline__ MkWhole mk_unit_whole(const MkParams &p, const MkUnit &u) {
  return mk_whole<S>(p, u, mk_seen(p, u, u.row0).hi, mk_seen(p, u, u.row0 + S::kTileRows - 1).lo);
}

// ---------------------------------------------------------------------------
// Softmax pieces.

struct MkRow {
  float m = -INFINITY;                                 // reference
  float sum = 0.0f;                                    // denominator under it
  int eg = 0;                                          // value scales are held over 2^eg
};

// 16 columns of this thread's TMEM lane, not waited for; done: after tmem_wait_ld, before
// any use.
__device__ __forceinline__ void mk_ld16_start(uint32_t taddr, float *x) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
               "%11, %12, %13, %14, %15}, [%16];\n"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
               : "r"(taddr) : "memory");
}
__device__ __forceinline__ void mk_ld16_done(float *x) {
  asm volatile("" : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]), "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15]) :: "memory");
}

// max_j (u_j + log2 of the value scale) over 16 tokens, those of `bits`.
__device__ __forceinline__ float mk_top16(const float (&x)[16], const float *ks, const float *lg,
                                          uint64_t rowf, uint32_t bits, float top) {
  float m[2] = {top, -INFINITY};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 k4 = reinterpret_cast<const float4 *>(ks)[q];
    const float4 l4 = reinterpret_cast<const float4 *>(lg)[q];
    const uint64_t kk[2] = {pack_f32x2(k4.x, k4.y), pack_f32x2(k4.z, k4.w)};
    const uint64_t ll[2] = {pack_f32x2(l4.x, l4.y), pack_f32x2(l4.z, l4.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 4 * q + 2 * i;
      float a, b;
      unpack_f32x2(fma_f32x2(mul_f32x2(pack_f32x2(x[e], x[e + 1]), kk[i]), rowf, ll[i]), a, b);
      a = (bits >> e) & 1u ? a : -INFINITY;
      b = (bits >> (e + 1)) & 1u ? b : -INFINITY;
      m[i] = mk_max3(m[i], a, b);
    }
  }
  return fmaxf(m[0], m[1]);
}

// The reference moved where `top` is far above it, the denominator and (unless the
// chain has no earlier chunk of the unit) the O row brought under the new one.  de: by
// how much 2^Eg grew; weights stay as large as they were under a reference that is
// lower by as much (as long as the denominator stays below 2^100).
__device__ __forceinline__ void mk_meet(MkRow &row, float top, int de, bool fresh, uint32_t ocol) {
  const bool unset = row.m == -INFINITY;
  const float keep = row.m - static_cast<float>(de == 0 ? 0 : min(de, 100 - mk_ceil_log2(row.sum)));
  const bool move = unset ? top > -INFINITY : top - keep > kMkLazy;
  const float next = move ? top : keep;
  const float f = unset ? 1.0f : mk_ex2(row.m - next), fo = f * mk_pow2_down(-de);
  row.m = next;
  row.sum *= f;
  if (!fresh && __any_sync(0xFFFFFFFFu, fo != 1.0f && !unset)) {
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
}

// P'' of 16 scores as f16 in w, the sum of the p added to `sum`; tokens that are not in
// `bits` (kMasked) have p = 0.
template <bool kMasked>
__device__ __forceinline__ void mk_part16(const float *x, const float *ks, const float *vs,
                                          uint64_t rowf, uint64_t shift, uint32_t bits,
                                          uint64_t (&sum)[2], uint32_t (&w)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 k4 = reinterpret_cast<const float4 *>(ks)[q];
    const float4 v4 = reinterpret_cast<const float4 *>(vs)[q];
    const uint64_t kk[2] = {pack_f32x2(k4.x, k4.y), pack_f32x2(k4.z, k4.w)};
    const uint64_t vv[2] = {pack_f32x2(v4.x, v4.y), pack_f32x2(v4.z, v4.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 4 * q + 2 * i;
      float a, b;
      unpack_f32x2(fma_f32x2(mul_f32x2(pack_f32x2(x[e], x[e + 1]), kk[i]), rowf, shift), a, b);
      if (kMasked) {
        a = (bits >> e) & 1u ? a : -INFINITY;
        b = (bits >> (e + 1)) & 1u ? b : -INFINITY;
      }
      const uint64_t p = pack_f32x2(mk_ex2(a), mk_ex2(b));
      sum[i] = mk_add2(sum[i], p);
      unpack_f32x2(mul_f32x2(p, vv[i]), a, b);
      w[2 * q + i] = pack_f16x2(a, b);
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

// A row's keys of a chunk: groups of 16 tokens, group g at the scores' (and the scales')
// column 16 (kHeads g + its head), its P'' at column mk_pcol of that (the halves of the 128
// keys each start at their own scores' place).
template <int kHeads>
__device__ __forceinline__ int mk_col(int g, int hu) {
  return 16 * (kHeads * g + hu);
}
__device__ __forceinline__ int mk_pcol(int col) { return (col & 64) + ((col & 63) >> 1); }

// The other heads' P'' columns of half h are 0.
template <int kHeads>
__device__ __forceinline__ void mk_zero(uint32_t scol, int h, int hu) {
  if (kHeads == 1) return;
  const uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c % kHeads != hu) tmem_st8u(scol + 64 * h + 8 * c, z);
}

// One chunk of one row whose warp sees all of it: S from TMEM, the row's statistics
// brought up to date, P'' over S's columns, its halves announced one after the other.
// ks: the chunk's key scales, value scales and their log2; meta: the largest key scale,
// the log2 of the largest value scale, Eg.
template <int kHeads, bool kHalves>
__device__ __forceinline__ void mk_softmax(uint32_t scol, uint32_t ocol, const float *ks,
                                           const float4 meta, float rowf, int hu, bool fresh,
                                           uint32_t ready, int lane, MkRow &row) {
  constexpr int kGroups = 8 / kHeads, kHalf = kGroups / 2;
  const int eg = __float_as_int(meta.z);
  const int de = fresh ? 0 : eg - row.eg;
  row.eg = eg;
  const float *vs = ks + kMkTok, *lg = vs + kMkTok;
  const uint64_t rf = pack_f32x2(rowf, rowf);
  // Scores in registers: of one head, 64 of the 128 at a time.
  constexpr int kRegs = kGroups > 4 ? 4 : kGroups;     // groups
  float x[16 * kRegs];
  auto load = [&](int h) {
    if (kHeads == 1) {
      tmem_ld64(scol + 64 * h, x);
    } else {
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        mk_ld16_start(scol + mk_col<kHeads>(g, hu), x + 16 * g % (16 * kRegs));
      tmem_wait_ld();
#pragma unroll
      for (int g = 0; g < kRegs; ++g) mk_ld16_done(x + 16 * g);
    }
  };
  // the largest a score can be under the chunk's largest scales
  float mx[2] = {0.0f, 0.0f};
#pragma unroll 1
  for (int h = kHeads == 1 ? 1 : 0; h >= 0; --h) {
    load(h);
#pragma unroll
    for (int i = 0; i < 16 * kRegs; i += 4)
#pragma unroll
      for (int q = 0; q < 2; ++q) mx[q] = mk_max3(mx[q], x[i + q], x[i + q + 2]);
  }
  const float most = fmaxf(mx[0], mx[1]) * meta.x * rowf + meta.y;
  if (de != 0 || __any_sync(0xFFFFFFFFu, !(most - row.m <= kMkLazy))) {
    float top = -INFINITY;
#pragma unroll 1
    for (int g = 0; g < kGroups; ++g) {
      float y[16];
      const int col = mk_col<kHeads>(g, hu);
      tmem_ld16(scol + col, y);
      top = mk_top16(y, ks + col, lg + col, rf, 0xFFFFu, top);
    }
    mk_meet(row, top, de, fresh, ocol);
  }
  const float sh = row.m == -INFINITY ? 0.0f : -row.m;
  const uint64_t s2 = pack_f32x2(sh, sh);
  uint64_t sum[2] = {pack_f32x2(0.0f, 0.0f), pack_f32x2(0.0f, 0.0f)};
  // (a half's P'' lies over its own scores, or of several heads over others')
#pragma unroll 1
  for (int h = 0; h < (kHeads == 1 ? 2 : 1); ++h) {
    if (h == 1) load(1);
#pragma unroll
    for (int g = 0; g < kRegs; ++g) {
      uint32_t w[8];
      const int col = mk_col<kHeads>(kHeads == 1 ? 4 * h + g : g, hu);
      mk_part16<false>(x + 16 * g, ks + col, vs + col, rf, s2, 0u, sum, w);
      tmem_st8u(scol + mk_pcol(col), w);
      if ((g + 1) % kHalf == 0) {
        const int half = kHeads == 1 ? h : g / kHalf;
        mk_zero<kHeads>(scol, half, hu);
        if (kHalves || half == 1) mk_announce(ready + (kHalves ? 8 * half : 0), lane);
      }
    }
  }
  float a, b;
  unpack_f32x2(mk_add2(sum[0], sum[1]), a, b);
  row.sum += a + b;
}

// The same where some of the warp's rows do not see some of the chunk's tokens, from x0
// on: seldom, so small rather than fast (the roles share an instruction cache).  bad:
// keys whose value was cleared, 16 a word; returns whether the row sees one of them.
template <int kHeads, bool kHalves>
__device__ __forceinline__ bool mk_softmax_masked(const MkParams &p, const MkSeen &seen, int x0,
                                                  int X, const uint16_t *bad, const uint16_t *bad_sc,
                                                  uint32_t scol, uint32_t ocol, const float *ks,
                                                  const float4 meta, float rowf, int hu, bool fresh,
                                                  uint32_t ready, int lane, MkRow &row) {
  constexpr int kGroups = 8 / kHeads, kHalf = kGroups / 2;
  const int eg = __float_as_int(meta.z);
  const int de = fresh ? 0 : eg - row.eg;
  row.eg = eg;
  const float *vs = ks + kMkTok, *lg = vs + kMkTok;
  const uint64_t rf = pack_f32x2(rowf, rowf);
  float top = -INFINITY;
  uint64_t lo = 0u, hi = 0u;                           // what the row sees, 16 bits a group
  uint32_t hit = 0u, word = 0u;
#pragma unroll 1
  for (int g = 0; g < kGroups; ++g) {
    float x[16];
    const int col = mk_col<kHeads>(g, hu);
    word = (g & 1) == 0 ? seen.bits(p, x0 + 16 * g, X) : word >> 16;
    const uint32_t bits = word & 0xFFFFu;
    hi = (hi >> 16) | (lo << 48);
    lo = (lo >> 16) | (static_cast<uint64_t>(bits) << 48);
    hit |= bits & (bad[col >> 4] | (meta.w != 0.0f ? bad_sc[col >> 4] : 0u));
    tmem_ld16(scol + col, x);
    top = mk_top16(x, ks + col, lg + col, rf, bits, top);
  }
  mk_meet(row, top, de, fresh, ocol);
  const float sh = row.m == -INFINITY ? 0.0f : -row.m;
  uint64_t sum[2] = {pack_f32x2(0.0f, 0.0f), pack_f32x2(0.0f, 0.0f)};
  // (the groups' bits: the first are the lowest 16 of hi, or of what of lo is in use)
  uint64_t bits = kGroups == 8 ? hi : (kGroups == 4 ? lo : lo >> 32);
#pragma unroll 1
  for (int g = 0; g < kGroups; ++g) {
    float x[16];
    uint32_t w[8];
    const int col = mk_col<kHeads>(g, hu);
    tmem_ld16(scol + col, x);
    mk_part16<true>(x, ks + col, vs + col, rf, pack_f32x2(sh, sh), static_cast<uint32_t>(bits) & 0xFFFFu,
                    sum, w);
    bits >>= 16;
    if (kGroups == 8 && g == 3) bits = lo;
    tmem_st8u(scol + mk_pcol(col), w);
    if ((g + 1) % kHalf == 0) {
      mk_zero<kHeads>(scol, g / kHalf, hu);
      if (kHalves || g / kHalf == 1) mk_announce(ready + (kHalves ? 8 * (g / kHalf) : 0), lane);
    }
  }
  float a, b;
  unpack_f32x2(mk_add2(sum[0], sum[1]), a, b);
  row.sum += a + b;
  return hit != 0u;
}

// Query rows wait for their largest magnitude in their pieces' own place in a K-major,
// 128-byte swizzled tile (two pieces of 128 bytes a row): of 16 dims, the first 8 where the
// first piece goes, the others where the second goes.
__device__ __forceinline__ uint8_t *mk_query_place(uint8_t *tile, int row, int c) {   // dims 8 c ..
  return tile + (c & 1) * 128 * kHeadDim + row * kHeadDim + (((c >> 1) ^ (row & 7)) << 4);
}
// The row's largest magnitude, as bf16 bits.
__device__ __forceinline__ uint32_t mk_query_top(uint8_t *tile, int row) {
  uint32_t mg = 0u;
#pragma unroll 4
  for (int c = 0; c < 16; ++c) {
    const uint4 v = *reinterpret_cast<const uint4 *>(mk_query_place(tile, row, c));
    mg = __vmaxu2(mg, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
    mg = __vmaxu2(mg, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  }
  return max(mg & 0xFFFFu, mg >> 16);
}
// e4m3 pieces of two elements that f16 holds: p1 = e4m3(x), p2 = e4m3(x - p1).
__device__ __forceinline__ void mk_pieces2(uint32_t x, uint32_t &p1, uint32_t &p2) {
  asm("{\n .reg .b16 a, b;\n .reg .b32 y, z;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 a, %2;\n cvt.rn.f16x2.e4m3x2 y, a;\n sub.rn.f16x2 z, %2, y;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 b, z;\n cvt.u32.u16 %0, a;\n cvt.u32.u16 %1, b;\n}\n"
      : "=r"(p1), "=r"(p2) : "r"(x));
}
// Dims [16 c0, 16 c1) of the row, largest magnitude `top`, as two e4m3 pieces (x = 2^e (p1
// + p2); elements below 2^-14 of 2^e in f16 are 2^-32 of the largest); returns 2^e |sm_scale|
// log2(e), which takes the row's scores to log2 units.
__device__ __forceinline__ float mk_query_pieces(uint8_t *tile, int row, int c0, int c1,
                                                 uint32_t top, float scale2, uint32_t flip) {
  const int ex = static_cast<int>(top >> 7);
  int e = ex == 0 ? -126 : ex - 127 - 7;
  e = e < -126 ? -126 : e;
  const float inv = top == 0u ? 0.0f : mk_pow2(-e);
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    uint4 *to1 = reinterpret_cast<uint4 *>(mk_query_place(tile, row, 2 * c)), *to2 = to1 + 8 * kHeadDim;
    const uint4 y[2] = {*to1, *to2};
    uint32_t p1[8], p2[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 &q = y[i >> 2];
      const uint32_t w = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
      mk_pieces2(pack_f16x2(bf16_lo(w) * inv, bf16_hi(w) * inv), p1[i], p2[i]);
    }
    *to1 = make_uint4((p1[0] | p1[1] << 16) ^ flip, (p1[2] | p1[3] << 16) ^ flip,
                      (p1[4] | p1[5] << 16) ^ flip, (p1[6] | p1[7] << 16) ^ flip);
    *to2 = make_uint4((p2[0] | p2[1] << 16) ^ flip, (p2[2] | p2[3] << 16) ^ flip,
                      (p2[4] | p2[5] << 16) ^ flip, (p2[6] | p2[7] << 16) ^ flip);
  }
  // (a row with an infinity or a NaN has no scores)
  return ex == 255 ? __uint_as_float(0x7FC00000u) : mk_pow2(e) * scale2;
}

template <bool kPair, int kRows>
__global__ void __launch_bounds__(kMkThreads, 1)
attn_masked_kernel(const MkParams p, const __grid_constant__ MkMaps maps) {
  using S = MkShape<kPair, kRows>;
  extern __shared__ uint8_t smem_raw[];
  // (an offset from the array, not a rounded address: the compiler keeps to shared memory)
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bar0 = smem_addr(smem + S::kOffBar);
  auto BAR = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffMisc);
  volatile int *abort_s = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
  MkUnit *unit_s = reinterpret_cast<MkUnit *>(smem + S::kOffUnit);
  volatile float *sum_s = reinterpret_cast<volatile float *>(smem + S::kOffSum);
  volatile float *ref_s = reinterpret_cast<volatile float *>(smem + S::kOffRef);
  volatile int *eg_s = reinterpret_cast<volatile int *>(smem + S::kOffEg);
  uint32_t *bad_s = reinterpret_cast<uint32_t *>(smem + S::kOffBad);
  volatile uint32_t *nan_s = reinterpret_cast<volatile uint32_t *>(smem + S::kOffNan);
  int *pre = reinterpret_cast<int *>(smem + S::kOffPre);

  allow_dependents_launch();
  if (tid < S::kBars) {
    uint32_t count = 1;
    const int i = tid;
    // commits of the chains that read it, and arrivals of the converting warps
    if (i >= S::kVfEmpty && i < S::kVfEmpty + 2) count = kPair ? 2 : 4;
    if (i >= S::kVfFull && i < S::kVfFull + 2) count = 4;
    if (i >= S::kKvFull && i < S::kKvFull + S::kStages) count = kPair ? 1 : 2;   // copies, scales
    if (i >= S::kKvEmpty && i < S::kKvEmpty + S::kStages) count = kPair ? 4 + 2 : 1;
    if (i >= S::kScEmpty && i < S::kScEmpty + S::kScales) count = 8;
    if (i >= S::kQFull && i < S::kQFull + 2) count = kPair ? 4 : 8;
    if (i >= S::kQRows && i < S::kQRows + 4) count = 2;  // the chains' warps of those rows
    if (i >= S::kPReady && i < S::kPReady + 4) count = kPair ? 4 : 8;   // a chain's softmax; values
    if ((i >= S::kOEmpty && i < S::kOEmpty + 2) || (i >= S::kSumFull && i < S::kSumFull + 2))
      count = 4;                                       // a chain's softmax or the epilogue
    if (i >= S::kUnitEmpty && i < S::kUnitEmpty + kMkUnits)
      count = 8 + 4 + 2 + 1;                           // softmax, conversion, MMAs, scales
    mbar_init(BAR(i), count);
    fence_mbarrier_init();
  }
  if (tid == 0) *abort_s = 0;
  // (The maps are not prefetched: a form that did, with other maps, faulted now and then for a
  // reason that was not found.)
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
#pragma unroll 1
    for (int t = 0; t < p.T; ++t) w += mk_positions<S>(mk_span<S::kTileRows>(p, Lc, t).X);
    return w * p.HG;
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
  const int B = max(p.least, static_cast<int>((static_cast<int64_t>(total) + gridDim.x - 1) / gridDim.x));

  // Unit t of this block is announced (unit_s[t % kMkUnits], read where it is needed:
  // registers are few); each warp of the other roles releases it once.
  auto wait_unit = [&](int t) -> bool {
    return mk_wait_all(BAR(S::kUnitFull + t % kMkUnits), (t / kMkUnits) & 1, abort_s);
  };
  auto release_unit = [&](int t) {
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(S::kUnitEmpty + t % kMkUnits));
  };
  // chunks of chain a in a unit, and whether it has any
  auto chain_chunks = [&](const MkUnit &u, int a) -> int {
    if (kPair) return a == 0 || u.row0 + 128 < p.M ? u.n : 0;
    return (u.n + 1 - a) / 2;
  };
  bool gave_up = false;

  if (warp < kMkWarpConv) {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n");
    const int a = warp >> 2, q4 = warp & 3;
    const int lane_row = 32 * q4 + lane;               // TMEM lane
    const int hu = kPair ? 0 : lane_row / kRows;       // its head and its row, of the unit's
    const int trow = kPair ? 128 * a + lane_row : lane_row % kRows;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    uint32_t steps = 0, done = 0, seq = 0;             // chunks and units of this chain, chunks of all
    uint32_t sc = 0, sc_par = 0;                       // place in the scales' ring
    uint32_t edge_par = 0;
    uint32_t q_units = 0;                              // units with rows of chain a
    for (int t = 0;; ++t) {
      if (!wait_unit(t)) {
        gave_up = true;
        break;
      }
      const MkUnit &u = unit_s[t % kMkUnits];
      const int un = u.n, n = chain_chunks(u, a);
      if (un == 0) break;
      float rowf = 0.0f;
      if (!kPair || n > 0) {
        // the warp's queries; the tile's space is free once the last unit's products with it
        // are done.  (Where the chains share a tile, a warp of each has half of its rows to
        // load and half of their dims to convert.)
        bool ok = true;
        if (kPair) {
          if (q_units > 0) ok = mk_wait_all(BAR(S::kQEmpty + a), (q_units - 1) & 1, abort_s);
        } else {
          if (q_units > 0)
            ok = mk_wait_all(BAR(S::kQEmpty), (q_units - 1) & 1, abort_s) &&
                 mk_wait_all(BAR(S::kQEmpty + 1), (q_units - 1) & 1, abort_s);
        }
        if (!ok) gave_up = true;
        uint8_t *tile = smem + S::kOffQ + (kPair ? a : 0) * 2 * S::kQPiece;
        const int r0 = kPair ? 0 : 16 * a;
#pragma unroll 1
        for (int r = r0 + (lane >> 4); r < r0 + (kPair ? 32 : 16); r += 2) {
          const int row = 32 * q4 + r, m = u.row0 + (kPair ? 128 * a + row : row % kRows);
          const int head = u.h + (kPair ? 0 : row / kRows), i = mk_query(p, m), c = lane & 15;
          const bool have = m < p.M && head < p.H;
          const int64_t at = (static_cast<int64_t>(u.r) * p.R + i) * p.Hq + head * p.G + (m - i * p.G);
          cp_async_16(mk_query_place(tile, row, c), p.q + (have ? at * kHeadDim + 8 * c : 0), have ? 16u : 0u);
        }
        cp_async_commit();
        cp_async_wait<0>();
        auto both = [&](uint32_t parity) {
          __syncwarp();
          if (kPair) return;
          if (lane == 0) mbar_arrive(BAR(S::kQRows + q4));
          if (!mk_wait_all(BAR(S::kQRows + q4), parity, abort_s)) gave_up = true;
        };
        both(0);
        const uint32_t top = mk_query_top(tile, lane_row);
        both(1);
        rowf = mk_query_pieces(tile, lane_row, kPair ? 0 : 4 * a, kPair ? 8 : 4 * a + 4, top, p.scale2, p.flip);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(S::kQFull + (kPair ? a : 0)));
        if (gave_up) break;
      }
      q_units += kPair ? n > 0 : 1;
      const MkSeen seen = mk_seen(p, u, u.row0 + trow);
      // the warp's first and last row
      const MkWhole whole = mk_whole<S>(p, u, __shfl_sync(0xFFFFFFFFu, seen.hi, 0),
                                     __shfl_sync(0xFFFFFFFFu, seen.lo, 31));
      const MkWhole all_whole = mk_unit_whole<S>(p, u);
      MkRow row;
      bool nan_row = false, fresh = true;
#pragma unroll 1
      for (int k = 0; k < un; ++k, ++seq, sc_par ^= sc == S::kScales - 1, sc = sc == S::kScales - 1 ? 0 : sc + 1) {
        if (!kPair && (k & 1) != a) continue;
        bool ok = !kPair || mk_wait_all(BAR(S::kScFull + sc), sc_par, abort_s);
        if (ok && n > 0) ok = mk_wait_all(BAR(S::kSFull + a), steps & 1, abort_s);
        if (!ok) {
          gave_up = true;
          break;
        }
        if (n > 0) {
          tc_fence_after();
          const float *ks = reinterpret_cast<const float *>(smem + S::kOffSc) + sc * 3 * kMkTok;
          const float4 meta = reinterpret_cast<const float4 *>(smem + S::kOffMeta)[sc];
          const uint32_t ready = BAR(S::kPReady + 2 * a);
          const uint32_t scol = tl + mk_s(a), ocol = tl + mk_o(a);
          const uint16_t *bad = reinterpret_cast<const uint16_t *>(bad_s + 4 * (seq % S::kVfs));
          const uint16_t *bad_sc = reinterpret_cast<const uint16_t *>(bad_s + 4 * (S::kVfs + sc));
          const bool see_all = whole.at(k), edge = !all_whole.at(k);
          // where some row of the unit does not see all of the chunk, value rows with a NaN
          // code have been cleared (scales that are not finite in every chunk)
          if (edge) {
            ok = kPair ? mk_wait_all(BAR(S::kVfFull + seq % S::kVfs), (seq / S::kVfs) & 1, abort_s)
                       : mk_wait_all(BAR(S::kVfFull + a), edge_par, abort_s);
            edge_par ^= 1u;
            if (!ok) {
              gave_up = true;
              break;
            }
          }
          if (see_all) {
            if (edge || meta.w != 0.0f) {
#pragma unroll 1
              for (int g = 0; g < 8 / S::kHeads; ++g) {
                const int c = mk_col<S::kHeads>(g, hu) >> 4;
                if (edge) nan_row |= bad[c] != 0;
                if (meta.w != 0.0f) nan_row |= bad_sc[c] != 0;
              }
            }
            mk_softmax<S::kHeads, kPair>(scol, ocol, ks, meta, rowf, hu, fresh, ready, lane, row);
          } else {
            nan_row |= mk_softmax_masked<S::kHeads, kPair>(p, seen, (u.c0 + k) * S::kTok, u.X, bad, bad_sc, scol,
                                                    ocol, ks, meta, rowf, hu, fresh, ready, lane, row);
          }
          fresh = false;
          ++steps;
        }
        if (kPair) {
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(S::kScEmpty + sc));
        }
      }
      if (gave_up) break;
      release_unit(t);
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
  } else if (warp < kMkWarpLoad) {
    // ------------------------- value codes to f16 values, and the epilogue
    // A unit's epilogue comes after the conversion of the next one's first chunk.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;\n");
    const int q4 = warp & 3;
    const int lane_row = 32 * q4 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    uint32_t par = 0;                                  // barrier parities, bit a
    auto out_row = [&](int r, int h, int m) -> uint16_t * {
      const int i = mk_query(p, m);
      return p.out + ((static_cast<int64_t>(r) * p.R + i) * p.Hq + h * p.G + (m - i * p.G)) * kHeadDim;
    };
    auto epilogue = [&](const MkUnit &u, int t) -> bool {
      // heads that had a NaN code in a chunk that all rows see whole
      uint32_t nan_heads = 0u;
      if (S::kHeads > 1) {
        if (!mk_wait_all(BAR(S::kVfEmpty + (t & 1)), (t >> 1) & 1, abort_s)) return false;
        for (int i = 0; i < 4; ++i) nan_heads |= nan_s[4 * (t & 1) + i];
      }
      const int64_t piece = static_cast<int64_t>(u.slot) * S::kLanes;
      const bool both = !kPair && u.n >= 2;
#pragma unroll 1
      for (int a = 0; a < (kPair ? 2 : 1); ++a) {
        if (chain_chunks(u, a) == 0) continue;
        bool got = mk_wait_all(BAR(S::kSumFull + a), (par >> a) & 1, abort_s) &&
                   mk_wait_all(BAR(S::kOFull + a), (par >> a) & 1, abort_s);
        if (both)
          got = got && mk_wait_all(BAR(S::kSumFull + 1), par >> 1, abort_s) &&
                mk_wait_all(BAR(S::kOFull + 1), par >> 1, abort_s);
        if (!got) return false;
        tc_fence_after();
        par ^= 1u << a;
        if (both) par ^= 2u;
        // the row's parts under their larger reference (one that saw nothing has no
        // reference and a sum of 0, or NaN)
        const float m0 = ref_s[128 * a + lane_row], m1 = both ? ref_s[128 + lane_row] : -INFINITY;
        const float top = fmaxf(m0, m1);
        const float w0 = m0 == -INFINITY ? 0.0f : mk_ex2(m0 - top), w1 = m1 == -INFINITY ? 0.0f : mk_ex2(m1 - top);
        float all = m0 == -INFINITY ? sum_s[128 * a + lane_row] : w0 * sum_s[128 * a + lane_row];
        if (both) all += m1 == -INFINITY ? sum_s[128 + lane_row] : w1 * sum_s[128 + lane_row];
        if (S::kHeads > 1 && (nan_heads >> (lane_row / kRows)) & 1u) all = __uint_as_float(0x7FC00000u);
        const bool none = all == 0.0f;                 // (the row has seen nothing)
        const float f0 = w0 / all * mk_pow2(eg_s[a]), f1 = both ? w1 / all * mk_pow2(eg_s[1]) : 0.0f;
        const int head = u.h + (kPair ? 0 : lane_row / kRows);
        const int m = u.row0 + (kPair ? 128 * a + lane_row : lane_row % kRows);
        const bool mine = m < p.M && head < p.H;
        uint16_t *dst = out_row(u.r, mine ? head : 0, mine ? m : 0);
        const int64_t prow = piece + (kPair ? 128 * a : 0) + lane_row;
        const bool direct = u.direct != 0;
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 32) {
          float o[32];
          tmem_ld32(tl + mk_o(a) + c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = none ? 0.0f : o[i] * f0;
          if (both) {
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              float o1[16];
              tmem_ld16(tl + mk_o(1) + c + h, o1);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[h + i] = none ? 0.0f : fmaf(o1[i], f1, o[h + i]);
            }
          }
          if (mine) {
            if (direct) {
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
        if (!direct && mine) p.ml_part[prow] = make_float2(top, all);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(BAR(S::kOEmpty + a));
          if (both) mbar_arrive(BAR(S::kOEmpty + 1));
        }
      }
      return true;
    };
    // chunk k of a unit, the seq-th of all: thread j converts key j, MN-major and 128-byte
    // swizzled, dims 0-63 and 64-127 in a block each; tokens past the unit's are cleared,
    // and where some row does not see all of the chunk, values with a NaN code.  Of several
    // heads all are: the product runs over the other heads' keys too, whose weights are 0.
    // In place the blocks are the key's and the value's own codes, which one thread reads
    // before it writes.
    const int j = lane_row;
    uint32_t nan_heads = 0u;                           // of the warp's keys in whole chunks of the unit
    uint32_t chain_par = 0;                            // parity of chain a's chunks, bit a
    auto convert = [&](const MkUnit &u, int k, uint32_t seq, bool whole) -> bool {
      const uint32_t b = seq % S::kStages, v = seq % S::kVfs;
      bool ok;
      if (kPair) {
        ok = mk_wait_all(BAR(S::kKvFull + b), (seq / S::kStages) & 1, abort_s);
        if (ok && seq >= 2) ok = mk_wait_all(BAR(S::kVfEmpty + v), ((seq >> 1) - 1) & 1, abort_s);
      } else {
        const int a = k & 1;                           // its scores are made
        ok = mk_wait_all(BAR(S::kSFull + a), (chain_par >> a) & 1, abort_s);
        chain_par ^= 1u << a;
        tc_fence_after();
      }
      if (!ok) return false;
      // (key j: box of 16 tokens and all heads, head, token)
      const int x = (u.c0 + k) * S::kTok + (S::kHeads == 1 ? j : 16 * (j / (16 * S::kHeads)) + (j & 15));
      uint8_t *stage = smem + S::kOffKv + b * S::kStage + (j >> 3) * S::kGroup + (j & 7) * 128;
      const uint8_t *src = stage + S::kVOff;
      uint8_t *dst = kPair ? smem + S::kOffVf + v * S::kVfBytes + j * 128 : stage;
      constexpr int block = S::kVfBytes / 2;
      uint4 w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = *reinterpret_cast<const uint4 *>(src + ((c ^ (j & 7)) << 4));
      bool keep = x < u.X && (S::kHeads == 1 || (j >> 4) % S::kHeads < p.H - u.h);
      if (S::kHeads > 1 || !whole) {
        // (a NaN code is 0x7F but for its sign: one more carries into bit 7, and no further)
        uint32_t bad = 0u;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          bad |= ((w[c].x & 0x7F7F7F7Fu) + 0x01010101u) | ((w[c].y & 0x7F7F7F7Fu) + 0x01010101u) |
                 ((w[c].z & 0x7F7F7F7Fu) + 0x01010101u) | ((w[c].w & 0x7F7F7F7Fu) + 0x01010101u);
        const bool clear = (bad & 0x80808080u) != 0u;
        const uint32_t word = __ballot_sync(0xFFFFFFFFu, keep && clear);
        if (!whole) {
          if (lane == 0) {
            bad_s[4 * v + q4] = word;
            if (!kPair) mbar_arrive(BAR(S::kVfFull + (k & 1)));
          }
        } else {
          // (the warp's keys: 16 of a head, 16 of the next)
          if ((word & 0xFFFFu) != 0u) nan_heads |= 1u << (2 * q4 % S::kHeads);
          if ((word >> 16) != 0u) nan_heads |= 1u << ((2 * q4 + 1) % S::kHeads);
        }
        keep = keep && !clear;
      }
      if (!keep) {
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 lo = make_uint4(e4m3x2_to_f16x2(w[c].x & 0xFFFFu), e4m3x2_to_f16x2(w[c].x >> 16),
                                    e4m3x2_to_f16x2(w[c].y & 0xFFFFu), e4m3x2_to_f16x2(w[c].y >> 16));
        const uint4 hi = make_uint4(e4m3x2_to_f16x2(w[c].z & 0xFFFFu), e4m3x2_to_f16x2(w[c].z >> 16),
                                    e4m3x2_to_f16x2(w[c].w & 0xFFFFu), e4m3x2_to_f16x2(w[c].w >> 16));
        uint8_t *to = dst + (c >> 2) * block;
        *reinterpret_cast<uint4 *>(to + (((2 * (c & 3)) ^ (j & 7)) << 4)) = lo;
        *reinterpret_cast<uint4 *>(to + (((2 * (c & 3) + 1) ^ (j & 7)) << 4)) = hi;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (kPair) mbar_arrive(BAR(S::kKvEmpty + b));
        mbar_arrive(kPair ? BAR(S::kVfFull + v) : BAR(S::kPReady + 2 * (k & 1)));
      }
      return true;
    };
    uint32_t seq = 0;
    int last = -1;                                     // the unit whose epilogue is to come
    for (int t = 0;; ++t) {
      if (!wait_unit(t)) {
        gave_up = true;
        break;
      }
      const MkUnit &u = unit_s[t % kMkUnits];
      const int un = u.n;
      const MkWhole all_whole = mk_unit_whole<S>(p, u);
#pragma unroll 1
      for (int k = 0; k < max(un, 1) && !gave_up; ++k) {
        if (un != 0) {
          gave_up = !convert(u, k, seq, all_whole.at(k));
          ++seq;
          // (the slot of the unit before the last is read by now: this unit's first scores
          // come after all warps' epilogues of it)
          if (S::kHeads > 1 && k == un - 1) {
            if (lane == 0) {
              nan_s[4 * (t & 1) + q4] = nan_heads;
              mbar_arrive(BAR(S::kVfEmpty + (t & 1)));
            }
            nan_heads = 0u;
          }
        }
        if (k == 0 && last >= 0 && !gave_up) {
          gave_up = !epilogue(unit_s[last % kMkUnits], last);
          release_unit(last);
        }
      }
      if (gave_up || un == 0) break;
      last = t;
    }
    // units whose rows see no token: zero rows, a request per block
#pragma unroll 1
    for (int r = blockIdx.x; r < p.N && !gave_up; r += gridDim.x) {
      const int L = mk_len(p, r);
#pragma unroll 1
      for (int t = 0; t < p.T; ++t) {
        if (mk_span<S::kTileRows>(p, L, t).X > 0) break;           // (later rows see no less)
#pragma unroll 1
        for (int m = t * S::kTileRows + q4; m < min(p.M, (t + 1) * S::kTileRows); m += 4)
#pragma unroll 1
          for (int h = 0; h < p.H; ++h)
            *reinterpret_cast<uint2 *>(out_row(r, h, m) + 4 * lane) = make_uint2(0u, 0u);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
    // Pages are looked up for 32 boxes at a time, a lane each: `per` chunks.
    const int log2_box = 31 - __clz(p.box), boxes = S::kTok >> log2_box, per = 32 >> (S::kTokLog2 - log2_box);
    auto box_pos = [&](const MkUnit &u, int kb, int *pos) -> bool {
      const int x = (u.c0 + kb) * S::kTok + lane * p.box;
      *pos = x < u.s16 ? x : x + u.shift;
      return x < u.X && (lane >> (S::kTokLog2 - log2_box)) < u.n - kb;
    };
    auto read_page = [&](const MkUnit &u, int kb) -> int {
      int pos;
      if (!box_pos(u, kb, &pos)) return -1;
      return __ldg(p.tables + static_cast<int64_t>(u.r) * p.width + (pos >> p.log2_bs));
    };
    // a box's first slot, -1 if it has none (bad: a page outside the cache)
    auto to_slot = [&](const MkUnit &u, int kb, int page, bool &bad) -> int {
      int pos;
      if (!box_pos(u, kb, &pos)) return -1;
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_blocks)) {
        bad = true;
        return -1;
      }
      return static_cast<int>((static_cast<uint32_t>(page) << p.log2_bs) | (pos & ((1 << p.log2_bs) - 1)));
    };
    if (warp == kMkWarpLoad) {
      // --------------------------------------------- units, copies of codes
      int x = static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * B, static_cast<int64_t>(total)));
      const int x_end = static_cast<int>(min(static_cast<int64_t>(x) + B, static_cast<int64_t>(total)));
      // the unit that position x is in or in front of: request, head, tile, where it starts
      int lo = 0, h = 0, t = 0, at = 0, L = 0;
      if (x < x_end) {
        int hi = p.N - 1;                              // the last request with pre[r] <= x
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (pre[mid] <= x) lo = mid;
          else hi = mid - 1;
        }
        L = mk_len(p, lo);
        const unsigned W = static_cast<unsigned>(pre[lo + 1] - pre[lo]) / static_cast<unsigned>(p.HG);
        h = static_cast<int>(static_cast<unsigned>(x - pre[lo]) / W);
        at = pre[lo] + h * static_cast<int>(W);
      }
      int4 cut = make_int4(-1, 0, 0, 0);               // (lane 0's)
      // the next piece of the block's range with chunks, into the announcements' entry u;
      // returns its chunks (0: none left)
      auto next_unit = [&](MkUnit &u) -> int {
        int n = 0;
#pragma unroll 1
        while (x < x_end) {
          const MkSpan s = mk_span<S::kTileRows>(p, L, t);
          const int V = mk_positions<S>(s.X), ut = t, uh = h, ur = lo, ua = at, uL = L;
          if (x >= at + V || at + V <= x_end) {        // (nothing of it is left after this)
            at += V;
            if (++t == p.T) {
              t = 0;
              if (++h == p.HG) {
                h = 0;
                do ++lo;
                while (lo < p.N && pre[lo + 1] <= at);
                if (lo < p.N) L = mk_len(p, lo);
              }
            }
          }
          if (x >= ua + V) continue;
          const int first = ua + S::kCharge, end = min(ua + V, x_end), from = max(x, first);
          x = end;
          if (from >= end) continue;
          n = end - from;
          if (lane == 0) {
            u.r = ur;
            u.h = uh * S::kHeads;
            u.row0 = ut * S::kTileRows;
            u.c0 = from - first;
            u.X = s.X;
            u.s16 = s.s16;
            u.shift = s.shift;
            u.base = uL - p.R;
            u.direct = n == V - S::kCharge;
            const int b_first = static_cast<int>(static_cast<unsigned>(first) / static_cast<unsigned>(B));
            const bool starts = static_cast<int>(blockIdx.x) == b_first;
            u.slot = 2 * static_cast<int>(blockIdx.x) + (starts ? 1 : 0);
            if (starts && n != V - S::kCharge)
              cut = make_int4(ur, uh * S::kHeads, ut * S::kTileRows,
                              static_cast<int>(static_cast<unsigned>(ua + V - 1) / static_cast<unsigned>(B)));
          }
          break;
        }
        if (lane == 0) u.n = n;
        __syncwarp();
        return n;
      };
      // (pages that only one unit reads need not stay: tree batch 200 -> 194 us)
      const uint64_t pol = p.T == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
      // A batch: the pages of 32 boxes, one a lane, read while the batch before is copied.
      int t_cur = 0, un = next_unit(unit_s[0]);
      if (lane == 0) mbar_arrive(BAR(S::kUnitFull));
      int kb = -1, j = 0, id = un != 0 ? read_page(unit_s[0], 0) : -1;
      int next_un = un, next_kb = 0, next_t = 0;       // of the batch that `id` belongs to
      int slot = -1, uh = 0;
      uint32_t have = 0u, n = 0u;
      bool ok = true, bad = false;
#pragma unroll 1
      for (;;) {
        if (kb < 0 || j == per || kb + j == un) {
          // the next batch
          un = next_un;
          kb = next_kb;
          t_cur = next_t;
          j = 0;
          if (un == 0) break;
          const MkUnit &u = unit_s[t_cur % kMkUnits];
          slot = to_slot(u, kb, id, bad);
          uh = u.h;
          have = __ballot_sync(0xFFFFFFFFu, slot >= 0);
          next_kb = kb + per;
          if (next_kb >= un) {
            // the next unit, announced
            next_kb = 0;
            ++next_t;
            const int e = next_t % kMkUnits;
            if (next_t >= kMkUnits)
              ok = mk_wait_all(BAR(S::kUnitEmpty + e), (next_t / kMkUnits - 1) & 1, abort_s);
            if (!ok) break;
            next_un = next_unit(unit_s[e]);
            if (lane == 0) mbar_arrive(BAR(S::kUnitFull + e));
          }
          id = next_un != 0 ? read_page(unit_s[next_t % kMkUnits], next_kb) : -1;
        }
        const uint32_t b = n % S::kStages;
        constexpr int kBoxes = 8 / S::kHeads;          // at most
        int z[kBoxes];                                 // in groups of 8 slots
#pragma unroll
        for (int i = 0; i < kBoxes; ++i) z[i] = __shfl_sync(0xFFFFFFFFu, slot >> 3, j * boxes + i);
        const uint32_t now = (have >> (j * boxes)) & ((1u << boxes) - 1u);
        if (n >= S::kStages)
          ok = mk_wait_all(BAR(S::kKvEmpty + b), (n / S::kStages - 1) & 1, abort_s);
        if (!ok) break;
        if (mk_elect()) {
          const uint32_t dst = smem_addr(smem + S::kOffKv) + b * S::kStage;
          const uint32_t full = BAR(S::kKvFull + b), step = p.box * S::kHeads / 8 * S::kGroup;
          const bool tail = S::kHeads > 1 && uh >= p.tail;
          const int head = tail ? 0 : uh, heads = tail ? p.H - p.tail : S::kHeads;
          mbar_arrive_expect_tx(full, __popc(now) * 2 * p.box * heads * kHeadDim);
#pragma unroll 1
          for (int plane = 0; plane < 2; ++plane) {
            const CUtensorMap *map = plane == 0 ? (tail ? &maps.k_tail : &maps.k)
                                                : (tail ? &maps.v_tail : &maps.v);
#pragma unroll
            for (int i = 0; i < kBoxes; ++i)
              if ((now >> i) & 1u)
                mk_load_box(dst + plane * S::kVOff + i * step, map, z[i], head, full, pol);
          }
        }
        __syncwarp();
        ++j;
        ++n;
      }
      gave_up = !ok;
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (lane == 0) {
        p.cuts[blockIdx.x] = cut;
        if (bad && p.err_flags) atomicOr(p.err_flags, KVQ_ERRF_BLOCK_RANGE);
        // copies in flight land before the block leaves
        for (uint32_t v = n > S::kStages ? n - S::kStages : 0; v < n; ++v)
          mbar_wait_sleep_bounded(BAR(S::kKvFull + v % S::kStages), (v / S::kStages) & 1);
      }
    } else if (warp == kMkWarpScale) {
      // -------------------------------------------------------------- scales
      // Copied two chunks ahead; value scales brought over 2^Eg, the chunk's largest scales
      // found.  Lane l has the tokens 4 l .. 4 l + 3.
      constexpr int kAhead = 2;
      const int box_of = 4 * lane / (p.box * S::kHeads), tok_of = 4 * lane & (p.box - 1);
      const int head_of = (4 * lane >> log2_box) & (S::kHeads - 1);
      bool ok = wait_unit(0), bad_page = false;
      int un = ok ? unit_s[0].n : 0;
      int t_cur = 0, kb = -1, j = 0, next_un = un, next_kb = 0, next_t = 0;
      int id = un != 0 ? read_page(unit_s[0], 0) : -1;
      int slot = -1, eg = 0;
      const float *kp = p.k_scales, *vp = p.v_scales;
      int left = 0;                                    // tokens of the unit from the lane's first on
      uint32_t n = 0u, done = 0u, hist = 0u;           // hist: a bit a chunk: a unit's first
      bool more = ok;
#pragma unroll 1
      for (;;) {
        if (more && (kb < 0 || j == per || kb + j == un)) {
          // the next batch
          if (kb >= 0 && next_t != t_cur) release_unit(t_cur);
          un = next_un;
          kb = next_kb;
          t_cur = next_t;
          j = 0;
          more = un != 0;
          if (more) {
            const MkUnit &u = unit_s[t_cur % kMkUnits];
            slot = to_slot(u, kb, id, bad_page);
            kp = p.k_scales + u.h + head_of;
            vp = p.v_scales + u.h + head_of;
            // (keys 4 lane ..: box, head, tokens from `tok` of the box on)
            left = head_of < p.H - u.h ? u.X - (u.c0 + kb) * S::kTok - box_of * p.box - tok_of : INT_MIN;
            next_kb = kb + per;
            if (next_kb >= un) {
              next_kb = 0;
              ++next_t;
              ok = wait_unit(next_t);
              if (!ok) break;
              next_un = unit_s[next_t % kMkUnits].n;
            }
            id = next_un != 0 ? read_page(unit_s[next_t % kMkUnits], next_kb) : -1;
          }
        }
        if (more) {
          const uint32_t b = n % S::kScales;
          if (n >= S::kScales)
            ok = mk_wait_all(BAR(kPair ? S::kScEmpty + b : S::kKvEmpty + b), (n / S::kScales - 1) & 1, abort_s);
          if (!ok) break;
          const int first = __shfl_sync(0xFFFFFFFFu, slot, j * boxes + box_of);
          const int len = first < 0 ? 0 : left;
          const int64_t at = len > 0 ? (static_cast<int64_t>(first) + tok_of) * p.H : 0;
          float *ks = reinterpret_cast<float *>(smem + S::kOffSc) + b * 3 * kMkTok + 4 * lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t size = i < len ? 4u : 0u;
            const int of = i < len ? i * p.H : 0;
            cp_async_4(ks + i, kp + at + of, size);
            cp_async_4(ks + kMkTok + i, vp + at + of, size);
          }
          hist = (hist << 1) | (kb + j == 0 ? 1u : 0u);
          if (left > INT_MIN / 2) left -= S::kTok;
          ++j;
          ++n;
        }
        cp_async_commit();
        if (!more && done == n) break;
        if (more && n - done <= kAhead) continue;
        // chunk `done`, copied kAhead chunks ago
        if (more) cp_async_wait<kAhead>();
        else cp_async_wait<0>();
        __syncwarp();
        const uint32_t b = done % S::kScales;
        float4 *ks = reinterpret_cast<float4 *>(smem + S::kOffSc + b * 3 * kMkTok * 4) + lane;
        const float4 kk = ks[0];
        const float4 v4 = ks[kMkTok / 4];
        float vv[4] = {v4.x, v4.y, v4.z, v4.w}, lg[4];
        const bool first_chunk = ((hist >> (n - 1 - done)) & 1u) != 0u;
        // Scales that are not finite reach nobody by a product (an infinite one would put the
        // references so high that every weight, and with them the denominator, is 0); rows that
        // see them become NaN.
        float flagged = 0.0f;
        uint32_t bad = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(vv[i] - vv[i] == 0.0f)) {
            vv[i] = 0.0f;
            bad |= 1u << i;
          }
        if (__any_sync(0xFFFFFFFFu, bad != 0u)) {
          flagged = 1.0f;
          if (lane < 4) bad_s[4 * (S::kVfs + b) + lane] = 0u;
          __syncwarp();
          if (bad != 0u) atomicOr(bad_s + 4 * (S::kVfs + b) + (lane >> 3), bad << (4 * (lane & 7)));
        }
        // (fmaxf leaves NaN out)
        const float km4 = fmaxf(fmaxf(kk.x, kk.y), fmaxf(kk.z, kk.w));
        const float vm4 = fmaxf(fmaxf(vv[0], vv[1]), fmaxf(vv[2], vv[3]));
        const uint32_t km = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fmaxf(km4, 0.0f)));
        const uint32_t vm = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fmaxf(vm4, 0.0f)));
        const int ev = min(mk_ceil_log2(__uint_as_float(vm)), 126);
        if (first_chunk) eg = min(ev, kMkMaxEg);
        else if (ev > eg) eg = min(ev + 2, kMkMaxEg);
        const float down = mk_pow2(-eg);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vv[i] *= down;
          lg[i] = fmaxf(static_cast<float>(mk_ceil_log2(vv[i])), kMkFloor);
        }
        ks[kMkTok / 4] = make_float4(vv[0], vv[1], vv[2], vv[3]);
        ks[kMkTok / 2] = make_float4(lg[0], lg[1], lg[2], lg[3]);
        if (lane == 0)
          reinterpret_cast<float4 *>(smem + S::kOffMeta)[b] =
              make_float4(__uint_as_float(km), fmaxf(static_cast<float>(ev - eg), kMkFloor),
                          __int_as_float(eg), flagged);
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(kPair ? S::kScFull + b : S::kKvFull + b));
        ++done;
      }
      cp_async_wait<0>();
      gave_up = !ok;
    } else {
      // ---------------------------------------------------- MMAs of a chain
      // Each step: PV of one of the chain's chunks and QK^T of its next.  kPair: chain 0's
      // and chain 1's steps one after the other, all but the second half of P'' waited for
      // before the turn (without turns the chunks of prompts took 638 us, with them 586).
      // Chains that share a tile have half the softmax work and take no turns (window of 64
      // requests: 107 us with turns, 100 without).
      const int a = warp - kMkWarpMma;
      const uint32_t q1 = (smem_addr(smem + S::kOffQ + (kPair ? a : 0) * 2 * S::kQPiece) >> 4) | kMkKMajor;
      const uint32_t q2 = q1 + (S::kQPiece >> 4);
      const uint32_t k0 = (smem_addr(smem + S::kOffKv) >> 4) | kMkKMajor;
      const uint32_t k_hi = (static_cast<uint32_t>(S::kGroup) >> 4) | (1u << 14) | (kSmemSwizzle128 << 29);
      // (values: blocks of 64 dims, groups of 8 keys, by bytes)
      constexpr uint32_t v_group = S::kGroup;
      constexpr uint32_t v_block = S::kVfBytes / 2;
      const uint32_t v_hi = (v_group >> 4) | (1u << 14) | (kSmemSwizzle128 << 29), v_step = 2 * v_group >> 4;
      const uint32_t v0 = (smem_addr(smem + S::kOffVf) >> 4) | (v_block >> 4) << 16;
      const uint32_t s_col = tmem + mk_s(a), o_col = tmem + mk_o(a);
      uint32_t base = 0;                               // chunks of earlier units
      uint32_t par_q = 0, par_p = 0, par_o = 1, par_turn = a ^ 1;
      bool ok = true;
      for (int t = 0; ok; ++t) {
        ok = wait_unit(t);
        if (!ok) break;
        const MkUnit &u = unit_s[t % kMkUnits];
        const int un = u.n;
        if (un == 0) break;
        const int steps = kPair ? un : (un + 1) / 2;
        const bool turns = kPair && chain_chunks(u, 1) > 0;    // (a lone chain 0 need not take them)
        const bool live = chain_chunks(u, a) > 0;      // (the chain has products)
        release_unit(t);
        for (int j = 0; j <= steps; ++j) {
          const int cv = kPair ? j - 1 : 2 * (j - 1) + a, cq = kPair ? j : 2 * j + a;
          const bool use_v = j > 0 && cv < un, use_k = cq < un;
          const bool pv = use_v && live, qk = use_k && live;
          const uint32_t sv = base + cv, sq = base + cq;
          const uint32_t bk = sq % S::kStages, bv = sv % S::kVfs;
          if (kPair && use_v) ok = mk_wait_all(BAR(S::kVfFull + bv), (sv / S::kVfs) & 1, abort_s);
          if (kPair && ok && use_k) ok = mk_wait_all(BAR(S::kKvFull + bk), (sq / S::kStages) & 1, abort_s);
          if (ok && j == 0 && (qk || !kPair))
            ok = mk_wait_all(BAR(S::kQFull + (kPair ? a : 0)), kPair ? par_q : t & 1, abort_s);
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
                mk_mma_pv(o_col, s_col + 8 * kk, v_lo + v_step * kk, v_hi, (j == 1 && kk == 0) ? 0u : 1u);
            }
            if (kPair) ok = mk_wait_all(BAR(S::kPReady + 2 * a + 1), par_p, abort_s);
            if (!ok) break;
            par_p ^= 1u;
            tc_fence_after();
            if (mk_elect()) {
#pragma unroll
              for (int kk = 4; kk < 8; ++kk)
                mk_mma_pv(o_col, s_col + 32 + 8 * kk, v_lo + v_step * kk, v_hi, 1u);
              if (!kPair) tc_commit(BAR(S::kKvEmpty + bv));
            }
          }
          if (!kPair && use_k) {
            ok = mk_wait_all(BAR(S::kKvFull + bk), (sq / S::kStages) & 1, abort_s);
            if (!ok) break;
          }
          if (qk) {
            const uint32_t k_lo = k0 + bk * (S::kStage >> 4);
            tc_fence_after();
            if (mk_elect()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mk_mma_qk(s_col, q1 + 2 * kk, k_lo + 2 * kk, k_hi, kk != 0);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mk_mma_qk(s_col, q2 + 2 * kk, k_lo + 2 * kk, k_hi, 1u);
              tc_commit(BAR(S::kSFull + a));
            }
          }
          __syncwarp();
          if (mk_elect()) {
            if (turns) mbar_arrive(BAR(S::kTurn + (a ^ 1)));
            if (pv && (kPair ? cv == un - 1 : cv + 2 >= un)) tc_commit(BAR(S::kOFull + a));
            if (qk && (kPair ? cq == un - 1 : cq + 2 >= un)) tc_commit(BAR(S::kQEmpty + a));
            if (!kPair && !live && j == 0) mbar_arrive(BAR(S::kQEmpty + a));   // (each unit's queries)
            if (kPair && use_v) tc_commit(BAR(S::kVfEmpty + bv));
            if (kPair && use_k) tc_commit(BAR(S::kKvEmpty + bk));
          }
          __syncwarp();
        }
        if (live) par_q ^= 1u;
        base += un;
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

// The pieces of the units that are cut, joined: `parts` blocks for each block of the first
// launch that was the first of several to work on a unit, a warp per row at a time, four
// dims a lane.
constexpr int kMkJoinParts = 32, kMkJoinWarps = 4;     // (parts at most)

__global__ void __launch_bounds__(32 * kMkJoinWarps)
attn_masked_join_kernel(const MkParams p, int parts, int lanes, int heads) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b_first = static_cast<int>(blockIdx.x) / parts, part = static_cast<int>(blockIdx.x) % parts;
  allow_dependents_launch();
  grid_dependency_wait();
  const int4 cut = __ldcg(p.cuts + b_first);           // request, first head, first row, last block
  if (cut.x < 0) return;
  const int pieces = cut.w - b_first + 1, step = parts * kMkJoinWarps;
  const int head_lanes = lanes / heads, rows = min(head_lanes, p.M - cut.z);
  auto place = [&](int b, int r) -> int64_t {
    return static_cast<int64_t>(2 * (b_first + b) + (b == 0 ? 1 : 0)) * lanes + r;
  };
  for (int n = part * kMkJoinWarps + warp; n < rows * min(heads, p.H - cut.y); n += step) {
    const int of = n / rows, head = cut.y + of, m = cut.z + n - of * rows;
    const int r = of * head_lanes + n - of * rows;
    float top = -INFINITY, all = 0.0f;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int b0 = 0; b0 < pieces; b0 += 8) {
      float2 ml[8];
      float4 o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t at = place(b0 + i, r);
        const bool get = b0 + i < pieces;
        ml[i] = get ? __ldcg(p.ml_part + at) : make_float2(-INFINITY, 0.0f);
        o[i] = get ? __ldcg(reinterpret_cast<const float4 *>(p.o_part + at * kHeadDim) + lane)
                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      float next = top;
#pragma unroll
      for (int i = 0; i < 8; ++i) next = fmaxf(next, ml[i].x);
      const float f = top == -INFINITY ? 0.0f : mk_ex2(top - next);
      all *= top == -INFINITY ? 1.0f : f;              // (NaN stays)
      y.x *= f;
      y.y *= f;
      y.z *= f;
      y.w *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // (a part that saw nothing has no reference and a sum of 0, or NaN)
        const float w = ml[i].x == -INFINITY ? ml[i].y : mk_ex2(ml[i].x - next) * ml[i].y;
        all += w;
        y.x = fmaf(o[i].x, w, y.x);
        y.y = fmaf(o[i].y, w, y.y);
        y.z = fmaf(o[i].z, w, y.z);
        y.w = fmaf(o[i].w, w, y.w);
      }
      top = next;
    }
    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
    const int i = mk_query(p, m);
    uint16_t *dst = p.out + ((static_cast<int64_t>(cut.x) * p.R + i) * p.Hq + head * p.G + (m - i * p.G)) * kHeadDim;
    *reinterpret_cast<uint2 *>(dst + 4 * lane) =
        make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
  }
}

// Rows of a unit and head, and its heads.
int mk_tile_rows(int M) { return M <= 32 ? 32 : (M <= 64 ? 64 : (M <= 128 ? 128 : 256)); }
int mk_charge(int rows) { return rows > 128 ? MkShape<true, 128>::kCharge : MkShape<false, 32>::kCharge; }
int mk_heads(int rows) { return rows >= 128 ? 1 : 128 / rows; }

template <bool kPair, int kRows>
cudaError_t mk_launch(const MkParams &p, const MkMaps &maps, int grid, cudaStream_t stream) {
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
  e = launch_overlapped(kernel, dim3(static_cast<unsigned>(grid)), dim3(kMkThreads), kSmem, stream, p,
                        maps);
  if (e != cudaSuccess) return e;
  using S = MkShape<kPair, kRows>;
  const int rows = S::kHeads * std::min(p.M, S::kTileRows);
  const int parts = std::min((rows + kMkJoinWarps - 1) / kMkJoinWarps, kMkJoinParts);
  return launch_overlapped(attn_masked_join_kernel, dim3(static_cast<unsigned>(grid * parts)),
                           dim3(32 * kMkJoinWarps), 0, stream, p, parts, S::kLanes, S::kHeads);
}

size_t mk_round(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Positions in the work sequence of a launch, at most; 2^31 are too many to number.
bool attn_masked_too_long(const MaskedArgs &a, int32_t num_kv_heads) {
  const int M = a.rows_per_request * (a.num_q_heads / num_kv_heads);
  const int rows = mk_tile_rows(M), heads = mk_heads(rows), tokens = kMkTok / heads;
  const double units = static_cast<double>(std::min(a.num_requests, kMkMaxRequests)) *
                       ((num_kv_heads + heads - 1) / heads) * ((M + rows - 1) / rows);
  return units * (a.max_context_len / tokens + 1 + mk_charge(rows)) >= 2147483648.0;
}

size_t attn_masked_workspace_bytes(const MaskedArgs &a, int32_t num_kv_heads) {
  const int64_t M = static_cast<int64_t>(a.rows_per_request) * (a.num_q_heads / num_kv_heads);
  const int rows = mk_tile_rows(static_cast<int>(M));
  const size_t slots = static_cast<size_t>(a.sms) * 2 * std::max(rows, 128);
  return mk_round(a.sms * sizeof(int4)) + mk_round(slots * kHeadDim * sizeof(float)) +
         mk_round(slots * sizeof(float2));
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
  p.inv_g = static_cast<uint32_t>(((uint64_t(1) << 32) + p.G - 1) / p.G);
  const int rows = mk_tile_rows(p.M);
  const int heads = mk_heads(rows), tokens = kMkTok / heads;
  p.T = (p.M + rows - 1) / rows;
  p.HG = (H + heads - 1) / heads;
  p.width = a.max_blocks_per_req;
  p.num_blocks = static_cast<int32_t>(c.num_slots >> a.log2_block);
  p.log2_bs = a.log2_block;
  // tokens of a box: a window and its sinks start on any 16 of a page, and of several heads
  // a chunk has no more
  p.box = a.tree_mask != nullptr && heads == 1 ? std::min(1 << a.log2_block, kMkTok) : 16;
  // (beyond the longest context neither bound means anything)
  p.window = std::min(a.window, a.max_context_len + p.R);
  p.sinks = std::min(a.num_sinks, a.max_context_len);
  p.words = (p.R + 31) / 32;
  p.scale2 = (a.sm_scale < 0.0f ? -a.sm_scale : a.sm_scale) * 1.4426950408889634f;
  p.flip = a.sm_scale < 0.0f ? 0x80808080u : 0u;
  // Ranges of at least 128 tokens (and a chunk): shorter ones are joined from more pieces
  // than they save (one row, 1,028 tokens: 21 us with ranges of three chunks of 32 tokens, 19
  // with five or six, 21 with seven).
  p.least = kMkTok / tokens + 1;
  p.k_scales = c.k_scales;
  p.v_scales = c.v_scales;
  p.err_flags = a.err_flags;
  // A map per plane for the whole groups of heads, and one for a last group of fewer: the
  // keys of its other places are not loaded (their scores reach no row, their values are
  // cleared).
  const int64_t slots = static_cast<int64_t>(p.num_blocks) << a.log2_block;
  const int last = H % heads;
  p.tail = H - last;
  MkMaps maps{};
  if ((p.tail > 0 &&
       (!encode_plane_tensor_map(&maps.k, c.k_codes, slots, H, 0, p.tail, p.box, heads) ||
        !encode_plane_tensor_map(&maps.v, c.v_codes, slots, H, 0, p.tail, p.box, heads))) ||
      (last > 0 &&
       (!encode_plane_tensor_map(&maps.k_tail, c.k_codes, slots, H, p.tail, last, p.box, last) ||
        !encode_plane_tensor_map(&maps.v_tail, c.v_codes, slots, H, p.tail, last, p.box, last))))
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
    const size_t slots_ws = static_cast<size_t>(grid) * 2 * std::max(rows, 128);
    p.cuts = reinterpret_cast<int4 *>(ws);
    ws += mk_round(grid * sizeof(int4));
    p.o_part = reinterpret_cast<float *>(ws);
    ws += mk_round(slots_ws * kHeadDim * sizeof(float));
    p.ml_part = reinterpret_cast<float2 *>(ws);
    const cudaError_t e = rows == 32    ? mk_launch<false, 32>(p, maps, grid, stream)
                          : rows == 64  ? mk_launch<false, 64>(p, maps, grid, stream)
                          : rows == 128 ? mk_launch<false, 128>(p, maps, grid, stream)
                                        : mk_launch<true, 128>(p, maps, grid, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kvq
