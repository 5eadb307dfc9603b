// tree_attn.cuh - the kernel behind gdn_tree_attention: attention of the drafted
// tokens of a tree over a request's paged cache and over each other, on tcgen05.
// tree_attn_bf16.cu and tree_attn_e4m3.cu compile it for the two cache formats.
//
// Math, per query row (node j, query head h), over the tokens t that it sees:
//   s_t = scale (q . k_t),  m = max s_t,  l = sum e^(s_t - m),  out = sum e^(s_t - m) v_t / l
// and with a gate out <- out / (1 + e^-gate).
//
// Work. The unit of work is a tile of 128 cached tokens for one (request, kv head,
// row tile): the query rows of the Hq / Hkv heads of all P nodes, up to kRows of
// them. The tiles of all requests stand in one line, cut into equal pieces, one
// per CTA (one CTA per SM): every SM streams the same number of keys and values,
// whatever the lengths, and a single long request uses the whole GPU. What a CTA
// does once per unit (request, kv head, row tile) counts as kSegCost tiles: with
// the tiles alone, CTAs with eight short units were 90 us behind the others. The
// lengths are read on the device, so a captured graph takes new ones. A unit that
// lies in several CTAs' pieces leaves a partial result per CTA in the workspace,
// and a second kernel adds them up in the order of the tiles. (With the CTA that
// arrived last doing it, two tickets and a chain of trips to L2 took up to 45 us
// for 64 rows.)
//
// Both products take the cache as their first operand, so a tile costs the tensor
// cores the same 128 lanes for few query rows as for many columns:
//   S^T [128 tokens x rows] = K Q^T    (K from shared memory as it lies in the cache)
//   O^T [128 of D x rows]   = V^T P^T  (V the same, read along its other dimension)
// A bf16 cache runs them in bf16. An E4M3 cache stays E4M3 in shared memory, and
// the other operand is written as the sum of two E4M3 terms, the value and what
// its rounding left: 4 + 4 significant bits, as many as bf16 has. For Q (bf16
// values, scaled by a power of two per row) that is exact down to 2^-17 of the
// row's largest value; a weight of P, which is one of the softmax times its value's
// scale, is off by 2^-8 + 2^-11 of itself or 2^-17 of the row's largest in the tile.
// The two terms are columns of one MMA, added up as they are read, or from 33 rows
// on two MMAs into the same columns. The key's scale multiplies the score.
// (A bf16 cache's weights go to bf16, 2^-8 of each; their sum is that of the fp32
// weights either way.)
//
// Softmax without a chain between tiles: a tile's weights are taken relative to
// its own maximum, and the accumulators of the output, in registers, take the
// tile's product times e^(tile's maximum - running maximum). So the next tile's
// scores never wait for the last one's.
//
// With an E4M3 cache the maximum is that of s_t log2(e) + e_t, 2^e_t the power of two
// of the value's scale v_t: what E4M3 holds best are a row's largest weights with
// their scales, not those of a token that it does not see or hardly weighs. (With
// the weights alone relative to their maximum and the scales to the tile's largest,
// a sibling node's scale of 2^14 times the others' put its neighbours' rows off by 14 %.)
// The fp32 weight 2^(s_t log2(e) + e_t - maximum) goes to P times v_t / 2^e_t, to the
// sum times 1 / 2^e_t. It costs a multiply-add for two scores and saves the scales'
// maximum: 64 rows on 131071 tokens 303 us, 308 with the two maxima apart; with a test
// of each tile's scales and a second pass where they are far apart, 323 .. 337.
//
// Roles: two groups of four warps for the softmax (a thread has four tokens and a
// quarter of the rows), which take turns at the tiles, or, from 33 rows on, half
// of a tile's rows each; one
// group of four warps for the output (a thread per value of D, mod 128), from 17
// rows on two with half of D each, or half of the rows at D = 128; a warp for the
// copies (TMA, 16 KB blocks of 128 tokens x 128 bytes into a ring), one for the
// MMAs, one for the query rows, one that checks pages and clears values behind the
// last token. Every wait is bounded: one that runs out sets
// GDN_DEVERR_TIMEOUT and the CTA leaves.
//
// What bounds it, with 24 query and 4 kv heads of 256:
//   one token per request: HBM. 256 requests of 1k..8k tokens, E4M3: 284 us, 6.5
//   TB/s. One request of 509 tokens: 11 us, the launches and one tile's chain.
//   Heads of 128, 32 over 8: 128 requests of 129..8192 tokens, E4M3: 134 us, 3.9
//   TB/s, a unit's fixed work, about six of its small tiles' time, 1024 units.
//   48 rows (trees of 8 nodes), bf16, 32 requests of 129..16384 tokens: 103 us,
//   4.4 TB/s. The copies wait for room: a tile is 128 KB, the ring 128 KB (96 KB for
//   64 rows: 109 us), and V stays in it until its weights are there; a unit costs
//   about five tiles' time. E4M3: 107 us, 2.2 TB/s, a unit about nine tiles' time.
//   64 rows, 131071 tokens, E4M3: 300 us, the softmax: 8 warps at 0.62 instructions
//   a cycle and scheduler in chains of exchanges, conversions and barriers, 3.6 k
//   cycles a tile, of which the MMAs need 1.1 k. bf16: 421 us, the ring as above, the
//   six row tiles each reading the cache.
#pragma once

#include "device.cuh"
#include "launch.h"
#include "umma.cuh"

namespace gdn {
namespace tree_attn {

constexpr int kTile = 128;               // tokens per tile
constexpr uint32_t kBlock = 128 * 128;   // bytes of one ring block: 128 tokens x 128 bytes
constexpr int kMaxCtas = 152;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kDescBytes = 4096;          // of the workspace: a Desc per CTA
constexpr int kScSlots = 4;              // tiles of scales in flight
// A barrier's parity tells a phase from the next one only. So there are more of them than their writer can be
// ahead of their reader: the ring (at most 11 blocks) holds K or V of fewer than 8 tiles.
constexpr int kSlots = 8, kMarks = 16;
constexpr int kBarBytes = 1216;
constexpr float kLog2e = 1.4426950408889634f;
// E4M3: the largest of a row's fp32 weights in a tile is 2^kTopExp, so that one of 2^-190 of it, a value scale of the
// smallest next to the largest, counts in the sum, and 128 of the most by 2 / 2^kMinScaleExp are no more than a number.
// As E4M3 terms, before v_t / 2^e_t in [1, 2), that weight is kTermTop: 448 is the largest.
constexpr int kTopExp = 64;
constexpr float kTermTop = 224.f;
// Exponents of the value scales: none below this. A write leaves -49 at least; a smaller scale, or none, counts as 2^-50
// here, and beside a weight with such a value a row's others are held to 2^-17 of 2^-50 times that weight.
constexpr int kMinScaleExp = -50;

struct Args {
  TreeAttnArgs p;
  KvArgs c;
  int rows;       // query rows per row tile (the last one may have fewer)
  int row_tiles;
  int box;        // tokens per TMA box: a power of two that divides the page, at most 128
  int slot_floats;  // workspace floats per partial
};

// A unit (request x head x row tile) that lies in several CTAs' pieces, noted by the CTA that has its first tile.
struct Desc {
  int valid, n, u, last;  // `last`: the CTA that has its last tile
};

// A partial result: the rows' maxima and sums, two words that are 0 once an output group has written its part
// and no page was out of the pool, then [rows][D] fp32. A CTA has two: of the unit that ends in its piece (or
// runs through it) and of the one that begins there.
__host__ __device__ __forceinline__ int head_floats(int rows) { return (2 * rows + 2 + 3) / 4 * 4; }
__device__ __forceinline__ float* partial(const Args& a, int cta, bool begins) {
  return reinterpret_cast<float*>(static_cast<unsigned char*>(a.p.workspace) + kDescBytes) +
         (size_t)(2 * cta + (begins ? 1 : 0)) * a.slot_floats;
}

template <int D, bool kE4m3, int kRows>
struct Cfg {
  static constexpr int kBlk = D * (kE4m3 ? 1 : 2) / 128;  // ring blocks of a tile's K, and of its V
  static constexpr int kHalves = D / 128;
  static constexpr int kTerms = kE4m3 ? 2 : 1;
  // The two terms of P are neighbouring columns of one product, those of Q rp columns apart, added as the result is
  // read; with 64 rows two products add them up in tensor memory instead (the MMAs have the time, the threads half the
  // columns to read).
  static constexpr bool kSumTerms = kE4m3 && kRows == 64;
  static constexpr int kOTerms = kSumTerms ? 1 : kTerms;
  static constexpr int kCols = kOTerms * kRows;               // of the scores
  static constexpr int kOCols = kOTerms * kRows;              // of the output
  static constexpr int kOBuf = 2;                             // outputs, as many as tiles of weights: see o_empty
  static constexpr bool kSplit = kRows == 64;               // the softmax groups share each tile's rows
  // Tiles whose scores are ahead of the output: when a softmax group ends a tile, its next one's scores are there.
  static constexpr int kAhead = kSplit ? 1 : 2;
  // query buffers: a tile's scores wait for no output that follows them, though every segment have one tile
  static constexpr int kQBuf = kAhead + 1;
  // A unit's fixed work (its query rows, its result, the ends of its pipeline) in tiles, for the cut of the line. It takes
  // as long as so many. Measured with 0 / 2 / 4 / 5 / 7 / 9 / 12:
  //   32 trees of 48 rows on 129..16384 tokens, E4M3       185 / 144 / 129 / 116 / 104 / 108 / 110 us
  //   the same with 32 query and 8 kv heads of 128         200 / 149 / 125 / 122 / 106 /  99 /  92
  //   the same of 30 rows, heads of 256                    119 /  94 /  87 /  86 /  86 /  89 /  94
  //   32 trees of 48 rows on 129..16384 tokens, bf16       164 / 124 / 111 / 110 / 111 / 115 / 122
  //   the same of 30 rows                                  112 /  94 /  95 /  98 / 102 / 106 / 111
  //   128 single tokens on 129..8192, bf16                 171 / 161 / 164 / 166 / 169 / 172 / 180
  //   256 single tokens on 1k..8k, E4M3                    284 / 282 / 288 / 290 / 297 / 298 / 306
  //   128 on 129..8192, E4M3, 32 / 8 heads of 128          167 / 129 / 128 / 131 / 140 / 143 / 155 (6: 134)
  static constexpr int kSegCost = kRows > 16 ? (kE4m3 ? 9 : 5) : !kE4m3 ? 2 : D == 256 ? 4 : 6;
  // The launch may begin before the kernel in front of it ends: one request of 509 tokens 11.9 -> 10.9 us, and 14.1 -> 11.1
  // us call after call. Not for more rows: 64 on 131071 tokens in E4M3 306 -> 319 us, 64 x 24 rows 85 -> 88 us.
  static constexpr bool kEarly = kRows == 16;
  static constexpr int kOutGroups = kRows == 16 ? 1 : 2;    // at few rows a group's fixed work outweighs the rows'
  static constexpr int kOutWarp = 8, kCopyWarp = kOutWarp + 4 * kOutGroups;  // first warps of the roles
  static constexpr int kMmaWarp = kCopyWarp + 1, kQueryWarp = kCopyWarp + 2, kCheckWarp = kCopyWarp + 3;
  static constexpr int kThreads = 32 * (kCopyWarp + 4);
  static constexpr int kSoftRows = kSplit ? kRows / 2 : kRows;  // rows of a softmax thread
  static constexpr int kSoftWarps = kSplit ? 8 : 4;         // softmax warps at one tile
  static constexpr int kOutHalves = kHalves / kOutGroups > 0 ? kHalves / kOutGroups : 1;  // values of an output thread
  static constexpr int kOutRows = kHalves >= kOutGroups ? kRows : kRows / 2;               // and its rows
  // shared memory behind the ring, by byte offsets from its end
  static constexpr int oP = 0;
  static constexpr int oSc = oP + 2 * (int)kBlock;                          // [kScSlots][2][128] fp32
  static constexpr int oMax = oSc + (kE4m3 ? kScSlots * 2 * kTile * 4 : 0);  // [2][4 warps][kRows + 4]
  static constexpr int oSum = oMax + 2 * (kRows + 4) * 16;                  // [2][4 warps][kRows]
  static constexpr int oWarp = oSum + 2 * kRows * 16;                       // [8 warps][kSoftRows]
  static constexpr int oTile = oWarp + 8 * kSoftRows * 4;                   // [2][kRows]: maxima
  static constexpr int oAb = oTile + 2 * kRows * 4;                         // [2 groups][2][2][kRows]
  static constexpr int oMask = oAb + 8 * kRows * 4;                         // [kQBuf][kRows] uint64
  static constexpr int oQs = oMask + kQBuf * kRows * 8;                     // [kQBuf][kRows] fp32
  static constexpr int oFin = oQs + kQBuf * kRows * 4;                      // [2 groups][kRows] fp32
  static constexpr int kStageRows = kOutHalves == 2 ? 4 : 8;                // rows of a result on their way out at a time
  static constexpr int oStage = oFin + 2 * kRows * 4;                       // [kOutGroups][kStageRows][kOutHalves * 128] fp32
  static constexpr int oBars = oStage + kOutGroups * kStageRows * kOutHalves * 512;
  // Q's buffers at the end, for the rows that there are: what they leave is the ring's. 48 rows of a bf16 cache of 256
  // wide heads have eight blocks, two more than 64. (Not for summed terms: their loops are slower with sizes of the run,
  // 311 us against 306 for 64 rows on 131071 tokens, 100 against 95 for 32 x 48 rows.)
  static constexpr int oQ = (oBars + kBarBytes + 1023) / 1024 * 1024;
  static __host__ __device__ constexpr int row_pad(int rows) { return kE4m3 ? (rows + 7) / 8 * 8 : (rows + 15) / 16 * 16; }
  static __host__ __device__ constexpr int q_block(int rows) { return kTerms * (kSumTerms ? kRows : row_pad(rows)) * 128; }
  static __host__ __device__ constexpr int q_bytes(int rows) { return q_block(rows) * kBlk; }
  static __host__ __device__ constexpr int rest_bytes(int rows) { return oQ + kQBuf * q_bytes(rows); }  // behind the ring
  static __host__ __device__ constexpr int stages(int rows) {
    const int fit = (kSmemLimit - rest_bytes(rows)) / (int)kBlock, most = fit < 11 ? fit : 11;
    // an even number of blocks keeps the two bf16 blocks of a 128-wide half of V side by side
    return kE4m3 ? most : most / 2 * 2;
  }
  static_assert(stages(kRows) >= kBlk + 2, "a tile's whole V stays until its weights are there");
  static_assert(2 * kCols + kOBuf * kHalves * kOCols <= 512, "tensor memory");
  // Columns of the MMAs: an MMA of 128 lanes takes them by sixteens, up to 256.
  static __host__ __device__ constexpr int mma_cols(int rows) {
    return kSumTerms ? (row_pad(rows) + 15) / 16 * 16 : kTerms * row_pad(rows);
  }
  static constexpr bool cols_ok() {
    for (int rows = 1; rows <= kRows; ++rows)
      if (mma_cols(rows) % 16 != 0 || mma_cols(rows) < rows || mma_cols(rows) > kCols || kCols > 256) return false;
    return true;
  }
};

// One CTA's piece of the line. `t`: where it begins in the unit, whose first kSegCost places hold no tile.
struct Plan {
  long long total, lo;
  int count, n, u, t;
};

struct Bars {
  uint64_t empty[12];                     // by ring block
  uint64_t k_full[kSlots], v_full[kSlots];  // by tile
  uint64_t v_issued[kMarks];              // by last tile (one with drafted tokens) of the piece: V's copies run
  uint64_t v_clean[kMarks];               // and V is ready for the MMAs
  uint64_t checked[kMarks];               // by segment
  uint64_t q_full[3], q_empty[3], s_full[2], s_empty[2], p_full[2], o_full[2], o_empty[2];
  uint64_t st_full[2], sc_full[kScSlots], sc_empty[kScSlots], drain;
  uint32_t tmem;
  int abort;
  int bad[kMarks];                        // the segment has a page out of the pool
  unsigned long long dirty[kMarks];       // nodes whose values in the last tile are no numbers
  Plan plan;
  long long warp_total[20];
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier area");

// The piece's segments: runs of tiles of one (request n, unit u = head x row tiles + row tile).
struct Seg {
  int n, u, t0, t1, tiles, len, ctx;
  long long first;  // the unit's first place in the line
};

__device__ __forceinline__ int tiles_of(const Args& a, int ctx, bool* too_long = nullptr) {
  if (ctx < 0) return 0;
  const long long len = (long long)ctx + a.p.P;
  if ((len + a.c.page - 1) / a.c.page > a.p.max_pages || len > INT32_MAX - kTile) {
    if (too_long) *too_long = true;
    return 0;
  }
  return (int)((len + kTile - 1) / kTile);
}

template <int kSegCost>
struct Walk {
  int n, u, t, left, units, tiles, ctx;
  long long at;
  __device__ __forceinline__ Walk(const Args& a, const Plan& p)
      : n(p.n), u(p.u), t(p.t), left(p.count), units(a.c.Hkv * a.row_tiles), tiles(0), ctx(0), at(p.lo) {
    if (left > 0) load(a);
  }
  __device__ __forceinline__ void load(const Args& a) {
    ctx = __ldg(a.p.ctx + n);
    tiles = tiles_of(a, ctx);
  }
  __device__ __forceinline__ bool next(const Args& a, Seg& s) {
    while (left > 0) {
      while (tiles == 0) {  // the piece has places left, so a request with some follows
        ++n;
        load(a);
      }
      const int take = min(tiles + kSegCost - t, left);
      s = Seg{n, u, max(t - kSegCost, 0), t + take - kSegCost, tiles, ctx + a.p.P, ctx, at - t};
      left -= take;
      at += take;
      t = 0;
      if (++u == units) {
        u = 0;
        ++n;
        if (left > 0) load(a);
      }
      if (s.t1 > 0) return true;
    }
    return false;
  }
};

// Waits for a phase of the barrier, no longer than the time limit or until another role gave up. Whoever
// gives up sets the flag, and all later waits of the CTA end at once: the softmax and output warps run
// through their tiles without effect (a result is written only while the flag is clear), the copies and
// the MMAs stop.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* abort) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 0; it < kWaitMaxIters; ++it) {
    if (*(volatile int*)abort) return false;
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 31u && globaltimer_ns() - t0 > kWaitLimitNs) break;
  }
  *(volatile int*)abort = 1;
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort);
}
// The same for a converged warp.
__device__ __forceinline__ void wait_warp(uint64_t* bar, uint32_t parity, int* abort) {
  wait(bar, parity, abort);
  __syncwarp();
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The warp's largest value (NaN is passed over).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// A warp's 32 tokens (lanes of tensor memory) by eight columns: this thread has tokens lane / 4 + 8 i, i = 0..3, and
// columns 2 (lane % 4) and the next of each. `lanes16`: the address of the upper sixteen lanes. Without waiting.
__device__ __forceinline__ void ld_tile8(uint32_t taddr, uint32_t lanes16, uint32_t (&r)[4][2]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0][0]), "=r"(r[0][1]), "=r"(r[1][0]), "=r"(r[1][1])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[2][0]), "=r"(r[2][1]), "=r"(r[3][0]), "=r"(r[3][1])
               : "r"(lanes16)
               : "memory");
}

// The same distribution of 16-bit pairs back to shared memory: register i holds the pair of token lane / 4 + 8 i, and
// each lane names the 16-byte row of token `lane`.
__device__ __forceinline__ void st_tile8(uint32_t row, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(row), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

// Of 2 kC values a lane, kC pairs of columns, the reduction over the eight lanes with the same lane % 4, the values
// shared out on the way. Afterwards the lane has the result of pair `pair`, value `second` of it.
template <int kC, typename Op>
__device__ __forceinline__ float reduce_pairs(const float2 (&v)[kC], int lane, Op op) {
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
  float a;
  if constexpr (kC == 1) {
    a = op(b4 ? v[0].y : v[0].x, __shfl_xor_sync(0xffffffffu, b4 ? v[0].x : v[0].y, 16));
    a = op(a, __shfl_xor_sync(0xffffffffu, a, 8));
    a = op(a, __shfl_xor_sync(0xffffffffu, a, 4));
  } else {
    constexpr int kN = kC / 2;
    float2 h[kN];  // the upper or the lower pairs
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float2 stay = b4 ? v[kN + i] : v[i], give = b4 ? v[i] : v[kN + i];
      h[i].x = op(stay.x, __shfl_xor_sync(0xffffffffu, give.x, 16));
      h[i].y = op(stay.y, __shfl_xor_sync(0xffffffffu, give.y, 16));
    }
    float2 t = h[0];
    if constexpr (kN == 2) {
      const float2 stay = b3 ? h[1] : h[0], give = b3 ? h[0] : h[1];
      t.x = op(stay.x, __shfl_xor_sync(0xffffffffu, give.x, 8));
      t.y = op(stay.y, __shfl_xor_sync(0xffffffffu, give.y, 8));
      a = op(b2 ? t.y : t.x, __shfl_xor_sync(0xffffffffu, b2 ? t.x : t.y, 4));
    } else {
      a = op(b3 ? t.y : t.x, __shfl_xor_sync(0xffffffffu, b3 ? t.x : t.y, 8));
      a = op(a, __shfl_xor_sync(0xffffffffu, a, 4));
    }
  }
  return a;
}
// The column (of 8 kC) whose result reduce_pairs leaves in this lane.
template <int kC>
__device__ __forceinline__ int reduced_column(int lane) {
  const int b4 = lane >> 4 & 1, b3 = lane >> 3 & 1, b2 = lane >> 2 & 1;
  const int pair = kC == 1 ? 0 : kC == 2 ? b4 : b4 * 2 + b3, second = kC == 1 ? b4 : kC == 2 ? b3 : b2;
  return pair * 8 + (lane & 3) * 2 + second;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}
// 2^e.
constexpr float exp2_of(int e) { return e == 0 ? 1.f : e < 0 ? 0.5f * exp2_of(e + 1) : 2.f * exp2_of(e - 1); }
// The exponent of a value scale, 128 of one that is no number, and 2 / 2^exponent, which is 0 then.
__device__ __forceinline__ int scale_exp(float s) {
  return max((int)(__float_as_uint(s) >> 23 & 255u) - 127, kMinScaleExp);
}
__device__ __forceinline__ float two_over_exp(float s) { return __uint_as_float((uint32_t)(128 - scale_exp(s)) << 23); }

// Two values as E4M3 (lower half) and what their rounding left, again as E4M3 (upper half). By way of fp16, whose 11
// bits hold the two terms' 4 + 4 and what is lost to it (2^-11) is below what is lost to them (2^-8).
__device__ __forceinline__ uint32_t two_terms(float2 x) {
  uint32_t h, back;
  uint16_t first, rest;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x.y), "f"(x.x));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(first) : "r"(h));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(first));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(rest) : "r"(h));
  return (uint32_t)first | ((uint32_t)rest << 16);
}
// Eight values as E4M3 (first) and what their rounding left, again as E4M3 (rest).
__device__ __forceinline__ void two_terms(const float (&x)[8], uint2& first, uint2& rest) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = e4m3x2(x[2 * i], x[2 * i + 1]);
    const float2 f = from_e4m3x2(a[i]);
    const float2 r = __fadd2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(-f.x, -f.y));
    b[i] = e4m3x2(r.x, r.y);
  }
  first = make_uint2(a[0] | (a[1] << 16), a[2] | (a[3] << 16));
  rest = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
}
__device__ __forceinline__ uint4 to_bf16x8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)f32_to_bf16(x[2 * i]) | ((uint32_t)f32_to_bf16(x[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four values as bf16, with a gate taken times 1 / (1 + e^-gate) first.
__device__ __forceinline__ uint2 to_out(float4 o, bool gated, uint2 gate) {
  if (gated) {
    o.x = __fdividef(o.x, 1.f + __expf(-bf16_to_f32((uint16_t)(gate.x & 0xffff))));
    o.y = __fdividef(o.y, 1.f + __expf(-bf16_to_f32((uint16_t)(gate.x >> 16))));
    o.z = __fdividef(o.z, 1.f + __expf(-bf16_to_f32((uint16_t)(gate.y & 0xffff))));
    o.w = __fdividef(o.w, 1.f + __expf(-bf16_to_f32((uint16_t)(gate.y >> 16))));
  }
  return make_uint2((uint32_t)f32_to_bf16(o.x) | ((uint32_t)f32_to_bf16(o.y) << 16),
                    (uint32_t)f32_to_bf16(o.z) | ((uint32_t)f32_to_bf16(o.w) << 16));
}

// Byte `at` of row `row` in a block of 128-byte rows under the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(int row, int at) {
  return (uint32_t)(row * 128 + ((((at >> 4) ^ (row & 7)) << 4) | (at & 15)));
}

// Descriptor of 128-byte swizzled rows read along their other dimension: a row is one step of the
// contraction, its 128 bytes run along M or N; eight-row groups 1024 bytes apart, and the next 128
// bytes of M one ring block further (used by bf16 alone, where 128 values are two blocks).
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kBlock >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// Eight consecutive columns of this thread's lane, without waiting.
__device__ __forceinline__ void ld8_nowait(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

__device__ __forceinline__ void sync_group(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// 128 threads of barrier `id`: whether any of them says so.
__device__ __forceinline__ bool any_in_group(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ int cta_of(long long tile, long long total, int grid) {
  return (int)(((tile + 1) * grid - 1) / total);
}

// The query rows of a segment into query buffer qb, as rows of the MMAs' second operand, with their masks and
// factors. `share` of `shares` warps take eight rows at a time.
template <int D, bool kE4m3, int kRows>
__device__ __noinline__ void load_queries(const Args& a, const Seg& s, unsigned char* rest, int qb, int share, int shares) {
  using C = Cfg<D, kE4m3, kRows>;
  const TreeAttnArgs& p = a.p;
  const int lane = threadIdx.x & 31;
  const int rp = C::row_pad(a.rows), q_block = C::q_block(a.rows);
  // scores are maxima before they are scaled: a negative scale turns the query's sign, none leaves zeros
  const uint32_t sign = p.scale < 0.f ? 0x80008000u : 0u, mask_q = p.scale == 0.f ? 0u : ~0u;
  const float to_log2 = p.scale == 0.f ? 1.f : fabsf(p.scale) * kLog2e;
  const int h = s.u / a.row_tiles, r0 = (s.u % a.row_tiles) * a.rows;
  unsigned char* q_s = rest + C::oQ + qb * C::q_bytes(a.rows);
  float* qs_s = reinterpret_cast<float*>(rest + C::oQs) + qb * kRows;
  uint64_t* mask_s = reinterpret_cast<uint64_t*>(rest + C::oMask) + qb * kRows;
  if (share == 0)
    for (int r = lane; r < rp; r += 32) {
      const int j = (r0 + r) / p.G;
      uint64_t m = 0;
      if (r < a.rows && j < p.P) m = p.mask ? __ldg(p.mask + (size_t)s.n * p.P + j) : j == 63 ? ~0ull : (2ull << j) - 1;
      mask_s[r] = m & ~0ull >> (64 - p.P);
    }
  // rows on their way at once: more hide their loads at the start of a short segment, fewer leave the instruction
  // cache to the loops (256 x 1k..8k tokens with 6 rows: 288 us with four, 294 with eight; 32 trees of 48 rows: 196 and 177)
  constexpr int kBatch = kRows == 16 ? 4 : 8;
  for (int rb = share * kBatch; rb < rp; rb += shares * kBatch) {
    uint4 raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = rb + i, j = (r0 + r) / p.G, g = (r0 + r) % p.G;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < a.rows && j < p.P && lane < D / 8)
        raw[i] = *reinterpret_cast<const uint4*>(p.q + (((size_t)s.n * p.P + j) * p.Hq + h * p.G + g) * D + lane * 8);
      raw[i] = make_uint4((raw[i].x ^ sign) & mask_q, (raw[i].y ^ sign) & mask_q, (raw[i].z ^ sign) & mask_q,
                          (raw[i].w ^ sign) & mask_q);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = rb + i;
      if constexpr (!kE4m3) {
        // eight values are one 16-byte piece of block lane / 8
        if (lane < D / 8)
          *reinterpret_cast<uint4*>(q_s + (lane >> 3) * q_block + swz(r, (lane & 7) * 16)) = raw[i];
        if (lane == 0) qs_s[r] = fmaxf(to_log2, 1e-37f);
      } else {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float x[8], most = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = __uint_as_float(w[e] << 16);
          x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(x[e]));
        most = warp_max(most);
        // a power of two that takes the largest value below 256; a row with an infinity has no scores
        const int ex = (int)(__float_as_uint(most) >> 23) - 127;
        const int up = most == 0.f ? 0 : min(7 - ex, 120);
        const float f = __uint_as_float((uint32_t)(up + 127) << 23);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= f;
        uint2 first, second;
        two_terms(x, first, second);
        if (lane < D / 8) {
          unsigned char* blk = q_s + (lane >> 4) * q_block;
          *reinterpret_cast<uint2*>(blk + swz(r, (lane & 15) * 8)) = first;
          *reinterpret_cast<uint2*>(blk + swz(rp + r, (lane & 15) * 8)) = second;
        }
        const float down = __uint_as_float((uint32_t)(127 - up) << 23);
        if (lane == 0) qs_s[r] = ex == 128 ? __uint_as_float(0x7fffffffu) : fmaxf(to_log2 * down, 1e-37f);
      }
    }
  }
}

template <int D, bool kE4m3, int kRows>
__global__ void __launch_bounds__(Cfg<D, kE4m3, kRows>::kThreads, 1) tree_attn_kernel(const Args a, const __grid_constant__ CUtensorMap tmk,
                                                      const __grid_constant__ CUtensorMap tmv) {
  using C = Cfg<D, kE4m3, kRows>;
  constexpr int kThreads = C::kThreads;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int stages = C::stages(a.rows);
  unsigned char* rest = smem + stages * kBlock;
  Bars* B = reinterpret_cast<Bars*>(rest + C::oBars);
  const TreeAttnArgs& p = a.p;
  const KvArgs& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem);

  auto set_up = [&] {
    if (tid != 0) return;
    for (int i = 0; i < stages; ++i) mbar_init(&B->empty[i], 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&B->k_full[i], 1);
      mbar_init(&B->v_full[i], 1);
    }
    for (int i = 0; i < kMarks; ++i) {
      mbar_init(&B->v_issued[i], 1);
      mbar_init(&B->v_clean[i], 32);
      mbar_init(&B->checked[i], 1);
    }
    for (int i = 0; i < C::kQBuf; ++i) {
      mbar_init(&B->q_full[i], 32);
      mbar_init(&B->q_empty[i], 1 + 8 + 4 * C::kOutGroups);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->s_full[i], 1);
      mbar_init(&B->s_empty[i], C::kSoftWarps);
      mbar_init(&B->p_full[i], C::kSoftWarps * 32);
      mbar_init(&B->o_full[i], 1);
      mbar_init(&B->o_empty[i], 4 * C::kOutGroups);
      mbar_init(&B->st_full[i], C::kSoftWarps * 32);
    }
    for (int i = 0; i < kScSlots; ++i) {
      mbar_init(&B->sc_full[i], 1);
      mbar_init(&B->sc_empty[i], C::kSoftWarps);
    }
    mbar_init(&B->drain, 1);
    B->abort = 0;
    B->plan.count = 0;
    fence_mbar_init();
  };
  if constexpr (C::kEarly) {
    set_up();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing of the kernel before is read or written earlier
  }
  // ---- this CTA's piece: a scan over the requests' tiles
  {
    const int per = (p.N + kThreads - 1) / kThreads, n0 = min(p.N, tid * per), n1 = min(p.N, n0 + per);
    long long mine = 0;
    bool too_long = false;
    for (int n = n0; n < n1; ++n) {
      const int tiles = tiles_of(a, p.ctx[n], &too_long);
      mine += tiles + (tiles > 0 ? C::kSegCost : 0);
    }
    if (too_long && blockIdx.x == 0) report(p.dev_err, GDN_DEVERR_OFFSETS);
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 31) B->warp_total[warp] = upto;
    if constexpr (!C::kEarly) set_up();
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += B->warp_total[w];
      total += B->warp_total[w];
    }
    before += upto - mine;
    const int units = c.Hkv * a.row_tiles;
    total *= units;
    const long long ctas = min((long long)gridDim.x, total);  // with a piece: none of them empty
    const long long lo = ctas ? total * blockIdx.x / ctas : 0, hi = ctas ? total * (blockIdx.x + 1) / ctas : 0;
    if (blockIdx.x < ctas && before * units <= lo && lo < (before + mine) * units) {
      long long at = before * units;
      for (int n = n0; n < n1; ++n) {
        const int tiles = tiles_of(a, p.ctx[n]), places = tiles + (tiles > 0 ? C::kSegCost : 0);
        const long long here = (long long)places * units;
        if (lo < at + here) {
          B->plan = Plan{total, lo, (int)(hi - lo), n, (int)((lo - at) / places), (int)((lo - at) % places)};
          break;
        }
        at += here;
      }
    }
    if (warp == C::kMmaWarp) umma::tmem_alloc(&B->tmem, 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
  }
  const Plan plan = B->plan;
  asm volatile("griddepcontrol.launch_dependents;");  // the join may be set up; it waits for this grid's end
  if (tid == 0) {
    static_cast<Desc*>(p.workspace)[blockIdx.x].valid = 0;
    for (int k = 0; k < 2; ++k) {
      int* written = reinterpret_cast<int*>(partial(a, blockIdx.x, k)) + 2 * a.rows;
      written[0] = written[1] = 1;
    }
  }
  // All warps but the copies' load the first query rows: no tile can be scored before.
  if (warp != C::kCopyWarp) {
    Walk<C::kSegCost> walk(a, plan);
    Seg s;
    if (walk.next(a, s)) {
      load_queries<D, kE4m3, kRows>(a, s, rest, 0, warp < C::kCopyWarp ? warp : warp - 1, kThreads / 32 - 1);
      umma::fence_proxy_async_smem();
    }
    asm volatile("bar.sync 5, %0;" ::"n"(C::kThreads - 32) : "memory");
  }
  const uint32_t tmem = B->tmem;
  int* abort = &B->abort;

  if (warp == C::kCopyWarp) {
    // ------------------------------------------------------------ copies
    // K of a tile (with the tile's scales), then V of the tile kAhead before it: the order in which the
    // MMAs take them.
    const int boxes = kTile / a.box, total_rows = c.slots * c.Hkv;
    int st = 0, phase = 1, i = 0;
    bool ok = true;
    auto blocks = [&](const CUtensorMap* map, int row, uint64_t* full) {
      if (lane == 0) mbar_arrive_expect_tx(full, C::kBlk * kBlock);
      __syncwarp();
      for (int b = 0; b < C::kBlk; ++b) {
        ok = __all_sync(0xffffffffu, ok && wait(&B->empty[st], phase, abort));
        if (ok && lane < boxes)
          tma_load_2d(smem + st * kBlock + lane * a.box * 128, map, b * (kE4m3 ? 128 : 64), row, full);
        if (++st == stages) st = 0, phase ^= 1;
      }
    };
    Walk<C::kSegCost> walk(a, plan);
    Seg s;
    int held[C::kAhead];  // rows of the last tiles, their V still to come
    int marks = 0;
    uint32_t last_tiles = 0;  // bit i % 32: tile i has drafted tokens
    auto value_blocks = [&](int j, int row) {
      blocks(&tmv, row, &B->v_full[j % kSlots]);
      if ((last_tiles >> (j & 31)) & 1) {
        if (lane == 0) arrive(&B->v_issued[marks % kMarks]);
        ++marks;
      }
    };
    while (ok && walk.next(a, s)) {
      const int h = s.u / a.row_tiles;
      const int32_t* table = p.table + (size_t)s.n * p.max_pages;
      auto row_of = [&](int t) {  // first row of this lane's box; behind the last token: rows that read as zeros
        const int tok = t * kTile + lane * a.box;
        if (lane >= boxes || tok >= s.len) return total_rows;
        const int page = __ldg(table + tok / c.page);
        if (page < 0 || page >= c.pages) return total_rows;
        return (page * c.Hkv + h) * c.page + tok % c.page;
      };
      int row = row_of(s.t0);
      for (int t = s.t0; t < s.t1 && ok; ++t, ++i) {
        const int next = t + 1 < s.t1 ? row_of(t + 1) : 0;
        if constexpr (kE4m3) {
          const int slot = i % kScSlots;
          ok = __all_sync(0xffffffffu, ok && wait(&B->sc_empty[slot], ((i / kScSlots) & 1) ^ 1, abort));
          if (!ok) break;
          const bool in = row < total_rows;
          const uint32_t bytes = a.box * 4, all = 2 * bytes * __popc(__ballot_sync(0xffffffffu, in));
          if (lane == 0) mbar_arrive_expect_tx(&B->sc_full[slot], all);
          __syncwarp();
          if (in) {
            unsigned char* dst = rest + C::oSc + slot * 2 * kTile * 4 + lane * bytes;
            bulk_g2s_plain(dst, c.k_scale + row, bytes, &B->sc_full[slot]);
            bulk_g2s_plain(dst + kTile * 4, c.v_scale + row, bytes, &B->sc_full[slot]);
          }
        }
        blocks(&tmk, row, &B->k_full[i % kSlots]);
        if (ok && i >= C::kAhead) value_blocks(i - C::kAhead, held[0]);
        if constexpr (C::kAhead == 2) held[0] = held[1];
        held[C::kAhead - 1] = row;
        last_tiles = (last_tiles & ~(1u << (i & 31))) | (((t + 1) * kTile > s.ctx ? 1u : 0u) << (i & 31));
        row = next;
      }
    }
    if constexpr (C::kAhead == 2)
      if (ok && i > 1) value_blocks(i - 2, held[0]);
    if (ok && i > 0) value_blocks(i - 1, held[C::kAhead - 1]);
    if (!ok) {
      // copies in flight land before the CTA may leave (bounded: a barrier whose copies were not all issued
      // runs into the limit)
      for (int k = max(0, i - kSlots); k <= i; ++k) {
        if (!mbar_wait_bounded(&B->k_full[k % kSlots], (k / kSlots) & 1)) break;
        if (k > C::kAhead && !mbar_wait_bounded(&B->v_full[(k - C::kAhead) % kSlots], ((k - C::kAhead) / kSlots) & 1)) break;
      }
      if constexpr (kE4m3)
        for (int k = max(0, i - kScSlots); k < i; ++k) mbar_wait_bounded(&B->sc_full[k % kScSlots], (k / kScSlots) & 1);
    }
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMAs
    // The whole warp walks and waits, one elected thread issues: with `if (lane == 0)` instead an MMA took
    // 73 cycles to issue on an idle SM, and about 200 next to the other warps; its work is 41 at 16 columns.
    const int rp = C::row_pad(a.rows);  // rows as columns of the MMAs
    const int q_block = C::q_block(a.rows), q_bytes = C::q_bytes(a.rows);
    static_assert(C::cols_ok(), "columns of the MMAs, for every number of rows");
    const int N = C::mma_cols(a.rows);
    constexpr uint32_t kKind = kE4m3 ? umma::kKindF8 : umma::kKindF16, kType = kE4m3 ? umma::kE4M3 : umma::kBF16;
    const uint32_t id_s = umma::idesc(kType, false, false, kTile, N), id_o = umma::idesc(kType, true, true, kTile, N);
    const uint32_t sQ = smem_u32(rest + C::oQ), sP = smem_u32(rest + C::oP);
    int st = 0, i = 0, seg = 0, marks = 0;
    uint32_t last_tiles = 0;  // bit i % 32: tile i has drafted tokens, the check warp cleans its V
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && wait(bar, parity, abort);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    // two at once: a wait whose phase is over costs 130 cycles of this warp, the tightest of all at few rows
    auto wait_both = [&](uint64_t* x, uint32_t px, uint64_t* y, uint32_t py) {
      const bool x_done = mbar_try_wait(x, px), y_done = mbar_try_wait(y, py);
      if (!x_done || !y_done) ok = ok && wait(x, px, abort) && wait(y, py, abort);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    auto product_o = [&](int j) {
      const int b = j & 1, ob = j % C::kOBuf;
      // (the softmax waited for the output of two tiles back: its place in tensor memory is free)
      if (!wait_both(&B->p_full[b], (j >> 1) & 1, &B->v_full[j % kSlots], (j / kSlots) & 1)) return;
      if ((last_tiles >> (j & 31)) & 1) {
        if (!wait_all(&B->v_clean[marks % kMarks], (marks / kMarks) & 1)) return;
        ++marks;
      }
#pragma unroll
      for (int h = 0; h < C::kHalves; ++h) {
        const int st2 = kE4m3 ? st : st + 1;  // two bf16 blocks are side by side
        umma::fence_after_sync();
        if (elect_one()) {
          const uint32_t d = tmem + 2 * C::kCols + (ob * C::kHalves + h) * C::kOCols;
          constexpr int kSteps = kE4m3 ? 4 : 8, kStepBytes = kE4m3 ? 4096 : 2048;  // 32 or 16 tokens a step
          const uint64_t va = desc_mn(ring + st * kBlock), pa = desc_mn(sP + b * kBlock);
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
            umma::mma<kKind>(d, va + k * (kStepBytes >> 4), pa + k * (kStepBytes >> 4), id_o, k > 0);
          if constexpr (C::kSumTerms) {  // the second terms, 64 bytes on
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
              umma::mma<kKind>(d, va + k * (kStepBytes >> 4), pa + 4 + k * (kStepBytes >> 4), id_o, 1);
          }
          umma::commit(&B->empty[st]);
          if (!kE4m3) umma::commit(&B->empty[st2]);
          if (h == C::kHalves - 1) {
            umma::commit(&B->o_full[ob]);
          }
        }
        __syncwarp();
        st = st2 + 1 == stages ? 0 : st2 + 1;
      }
    };
    Walk<C::kSegCost> walk(a, plan);
    Seg s;
    while (ok && walk.next(a, s)) {
      const int qb = seg % C::kQBuf;
      if (!wait_all(&B->q_full[qb], (seg / C::kQBuf) & 1)) break;
      for (int t = s.t0; t < s.t1 && ok; ++t, ++i) {
        const int b = i & 1;
        if (!wait_both(&B->s_empty[b], ((i >> 1) & 1) ^ 1, &B->k_full[i % kSlots], (i / kSlots) & 1)) break;
        const bool last = (t + 1) * kTile > s.ctx;
        last_tiles = (last_tiles & ~(1u << (i & 31))) | ((last ? 1u : 0u) << (i & 31));
        for (int kb = 0; kb < C::kBlk; ++kb) {
          umma::fence_after_sync();
          if (elect_one()) {
            const uint64_t ka = umma::smem_desc_sw128(ring + st * kBlock);
            const uint64_t qa = umma::smem_desc_sw128(sQ + qb * q_bytes + kb * q_block);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma::mma<kKind>(tmem + b * C::kCols, ka + 2 * k, qa + 2 * k, id_s, kb + k > 0);
            if constexpr (C::kSumTerms) {  // the second terms, rp rows on
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma::mma<kKind>(tmem + b * C::kCols, ka + 2 * k, qa + rp * 8 + 2 * k, id_s, 1);
            }
            umma::commit(&B->empty[st]);
            if (kb == C::kBlk - 1) {
              umma::commit(&B->s_full[b]);
              if (t + 1 == s.t1) umma::commit(&B->q_empty[qb]);
            }
          }
          __syncwarp();
          if (++st == stages) st = 0;
        }
        if (ok && i >= C::kAhead) product_o(i - C::kAhead);
      }
      ++seg;
    }
    for (int j = max(0, i - C::kAhead); j < i && ok; ++j) product_o(j);
    if (elect_one()) {  // nothing of the tensor core's is in flight when the CTA leaves
      umma::commit(&B->drain);
      mbar_wait_bounded(&B->drain, 0);
    }
    __syncwarp();
  } else if (warp == C::kQueryWarp) {
    // ------------------------------------------------------------ query rows (the first segment's are there)
    Walk<C::kSegCost> walk(a, plan);
    Seg s;
    int seg = 0;
    bool ok = true;
    while (ok && walk.next(a, s)) {
      const int qb = seg % C::kQBuf;
      if (seg > 0) {
        ok = __all_sync(0xffffffffu, wait(&B->q_empty[qb], ((seg / C::kQBuf) & 1) ^ 1, abort));
        if (!ok) break;
        load_queries<D, kE4m3, kRows>(a, s, rest, qb, 0, 1);
        umma::fence_proxy_async_smem();
      }
      arrive(&B->q_full[qb]);
      ++seg;
    }
  } else if (warp == C::kCheckWarp) {
    // ------------------------------------------------------------ pages, and V of the tiles with drafted tokens
    // A weight of zero does not take a NaN or an infinity out of a product. Values behind the last token
    // become zeros (as far as its box goes: behind it they are zeros already); a drafted token's that are no
    // numbers too, and the output warps add them to the rows that see the token.
    Walk<C::kSegCost> walk(a, plan);
    Seg s;
    int seg = 0, marks = 0, i0 = 0, tiles = 0;  // `tiles`: of the piece
    for (Walk<C::kSegCost> all(a, plan); all.next(a, s);) tiles += s.t1 - s.t0;
    bool ok = true;
    while (ok && walk.next(a, s)) {
      const int h = s.u / a.row_tiles;
      const int32_t* table = p.table + (size_t)s.n * p.max_pages;
      bool bad = false;
      const int last_page = (min(s.len, s.t1 * kTile) - 1) / c.page;
      for (int k = s.t0 * kTile / c.page + lane; k <= last_page; k += 32) {
        const int page = __ldg(table + k);
        bad |= page < 0 || page >= c.pages;
      }
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) {
        B->bad[seg % kMarks] = bad;
        arrive(&B->checked[seg % kMarks]);
      }
      for (int t = max(s.t0, s.ctx / kTile); t < s.t1; ++t, ++marks) {
        const int i = i0 + t - s.t0, row0 = max(0, s.ctx - t * kTile), end = min(kTile, s.len - t * kTile);
        const int row1 = (end + a.box - 1) / a.box * a.box;
        uint32_t odd[2] = {0u, 0u};  // nodes with values that are no numbers
        if constexpr (kE4m3)
          for (int row = row0 + lane; row < end; row += 32) {
            const int tok = t * kTile + row, page = __ldg(table + tok / c.page), node = tok - s.ctx;
            if (page < 0 || page >= c.pages) continue;
            const float sv = c.v_scale[((size_t)page * c.Hkv + h) * c.page + tok % c.page];
            if (!(fabsf(sv) < INFINITY)) odd[node >> 5] |= 1u << (node & 31);
          }
        // the copies' warp says when this tile's phase of the barrier has begun: it may be many phases off
        ok = wait(&B->v_issued[marks % kMarks], (marks / kMarks) & 1, abort) &&
             wait(&B->v_full[i % kSlots], (i / kSlots) & 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // V's place in the order of copies
        const int first = C::kBlk * min(i + 1 + C::kAhead, tiles) + C::kBlk * i;
        auto piece = [&](int k) {
          const int row = row0 + k / (8 * C::kBlk), x = k % (8 * C::kBlk);
          return reinterpret_cast<uint4*>(smem + (first + (x >> 3)) % stages * kBlock + row * 128) + (x & 7);
        };
        const int kept = (end - row0) * (8 * C::kBlk), all = (row1 - row0) * (8 * C::kBlk);
#pragma unroll 1
        for (int k = lane; k < kept; k += 32) {
          uint4 v = *piece(k);
          uint32_t* w = reinterpret_cast<uint32_t*>(&v);
          uint32_t any = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t o = 0;
#pragma unroll
            for (int y = 0; y < 32; y += kE4m3 ? 8 : 16) {
              const uint32_t m = (kE4m3 ? 0x7fu : 0x7f80u) << y;
              if ((w[e] & m) == m) o |= (kE4m3 ? 0xffu : 0xffffu) << y;
            }
            w[e] &= ~o;
            any |= o;
          }
          if (any) {
            const int node = t * kTile + row0 + k / (8 * C::kBlk) - s.ctx;
            *piece(k) = v;
            odd[node >> 5] |= 1u << (node & 31);
          }
        }
#pragma unroll 4
        for (int k = kept + lane; k < all; k += 32) *piece(k) = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t lo = __reduce_or_sync(0xffffffffu, odd[0]), hi = __reduce_or_sync(0xffffffffu, odd[1]);
        if (lane == 0) B->dirty[marks % kMarks] = lo | ((unsigned long long)hi << 32);
        umma::fence_proxy_async_smem();
        arrive(&B->v_clean[marks % kMarks]);
      }
      i0 += s.t1 - s.t0;
      ++seg;
    }
  } else if (warp < C::kOutWarp) {
    // ------------------------------------------------------------ softmax
    // A warp has 32 of the tile's tokens; a thread four of them (lane / 4 + 8 i) with a quarter of the rows (2 (lane % 4)
    // and the next of every eight): the reductions over the tokens are three quarters done before the first exchange
    // between lanes. (A token a thread, with all its rows, took 36 exchanges for 32 rows instead of 7, and a reduction
    // instruction for each row's maximum twice as long.)
    const int wg = warp >> 2, w4 = warp & 3, a4 = lane & 3;
    constexpr int kR = C::kSoftRows, kC = kR / 8;
    const int rp = C::row_pad(a.rows);
    const int roff = C::kSplit ? wg * kR : 0;                            // this group's first row
    const int used = min(kC, max(0, (a.rows - roff + 7) / 8));           // its groups of eight rows
    const int mine = reduced_column<kC>(lane);                           // the row whose statistics end in this lane
    const int tt = 32 * w4 + (lane >> 2);                                // the first of this thread's tokens
    float* sums = reinterpret_cast<float*>(rest + C::oSum);
    float* maxima = reinterpret_cast<float*>(rest + C::oMax);
    float* tile_s = reinterpret_cast<float*>(rest + C::oTile);
    float* warp_s = reinterpret_cast<float*>(rest + C::oWarp) + warp * kR;
    const float* scales = reinterpret_cast<const float*>(rest + C::oSc);
    Walk<C::kSegCost> walk(a, plan);
    Seg s;
    int i = 0, seg = 0;
    while (walk.next(a, s)) {
      const int qb = seg % C::kQBuf;
      wait_warp(&B->q_full[qb], (seg / C::kQBuf) & 1, abort);
      const float* qs_s = reinterpret_cast<const float*>(rest + C::oQs) + qb * kRows + roff;
      const uint64_t* mask_s = reinterpret_cast<const uint64_t*>(rest + C::oMask) + qb * kRows + roff;
      for (int t = s.t0; t < s.t1; ++t, ++i) {
        const int b = i & 1, ph = (i >> 1) & 1;
        if (!C::kSplit && b != wg) continue;
        float sk[4], sv[4], ev[4];  // the scales, and the exponents of the values'
        if constexpr (kE4m3) {
          const int slot = i % kScSlots;
          wait_warp(&B->sc_full[slot], (i / kScSlots) & 1, abort);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sk[k] = scales[slot * 2 * kTile + tt + 8 * k];
            sv[k] = t * kTile + tt + 8 * k < s.len ? scales[slot * 2 * kTile + kTile + tt + 8 * k] : 0.f;
          }
          __syncwarp();
          if (lane == 0) arrive(&B->sc_empty[slot]);
          if ((t + 1) * kTile > s.ctx) {
#pragma unroll
            for (int k = 0; k < 4; ++k)  // the values of such a node are zeros, see the check warp
              if (t * kTile + tt + 8 * k >= s.ctx && !(fabsf(sv[k]) < INFINITY)) sv[k] = 0.f;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) ev[k] = (float)scale_exp(sv[k]);
        }
        wait_warp(&B->s_full[b], ph, abort);
        umma::fence_after_sync();
        // scores, not yet taken times the row's factor; E4M3: to base 2, with the exponent of the token's value scale
        float2 x[kC][4];
        const uint32_t ts = umma::taddr(tmem, 32 * w4, b * C::kCols + roff);
#pragma unroll
        for (int g = 0; g < kC; ++g)
          if (g < used) {
            uint32_t u[4][2], w[4][2];
            ld_tile8(ts + g * 8, ts + (16u << 16) + g * 8, u);
            if constexpr (C::kOTerms == 2) ld_tile8(ts + rp + g * 8, ts + (16u << 16) + rp + g * 8, w);
            float2 q2;
            if constexpr (kE4m3) q2 = *reinterpret_cast<const float2*>(qs_s + g * 8 + a4 * 2);
            umma::wait_ld();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float2 v = make_float2(__uint_as_float(u[k][0]), __uint_as_float(u[k][1]));
              if constexpr (C::kOTerms == 2)
                v = __fadd2_rn(v, make_float2(__uint_as_float(w[k][0]), __uint_as_float(w[k][1])));
              if constexpr (kE4m3) v = __ffma2_rn(__fmul2_rn(v, make_float2(sk[k], sk[k])), q2, make_float2(ev[k], ev[k]));
              x[g][k] = v;
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[g][k] = make_float2(0.f, 0.f);
          }
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(&B->s_empty[b]);
        // the output of two tiles back has been read: its statistics, its product and the weights are done with
        wait_warp(&B->o_empty[b], ph ^ 1, abort);
        if ((t + 1) * kTile > s.ctx) {  // drafted tokens, or tokens behind the last
          // of each row, bit 8 k: this thread's token k is seen (one of the context, or a node whose bit is set)
          const int node0 = t * kTile + tt - s.ctx;
          uint32_t before = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) before |= node0 + 8 * k < 0 ? 1u << (8 * k) : 0u;
          auto see = [&](uint64_t m) {
            return before | (uint32_t)(node0 >= 64 || node0 <= -64 ? 0ull : node0 >= 0 ? m >> node0 : m << -node0);
          };
#pragma unroll
          for (int g = 0; g < kC; ++g)
            if (g < used) {
              const uint32_t lo = see(mask_s[g * 8 + a4 * 2]), hi = see(mask_s[g * 8 + a4 * 2 + 1]);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (!((lo >> (8 * k)) & 1)) x[g][k].x = -INFINITY;
                if (!((hi >> (8 * k)) & 1)) x[g][k].y = -INFINITY;
              }
            }
        }
        // ---- the tile's maximum of each row: of the warp first, then of the four warps
        float* max_b = maxima + b * 4 * (kRows + 4);
        {
          float2 m[kC];
#pragma unroll
          for (int g = 0; g < kC; ++g)
            m[g] = make_float2(fmaxf(fmaxf(x[g][0].x, x[g][1].x), fmaxf(x[g][2].x, x[g][3].x)),
                               fmaxf(fmaxf(x[g][0].y, x[g][1].y), fmaxf(x[g][2].y, x[g][3].y)));
          max_b[w4 * (kRows + 4) + roff + mine] = reduce_pairs<kC>(m, lane, [](float u, float v) { return fmaxf(u, v); });
        }
        sync_group(1 + wg);
        if (lane < kR) {
          const float* at = max_b + roff + lane;
          const float m = fmaxf(fmaxf(at[0], at[kRows + 4]), fmaxf(at[2 * (kRows + 4)], at[3 * (kRows + 4)]));
          const float scaled = kE4m3 || m == -INFINITY ? m : m * qs_s[lane];
          warp_s[lane] = m == -INFINITY ? 0.f : kE4m3 ? kTopExp - scaled : -scaled;
          if (w4 == 0) tile_s[b * kRows + roff + lane] = scaled;
        }
        // what makes of a weight with its value's power of two the one with its scale, as a term, and twice the plain one
        float f[4], part[4];
        if constexpr (kE4m3) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            part[k] = two_over_exp(sv[k]);
            f[k] = sv[k] * part[k] * (0.5f * kTermTop * exp2_of(-kTopExp));
          }
        }
        __syncwarp();
        const uint32_t prow = smem_u32(rest + C::oP + b * kBlock) + (32 * w4 + lane) * 128;
        uint32_t even[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int g = 0; g < kC; ++g)
          if (g < used) {
            float2 q2;
            if constexpr (!kE4m3) q2 = *reinterpret_cast<const float2*>(qs_s + g * 8 + a4 * 2);
            const float2 m2 = *reinterpret_cast<const float2*>(warp_s + g * 8 + a4 * 2);
            uint32_t r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 v = kE4m3 ? __fadd2_rn(x[g][k], m2) : __ffma2_rn(x[g][k], q2, m2);
              x[g][k] = make_float2(ex2(v.x), ex2(v.y));
              if constexpr (kE4m3) {
                r[k] = two_terms(__fmul2_rn(x[g][k], make_float2(f[k], f[k])));
              } else {
                const __nv_bfloat162 w = __floats2bfloat162_rn(x[g][k].x, x[g][k].y);
                r[k] = *reinterpret_cast<const uint32_t*>(&w);
              }
            }
            if constexpr (C::kSumTerms) {
              // sixteen rows' first terms are 16 bytes of a token's row of P, two of the one group and two of the
              // other in turn; their second terms 64 bytes on
              if (g % 2 == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) even[k] = r[k];
              }
              if (g % 2 == 1 || g + 1 >= used) {
                uint32_t first[4], second[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t odd = g % 2 ? r[k] : 0u;
                  first[k] = __byte_perm(even[k], odd, 0x5410);
                  second[k] = __byte_perm(even[k], odd, 0x7632);
                }
                st_tile8(prow + (((roff / 16 + g / 2) ^ (lane & 7)) << 4), first);
                st_tile8(prow + (((4 + roff / 16 + g / 2) ^ (lane & 7)) << 4), second);
              }
            } else {
              // eight rows are 16 bytes of a token's row of P, in E4M3 too: two rows' first terms, then their second
              st_tile8(prow + (((roff / 8 + g) ^ (lane & 7)) << 4), r);
            }
          }
        umma::fence_proxy_async_smem();
        arrive(&B->p_full[b]);
        // ---- the warp's sums
        {
          float2 v[kC];
#pragma unroll
          for (int g = 0; g < kC; ++g)
            if constexpr (kE4m3) {
              v[g] = __fmul2_rn(x[g][0], make_float2(part[0], part[0]));
#pragma unroll
              for (int k = 1; k < 4; ++k) v[g] = __ffma2_rn(x[g][k], make_float2(part[k], part[k]), v[g]);
            } else {
              v[g] = __fadd2_rn(__fadd2_rn(x[g][0], x[g][1]), __fadd2_rn(x[g][2], x[g][3]));
            }
          sums[(b * 4 + w4) * kRows + roff + mine] = reduce_pairs<kC>(v, lane, [](float u, float w) { return u + w; });
        }
        arrive(&B->st_full[b]);
      }
      __syncwarp();
      if (lane == 0) arrive(&B->q_empty[qb]);
      ++seg;
    }
  } else {
    // ------------------------------------------------------------ output: thread = value of D
    const int og = (warp - C::kOutWarp) >> 2, ot = tid & 127, bar = 3 + og;
    constexpr int kR = C::kOutRows;
    constexpr int kH = C::kOutHalves;
    const int half = C::kHalves > kH ? og : 0, dim = half * 128 + ot;    // this thread's first value
    const int roff = kR < kRows ? og * kR : 0;                           // its first row
    const int used = min(kR / 8, max(0, (a.rows - roff + 7) / 8));       // its groups of eight rows
    const float* sums = reinterpret_cast<const float*>(rest + C::oSum);
    const float* tile_s = reinterpret_cast<const float*>(rest + C::oTile);
    float* ab = reinterpret_cast<float*>(rest + C::oAb) + og * 4 * kRows;
    float* fin = reinterpret_cast<float*>(rest + C::oFin) + og * kRows;
    int marks = 0;
    Walk<C::kSegCost> walk(a, plan);
    Seg s;
    int i = 0, seg = 0;
    while (walk.next(a, s)) {
      const int qb = seg % C::kQBuf;
      const int h = s.u / a.row_tiles, r0 = (s.u % a.row_tiles) * a.rows + roff;
      const int rows = max(0, min(min(kR, a.rows - roff), p.P * p.G - r0));  // of this thread, in this row tile
      const int32_t* table = p.table + (size_t)s.n * p.max_pages;
      const uint64_t* mask_s = reinterpret_cast<const uint64_t*>(rest + C::oMask) + qb * kRows + roff;
      wait_warp(&B->q_full[qb], (seg / C::kQBuf) & 1, abort);
      float2 acc[kH][kR / 2];
#pragma unroll
      for (int k = 0; k < kH; ++k)
#pragma unroll
        for (int r = 0; r < kR / 2; ++r) acc[k][r] = make_float2(0.f, 0.f);
      float m_run = -INFINITY, l_run = 0.f;  // of row ot of the row tile
      for (int t = s.t0; t < s.t1; ++t, ++i) {
        const int b = i & 1, ph = (i >> 1) & 1, ob = i % C::kOBuf;
        wait_warp(&B->st_full[b], ph, abort);
        float* keep_s = ab + b * 2 * kRows;
        float* w_s = keep_s + kRows;
        bool moved = false;  // a running maximum has changed
        if (ot < a.rows) {
          const float mt = tile_s[b * kRows + ot];
          const float* l4 = sums + b * 4 * kRows + ot;
          float lt = (l4[0] + l4[kRows]) + (l4[2 * kRows] + l4[3 * kRows]);
          const float mn = fmaxf(m_run, mt);
          // E4M3: the maxima are those of the weights with the value scales, the sums are not. A sum may hold against a
          // factor that is too small for a number, so it is taken times the factor's root twice.
          constexpr float kPart = kE4m3 ? 0.5f : 1.f;
          float keep = m_run == -INFINITY ? 0.f : ex2((m_run - mn) * kPart), w = mt == -INFINITY ? 0.f : ex2((mt - mn) * kPart);
          if constexpr (kE4m3) {
            lt *= exp2_of(-kTopExp - 1);
            l_run = l_run * keep * keep + lt * w * w;
            keep *= keep;
            w *= w;
          } else {
            l_run = l_run * keep + lt * w;
          }
          moved = keep != 1.f;
          m_run = mn;
          keep_s[ot] = keep;
          w_s[ot] = kE4m3 ? w * (1.f / kTermTop) : w;
        }
        moved = any_in_group(bar, moved);
        wait_warp(&B->o_full[ob], (i / C::kOBuf) & 1, abort);
        umma::fence_after_sync();
        const uint32_t to = umma::taddr(tmem, 32 * (warp & 3), 2 * C::kCols + (ob * C::kHalves + half) * C::kOCols + roff * C::kOTerms);
        // kN columns at a time hold rows r .. r + 3 and, behind or between them (where P is stored says which), the next
        // four, or with summed terms the same four of the next eight
        constexpr int kN = C::kOTerms * 8, kOn = C::kSumTerms ? 8 : 4;
#pragma unroll
        for (int g = 0; g < kR / 8; ++g)
          if (C::kSumTerms ? g / 2 * 2 < used : g < used) {
            uint32_t u[kH][kN];
#pragma unroll
            for (int k = 0; k < kH; ++k) {
              if constexpr (kN == 16) umma::ld16_nowait(to + k * C::kOCols + g * kN, u[k]);
              else ld8_nowait(to + k * C::kOCols + g * kN, u[k]);
            }
            umma::wait_ld();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = (C::kSumTerms ? g / 2 * 16 + g % 2 * 4 : g * 8) + e * kOn;
              const float4 w4 = *reinterpret_cast<const float4*>(w_s + roff + r);
              float4 k4 = make_float4(1.f, 1.f, 1.f, 1.f);
              if (moved) k4 = *reinterpret_cast<const float4*>(keep_s + roff + r);
#pragma unroll
              for (int k = 0; k < kH; ++k) {
                float2 o[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int at = C::kSumTerms ? 2 * e + 4 * y : kE4m3 ? 8 * e + 4 * y : 4 * e + 2 * y;
                  o[y] = make_float2(__uint_as_float(u[k][at]), __uint_as_float(u[k][at + 1]));
                  if constexpr (C::kOTerms == 2)
                    o[y] = __fadd2_rn(o[y], make_float2(__uint_as_float(u[k][at + 2]), __uint_as_float(u[k][at + 3])));
                }
                float2 &lo = acc[k][r / 2], &hi = acc[k][r / 2 + 1];
                if (moved) {
                  lo = __fmul2_rn(lo, make_float2(k4.x, k4.y));
                  hi = __fmul2_rn(hi, make_float2(k4.z, k4.w));
                }
                lo = __ffma2_rn(o[0], make_float2(w4.x, w4.y), lo);
                hi = __ffma2_rn(o[1], make_float2(w4.z, w4.w), hi);
              }
            }
          }
        umma::fence_before_sync();
        unsigned long long dirty = 0;
        if ((t + 1) * kTile > s.ctx) {
          wait_warp(&B->v_clean[marks % kMarks], (marks / kMarks) & 1, abort);
          dirty = *(volatile unsigned long long*)&B->dirty[marks % kMarks];
          ++marks;
        }
        if (dirty) {
          // drafted tokens whose values are no numbers: to the rows that see them
          for (int node = 0; node < p.P; ++node) {
            if (!((dirty >> node) & 1)) continue;
            const int tok = s.ctx + node, page = __ldg(table + tok / c.page);
            if (page < 0 || page >= c.pages) continue;
            const size_t row = ((size_t)page * c.Hkv + h) * c.page + tok % c.page;
#pragma unroll
            for (int k = 0; k < kH; ++k) {
              const size_t at = row * D + k * 128 + dim;
              float v;
              if constexpr (kE4m3) v = from_e4m3x2(static_cast<const uint8_t*>(c.v)[at]).x * c.v_scale[row];
              else v = bf16_to_f32(static_cast<const uint16_t*>(c.v)[at]);
              if (!(fabsf(v) < INFINITY)) {
#pragma unroll
                for (int r = 0; r < kR; ++r)
                  if (r < rows && ((mask_s[r] >> node) & 1)) (r & 1 ? acc[k][r / 2].y : acc[k][r / 2].x) += v;
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) {
          arrive(&B->o_empty[ob]);
        }
      }
      wait_warp(&B->checked[seg % kMarks], (seg / kMarks) & 1, abort);
      const bool bad = *(volatile int*)&B->bad[seg % kMarks] != 0;
      if (lane == 0) arrive(&B->q_empty[qb]);
      ++seg;
      // ---- the segment's result: whole, or a partial for the join
      if (any_in_group(bar, *(volatile int*)abort)) continue;
      if (bad && ot == 0) report(p.dev_err, GDN_DEVERR_SLOT);
      if (s.t0 == 0 && s.t1 == s.tiles) {
        if (bad) continue;
        if (ot < a.rows) fin[ot] = l_run == 0.f ? 0.f : __fdividef(1.f, l_run);
        // A few rows at a time through shared memory, a thread then has neighbouring values of one or two rows. The
        // loop is not unrolled (the registers' choice is): code that runs once per segment costs its fetches.
        constexpr int kS = C::kStageRows, kY = kS / 4;
        float* stage = reinterpret_cast<float*>(rest + C::oStage) + og * (kS * kH * 128);
        const int mine = ot >> 5, col = (ot & 31) * (4 * kH);  // rows `mine` and `mine` + 4 of the eight, first value
#pragma unroll 1
        for (int rs = 0; rs < rows; rs += kS) {
          size_t at[kY];
          uint2 gate[kY][kH];
#pragma unroll
          for (int y = 0; y < kY; ++y) {
            const int r = rs + mine + 4 * y, rr = r0 + r, j = rr / p.G, g = rr - j * p.G;
            at[y] = (((size_t)s.n * p.P + j) * p.Hq + h * p.G + g) * D + half * 128 + col;
            if (p.gate && r < rows) {
#pragma unroll
              for (int e = 0; e < kH; ++e) gate[y][e] = *reinterpret_cast<const uint2*>(p.gate + at[y] + 4 * e);
            }
          }
          sync_group(bar);
#pragma unroll
          for (int c = 0; c < kR; c += kS)
            if (c == rs) {
#pragma unroll
              for (int k = 0; k < kH; ++k)
#pragma unroll
                for (int e = 0; e < kS; ++e)
                  stage[e * (kH * 128) + k * 128 + ot] = e & 1 ? acc[k][(c + e) / 2].y : acc[k][(c + e) / 2].x;
            }
          sync_group(bar);
#pragma unroll
          for (int y = 0; y < kY; ++y) {
            const int r = rs + mine + 4 * y;
            if (r >= rows) continue;
            const float f = fin[roff + r];
#pragma unroll
            for (int e = 0; e < kH; ++e) {
              const float4 o = *reinterpret_cast<const float4*>(stage + (mine + 4 * y) * (kH * 128) + col + 4 * e);
              *reinterpret_cast<uint2*>(p.out + at[y] + 4 * e) =
                  to_out(make_float4(o.x * f, o.y * f, o.z * f, o.w * f), p.gate, gate[y][e]);
            }
          }
        }
        continue;
      }
      float* mine = partial(a, blockIdx.x, s.t0 == 0);
      if (ot < a.rows && og == 0) {
        mine[ot] = m_run;
        mine[a.rows + ot] = l_run;
      }
      float* rows_at = mine + head_floats(a.rows) + roff * D + dim;
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if (r < rows) {
#pragma unroll
          for (int k = 0; k < kH; ++k) rows_at[r * D + k * 128] = r & 1 ? acc[k][r / 2].y : acc[k][r / 2].x;
        }
      if (ot == 0) {
        reinterpret_cast<int*>(mine)[2 * a.rows + og] = bad;
        if (C::kOutGroups == 1) reinterpret_cast<int*>(mine)[2 * a.rows + 1] = 0;
        if (s.t0 == 0 && og == 0) {
          const int ctas = (int)min((long long)gridDim.x, plan.total);
          static_cast<Desc*>(p.workspace)[blockIdx.x] = Desc{1, s.n, s.u, cta_of(s.first + C::kSegCost + s.tiles - 1, plan.total, ctas)};
        }
      }
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == C::kMmaWarp) umma::tmem_dealloc(tmem, 512);
  if (tid == 0 && *(volatile int*)abort) report(p.dev_err, GDN_DEVERR_TIMEOUT);
}

template <int D, bool kE4m3, int kRows>
cudaError_t launch_rows(const Args& a, const CUtensorMap& tmk, const CUtensorMap& tmv, int grid, cudaStream_t stream) {
  using C = Cfg<D, kE4m3, kRows>;
  const cudaError_t err =
      ensure_dynamic_smem(reinterpret_cast<const void*>(&tree_attn_kernel<D, kE4m3, kRows>), kSmemLimit);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)C::stages(a.rows) * kBlock + C::rest_bytes(a.rows);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = C::kEarly;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, kE4m3, kRows>, a, tmk, tmv);
}

template <bool kE4m3>
cudaError_t launch_format(const Args& a, const CUtensorMap& tmk, const CUtensorMap& tmv, int grid, cudaStream_t stream) {
  if (a.p.D == 256) {
    if (a.rows <= 16) return launch_rows<256, kE4m3, 16>(a, tmk, tmv, grid, stream);
    if (a.rows <= 32) return launch_rows<256, kE4m3, 32>(a, tmk, tmv, grid, stream);
    return launch_rows<256, kE4m3, 64>(a, tmk, tmv, grid, stream);
  }
  if (a.rows <= 16) return launch_rows<128, kE4m3, 16>(a, tmk, tmv, grid, stream);
  if (a.rows <= 32) return launch_rows<128, kE4m3, 32>(a, tmk, tmv, grid, stream);
  return launch_rows<128, kE4m3, 64>(a, tmk, tmv, grid, stream);
}

cudaError_t launch_bf16(const Args& a, const CUtensorMap& tmk, const CUtensorMap& tmv, int grid, cudaStream_t stream);
cudaError_t launch_e4m3(const Args& a, const CUtensorMap& tmk, const CUtensorMap& tmv, int grid, cudaStream_t stream);

}  // namespace tree_attn
}  // namespace gdn
