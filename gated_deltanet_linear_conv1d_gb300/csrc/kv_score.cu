// kv_score.cu - gdn_kv_score: the attention weight that every cached token receives from the query rows of its request,
// added to what it has received before.
//
// Math, per request, kv head and cached token t, over the rows r (node j, query head g of the kv head's) that see it:
//   w_t <- decay w_t + sum_r e^(scale (q_r . k_t) - lse_r)
// lse_r is what the attention of the row leaves (gdn_tree_attention_lse): with it a token's weight is a sum over the rows
// alone, and one pass over the keys does, without the values, without a maximum, and with no two CTAs at one token.
//
// S^T [128 tokens x rows] = K Q^T on the tensor cores (tcgen05): the keys are the first operand, from shared memory as
// they lie in the cache, so a token is a lane of tensor memory, and its sum over the rows is one thread's, in the order of
// the rows. An E4M3 cache stays E4M3, and Q (bf16, scaled by a power of two) is written as the sum of two E4M3 terms, exact
// down to 2^-17 of the largest value of the kv head's rows, or, where a row's own power of two is used, 2^-15 of the row's
// largest; the two are columns of one MMA, added as they are read.
//
// Work. The tiles of 128 tokens of all (request, kv head) units stand in one line, cut into equal pieces, one per CTA. A
// unit's rows, up to 64, stay in shared memory for its tiles; more go to kv_score_pair.cu.
//
// Roles: two groups of four warps that take the tiles in turn (a thread has one token), two warps for the copies (TMA, 16 KB
// blocks of 128 tokens x 128 bytes into a ring), one for the MMAs, four for the query rows. Every wait is bounded.
//
// Bound by HBM where there are few rows: 256 requests of 1k .. 8k tokens, 6 rows, E4M3, 152 us for 949 MB, 92 % of the
// copy bandwidth. With more rows a unit's beginning (its pages, its query rows and their constants, its first keys, each a
// trip to memory) is a good part: 32 trees of 8 nodes, 48 rows, on 129 .. 16384 tokens in pages of 16 32 us, for 118 MB.
#include "kv_score.cuh"

namespace gdn {
namespace kv_score {

namespace {

constexpr int kMaxRows = 64;   // more go to pairs
constexpr int kGroups = 2;     // of four warps for the weights
constexpr int kCopyWarp = 4 * kGroups, kCopyWarps = 2, kMmaWarp = kCopyWarp + kCopyWarps, kQueryWarp = kMmaWarp + 1,
              kQueryWarps = 4;
constexpr int kLoaders = 4 * kGroups + kQueryWarps;  // all but those of the copies and the MMAs
constexpr int kThreads = 32 * (kQueryWarp + kQueryWarps);
constexpr int kMaxStages = 12;

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t s_full[kGroups], s_empty[kGroups], q_full[2], q_empty[2], r_empty[2], drain;
  uint32_t tmem;
  int abort;
  int rows[2];      // of the segment, without those that add nothing
  float factor[2];  // what takes its scores to base 2
  uint32_t most[kLoaders], least[kLoaders];
  int uneven[2];    // rows have factors of their own
  Plan plan;
  long long warp_total[kThreads / 32];
};

template <int D, bool kE4m3, int kRows>
struct Cfg {
  static constexpr int kBlk = D * (kE4m3 ? 1 : 2) / 128;  // ring blocks of a tile
  static constexpr int kTerms = kE4m3 ? 2 : 1;
  static constexpr int kBufs = kGroups;                    // tiles' scores in tensor memory
  static constexpr int kCols = 2 * kTerms * kRows;
  static constexpr int kQBytes = kRows * D * 2;            // query rows of a segment
  // behind the ring, for two segments each: Q, then by row -lse to base 2, and the nodes that the row sees (in two words)
  static constexpr int oLse = 2 * kQBytes;
  static constexpr int oSees = oLse + 2 * kRows * 4;
  static constexpr int oOwn = oSees + 2 * 2 * kRows * 4;  // by row, its own factor (E4M3)
  static constexpr int oBars = oOwn + (kE4m3 ? 2 * kRows * 4 : 0);
  static constexpr int kRest = oBars + (sizeof(Bars) + 15) / 16 * 16;
  static constexpr int kFit = (kSmemLimit - kRest) / (int)kBlock;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static_assert(kStages >= 2, "a ring");
};

// The query rows of a segment, number `seg` of the piece, as rows of the MMAs' second operand, with their constants. Rows
// that add nothing (without a finite lse) are left out: the others move up. `shares` warps have an equal part of the rows
// each, a lane what goes by the row. The rows are copied past the registers, all of them on their way at once. An E4M3
// cache's are then taken apart into their two terms in place (a row's 2 D bytes are its own).
template <int D, bool kE4m3, int kRows>
__device__ __noinline__ void load_queries(const Args& a, const Seg& s, unsigned char* rest, Bars* B, int seg, int share,
                                          int shares) {
  using C = Cfg<D, kE4m3, kRows>;
  const ScoreArgs& p = a.p;
  const int lane = threadIdx.x & 31, rp = (a.rows + 15) / 16 * 16;
  const uint32_t q_block = C::kTerms * rp * 128, lower = (1u << lane) - 1u;
  const int r0 = s.c * a.rows, all = min(a.rows, p.P * p.G - r0), b = seg & 1;
  const int per = (all + shares - 1) / shares;
  unsigned char* q_s = rest + b * C::kQBytes;
  float* lse = reinterpret_cast<float*>(rest + C::oLse) + b * kRows;
  uint32_t* sees = reinterpret_cast<uint32_t*>(rest + C::oSees) + b * 2 * kRows;
  const int first = min(all, share * per), end = min(all, first + per);
  const float* lse_g = p.lse + (size_t)s.n * p.P * p.Hq + s.h * p.G;
  const uint16_t* q_g = p.q + ((size_t)s.n * p.P * p.Hq + s.h * p.G) * D;
  auto row_of = [&](int r) {  // from the first position's first row of this kv head
    const int j = (r0 + r) / p.G;
    return j * p.Hq + (r0 + r - j * p.G);
  };
  // every 32 rows' lse up to this warp's last, at once: a lane has the rows g + lane (a plain load: the attention in front
  // may have been writing them when this kernel began)
  constexpr int kMost = (kRows + 31) / 32;
  float l_all[kMost];
#pragma unroll
  for (int g = 0; g < kMost; ++g) {
    const int r = 32 * g + lane;
    l_all[g] = r < end ? lse_g[row_of(r)] : INFINITY;
  }
  // piece `lane` (16 bytes) of row r: where it lies, bf16 values
  const uint32_t q_a = smem_u32(q_s) + (lane >> 3) / C::kTerms * q_block + (lane >> 3) % C::kTerms * rp * 128, piece_at = lane & 7;
  auto piece = [&](int r) { return q_a + r * 128 + ((piece_at ^ (r & 7)) << 4); };
  auto copy = [&](int r, int from) {
    if (lane < D / 8)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(piece(r)), "l"(q_g + (size_t)from * D + lane * 8)
                   : "memory");
  };
  int at = 0;  // live rows so far
  int begin = 0;  // of those before this warp's
#pragma unroll
  for (int g = 0; g < kMost; ++g) {
    if (32 * g >= end) break;
    const int r = 32 * g + lane;
    const float l = l_all[g];
    const uint32_t finite = __ballot_sync(0xffffffffu, fabsf(l) < INFINITY);
    const uint32_t own = first <= 32 * g ? ~0u : first >= 32 * g + 32 ? 0u : ~0u << (first - 32 * g);
    const uint32_t live = finite & own;
    at += __popc(finite & ~own);
    begin += __popc(finite & ~own);
    const int from = row_of(r);
    int to = at;
#pragma unroll 4
    for (uint32_t left = live; left; left &= left - 1) copy(to++, __shfl_sync(0xffffffffu, from, __ffs(left) - 1));
    if (live >> lane & 1) {
      const int mine = at + __popc(live & lower), j = (r0 + r) / p.G;
      uint64_t m = p.mask ? __ldg(p.mask + (size_t)s.n * p.P + j) : j == 63 ? ~0ull : (2ull << j) - 1;
      m &= ~0ull >> (64 - p.P);
      lse[mine] = -l * kLog2e;
      sees[mine] = (uint32_t)m;
      sees[kRows + mine] = (uint32_t)(m >> 32);
    }
    at += __popc(live);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (share == shares - 1 && lane == 0) B->rows[b] = at;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  const float f0 = p.scale * kLog2e;
  if constexpr (!kE4m3) {
    if (share == 0 && lane == 0) B->factor[b] = f0;
  } else {
    __syncwarp();
    auto values = [&](int r) {
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (lane < D / 8)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w) : "r"(piece(r)));
      return raw;
    };
    // the largest magnitude of all loaders' rows, as the bits of a bf16
    auto largest = [](const uint4& w) {
      const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
      return max(m & 0xffffu, m >> 16);
    };
    constexpr uint32_t kInf = 0x7f80u;
    uint32_t row_most = 0;  // of row begin + lane
#pragma unroll 4
    for (int r = begin; r < at; ++r) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, largest(values(r)));
      if (lane == r - begin) row_most = m;
    }
    if (row_most >= kInf) {  // a row with values that are no numbers has no scores, and no say in it
      lse[begin + lane] = __uint_as_float(0x7fffffffu);
      row_most = 0;
    }
    uint32_t most = __reduce_max_sync(0xffffffffu, row_most);
    uint32_t least = __reduce_min_sync(0xffffffffu, row_most > 0 ? row_most : ~0u);
    if (lane == 0) B->most[share] = most, B->least[share] = least;
    asm volatile("bar.sync 1, %0;" ::"r"(32 * shares) : "memory");
    most = __reduce_max_sync(0xffffffffu, lane < shares ? B->most[lane] : 0u);
    least = __reduce_min_sync(0xffffffffu, lane < shares ? B->least[lane] : ~0u);
    asm volatile("bar.sync 1, %0;" ::"r"(32 * shares) : "memory");  // before the next segment's
    const int up = power_of(most), own = power_of(row_most, most);
    if (lane < at - begin) reinterpret_cast<float*>(rest + C::oOwn)[b * kRows + begin + lane] = two_to(up - own);
    if (share == 0 && lane == 0) {
      B->factor[b] = f0 * two_to(-up);
      B->uneven[b] = smaller(least, most);
    }
#pragma unroll 2
    for (int r = begin; r < at; ++r) {
      const float by = two_to(__shfl_sync(0xffffffffu, own, r - begin));
      const uint4 raw = values(r);
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      uint32_t t[4];  // first terms of two values, then their second ones
#pragma unroll
      for (int e = 0; e < 4; ++e)
        t[e] = tree_attn::two_terms(make_float2(__uint_as_float(w[e] << 16) * by, __uint_as_float(w[e] & 0xffff0000u) * by));
      __syncwarp();
      if (lane < D / 8) {
        unsigned char* blk = q_s + (lane >> 4) * q_block + swz(r, (lane & 15) * 8);
        *reinterpret_cast<uint2*>(blk) = make_uint2(__byte_perm(t[0], t[1], 0x5410), __byte_perm(t[2], t[3], 0x5410));
        *reinterpret_cast<uint2*>(blk + rp * 128) =
            make_uint2(__byte_perm(t[0], t[1], 0x7632), __byte_perm(t[2], t[3], 0x7632));
      }
    }
  }
}

template <int D, bool kE4m3, int kRows>
__global__ void __launch_bounds__(kThreads, 1) score_kernel(const Args a, const __grid_constant__ CUtensorMap tmk) {
  using C = Cfg<D, kE4m3, kRows>;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* rest = smem + C::kStages * kBlock;
  Bars* B = reinterpret_cast<Bars*>(rest + C::oBars);
  const ScoreArgs& p = a.p;
  const KvArgs& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&B->s_full[i], 1);
      mbar_init(&B->s_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->q_full[i], kQueryWarps);
      mbar_init(&B->q_empty[i], 1);
      mbar_init(&B->r_empty[i], 4 * kGroups);
    }
    mbar_init(&B->drain, 1);
    B->abort = 0;
    B->plan.count = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing of the kernel before is read or written earlier
  asm volatile("griddepcontrol.launch_dependents;");
  make_plan<kTile, kThreads>(a, blockIdx.x, gridDim.x, B->warp_total, &B->plan);
  if (warp == kMmaWarp) umma::tmem_alloc(&B->tmem, C::kCols);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const Plan plan = B->plan;
  const uint32_t tmem = B->tmem;
  int* abort = &B->abort;
  // The first segment's query rows are loaded by all warps but the copies' and the MMAs', the later ones by the query warps
  // while the segment before is worked on. (Whoever gives up a wait goes on without effect: no warp is missing at a barrier
  // of several.)
  auto load_segment = [&](const Seg& s, int seg, int share) {
    const int qb = seg & 1, parity = ((seg >> 1) & 1) ^ 1;
    wait_warp(&B->q_empty[qb], parity, abort);
    wait_warp(&B->r_empty[qb], parity, abort);
    const bool together = seg == 0;
    load_queries<D, kE4m3, kRows>(a, s, rest, B, seg, together ? share : share - 4 * kGroups, together ? kLoaders : kQueryWarps);
    umma::fence_proxy_async_smem();
    if (together) asm volatile("bar.sync 2, %0;" ::"n"(32 * kLoaders) : "memory");
    else __syncwarp();
    if (share >= 4 * kGroups && lane == 0) arrive(&B->q_full[qb]);
  };

  if (warp >= kCopyWarp && warp < kMmaWarp) {
    // ------------------------------------------------------------ copies
    // The warps take the blocks in turn: a box takes one about 100 cycles, and of pages of 16 tokens there are eight a block.
    // The pages of `span` tiles are loaded at once, a lane per box, and the next tiles' before these are copied.
    const int boxes = kTile / a.box, total_rows = c.slots * c.Hkv, span = 32 / boxes, mine = warp - kCopyWarp;
    int st = 0, phase = 1, issued = 0;
    bool ok = true;
    Walk<kTile> walk(a, plan);
    Seg s;
    bool more = walk.next(a, s);
    auto load_page = [&](const Seg& x, int t) {  // of box `lane` from tile t on; -1 behind the last token
      const long long tok = (long long)t * kTile + lane * a.box;
      return tok < x.len && t + lane / boxes < x.t1 ? __ldg(p.table + (size_t)x.n * p.max_pages + tok / c.page) : -1;
    };
    int page = more ? load_page(s, s.t0) : -1;
    while (ok && more) {
      const Seg cur = s;
      more = walk.next(a, s);
      for (int t0 = cur.t0; t0 < cur.t1 && ok; t0 += span) {
        // the first row of this lane's box; a page out of the pool and behind the last token: rows that read as zeros
        const int tok = t0 * kTile + lane * a.box;
        const int row = page < 0 || page >= c.pages ? total_rows : (page * c.Hkv + cur.h) * c.page + tok % c.page;
        page = t0 + span < cur.t1 ? load_page(cur, t0 + span) : more ? load_page(s, s.t0) : -1;
        for (int t = t0; t < min(cur.t1, t0 + span) && ok; ++t) {
          const int r = __shfl_sync(0xffffffffu, row, (t - t0) * boxes + lane % boxes);
          for (int b = 0; b < C::kBlk; ++b) {
            if (issued % kCopyWarps == mine) {
              ok = __all_sync(0xffffffffu, ok && wait(&B->empty[st], phase, abort));
              if (!ok) break;
              if (lane == 0) mbar_arrive_expect_tx(&B->full[st], kBlock);
              __syncwarp();
              if (lane < boxes)
                tma_load_2d(smem + st * kBlock + lane * a.box * 128, &tmk, b * (kE4m3 ? 128 : 64), r, &B->full[st]);
            }
            ++issued;
            if (++st == C::kStages) st = 0, phase ^= 1;
          }
        }
      }
    }
    // copies in flight land before the CTA may leave
    if (!ok)
      for (int k = max(0, issued - C::kStages); k < issued; ++k)
        if (k % kCopyWarps == mine && !mbar_wait_bounded(&B->full[k % C::kStages], (k / C::kStages) & 1)) break;
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMAs
    const int rp = (a.rows + 15) / 16 * 16;
    const uint32_t q_block = C::kTerms * rp * 128;
    constexpr uint32_t kKind = kE4m3 ? umma::kKindF8 : umma::kKindF16, kType = kE4m3 ? umma::kE4M3 : umma::kBF16;
    const uint32_t ring = smem_u32(smem), sQ = smem_u32(rest);
    int st = 0, phase = 0, seg = 0;
    uint32_t used = 0;  // bit b: parity of buffer b's uses
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && wait(bar, parity, abort);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    Walk<kTile> walk(a, plan);
    Seg s;
    while (ok && walk.next(a, s)) {
      const int qb = seg & 1;
      if (!wait_all(&B->q_full[seg & 1], (seg >> 1) & 1)) break;
      // bf16: the rows that there are; E4M3: the two terms of a row are rp columns apart
      const int cols = kE4m3 ? 2 * rp : max(16, (*(volatile int*)&B->rows[seg & 1] + 15) / 16 * 16);
      const uint32_t id = umma::idesc(kType, false, false, kTile, cols);
      for (int t = s.t0; t < s.t1 && ok; ++t) {
        const int b = (s.at + t - s.t0) % C::kBufs;
        if (!wait_all(&B->s_empty[b], (used >> b & 1) ^ 1)) break;
        used ^= 1u << b;
        for (int kb = 0; kb < C::kBlk; ++kb) {
          if (!wait_all(&B->full[st], phase)) break;
          umma::fence_after_sync();
          if (elect_one()) {
            const uint64_t ka = umma::smem_desc_sw128(ring + st * kBlock);
            const uint64_t qa = umma::smem_desc_sw128(sQ + qb * C::kQBytes + kb * q_block);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma::mma<kKind>(tmem + b * C::kTerms * kRows, ka + 2 * k, qa + 2 * k, id, kb + k > 0);
            umma::commit(&B->empty[st]);
            if (kb == C::kBlk - 1) {
              umma::commit(&B->s_full[b]);
              if (t + 1 == s.t1) umma::commit(&B->q_empty[qb]);
            }
          }
          __syncwarp();
          if (++st == C::kStages) st = 0, phase ^= 1;
        }
      }
      ++seg;
    }
    if (elect_one()) {  // nothing of the tensor core's is in flight when the CTA leaves
      umma::commit(&B->drain);
      mbar_wait_bounded(&B->drain, 0);
    }
    __syncwarp();
  } else if (warp >= kQueryWarp) {
    // ------------------------------------------------------------ query rows
    Walk<kTile> walk(a, plan);
    Seg s;
    int seg = 0;
    while (walk.next(a, s)) {
      load_segment(s, seg, 4 * kGroups + warp - kQueryWarp);
      ++seg;
    }
  } else {
    // ------------------------------------------------------------ weights: thread = token
    const int wg = warp >> 2, w4 = warp & 3, mine = 32 * w4 + lane;
    const int rp = (a.rows + 15) / 16 * 16;
    const float* lse_s = reinterpret_cast<const float*>(rest + C::oLse);
    const uint32_t* sees_s = reinterpret_cast<const uint32_t*>(rest + C::oSees);
    Walk<kTile> walk(a, plan);
    Seg s;
    int seg = 0, used = 0;
    while (walk.next(a, s)) {
      const int rb = seg & 1;
      const int32_t* table = p.table + (size_t)s.n * p.max_pages;
      const bool fresh = p.init && !p.init[s.n];
      float* out = p.score + ((size_t)__ldg(p.slot + s.n) * c.Hkv + s.h) * p.max_tokens;
      // A token's page, then its key's scale and its score so far, are loaded two tiles and one tile ahead of their use.
      auto load_page = [&](int t) {
        const int tok = t * kTile + mine;
        return t < s.t1 && tok < s.len ? __ldg(table + page_of(a, tok)) : -1;
      };
      float key_scale = 1.f, before = 0.f;
      auto load_token = [&](int t, int page, float& ks, float& w) {
        const int tok = t * kTile + mine;
        ks = 1.f;
        w = 0.f;
        if (page < 0 || page >= c.pages) return;
        if constexpr (kE4m3) ks = __ldg(c.k_scale + ((size_t)page * c.Hkv + s.h) * c.page + tok - page_of(a, tok) * c.page);
        if (!fresh && tok < s.ctx) w = out[tok];
      };
      int t = s.t0 + (wg - s.at) % C::kBufs;
      if (t < s.t0) t += C::kBufs;
      int page = load_page(t), next_page = load_page(t + C::kBufs);
      load_token(t, page, key_scale, before);
      if (seg == 0) load_segment(s, seg, warp);
      wait_warp(&B->q_full[rb], (seg >> 1) & 1, abort);
      const int rows = *(volatile int*)&B->rows[rb];
      const float f0 = *(volatile float*)&B->factor[rb];
      const float* lse = lse_s + rb * kRows;
      const uint32_t* sees = sees_s + rb * 2 * kRows;
      const float* own = reinterpret_cast<const float*>(rest + C::oOwn) + rb * kRows;
      const bool uneven = kE4m3 && *(volatile int*)&B->uneven[rb] != 0;
      for (; t < s.t1; t += C::kBufs, ++used) {
        const int this_page = page;
        const float ks = key_scale, w = before;
        page = next_page;
        next_page = load_page(t + 2 * C::kBufs);
        load_token(t + C::kBufs, page, key_scale, before);
        wait_warp(&B->s_full[wg], used & 1, abort);
        umma::fence_after_sync();
        const uint32_t ts = umma::taddr(tmem, 32 * w4, wg * C::kTerms * kRows);
        const float f = kE4m3 ? f0 * ks : f0;
        const int node = t * kTile + mine - s.ctx;
        const bool masked = (t + 1) * kTile > s.ctx;
        constexpr int kN = 16;  // rows at a time
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        struct Scores {
          uint32_t u[kN], v[kE4m3 ? kN : 1];  // v: the second terms'
        };
        auto load = [&](int r0, Scores& x) {
          umma::ld16_nowait(ts + r0, x.u);
          if constexpr (kE4m3) umma::ld16_nowait(ts + rp + r0, x.v);
        };
        auto arrived = [&](Scores& x) {
          loaded(x.u);
          if constexpr (kE4m3) {
            loaded(x.v);
#pragma unroll
            for (int i = 0; i < kN; ++i) x.u[i] = __float_as_uint(__uint_as_float(x.u[i]) + __uint_as_float(x.v[i]));
          }
        };
        auto constants = [&](int r0, float4 (&l)[kN / 4]) {
#pragma unroll
          for (int i = 0; i < kN / 4; ++i) l[i] = *reinterpret_cast<const float4*>(lse + r0 + 4 * i);
        };
        // The weights of four rows' scores. (32 rows of a warp alone: 443 cycles two at a time in packed operations, 198 like
        // this; the exponentials' pipe is busy for 128.)
        auto weights = [&](const uint32_t* u, const float4& l, float (&e)[4], const float4& f) {
          e[0] = ex2(fmaf(__uint_as_float(u[0]), f.x, l.x));
          e[1] = ex2(fmaf(__uint_as_float(u[1]), f.y, l.y));
          e[2] = ex2(fmaf(__uint_as_float(u[2]), f.z, l.z));
          e[3] = ex2(fmaf(__uint_as_float(u[3]), f.w, l.w));
        };
        auto add = [&](const float (&e)[4]) {
#pragma unroll
          for (int y = 0; y < 4; ++y) sum[y] += e[y];
        };
        auto compute = [&](int r0, const uint32_t (&u)[kN], const float4 (&l)[kN / 4]) {
          if (!masked && !uneven && r0 + kN <= rows) {  // no branch inside: the chains of all rows run side by side
#pragma unroll
            for (int i = 0; i < kN; i += 4) {
              float e[4];
              weights(u + i, l[i / 4], e, make_float4(f, f, f, f));
              add(e);
            }
          } else {
            // rows behind the last and nodes that a row does not see: by selection, whatever the score is
#pragma unroll
            for (int i = 0; i < kN; i += 8)
              if (r0 + i < rows) {
#pragma unroll
                for (int y0 = i; y0 < i + 8; y0 += 4) {
                  float e[4];
                  const int r = r0 + y0;
                  float4 fr = make_float4(f, f, f, f);
                  if constexpr (kE4m3) {
                    const float4 o = *reinterpret_cast<const float4*>(own + r);
                    fr = make_float4(f * o.x, f * o.y, f * o.z, f * o.w);
                  }
                  weights(u + y0, l[y0 / 4], e, fr);
                  if (masked && node >= 0) {
                    const uint4 w = *reinterpret_cast<const uint4*>(sees + (node < 32 ? 0 : kRows) + r);
                    const int bit = node & 31;
                    e[0] = (w.x >> bit) & 1u ? e[0] : 0.f;
                    e[1] = (w.y >> bit) & 1u ? e[1] : 0.f;
                    e[2] = (w.z >> bit) & 1u ? e[2] : 0.f;
                    e[3] = (w.w >> bit) & 1u ? e[3] : 0.f;
                  }
#pragma unroll
                  for (int y = 0; y < 4; ++y) e[y] = r + y < rows ? e[y] : 0.f;
                  add(e);
                }
              }
          }
        };
        Scores x, y;  // one is on its way while the other is worked on
        float4 l[kN / 4];
        load(0, x);
        constants(0, l);
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 2 * kN) {
          const int r1 = r0 + kN, r2 = r0 + 2 * kN;
          const bool more = kRows > kN && r1 < rows;
          arrived(x);
          if (more) load(r1, y);
          compute(r0, x.u, l);
          if (more) {
            constants(r1, l);
            arrived(y);
            if (r2 < rows) load(r2, x);
            compute(r1, y.u, l);
            if (r2 < rows) constants(r2, l);
          }
        }
        umma::wait_ld();  // of the first rows, where there are none
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(&B->s_empty[wg]);
        if (t * kTile + mine < s.len && !*(volatile int*)abort) {
          if (this_page < 0 || this_page >= c.pages) report(p.dev_err, GDN_DEVERR_SLOT);
          else out[t * kTile + mine] = fmaf(w, p.decay, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        }
      }
      __syncwarp();
      if (lane == 0) arrive(&B->r_empty[rb]);
      ++seg;
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == kMmaWarp) umma::tmem_dealloc(tmem, C::kCols);
  if (tid == 0 && *(volatile int*)abort) report(p.dev_err, GDN_DEVERR_TIMEOUT);
}

template <int D, bool kE4m3, int kRows>
cudaError_t launch_rows(const Args& a, const CUtensorMap& tmk, int grid, cudaStream_t stream) {
  using C = Cfg<D, kE4m3, kRows>;
  constexpr int kSmem = C::kStages * (int)kBlock + C::kRest;
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(&score_kernel<D, kE4m3, kRows>), kSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, score_kernel<D, kE4m3, kRows>, a, tmk);
}

template <int D, bool kE4m3>
cudaError_t launch_dim(const Args& a, const CUtensorMap& tmk, int grid, cudaStream_t stream) {
  if (a.rows <= 16) return launch_rows<D, kE4m3, 16>(a, tmk, grid, stream);
  return launch_rows<D, kE4m3, 64>(a, tmk, grid, stream);
}

}  // namespace

}  // namespace kv_score

cudaError_t launch_kv_score(const ScoreArgs& p, const KvArgs& c, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  kv_score::Args a{};
  a.p = p;
  a.c = c;
  a.box = tree_attn::box_tokens(c.page);
  a.shift = -1;
  if ((c.page & (c.page - 1)) == 0)
    for (a.shift = 0; 1 << a.shift < c.page;) ++a.shift;
  CUtensorMap tmk{};
  if (!tree_attn::encode_rows(&tmk, c.k, c, p.D, a.box)) return cudaErrorInvalidValue;
  if (p.P * p.G > kv_score::kMaxRows) return kv_score::launch_pairs(a, tmk, p.D, stream);
  a.rows = p.P * p.G;
  a.chunks = 1;
  // the wait for a unit's query rows: trees of 48 rows on 129 .. 16384 tokens 38 us with one tile, 34 with three
  a.cost = a.rows > 16 ? 3 : 1;
  if (p.D == 256) return c.e4m3 ? kv_score::launch_dim<256, true>(a, tmk, sms, stream)
                                : kv_score::launch_dim<256, false>(a, tmk, sms, stream);
  return c.e4m3 ? kv_score::launch_dim<128, true>(a, tmk, sms, stream)
                : kv_score::launch_dim<128, false>(a, tmk, sms, stream);
}

}  // namespace gdn
