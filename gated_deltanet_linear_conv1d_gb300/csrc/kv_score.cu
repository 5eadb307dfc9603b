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
// the rows. An E4M3 cache stays E4M3, and Q (bf16, scaled by a power of two per row) is written as the sum of two E4M3
// terms, exact down to 2^-17 of the row's largest value; the second term's MMAs add to the same columns.
//
// Work. The tiles of 128 tokens of all (request, kv head) units stand in one line, cut into equal pieces, one per CTA. Up
// to 128 rows stay in shared memory for a unit's tiles. More are taken in chunks: the piece goes through kSub tiles with
// one chunk after the other, the keys coming from L2 from the second on, and a tile's later chunks add to the weights
// that the same thread has stored.
//
// Roles: two groups of four warps that take the tiles in turn (a thread has one token), a warp for the copies (TMA, 16 KB
// blocks of 128 tokens x 128 bytes into a ring), one for the MMAs, four for the query rows. Every wait is bounded.
#include <type_traits>

#include "tree_attn.cuh"

namespace gdn {
namespace kv_score {

using tree_attn::arrive;
using tree_attn::elect_one;
using tree_attn::ex2;
using tree_attn::kBlock;
using tree_attn::kLog2e;
using tree_attn::kSmemLimit;
using tree_attn::kTile;
using tree_attn::swz;
using tree_attn::wait;
using tree_attn::wait_warp;

constexpr int kMaxRows = 128;  // of a chunk
constexpr int kSub = 8;        // tiles that the chunks of more rows go through in turn
constexpr int kUnitCost = 1;   // what a unit takes beside its tiles, in tiles
constexpr int kQBuf = 2;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kQueryWarp = 10, kQueryWarps = 4;
static_assert(kQueryWarps == 4, "see where their flags are read");
constexpr int kThreads = 32 * (kQueryWarp + kQueryWarps);
constexpr int kMaxStages = 12;

struct Args {
  ScoreArgs p;
  KvArgs c;
  int rows, chunks;  // rows of a chunk (the last one may have fewer)
  int box;           // tokens per TMA box
};

struct Plan {
  long long lo;
  int count, n, h, t;  // t: where the piece begins in the unit, whose first kUnitCost places hold no tile
};

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t s_full[2], s_empty[2], q_full[kQBuf], q_empty[kQBuf], drain;
  uint32_t tmem;
  int abort;
  int dead[kQBuf][kQueryWarps];  // the buffer has a row that adds nothing
  Plan plan;
  long long warp_total[kThreads / 32];
};

template <int D, bool kE4m3, int kRows>
struct Cfg {
  static constexpr int kBlk = D * (kE4m3 ? 1 : 2) / 128;  // ring blocks of a tile
  static constexpr int kTerms = kE4m3 ? 2 : 1;
  static constexpr int kCols = 2 * kRows < 32 ? 32 : 2 * kRows;  // of tensor memory: two tiles' scores
  static constexpr int kQBytes = kRows * D * 2;            // one buffer
  static constexpr int kBarBytes = (sizeof(Bars) + 15) / 16 * 16;
  // behind the ring: Q, then by row what makes a score a base-2 logarithm of its weight (factor and -lse), then which
  // tokens the row sees: bit i of words 0 and 1: node i, bit 0 of word 2: those of the context
  static constexpr int oFac = kQBuf * kQBytes;
  static constexpr int oLse = oFac + kQBuf * kRows * 4;
  static constexpr int oSees = oLse + kQBuf * kRows * 4;
  static constexpr int oBars = oSees + kQBuf * 3 * kRows * 4;
  static constexpr int kRest = oBars + kBarBytes;
  static constexpr int kFit = (kSmemLimit - kRest) / (int)kBlock;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static_assert(kStages >= 2, "a ring");
};

// What the roles go through: tiles t0 .. t1 - 1 of (request n, kv head h) with the rows of chunk c. `at`: the number of
// tiles before t0 in the piece, each counted once; tile t's scores are in buffer (at + t - t0) % 2, whatever the chunk.
struct Seg {
  int n, h, c, t0, t1, len, ctx, at;
};

// The tiles of a request; none where it is a padding request or breaks the limits.
__device__ __forceinline__ int tiles_of(const Args& a, int n, int* why = nullptr) {
  const ScoreArgs& p = a.p;
  const int ctx = __ldg(p.ctx + n), slot = __ldg(p.slot + n);
  if (ctx < 0 || slot < 0) return 0;
  const long long len = (long long)ctx + p.P;
  int bad = slot >= p.Rs ? GDN_DEVERR_SLOT : 0;
  if ((len + a.c.page - 1) / a.c.page > p.max_pages || len > p.max_tokens) bad |= GDN_DEVERR_OFFSETS;
  if (why) *why |= bad;
  return bad ? 0 : (int)((len + kTile - 1) / kTile);
}

struct Walk {
  int n, h, t, left, tiles, at;
  Seg cur;
  __device__ __forceinline__ Walk(const Args& a, const Plan& p) : n(p.n), h(p.h), t(p.t), left(p.count), tiles(0), at(0) {
    cur.c = a.chunks;  // none
    if (left > 0) tiles = tiles_of(a, n);
  }
  __device__ __forceinline__ bool next(const Args& a, Seg& s) {
    if (cur.c + 1 < a.chunks) {
      ++cur.c;
      s = cur;
      return true;
    }
    while (left > 0) {
      while (tiles == 0) tiles = tiles_of(a, ++n);  // the piece has places left, so a request with some follows
      const int places = tiles + kUnitCost;
      int take = min(places - t, left);
      if (a.chunks > 1) take = min(take, max(kUnitCost - t, 0) + kSub);
      const int ctx = __ldg(a.p.ctx + n);
      cur = Seg{n, h, 0, max(t - kUnitCost, 0), t + take - kUnitCost, ctx + a.p.P, ctx, at};
      left -= take;
      t += take;
      if (t == places) {
        t = 0;
        if (++h == a.c.Hkv) {
          h = 0;
          tiles = 0;
        }
      }
      if (cur.t1 > 0) {
        at += cur.t1 - cur.t0;
        s = cur;
        return true;
      }
    }
    cur.c = a.chunks;
    return false;
  }
};

// The registers of a tensor-memory load, after the wait for it: nothing that uses them moves in front of the wait.
template <int kN>
__device__ __forceinline__ void loaded(uint32_t (&u)[kN]) {
  umma::wait_ld();
#pragma unroll
  for (int i = 0; i < kN; ++i) asm volatile("" : "+r"(u[i]));
}

// The query rows of a segment into buffer qb, as rows of the MMAs' second operand, with their factors and what they see.
// A warp has up to 32 rows in a row, a lane what goes by the row. The rows are copied past the registers, all of them on
// their way at once. An E4M3 cache's are then taken apart into their two terms in place: a row's 2 D bytes are its own.
template <int D, bool kE4m3, int kRows>
__device__ __forceinline__ void load_queries(const Args& a, const Seg& s, unsigned char* rest, Bars* B, int qb, int share) {
  using C = Cfg<D, kE4m3, kRows>;
  static_assert(kRows <= 32 * kQueryWarps, "a lane per row");
  const ScoreArgs& p = a.p;
  const int lane = threadIdx.x & 31, rp = (a.rows + 15) / 16 * 16, per = rp / kQueryWarps;
  const uint32_t q_block = rp * 128;
  const int r0 = s.c * a.rows, all = min(a.rows, p.P * p.G - r0);
  unsigned char* q_s = rest + qb * C::kQBytes;
  float* fac = reinterpret_cast<float*>(rest + C::oFac) + qb * kRows;
  float* lse = reinterpret_cast<float*>(rest + C::oLse) + qb * kRows;
  uint32_t* sees = reinterpret_cast<uint32_t*>(rest + C::oSees) + qb * 3 * kRows;
  const int first = share * per, mine = first + lane;
  const bool have = lane < per && mine < all;
  const int j = (r0 + mine) / p.G;
  const size_t row = ((size_t)s.n * p.P + j) * p.Hq + s.h * p.G + (r0 + mine) % p.G;
  const size_t off = have ? row * D : 0;
  // piece `lane` (16 bytes) of row r: where it lies, bf16 values
  auto piece = [&](int r) { return q_s + (lane >> 3) * q_block + swz(r, (lane & 7) * 16); };
  for (int i = 0; i < per; ++i) {
    const size_t o = __shfl_sync(0xffffffffu, off, i);
    const int r = first + i;
    if (lane < D / 8) {
      const uint32_t bytes = r < all ? 16u : 0u;  // zeros behind the last row
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(piece(r))), "l"(p.q + o + lane * 8), "r"(bytes)
                   : "memory");
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  const float l = have ? __ldg(p.lse + row) : INFINITY;
  uint64_t m = 0;
  if (have) m = p.mask ? __ldg(p.mask + (size_t)s.n * p.P + j) : j == 63 ? ~0ull : (2ull << j) - 1;
  const bool live = fabsf(l) < INFINITY;  // a row without a finite sum adds nothing
  m = live ? m & ~0ull >> (64 - p.P) : 0ull;
  if (lane < per) {
    lse[mine] = live ? -l * kLog2e : -INFINITY;
    sees[mine] = (uint32_t)m;
    sees[kRows + mine] = (uint32_t)(m >> 32);
    sees[2 * kRows + mine] = live;
  }
  const bool dead = __any_sync(0xffffffffu, have && !live);
  if (lane == 0) B->dead[qb][share] = dead;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if constexpr (kE4m3) {
    const float f0 = p.scale * kLog2e;
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < per; ++i) {
      const int r = first + i;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (lane < D / 8) raw = *reinterpret_cast<const uint4*>(piece(r));
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      float x[8], most = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(x[e]));
      most = tree_attn::warp_max(most);
      // a power of two that takes the largest value below 256; a row with an infinity has no scores
      const int ex = (int)(__float_as_uint(most) >> 23) - 127;
      const int up = most == 0.f ? 0 : min(7 - ex, 120);
      const float by = __uint_as_float((uint32_t)(up + 127) << 23);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= by;
      uint2 one, two;
      tree_attn::two_terms(x, one, two);
      __syncwarp();
      if (lane < D / 8) {
        unsigned char* blk = q_s + (lane >> 4) * q_block + swz(r, (lane & 15) * 8);
        *reinterpret_cast<uint2*>(blk) = one;
        *reinterpret_cast<uint2*>(blk + C::kBlk * q_block) = two;
      }
      if (lane == 0)
        fac[r] = ex == 128 ? __uint_as_float(0x7fffffffu) : f0 * __uint_as_float((uint32_t)(127 - up) << 23);
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->s_full[i], 1);
      mbar_init(&B->s_empty[i], 4);
    }
    for (int i = 0; i < kQBuf; ++i) {
      mbar_init(&B->q_full[i], kQueryWarps);
      mbar_init(&B->q_empty[i], 1 + 8);
    }
    mbar_init(&B->drain, 1);
    B->abort = 0;
    B->plan.count = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing of the kernel before is read or written earlier
  asm volatile("griddepcontrol.launch_dependents;");
  // ---- this CTA's piece: a scan over the requests' tiles
  {
    const int per = (p.N + kThreads - 1) / kThreads, n0 = min(p.N, tid * per), n1 = min(p.N, n0 + per);
    long long mine = 0;
    int why = 0;
    for (int n = n0; n < n1; ++n) {
      const int tiles = tiles_of(a, n, &why);
      mine += tiles + (tiles > 0 ? kUnitCost : 0);
    }
    if (why && blockIdx.x == 0) report(p.dev_err, why);
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 31) B->warp_total[warp] = upto;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += B->warp_total[w];
      total += B->warp_total[w];
    }
    before += upto - mine;
    total *= c.Hkv;
    const long long ctas = min((long long)gridDim.x, total);  // with a piece: none of them empty
    const long long lo = ctas ? total * blockIdx.x / ctas : 0, hi = ctas ? total * (blockIdx.x + 1) / ctas : 0;
    if (blockIdx.x < ctas && before * c.Hkv <= lo && lo < (before + mine) * c.Hkv) {
      long long at = before * c.Hkv;
      for (int n = n0; n < n1; ++n) {
        const int tiles = tiles_of(a, n), places = tiles + (tiles > 0 ? kUnitCost : 0);
        const long long here = (long long)places * c.Hkv;
        if (lo < at + here) {
          B->plan = Plan{lo, (int)(hi - lo), n, (int)((lo - at) / places), (int)((lo - at) % places)};
          break;
        }
        at += here;
      }
    }
    if (warp == kMmaWarp) umma::tmem_alloc(&B->tmem, C::kCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
  }
  const Plan plan = B->plan;
  const uint32_t tmem = B->tmem;
  int* abort = &B->abort;

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------ copies
    const int boxes = kTile / a.box, total_rows = c.slots * c.Hkv;
    int st = 0, phase = 1, issued = 0;
    bool ok = true;
    Walk walk(a, plan);
    Seg s;
    while (ok && walk.next(a, s)) {
      const int32_t* table = p.table + (size_t)s.n * p.max_pages;
      auto row_of = [&](int t) {  // first row of this lane's box; behind the last token: rows that read as zeros
        const int tok = t * kTile + lane * a.box;
        if (lane >= boxes || tok >= s.len) return total_rows;
        const int page = __ldg(table + tok / c.page);
        if (page < 0 || page >= c.pages) return total_rows;
        return (page * c.Hkv + s.h) * c.page + tok % c.page;
      };
      int row = row_of(s.t0);
      for (int t = s.t0; t < s.t1 && ok; ++t) {
        const int next = t + 1 < s.t1 ? row_of(t + 1) : 0;
        for (int b = 0; b < C::kBlk; ++b) {
          ok = __all_sync(0xffffffffu, ok && wait(&B->empty[st], phase, abort));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&B->full[st], kBlock);
          __syncwarp();
          if (lane < boxes) tma_load_2d(smem + st * kBlock + lane * a.box * 128, &tmk, b * (kE4m3 ? 128 : 64), row, &B->full[st]);
          ++issued;
          if (++st == C::kStages) st = 0, phase ^= 1;
        }
        row = next;
      }
    }
    // copies in flight land before the CTA may leave
    if (!ok)
      for (int k = max(0, issued - C::kStages); k < issued; ++k)
        if (!mbar_wait_bounded(&B->full[k % C::kStages], (k / C::kStages) & 1)) break;
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMAs
    const int rp = (a.rows + 15) / 16 * 16;
    const uint32_t q_block = rp * 128;
    constexpr uint32_t kKind = kE4m3 ? umma::kKindF8 : umma::kKindF16, kType = kE4m3 ? umma::kE4M3 : umma::kBF16;
    const uint32_t id = umma::idesc(kType, false, false, kTile, rp);
    const uint32_t ring = smem_u32(smem), sQ = smem_u32(rest);
    int st = 0, phase = 0, seg = 0, used[2] = {0, 0};
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && wait(bar, parity, abort);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    Walk walk(a, plan);
    Seg s;
    while (ok && walk.next(a, s)) {
      const int qb = seg % kQBuf;
      if (!wait_all(&B->q_full[qb], (seg / kQBuf) & 1)) break;
      for (int t = s.t0; t < s.t1 && ok; ++t) {
        const int b = (s.at + t - s.t0) & 1;
        const int use = b ? used[1]++ : used[0]++;
        if (!wait_all(&B->s_empty[b], (use & 1) ^ 1)) break;
        for (int kb = 0; kb < C::kBlk; ++kb) {
          if (!wait_all(&B->full[st], phase)) break;
          umma::fence_after_sync();
          if (elect_one()) {
            const uint64_t ka = umma::smem_desc_sw128(ring + st * kBlock);
#pragma unroll
            for (int term = 0; term < C::kTerms; ++term) {
              const uint64_t qa = umma::smem_desc_sw128(sQ + qb * C::kQBytes + (term * C::kBlk + kb) * q_block);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma::mma<kKind>(tmem + b * kRows, ka + 2 * k, qa + 2 * k, id, kb + term + k > 0);
            }
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
    Walk walk(a, plan);
    Seg s;
    int seg = 0;
    while (walk.next(a, s)) {
      const int qb = seg % kQBuf;
      if (!__all_sync(0xffffffffu, wait(&B->q_empty[qb], ((seg / kQBuf) & 1) ^ 1, abort))) break;
      load_queries<D, kE4m3, kRows>(a, s, rest, B, qb, warp - kQueryWarp);
      umma::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive(&B->q_full[qb]);
      ++seg;
    }
  } else {
    // ------------------------------------------------------------ weights: thread = token
    const int wg = warp >> 2, w4 = warp & 3, mine = 32 * w4 + lane;
    const float* fac_s = reinterpret_cast<const float*>(rest + C::oFac);
    const float* lse_s = reinterpret_cast<const float*>(rest + C::oLse);
    const uint32_t* sees_s = reinterpret_cast<const uint32_t*>(rest + C::oSees);
    Walk walk(a, plan);
    Seg s;
    int seg = 0, used = 0;
    while (walk.next(a, s)) {
      const int qb = seg % kQBuf;
      const int rows = min(a.rows, p.P * p.G - s.c * a.rows);
      const int32_t* table = p.table + (size_t)s.n * p.max_pages;
      const bool fresh = p.init && !p.init[s.n];
      float* out = p.score + ((size_t)__ldg(p.slot + s.n) * c.Hkv + s.h) * p.max_tokens;
      // A token's page, then its key's scale and its score so far, are loaded two tiles and one tile ahead of their use.
      auto load_page = [&](int t) {
        const int tok = t * kTile + mine;
        return t < s.t1 && tok < s.len ? __ldg(table + tok / c.page) : -1;
      };
      const bool again = s.c > 0, old = again || !fresh;
      const float decay = again ? 1.f : p.decay;
      float key_scale = 1.f, before = 0.f;
      auto load_token = [&](int t, int page, float& ks, float& w) {
        const int tok = t * kTile + mine;
        ks = 1.f;
        w = 0.f;
        if (page < 0 || page >= c.pages) return;
        if constexpr (kE4m3) ks = __ldg(c.k_scale + ((size_t)page * c.Hkv + s.h) * c.page + tok % c.page);
        if (old && (again || tok < s.ctx)) w = out[tok];
      };
      int t = s.t0 + ((s.at & 1) == wg ? 0 : 1);
      int page = load_page(t), next_page = load_page(t + 2);
      load_token(t, page, key_scale, before);
      wait_warp(&B->q_full[qb], (seg / kQBuf) & 1, abort);
      const volatile int* d4 = B->dead[qb];
      const bool dead = (d4[0] | d4[1] | d4[2] | d4[3]) != 0;
      const float* fac = fac_s + qb * kRows;
      const float* lse = lse_s + qb * kRows;
      const uint32_t* sees = sees_s + qb * 3 * kRows;
      const float f0 = p.scale * kLog2e;
      for (; t < s.t1; t += 2, ++used) {
        const int this_page = page;
        const float ks = key_scale, w = before;
        page = next_page;
        next_page = load_page(t + 4);
        load_token(t + 2, page, key_scale, before);
        wait_warp(&B->s_full[wg], used & 1, abort);
        umma::fence_after_sync();
        const uint32_t ts = umma::taddr(tmem, 32 * w4, wg * kRows);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // The weights of eight rows' scores. kMasked: not of rows that are left out or behind the last, nor of nodes that
        // a row does not see: by selection, whatever the score is.
        const int node = t * kTile + mine - s.ctx;
        const uint32_t* sees_t = sees + (node < 0 ? 2 : node < 32 ? 0 : 1) * kRows;
        const int bit = node < 0 ? 0 : node & 31;
        auto weights = [&](const uint32_t* u, int r0, auto masked) {
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const int r = r0 + i;
            float4 f = make_float4(f0, f0, f0, f0);
            if constexpr (kE4m3) f = *reinterpret_cast<const float4*>(fac + r);
            const float4 l = *reinterpret_cast<const float4*>(lse + r);
            float2 x[2] = {make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])),
                           make_float2(__uint_as_float(u[i + 2]), __uint_as_float(u[i + 3]))};
            if constexpr (kE4m3) {
              x[0] = __fmul2_rn(x[0], make_float2(ks, ks));
              x[1] = __fmul2_rn(x[1], make_float2(ks, ks));
            }
            x[0] = __ffma2_rn(x[0], make_float2(f.x, f.y), make_float2(l.x, l.y));
            x[1] = __ffma2_rn(x[1], make_float2(f.z, f.w), make_float2(l.z, l.w));
            float e[4] = {ex2(x[0].x), ex2(x[0].y), ex2(x[1].x), ex2(x[1].y)};
            if constexpr (decltype(masked)::value) {
              const uint4 w = *reinterpret_cast<const uint4*>(sees_t + r);
              e[0] = (w.x >> bit) & 1u ? e[0] : 0.f;
              e[1] = (w.y >> bit) & 1u ? e[1] : 0.f;
              e[2] = (w.z >> bit) & 1u ? e[2] : 0.f;
              e[3] = (w.w >> bit) & 1u ? e[3] : 0.f;
            }
            sum[0] = __fadd2_rn(sum[0], make_float2(e[0], e[1]));
            sum[1] = __fadd2_rn(sum[1], make_float2(e[2], e[3]));
          }
        };
        constexpr int kN = kRows < 32 ? 16 : 32;  // rows at a time
        const bool masked = dead || (t + 1) * kTile > s.ctx;
        auto load = [&](int r0, uint32_t (&u)[kN]) {
          if constexpr (kN == 32) umma::ld32_nowait(ts + r0, u);
          else umma::ld16_nowait(ts + r0, u);
        };
        auto compute = [&](int r0, const uint32_t (&u)[kN]) {
          if (!masked && r0 + kN <= rows) {  // no branch inside: the chains of all rows run side by side
#pragma unroll
            for (int i = 0; i < kN; i += 8) weights(u + i, r0 + i, std::false_type());
          } else {
#pragma unroll
            for (int i = 0; i < kN; i += 8)
              if (r0 + i < rows) weights(u + i, r0 + i, std::true_type());
          }
        };
        uint32_t u[kN], v[kN];  // one is on its way while the other is worked on
        load(0, u);
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 2 * kN) {
          loaded(u);
          if (kRows > kN && r0 + kN < rows) load(r0 + kN, v);
          compute(r0, u);
          if (kRows > kN && r0 + kN < rows) {
            loaded(v);
            if (r0 + 2 * kN < rows) load(r0 + 2 * kN, u);
            compute(r0 + kN, v);
          }
        }
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(&B->s_empty[wg]);
        if (t * kTile + mine < s.len && !*(volatile int*)abort) {
          if (this_page < 0 || this_page >= c.pages) report(p.dev_err, GDN_DEVERR_SLOT);
          else out[t * kTile + mine] = fmaf(w, decay, (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
        }
      }
      __syncwarp();
      if (lane == 0) arrive(&B->q_empty[qb]);
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
  if (a.rows <= 64) return launch_rows<D, kE4m3, 64>(a, tmk, grid, stream);
  return launch_rows<D, kE4m3, 128>(a, tmk, grid, stream);
}

}  // namespace kv_score

cudaError_t launch_kv_score(const ScoreArgs& p, const KvArgs& c, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  kv_score::Args a{};
  a.p = p;
  a.c = c;
  const int all = p.P * p.G;
  a.chunks = (all + kv_score::kMaxRows - 1) / kv_score::kMaxRows;
  a.rows = (all + a.chunks - 1) / a.chunks;
  a.chunks = (all + a.rows - 1) / a.rows;
  a.box = tree_attn::box_tokens(c.page);
  CUtensorMap tmk{};
  if (!tree_attn::encode_rows(&tmk, c.k, c, p.D, a.box)) return cudaErrorInvalidValue;
  if (p.D == 256) return c.e4m3 ? kv_score::launch_dim<256, true>(a, tmk, sms, stream)
                                : kv_score::launch_dim<256, false>(a, tmk, sms, stream);
  return c.e4m3 ? kv_score::launch_dim<128, true>(a, tmk, sms, stream)
                : kv_score::launch_dim<128, false>(a, tmk, sms, stream);
}

}  // namespace gdn
