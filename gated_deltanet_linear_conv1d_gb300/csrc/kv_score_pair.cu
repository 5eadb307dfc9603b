// kv_score_pair.cu - gdn_kv_score with more than 64 query rows a kv head (the mathematics is in kv_score.cu): a prompt's last
// rows, wide trees.
//
// With many rows the tensor cores bound the work, 2 D operations a row and token, and what feeds them is shared memory:
// an MMA of one CTA reads 128 tokens and all its rows for each step of the contraction, 107 of the 128 bytes a cycle that
// there are with 192 rows of a 256-wide head, beside the copies. So CTAs go in pairs: an MMA (cta_group::2) takes 256
// tokens, 128 of each CTA, and the rows half from each, and every row's bytes are read for both CTAs' tokens at once. It
// also halves what a CTA keeps of Q: up to 384 rows stay for all tiles of a unit, so the keys are read once. (One CTA by
// itself had room for 192, went through the keys twice, from L2 the second time, and waited 5 us for each change of rows:
// 64 x 6 rows on 131071 tokens 115 us.)
//
// A pair tile is 256 tokens. Its rows are taken in up to two steps of up to 192 columns each, a buffer of tensor memory for
// each of two steps; columns 0 .. hs - 1 of a step are rows of the even CTA, the next hs of the odd one. Roles in each CTA:
// four groups of four warps that share a step's columns (two the even CTA's rows, two the odd one's), a warp for the copies,
// one for the MMAs (the even CTA's issues them). The groups load the query rows too. Every wait is bounded.
//
// 64 x 6 rows on 131071 tokens, bf16, 84 us (104 GFLOP, 66 % of the cuBLAS rate): 9 us to the first scores, then 54 steps of
// 192 rows at about 1.2 us each, 1.0 of them the MMAs', with the weights' loop just behind them; 10 us are in neither. 32 x 6
// rows of 8 prompts of 1500 .. 32768 tokens 43 us, 9 of them to the first scores; 11 x 6 rows 39 us: what a unit takes beside
// its tiles weighs most. 2 x 64 x 6 rows in one kv head on 40 .. 70 thousand tokens, E4M3, 33 us, 12 of them to the first
// scores, the rows' terms among them, and 14 the steps.
#include "kv_score.cuh"
#include "pair.cuh"

namespace gdn {
namespace kv_score {

namespace {

constexpr int kPairTile = 2 * kTile;
constexpr int kHalf = 192;       // rows of a chunk that a CTA keeps
constexpr int kStepRows = 96;    // of those, at most, in one step
constexpr int kGroups = 4;       // of four warps for the weights
constexpr int kLoaders = 4 * kGroups;
constexpr int kCopyWarp = kLoaders, kMmaWarp = kLoaders + 1;
constexpr int kThreads = 32 * (kLoaders + 2);
constexpr int kMaxStages = 12;
constexpr int kColsBuf = 256;    // columns of tensor memory from one buffer to the next
constexpr int kSums = 4;         // tiles whose sums the groups may have under way: see where they meet
// Bytes of keys that several chunks go through in turn, a CTA: what all CTAs have stays in L2.
constexpr int kSubBytes = 640 * 1024;

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];  // `full`: the even CTA's count both CTAs' copies
  uint64_t s_full[2], s_empty[2], q_full[2], q_empty, drain;
  uint32_t tmem;
  int abort;
  float factor[2][2];  // what takes the scores of each half's rows to base 2, by segment
  int dead[2][kLoaders];  // the segment has a row that adds nothing
  uint32_t most[kLoaders], least[kLoaders];
  int uneven[2][2];    // rows of the half have factors of their own
  Plan plan;
  long long warp_total[kThreads / 32];
};

template <int D, bool kE4m3>
struct Cfg {
  static constexpr int kBlk = D * (kE4m3 ? 1 : 2) / 128;  // ring blocks of a tile
  static constexpr int kTerms = kE4m3 ? 2 : 1;
  static constexpr int kQBytes = kHalf * D * 2;
  // behind the ring: Q, then by segment, half and row -lse to base 2, and what the row sees: the nodes, in two words, and
  // whether the context; its own factor (E4M3); then the groups' sums
  static constexpr int oLse = kQBytes;
  static constexpr int oSees = oLse + 2 * 2 * kHalf * 4;
  static constexpr int oOwn = oSees + 2 * 3 * 2 * kHalf * 4;
  static constexpr int oSum = oOwn + (kE4m3 ? 2 * 2 * kHalf * 4 : 0);
  static constexpr int oBars = oSum + kSums * kGroups * kTile * 4;
  static constexpr int kRest = oBars + (sizeof(Bars) + 15) / 16 * 16;
  static constexpr int kFit = (kSmemLimit - kRest) / (int)kBlock;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static_assert(kStages > kBlk, "a tile's keys stay for all its steps");
};

// The rows of a chunk: `steps` steps of `hs` rows from each CTA (hs a multiple of 8).
struct Rows {
  int steps, hs;
  __host__ __device__ explicit Rows(int rows) {
    const int half = (rows + 1) / 2;
    steps = (half + kStepRows - 1) / kStepRows;
    hs = ((half + steps - 1) / steps + 7) / 8 * 8;
  }
  // Row of the chunk of place q (step by step) in half g.
  __device__ __forceinline__ int of(int g, int q) const { return q / hs * 2 * hs + g * hs + q % hs; }
};

// Arrives on the barrier of both CTAs, what this thread has written, in either's shared memory, before it.
__device__ __forceinline__ void arrive_both(uint64_t* bar) {
#pragma unroll
  for (int r = 0; r < 2; ++r)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(bar, r)) : "memory");
}
// Waits for arrivals from both CTAs.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, int* abort) {
  return wait(bar, parity, abort) && try_wait_cluster(bar, parity);
}

// Sixteen lanes of tensor memory by sixteen columns, without waiting: this thread has lanes lane / 4 and 8 on, and of every
// eight columns 2 (lane % 4) and the next: registers 4 g .. 4 g + 1 of the one lane, 4 g + 2 .. 4 g + 3 of the other.
__device__ __forceinline__ void ld_rows(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

// The scores of 32 tokens, a warp's, with 16 rows.
struct Scores {
  uint32_t lo[8], hi[8];  // of the lower and the upper sixteen lanes
  __device__ __forceinline__ void load(uint32_t taddr) {
    ld_rows(taddr, lo);
    ld_rows(taddr + (16u << 16), hi);
  }
  // Waits for it: nothing that uses the registers moves in front.
  __device__ __forceinline__ void wait() {
    loaded(lo);
    loaded(hi);
  }
  // Token k (lane / 4 + 8 k), row 8 g + 2 (lane % 4) + y.
  __device__ __forceinline__ float at(int g, int k, int y) const {
    return __uint_as_float((k < 2 ? lo : hi)[4 * g + 2 * (k & 1) + y]);
  }
};

// This CTA's rows of a segment, number `seg` of the piece, as rows of the MMAs' second operand, and the constants of both
// CTAs' rows. The rows are copied past the registers, all of them on their way at once; an E4M3 cache's are then taken
// apart into their two terms in place (a row's 2 D bytes are its own).
template <int D, bool kE4m3>
__device__ __noinline__ void load_queries(const Args& a, const Seg& s, unsigned char* rest, Bars* B, int seg, int share, int pr) {
  using C = Cfg<D, kE4m3>;
  const ScoreArgs& p = a.p;
  const int lane = threadIdx.x & 31, b = seg & 1;
  const Rows rows(a.rows);
  const int held = rows.steps * rows.hs, most_rows = (held + kLoaders - 1) / kLoaders, first = min(held, share * most_rows);
  const int per = min(most_rows, held - first);
  const uint32_t q_block = held * 128;
  const int r0 = s.c * a.rows, all = min(a.rows, p.P * p.G - r0);
  const float* lse_g = p.lse + (size_t)s.n * p.P * p.Hq + s.h * p.G;
  const uint16_t* q_g = p.q + ((size_t)s.n * p.P * p.Hq + s.h * p.G) * D;
  auto row_of = [&](int r) {  // from the first position's first row of this kv head
    const int j = (r0 + r) / p.G;
    return j * p.Hq + (r0 + r - j * p.G);
  };
  // piece `lane` (16 bytes) of row q: where it lies, bf16 values
  const uint32_t q_a = smem_u32(rest) + (lane >> 3) * q_block, piece_at = lane & 7;
  auto piece = [&](int q) { return q_a + q * 128 + ((piece_at ^ (q & 7)) << 4); };
  const int mine = rows.of(pr, first + lane), from = lane < per && mine < all ? row_of(mine) : -1;
  // (plain loads of lse: the attention in front may have been writing it when this kernel began)
  const float own_lse = kE4m3 && from >= 0 ? lse_g[from] : INFINITY;
  const uint32_t there = __ballot_sync(0xffffffffu, from >= 0);
#pragma unroll 8
  for (int i = 0; i < per; ++i) {
    const int o = __shfl_sync(0xffffffffu, from, i);
    if (o >= 0 && lane < D / 8)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(piece(first + i)), "l"(q_g + (size_t)o * D + lane * 8)
                   : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  // ---- the constants
  float* lse = reinterpret_cast<float*>(rest + C::oLse) + b * 2 * kHalf;
  uint32_t* sees = reinterpret_cast<uint32_t*>(rest + C::oSees) + b * 3 * 2 * kHalf;
  bool dead = false;
  for (int i = share * 32 + lane; i < 2 * held; i += 32 * kLoaders) {
    const int g = i >= held, q = i - g * held, r = rows.of(g, q);
    float l = INFINITY;
    uint64_t m = 0;
    if (r < all) {
      const int j = (r0 + r) / p.G;
      l = lse_g[j * p.Hq + (r0 + r - j * p.G)];
      m = p.mask ? __ldg(p.mask + (size_t)s.n * p.P + j) : j == 63 ? ~0ull : (2ull << j) - 1;
      m &= ~0ull >> (64 - p.P);
    }
    const bool live = fabsf(l) < INFINITY;  // a row without a finite sum adds nothing
    if (!live) m = 0;
    dead |= r < all && !live;
    const int at = g * kHalf + q;
    lse[at] = live ? -l * kLog2e : -INFINITY;
    sees[at] = (uint32_t)m;
    sees[2 * kHalf + at] = (uint32_t)(m >> 32);
    sees[4 * kHalf + at] = live;
  }
  dead = __any_sync(0xffffffffu, dead);
  if (lane == 0) B->dead[b][share] = dead;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  float factor = p.scale * kLog2e;
  int uneven = 0;
  if constexpr (kE4m3) {
    __syncwarp();
    auto values = [&](int q) {
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (lane < D / 8)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w) : "r"(piece(q)));
      return raw;
    };
    // the largest magnitude of eight values, as the bits of a bf16
    auto largest = [](const uint4& w) {
      const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
      return max(m & 0xffffu, m >> 16);
    };
    constexpr uint32_t kInf = 0x7f80u;
    uint32_t row_most = 0;  // of row first + lane
#pragma unroll 4
    for (int i = 0; i < per; ++i) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, largest(values(first + i)));
      if (lane == i) row_most = m;
    }
    // one that is not there, adds nothing, or has values that are no numbers, has no say in it
    if (row_most >= kInf || !(fabsf(own_lse) < INFINITY)) row_most = 0;
    uint32_t most = __reduce_max_sync(0xffffffffu, row_most);
    uint32_t least = __reduce_min_sync(0xffffffffu, row_most > 0 ? row_most : ~0u);
    if (lane == 0) B->most[share] = most, B->least[share] = least;
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kLoaders) : "memory");
    most = __reduce_max_sync(0xffffffffu, B->most[lane % kLoaders]);
    least = __reduce_min_sync(0xffffffffu, B->least[lane % kLoaders]);
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kLoaders) : "memory");  // before the next segment's
    const int up = power_of(most), own = power_of(row_most, most);
    uneven = smaller(least, most);
    factor *= two_to(-up);
    if (lane < per) {
      float* at = reinterpret_cast<float*>(rest + C::oOwn) + (b * 2 + pr) * kHalf + first + lane;
#pragma unroll
      for (int r = 0; r < 2; ++r)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(at, r)), "f"(two_to(up - own)) : "memory");
    }
#pragma unroll 2
    for (int i = 0; i < per; ++i) {
      const float by = two_to(__shfl_sync(0xffffffffu, own, i));
      if (!(there >> i & 1)) continue;
      const int q = first + i;
      const uint4 raw = values(q);
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      uint32_t t[4];  // first terms of two values, then their second ones
      uint32_t odd = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[e] = tree_attn::two_terms(make_float2(__uint_as_float(w[e] << 16) * by, __uint_as_float(w[e] & 0xffff0000u) * by));
        // an infinity has no E4M3 value: a NaN in its place, so that the row has no scores
        if ((w[e] & 0x7fffu) >= kInf) odd |= 1u << (2 * e);
        if ((w[e] >> 16 & 0x7fffu) >= kInf) odd |= 2u << (2 * e);
      }
      if (odd) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (odd >> (2 * e) & 1) t[e] |= 0x7fu;
          if (odd >> (2 * e) & 2) t[e] |= 0x7f00u;
        }
      }
      __syncwarp();
      if (lane < D / 8) {
        unsigned char* blk = rest + (lane >> 4) * q_block + swz(q, (lane & 15) * 8);
        *reinterpret_cast<uint2*>(blk) = make_uint2(__byte_perm(t[0], t[1], 0x5410), __byte_perm(t[2], t[3], 0x5410));
        *reinterpret_cast<uint2*>(blk + C::kBlk * q_block) =
            make_uint2(__byte_perm(t[0], t[1], 0x7632), __byte_perm(t[2], t[3], 0x7632));
      }
    }
  }
  if (share == 0 && lane == 0) {  // for the groups of both CTAs that have this one's rows
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(&B->factor[b][pr], r)), "f"(factor) : "memory");
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&B->uneven[b][pr], r)), "r"(uneven) : "memory");
    }
  }
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1) pair_kernel(const Args a, const __grid_constant__ CUtensorMap tmk) {
  using C = Cfg<D, kE4m3>;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* rest = smem + C::kStages * kBlock;
  Bars* B = reinterpret_cast<Bars*>(rest + C::oBars);
  const ScoreArgs& p = a.p;
  const KvArgs& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pr = (int)cluster_ctarank();

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->s_full[i], 1);
      mbar_init(&B->s_empty[i], 2 * kLoaders);
      mbar_init(&B->q_full[i], 2 * kLoaders);
    }
    mbar_init(&B->q_empty, 1);
    mbar_init(&B->drain, 1);
    B->abort = 0;
    B->plan.count = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing of the kernel before is read or written earlier
  asm volatile("griddepcontrol.launch_dependents;");
  make_plan<kPairTile, kThreads>(a, blockIdx.x / 2, gridDim.x / 2, B->warp_total, &B->plan);
  if (warp == kMmaWarp) tmem_alloc_pair(&B->tmem, 512);
  umma::fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before either copies or arrives on them
  umma::fence_after_sync();
  const Plan plan = B->plan;
  const uint32_t tmem = B->tmem;
  int* abort = &B->abort;
  const Rows rows(a.rows);

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------ copies
    // The pages of `span` tiles are loaded at once, a lane per box, and the next tiles' before these are copied.
    const int boxes = kTile / a.box, total_rows = c.slots * c.Hkv, span = 32 / boxes;
    const uint64_t policy = l2_policy_evict_normal();
    int st = 0, phase = 1, issued = 0;
    bool ok = true;
    Walk<kPairTile> walk(a, plan);
    Seg s;
    bool more = walk.next(a, s);
    auto token_of = [&](int t) {  // of box `lane` from tile t on
      return (long long)(t + lane / boxes) * kPairTile + pr * kTile + lane % boxes * a.box;
    };
    auto load_page = [&](const Seg& x, int t) {  // -1 behind the last token
      const long long tok = token_of(t);
      return tok < x.len && t + lane / boxes < x.t1 ? __ldg(p.table + (size_t)x.n * p.max_pages + tok / c.page) : -1;
    };
    int page = more ? load_page(s, s.t0) : -1;
    while (ok && more) {
      const Seg cur = s;
      more = walk.next(a, s);
      for (int t0 = cur.t0; t0 < cur.t1 && ok; t0 += span) {
        // the first row of this lane's box; a page out of the pool and behind the last token: rows that read as zeros
        const int row = page < 0 || page >= c.pages ? total_rows : (page * c.Hkv + cur.h) * c.page + (int)(token_of(t0) % c.page);
        page = t0 + span < cur.t1 ? load_page(cur, t0 + span) : more ? load_page(s, s.t0) : -1;
        for (int t = t0; t < min(cur.t1, t0 + span) && ok; ++t) {
          const int r = __shfl_sync(0xffffffffu, row, (t - t0) * boxes + lane % boxes);
          for (int b = 0; b < C::kBlk; ++b) {
            ok = __all_sync(0xffffffffu, ok && wait(&B->empty[st], phase, abort));
            if (!ok) break;
            if (lane == 0 && pr == 0) mbar_arrive_expect_tx(&B->full[st], 2 * kBlock);  // the pair's
            __syncwarp();
            if (lane < boxes)
              tma_load_2d_pair(smem + st * kBlock + lane * a.box * 128, &tmk, b * (kE4m3 ? 128 : 64), r,
                               cluster_addr(&B->full[st], 0), policy);
            ++issued;
            if (++st == C::kStages) st = 0, phase ^= 1;
          }
        }
      }
    }
    // copies in flight, the other CTA's too, land before either CTA may leave
    if (!ok && pr == 0)
      for (int k = max(0, issued - C::kStages); k < issued; ++k)
        if (!mbar_wait_bounded(&B->full[k % C::kStages], (k / C::kStages) & 1)) break;
    if (!ok && pr == 1) {  // (only the even CTA's barriers know: the limit of a wait)
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t it = 0; it < kWaitMaxIters && globaltimer_ns() - t0 < kWaitLimitNs; ++it) __nanosleep(1000);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMAs
    if (pr == 0) {
      const uint32_t q_block = rows.steps * rows.hs * 128;
      constexpr uint32_t kType = kE4m3 ? umma::kE4M3 : umma::kBF16;
      const uint32_t id = umma::idesc(kType, false, false, kPairTile, 2 * rows.hs);
      const uint32_t ring = smem_u32(smem), sQ = smem_u32(rest);
      int st = 0, phase = 0, seg = 0, step = 0;
      bool ok = true;
      auto agree = [&](bool x) {
        ok = __all_sync(0xffffffffu, ok && x);
        return ok;
      };
      Walk<kPairTile> walk(a, plan);
      Seg s;
      while (ok && walk.next(a, s)) {
        if (!agree(wait_cluster(&B->q_full[seg & 1], (seg >> 1) & 1, abort))) break;
        for (int t = s.t0; t < s.t1 && ok; ++t) {
          int at = st, ph = phase;
          for (int sub = 0; sub < rows.steps && ok; ++sub, ++step) {
            const int b = step & 1;
            if (!agree(wait(&B->s_empty[b], ((step >> 1) & 1) ^ 1, abort))) break;
            const bool last = sub == rows.steps - 1;
            at = st, ph = phase;
            for (int kb = 0; kb < C::kBlk; ++kb) {
              if (sub == 0 && !agree(wait(&B->full[at], ph, abort))) break;
              umma::fence_after_sync();
              if (elect_one()) {
                const uint64_t ka = umma::smem_desc_sw128(ring + at * kBlock);
#pragma unroll
                for (int term = 0; term < C::kTerms; ++term) {
                  const uint64_t qa = umma::smem_desc_sw128(sQ + (term * C::kBlk + kb) * q_block + sub * rows.hs * 128);
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    mma_pair<kE4m3>(tmem + b * kColsBuf, ka + 2 * k, qa + 2 * k, id, kb + term + k > 0);
                }
                if (last) commit_pair(&B->empty[at], 3);
                if (kb == C::kBlk - 1) {
                  commit_pair(&B->s_full[b], 3);
                  if (last && t + 1 == s.t1) commit_pair(&B->q_empty, 3);
                }
              }
              __syncwarp();
              if (++at == C::kStages) at = 0, ph ^= 1;
            }
          }
          st = at;
          phase = ph;
        }
        ++seg;
      }
      if (elect_one()) {  // nothing of the tensor cores' is in flight when the CTAs leave
        commit_pair(&B->drain, 1);
        mbar_wait_bounded(&B->drain, 0);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ weights: a group has a quarter of the columns
    // A thread has four of its warp's tokens (lane / 4 + 8 k) with a quarter of the rows (2 (lane % 4) and the next of every
    // eight), so that what goes by the row is loaded for four tokens at once; at the end it has one token's sum.
    const int g = warp >> 3, part = warp >> 2 & 1, w4 = warp & 3, a4 = lane & 3, mine = 32 * w4 + (lane >> 2) + 8 * a4;
    float* sums = reinterpret_cast<float*>(rest + C::oSum);
    Walk<kPairTile> walk(a, plan);
    Seg s;
    int seg = 0, step = 0, tile = 0;
    while (walk.next(a, s)) {
      const int b2 = seg & 1, all = min(a.rows, p.P * p.G - s.c * a.rows);
      const int32_t* table = p.table + (size_t)s.n * p.max_pages;
      const bool fresh = p.init && !p.init[s.n];
      float* out = p.score + ((size_t)__ldg(p.slot + s.n) * c.Hkv + s.h) * p.max_tokens;
      // A token's page, then its key's scale and its score so far, are loaded two tiles and one tile ahead of their use.
      auto token_of = [&](int t) { return t * kPairTile + pr * kTile + mine; };
      auto load_page = [&](int t) {
        const int tok = token_of(t);
        return t < s.t1 && tok < s.len ? __ldg(table + page_of(a, tok)) : -1;
      };
      const bool again = s.c > 0, old = again || !fresh;
      const float decay = again ? 1.f : p.decay;
      float key_scale = 1.f, before = 0.f;
      auto load_token = [&](int t, int page) {
        const int tok = token_of(t);
        key_scale = 1.f;
        before = 0.f;
        if (page < 0 || page >= c.pages) return;
        if constexpr (kE4m3) key_scale = __ldg(c.k_scale + ((size_t)page * c.Hkv + s.h) * c.page + tok - page_of(a, tok) * c.page);
        if (t % kGroups == warp >> 2 && old && (again || tok < s.ctx)) before = out[tok];
      };
      int page = load_page(s.t0), next_page = load_page(s.t0 + 1);
      // The segment's query rows, once the MMAs of the one before are through. (Whoever gives up a wait goes on without
      // effect: no warp is missing at a barrier of several.)
      wait_warp(&B->q_empty, (seg & 1) ^ 1, abort);
      load_queries<D, kE4m3>(a, s, rest, B, seg, warp, pr);
      asm volatile("fence.proxy.async;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_both(&B->q_full[b2]);
      load_token(s.t0, page);
      wait_cluster(&B->q_full[b2], (seg >> 1) & 1, abort);
      __syncwarp();
      // rows that add nothing or have factors of their own: the way of masked tiles for all of them
      const bool dead = __any_sync(0xffffffffu, lane < kLoaders && *(volatile int*)&B->dead[b2][lane % kLoaders] != 0) ||
                        *(volatile int*)&B->uneven[b2][g] != 0;
      const float f0 = *(volatile float*)&B->factor[b2][g];
      const float* lse_h = reinterpret_cast<const float*>(rest + C::oLse) + (b2 * 2 + g) * kHalf + 2 * a4;
      const float* own_h = reinterpret_cast<const float*>(rest + C::oOwn) + (b2 * 2 + g) * kHalf + 2 * a4;
      const uint32_t* sees_h = reinterpret_cast<const uint32_t*>(rest + C::oSees) + b2 * 3 * 2 * kHalf + g * kHalf + 2 * a4;
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        const int this_page = page;
        const float ks = key_scale, w = before;
        page = next_page;
        next_page = load_page(t + 2);
        load_token(t + 1, page);
        const int tok = token_of(t), node0 = tok - 8 * a4 - s.ctx;
        const bool masked = dead || t * kPairTile + (pr + 1) * kTile > s.ctx;
        uint32_t context = 0;  // bit 8 k: token k is one of the context
        float f[4], sum[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          context |= node0 + 8 * k < 0 ? 1u << (8 * k) : 0u;
          f[k] = kE4m3 ? f0 * __shfl_sync(0xffffffffu, ks, (lane & ~3) | k) : f0;
          sum[k][0] = sum[k][1] = 0.f;
        }
        for (int sub = 0; sub < rows.steps; ++sub, ++step) {
          const int b = step & 1;
          const float* lse = lse_h + sub * rows.hs;
          // rows of this step's that there are, and of those the group's
          const int half = max(0, min(rows.hs, all - (2 * sub + g) * rows.hs)), mid = (half + 31) / 32 * 16;
          const int from = part ? mid : 0, here = part ? half : min(mid, half);
          // Sixteen rows at a time, their scores and constants loaded while the sixteen before are worked on. (With 32, or
          // with all constants in registers, the compiler has too few left to let the chains of several rows run side by
          // side: 96 rows of a tile took 1.45 us with 32, 0.8 with 16.)
          auto constants = [&](int r0, float2 (&l)[2]) {
            l[0] = *reinterpret_cast<const float2*>(lse + min(r0, kHalf - 8));
            l[1] = *reinterpret_cast<const float2*>(lse + min(r0 + 8, kHalf - 8));
          };
          // all rows there and seen by all tokens
          auto whole = [&](const Scores& u, const float2 (&l)[2]) {
            float x[2][4][2];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                x[q][k][0] = fmaf(u.at(q, k, 0), f[k], l[q].x);
                x[q][k][1] = fmaf(u.at(q, k, 1), f[k], l[q].y);
              }
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int y = 0; y < 2; ++y) x[q][k][y] = ex2(x[q][k][y]);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int y = 0; y < 2; ++y) sum[k][y] += x[q][k][y];
          };
          // rows behind the last and nodes that a row does not see: by selection, whatever the score is
          auto some = [&](const Scores& u, const float2 (&l)[2], int r0) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int r = r0 + 8 * q;
              uint32_t see[2] = {~0u, ~0u};
              float2 own = make_float2(1.f, 1.f);
              if (masked) {
                if constexpr (kE4m3) own = *reinterpret_cast<const float2*>(own_h + min(sub * rows.hs + r, kHalf - 8));
                const uint32_t* at = sees_h + min(sub * rows.hs + r, kHalf - 8);
                const uint2 w0 = *reinterpret_cast<const uint2*>(at), w1 = *reinterpret_cast<const uint2*>(at + 2 * kHalf),
                            live = *reinterpret_cast<const uint2*>(at + 4 * kHalf);
                auto nodes = [&](uint32_t x, uint32_t y) {
                  const uint64_t m = (uint64_t)y << 32 | x;
                  return (uint32_t)(node0 >= 64 || node0 <= -64 ? 0ull : node0 >= 0 ? m >> node0 : m << -node0);
                };
                see[0] = nodes(w0.x, w1.x) | (live.x ? context : 0u);
                see[1] = nodes(w0.y, w1.y) | (live.y ? context : 0u);
              }
              if (r + 2 * a4 >= here) see[0] = 0u;
              if (r + 2 * a4 + 1 >= here) see[1] = 0u;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float x = ex2(fmaf(u.at(q, k, 0), f[k] * own.x, l[q].x)),
                            y = ex2(fmaf(u.at(q, k, 1), f[k] * own.y, l[q].y));
                sum[k][0] += (see[0] >> (8 * k)) & 1u ? x : 0.f;
                sum[k][1] += (see[1] >> (8 * k)) & 1u ? y : 0.f;
              }
            }
          };
          auto work = [&](const Scores& u, const float2 (&l)[2], int r0) {
            if (!masked && r0 + 16 <= here) whole(u, l);
            else some(u, l, r0);
          };
          float2 lu[2], lv[2];
          constants(from, lu);
          constants(from + 16, lv);
          wait_warp(&B->s_full[b], (step >> 1) & 1, abort);
          umma::fence_after_sync();
          const uint32_t ts = umma::taddr(tmem, 32 * w4, b * kColsBuf + g * rows.hs);
          Scores u, v;
          if (from < here) u.load(ts + from);
#pragma unroll 1
          for (int r0 = from; r0 < here; r0 += 32) {
            u.wait();
            if (r0 + 16 < here) v.load(ts + r0 + 16);
            work(u, lu, r0);
            if (r0 + 16 < here) {
              constants(r0 + 32, lu);
              v.wait();
              if (r0 + 32 < here) u.load(ts + r0 + 32);
              work(v, lv, r0 + 16);
              constants(r0 + 48, lv);
            }
          }
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) arrive_cluster(cluster_addr(&B->s_empty[b], 0));
        }
        // the four lanes' parts of their four tokens: after two exchanges each lane has its own token's
        float mix[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mix[k] = sum[k][0] + sum[k][1];
        const bool up = a4 & 2, odd = a4 & 1;
        const float even_part = (up ? mix[2] : mix[0]) + __shfl_xor_sync(0xffffffffu, up ? mix[0] : mix[2], 2);
        const float odd_part = (up ? mix[3] : mix[1]) + __shfl_xor_sync(0xffffffffu, up ? mix[1] : mix[3], 2);
        float total = (odd ? odd_part : even_part) + __shfl_xor_sync(0xffffffffu, odd ? even_part : odd_part, 1);
        // The groups meet: the others' sums by way of shared memory to the one whose turn it is (by the tile, whatever the
        // chunk). They may be two steps ahead, since it has read a step's scores before the next but one's are made, so there
        // are sums and barriers for the tiles of that.
        float* all_sums = sums + tile % kSums * kGroups * kTile + mine;
        if (t % kGroups != warp >> 2) {
          all_sums[(warp >> 2) * kTile] = total;
          asm volatile("bar.arrive %0, %1;" ::"r"(2 + tile % kSums), "n"(32 * kLoaders) : "memory");
          continue;
        }
        asm volatile("bar.sync %0, %1;" ::"r"(2 + tile % kSums), "n"(32 * kLoaders) : "memory");
#pragma unroll
        for (int k = 1; k < kGroups; ++k) total += all_sums[((warp >> 2) + k) % kGroups * kTile];
        if (tok < s.len && !*(volatile int*)abort) {
          if (this_page < 0 || this_page >= c.pages) report(p.dev_err, GDN_DEVERR_SLOT);
          else out[tok] = fmaf(w, decay, total);
        }
      }
      ++seg;
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  // neither CTA leaves while the other may still copy into it, read its shared memory in an MMA, or arrive on its barriers
  cluster_sync_all();
  umma::fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem, 512);
  if (tid == 0 && *(volatile int*)abort) report(p.dev_err, GDN_DEVERR_TIMEOUT);
}

template <int D, bool kE4m3>
cudaError_t launch(const Args& a, const CUtensorMap& tmk, cudaStream_t stream) {
  using C = Cfg<D, kE4m3>;
  constexpr int kSmem = C::kStages * (int)kBlock + C::kRest;
  const void* fn = reinterpret_cast<const void*>(&pair_kernel<D, kE4m3>);
  const cudaError_t err = ensure_dynamic_smem(fn, kSmem);
  if (err != cudaSuccess) return err;
  const int pairs = resident_clusters(fn, kThreads, kSmem, 2);
  if (pairs <= 0) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pair_kernel<D, kE4m3>, a, tmk);
}

}  // namespace

cudaError_t launch_pairs(Args a, const CUtensorMap& tmk, int D, cudaStream_t stream) {
  const int all = a.p.P * a.p.G;
  a.chunks = (all + 2 * kHalf - 1) / (2 * kHalf);
  a.rows = (all + a.chunks - 1) / a.chunks;
  a.chunks = (all + a.rows - 1) / a.rows;
  a.sub = kSubBytes / (kTile * D * (a.c.e4m3 ? 1 : 2));
  a.cost = 2;
  if (D == 256) return a.c.e4m3 ? launch<256, true>(a, tmk, stream) : launch<256, false>(a, tmk, stream);
  return a.c.e4m3 ? launch<128, true>(a, tmk, stream) : launch<128, false>(a, tmk, stream);
}

}  // namespace kv_score
}  // namespace gdn
