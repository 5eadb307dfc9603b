// kv_score.cuh - what the two kernels behind gdn_kv_score share (kv_score.cu: up to 64 query rows a kv head, a CTA by
// itself; kv_score_pair.cu: more, in CTA pairs): the line of tiles and its cut, and small helpers.
#pragma once

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

struct Args {
  ScoreArgs p;
  KvArgs c;
  int rows, chunks;  // rows of a chunk (the last one may have fewer)
  int box;           // tokens per TMA box
  int sub;           // tiles that several chunks go through in turn
  int cost;          // what a unit takes beside its tiles, in tiles
  int shift;         // the page's tokens as a power of two, or -1
};

// Page of a request's table that has token `tok`. (A division for every token of a tile takes a good part of its time.)
__device__ __forceinline__ int page_of(const Args& a, int tok) { return a.shift >= 0 ? tok >> a.shift : tok / a.c.page; }

struct Plan {
  long long lo;
  int count, n, h, t;  // t: where the piece begins in the unit, whose first `cost` places hold no tile
};

// What the roles go through: tiles t0 .. t1 - 1 of (request n, kv head h) with the rows of chunk c. `at`: the number of
// tiles before t0 in the piece, each counted once.
struct Seg {
  int n, h, c, t0, t1, len, ctx, at;
};

// The tiles (of kTokens) of a request; none where it is a padding request or breaks the limits.
template <int kTokens>
__device__ __forceinline__ int tiles_of(const Args& a, int n, int* why = nullptr) {
  const ScoreArgs& p = a.p;
  const int ctx = __ldg(p.ctx + n), slot = __ldg(p.slot + n);
  if (ctx < 0 || slot < 0) return 0;
  const long long len = (long long)ctx + p.P;
  int bad = slot >= p.Rs ? GDN_DEVERR_SLOT : 0;
  if ((len + a.c.page - 1) / a.c.page > p.max_pages || len > p.max_tokens) bad |= GDN_DEVERR_OFFSETS;
  if (why) *why |= bad;
  return bad ? 0 : (int)((len + kTokens - 1) / kTokens);
}

template <int kTokens>
struct Walk {
  int n, h, t, left, tiles, at;
  Seg cur;
  __device__ __forceinline__ Walk(const Args& a, const Plan& p) : n(p.n), h(p.h), t(p.t), left(p.count), tiles(0), at(0) {
    cur.c = a.chunks;  // none
    if (left > 0) tiles = tiles_of<kTokens>(a, n);
  }
  __device__ __forceinline__ bool next(const Args& a, Seg& s) {
    if (cur.c + 1 < a.chunks) {
      ++cur.c;
      s = cur;
      return true;
    }
    while (left > 0) {
      while (tiles == 0) tiles = tiles_of<kTokens>(a, ++n);  // the piece has places left, so a request with some follows
      const int places = tiles + a.cost;
      int take = min(places - t, left);
      if (a.chunks > 1) take = min(take, max(a.cost - t, 0) + a.sub);
      const int ctx = __ldg(a.p.ctx + n);
      cur = Seg{n, h, 0, max(t - a.cost, 0), t + take - a.cost, ctx + a.p.P, ctx, at};
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

// An E4M3 cache's query rows are scaled by powers of two before they are taken apart into two terms: by one, `up`, that
// takes the largest value of all (`most`, a bf16's bits) below 256, so that one factor does for all scores; but a row whose
// own largest is more than two powers below has one of its own, and its scores a factor 2^(up - own) beside it.
__device__ __forceinline__ int power_of(uint32_t most) { return most == 0 ? 0 : min(134 - (int)(most >> 7), 120); }
__device__ __forceinline__ bool smaller(uint32_t row, uint32_t most) { return row > 0 && (row >> 7) + 2 < (most >> 7); }
__device__ __forceinline__ int power_of(uint32_t row, uint32_t most) {
  const int up = power_of(most);
  return smaller(row, most) ? min(power_of(row), up + 126) : up;
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Piece `index` of `pieces`: a scan over the requests' tiles by all threads of the block, `totals` a word a warp. The plan is
// there after the next barrier.
template <int kTokens, int kThreads>
__device__ __forceinline__ void make_plan(const Args& a, int index, int pieces, long long* totals, Plan* plan) {
  const ScoreArgs& p = a.p;
  const KvArgs& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.N + kThreads - 1) / kThreads, n0 = min(p.N, tid * per), n1 = min(p.N, n0 + per);
  long long mine = 0;
  int why = 0;
  for (int n = n0; n < n1; ++n) {
    const int tiles = tiles_of<kTokens>(a, n, &why);
    mine += tiles + (tiles > 0 ? a.cost : 0);
  }
  if (why && index == 0) report(p.dev_err, why);
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) totals[warp] = upto;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += totals[w];
    total += totals[w];
  }
  before += upto - mine;
  total *= c.Hkv;
  const long long with = min((long long)pieces, total);  // with a piece: none of them empty
  const long long lo = with ? total * index / with : 0, hi = with ? total * (index + 1) / with : 0;
  if (index < with && before * c.Hkv <= lo && lo < (before + mine) * c.Hkv) {
    long long at = before * c.Hkv;
    for (int n = n0; n < n1; ++n) {
      const int tiles = tiles_of<kTokens>(a, n), places = tiles + (tiles > 0 ? a.cost : 0);
      const long long here = (long long)places * c.Hkv;
      if (lo < at + here) {
        *plan = Plan{lo, (int)(hi - lo), n, (int)((lo - at) / places), (int)((lo - at) % places)};
        break;
      }
      at += here;
    }
  }
}

cudaError_t launch_pairs(Args a, const CUtensorMap& tmk, int D, cudaStream_t stream);

}  // namespace kv_score
}  // namespace gdn
