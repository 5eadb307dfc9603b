// kv_evict.cu - gdn_kv_evict: a request's cache cut down to its budget of tokens, per kv head those of the largest
// accumulated weight (gdn_kv_score), the first and the last ones always among them.
//
// Two kernels, one after the other on the stream:
//   select: per (request, kv head) the m-th largest weight by radix, 11 bits a pass from the top, and the indices of the
//           kept tokens in ascending order. Weights that are equal at the border go to the lowest indices.
//   move:   the kept tokens' keys, values, scales and weights, in the order of the tokens, to other pages (copy_kernel) or
//           to the front of the request's own (shift_kernel).
// Every kernel here may begin before the one in front of it ends, so what that one writes (the weights; the new lengths and
// the kept indices) is read by plain loads: read-only ones are for memory that nobody writes while the kernel is there.
#include <algorithm>

#include "device.cuh"
#include "launch.h"

namespace gdn {

namespace {

// ---------------------------------------------------------------- select

constexpr int kFew = 128;  // weights at the border that are put in order all at once

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// A 32-bit word of another CTA's shared memory, at the place of `mine` in this one's.
__device__ __forceinline__ int load_remote(const int* mine, uint32_t rank) {
  uint32_t addr;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int4 load_remote4(const int* mine, uint32_t rank) {
  uint32_t addr;
  int4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// The limits of request n: how many tokens it keeps, -1 if none are to be touched (a padding request, *why 0, or one
// that breaks a limit).
__device__ __forceinline__ int kept_of(const EvictArgs& p, const KvArgs& c, int n, int* why) {
  const int len = __ldg(p.len + n), slot = __ldg(p.slot + n), dst = __ldg(p.dst_slot + n), budget = __ldg(p.budget + n);
  const int m = min(len, budget);
  *why = 0;
  if (len < 0 || slot < 0) return -1;
  if (slot >= p.Rs || dst < 0 || dst >= p.Rs) *why |= GDN_DEVERR_SLOT;
  if (budget < 0 || m > p.max_kept || len > p.max_tokens || (len - 1) / c.page >= p.max_pages ||
      (m > 0 && (m - 1) / c.page >= p.dst_max_pages))
    *why |= GDN_DEVERR_OFFSETS;
  return *why ? -1 : m;
}

// Weights in their order as unsigned numbers: NaN lowest, -0 and 0 alike, below what is always kept.
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// kSplit CTAs, a cluster, have a (request, kv head), each an equal run of its tokens; a thread has kHeld of them at a
// time, and a CTA whose tokens are no more than its threads hold reads their weights once (else again, from L2, in each of
// the passes). A pass counts the keys with the border's upper bits by their next kBits. After two passes (after one of a
// short request) few have all the bits so far, as a rule: those are put in order at once, by counting for each the larger
// ones.
// Bound by the chain of loads, barriers and exchanges between the CTAs: of the 17 us that a CTA of eight takes for its part
// of 131071 tokens of four heads (floor, 2 MB: 0.3 us), 3.7 are the first loads, 3.3 and 3.5 the passes, 3 the few, 2.9 the
// kept indices. (With 8 bits a pass in 32 histograms, a lane's own each, a pass took 4.5 us, and one more was needed.)
template <int kSplit, int kHeld, int kThreads, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm) select_kernel(const EvictArgs p, const KvArgs c) {
  constexpr int kWarps = kThreads / 32, kBatch = kThreads * kHeld;
  constexpr int kBits = kThreads == 512 ? 11 : 10, kBins = 1 << kBits;
  __shared__ __align__(16) int hist[2][kBins];           // of two passes in turn: the others' CTAs read the one before
  __shared__ int above_s[kWarps];
  __shared__ int2 scan_s[2][kWarps];
  __shared__ int pick[3];                                // the bin of the m-th largest, those above it, and in it
  __shared__ __align__(16) uint32_t few_s[kFew];
  __shared__ uint32_t own_few_s[kFew];
  __shared__ int few[2], border_s[2];                    // few: of this CTA, those in the bin and those above it
  __shared__ int totals[2];                              // of this CTA: weights above the border, and equal to it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long unit = blockIdx.x / kSplit;
  const int n = (int)(unit / c.Hkv), h = (int)(unit % c.Hkv);
  const int rank = kSplit > 1 ? (int)cluster_rank() : 0;
  int why;
  const int m = kept_of(p, c, n, &why);
  const int len = __ldg(p.len + n);
  // this CTA's run of tokens
  const int per = ((max(len, 0) + kSplit - 1) / kSplit + 31) / 32 * 32;
  const int lo = min(len, rank * per), count = min(len, lo + per) - lo;
  const bool sift = m > 0 && m < len;
  const float* w = p.score;
  if (sift) w += ((size_t)__ldg(p.slot + n) * c.Hkv + h) * p.max_tokens + lo;
  const int last = len - min(p.recent, max(len, 0));  // the first of the last tokens
  // A warp has an equal run of these, or as many as it holds; a lane every 32nd of it.
  const bool held = count <= kBatch;
  const int run = held ? ((count + kWarps - 1) / kWarps + 31) / 32 * 32 : 32 * kHeld;
  uint32_t key[kHeld];
  int valid = 0;  // of this thread's tokens
  auto load = [&](int base) {
    const int i = base + warp * run + lane;
    valid = max(0, (min(count - base - warp * run, run) - lane + 31) >> 5);
    float x[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) x[j] = j < valid ? w[i + 32 * j] : 0.f;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int t = lo + i + 32 * j;
      key[j] = t < p.sinks || t >= last ? 0xffffffffu : key_of(x[j]);
    }
  };
  if (sift && held) load(0);
#pragma unroll
  for (int i = tid; i < 2 * kBins / 4; i += kThreads) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
  if (tid < 2) few[tid] = 0;
  bool bad = false;
  if (m >= 0) {
#pragma unroll 4
    for (int i = tid; (long long)i * c.page < len; i += kThreads) {
      const int page = __ldg(p.table + (size_t)n * p.max_pages + i);
      bad |= page < 0 || page >= c.pages;
    }
#pragma unroll 4
    for (int i = tid; (long long)i * c.page < m; i += kThreads) {
      const int page = __ldg(p.dst_table + (size_t)n * p.dst_max_pages + i);
      bad |= page < 0 || page >= c.pages;
    }
  }
  if (__syncthreads_or(bad)) why |= GDN_DEVERR_SLOT;
  if (h == 0 && rank == 0 && tid == 0) {
    if (why) report(p.dev_err, why);
    if (why) p.new_len[n] = -1;
    else if (m >= 0) p.new_len[n] = m;
  }
  if (m <= 0 || why) return;  // the same in the whole cluster
  int* kept = p.kept + ((size_t)n * c.Hkv + h) * p.max_kept;
  if (!sift) {
    for (int i = tid; i < count; i += kThreads) kept[lo + i] = lo + i;
    return;
  }
  auto batches = [&](auto work) {
    if (held) {
      work();
    } else {
      for (int base = 0; base < count; base += kBatch) {
        load(base);
        work();
      }
    }
  };

  uint32_t border = 0;  // the key of the m-th largest, from the top
  int need = m;         // how many of those with its upper bits
  int over_before = 0, equal_before = 0;  // keys above the border, and at it, in the CTAs before this one
  bool counted = false;
  for (int pass = 0, top = 32; top > 0; ++pass) {
    const int width = min(top, kBits), shift = top - width;
    top = shift;
    int* bins = hist[pass & 1];
    if (pass >= 2) {
      for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<int4*>(bins)[i] = make_int4(0, 0, 0, 0);
      __syncthreads();
    }
    batches([&] {
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        if (j < valid && (pass == 0 || ((key[j] ^ border) >> (shift + width)) == 0))
          atomicAdd(&bins[key[j] >> shift & ((1u << width) - 1)], 1);
    });
    if constexpr (kSplit > 1) cluster_sync();
    else __syncthreads();
    // this thread's four bins, and the keys in higher ones: a scan from the top
    static_assert(kBins == 4 * kThreads, "four bins a thread");
    int4 mine = reinterpret_cast<const int4*>(bins)[tid];
    if constexpr (kSplit > 1) {
      int4 theirs[kSplit - 1];
#pragma unroll
      for (int r = 1; r < kSplit; ++r) theirs[r - 1] = load_remote4(bins + 4 * tid, (rank + r) % kSplit);
#pragma unroll
      for (int r = 0; r < kSplit - 1; ++r) {
        mine.x += theirs[r].x;
        mine.y += theirs[r].y;
        mine.z += theirs[r].z;
        mine.w += theirs[r].w;
      }
    }
    const int sum = mine.x + mine.y + mine.z + mine.w;
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_down_sync(0xffffffffu, upto, d);
      if (lane + d < 32) upto += o;
    }
    if (lane == 0) above_s[warp] = upto;
    __syncthreads();
    int above = upto - sum + __reduce_add_sync(0xffffffffu, lane > warp && lane < kWarps ? above_s[lane] : 0);
    if (above < need && above + sum >= need) {
      const int in[4] = {mine.x, mine.y, mine.z, mine.w};
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        if (above < need && above + in[i] >= need) pick[0] = 4 * tid + i, pick[1] = above, pick[2] = in[i];
        above += in[i];
      }
    }
    __syncthreads();
    border |= (uint32_t)pick[0] << shift;
    need -= pick[1];
    const int in_bin = pick[2];
    if (shift > 0 && in_bin <= kFew) {
      uint32_t* own = kSplit > 1 ? own_few_s : few_s;
      batches([&] {
        uint32_t in = 0;
        int over = 0;
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
          in |= (j < valid && key[j] >> shift == border >> shift ? 1u : 0u) << j;
          if (kSplit > 1) over += j < valid && key[j] >> shift > border >> shift;
        }
        int upto = __popc(in);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += o;
        }
        if (kSplit > 1) over = __reduce_add_sync(0xffffffffu, over);
        int at = 0;
        if (lane == 31 && upto > 0) at = atomicAdd(&few[0], upto);
        if (kSplit > 1 && lane == 0 && over > 0) atomicAdd(&few[1], over);
        at = __shfl_sync(0xffffffffu, at, 31) + upto - __popc(in);
        if (in) {
#pragma unroll
          for (int j = 0; j < kHeld; ++j)
            if (in >> j & 1) own[at++] = key[j];
        }
      });
      int before = 0;  // keys of the CTAs before this one in few_s
      if constexpr (kSplit > 1) {  // every CTA's, one after the other
        cluster_sync();
        const int theirs = lane < kSplit ? load_remote(&few[0], lane) : 0;
        over_before = lane < rank ? load_remote(&few[1], lane) : 0;
        int upto = theirs;
#pragma unroll
        for (int d = 1; d < kSplit; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += o;
        }
        int r = 0, first = 0;
#pragma unroll
        for (int x = 0; x < kSplit - 1; ++x) {
          const int end = __shfl_sync(0xffffffffu, upto, x);
          if (tid >= end) r = x + 1, first = end;
        }
        static_assert(kFew <= kThreads, "a key a thread");
        if (tid < in_bin) few_s[tid] = (uint32_t)load_remote(reinterpret_cast<const int*>(own_few_s) + tid - first, r);
        before = __shfl_sync(0xffffffffu, upto - theirs, rank);
        over_before = __reduce_add_sync(0xffffffffu, over_before);
      }
      if (tid >= in_bin && tid < (in_bin + 3) / 4 * 4) few_s[tid] = 0;  // counted as the least of them
      __syncthreads();
      if constexpr (kSplit > 1) cluster_arrive();  // the others' have been read
      if (tid < in_bin) {
        const uint32_t mine_key = few_s[tid];
        int above = 0, reach = 0;  // larger ones, and those as large too
#pragma unroll 4
        for (int i = 0; i < in_bin; i += 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(few_s + i);
          above += (x.x > mine_key) + (x.y > mine_key) + (x.z > mine_key) + (x.w > mine_key);
          reach += (x.x >= mine_key) + (x.y >= mine_key) + (x.z >= mine_key) + (x.w >= mine_key);
        }
        if (above < need && reach >= need) border_s[0] = (int)mine_key, border_s[1] = need - above;
      }
      __syncthreads();
      border = (uint32_t)border_s[0];
      need = border_s[1];
      if constexpr (kSplit > 1) {
        int over = 0;
        for (int i = lane; i < before; i += 32) {
          over += few_s[i] > border;
          equal_before += few_s[i] == border;
        }
        over_before += __reduce_add_sync(0xffffffffu, over);
        equal_before = __reduce_add_sync(0xffffffffu, equal_before);
        counted = true;
      }
      break;
    }
  }

  // ---- the kept tokens' indices: those above the border, and the first `need` of those at it
  if (kSplit > 1 && !counted) {  // the numbers of both in the CTAs before this one
    if (tid < 2) totals[tid] = 0;
    __syncthreads();
    int over = 0, equal = 0;
    batches([&] {
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        over += j < valid && key[j] > border;
        equal += j < valid && key[j] == border;
      }
    });
    over = __reduce_add_sync(0xffffffffu, over);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
      atomicAdd(&totals[0], over);
      atomicAdd(&totals[1], equal);
    }
    cluster_sync();
    if (lane < rank) {
      over_before = load_remote(&totals[0], lane);
      equal_before = load_remote(&totals[1], lane);
    }
    over_before = __reduce_add_sync(0xffffffffu, over_before);
    equal_before = __reduce_add_sync(0xffffffffu, equal_before);
    cluster_arrive();
  }
  int buf = 0, base = 0;
  const uint32_t lower = (1u << lane) - 1u;
  batches([&] {
    int over = 0, equal = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      over += j < valid && key[j] > border;
      equal += j < valid && key[j] == border;
    }
    over = __reduce_add_sync(0xffffffffu, over);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) scan_s[buf][warp] = make_int2(over, equal);
    __syncthreads();
    const int2 theirs = lane < kWarps ? scan_s[buf][lane] : make_int2(0, 0);
    int o = over_before + __reduce_add_sync(0xffffffffu, lane < warp ? theirs.x : 0);
    int e = equal_before + __reduce_add_sync(0xffffffffu, lane < warp ? theirs.y : 0);
    int* to = kept + min(e, need);
    const int first = lo + base + warp * run + lane;
    if (equal == 0) {  // as a rule
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const bool is_over = j < valid && key[j] > border;
        const uint32_t overs = __ballot_sync(0xffffffffu, is_over);
        if (is_over) to[o + __popc(overs & lower)] = first + 32 * j;
        o += __popc(overs);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const bool is_over = j < valid && key[j] > border, is_equal = j < valid && key[j] == border;
        const uint32_t overs = __ballot_sync(0xffffffffu, is_over), equals = __ballot_sync(0xffffffffu, is_equal);
        const int mine = e + __popc(equals & lower);
        if (is_over || (is_equal && mine < need)) kept[o + __popc(overs & lower) + min(mine, need)] = first + 32 * j;
        o += __popc(overs);
        e += __popc(equals);
      }
    }
    over_before += __reduce_add_sync(0xffffffffu, theirs.x);
    equal_before += __reduce_add_sync(0xffffffffu, theirs.y);
    base += kBatch;
    buf ^= 1;
  });
  if constexpr (kSplit > 1) cluster_wait();  // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------- move

constexpr int kMoveThreads = 512;
constexpr int kUnroll = 8;

// Rows of the pool: of the page's first head and token, and of a token.
struct Rows {
  const int32_t* table;
  int h, shift;  // shift: the page's tokens as a power of two, or -1
  __device__ __forceinline__ int at(const KvArgs& c, int i) const {
    const int k = shift >= 0 ? i >> shift : i / c.page;
    return (__ldg(table + k) * c.Hkv + h) * c.page + (i - k * c.page);
  }
};

// To other pages: nothing that is read is written, so the kept tokens of all (request, kv head) units stand in one line of
// segments, cut into equal pieces, one per block. A segment is kUnroll pieces of 16 bytes a thread, of keys and values;
// where its tokens come from and go to is found once per token, a segment ahead, in shared memory.
// Bound by HBM: its reads and writes in turn, 64 KB on their way in each of two blocks an SM. 32 requests of 2k .. 32k
// tokens, E4M3, cut to half, 750 MB, 117 us; one of 131071 to a quarter, bf16, 272 MB, 42 us: 95 % of the copy bandwidth.
template <int kRowBytes>
__global__ void __launch_bounds__(kMoveThreads, 2) copy_kernel(const EvictArgs p, const KvArgs c, int shift) {
  constexpr int kPieces = kRowBytes / 16, kTokens = kMoveThreads * kUnroll / (2 * kPieces);
  static_assert(kTokens <= kMoveThreads, "a thread per token");
  __shared__ int2 place[2][kTokens];  // rows of the pool: from, to
  __shared__ long long warp_total[kMoveThreads / 32];
  __shared__ struct {
    long long left;
    int n, h, s;
  } plan;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto tokens_of = [&](int n) {
    const int m = __ldg(p.len + n) < 0 || __ldg(p.slot + n) < 0 ? 0 : p.new_len[n];
    return max(m, 0);
  };
  auto segments_of = [&](int n) { return (tokens_of(n) + kTokens - 1) / kTokens; };
  // ---- this block's piece: a scan over the requests' segments
  {
    if (tid == 0) plan.left = 0;
    const int per = (p.N + kMoveThreads - 1) / kMoveThreads, n0 = min(p.N, tid * per), n1 = min(p.N, n0 + per);
    long long mine = 0;
    for (int n = n0; n < n1; ++n) mine += segments_of(n);
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 31) warp_total[warp] = upto;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < kMoveThreads / 32; ++w) {
      if (w < warp) before += warp_total[w];
      total += warp_total[w];
    }
    before = (before + upto - mine) * c.Hkv;
    total *= c.Hkv;
    const long long lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
    if (hi > lo && before <= lo && lo < before + mine * c.Hkv) {
      long long at = before;
      for (int n = n0; n < n1; ++n) {
        const long long segs = segments_of(n), here = segs * c.Hkv;
        if (lo < at + here) {
          plan.left = hi - lo;
          plan.n = n;
          plan.h = (int)((lo - at) / segs);
          plan.s = (int)((lo - at) % segs);
          break;
        }
        at += here;
      }
    }
    __syncthreads();
  }
  long long left = plan.left;
  if (left == 0) return;
  // the segment whose places are looked up: request, head, first token, and the request's tokens
  int n = plan.n, h = plan.h, s = plan.s, m = tokens_of(n);
  struct Seg {
    int n, h, first, count;
  };
  auto next = [&](Seg& x) {
    if (left == 0) return false;
    while (s * kTokens >= m) {  // the unit is through; the piece has segments left, so one follows
      s = 0;
      if (++h == c.Hkv) {
        h = 0;
        do m = tokens_of(++n);
        while (m == 0);
      }
    }
    x = Seg{n, h, s * kTokens, min(kTokens, m - s * kTokens)};
    ++s;
    --left;
    return true;
  };
  auto index_of = [&](const Seg& x) {
    return tid < x.count ? p.kept[((size_t)x.n * c.Hkv + x.h) * p.max_kept + x.first + tid] : -1;
  };
  auto look_up = [&](const Seg& x, int index) {
    if (tid >= x.count) return make_int2(-1, -1);
    const Rows from{p.table + (size_t)x.n * p.max_pages, x.h, shift}, to{p.dst_table + (size_t)x.n * p.dst_max_pages, x.h, shift};
    return make_int2(from.at(c, index), to.at(c, x.first + tid));
  };
  Seg cur, after;
  next(cur);
  int index = index_of(cur);
  int2 mine = look_up(cur, index);
  if (tid < kTokens) place[0][tid] = mine;
  bool more = next(after);
  int next_index = more ? index_of(after) : -1;
  const uint4* k = static_cast<const uint4*>(c.k);
  const uint4* v = static_cast<const uint4*>(c.v);
  for (int b = 0;; b ^= 1) {
    __syncthreads();
    // a warp's pieces are of one token's keys or values, or of several of the one
    uint4 held[kUnroll];
    const int piece = tid % kPieces, part = tid / kPieces;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int x = part + u * (kMoveThreads / kPieces), t = x >> 1;
      if (t < cur.count) held[u] = __ldcs((x & 1 ? v : k) + (size_t)place[b][t].x * kPieces + piece);
    }
    float ks = 0.f, vs = 0.f, w = 0.f;
    if (tid < cur.count) {
      if (c.e4m3) {
        ks = __ldcs(c.k_scale + mine.x);
        vs = __ldcs(c.v_scale + mine.x);
      }
      w = __ldcs(p.score + ((size_t)__ldg(p.slot + cur.n) * c.Hkv + cur.h) * p.max_tokens + index);
    }
    // the next segment's places, and the one's after it indices
    const Seg now = cur;
    const int2 here = mine;
    const bool go_on = more;
    if (more) {
      cur = after;
      index = next_index;
      mine = look_up(cur, index);
      if (tid < kTokens) place[b ^ 1][tid] = mine;
      more = next(after);
      next_index = more ? index_of(after) : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int x = part + u * (kMoveThreads / kPieces), t = x >> 1;
      if (t < now.count)
        __stcs(static_cast<uint4*>(x & 1 ? c.v : c.k) + (size_t)place[b][t].y * kPieces + piece, held[u]);
    }
    if (tid < now.count) {
      if (c.e4m3) {
        __stcs(c.k_scale + here.y, ks);
        __stcs(c.v_scale + here.y, vs);
      }
      __stcs(p.score + ((size_t)__ldg(p.dst_slot + now.n) * c.Hkv + now.h) * p.max_tokens + now.first + tid, w);
    }
    if (!go_on) break;
  }
}

// In place: kept token i has index kept[i] >= i, so a chunk of tokens is stored where only earlier chunks' tokens, or this
// one's, were read: a block takes its chunks in order and has read a chunk before it stores it. Blocks share no byte: a
// block has one head's keys or values, or a slice of their rows, or its floats.
// Bound by the chunks of a block coming one after the other: 32 requests of 8192 tokens, E4M3, cut to half, 550 MB, 110 us
// where copy_kernel takes 88.
//
// Tokens [first, m) of one head: `lanes` threads a token, each with one T; chunks of kShift tokens a thread. `row` finds
// the place that a token comes from, `from` and `to` give its address and that of the place that it goes to. A chunk is
// read while the one before it is stored: what it reads lies behind where that goes. Its places come a chunk ahead of
// that, its indices two.
template <typename T, int kShift, typename Row, typename From, typename To>
__device__ __forceinline__ void shift_rows(int first, int m, int lanes, const int* kept, Row row, From from, To to) {
  const int per = kMoveThreads / lanes, r = threadIdx.x / lanes, chunk = per * kShift;
  T even[kShift], odd[kShift];
  int place[kShift], index[kShift];
  auto indices = [&](int base) {
#pragma unroll
    for (int u = 0; u < kShift; ++u) {
      const int i = base + u * per + r;
      index[u] = i < m ? kept[i] : -1;
    }
  };
  auto places = [&] {
#pragma unroll
    for (int u = 0; u < kShift; ++u) place[u] = index[u] >= 0 ? row(index[u]) : -1;
  };
  auto read = [&](T (&held)[kShift]) {
#pragma unroll
    for (int u = 0; u < kShift; ++u)
      if (place[u] >= 0) held[u] = *from(place[u]);
  };
  auto step = [&](int base, T (&now)[kShift], T (&next)[kShift]) {
    read(next);
    places();
    indices(base + 3 * chunk);
    __syncthreads();  // the whole chunk has been read: a part of it is where it goes
#pragma unroll
    for (int u = 0; u < kShift; ++u) {
      const int i = base + u * per + r;
      if (i < m) *to(i) = now[u];
    }
  };
  indices(first);
  places();
  indices(first + chunk);
  read(even);
  places();
  indices(first + 2 * chunk);
  for (int base = first; base < m; base += 2 * chunk) {
    step(base, even, odd);
    if (base + chunk < m) step(base + chunk, odd, even);
  }
}

// A unit's parts: its keys' slices, its values' slices, and its floats (scales and weights).
template <int kShift>
__global__ void __launch_bounds__(kMoveThreads, kShift > 4 ? 1 : 2) shift_kernel(const EvictArgs p, const KvArgs c, int slices, int shift) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int parts = 2 * slices + 1;
  const long long unit = blockIdx.x / parts;
  const int part = (int)(blockIdx.x % parts);
  const int n = (int)(unit / c.Hkv), h = (int)(unit % c.Hkv);
  int why;
  const int m = kept_of(p, c, n, &why);
  if (m <= 0 || p.new_len[n] < 0) return;
  const int* kept = p.kept + ((size_t)n * c.Hkv + h) * p.max_kept;
  const Rows rows{p.table + (size_t)n * p.max_pages, h, shift};
  // the tokens in front of the first that is gone stay where they are
  int first = 0, hi = m;
  while (first < hi) {
    const int mid = (first + hi) >> 1;
    if (kept[mid] == mid) first = mid + 1;
    else hi = mid;
  }
  auto row = [&](int i) { return rows.at(c, i); };
  if (part < 2 * slices) {
    const int pieces = p.D * (c.e4m3 ? 1 : 2) / 16, lanes = pieces / slices;
    uint4* pool = static_cast<uint4*>(part < slices ? c.k : c.v) + (part % slices) * lanes + threadIdx.x % lanes;
    shift_rows<uint4, kShift>(first, m, lanes, kept, row, [&](int at) { return pool + (size_t)at * pieces; },
                      [&](int i) { return pool + (size_t)row(i) * pieces; });
  } else {
    if (c.e4m3) {
      shift_rows<float, kShift>(first, m, 1, kept, row, [&](int at) { return c.k_scale + at; },
                        [&](int i) { return c.k_scale + row(i); });
      shift_rows<float, kShift>(first, m, 1, kept, row, [&](int at) { return c.v_scale + at; },
                        [&](int i) { return c.v_scale + row(i); });
    }
    float* w = p.score + ((size_t)__ldg(p.slot + n) * c.Hkv + h) * p.max_tokens;
    shift_rows<float, kShift>(first, m, 1, kept, [](int i) { return i; }, [&](int at) { return w + at; },
                      [&](int i) { return w + i; });
  }
}

template <int kSplit, int kHeld, int kThreads, int kPerSm>
cudaError_t launch_select(const EvictArgs& a, const KvArgs& c, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.N * c.Hkv * kSplit), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSplit;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel<kSplit, kHeld, kThreads, kPerSm>, a, c);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, const KvArgs& c, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  const long long units = (long long)a.N * c.Hkv;
  const long long most = std::min<long long>((long long)a.max_pages * c.page, a.max_tokens);
  // As many CTAs a head as hold the longest request that the tables allow in registers, up to 131072 tokens. What a CTA takes
  // is a chain of steps, whatever its tokens, so of many heads the fewer CTAs the better, and four small ones an SM: with 4
  // x 512 threads of 16 tokens, two an SM, 32 requests of 2k .. 32k took 150 us, selection and copy, with 4 x 256 of 32 143,
  // with 8 x 256 of 16 158. (With 1 x 512 of 16, three an SM, 128 of 300 .. 8k took 193, with 1 x 256 of 32 195.)
  // The host knows the tables' width only. Where they, and the slots of scores, are much wider than the requests are long, the
  // heads get more and larger CTAs than their tokens need: with room for 131072 tokens a request, 32 of 2k .. 32k took 247 us
  // instead of 141, 128 of 300 .. 8k 958 instead of 191, one of 1000 18 instead of 10.
  err = most <= 2048    ? launch_select<1, 4, 512, 2>(a, c, stream)
        : most <= 8192  ? launch_select<1, 16, 512, 3>(a, c, stream)
        : most <= 16384 ? launch_select<2, 32, 256, 4>(a, c, stream)
        : most <= 32768 ? launch_select<4, 32, 256, 4>(a, c, stream)
        : most <= 65536 ? launch_select<8, 32, 256, 4>(a, c, stream)
                        : launch_select<8, 32, 512, 1>(a, c, stream);
  if (err != cudaSuccess) return err;
  const int row_bytes = a.D * (c.e4m3 ? 1 : 2);
  int shift = -1;
  if ((c.page & (c.page - 1)) == 0)
    for (shift = 0; 1 << shift < c.page;) ++shift;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMoveThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (a.dst_table != a.table) {
    cfg.gridDim = dim3((unsigned)(2 * sms), 1, 1);
    return row_bytes == 512   ? cudaLaunchKernelEx(&cfg, copy_kernel<512>, a, c, shift)
           : row_bytes == 256 ? cudaLaunchKernelEx(&cfg, copy_kernel<256>, a, c, shift)
                              : cudaLaunchKernelEx(&cfg, copy_kernel<128>, a, c, shift);
  }
  // slices of the rows, down to a sector, while there are too few blocks to keep HBM busy
  int slices = 1;
  while (row_bytes / slices > 32 && units * 2 * slices < 2 * sms) slices *= 2;
  const long long blocks = units * (2 * slices + 1);
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  // A block that has an SM's registers for itself takes chunks twice as long: one request of 65536 tokens, bf16, to half,
  // selection and shift, 123 us, with the short ones 148. (Where there are more blocks, 32 of 8192, E4M3, 161 and 131.)
  return blocks <= sms ? cudaLaunchKernelEx(&cfg, shift_kernel<8>, a, c, slices, shift)
                       : cudaLaunchKernelEx(&cfg, shift_kernel<4>, a, c, slices, shift);
}

}  // namespace gdn
