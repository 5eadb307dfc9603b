// kv_evict.cu - gdn_kv_evict: a request's cache cut down to its budget of tokens, per kv head those of the largest
// accumulated weight (gdn_kv_score), the first and the last ones always among them.
//
// Two kernels, one after the other on the stream:
//   select: per (request, kv head) the m-th largest weight by radix, 8 bits a pass from the top, and the indices of the
//           kept tokens in ascending order. Weights that are equal at the border go to the lowest indices.
//   move:   the kept tokens' keys, values, scales and weights to the front of the request's pages, or of other pages, in
//           the order of the tokens. Kept token i has index kept[i] >= i, so in place a chunk of tokens is stored where
//           only earlier chunks' tokens, or this one's, were read: a block takes its chunks in order and has read a
//           chunk before it stores it. Blocks share no byte: a block has one head's keys, values or floats, or a slice of
//           its rows.
#include "device.cuh"
#include "launch.h"

namespace gdn {

namespace {

// ---------------------------------------------------------------- select

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCached = 16384;  // tokens of a CTA whose keys stay in shared memory

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A 32-bit word of another CTA's shared memory, at the place of `mine` in this one's.
__device__ __forceinline__ int load_remote(const int* mine, uint32_t rank) {
  uint32_t addr;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The limits of request n: how many tokens it keeps, -1 if none are to be touched (a padding request, *why 0, or one
// that breaks a limit).
__device__ __forceinline__ int kept_of(const EvictArgs& p, const KvArgs& c, int n, int* why) {
  const int len = __ldg(p.len + n), slot = __ldg(p.slot + n);
  *why = 0;
  if (len < 0 || slot < 0) return -1;
  const int dst = __ldg(p.dst_slot + n), budget = __ldg(p.budget + n), m = min(len, budget);
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

// kSplit CTAs, a cluster, have a (request, kv head), each an equal run of its tokens.
template <int kSplit>
__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const EvictArgs p, const KvArgs c) {
  extern __shared__ uint32_t keys[];                 // [kCached]
  __shared__ int hist[256 * 32];                     // [bin][lane]: no two lanes of a warp at one bank
  __shared__ int bins[256], above_s[kSelWarps], scan_s[2][kSelWarps];
  __shared__ int pick[2];                            // the bin of the m-th largest, and those above it
  __shared__ int totals[2];                          // of this CTA: weights above the border, and equal to it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long unit = blockIdx.x / kSplit;
  const int n = (int)(unit / c.Hkv), h = (int)(unit % c.Hkv);
  const int rank = kSplit > 1 ? (int)cluster_rank() : 0;
  int why;
  const int m = kept_of(p, c, n, &why);
  const int len = __ldg(p.len + n);
  bool bad = false;
  if (m >= 0) {
    for (int i = tid; (long long)i * c.page < len; i += kSelThreads) {
      const int page = __ldg(p.table + (size_t)n * p.max_pages + i);
      bad |= page < 0 || page >= c.pages;
    }
    for (int i = tid; (long long)i * c.page < m; i += kSelThreads) {
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
  const int per = ((len + kSplit - 1) / kSplit + 31) / 32 * 32;
  const int lo = min(len, rank * per), count = min(len, lo + per) - lo;
  if (m == len) {
    for (int i = tid; i < count; i += kSelThreads) kept[lo + i] = lo + i;
    return;
  }
  const float* w = p.score + ((size_t)__ldg(p.slot + n) * c.Hkv + h) * p.max_tokens + lo;
  const int last = len - min(p.recent, len);  // the first of the last tokens
  auto load_key = [&](int i) { return lo + i < p.sinks || lo + i >= last ? 0xffffffffu : key_of(__ldg(w + i)); };
  const bool cached = count <= kCached;
  if (cached) {
#pragma unroll 4
    for (int i = tid; i < count; i += kSelThreads) keys[i] = load_key(i);
  }
  auto key_at = [&](int i) { return cached ? keys[i] : load_key(i); };

  uint32_t border = 0;  // the key of the m-th largest, from the top
  int need = m;         // how many of those with its upper bits
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256 * 32; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < count; i += kSelThreads) {
      const uint32_t k = key_at(i);
      if (shift == 24 || (k >> (shift + 8)) == (border >> (shift + 8))) atomicAdd(&hist[(k >> shift & 255u) * 32 + lane], 1);
    }
    __syncthreads();
    int mine = 0;
    if (tid < 256) {
#pragma unroll
      for (int i = 0; i < 32; ++i) mine += hist[tid * 32 + (i + lane) % 32];
      bins[tid] = mine;
    }
    if constexpr (kSplit > 1) {
      cluster_sync();
      if (tid < 256) {
#pragma unroll
        for (int r = 0; r < kSplit; ++r)
          if (r != rank) mine += load_remote(&bins[tid], r);
      }
    }
    // keys in higher bins: a scan from the top, thread t has bin t
    int upto = mine;
    if (tid < 256) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_down_sync(0xffffffffu, upto, d);
        if (lane + d < 32) upto += o;
      }
      if (lane == 0) above_s[warp] = upto;
    }
    __syncthreads();
    if (tid < 256) {
      int above = upto - mine;
      for (int k = warp + 1; k < 8; ++k) above += above_s[k];
      if (above < need && above + mine >= need) pick[0] = tid, pick[1] = above;
    }
    if constexpr (kSplit > 1) cluster_sync();  // the bins have been read
    else __syncthreads();
    border |= (uint32_t)pick[0] << shift;
    need -= pick[1];
    __syncthreads();  // `pick` and `above_s` have been read
  }

  // ---- the kept tokens' indices: those above the border, and the first `need` of those at it
  int over = 0, equal = 0;
  if (tid < 2) totals[tid] = 0;
  __syncthreads();
  for (int i = tid; i < count; i += kSelThreads) {
    const uint32_t k = key_at(i);
    over += k > border;
    equal += k == border;
  }
  over = __reduce_add_sync(0xffffffffu, over);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    atomicAdd(&totals[0], over);
    atomicAdd(&totals[1], equal);
  }
  int over_before = 0, equal_before = 0;
  if constexpr (kSplit > 1) {
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      over_before += load_remote(&totals[0], r);
      equal_before += load_remote(&totals[1], r);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
  for (int i0 = 0, buf = 0; i0 < count; i0 += kSelThreads, buf ^= 1) {
    const int i = i0 + tid;
    const uint32_t k = i < count ? key_at(i) : 0u;
    const bool is_over = i < count && k > border, is_equal = i < count && k == border;
    const uint32_t vo = __ballot_sync(0xffffffffu, is_over), ve = __ballot_sync(0xffffffffu, is_equal);
    if (lane == 0) scan_s[buf][warp] = __popc(vo) | __popc(ve) << 16;
    __syncthreads();
    const int theirs = scan_s[buf][lane];  // of warp `lane`
    int upto = theirs;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const int before = __shfl_sync(0xffffffffu, upto - theirs, warp), all = __shfl_sync(0xffffffffu, upto, 31);
    const uint32_t lower = (1u << lane) - 1u;
    const int o = over_before + (before & 0xffff) + __popc(vo & lower);
    const int e = equal_before + (before >> 16) + __popc(ve & lower);
    if (is_over || (is_equal && e < need)) kept[o + min(e, need)] = lo + i;
    over_before += all & 0xffff;
    equal_before += all >> 16;
  }
}

// ---------------------------------------------------------------- move

constexpr int kMoveThreads = 512;
constexpr int kUnroll = 8;

// Kept tokens [first, m) of one head: `lanes` threads a token, each with one T; chunks of kUnroll tokens a thread. `at`
// gives the place of a token (page row or index) and thread, in units of T.
template <typename T, typename From, typename To>
__device__ __forceinline__ void move_rows(int first, int m, int lanes, const int* kept, From from, To to) {
  const int per = kMoveThreads / lanes, r = threadIdx.x / lanes, chunk = per * kUnroll;
  T held[kUnroll];
  int src[kUnroll];
  auto indices = [&](int base) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * per + r;
      src[u] = i < m ? __ldg(kept + i) : -1;
    }
  };
  auto load = [&] {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (src[u] >= 0) held[u] = *from(src[u]);
  };
  indices(first);
  for (int base = first; base < m; base += chunk) {
    load();
    indices(base + chunk);
    __syncthreads();  // the whole chunk has been read, in place a part of it is where it goes
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = base + u * per + r;
      if (i < m) *to(i) = held[u];
    }
  }
}

// A unit's parts: its keys' slices, its values' slices, and its floats (scales and weights).
__global__ void __launch_bounds__(kMoveThreads, 1) move_kernel(const EvictArgs p, const KvArgs c, int slices) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int parts = 2 * slices + 1;
  const long long unit = blockIdx.x / parts;
  const int part = (int)(blockIdx.x % parts);
  const int n = (int)(unit / c.Hkv), h = (int)(unit % c.Hkv);
  int why;
  const int m = kept_of(p, c, n, &why);
  if (m <= 0 || p.new_len[n] < 0) return;
  const int* kept = p.kept + ((size_t)n * c.Hkv + h) * p.max_kept;
  const int32_t* table = p.table + (size_t)n * p.max_pages;
  const int32_t* dst_table = p.dst_table + (size_t)n * p.dst_max_pages;
  const int slot = __ldg(p.slot + n), dst_slot = __ldg(p.dst_slot + n);
  // in place the tokens in front of the first that is gone stay where they are
  auto first_moved = [&] {
    int lo = 0, hi = m;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(kept + mid) == mid) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  };
  auto row = [&](const int32_t* t, int i) {
    const int k = i / c.page;
    return ((size_t)__ldg(t + k) * c.Hkv + h) * c.page + (i - k * c.page);
  };
  if (part < 2 * slices) {
    const int row_bytes = p.D * (c.e4m3 ? 1 : 2), lanes = row_bytes / 16 / slices;
    uint4* pool = static_cast<uint4*>(part < slices ? c.k : c.v) + (part % slices) * lanes + threadIdx.x % lanes;
    const int row_pieces = row_bytes / 16;
    move_rows<uint4>(p.table == p.dst_table ? first_moved() : 0, m, lanes, kept,
                     [&](int i) { return pool + row(table, i) * row_pieces; },
                     [&](int i) { return pool + row(dst_table, i) * row_pieces; });
  } else {
    if (c.e4m3) {
      const int first = p.table == p.dst_table ? first_moved() : 0;
      move_rows<float>(first, m, 1, kept, [&](int i) { return c.k_scale + row(table, i); },
                       [&](int i) { return c.k_scale + row(dst_table, i); });
      move_rows<float>(first, m, 1, kept, [&](int i) { return c.v_scale + row(table, i); },
                       [&](int i) { return c.v_scale + row(dst_table, i); });
    }
    const float* w = p.score + ((size_t)slot * c.Hkv + h) * p.max_tokens;
    float* to = p.score + ((size_t)dst_slot * c.Hkv + h) * p.max_tokens;
    move_rows<float>(slot == dst_slot ? first_moved() : 0, m, 1, kept, [&](int i) { return w + i; },
                     [&](int i) { return to + i; });
  }
}

template <int kSplit>
cudaError_t launch_select(const EvictArgs& a, const KvArgs& c, cudaStream_t stream) {
  constexpr int kSmem = kCached * (int)sizeof(uint32_t);
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(&select_kernel<kSplit>), kSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.N * c.Hkv * kSplit), 1, 1);
  cfg.blockDim = dim3(kSelThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
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
  return cudaLaunchKernelEx(&cfg, select_kernel<kSplit>, a, c);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, const KvArgs& c, cudaStream_t stream) {
  const long long units = (long long)a.N * c.Hkv;
  cudaError_t err = units * 8 <= 152 ? launch_select<8>(a, c, stream) : launch_select<1>(a, c, stream);
  if (err != cudaSuccess) return err;
  // slices of the rows, down to 64 bytes, while there are too few blocks to keep HBM busy
  const int row_bytes = a.D * (c.e4m3 ? 1 : 2);
  int slices = 1;
  while (row_bytes / slices > 64 && units * 2 * slices < 4 * 152) slices *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * (2 * slices + 1)), 1, 1);
  cfg.blockDim = dim3(kMoveThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, move_kernel, a, c, slices);
}

}  // namespace gdn
