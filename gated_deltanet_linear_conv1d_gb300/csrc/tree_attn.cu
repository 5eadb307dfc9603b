// tree_attn.cu - gdn_tree_attention: attention of the drafted tokens of a tree
// over a request's paged cache and over each other.
//
// Math, per query row (node j, query head h), over the tokens t that it sees:
//   s_t = scale (q . k_t),  m = max s_t,  l = sum e^(s_t - m),  out = sum e^(s_t - m) v_t / l
// and with a gate out <- out / (1 + e^-gate).
//
// One block per query row: its four warps take every fourth token each, a lane
// holding D / 32 of the row's values, with the running maximum and sum of the
// softmax; the warps' parts meet in shared memory.
#include "device.cuh"
#include "launch.h"

namespace gdn {

namespace {

template <int D, bool kE4m3>
__device__ __forceinline__ void load_row(const void* pool, const float* scale, size_t row, int lane, float (&x)[D / 32]) {
  constexpr int E = D / 32;
  if constexpr (kE4m3) {
    const uint8_t* src = static_cast<const uint8_t*>(pool) + row * D + lane * E;
    const float s = scale[row];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t c = src[e], ex = (c >> 3) & 15, m = c & 7;
      float v = ex ? __uint_as_float(((ex + 120) << 23) | (m << 20)) : (float)m * 0.001953125f;
      if (ex == 15 && m == 7) v = __uint_as_float(0x7fffffffu);
      x[e] = (c & 128 ? -v : v) * s;
    }
  } else {
    const uint16_t* src = static_cast<const uint16_t*>(pool) + row * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = bf16_to_f32(src[e]);
  }
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(128) tree_attn_kernel(const TreeAttnArgs p, const KvArgs c) {
  constexpr int E = D / 32;
  __shared__ float part[4][D + 2];
  const int hq = blockIdx.x % p.Hq, row = blockIdx.x / p.Hq, n = row / p.P, j = row % p.P;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = hq / p.G;
  const int ctx = p.ctx[n];
  if (ctx < 0) return;
  const int32_t* table = p.table + (size_t)n * p.max_pages;
  const long long len = (long long)ctx + p.P;
  bool bad = (len + c.page - 1) / c.page > p.max_pages;
  if (bad && threadIdx.x == 0) report(p.dev_err, GDN_DEVERR_OFFSETS);
  if (!bad) {
    for (long long i = threadIdx.x; i < (len + c.page - 1) / c.page; i += blockDim.x) bad |= table[i] < 0 || table[i] >= c.pages;
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) report(p.dev_err, GDN_DEVERR_SLOT);
  }
  if (bad) return;
  const uint64_t mask = p.mask ? p.mask[(size_t)n * p.P + j] : j == 63 ? ~0ull : (1ull << (j + 1)) - 1;
  const size_t qoff = ((size_t)row * p.Hq + hq) * D + lane * E;
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_to_f32(p.q[qoff + e]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (long long t = warp; t < len; t += 4) {
    if (t >= ctx && !((mask >> (t - ctx)) & 1)) continue;
    const size_t at = ((size_t)table[t / c.page] * c.Hkv + h) * c.page + t % c.page;
    float k[E], v[E];
    load_row<D, kE4m3>(c.k, c.k_scale, at, lane, k);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    s = warp_sum(s) * p.scale;
    load_row<D, kE4m3>(c.v, c.v_scale, at, lane, v);
    const float mn = fmaxf(m, s), a = m == mn ? 1.f : expf(m - mn), w = expf(s - mn);
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[e], acc[e] * a);
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
  if (lane == 0) {
    part[warp][D] = m;
    part[warp][D + 1] = l;
  }
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, part[w][D]);
  for (int w = 0; w < 4; ++w)
    if (part[w][D + 1] != 0.f) ll += part[w][D + 1] * expf(part[w][D] - mm);
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float o = 0.f;
    for (int w = 0; w < 4; ++w)
      if (part[w][D + 1] != 0.f) o += part[w][d] * expf(part[w][D] - mm);
    o = ll != 0.f ? o / ll : 0.f;
    const size_t at = ((size_t)row * p.Hq + hq) * D + d;
    if (p.gate) o = o / (1.f + expf(-bf16_to_f32(p.gate[at])));
    p.out[at] = f32_to_bf16(o);
  }
}

}  // namespace

size_t tree_attn_workspace_bytes(int N, int P, int Hq, int Hkv, int D, bool e4m3) { return 256; }

cudaError_t launch_tree_attn(const TreeAttnArgs& a, const KvArgs& c, cudaStream_t stream) {
  const unsigned grid = (unsigned)((long long)a.N * a.P * a.Hq);
  if (a.D == 256) {
    if (c.e4m3) tree_attn_kernel<256, true><<<grid, 128, 0, stream>>>(a, c);
    else tree_attn_kernel<256, false><<<grid, 128, 0, stream>>>(a, c);
  } else {
    if (c.e4m3) tree_attn_kernel<128, true><<<grid, 128, 0, stream>>>(a, c);
    else tree_attn_kernel<128, false><<<grid, 128, 0, stream>>>(a, c);
  }
  return cudaGetLastError();
}

}  // namespace gdn
