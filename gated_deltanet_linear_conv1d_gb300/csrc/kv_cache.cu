// kv_cache.cu - the attention layers' query/key preparation and their paged
// key/value cache: gdn_qk_norm_rope, gdn_kv_cache_write, gdn_kv_cache_read.
//
// Math, per head row x of D values (page "Qwen3.8-27B: from model structure to
// vLLM inference data flow", section 01, GQA rows; section 04, FP8 cache):
//   y = x / sqrt(mean(x^2) + eps) * gamma
//   (y_i, y_i') <- (y_i cos a_i - y_i' sin a_i, y_i' cos a_i + y_i sin a_i),  a_i = position * f_i
//   E4M3 cache: s = max(amax |y|, 1e-12) / 448, code = E4M3(y / s)
// Every byte is read once and written once, so HBM bounds all three at large
// token counts and the launch at small ones.
#include "device.cuh"
#include "launch.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.f;
constexpr float kMinAmax = 1e-12f;
constexpr int kMaxTokens = 16;  // tokens per block

__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)f32_to_bf16(x[i].x) | ((uint32_t)f32_to_bf16(x[i].y) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two fp32 values to two E4M3 codes (round to nearest even, saturate); lo lands in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 codes (low byte first) to fp32, exactly (every E4M3 value is an fp16 value).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

// A row group's largest magnitude (NaN is passed over); D / 8 lanes hold a row.
template <int kLanes>
__device__ __forceinline__ float row_amax(const float2 (&x)[4]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) a = fmaxf(a, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
  if constexpr (kLanes == 32) {
    asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(a));
  } else {
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
  }
  return a;
}

// Eight quotients x / s as E4M3 codes. The division is Markstein's (IBM J. Res. Dev. 34, 1990): with the correctly
// rounded reciprocal r of s, q = x r and its remainder x - q s, exact in one multiply-add, q + r (x - q s) rounds
// as x / s does: three packed operations for two values. Every pair of bf16 significands is tested against the
// division. An infinite s leaves zeros, and a NaN where x is infinite too.
__device__ __forceinline__ uint2 codes(const float2 (&x)[4], float s) {
  const bool finite = s < INFINITY;
  const float r = finite ? __frcp_rn(s) : 0.f, back = finite ? -s : 0.f;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = __fmul2_rn(x[i], make_float2(r, r));
    const float2 left = __ffma2_rn(q, make_float2(back, back), x[i]);
    const float2 y = __ffma2_rn(left, make_float2(r, r), q);
    w[i] = e4m3x2(y.x, y.y);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

enum { kNoCache = 0, kBf16Cache = 1, kE4m3Cache = 2 };

// The rows of a block's tokens, query heads, key heads and value heads of a token one after the other: a row group
// of D / 8 lanes takes kRows rows at a time, every kGroups-th of one token's, or, where a token has no more than
// kGroups of them, its one of kRows tokens. The next rows are on their way while these are worked on: with one batch
// in flight the loads, the arithmetic and the stores took turns (192 us for 16,384 tokens of 24 + 4 heads of 256).
// kNorm: the head norm, the rotation and the dense outputs; without it the rows go to the cache as they are.
// The angles of a token are the same for all its heads: a thread per (token, frequency) puts their cosine and sine
// into shared memory first. A position times a frequency is taken in turns, in 64-bit fixed point (one turn = 2^64),
// where the whole turns fall away by themselves: the error is the frequency's rounding to 2^-64 turns times the
// position, 2^-33 turns at the largest one.
template <int D, bool kNorm, int kCache>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RopeArgs p, const KvArgs c, int tokens_per_block) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes, kRows = 4;
  __shared__ uint64_t freq[kNorm ? D / 2 : 1];
  extern __shared__ float2 turn[];  // [tokens][half]
  const int tid = threadIdx.x, l = tid % kLanes, group = tid / kLanes;
  const int t0 = blockIdx.x * tokens_per_block;
  const int T = min(tokens_per_block, p.T - t0);
  const int half = p.rotary / 2;
  const bool rotate = kNorm && half > 0;
  // the lane's eight dimensions: rotated or not, and where the other dimensions of their pairs are
  const bool turns = rotate && l * 8 < p.rotary;
  const bool low = l < half / 8;
  const int partner = (tid & 31) + (!turns || p.interleaved ? 0 : low ? half / 8 : -(half / 8));
  const int Hq = kNorm && p.q ? p.Hq : 0, Hk = Hq + c.Hkv;
  const int per_token = Hk + (p.v ? c.Hkv : 0);
  const bool many = per_token > kGroups;              // rows of one token in a batch, else of kRows tokens
  const int step_h = many ? kGroups : 0, step_t = many ? 0 : 1;

  // row i of the batch at (tl, h0): token tl + i * step_t, head h0 + i * step_h + group
  auto fetch = [&](int tl, int h0, uint4 (&raw)[kRows], int (&slot)[kRows]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int ti = tl + i * step_t, h = h0 + i * step_h + group;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      slot[i] = -1;
      if (ti < T && h < per_token) {
        const int64_t t = t0 + ti;
        const uint16_t* src = h < Hq   ? p.q + t * p.q_t + h * p.q_h
                              : h < Hk ? p.k + t * p.k_t + (h - Hq) * p.k_h
                                       : p.v + t * p.v_t + (h - Hk) * p.v_h;
        raw[i] = *reinterpret_cast<const uint4*>(src + l * 8);
        if (kCache != kNoCache && h >= Hq) slot[i] = p.kv_slot[t];
      }
    }
  };
  uint4 raw[kRows];
  int slot[kRows];
  fetch(0, 0, raw, slot);
  if constexpr (kNorm) {
    if (rotate) {
      for (int i = tid; i < half; i += kThreads) {
        const double f = p.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi): turns per position
        freq[i] = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
      }
      __syncthreads();
      for (int i = tid; i < T * half; i += kThreads) {
        const int64_t pos = p.positions[t0 + i / half];
        // the upper 32 bits as a signed number: half turns in [-1, 1)
        const int32_t top = (int32_t)(((uint64_t)pos * freq[i % half]) >> 32);
        float s, co;
        sincospif((float)top * 4.656612873077393e-10f, &s, &co);
        turn[i] = make_float2(co, s);
      }
      __syncthreads();
    }
  }
  for (int tl = 0, h0 = 0; tl < T;) {
    const int tl_now = tl, h0_now = h0;
    if (many) {
      h0 += kGroups * kRows;
      if (h0 >= per_token) h0 = 0, ++tl;
    } else {
      tl += kRows;
    }
    uint4 next[kRows];
    int next_slot[kRows];
    if (tl < T) fetch(tl, h0, next, next_slot);
    float inv[kRows];
    if constexpr (kNorm) {
      // the sums of the rows' squares, each lane's part in `inv` first
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
          ss = __ffma2_rn(x, x, ss);
        }
        inv[i] = ss.x + ss.y;
      }
      // four rows in one butterfly: after two steps a lane has one row's sum, after the rest its whole
      const bool b1 = l & (kLanes / 2), b2 = l & (kLanes / 4);
      float a0 = b1 ? inv[2] : inv[0], a1 = b1 ? inv[3] : inv[1];
      a0 += __shfl_xor_sync(0xffffffffu, b1 ? inv[0] : inv[2], kLanes / 2);
      a1 += __shfl_xor_sync(0xffffffffu, b1 ? inv[1] : inv[3], kLanes / 2);
      float a = b2 ? a1 : a0;
      a += __shfl_xor_sync(0xffffffffu, b2 ? a0 : a1, kLanes / 4);
#pragma unroll
      for (int m = kLanes / 8; m > 0; m >>= 1) a += __shfl_xor_sync(0xffffffffu, a, m);
      a = rsqrtf(a * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < kRows; ++i)  // row i's is in the lanes with bits i / 2 and i % 2
        inv[i] = __shfl_sync(0xffffffffu, a, (tid & 31) - l + (i >> 1) * (kLanes / 2) + (i & 1) * (kLanes / 4));
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int ti = tl_now + i * step_t, h = h0_now + i * step_h + group;
      // nothing left for any group: the shuffles take whole warps
      if (ti >= T || h - group >= per_token) break;
      const int64_t t = t0 + ti;
      const bool live = h < per_token, is_q = h < Hq, is_v = h >= Hk;
      const int hk = is_q ? 0 : is_v ? h - Hk : h - Hq;
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      float2 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
      if constexpr (kNorm) {
        uint32_t o[4];
        if (rotate && !p.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = __shfl_sync(0xffffffffu, w[e], partner);
        }
        if (live && !is_v) {
          const float* gamma = is_q ? p.q_gamma : p.k_gamma;
          const float4 g0 = __ldg(reinterpret_cast<const float4*>(gamma) + 2 * l);
          const float4 g1 = __ldg(reinterpret_cast<const float4*>(gamma) + 2 * l + 1);
          const float2 f = make_float2(inv[i], inv[i]);
          x[0] = __fmul2_rn(__fmul2_rn(x[0], f), make_float2(g0.x, g0.y));
          x[1] = __fmul2_rn(__fmul2_rn(x[1], f), make_float2(g0.z, g0.w));
          x[2] = __fmul2_rn(__fmul2_rn(x[2], f), make_float2(g1.x, g1.y));
          x[3] = __fmul2_rn(__fmul2_rn(x[3], f), make_float2(g1.z, g1.w));
          if (turns) {
            if (p.interleaved) {
              const float4* cs = reinterpret_cast<const float4*>(turn + ti * half + l * 4);
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const float4 w2 = cs[e / 2];  // two pairs' cosine and sine
                const float2 u = x[e], v = x[e + 1];
                x[e] = make_float2(u.x * w2.x - u.y * w2.y, u.y * w2.x + u.x * w2.y);
                x[e + 1] = make_float2(v.x * w2.z - v.y * w2.w, v.y * w2.z + v.x * w2.w);
              }
            } else {
              const float4* pg = reinterpret_cast<const float4*>(gamma) + 2 * (low ? l + half / 8 : l - half / 8);
              const float4 p0 = __ldg(pg), p1 = __ldg(pg + 1);
              const float2 g[4] = {make_float2(p0.x, p0.y), make_float2(p0.z, p0.w), make_float2(p1.x, p1.y),
                                   make_float2(p1.z, p1.w)};
              const float4* cs = reinterpret_cast<const float4*>(turn + ti * half + (low ? l : l - half / 8) * 8);
              const float sign = low ? -1.f : 1.f;  // a' = a cos - b sin, b' = b cos + a sin
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 w2 = cs[e];
                const float2 other = __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(o[e] << 16),
                                                                       __uint_as_float(o[e] & 0xffff0000u)), f), g[e]);
                x[e] = __ffma2_rn(x[e], make_float2(w2.x, w2.z),
                                  __fmul2_rn(other, make_float2(sign * w2.y, sign * w2.w)));
              }
            }
          }
          if (is_q)
            *reinterpret_cast<uint4*>(p.q_out + ((size_t)t * p.Hq + h) * D + l * 8) = pack8(x);
          else if (p.k_out)
            *reinterpret_cast<uint4*>(p.k_out + ((size_t)t * c.Hkv + hk) * D + l * 8) = pack8(x);
        }
      }
      if constexpr (kCache != kNoCache) {
        const bool store = live && !is_q && slot[i] >= 0 && slot[i] < c.slots;
        if (slot[i] >= c.slots && l == 0) report(p.dev_err, GDN_DEVERR_SLOT);
        if (!__any_sync(0xffffffffu, store)) continue;
        const int page = store ? slot[i] / c.page : 0, row = store ? slot[i] - page * c.page : 0;
        const size_t at = ((size_t)page * c.Hkv + hk) * c.page + row;
        if constexpr (kCache == kE4m3Cache) {
          const float s = __fdiv_rn(fmaxf(row_amax<kLanes>(x), kMinAmax), kE4m3Max);
          if (store) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + at * D + l * 8) = codes(x, s);
            if (l == 0) (is_v ? c.v_scale : c.k_scale)[at] = s;
          }
        } else if (store) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? c.v : c.k) + at * D + l * 8) = pack8(x);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      raw[i] = next[i];
      slot[i] = next_slot[i];
    }
  }
}

// Cached rows back to bf16: a block takes kReadTokens output tokens, a thread 16
// values of one (token, k or v, head) row at a time. The request of the block's
// first token is found by bisection, the others' by walking on from it.
constexpr int kReadTokens = 8;

template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs p, const KvArgs c) {
  __shared__ long long src[kReadTokens];  // row of the first head of the token's page, -1: nothing to read
  const int t0 = blockIdx.x * kReadTokens;
  if (threadIdx.x < kReadTokens) {
    const int t = t0 + threadIdx.x;
    long long at = -1;
    if (t < p.T) {
      int lo = 0, hi = p.N;  // the last request that starts at or before t: start[lo] <= t < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.start[mid] <= t) lo = mid; else hi = mid;
      }
      const int s = p.start[lo], e = p.start[lo + 1], i = t - s;
      if (s < 0 || i < 0 || t >= e || e > p.T || (e - s - 1) / c.page >= p.max_pages) {
        report(p.dev_err, GDN_DEVERR_OFFSETS);
      } else {
        const int page = p.table[(size_t)lo * p.max_pages + i / c.page];
        if (page < 0 || page >= c.pages) report(p.dev_err, GDN_DEVERR_SLOT);
        else at = (long long)page * c.Hkv * c.page + i % c.page;
      }
    }
    src[threadIdx.x] = at;
  }
  __syncthreads();
  constexpr int kChunks = D / 16;
  const int per_token = 2 * c.Hkv * kChunks;
  const int total = min(kReadTokens, p.T - t0) * per_token;
#pragma unroll 4
  for (int i = threadIdx.x; i < total; i += kThreads) {
    const int tl = i / per_token;
    int rest = i - tl * per_token;
    const bool value = rest >= c.Hkv * kChunks;
    if (value) rest -= c.Hkv * kChunks;
    const int h = rest / kChunks, ch = rest % kChunks;
    const long long first = src[tl];
    if (first < 0) continue;
    const size_t row = (size_t)first + (size_t)h * c.page;
    uint4 out[2];
    if (c.e4m3) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(value ? c.v : c.k) + row * D) + ch);
      const float s = (value ? c.v_scale : c.k_scale)[row];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        float2 x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t word = w[2 * o + (e >> 1)];
          x[e] = __fmul2_rn(e4m3x2_to_f32((uint16_t)((e & 1) ? word >> 16 : word & 0xffff)), make_float2(s, s));
        }
        out[o] = pack8(x);
      }
    } else {
      const uint4* u = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(value ? c.v : c.k) + row * D) + 2 * ch;
      out[0] = __ldcs(u);
      out[1] = __ldcs(u + 1);
    }
    uint4* dst = reinterpret_cast<uint4*>((value ? p.v_out : p.k_out) + ((size_t)(t0 + tl) * c.Hkv + h) * D) + 2 * ch;
    __stcs(dst, out[0]);
    __stcs(dst + 1, out[1]);
  }
}

}  // namespace

namespace {

template <int D>
void run_rows(const RopeArgs& a, const KvArgs& c, bool norm, unsigned grid, int per, cudaStream_t stream) {
  const int cache = !c.k ? kNoCache : c.e4m3 ? kE4m3Cache : kBf16Cache;
  const size_t smem = norm ? (size_t)per * (a.rotary / 2) * sizeof(float2) : 0;
  if (norm) {
    if (cache == kNoCache) rows_kernel<D, true, kNoCache><<<grid, kThreads, smem, stream>>>(a, c, per);
    else if (cache == kBf16Cache) rows_kernel<D, true, kBf16Cache><<<grid, kThreads, smem, stream>>>(a, c, per);
    else rows_kernel<D, true, kE4m3Cache><<<grid, kThreads, smem, stream>>>(a, c, per);
  } else {
    if (cache == kBf16Cache) rows_kernel<D, false, kBf16Cache><<<grid, kThreads, smem, stream>>>(a, c, per);
    else rows_kernel<D, false, kE4m3Cache><<<grid, kThreads, smem, stream>>>(a, c, per);
  }
}

}  // namespace

cudaError_t launch_rows(const RopeArgs& a, const KvArgs& c, bool norm, int D, cudaStream_t stream) {
  // enough blocks for every SM before a block takes several tokens
  int per = 1;
  while (per < kMaxTokens && a.T / (2 * per) >= 4 * 152) per *= 2;
  const unsigned grid = (unsigned)((a.T + per - 1) / per);
  if (D == 256) run_rows<256>(a, c, norm, grid, per, stream);
  else run_rows<128>(a, c, norm, grid, per, stream);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const ReadArgs& a, const KvArgs& c, int D, cudaStream_t stream) {
  const unsigned grid = (unsigned)((a.T + kReadTokens - 1) / kReadTokens);
  if (D == 256) read_kernel<256><<<grid, kThreads, 0, stream>>>(a, c);
  else read_kernel<128><<<grid, kThreads, 0, stream>>>(a, c);
  return cudaGetLastError();
}

}  // namespace gdn
