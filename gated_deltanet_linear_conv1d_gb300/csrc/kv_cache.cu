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
constexpr int kMaxTokens = 8;  // tokens per block

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)f32_to_bf16(x[2 * i]) | ((uint32_t)f32_to_bf16(x[2 * i + 1]) << 16);
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

// One row of D values, eight per lane, into its place in the cache. kLanes = D / 8 lanes hold the row.
template <int kLanes>
__device__ __forceinline__ void store_row(const KvArgs& c, bool value, int slot, int head, int l, float (&x)[8]) {
  const int page = slot / c.page, row = slot % c.page;
  const size_t at = ((size_t)page * c.Hkv + head) * c.page + row;
  if (c.e4m3) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
    const float s = __fdiv_rn(fmaxf(a, kMinAmax), kE4m3Max);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], s);
    if (slot < 0) return;
    uint8_t* pool = static_cast<uint8_t*>(value ? c.v : c.k);
    *reinterpret_cast<uint2*>(pool + at * (kLanes * 8) + l * 8) =
        make_uint2(e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16), e4m3x2(x[4], x[5]) | (e4m3x2(x[6], x[7]) << 16));
    if (l == 0) (value ? c.v_scale : c.k_scale)[at] = s;
  } else {
    if (slot < 0) return;
    uint16_t* pool = static_cast<uint16_t*>(value ? c.v : c.k);
    *reinterpret_cast<uint4*>(pool + at * (kLanes * 8) + l * 8) = pack8(x);
  }
}

// The rows of a block's tokens, (query heads), key heads and (value heads) of a
// token one after the other, dealt to its row groups of D / 8 lanes; a group
// loads kRows rows before it works on the first. kNorm: the head norm, the
// rotation and the dense outputs; without it the rows go to the cache as they are.
// The angles of a token are the same for all its heads: a thread per (token,
// frequency) puts their cosine and sine into shared memory first. A position
// times a frequency is taken in turns, in 64-bit fixed point (one turn = 2^64),
// where the whole turns fall away by themselves: the error is the frequency's
// rounding to 2^-64 turns times the position, 2^-33 turns at the largest one.
template <int D, bool kNorm>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RopeArgs p, const KvArgs c, int tokens_per_block) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes, kRows = 4;
  __shared__ uint64_t freq[D / 2];
  __shared__ float2 turn[kNorm ? kMaxTokens * D / 2 : 1];
  const int tid = threadIdx.x, l = tid % kLanes, group = tid / kLanes;
  const int t0 = blockIdx.x * tokens_per_block;
  const int T = min(tokens_per_block, p.T - t0);
  const int half = p.rotary / 2;
  const bool rotate = kNorm && half > 0;
  float qg[8], kg[8];
  if constexpr (kNorm) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 kv = *reinterpret_cast<const float4*>(p.k_gamma + l * 8 + i);
      kg[i] = kv.x; kg[i + 1] = kv.y; kg[i + 2] = kv.z; kg[i + 3] = kv.w;
      const float4 qv = p.q ? *reinterpret_cast<const float4*>(p.q_gamma + l * 8 + i) : kv;
      qg[i] = qv.x; qg[i + 1] = qv.y; qg[i + 2] = qv.z; qg[i + 3] = qv.w;
    }
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
  const int Hq = kNorm && p.q ? p.Hq : 0;
  const int per_token = Hq + c.Hkv + (c.v ? c.Hkv : 0);
  const int total = T * per_token;
  for (int r0 = group; r0 - group < total; r0 += kGroups * kRows) {
    uint4 raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + i * kGroups;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < total) {
        const int tl = r / per_token, h = r - tl * per_token;
        const int64_t t = t0 + tl;
        const uint16_t* src = h < Hq            ? p.q + t * p.q_t + h * p.q_h
                              : h < Hq + c.Hkv ? p.k + t * p.k_t + (h - Hq) * p.k_h
                                               : p.v + t * p.v_t + (h - Hq - c.Hkv) * p.v_h;
        raw[i] = *reinterpret_cast<const uint4*>(src + l * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + i * kGroups;
      if (r0 - group + i * kGroups >= total) break;  // for every group at once: the shuffles take whole warps
      const bool live = r < total;
      const int tl = live ? r / per_token : 0, h = live ? r - tl * per_token : 0;
      const int64_t t = t0 + tl;
      const bool is_q = h < Hq, is_v = h >= Hq + c.Hkv;
      const int hk = is_q ? 0 : is_v ? h - Hq - c.Hkv : h - Hq;
      float x[8];
      unpack8(raw[i], x);
      if constexpr (kNorm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int m = kLanes / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (!is_v) {
          const float inv = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * (is_q ? qg[e] : kg[e]);
        }
        if (rotate) {
          const float2* cs = turn + tl * half;
          if (p.interleaved) {
            if (!is_v && l * 8 < p.rotary) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 w = cs[l * 4 + e];
                const float a = x[2 * e], b = x[2 * e + 1];
                x[2 * e] = a * w.x - b * w.y;
                x[2 * e + 1] = b * w.x + a * w.y;
              }
            }
          } else {
            // element i's partner, half away, is the same element of another lane
            const int hl = half / 8;
            const bool low = l < hl, in = l < 2 * hl && !is_v;
            const int from = low ? l + hl : l - hl;
            const int src = (tid & 31) - l + (l < 2 * hl ? from : l);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float other = __shfl_sync(0xffffffffu, x[e], src);
              if (in) {
                const float2 w = cs[(low ? l : l - hl) * 8 + e];
                x[e] = x[e] * w.x + (low ? -other : other) * w.y;
              }
            }
          }
        }
        if (live && !is_v) {
          if (is_q)
            *reinterpret_cast<uint4*>(p.q_out + ((size_t)t * p.Hq + h) * D + l * 8) = pack8(x);
          else if (p.k_out)
            *reinterpret_cast<uint4*>(p.k_out + ((size_t)t * c.Hkv + hk) * D + l * 8) = pack8(x);
        }
      }
      if (c.k && __any_sync(0xffffffffu, live && !is_q)) {
        int slot = -1;
        if (live && !is_q) {
          slot = p.kv_slot[t];
          if (slot >= c.slots) {
            if (l == 0) report(p.dev_err, GDN_DEVERR_SLOT);
            slot = -1;
          }
        }
        store_row<kLanes>(c, is_v, slot, hk, l, x);
      }
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
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t word = w[2 * o + (e >> 1)];
          const float2 f = e4m3x2_to_f32((uint16_t)((e & 1) ? word >> 16 : word & 0xffff));
          x[2 * e] = f.x * s;
          x[2 * e + 1] = f.y * s;
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

cudaError_t launch_rows(const RopeArgs& a, const KvArgs& c, bool norm, int D, cudaStream_t stream) {
  // enough blocks for every SM before a block takes several tokens
  int per = 1;
  while (per < kMaxTokens && a.T / (2 * per) >= 4 * 152) per *= 2;
  const unsigned grid = (unsigned)((a.T + per - 1) / per);
  if (D == 256) {
    if (norm) rows_kernel<256, true><<<grid, kThreads, 0, stream>>>(a, c, per);
    else rows_kernel<256, false><<<grid, kThreads, 0, stream>>>(a, c, per);
  } else {
    if (norm) rows_kernel<128, true><<<grid, kThreads, 0, stream>>>(a, c, per);
    else rows_kernel<128, false><<<grid, kThreads, 0, stream>>>(a, c, per);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const ReadArgs& a, const KvArgs& c, int D, cudaStream_t stream) {
  const unsigned grid = (unsigned)((a.T + kReadTokens - 1) / kReadTokens);
  if (D == 256) read_kernel<256><<<grid, kThreads, 0, stream>>>(a, c);
  else read_kernel<128><<<grid, kThreads, 0, stream>>>(a, c);
  return cudaGetLastError();
}

}  // namespace gdn
