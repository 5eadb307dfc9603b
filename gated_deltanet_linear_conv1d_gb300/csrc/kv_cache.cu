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

__device__ __forceinline__ uint32_t bf16x2(float2 x) {  // x.x in the low half
  const __nv_bfloat162 v = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  return make_uint4(bf16x2(x[0]), bf16x2(x[1]), bf16x2(x[2]), bf16x2(x[3]));
}
__device__ __forceinline__ void unpack8(const uint2 (&u)[2], float2 (&x)[4]) {
  const uint32_t w[4] = {u[0].x, u[0].y, u[1].x, u[1].y};
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
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

enum { kPartial = 0, kWhole = 1, kInterleaved = 2 };  // up to D / 2 rotated dimensions, all D, neighbours as pairs

// Batches of four rows per group on their way to shared memory, past the registers, next to the one that is worked on.
constexpr int kAhead = 2, kBuffers = kAhead + 1, kRows = 4;
constexpr int kBatchBytes = kThreads * kRows * 16;  // a lane has eight values of a row

__device__ __forceinline__ void copy16(void* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}

// The query rows (kQuery) or the key and value rows of a block's T tokens, H of them a token. D / 8 lanes hold a row:
// lane l has four values from 4 l on, and four from D / 2 + 4 l on. A row group keeps its head over the tokens, so that
// what goes by the head (addresses, gains) is found once. A batch is four rows, loaded before the first is worked on:
// every kGroups-th head of one token (kMany), or, where a token has no more rows than there are groups, one head of
// four tokens.
// A rotated value is inv (x A + x' B): x' the other value of its pair, inv the row's 1 / sqrt(mean + eps), A the cosine
// times x's gain, B the signed sine times the gain of x'. Up to D / 2 rotated dimensions are in the first four values of
// the first lanes, and pairs half a rotation apart are in lanes l and l ^ (half / 4); with all D rotated they are a lane's
// first and second four.
template <int D, bool kNorm, int kCache, bool kQuery, bool kMany, int kRot>
__device__ __forceinline__ void rows_pass(const RopeArgs& p, const KvArgs& c, const float2* turn, unsigned char* stage,
                                          int* place, int t0, int T, int H) {
  constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
  constexpr int kStep = kMany ? 1 : kRows;  // tokens of a batch
  const int tid = threadIdx.x, l = tid % kLanes, group = tid / kLanes;
  const int half = p.rotary / 2;
  const bool turns = kNorm && l * 4 < (kRot == kWhole ? D / 2 : p.rotary);
  const bool low = kRot == kWhole || (l * 4 & half) == 0;  // the lane's first four are their pairs' first values

  for (int h0 = 0; h0 < H; h0 += kGroups * (kMany ? kRows : 1)) {
    const int h = h0 + group;
    const bool value = !kQuery && h >= c.Hkv, live = h < H;
    const int hh = value ? h - c.Hkv : h;
    const int64_t st = kQuery ? p.q_t : value ? p.v_t : p.k_t;
    // row i of a batch: i steps on from the first
    const uint16_t* src = (kQuery ? p.q + hh * p.q_h : value ? p.v + hh * p.v_h : p.k + hh * p.k_h) + t0 * st + l * 8;
    const int64_t step = kMany ? kGroups * p.q_h : st;
    uint16_t* dst = kQuery ? p.q_out : value ? nullptr : p.k_out;  // dense output, or none
    const int64_t out_t = (int64_t)(kQuery ? p.Hq : c.Hkv) * D, out_step = kMany ? kGroups * D : out_t;
    if (dst) dst += t0 * out_t + hh * D + l * 4;
    float2 gain[4], other_gain[2];
    if constexpr (kNorm) {
      const float* gamma = kQuery ? p.q_gamma : p.k_gamma;
      const float4 g0 = __ldg(reinterpret_cast<const float4*>(gamma + l * 4));
      const float4 g1 = __ldg(reinterpret_cast<const float4*>(gamma + D / 2 + l * 4));
      const float4 o = __ldg(reinterpret_cast<const float4*>(gamma + (kRot == kPartial && turns ? (l * 4) ^ half : l * 4)));
      gain[0] = make_float2(g0.x, g0.y);
      gain[1] = make_float2(g0.z, g0.w);
      gain[2] = make_float2(g1.x, g1.y);
      gain[3] = make_float2(g1.z, g1.w);
      other_gain[0] = make_float2(o.x, o.y);
      other_gain[1] = make_float2(o.z, o.w);
    }
    unsigned char* rows = stage + group * (kRows * D * 2);  // of the group, in the first buffer
    auto fetch = [&](int tl, int buf) {  // the batch from token tl on
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (kMany ? tl < T && h + i * kGroups < H : live && tl + i < T)
          copy16(rows + buf * kBatchBytes + i * (D * 2) + l * 16, src + tl * st + i * step);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncwarp();  // the buffers have been read
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(k * kStep, k);
    if constexpr (kCache != kNoCache && !kQuery) {
      // where the tokens go: the row of the page's first head, -1: nowhere
      if (h0 == 0) {
        for (int t = tid; t < T; t += kThreads) {
          const int to = __ldg(p.kv_slot + t0 + t), page = to / c.page;
          if (to >= c.slots) report(p.dev_err, GDN_DEVERR_SLOT);
          place[t] = to < 0 || to >= c.slots ? -1 : page * c.Hkv * c.page + (to - page * c.page);
        }
        __syncthreads();
      }
    }
    int buf = 0;
    for (int tl = 0; tl < T; tl += kStep) {
      __syncwarp();  // the batch before has been read, by lanes other than those that copied it: its buffer is next
      fetch(tl + kAhead * kStep, buf == 0 ? kAhead : buf - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
      __syncwarp();
      const unsigned char* batch = rows + buf * kBatchBytes + l * 8;
      auto load = [&](int i, uint2 (&raw)[2]) {
        raw[0] = *reinterpret_cast<const uint2*>(batch + i * (D * 2));
        raw[1] = *reinterpret_cast<const uint2*>(batch + i * (D * 2) + D);
      };
      if (++buf == kBuffers) buf = 0;
      float inv[kRows];
      if constexpr (kNorm) {
        // the sums of the rows' squares, each lane's part in `inv` first
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          float2 x[4], ss = make_float2(0.f, 0.f);
          uint2 raw[2];
          load(i, raw);
          unpack8(raw, x);
#pragma unroll
          for (int e = 0; e < 4; ++e) ss = __ffma2_rn(x[e], x[e], ss);
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
      float2 A[4], B[4];
      auto coefficients = [&](int ti) {
#pragma unroll
        for (int e = 0; e < 4; ++e) A[e] = gain[e], B[e] = make_float2(0.f, 0.f);
        if (!turns) return;
        if constexpr (kRot == kInterleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < 2 || p.rotary == D) {
              const float2 w = turn[ti * half + (e < 2 ? 0 : D / 4) + l * 2 + (e & 1)];
              B[e] = make_float2(-w.y * gain[e].y, w.y * gain[e].x);
              A[e] = make_float2(w.x * gain[e].x, w.x * gain[e].y);
            }
        } else {
          const float4* w = reinterpret_cast<const float4*>(turn + ti * half + (l * 4 & (half - 1)));
          const float sign = low ? -1.f : 1.f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 v = w[e];
            const float2 co = make_float2(v.x, v.z), si = make_float2(v.y, v.w);
            A[e] = __fmul2_rn(gain[e], co);
            B[e] = __fmul2_rn(kRot == kWhole ? gain[2 + e] : other_gain[e], make_float2(sign * si.x, sign * si.y));
            if (kRot == kWhole) {
              A[2 + e] = __fmul2_rn(gain[2 + e], co);
              B[2 + e] = __fmul2_rn(gain[e], si);
            }
          }
        }
      };
      if (kNorm && kMany) coefficients(tl);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int ti = tl + (kMany ? 0 : i), hi = h + (kMany ? i * kGroups : 0);
        // nothing left for any group: the shuffles take whole warps
        if (ti >= T || hi - group >= H) break;
        float2 x[4];
        uint2 raw[2];
        load(i, raw);
        unpack8(raw, x);
        if constexpr (kNorm) {
          uint2 o = raw[0];
          if (kRot == kPartial && half > 0) {
            const int from = (tid & 31) ^ (turns ? half / 4 : 0);
            o.x = __shfl_sync(0xffffffffu, o.x, from);
            o.y = __shfl_sync(0xffffffffu, o.y, from);
          }
          if (!value) {
            if (!kMany) coefficients(ti);
            float2 y[4];
            if constexpr (kRot == kInterleaved) {
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = make_float2(x[e].y, x[e].x);
            } else if constexpr (kRot == kWhole) {
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = x[e ^ 2];
            } else {
              const uint2 both[2] = {o, o};
              unpack8(both, y);
            }
            const float2 f = make_float2(inv[i], inv[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = __fmul2_rn(x[e], A[e]);
              if (e < 2 || kRot != kPartial) x[e] = turns ? __ffma2_rn(y[e], B[e], x[e]) : x[e];
              x[e] = __fmul2_rn(x[e], f);
            }
            if (dst && (kMany ? hi < H : live)) {
              uint16_t* to = dst + i * out_step;
              *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2(x[0]), bf16x2(x[1]));
              *reinterpret_cast<uint2*>(to + D / 2) = make_uint2(bf16x2(x[2]), bf16x2(x[3]));
            }
          }
        }
        if constexpr (kCache != kNoCache && !kQuery) {
          const int to = place[ti];
          const bool store = live && to >= 0;
          if (!__any_sync(0xffffffffu, store)) continue;
          const size_t at = (size_t)to + (size_t)hh * c.page;
          if constexpr (kCache == kE4m3Cache) {
            // a / 448, rounded once, as in codes()
            constexpr float kInv = 1.f / kE4m3Max;
            const float a = fmaxf(row_amax<kLanes>(x), kMinAmax), s0 = a * kInv;
            const float s = a < INFINITY ? fmaf(fmaf(-s0, kE4m3Max, a), kInv, s0) : a;
            if (store) {
              const uint2 w = codes(x, s);
              uint8_t* pool = static_cast<uint8_t*>(value ? c.v : c.k) + at * D + l * 4;
              *reinterpret_cast<uint32_t*>(pool) = w.x;
              *reinterpret_cast<uint32_t*>(pool + D / 2) = w.y;
              if (l == 0) (value ? c.v_scale : c.k_scale)[at] = s;
            }
          } else if (store) {
            uint16_t* pool = static_cast<uint16_t*>(value ? c.v : c.k) + at * D + l * 4;
            *reinterpret_cast<uint2*>(pool) = make_uint2(bf16x2(x[0]), bf16x2(x[1]));
            *reinterpret_cast<uint2*>(pool + D / 2) = make_uint2(bf16x2(x[2]), bf16x2(x[3]));
          }
        }
      }
      if (dst) dst += kMany ? out_t : kRows * out_t;
    }
  }
}

// blockIdx.y 0: the key and value rows of the block's tokens, 1: their query rows.
// kNorm: the head norm, the rotation and the dense outputs; without it the rows go to the cache as they are.
// The angles: a thread per (token, frequency) puts their cosine and sine into shared memory first. A position times a
// frequency is taken in turns, in 64-bit fixed point (one turn = 2^64), where the whole turns fall away by themselves.
// The frequency in turns is an fp64 product with 1 / (2 pi), off by up to 2^-52 of itself, and so is the angle: 2^-24
// turns at the largest position and a radian a position, about what the fp64 product of the two is off by. The fixed
// point adds 2^-65 turns a position, the cut to the upper 32 bits up to 2^-32.
// What bounds it: HBM at many tokens, the launch and the angles' chain at few. A batch is copied to shared memory while
// the one before it is worked on: loads into registers left none in flight meanwhile, and a second batch of registers
// spills at three blocks an SM. 16,384 tokens of 24 + 4 heads of 256, the keys dense and into a bf16 cache, 571 MB: 95
// us, 6.0 TB/s (116 us with loads into registers; 106 us with three blocks of 80 registers, which spill; 100 us one
// batch ahead instead of two; 96 us with 28 tokens a block instead of 16). A token's place in the pool is found once per
// block: with the page's division and the slot's load in every row, writing 16,384 tokens of 4 heads into an E4M3 cache,
// 101 MB, was bound by instructions, 24 us; now 18 us. 256 tokens with their queries: 4.1 us with two tokens a block,
// one block of each kind per SM; 5.4 us with one.
template <int D, bool kNorm, int kCache, int kRot>
__global__ void __launch_bounds__(kThreads, 2) rows_kernel(const RopeArgs p, const KvArgs c, int tokens_per_block) {
  __shared__ uint64_t freq[kNorm ? D / 2 : 1];
  __shared__ int place[kMaxTokens];
  extern __shared__ __align__(16) unsigned char stage[];  // [kBuffers][groups][kRows][D] bf16
  float2* turn = reinterpret_cast<float2*>(stage + kBuffers * kBatchBytes);  // [tokens][half]
  constexpr int kGroups = kThreads / (D / 8);
  const int t0 = blockIdx.x * tokens_per_block;
  const int T = min(tokens_per_block, p.T - t0);
  if constexpr (kNorm) {
    const int half = p.rotary / 2;
    if (half > 0) {
      for (int i = threadIdx.x; i < half; i += kThreads) {
        const double f = p.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi): turns per position
        freq[i] = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < T * half; i += kThreads) {
        const int64_t pos = p.positions[t0 + i / half];
        // the upper 32 bits as a signed number: half turns in [-1, 1)
        const int32_t top = (int32_t)(((uint64_t)pos * freq[i % half]) >> 32);
        // what the conversion to fp32 rounds off, up to 2^-25 half turns, turns sine and cosine on to first order
        const float half_turns = (float)top, off = (float)(top - (int32_t)half_turns) * 1.4629180792671596e-09f;  // pi 2^-31
        float s, co;
        sincospif(half_turns * 4.656612873077393e-10f, &s, &co);
        turn[i] = make_float2(fmaf(-s, off, co), fmaf(co, off, s));
      }
      __syncthreads();
    }
    if (blockIdx.y == 1) {
      if (p.Hq > kGroups) rows_pass<D, true, kNoCache, true, true, kRot>(p, c, turn, stage, place, t0, T, p.Hq);
      else rows_pass<D, true, kNoCache, true, false, kRot>(p, c, turn, stage, place, t0, T, p.Hq);
      return;
    }
  }
  rows_pass<D, kNorm, kCache, false, false, kRot>(p, c, turn, stage, place, t0, T, c.Hkv + (p.v ? c.Hkv : 0));
}

// Cached rows back to bf16: a block takes kReadTokens output tokens, a thread 16
// values of one (token, k or v, head) row at a time. A thread per token finds its
// request by bisection and its page in the table. Bound by HBM: 64 prefixes of up
// to 8192 tokens, E4M3, 518 MB: 80 us, 6.5 TB/s; one of 2047 tokens 4.5 us, the
// launch and the chain of two loads before the first row's.
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

template <int D, bool kNorm, int kCache, int kRot>
cudaError_t run(const RopeArgs& a, const KvArgs& c, dim3 grid, int per, cudaStream_t stream) {
  const int smem = kBuffers * kBatchBytes + (kNorm ? per * (a.rotary / 2) * (int)sizeof(float2) : 0);
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(&rows_kernel<D, kNorm, kCache, kRot>),
                                              kBuffers * kBatchBytes + kMaxTokens * D / 2 * (int)sizeof(float2));
  if (err != cudaSuccess) return err;
  rows_kernel<D, kNorm, kCache, kRot><<<grid, kThreads, smem, stream>>>(a, c, per);
  return cudaGetLastError();
}

template <int D, int kRot>
cudaError_t run_norm(const RopeArgs& a, const KvArgs& c, dim3 grid, int per, cudaStream_t stream) {
  if (!c.k) return run<D, true, kNoCache, kRot>(a, c, grid, per, stream);
  return c.e4m3 ? run<D, true, kE4m3Cache, kRot>(a, c, grid, per, stream)
                : run<D, true, kBf16Cache, kRot>(a, c, grid, per, stream);
}

template <int D>
cudaError_t run_rows(const RopeArgs& a, const KvArgs& c, bool norm, dim3 grid, int per, cudaStream_t stream) {
  if (norm) {
    if (a.interleaved) return run_norm<D, kInterleaved>(a, c, grid, per, stream);
    return a.rotary == D ? run_norm<D, kWhole>(a, c, grid, per, stream)
                         : run_norm<D, kPartial>(a, c, grid, per, stream);
  }
  return c.e4m3 ? run<D, false, kE4m3Cache, kPartial>(a, c, grid, per, stream)
                : run<D, false, kBf16Cache, kPartial>(a, c, grid, per, stream);
}

}  // namespace

cudaError_t launch_rows(const RopeArgs& a, const KvArgs& c, bool norm, int D, cudaStream_t stream) {
  // as many blocks (of each kind) as SMs, or the fewest whole multiples that keep a block at kMaxTokens, in fours
  const int most = 152 * kMaxTokens, waves = a.T / most + (a.T % most != 0), blocks = 152 * waves;
  int per = a.T / blocks + (a.T % blocks != 0);
  if (per > 4) per = (per + 3) / 4 * 4;
  const dim3 grid((unsigned)(((long long)a.T + per - 1) / per), norm && a.q ? 2 : 1, 1);
  return D == 256 ? run_rows<256>(a, c, norm, grid, per, stream) : run_rows<128>(a, c, norm, grid, per, stream);
}

cudaError_t launch_kv_read(const ReadArgs& a, const KvArgs& c, int D, cudaStream_t stream) {
  const unsigned grid = (unsigned)(((long long)a.T + kReadTokens - 1) / kReadTokens);
  if (D == 256) read_kernel<256><<<grid, kThreads, 0, stream>>>(a, c);
  else read_kernel<128><<<grid, kThreads, 0, stream>>>(a, c);
  return cudaGetLastError();
}

}  // namespace gdn
