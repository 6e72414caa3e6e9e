// Rotary positions in either pair layout over all or part of a head, and the
// append of rotated keys and of values to a paged cache (sm_103a).
//
// Pair i of a row at position p turns by p f_i.  The pair is (i, i + r/2)
// ("half") or (2i, 2i + 1) ("interleaved") of the head's first r dimensions;
// the others pass unchanged.
//
// The angle.  f_i / 2 pi, the turns per position, is kept as a 64-bit fraction
// of a turn: p times it modulo 2^64 is the angle modulo one turn, exactly, so
// that the wrap-around of an integer product is the whole range reduction.  The
// frequency is a float64, its turns rounded to that fraction: the angle of position
// 2^24 is off by at most 2^24 * 2^-65 turns.  The nearest quarter turn is taken off
// as an integer; sine and cosine of the eighth of a turn at most that remains
// are their Taylor sums in pairs of float32 (about 46 bits; this GPU does
// float64 at a small part of its float32 rate), so that the float32 factors are
// the ones nearest to the true values but for one in some thousands.
//
// The rotation and the head norm round every step once, in the order written
// in include/dsb.h, with no fused multiply-add: a 4-bit code next to a border
// is then the code that these steps define, on whatever path they are taken.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "dsb_kernels.h"
#include "dsb_ptx.cuh"
#include "dsb_q4.cuh"

namespace dsbk {

namespace {

template <int NP>
struct Turns {
  unsigned long long f[NP];  // turns per position of pair i, times 2^64
  float gain, gain_lo;       // every rotated value is multiplied by gain + gain_lo
  int rd;                    // rotated dimensions
  int interleaved;
};

// A value as the unevaluated sum of two float32, hi the nearest to it.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_mul(Two a, Two b) {
  const float p = __fmul_rn(a.hi, b.hi);
  float e = __fmaf_rn(a.hi, b.hi, -p);
  e = __fmaf_rn(a.hi, b.lo, e);
  e = __fmaf_rn(a.lo, b.hi, e);
  const float s = __fadd_rn(p, e);
  return Two{s, __fsub_rn(e, __fsub_rn(s, p))};
}
// c + x, |c| >= |x|
__device__ __forceinline__ Two two_add(Two c, Two x) {
  const float s = __fadd_rn(c.hi, x.hi);
  const float e = __fadd_rn(__fsub_rn(x.hi, __fsub_rn(s, c.hi)), __fadd_rn(c.lo, x.lo));
  const float r = __fadd_rn(s, e);
  return Two{r, __fsub_rn(e, __fsub_rn(r, s))};
}

__device__ __forceinline__ float2 turn_cs(unsigned long long f, int pos, float gain, float gain_lo) {
  const unsigned long long p = f * (unsigned long long)(unsigned)pos;
  const unsigned quarter = (unsigned)((p + (1ull << 61)) >> 62);
  const long long r = (long long)(p - ((unsigned long long)quarter << 62));  // [-2^61, 2^61)
  // t: the rest in half turns, at most 1/4; u = t^2
  Two t;
  t.hi = __ll2float_rn(r);
  t.lo = __fmul_rn(__ll2float_rn(r - __float2ll_rn(t.hi)), 0x1p-63f);
  t.hi = __fmul_rn(t.hi, 0x1p-63f);
  const Two u = two_mul(t, t);
  // sin(pi t) = t (pi - pi^3/3! u + pi^5/5! u^2 - ...), cos(pi t) alike; the terms
  // from u^3 on, below 2^-12 of the sum, in one float32
  float a = __fmaf_rn(0x1.e8f434p-12f, u.hi, -0x1.e30750p-8f);
  a = __fmaf_rn(a, u.hi, 0x1.507834p-4f);
  a = __fmaf_rn(a, u.hi, -0x1.32d2ccp-1f);
  Two s = two_add(Two{0x1.466bc6p+1f, 0x1.dd6ab8p-25f}, two_mul(u, Two{a, 0.0f}));
  s = two_add(Two{-0x1.4abbcep+2f, -0x1.896f94p-24f}, two_mul(u, s));
  s = two_add(Two{0x1.921fb6p+1f, -0x1.777a5cp-24f}, two_mul(u, s));
  s = two_mul(t, s);
  float b = __fmaf_rn(-0x1.b6e250p-14f, u.hi, 0x1.f9d38ap-10f);
  b = __fmaf_rn(b, u.hi, -0x1.a6d1f2p-6f);
  b = __fmaf_rn(b, u.hi, 0x1.e1f506p-3f);
  Two c = two_add(Two{-0x1.55d3c8p+0f, 0x1.c34006p-28f}, two_mul(u, Two{b, 0.0f}));
  c = two_add(Two{0x1.03c1f0p+2f, 0x1.036b58p-23f}, two_mul(u, c));
  c = two_add(Two{-0x1.3bd3ccp+2f, -0x1.37c8bcp-23f}, two_mul(u, c));
  c = two_add(Two{1.0f, 0.0f}, two_mul(u, c));
  if (quarter & 1) {
    const Two x = c;
    c = Two{-s.hi, -s.lo};
    s = x;
  }
  const float sign = quarter & 2 ? -1.0f : 1.0f;
  const Two g{__fmul_rn(sign, gain), __fmul_rn(sign, gain_lo)};
  return make_float2(two_mul(c, g).hi, two_mul(s, g).hi);
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float2 cs) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, cs.y));
  b = __fadd_rn(__fmul_rn(x, cs.y), __fmul_rn(y, cs.x));
}

constexpr int kRotThreads = 256;
constexpr int kRotUnroll = 4;  // pieces per thread, all loaded before the first is stored

// grid (n_tok, pieces / (256 * 4)).  A piece is four pairs (half layout: four
// values from each half), two pairs (interleaved) or, without VEC, one pair.
// In place: a pair is read and written by one thread.  The pairs' sines and
// cosines are worked out once per CTA while the loads are on their way.  Bound by
// memory: 6000 rows of 48 heads, 64 dimensions turned (147 MB): 25 us, 5.9 TB/s, 0.87
// of the copy rate.  One row: 4 us, a launch's latency.
template <int NP, bool VEC, int N>
__global__ void __launch_bounds__(kRotThreads) rope_rotary_kernel(float* __restrict__ q, long long q_stride, int hq,
                                                                  float* __restrict__ k, long long k_stride, int hkv,
                                                                  int head_dim,
                                                                  const __grid_constant__ Turns<NP> tab,
                                                                  int runs,
                                                                  const __grid_constant__ ParamWords<N> words,
                                                                  const int32_t* __restrict__ meta_dev) {
  __shared__ float2 cs[NP];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, half = tab.rd >> 1;
  const int per_head = !VEC ? half : tab.interleaved ? tab.rd >> 2 : tab.rd >> 3;
  const int pieces = (hq + hkv) * per_head;
  float* at[kRotUnroll];
  int first[kRotUnroll];  // the piece's first pair
  float4 a[kRotUnroll], b[kRotUnroll];
#pragma unroll
  for (int u = 0; u < kRotUnroll; ++u) {
    const int e = (blockIdx.y * kRotUnroll + u) * kRotThreads + threadIdx.x;
    at[u] = nullptr;
    if (e < pieces) {
      const int h = e / per_head, i = e - h * per_head;
      float* row = h < hq ? q + (size_t)t * q_stride + (size_t)h * head_dim
                          : k + (size_t)t * k_stride + (size_t)(h - hq) * head_dim;
      if (!VEC) {
        first[u] = i;
        at[u] = row + (tab.interleaved ? 2 * i : i);
        a[u].x = at[u][0];
        b[u].x = at[u][tab.interleaved ? 1 : half];
      } else if (tab.interleaved) {
        first[u] = 2 * i;
        at[u] = row + 4 * i;
        a[u] = *reinterpret_cast<const float4*>(at[u]);
      } else {
        first[u] = 4 * i;
        at[u] = row + 4 * i;
        a[u] = *reinterpret_cast<const float4*>(at[u]);
        b[u] = *reinterpret_cast<const float4*>(at[u] + half);
      }
    }
  }
  // the run of consecutive positions that token t is in
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  int lo = 0, hi = runs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (meta[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int pos = runs == 0 ? meta[t] : meta[runs + lo] + t - meta[lo];
  for (int i = threadIdx.x; i < half; i += kRotThreads) cs[i] = turn_cs(tab.f[i], pos, tab.gain, tab.gain_lo);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kRotUnroll; ++u) {
    if (!at[u]) continue;
    const float2* c = cs + first[u];
    if (!VEC) {
      turn_pair(a[u].x, b[u].x, c[0]);
      at[u][0] = a[u].x;
      at[u][tab.interleaved ? 1 : half] = b[u].x;
    } else if (tab.interleaved) {
      turn_pair(a[u].x, a[u].y, c[0]);
      turn_pair(a[u].z, a[u].w, c[1]);
      *reinterpret_cast<float4*>(at[u]) = a[u];
    } else {
      turn_pair(a[u].x, b[u].x, c[0]);
      turn_pair(a[u].y, b[u].y, c[1]);
      turn_pair(a[u].z, b[u].z, c[2]);
      turn_pair(a[u].w, b[u].w, c[3]);
      *reinterpret_cast<float4*>(at[u]) = a[u];
      *reinterpret_cast<float4*>(at[u] + half) = b[u];
    }
  }
}

// ---- append --------------------------------------------------------------------

// Small CTAs: a token's set-up (its sequence, page, sines and cosines) is a chain
// that others hide.  5178 tokens of 56 heads, append and read-back: 64 threads 61 us,
// 128 with 6, 7 or 8 CTAs an SM 62, 58 and 58, 256 62 (all as far as registers allow).
constexpr int kAppThreads = 128, kAppPerSm = 7;

// Two float32 operations at once, each rounded as by itself.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Not of two packed products: that would be compiled to a fused multiply-add, which
// rounds once less.
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Largest of a and b; NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Largest and smallest value over the D/8 lanes that hold a head (NaN where any is).
// Neighbours share the work: after the first exchange even lanes carry the largest,
// odd ones the smallest negated.
template <int D>
__device__ __forceinline__ void head_range(float& most, float& least, int lane) {
  const bool odd = lane & 1;
  const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? most : -least, 1);
  float v = max_nan(odd ? -least : most, other);
#pragma unroll
  for (int o = 2; o < D / 8; o <<= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  const float w = __shfl_xor_sync(0xFFFFFFFFu, v, 1);
  most = odd ? w : v;
  least = odd ? -v : -w;
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Sum of the squares of a head's D values, lane l of its D/8 holding values 4l ..
// and D/2 + 4l ...  The order is that of 32 running sums, the i-th over dimensions i,
// i + 32, ..., added pairwise, neighbours first.  D = 64: a lane holds both terms of
// four running sums; D = 128: two of the four terms, and an exchange with the lane
// that holds the others leaves two running sums to each.
template <int D>
__device__ __forceinline__ float sum_squares(const float (&y)[8], int lane) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; e += 2) unpack2(mul2(pack2(y[e], y[e + 1]), pack2(y[e], y[e + 1])), v[e], v[e + 1]);
  float ss;
  if constexpr (D == 128) {
    const bool up = lane & 8;
    float t[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float a = up ? v[e + 2] : v[e], b = up ? v[e + 6] : v[e + 4];
      const float a1 = __shfl_xor_sync(0xFFFFFFFFu, up ? v[e] : v[e + 2], 8);
      const float b1 = __shfl_xor_sync(0xFFFFFFFFu, up ? v[e + 4] : v[e + 6], 8);
      t[e] = __fadd_rn(__fadd_rn(__fadd_rn(a, a1), up ? b1 : b), up ? b : b1);
    }
    ss = __fadd_rn(t[0], t[1]);
    ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, 8));
  } else {
    ss = __fadd_rn(__fadd_rn(__fadd_rn(v[0], v[4]), __fadd_rn(v[1], v[5])),
                   __fadd_rn(__fadd_rn(v[2], v[6]), __fadd_rn(v[3], v[7])));
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, o));
  return ss;
}

// How the cache rows are stored.
struct StoreQ4 {};

// The eight 4-bit codes of y / d about z.  The quotient by the reciprocal, held to
// the codes' range, is within 2^-20 of the rounded quotient; only where it lies
// closer than that to a half does the code need the division itself.  Adding 1.5 2^23
// (and the code's 8) rounds to the nearest integer, ties to even, and leaves the code
// in the low bits.
__device__ __forceinline__ uint32_t q4_codes(const float (&y)[8], float d, float z) {
  constexpr float kRound = 12582920.0f;
  const float inv = __frcp_rn(d);
  const f2 inv2 = pack2(inv, inv), z2 = pack2(-z, -z), up = pack2(kRound, kRound), down = pack2(-kRound, -kRound);
  uint32_t code = 0;
  bool near = false;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    float v0, v1, t0, t1, r0, r1;
    unpack2(mul2(add2(pack2(y[e], y[e + 1]), z2), inv2), v0, v1);
    v0 = fminf(fmaxf(v0, -8.0f), 7.0f);
    v1 = fminf(fmaxf(v1, -8.0f), 7.0f);
    const f2 t = add2(pack2(v0, v1), up);
    const f2 n = add2(t, down);
    unpack2(t, t0, t1);
    unpack2(n, r0, r1);
    near |= !(fabsf(fabsf(v0 - r0) - 0.5f) > 0x1p-18f) || !(fabsf(fabsf(v1 - r1) - 0.5f) > 0x1p-18f);
    code += __float_as_uint(t0) << (4 * e);
    code += __float_as_uint(t1) << (4 * e + 4);
  }
  // the bits above the codes, the same in each
  constexpr uint32_t kBits = 0x4B400000u;
  code -= kBits * 0x11111111u;
  if (near) {
    code = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float n = rintf(__fdiv_rn(__fsub_rn(y[e], z), d));
      code |= (uint32_t)(int)fminf(fmaxf(n + 8.0f, 0.0f), 15.0f) << (4 * e);
    }
  }
  return d == 0.0f ? 0x88888888u : code;
}

// grid (n_tok, shares of the heads): D/8 lanes hold one head's vector, eight values
// each: four of its first half and the four at the same place of its second, so that a
// rotated value's partner is in the lane (both pair layouts, the whole head rotated; else
// it is fetched from shared memory) and norm and extremes stay inside a warp.  A lane
// handles the same dimensions of one head after the other, the next one's values on
// their way, with one set of sines and cosines.  Head h of the row: query heads, then
// key heads, then value heads.  With many tokens one CTA takes all heads of its token,
// so the token's set-up is paid once.  Those 5178 tokens read and write 266 MB (39 us at
// the copy rate) in 45 us, with 0.71 of the issue slots full: the token's set-up and the
// shuffles wait.  Into 16-bit pages (276 MB) they take 1 us less.  16 tokens: 4.5 us, the
// latency of the chain.
// Metadata: tok_off[n + 1] | pos0[n] | pg_off[n + 1] | pages of every sequence,
// from the page of its first new key on.
template <int D, typename Store, int N>
__global__ void __launch_bounds__(kAppThreads, kAppPerSm)
    kv_append_kernel(float* __restrict__ qkv, long long stride, int hq, int hkv, uint8_t* __restrict__ kc,
                     uint8_t* __restrict__ vc, const __grid_constant__ Turns<64> tab, const float* __restrict__ q_norm,
                     const float* __restrict__ k_norm, float eps, int n_seq,
                     const __grid_constant__ ParamWords<N> words, const int32_t* __restrict__ meta_dev) {
  constexpr int LPH = D / 8, SLOTS = kAppThreads / LPH;
  __shared__ __align__(16) float cosines[D], sines[D];  // of every dimension; a sine with the sign its term takes
  __shared__ __align__(16) float swap[kAppThreads * 8];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, tid = threadIdx.x, l = tid & (LPH - 1), slot = tid / LPH;
  const int heads = hq + 2 * hkv, rd = tab.rd, half = rd >> 1;
  const int d0 = 4 * l, d1 = D / 2 + 4 * l;  // the lane's dimensions
  // query values past the rotated part stay where they are
  const bool touched0 = q_norm || d0 < rd, touched1 = q_norm || d1 < rd;
  float* row = qkv + (size_t)t * stride;
  float4 x[2];
  auto fetch = [&](int h) {
    x[0] = x[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (h < heads && (h >= hq || touched0)) x[0] = __ldcg(reinterpret_cast<const float4*>(row + h * D + d0));
    if (h < heads && (h >= hq || touched1)) x[1] = __ldcg(reinterpret_cast<const float4*>(row + h * D + d1));
  };
  int h = blockIdx.y * SLOTS + slot;
  fetch(h);
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  int lo = 0, hi = n_seq - 1;  // the sequence of token t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (meta[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int pos0 = meta[n_seq + 1 + lo], pos = pos0 + t - meta[lo];
  const int32_t* pg_off = meta + 2 * n_seq + 1;
  const int page = pg_off[n_seq + 1 + pg_off[lo] + (pos >> 7) - (pos0 >> 7)];
  const int r = pos & 127;
  for (int i = tid; i < half; i += kAppThreads) {
    const float2 v = turn_cs(tab.f[i], pos, tab.gain, tab.gain_lo);
    const int a = tab.interleaved ? 2 * i : i, b = tab.interleaved ? a + 1 : a + half;
    cosines[a] = cosines[b] = v.x;
    sines[a] = -v.y;
    sines[b] = v.y;
  }
  for (int i = rd + tid; i < D; i += kAppThreads) {
    cosines[i] = 1.0f;
    sines[i] = 0.0f;
  }
  __syncthreads();
  const int turned0 = min(max(rd - d0, 0), 4), turned1 = min(max(rd - d1, 0), 4);  // of its dimensions
  const bool whole = rd == D;
  const float4 c[2] = {*reinterpret_cast<const float4*>(&cosines[d0]), *reinterpret_cast<const float4*>(&cosines[d1])};
  const float4 s[2] = {*reinterpret_cast<const float4*>(&sines[d0]), *reinterpret_cast<const float4*>(&sines[d1])};
  for (;;) {
    const bool live = h < heads, is_q = h < hq, is_k = !is_q && h < hq + hkv, is_v = live && !is_q && !is_k;
    float y[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    const int next = h + gridDim.y * SLOTS;
    if (next - slot < heads) fetch(next);
    const float* norm = is_q ? q_norm : is_k ? k_norm : nullptr;
    if (__any_sync(0xFFFFFFFFu, norm != nullptr)) {
      const float ss = sum_squares<D>(y, tid & 31);
      if (norm) {
        const float inv = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / D), eps));
        const f2 inv2 = pack2(inv, inv);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(norm + (e ? d1 : d0)));
          unpack2(mul2(mul2(pack2(y[e], y[e + 1]), inv2), pack2(w.x, w.y)), y[e], y[e + 1]);
          unpack2(mul2(mul2(pack2(y[e + 2], y[e + 3]), inv2), pack2(w.z, w.w)), y[e + 2], y[e + 3]);
        }
      }
    }
    if (__any_sync(0xFFFFFFFFu, live && !is_v)) {
      float p[8];
      if (tab.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = y[e ^ 1];
      } else if (whole) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = y[e ^ 4];
      } else {
        float* mine = swap + slot * D;
        __syncwarp();
        *reinterpret_cast<float4*>(mine + d0) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4*>(mine + d1) = make_float4(y[4], y[5], y[6], y[7]);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int dim = e < 4 ? d0 + e : d1 + e - 4;
          p[e] = mine[dim >= rd ? dim : dim >= half ? dim - half : dim + half];
        }
      }
      if (!is_v) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float a[4], b[4];
          unpack2(mul2(pack2(y[4 * i], y[4 * i + 1]), pack2(c[i].x, c[i].y)), a[0], a[1]);
          unpack2(mul2(pack2(y[4 * i + 2], y[4 * i + 3]), pack2(c[i].z, c[i].w)), a[2], a[3]);
          unpack2(mul2(pack2(p[4 * i], p[4 * i + 1]), pack2(s[i].x, s[i].y)), b[0], b[1]);
          unpack2(mul2(pack2(p[4 * i + 2], p[4 * i + 3]), pack2(s[i].z, s[i].w)), b[2], b[3]);
          if (whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[4 * i + e] = __fadd_rn(a[e], b[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[4 * i + e] = e < (i ? turned1 : turned0) ? __fadd_rn(a[e], b[e]) : y[4 * i + e];
          }
        }
      }
    }
    if (is_q && touched0) *reinterpret_cast<float4*>(row + h * D + d0) = make_float4(y[0], y[1], y[2], y[3]);
    if (is_q && touched1) *reinterpret_cast<float4*>(row + h * D + d1) = make_float4(y[4], y[5], y[6], y[7]);
    const int g = h - hq - (is_k ? 0 : hkv);  // kv head
    if constexpr (std::is_same<Store, StoreQ4>::value) {
      if (__any_sync(0xFFFFFFFFu, live && !is_q)) {
        float most = max_nan(max_nan(max_nan(y[0], y[1]), max_nan(y[2], y[3])),
                             max_nan(max_nan(y[4], y[5]), max_nan(y[6], y[7])));
        float least = -max_nan(max_nan(max_nan(-y[0], -y[1]), max_nan(-y[2], -y[3])),
                               max_nan(max_nan(-y[4], -y[5]), max_nan(-y[6], -y[7])));
        head_range<D>(most, least, tid & 31);
        const float span = __fsub_rn(most, least);
        __half dh = __float2half_rn(__fmul_rn(span, 1.0f / 15.0f));
        __half zh = __float2half_rn(__fadd_rn(least, __fmul_rn(8.0f, __half2float(dh))));
        if (!(span <= FLT_MAX)) {  // a vector with a NaN or an infinity is stored as NaN
          dh = __ushort_as_half(0);
          zh = __ushort_as_half(0x7FFF);
        }
        if (live && !is_q) {
          const uint32_t code = q4_codes(y, __half2float(dh), __half2float(zh));
          using B = Q4Block<D>;
          uint8_t* blk = kc + ((size_t)page * hkv + g) * B::bytes;
          // 16 bits of codes for four dimensions; V's words hold a key pair's
          uint8_t* dst = is_k ? blk + r * (D / 2) + d0 / 2 : blk + B::v + (r >> 1) * D + d0 + 2 * (r & 1);
          *reinterpret_cast<uint16_t*>(dst) = (uint16_t)code;
          *reinterpret_cast<uint16_t*>(dst + (is_k ? D / 4 : D / 2)) = (uint16_t)(code >> 16);
          if (l == 0) *reinterpret_cast<__half2*>(blk + (is_k ? B::kz : B::vz) + 4 * r) = __halves2half2(dh, zh);
        }
      }
    } else {
      if (live && !is_q) {
        uint8_t* dst = (is_k ? kc : vc) + ((((size_t)page * hkv + g) * kQ4Page + r) * D + d0) * 2;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<Store>(y[0], y[1]), pack16<Store>(y[2], y[3]));
        *reinterpret_cast<uint2*>(dst + D) = make_uint2(pack16<Store>(y[4], y[5]), pack16<Store>(y[6], y[7]));
      }
    }
    h = next;
    if (h - slot >= heads) break;
  }
}

template <int NP>
void fill_turns(const RotaryTable& rot, Turns<NP>* out) {
  for (int i = 0; i < NP; ++i) out->f[i] = i < rot.rd / 2 ? rot.turns[i] : 0;
  out->gain = (float)rot.gain;
  out->gain_lo = (float)(rot.gain - (double)out->gain);
  out->rd = rot.rd;
  out->interleaved = rot.interleaved;
}

template <int NP, bool VEC, int N>
cudaError_t rope_go(float* q, long long q_stride, int hq, float* k, long long k_stride, int hkv, int head_dim, int n_tok,
                    const RotaryTable& rot, int runs, const MetaArg& meta, cudaStream_t st) {
  Turns<NP> tab;
  fill_turns(rot, &tab);
  ParamWords<N> w;
  fill_words(meta, &w);
  const int per_head = !VEC ? rot.rd / 2 : rot.interleaved ? rot.rd / 4 : rot.rd / 8;
  const long long pieces = (long long)(hq + hkv) * per_head;
  const unsigned gy = (unsigned)((pieces + kRotThreads * kRotUnroll - 1) / (kRotThreads * kRotUnroll));
  return launch_kernel(rope_rotary_kernel<NP, VEC, N>, dim3((unsigned)n_tok, gy), dim3(kRotThreads), 0, st, q, q_stride,
                       hq, k, k_stride, hkv, head_dim, tab, runs, w, meta.dev);
}

template <int NP, int N>
cudaError_t rope_vec(float* q, long long q_stride, int hq, float* k, long long k_stride, int hkv, int head_dim,
                     int n_tok, const RotaryTable& rot, int runs, const MetaArg& meta, cudaStream_t st) {
  // 16-byte pieces where every head starts on 16 bytes and the rotated part is
  // a whole number of pieces
  const bool vec = head_dim % 4 == 0 && q_stride % 4 == 0 && k_stride % 4 == 0 &&
                   rot.rd % (rot.interleaved ? 4 : 8) == 0;
  return vec ? rope_go<NP, true, N>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, runs, meta, st)
             : rope_go<NP, false, N>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, runs, meta, st);
}

template <int D, typename Store, int N>
cudaError_t append_go(const AppendArgs& a, const RotaryTable& rot, const MetaArg& meta, cudaStream_t st) {
  Turns<64> tab;
  fill_turns(rot, &tab);
  ParamWords<N> w;
  fill_words(meta, &w);
  // as many shares of a token's heads as fill the GPU, no more than there are
  const int slots = kAppThreads / (D / 8), most = (a.hq + 2 * a.hkv + slots - 1) / slots;
  const int shares = std::min(most, std::max(1, kAppPerSm * a.sms / a.n_tok));
  const dim3 grid((unsigned)a.n_tok, (unsigned)shares);
  return launch_kernel(kv_append_kernel<D, Store, N>, grid, dim3(kAppThreads), 0, st, a.qkv, a.stride, a.hq, a.hkv,
                       static_cast<uint8_t*>(a.kc), static_cast<uint8_t*>(a.vc), tab, a.q_norm, a.k_norm, a.eps, a.n_seq,
                       w, meta.dev);
}

template <int D, typename Store>
cudaError_t append_pick(const AppendArgs& a, const RotaryTable& rot, const MetaArg& meta, cudaStream_t st) {
  return with_words(meta, [&](auto n) { return append_go<D, Store, decltype(n)::value>(a, rot, meta, st); });
}

}  // namespace

cudaError_t launch_rope_rotary(float* q, long long q_stride, int hq, float* k, long long k_stride, int hkv, int head_dim,
                               int n_tok, const RotaryTable& rot, int runs, const MetaArg& meta, cudaStream_t st) {
  if (n_tok == 0) return cudaSuccess;
  return with_words(meta, [&](auto n) {
    constexpr int N = decltype(n)::value;
    return rot.rd <= 128 ? rope_vec<64, N>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, runs, meta, st)
                         : rope_vec<kRopeMaxPairs, N>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, runs, meta, st);
  });
}

cudaError_t launch_kv_append(const AppendArgs& a, int head_dim, KvStore store, const RotaryTable& rot,
                             const MetaArg& meta, cudaStream_t st) {
  if (a.n_tok == 0) return cudaSuccess;
  if (head_dim == 128) {
    if (store == KvStore::kQ4) return append_pick<128, StoreQ4>(a, rot, meta, st);
    return store == KvStore::kF16 ? append_pick<128, __half>(a, rot, meta, st)
                                  : append_pick<128, __nv_bfloat16>(a, rot, meta, st);
  }
  if (head_dim == 64) {
    if (store == KvStore::kQ4) return append_pick<64, StoreQ4>(a, rot, meta, st);
    return store == KvStore::kF16 ? append_pick<64, __half>(a, rot, meta, st)
                                  : append_pick<64, __nv_bfloat16>(a, rot, meta, st);
  }
  return cudaErrorInvalidValue;
}

// Turns per position as 64-bit fractions, the nearest to freq / 2 pi: that quotient
// in two float64 (one is 2^-53 of it off, 2^-30 of a turn at position 2^24: there one
// factor in a hundred would not be the nearest float32).  Only the fraction of a turn
// counts, because positions are whole numbers.
void rotary_table(const double* freq, int rd, bool interleaved, double gain, RotaryTable* out) {
  constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLo = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
  out->rd = rd;
  out->interleaved = interleaved ? 1 : 0;
  out->gain = gain;
  for (int i = 0; i < rd / 2; ++i) {
    double hi = freq[i] * kTurn;
    double lo = std::fma(freq[i], kTurn, -hi) + freq[i] * kTurnLo;
    hi -= std::floor(hi);
    lo -= std::rint(lo);  // of turns from 2^52 on
    hi *= 0x1p64;
    const double whole = std::floor(hi);
    lo = lo * 0x1p64 + (hi - whole);
    // whole < 2^64; |lo| <= 2^63, halved before its conversion where it is that large
    const unsigned long long rest = std::fabs(lo) < 0x1p62 ? (unsigned long long)std::llrint(lo)
                                                           : 2ull * (unsigned long long)std::llrint(0.5 * lo);
    out->turns[i] = (unsigned long long)whole + rest;
  }
}

}  // namespace dsbk
