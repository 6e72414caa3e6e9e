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
// frequency is a float64 rounded to that fraction: the angle of position 2^24
// is off by at most 2^24 * 2^-53 turns.  The nearest quarter turn is taken off
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
// cosines are worked out once per CTA while the loads are on their way.
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

constexpr int kAppThreads = 256;

// Two float32 products at once, each rounded as by itself.
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

// Largest of a and b; NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Over the D/4 lanes that hold a head.
template <int D>
__device__ __forceinline__ float head_max_nan(float v) {
  if constexpr (D == 128) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int o = D / 8; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  }
}
// Whether any head of the warp is concerned; a warp holds one head at D = 128.
template <int D>
__device__ __forceinline__ bool warp_any(bool x) {
  return D == 128 ? x : __any_sync(0xFFFFFFFFu, x);
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

// Sum of the squares of a head's D values, lane l of its D/4 holding values
// 4l .. 4l+3.  The order is that of 32 running sums, the i-th over dimensions i,
// i + 32, ..., added pairwise, neighbours first.  D = 128: the four terms of a
// running sum sit 8 lanes apart; a transpose of the 4 x 4 (lane group, element)
// brings them into one lane, the i-th group taking element i.  D = 64: two terms,
// half of the elements to each group.
template <int D>
__device__ __forceinline__ float sum_squares(const float (&y)[4], int lane) {
  float v[4];
  unpack2(mul2(pack2(y[0], y[1]), pack2(y[0], y[1])), v[0], v[1]);
  unpack2(mul2(pack2(y[2], y[3]), pack2(y[2], y[3])), v[2], v[3]);
  float ss;
  if constexpr (D == 128) {
    const bool up = lane & 16, odd = lane & 8;
    const float a = __shfl_xor_sync(0xFFFFFFFFu, up ? v[0] : v[2], 16);
    const float b = __shfl_xor_sync(0xFFFFFFFFu, up ? v[1] : v[3], 16);
    if (up) {
      v[0] = a, v[1] = b;
    } else {
      v[2] = a, v[3] = b;
    }
    const float c = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[0] : v[1], 8);
    const float d = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[2] : v[3], 8);
    if (odd) {
      v[0] = c, v[2] = d;
    } else {
      v[1] = c, v[3] = d;
    }
    ss = __fadd_rn(__fadd_rn(__fadd_rn(v[0], v[1]), v[2]), v[3]);
    ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, 8));
    ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, 16));
  } else {
    const bool odd = lane & 8;
    const float a = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[0] : v[2], 8);
    const float b = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[1] : v[3], 8);
    ss = odd ? __fadd_rn(__fadd_rn(v[2], a), __fadd_rn(v[3], b)) : __fadd_rn(__fadd_rn(v[0], a), __fadd_rn(v[1], b));
    ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, 8));
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, o));
  return ss;
}

// How the cache rows are stored.
struct StoreQ4 {};

// grid (n_tok, shares of the heads), 256 threads: D/4 lanes hold one head's vector,
// four values each, so that its norm, its extremes and the partner of a rotated
// value stay inside a warp.  A lane handles the same four dimensions of one head
// after the other, HPS of them loaded before the first is used, with one set of
// sines and cosines.  Head h of the row: query heads, then key heads, then value
// heads.  With many tokens one CTA takes all heads of its token: the kernel is
// bound by instruction issue (a prompt of 5178 tokens of 56 heads: 254 MB, 78 us
// and 253 instructions a head before, see the launch for the time now), so the
// token's set-up is paid once.
// Metadata: tok_off[n + 1] | pos0[n] | pg_off[n + 1] | pages of every sequence,
// from the page of its first new key on.
template <int D, typename Store, int HPS, int N>
__global__ void __launch_bounds__(kAppThreads, 4) kv_append_kernel(float* __restrict__ qkv, long long stride, int hq,
                                                                int hkv, uint8_t* __restrict__ kc,
                                                                uint8_t* __restrict__ vc,
                                                                const __grid_constant__ Turns<64> tab,
                                                                const float* __restrict__ q_norm,
                                                                const float* __restrict__ k_norm, float eps, int n_seq,
                                                                const __grid_constant__ ParamWords<N> words,
                                                                const int32_t* __restrict__ meta_dev) {
  constexpr int LPH = D / 4, SLOTS = kAppThreads / LPH;
  __shared__ float2 cs[D / 2];
  __shared__ float swap[kAppThreads * 4];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, tid = threadIdx.x, l = tid & (LPH - 1), slot = tid / LPH;
  const int heads = hq + 2 * hkv, rd = tab.rd, half = rd >> 1;
  const bool touched = q_norm || 4 * l < rd;  // query values past the rotated part stay where they are
  float* row = qkv + (size_t)t * stride + 4 * l;
  float4 x[HPS];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int u = 0; u < HPS; ++u) {
      const int h = h0 + u * SLOTS;
      x[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (h < heads && (h >= hq || touched)) x[u] = __ldcg(reinterpret_cast<const float4*>(row + h * D));
    }
  };
  fetch(blockIdx.y * (HPS * SLOTS) + slot);
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
  if (tid < half) cs[tid] = turn_cs(tab.f[tid], pos, tab.gain, tab.gain_lo);
  __syncthreads();
  float c[4], s[4];  // of this lane's four dimensions; s with the sign its term takes
  bool turned[4];
  int partner[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int dim = 4 * l + e;
    c[e] = 1.0f;
    s[e] = 0.0f;
    partner[e] = dim;
    turned[e] = dim < rd;
    if (turned[e]) {
      const bool second = tab.interleaved ? (dim & 1) : dim >= half;
      const float2 v = cs[tab.interleaved ? dim >> 1 : second ? dim - half : dim];
      c[e] = v.x;
      s[e] = second ? v.y : -v.y;
      partner[e] = tab.interleaved ? dim ^ 1 : second ? dim - half : dim + half;
    }
  }
  const int src = (tid & 31 & ~(LPH - 1)) + (partner[0] >> 2);  // lane of the partners, half layout in whole lanes
  const bool lanes = (rd & 7) == 0, all = rd == D;
  const float4 qw = q_norm ? __ldg(reinterpret_cast<const float4*>(q_norm) + l) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 kw = k_norm ? __ldg(reinterpret_cast<const float4*>(k_norm) + l) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int h0 = blockIdx.y * (HPS * SLOTS) + slot;; ) {
#pragma unroll
    for (int u = 0; u < HPS; ++u) {
      const int h = h0 + u * SLOTS;
      if (D == 128 && h >= heads) break;
      const bool live = h < heads, is_q = h < hq, is_k = !is_q && h < hq + hkv, is_v = live && !is_q && !is_k;
      float y[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      const bool normed = (is_q && q_norm) || (is_k && k_norm);
      if (warp_any<D>(normed)) {
        const float ss = sum_squares<D>(y, tid & 31);
        if (normed) {
          const float inv = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / D), eps));
          const float4 wv = is_q ? qw : kw;
          const f2 inv2 = pack2(inv, inv);
          unpack2(mul2(mul2(pack2(y[0], y[1]), inv2), pack2(wv.x, wv.y)), y[0], y[1]);
          unpack2(mul2(mul2(pack2(y[2], y[3]), inv2), pack2(wv.z, wv.w)), y[2], y[3]);
        }
      }
      if (warp_any<D>(live && !is_v)) {
        float p[4];
        if (tab.interleaved) {
          p[0] = y[1], p[1] = y[0], p[2] = y[3], p[3] = y[2];
        } else if (lanes) {
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = __shfl_sync(0xFFFFFFFFu, y[e], src);
        } else {
          float* mine = swap + slot * D;
          __syncwarp();
          *reinterpret_cast<float4*>(mine + 4 * l) = make_float4(y[0], y[1], y[2], y[3]);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = mine[partner[e]];
        }
        if (!is_v) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            // the sums one by one: a packed sum of packed products is compiled to a
            // fused multiply-add, which rounds once less
            float a0, a1, b0, b1;
            unpack2(mul2(pack2(y[e], y[e + 1]), pack2(c[e], c[e + 1])), a0, a1);
            unpack2(mul2(pack2(p[e], p[e + 1]), pack2(s[e], s[e + 1])), b0, b1);
            const float z0 = __fadd_rn(a0, b0), z1 = __fadd_rn(a1, b1);
            y[e] = all || turned[e] ? z0 : y[e];
            y[e + 1] = all || turned[e + 1] ? z1 : y[e + 1];
          }
        }
      }
      if (is_q && touched) *reinterpret_cast<float4*>(row + h * D) = make_float4(y[0], y[1], y[2], y[3]);
      const int g = h - hq - (is_k ? 0 : hkv);  // kv head
      if constexpr (std::is_same<Store, StoreQ4>::value) {
        if (!warp_any<D>(live && !is_q)) continue;
        const float most = head_max_nan<D>(max_nan(max_nan(y[0], y[1]), max_nan(y[2], y[3])));
        const float least = -head_max_nan<D>(max_nan(max_nan(-y[0], -y[1]), max_nan(-y[2], -y[3])));
        const float span = __fsub_rn(most, least);
        __half dh = __float2half_rn(__fmul_rn(span, 1.0f / 15.0f));
        __half zh = __float2half_rn(__fadd_rn(least, __fmul_rn(8.0f, __half2float(dh))));
        if (!(span <= FLT_MAX)) {  // a vector with a NaN or an infinity is stored as NaN
          dh = __ushort_as_half(0);
          zh = __ushort_as_half(0x7FFF);
        }
        const float d = __half2float(dh), z = __half2float(zh);
        // The quotient by the reciprocal, at most 8, is within 2^-20 of the rounded
        // quotient; only where it lies closer than that to a half does the code
        // need the division itself.
        const float inv = __frcp_rn(d);
        uint32_t code = 0;
        bool near = false;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = __fmul_rn(__fsub_rn(y[e], z), inv);
          const float n = rintf(v[e]);
          near |= !(fabsf(fabsf(v[e] - n) - 0.5f) > 0x1p-18f);
          v[e] = n;
        }
        if (near) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = rintf(__fdiv_rn(__fsub_rn(y[e], z), d));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) code |= (uint32_t)(int)fminf(fmaxf(v[e] + 8.0f, 0.0f), 15.0f) << (4 * e);
        if (d == 0.0f) code = 0x8888u;
        if (live && !is_q) {
          using B = Q4Block<D>;
          uint8_t* blk = kc + ((size_t)page * hkv + g) * B::bytes;
          uint8_t* dst = is_k ? blk + r * (D / 2) + 2 * l : blk + B::v + (r >> 1) * D + 4 * l + 2 * (r & 1);
          *reinterpret_cast<uint16_t*>(dst) = (uint16_t)code;
          if (l == 0) *reinterpret_cast<__half2*>(blk + (is_k ? B::kz : B::vz) + 4 * r) = __halves2half2(dh, zh);
        }
      } else {
        if (live && !is_q) {
          uint8_t* dst = (is_k ? kc : vc) + ((((size_t)page * hkv + g) * kQ4Page + r) * D + 4 * l) * 2;
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<Store>(y[0], y[1]), pack16<Store>(y[2], y[3]));
        }
      }
    }
    h0 += gridDim.y * (HPS * SLOTS);
    if (h0 - slot >= heads) break;
    fetch(h0);
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

template <int D, typename Store, int HPS, int N>
cudaError_t append_go(const AppendArgs& a, const RotaryTable& rot, const MetaArg& meta, cudaStream_t st) {
  Turns<64> tab;
  fill_turns(rot, &tab);
  ParamWords<N> w;
  fill_words(meta, &w);
  // as many shares of a token's heads as fill the GPU (8 CTAs on each of some 150
  // SMs), no more than there are
  const int slots = kAppThreads / (D / 4) * HPS, most = (a.hq + 2 * a.hkv + slots - 1) / slots;
  const int shares = std::min(most, std::max(1, 1200 / a.n_tok));
  const dim3 grid((unsigned)a.n_tok, (unsigned)shares);
  return launch_kernel(kv_append_kernel<D, Store, HPS, N>, grid, dim3(kAppThreads), 0, st, a.qkv, a.stride, a.hq, a.hkv,
                       static_cast<uint8_t*>(a.kc), static_cast<uint8_t*>(a.vc), tab, a.q_norm, a.k_norm, a.eps, a.n_seq,
                       w, meta.dev);
}

template <int D, typename Store>
cudaError_t append_pick(const AppendArgs& a, const RotaryTable& rot, const MetaArg& meta, cudaStream_t st) {
  // few tokens: one head per lane group, the most CTAs; else four
  const bool few = a.n_tok <= 64;
  return with_words(meta, [&](auto n) {
    constexpr int N = decltype(n)::value;
    return few ? append_go<D, Store, 1, N>(a, rot, meta, st) : append_go<D, Store, 4, N>(a, rot, meta, st);
  });
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

// Turns per position as 64-bit fractions; only the fraction of a turn counts,
// because positions are whole numbers.
void rotary_table(const double* freq, int rd, bool interleaved, double gain, RotaryTable* out) {
  out->rd = rd;
  out->interleaved = interleaved ? 1 : 0;
  out->gain = gain;
  for (int i = 0; i < rd / 2; ++i) {
    double turns = freq[i] * 0.15915494309189533577;
    turns -= std::floor(turns);
    const double scaled = std::ldexp(turns, 64);
    out->turns[i] = scaled >= 18446744073709551616.0 ? 0ull : (unsigned long long)scaled;
  }
}

}  // namespace dsbk
