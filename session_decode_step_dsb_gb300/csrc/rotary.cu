// Rotary positions in either pair layout over all or part of a head, and the
// append of rotated keys and of values to a paged cache (sm_103a).
//
// Pair i of a row at position p turns by p f_i.  The pair is (i, i + r/2)
// ("half") or (2i, 2i + 1) ("interleaved") of the head's first r dimensions;
// the others pass unchanged.
//
// The angle.  f_i / 2 pi, the turns per position, is kept as a 64-bit fraction
// of a turn: p times it modulo 2^64 is the angle modulo one turn, exactly, so
// that the wrap-around of an integer product is the whole range reduction (no
// float64 work, which this GPU does at a small part of its float32 rate).  The frequency is
// a float64 rounded to that fraction: the angle of position 2^24 is off by at
// most 2^24 * 2^-53 turns.  The nearest quarter turn is taken off as an
// integer, and the sine and cosine of the remaining eighth of a turn at most
// are a float32 sincospif.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

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
  float gain;                // every rotated value is multiplied by it
  int rd;                    // rotated dimensions
  int interleaved;
};

__device__ __forceinline__ float2 turn_cs(unsigned long long f, int pos, float gain) {
  const unsigned long long p = f * (unsigned long long)(unsigned)pos;
  const unsigned quarter = (unsigned)((p + (1ull << 61)) >> 62);
  const long long r = (long long)(p - ((unsigned long long)quarter << 62));  // [-2^61, 2^61)
  float s, c;
  sincospif((float)(int)(r >> 30) * 0x1p-33f, &s, &c);
  float2 o = make_float2(c, s);
  if (quarter & 1) o = make_float2(-s, c);
  if (quarter & 2) o = make_float2(-o.x, -o.y);
  return make_float2(__fmul_rn(o.x, gain), __fmul_rn(o.y, gain));
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float2 cs) {
  const float x = a, y = b;
  a = __fmaf_rn(x, cs.x, __fmul_rn(-y, cs.y));
  b = __fmaf_rn(x, cs.y, __fmul_rn(y, cs.x));
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
                                                                  const __grid_constant__ ParamWords<N> words,
                                                                  const int32_t* __restrict__ pos_dev) {
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
  const int pos = N > 1 ? words.w[t] : pos_dev[t];
  for (int i = threadIdx.x; i < half; i += kRotThreads) cs[i] = turn_cs(tab.f[i], pos, tab.gain);
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

__device__ __forceinline__ float lanes_max(float v, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
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

// How the cache rows are stored.
struct StoreQ4 {};

// grid (n_tok, groups of heads), 256 threads: D/4 lanes hold one head's vector,
// four values each, so that its norm, its extremes and the partner of a rotated
// value stay inside a warp.  A lane handles the same four dimensions of HPS
// heads, all loaded before the first is used, with one set of sines and cosines.
// Head h of the row: query heads, then key heads, then value heads.
// Metadata: tok_off[n + 1] | pos0[n] | pg_off[n + 1] | pages of every sequence,
// from the page of its first new key on.
template <int D, typename Store, int HPS, int N>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(float* __restrict__ qkv, long long stride, int hq,
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
  float* row = qkv + (size_t)t * stride;
  float4 x[HPS];
  const int h0 = blockIdx.y * (HPS * SLOTS) + slot;
#pragma unroll
  for (int u = 0; u < HPS; ++u) {
    const int h = h0 + u * SLOTS;
    x[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // query values past the rotated part stay where they are
    if (h < heads && (h >= hq || q_norm || 4 * l < rd))
      x[u] = __ldcg(reinterpret_cast<const float4*>(row + (size_t)h * D) + l);
  }
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
  if (tid < half) cs[tid] = turn_cs(tab.f[tid], pos, tab.gain);
  __syncthreads();
  float c[4], s[4];  // of this lane's four dimensions; s with the sign its term takes
  int partner[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int dim = 4 * l + e;
    c[e] = 1.0f;
    s[e] = 0.0f;
    partner[e] = dim;
    if (dim < rd) {
      const bool second = tab.interleaved ? (dim & 1) : dim >= half;
      const float2 v = cs[tab.interleaved ? dim >> 1 : second ? dim - half : dim];
      c[e] = v.x;
      s[e] = second ? v.y : -v.y;
      partner[e] = tab.interleaved ? dim ^ 1 : second ? dim - half : dim + half;
    }
  }
#pragma unroll
  for (int u = 0; u < HPS; ++u) {
    const int h = h0 + u * SLOTS;
    const bool live = h < heads, is_q = h < hq, is_k = !is_q && h < hq + hkv;
    float y[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
    const float* w = !live ? nullptr : is_q ? q_norm : is_k ? k_norm : nullptr;
    if (__any_sync(0xFFFFFFFFu, w != nullptr)) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = __fmaf_rn(y[e], y[e], ss);
#pragma unroll
      for (int o = LPH >> 1; o > 0; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, o));
      if (w) {
        const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)D), eps)));
        const float4 wv = __ldg(reinterpret_cast<const float4*>(w) + l);
        y[0] = __fmul_rn(__fmul_rn(y[0], inv), wv.x);
        y[1] = __fmul_rn(__fmul_rn(y[1], inv), wv.y);
        y[2] = __fmul_rn(__fmul_rn(y[2], inv), wv.z);
        y[3] = __fmul_rn(__fmul_rn(y[3], inv), wv.w);
      }
    }
    if (__any_sync(0xFFFFFFFFu, live && (is_q || is_k))) {
      float p[4];
      if (tab.interleaved) {
        p[0] = y[1], p[1] = y[0], p[2] = y[3], p[3] = y[2];
      } else if ((rd & 7) == 0) {  // the partners are another lane's four values
        const int src = (tid & 31 & ~(LPH - 1)) + (partner[0] >> 2);
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
      if (is_q || is_k) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * l + e < rd) y[e] = __fmaf_rn(y[e], c[e], __fmul_rn(p[e], s[e]));
      }
    }
    if (live && is_q && (q_norm || 4 * l < rd))
      *(reinterpret_cast<float4*>(row + (size_t)h * D) + l) = make_float4(y[0], y[1], y[2], y[3]);
    const int g = h - hq - (is_k ? 0 : hkv);  // kv head
    if constexpr (std::is_same<Store, StoreQ4>::value) {
      if (!__any_sync(0xFFFFFFFFu, live && !is_q)) continue;
      float least = fminf(fminf(y[0], y[1]), fminf(y[2], y[3])), most = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
      most = lanes_max(most, LPH);
      least = -lanes_max(-least, LPH);
      const bool odd = !(fabsf(y[0]) <= FLT_MAX) || !(fabsf(y[1]) <= FLT_MAX) || !(fabsf(y[2]) <= FLT_MAX) ||
                       !(fabsf(y[3]) <= FLT_MAX);
      const uint32_t seen = __ballot_sync(0xFFFFFFFFu, odd);
      const uint32_t group = LPH == 32 ? 0xFFFFFFFFu : 0xFFFFu << (tid & 16);
      __half dh = __float2half_rn(__fdiv_rn(__fsub_rn(most, least), 15.0f));
      __half zh = __float2half_rn(__fadd_rn(least, __fmul_rn(8.0f, __half2float(dh))));
      if (seen & group) {  // a vector with a NaN or an infinity is stored as NaN
        dh = __ushort_as_half(0);
        zh = __ushort_as_half(0x7FFF);
      }
      const float d = __half2float(dh), z = __half2float(zh);
      uint32_t code = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = rintf(__fdiv_rn(__fsub_rn(y[e], z), d)) + 8.0f;
        const int n = d == 0.0f ? 8 : (int)fminf(fmaxf(v, 0.0f), 15.0f);
        code |= (uint32_t)n << (4 * e);
      }
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
}

template <int NP>
void fill_turns(const RotaryTable& rot, Turns<NP>* out) {
  for (int i = 0; i < NP; ++i) out->f[i] = i < rot.rd / 2 ? rot.turns[i] : 0;
  out->gain = rot.gain;
  out->rd = rot.rd;
  out->interleaved = rot.interleaved;
}

template <int N>
void fill_words(const MetaArg& m, ParamWords<N>* out) {
  for (int i = 0; i < N; ++i) out->w[i] = N > 1 && i < m.n_words ? m.host[i] : 0;
}

template <int NP, bool VEC, int N>
cudaError_t rope_go(float* q, long long q_stride, int hq, float* k, long long k_stride, int hkv, int head_dim, int n_tok,
                    const RotaryTable& rot, const MetaArg& meta, cudaStream_t st) {
  Turns<NP> tab;
  fill_turns(rot, &tab);
  ParamWords<N> w;
  fill_words(meta, &w);
  const int per_head = !VEC ? rot.rd / 2 : rot.interleaved ? rot.rd / 4 : rot.rd / 8;
  const long long pieces = (long long)(hq + hkv) * per_head;
  const unsigned gy = (unsigned)((pieces + kRotThreads * kRotUnroll - 1) / (kRotThreads * kRotUnroll));
  return launch_kernel(rope_rotary_kernel<NP, VEC, N>, dim3((unsigned)n_tok, gy), dim3(kRotThreads), 0, st, q, q_stride,
                       hq, k, k_stride, hkv, head_dim, tab, w, meta.dev);
}

template <int NP, int N>
cudaError_t rope_vec(float* q, long long q_stride, int hq, float* k, long long k_stride, int hkv, int head_dim,
                     int n_tok, const RotaryTable& rot, const MetaArg& meta, cudaStream_t st) {
  // 16-byte pieces where every head starts on 16 bytes and the rotated part is
  // a whole number of pieces
  const bool vec = head_dim % 4 == 0 && q_stride % 4 == 0 && k_stride % 4 == 0 &&
                   rot.rd % (rot.interleaved ? 4 : 8) == 0;
  return vec ? rope_go<NP, true, N>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, meta, st)
             : rope_go<NP, false, N>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, meta, st);
}

template <int D, typename Store, int HPS, int N>
cudaError_t append_go(const AppendArgs& a, const RotaryTable& rot, const MetaArg& meta, cudaStream_t st) {
  Turns<64> tab;
  fill_turns(rot, &tab);
  ParamWords<N> w;
  fill_words(meta, &w);
  const int slots = kAppThreads / (D / 4) * HPS;
  const dim3 grid((unsigned)a.n_tok, (unsigned)((a.hq + 2 * a.hkv + slots - 1) / slots));
  return launch_kernel(kv_append_kernel<D, Store, HPS, N>, grid, dim3(kAppThreads), 0, st, a.qkv, a.stride, a.hq, a.hkv,
                       static_cast<uint8_t*>(a.kc), static_cast<uint8_t*>(a.vc), tab, a.q_norm, a.k_norm, a.eps, a.n_seq,
                       w, meta.dev);
}

template <int D, typename Store>
cudaError_t append_pick(const AppendArgs& a, const RotaryTable& rot, const MetaArg& meta, cudaStream_t st) {
  // few tokens: one head per lane group, the most CTAs; else four
  const bool few = a.n_tok <= 64;
  if (meta.dev) return few ? append_go<D, Store, 1, 1>(a, rot, meta, st) : append_go<D, Store, 4, 1>(a, rot, meta, st);
  return few ? append_go<D, Store, 1, kParamWords>(a, rot, meta, st)
             : append_go<D, Store, 4, kParamWords>(a, rot, meta, st);
}

}  // namespace

cudaError_t launch_rope_rotary(float* q, long long q_stride, int hq, float* k, long long k_stride, int hkv, int head_dim,
                               int n_tok, const RotaryTable& rot, const MetaArg& meta, cudaStream_t st) {
  if (n_tok == 0) return cudaSuccess;
  if (rot.rd <= 128)
    return meta.dev ? rope_vec<64, 1>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, meta, st)
                    : rope_vec<64, kParamWords>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, meta, st);
  return meta.dev ? rope_vec<kRopeMaxPairs, 1>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, meta, st)
                  : rope_vec<kRopeMaxPairs, kParamWords>(q, q_stride, hq, k, k_stride, hkv, head_dim, n_tok, rot, meta,
                                                         st);
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
void rotary_table(const double* freq, int rd, bool interleaved, float gain, RotaryTable* out) {
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
