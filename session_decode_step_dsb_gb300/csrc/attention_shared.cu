// Decode attention over 16-bit pages for up to a few query rows on a kv head: the pages
// of one sequence, of a few that share theirs, or those that a selection lists
// (sm_103a).  And the join of the parts, for these and for the tcgen05 kernel.
//
//   out = sum_k exp(s_k - max s) v_k / sum_k exp(s_k - max s),  s_k = q . k / sqrt(D)
//
// Few rows read every key for little work: bound by memory, 4 D bytes a key and kv head.
// So the design is about loads in flight and nothing else.  A CTA of four warps walks over
// pages, each warp over its own 32 keys of every page with its own running reference, sums
// and output: no barrier until a part ends.  A warp asks for 16 keys of K and V at a time,
// cp.async into a ring of stages of its own, from which each lane reads only what it
// asked for itself: the pieces are laid out so that they are the lane's parts of the
// matrix operands (below), so no lane waits for another.
//
// Products: m16n8k16 in the cache's type, float32 sums.  A tile has 8 query rows; their
// upper parts are rows 0 to 7 of the left operand and their lower parts rows 8 to 15, so
// that one product makes both halves of a float32 product, which a lane then holds side by
// side.  (bf16 queries have a third part, in a product of its own; weights have two.)  The
// order of the dimensions along a product's sum is free, so lane (g, c) of the K operand
// takes 16-byte pieces c, c + 4, .. of key g; and the order of the dimensions across the
// second product's columns is free, so it takes pieces g and g + 8 of keys 2c, 2c + 1, 2c + 8,
// 2c + 9 of V and pairs up the keys' halves.
//
// The tensor core's sums round toward zero, which would tell over the pages of a part: each
// product of weights and V starts from zero, and its two halves are added to the output
// in float32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "attention_shared.cuh"
#include "dsb_kernels.h"
#include "dsb_ptx.cuh"

namespace dsbk {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kRows = 8;
constexpr int kStep = 16;  // keys of a stage

template <int D>
struct Ring {
  static constexpr int pieces = D / 8;           // of a lane, 16 bytes each: half of them K
  static constexpr int stage = pieces * 512;     // bytes
  static constexpr int stages = 24576 / stage;   // 24 KB a warp
  static constexpr int bytes = kWarps * stages * stage;
  static constexpr int join = kWarps * kRows * D * 4;
  static constexpr int smem = bytes + join + kWarps * kRows * 8;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// d = a b + c, c given or zero
#define DSB_MMA(TYPE)                                                                                              \
  asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "        \
      "{%10,%11,%12,%13};"                                                                                         \
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                                             \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3))
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, float c0, float c1, float c2, float c3) {
  if constexpr (std::is_same_v<T, __half>)
    DSB_MMA("f16");
  else
    DSB_MMA("bf16");
}
#undef DSB_MMA
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  mma<T>(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

template <typename T>
__device__ __forceinline__ float value(T x);
template <>
__device__ __forceinline__ float value<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// Whether a pair of 16-bit values holds an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool odd(uint32_t w) {
  constexpr uint32_t e = std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u;
  return (w & e) == e || (w & e << 16) == e << 16;
}
template <typename T>
__device__ __forceinline__ bool odd(uint4 v) { return odd<T>(v.x) || odd<T>(v.y) || odd<T>(v.z) || odd<T>(v.w); }

template <int D, typename T, typename Walk, int N>
__global__ void __launch_bounds__(kThreads, 2) attention_pages_kernel(
    const float* __restrict__ q, long long q_stride, int hq, int hkv, const T* __restrict__ kp, const T* __restrict__ vp,
    int n_seg, int n_tok, const int32_t* __restrict__ selected, int n_select, int sel_stride, int sel_cap, float scale_log2e,
    PartialsOut to, const __grid_constant__ ParamWords<N> words, const int32_t* __restrict__ meta_dev) {
  using R = Ring<D>;
  constexpr int PG = D / 32, VH = D / 64;  // 16-byte pieces of a lane: of a K row, of a V row
  extern __shared__ __align__(128) uint8_t smem[];
  float* joined = reinterpret_cast<float*>(smem + R::bytes);                     // [warp][row][D]
  float2* joined_stat = reinterpret_cast<float2*>(smem + R::bytes + R::join);    // [warp][row]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * R::stages * R::stage + lane * 16;
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  const int cta = blockIdx.x, ctas = gridDim.x;
  pdl_wait();
  pdl_trigger();

  Walk cur, ahead;
  if constexpr (std::is_same_v<Walk, SharedWalk>)
    cur.begin(meta, n_seg, hkv, hq / hkv, kRows, cta, ctas);
  else
    cur.begin(meta, n_seg, selected, n_select, sel_stride, sel_cap, n_tok, hkv, hq / hkv, kRows, cta, ctas);
  ahead = cur;

  // ---- asking: entry `e` of ahead's run, its half `half`; 32 entries' blocks and pages
  // in the lanes
  int e = ahead.i, half = 0, list_at = 0, list_block = 0, list_page = 0, filled = 0;
  bool asking = true;
  const auto list = [&]() {
    list_at = e;
    if (e + lane < ahead.n_pages) {
      const int got = ahead.listed(e + lane);
      list_block = ahead.block(e + lane, got);
      if constexpr (std::is_same_v<Walk, SharedWalk>)
        list_page = ahead.page(e + lane);
      else
        list_page = ahead.seen(list_block * kPgKeys, 1) ? meta[ahead.pg_at + got] : 0;
    }
  };
  list();
  const auto ask = [&]() {
    if (asking) {
      const int block = __shfl_sync(0xFFFFFFFFu, list_block, e - list_at);
      const int page = __shfl_sync(0xFFFFFFFFu, list_page, e - list_at);
      const int in_page = 32 * warp + kStep * half;
      if (ahead.seen(block * kPgKeys + in_page, kStep)) {
        const size_t row0 = ((size_t)page * hkv + ahead.h) * kPgKeys + in_page;
        const uint32_t dst = ring + filled * R::stage;
        const T* ks = kp + (row0 + g) * D + 8 * c;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int p = 0; p < PG; ++p) cp16(dst + (kt * PG + p) * 512, ks + kt * 8 * D + p * 32);
        const T* vs = vp + (row0 + 2 * c) * D + 8 * g;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int v = 0; v < VH; ++v)
            cp16(dst + (2 * PG + n * VH + v) * 512, vs + ((n >> 1) * 8 + (n & 1)) * D + v * 64);
      }
      if (++filled == R::stages) filled = 0;
      if ((half ^= 1) == 0) {
        if (++e == ahead.i_end) {
          if (ahead.another()) {
            ahead.next();
            e = ahead.i;
            list();
          } else {
            asking = false;
          }
        } else if (e - list_at == 32) {
          list();
        }
      }
    }
    cp_commit();
  };
#pragma unroll 1
  for (int i = 0; i < R::stages; ++i) ask();

  int stage = 0;
  for (;;) {
    // ---- the tile's rows: lane (g, c) holds row g, the pieces of its dimensions that it
    // has of a key
    const int live = cur.tile_rows();
    RowAt at{0, 0, 0, 0x7FFFFFFF};
    if (g < live) at = cur.row(g, hq);
    int min_hi = at.hi, max_hi = g < live ? at.hi : -1, min_lo = g < live ? at.lo : 0x7FFFFFFF, max_lo = at.lo;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      min_hi = min(min_hi, __shfl_xor_sync(0xFFFFFFFFu, min_hi, o));
      max_hi = max(max_hi, __shfl_xor_sync(0xFFFFFFFFu, max_hi, o));
      min_lo = min(min_lo, __shfl_xor_sync(0xFFFFFFFFu, min_lo, o));
      max_lo = max(max_lo, __shfl_xor_sync(0xFFFFFFFFu, max_lo, o));
    }
    uint32_t qa[PG][2][4];                                               // upper and lower parts
    uint32_t qb[Parts<T>::kScore > 2 ? PG : 1][2][2];                    // the third
    float rs;
    {
      float x[PG][8];
      const float* src = q + (size_t)at.tok * q_stride + (size_t)(at.row - at.tok * hq) * D + 8 * c;
      float m = 0.0f;
#pragma unroll
      for (int p = 0; p < PG; ++p) {
        float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
        if (g < live) {
          v0 = __ldg(reinterpret_cast<const float4*>(src + 32 * p));
          v1 = __ldg(reinterpret_cast<const float4*>(src + 32 * p + 4));
        }
        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[p][i] = v[i] * scale_log2e;
          m = fmaxf(m, fabsf(x[p][i]));
        }
      }
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      // the row over a power of two that brings its largest value to [2^10, 2^11): the parts
      // keep their bits whatever q's size
      const int ex = min(max((int)(__float_as_uint(m) >> 23), 11), 254);
      const float inv = __uint_as_float((uint32_t)(264 - ex) << 23);
      rs = __uint_as_float((uint32_t)(ex - 10) << 23);
#pragma unroll
      for (int p = 0; p < PG; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x0 = x[p][4 * j + 2 * k] * inv, x1 = x[p][4 * j + 2 * k + 1] * inv;
            qa[p][j][2 * k] = Parts<T>::take(x0, x1);
            qa[p][j][2 * k + 1] = Parts<T>::take(x0, x1);
            if constexpr (Parts<T>::kScore > 2) qb[p][j][k] = Parts<T>::take(x0, x1);
          }
    }

    f2 o[VH][8];  // of row g: columns 2c and 2c + 1 of each product
#pragma unroll
    for (int v = 0; v < VH; ++v)
#pragma unroll
      for (int t = 0; t < 8; ++t) o[v][t] = 0;
    float minus = kNoRef, l = 0.0f;

    int blocks_at = 0, blocks = 0;
    for (int i = cur.i; i < cur.i_end; ++i) {
      int block;
      if constexpr (std::is_same_v<Walk, SharedWalk>) {
        block = cur.block(i, 0);
      } else {
        if (i == cur.i || i - blocks_at == 32) {
          blocks_at = i;
          if (i + lane < cur.n_pages) blocks = cur.listed(i + lane);
        }
        block = __shfl_sync(0xFFFFFFFFu, blocks, i - blocks_at);
      }
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        cp_wait<R::stages - 1>();
        const int key0 = block * kPgKeys + 32 * warp + kStep * hf;
        if (cur.seen(key0, kStep)) {
          const uint32_t from = ring + stage * R::stage;
          // ---- scores of row g with keys 2c, 2c + 1 of both tiles of eight
          float s[2][4];
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            s[kt][0] = s[kt][1] = s[kt][2] = s[kt][3] = 0.0f;
#pragma unroll
            for (int p = 0; p < PG; ++p) {
              const uint4 k = lds16(from + (kt * PG + p) * 512);
              mma<T>(s[kt], qa[p][0][0], qa[p][0][1], qa[p][0][2], qa[p][0][3], k.x, k.y);
              mma<T>(s[kt], qa[p][1][0], qa[p][1][1], qa[p][1][2], qa[p][1][3], k.z, k.w);
              if constexpr (Parts<T>::kScore > 2) {
                mma<T>(s[kt], 0u, qb[p][0][0], 0u, qb[p][0][1], k.x, k.y);
                mma<T>(s[kt], 0u, qb[p][1][0], 0u, qb[p][1][1], k.z, k.w);
              }
            }
          }
          uint4 v[4][VH];
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int h2 = 0; h2 < VH; ++h2) v[n][h2] = lds16(from + (2 * PG + n * VH + h2) * 512);
          // n: key 8 (n >> 1) + 2c + (n & 1) of the step
          float x[4], p[4];
          bool hidden[4] = {false, false, false, false};
#pragma unroll
          for (int n = 0; n < 4; ++n) x[n] = s[n >> 1][n & 1] + s[n >> 1][2 + (n & 1)];
          const bool whole = key0 >= max_lo && key0 + kStep - 1 <= min_hi;
          unsigned strange = 0;
          if (!whole) {
            bool bad[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const int key = key0 + 8 * (n >> 1) + 2 * c + (n & 1);
              hidden[n] = key > at.hi || key < at.lo;
              // a key that no row sees may hold anything; nothing of it enters a product
              const bool none = key > max_hi || key < min_lo;
              bad[n] = false;
#pragma unroll
              for (int h2 = 0; h2 < VH; ++h2) {
                if (none) v[n][h2] = make_uint4(0, 0, 0, 0);
                bad[n] = bad[n] || odd<T>(v[n][h2]);
              }
            }
            // one that some rows see, with an infinity or a NaN: 0 times it is no 0, so it
            // is left out of the product and added below to the rows that see it
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              unsigned b = __ballot_sync(0xFFFFFFFFu, bad[n]);  // any lane (., c): the same keys
              b |= b >> 4;
              b |= b >> 8;
              b |= b >> 16;
              strange |= (b & 15u) << (4 * n);
              if (b >> c & 1u) {
#pragma unroll
                for (int h2 = 0; h2 < VH; ++h2) v[n][h2] = make_uint4(0, 0, 0, 0);
              }
            }
          }
          float top = -INFINITY;
#pragma unroll
          for (int n = 0; n < 4; ++n) top = fmaxf(top, hidden[n] ? -INFINITY : x[n] * rs);
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const bool grown = top + minus > kRoom + kSlack;
          if (__any_sync(0xFFFFFFFFu, grown)) {
            const float to_minus = grown ? kRoom - top : minus, f = exp2_of(to_minus - minus);
            minus = to_minus;
            l *= f;
#pragma unroll
            for (int h2 = 0; h2 < VH; ++h2)
#pragma unroll
              for (int t = 0; t < 8; ++t) o[h2][t] = mul2(o[h2][t], pack(f, f));
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            p[n] = hidden[n] ? 0.0f : exp2_of(fmaf(x[n], rs, minus));
            l += p[n];
          }
          if (strange) {
            // rows 0 to 15 of key n's 4 lanes c: bit 4 n + c
#pragma unroll 1
            for (int b = 0; b < 16; ++b) {
              if (!(strange >> b & 1u)) continue;
              const int n = b >> 2, from_lane = (lane & ~3) | (b & 3);
              const float pn = n == 0 ? p[0] : n == 1 ? p[1] : n == 2 ? p[2] : p[3];
              const bool hn = n == 0 ? hidden[0] : n == 1 ? hidden[1] : n == 2 ? hidden[2] : hidden[3];
              const float w = __shfl_sync(0xFFFFFFFFu, pn, from_lane);
              const bool no = __shfl_sync(0xFFFFFFFFu, (int)hn, from_lane);
              const int page = [&] {
                if constexpr (std::is_same_v<Walk, SharedWalk>)
                  return cur.page(i);
                else
                  return meta[cur.pg_at + block];
              }();
              const T* row = vp + (((size_t)page * hkv + cur.h) * kPgKeys + 32 * warp + kStep * hf + 8 * (n >> 1) +
                                   2 * (b & 3) + (n & 1)) * D;
              if (!no) {
#pragma unroll
                for (int h2 = 0; h2 < VH; ++h2)
#pragma unroll
                  for (int t = 0; t < 8; ++t)
                    o[h2][t] = fma2(pack(w, w), pack(value<T>(row[8 * (2 * c + 8 * h2) + t]),
                                                     value<T>(row[8 * (2 * c + 1 + 8 * h2) + t])), o[h2][t]);
              }
            }
          }
          // ---- output: columns t of half h2 are dimensions 8 (n + 8 h2) + t
          uint32_t a[4];
          {
            float p0 = p[0], p1 = p[1], p2 = p[2], p3 = p[3];
            a[0] = Parts<T>::take(p0, p1);
            a[1] = Parts<T>::take(p0, p1);
            a[2] = Parts<T>::take(p2, p3);
            a[3] = Parts<T>::take(p2, p3);
          }
#pragma unroll
          for (int h2 = 0; h2 < VH; ++h2) {
            const uint32_t w[4][4] = {{v[0][h2].x, v[0][h2].y, v[0][h2].z, v[0][h2].w},
                                      {v[1][h2].x, v[1][h2].y, v[1][h2].z, v[1][h2].w},
                                      {v[2][h2].x, v[2][h2].y, v[2][h2].z, v[2][h2].w},
                                      {v[3][h2].x, v[3][h2].y, v[3][h2].z, v[3][h2].w}};
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              const uint32_t pick = t & 1 ? 0x7632u : 0x5410u;
              float d[4];
              mma<T>(d, a[0], a[1], a[2], a[3], __byte_perm(w[0][t >> 1], w[1][t >> 1], pick),
                     __byte_perm(w[2][t >> 1], w[3][t >> 1], pick), 0.0f, 0.0f, 0.0f, 0.0f);
              o[h2][t] = add2(o[h2][t], add2(pack(d[0], d[1]), pack(d[2], d[3])));
            }
          }
        }
        if (++stage == R::stages) stage = 0;
        ask();
      }
    }

    // ---- the part's end: the four warps' rows joined
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
    __syncthreads();  // the last part's have been read
    {
      float* row = joined + (warp * kRows + g) * D;
#pragma unroll
      for (int h2 = 0; h2 < VH; ++h2)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float4* d = reinterpret_cast<float4*>(row + 8 * (2 * c + k + 8 * h2));
          float x[8];
#pragma unroll
          for (int t = 0; t < 8; ++t) x[t] = k ? unpack(o[h2][t]).y : unpack(o[h2][t]).x;
          d[0] = make_float4(x[0], x[1], x[2], x[3]);
          d[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
      if (c == 0) joined_stat[warp * kRows + g] = make_float2(-minus, l);
    }
    __syncthreads();
    {
      const int r = tid >> 4, d0 = (tid & 15) * (D / 16);
      if (r < live) {
        const RowAt mine = cur.row(r, hq);
        float2 st[kWarps];
        float ref = -kNoRef;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          st[w] = joined_stat[w * kRows + r];
          ref = fmaxf(ref, st[w].x);
        }
        float sum = 0.0f, x[D / 16];
#pragma unroll
        for (int k = 0; k < D / 16; ++k) x[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = exp2_of(st[w].x - ref);
          sum = fmaf(f, st[w].y, sum);
          const float4* src = reinterpret_cast<const float4*>(joined + (w * kRows + r) * D + d0);
#pragma unroll
          for (int k = 0; k < D / 64; ++k) {
            const float4 y = src[k];
            x[4 * k] = fmaf(f, y.x, x[4 * k]);
            x[4 * k + 1] = fmaf(f, y.y, x[4 * k + 1]);
            x[4 * k + 2] = fmaf(f, y.z, x[4 * k + 2]);
            x[4 * k + 3] = fmaf(f, y.w, x[4 * k + 3]);
          }
        }
        const int cap = cur.slot_cap();
        float* dst;
        float2* stat = to.stat + (size_t)mine.row * to.slots + cur.slot_base();
        if (cur.alone() && cur.i == 0 && cur.i_end == cur.n_pages) {  // the row is done
          dst = to.out + (size_t)mine.row * D;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) x[k] = sum == 0.0f ? 0.0f : __fdiv_rn(x[k], sum);
          if (cap > 1 && d0 == 0) stat[0] = make_float2(0.0f, -1.0f);
        } else {
          const int part = cur.part(cta, ctas);
          dst = to.acc + ((size_t)mine.row * to.slots + cur.slot_base() + part) * D;
          if (d0 == 0) {
            stat[part] = make_float2(ref, sum);
            if (part == 0)
              for (int k = cur.parts(ctas); k < cap; ++k) stat[k] = make_float2(0.0f, 0.0f);
          }
        }
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
          reinterpret_cast<float4*>(dst + d0)[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
      }
    }
    if (!cur.another()) break;
    cur.next();
  }
  cp_wait<0>();
}

// One warp per row: the parts' sums at the largest of their references, in slot order.
template <int D, int N>
__global__ void __launch_bounds__(kThreads) attention_join_kernel(int n_seq, int rows, int hq, PartialsOut from,
                                                                  const __grid_constant__ ParamWords<N> words) {
  constexpr int V = D / 32;  // dimensions of a lane
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int tok = row / hq;
  int s = 0, hi = n_seq - 1;
  while (s < hi) {
    const int mid = (s + hi + 1) >> 1;
    if (words.w[2 * mid] <= tok)
      s = mid;
    else
      hi = mid - 1;
  }
  const int n = words.w[2 * s + 1];
  if (n == 0) return;
  const float2* stat = from.stat + (size_t)row * from.slots;
  const float* acc = from.acc + (size_t)row * from.slots * D + lane * V;
  float2 mine = make_float2(0.0f, 0.0f);
  if (lane < n) mine = __ldcg(stat + lane);
  if (__shfl_sync(0xFFFFFFFFu, mine.y, 0) == -1.0f) return;
  float ref = mine.y == 0.0f ? -kNoRef : mine.x;
  for (int i = lane + 32; i < n; i += 32) {
    const float2 x = __ldcg(stat + i);
    if (x.y != 0.0f) ref = fmaxf(ref, x.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, o));
  float sum = 0.0f, x[V];
#pragma unroll
  for (int k = 0; k < V; ++k) x[k] = 0.0f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    if (i0 > 0) mine = i0 + lane < n ? __ldcg(stat + i0 + lane) : make_float2(0.0f, 0.0f);
    const float f = mine.y == 0.0f ? 0.0f : exp2_of(mine.x - ref);
    const float fl = mine.y == 0.0f ? 0.0f : f * mine.y;
    const unsigned there = __ballot_sync(0xFFFFFFFFu, mine.y != 0.0f);
    const int m = min(32, n - i0);
    for (int j0 = 0; j0 < m; j0 += 8) {
      float y[8][V];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (there >> (j0 + j) & 1u) {
          const float* src = acc + (size_t)(i0 + j0 + j) * D;
          if constexpr (V == 4) {
            const float4 z = __ldcg(reinterpret_cast<const float4*>(src));
            y[j][0] = z.x, y[j][1] = z.y, y[j][2] = z.z, y[j][3] = z.w;
          } else {
            const float2 z = __ldcg(reinterpret_cast<const float2*>(src));
            y[j][0] = z.x, y[j][1] = z.y;
          }
        }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float fj = __shfl_sync(0xFFFFFFFFu, f, j0 + j), lj = __shfl_sync(0xFFFFFFFFu, fl, j0 + j);
        if (there >> (j0 + j) & 1u) {
          sum += lj;
#pragma unroll
          for (int k = 0; k < V; ++k) x[k] = fmaf(fj, y[j][k], x[k]);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) x[k] = sum == 0.0f ? 0.0f : __fdiv_rn(x[k], sum);
  float* out = from.out + (size_t)row * D + lane * V;
  if constexpr (V == 4)
    *reinterpret_cast<float4*>(out) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *reinterpret_cast<float2*>(out) = make_float2(x[0], x[1]);
}

template <int D, typename T, typename Walk, int N>
cudaError_t pages_go(const PageAttnArgs& a, const MetaArg& meta, cudaStream_t st) {
  using R = Ring<D>;
  static_assert(2 * (R::smem + 1024) <= 228 * 1024, "two CTAs an SM");
  auto kern = attention_pages_kernel<D, T, Walk, N>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::smem);
  if (e != cudaSuccess) return e;
  ParamWords<N> w;
  fill_words(meta, &w);
  const PartialsOut to{reinterpret_cast<float2*>(a.stat), a.acc, a.out, a.slots};
  return launch_kernel(kern, dim3((unsigned)a.ctas), dim3(kThreads), (size_t)R::smem, st, a.q, a.q_stride, a.hq, a.hkv,
                       static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.n_seg, a.n_tok, a.selected, a.n_select,
                       a.sel_stride, a.sel_cap, (float)(1.4426950408889634 / std::sqrt((double)D)), to, w, meta.dev);
}

template <int D, typename T>
cudaError_t pages_walk(const PageAttnArgs& a, const MetaArg& meta, cudaStream_t st) {
  return with_words(meta, [&](auto n) {
    constexpr int N = decltype(n)::value;
    return a.selected ? pages_go<D, T, SelectedWalk, N>(a, meta, st) : pages_go<D, T, SharedWalk, N>(a, meta, st);
  });
}

}  // namespace

int page_attn_resident(int sms) { return 2 * sms; }

cudaError_t launch_attention_pages(const PageAttnArgs& a, int dtype, int head_dim, const MetaArg& meta, cudaStream_t st) {
  if (head_dim == 128)
    return dtype == 0 ? pages_walk<128, __half>(a, meta, st) : pages_walk<128, __nv_bfloat16>(a, meta, st);
  return dtype == 0 ? pages_walk<64, __half>(a, meta, st) : pages_walk<64, __nv_bfloat16>(a, meta, st);
}

cudaError_t launch_attention_join(const PageAttnArgs& a, int n_seq, int head_dim, const MetaArg& meta, cudaStream_t st) {
  const PartialsOut from{reinterpret_cast<float2*>(a.stat), a.acc, a.out, a.slots};
  const int rows = a.n_tok * a.hq;
  const dim3 grid((unsigned)((rows + kWarps - 1) / kWarps));
  const auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    ParamWords<N> w;
    fill_words(meta, &w);
    return head_dim == 128 ? launch_kernel(attention_join_kernel<128, N>, grid, dim3(kThreads), 0, st, n_seq, rows, a.hq, from, w)
                           : launch_kernel(attention_join_kernel<64, N>, grid, dim3(kThreads), 0, st, n_seq, rows, a.hq, from, w);
  };
  if (meta.n_words <= kParamFew) return go(std::integral_constant<int, kParamFew>{});
  return go(std::integral_constant<int, kParamWords>{});
}

}  // namespace dsbk
