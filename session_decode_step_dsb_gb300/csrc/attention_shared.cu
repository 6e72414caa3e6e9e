// Decode attention over 16-bit pages for up to a few query rows on a kv head: the pages
// of one sequence, of a few that share theirs, or those that a selection lists
// (sm_103a).  And the join of the parts, for these and for the tcgen05 kernel.
//
//   out = sum_k exp(s_k - max s) v_k / sum_k exp(s_k - max s),  s_k = q . k / sqrt(D)
//
// Few rows read every key for little work: bound by memory, 4 D bytes a key and kv head.
// So the design is about bytes on their way and few instructions.  A CTA of four warps walks
// over pages, each warp over its own 32 keys of every page with its own running reference,
// sums and output: no barrier until a part ends.  A warp has a ring of three slots of 32 keys
// of K or V, which one lane fills by TMA tensor copies (128-byte swizzle, so that ldmatrix
// reads without bank conflicts) as soon as one is free.
//
// Products: m16n8k16 in the cache's type, float32 sums.  A tile has 8 query rows; their
// upper parts are rows 0 to 7 of the left operand and their lower parts rows 8 to 15, so
// that one product makes both halves of a float32 product, which a lane then holds side by
// side.  (bf16 has a third part, in a product of its own.)  The scores of a lane's row and
// keys are where the left operand of the second product wants their weights.
//
// The tensor core's sums round toward zero, which would tell over the pages of a part: each
// page's products of weights and V start from zero, and their halves are added to the
// output in float32.
//
// Measured (GB300): 64 selected pages of bf16 for each of 16 sessions and 8 kv heads of 128,
// 537 MB: 92 us, 0.86 of the copy rate; two CTAs an SM take 1.3 us for a page each, and 5 us
// until their first.  What is left are latencies of eight warps an SM (issue slots 0.25 full,
// the tensor pipe 0.36); a third CTA has no room, 255 registers a thread being in use.  16
// sessions of 5 rows behind 16 common pages (bf16, 76 MB): 26 us, 3 of them the join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "attention_shared.cuh"
#include "dsb_kernels.h"
#include "dsb_ptx.cuh"
#include "kv_tensor_map.h"

namespace dsbk {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kRows = 8;

__device__ unsigned int g_err_attention_pages = 0;

template <int D>
struct Ring {
  static constexpr int keys = 32;                // of a slot, K or V
  static constexpr int slab = keys * 128;        // 64 columns of them
  static constexpr int slot = D / 64 * slab;
  static constexpr int slots = 24576 / slot;     // 24 KB a warp
  static constexpr int bytes = kWarps * slots * slot;
  static constexpr int join = bytes;             // [warp][row][D] sums, [warp][row] statistics
  static constexpr int stat = join + kWarps * kRows * D * 4;
  static constexpr int bars = stat + kWarps * kRows * 8;
  static constexpr int smem = bars + kWarps * slots * 8;
};

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

#define DSB_MMA(TYPE)                                                                                              \
  asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "        \
      "{%0,%1,%2,%3};"                                                                                             \
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                             \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (std::is_same_v<T, __half>)
    DSB_MMA("f16");
  else
    DSB_MMA("bf16");
}
#undef DSB_MMA

template <typename T>
__device__ __forceinline__ float value(T x);
template <>
__device__ __forceinline__ float value<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <int D, typename T, typename Walk, int N>
__global__ void __launch_bounds__(kThreads, 2) attention_pages_kernel(
    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const float* __restrict__ q,
    long long q_stride, int hq, int hkv, const T* __restrict__ vp, int n_seg, int n_tok,
    const int32_t* __restrict__ selected, int n_select, int sel_stride, int sel_cap, float scale_log2e, float unit,
    PartialsOut to, bool wide, bool beside, const __grid_constant__ ParamWords<N> words, const int32_t* __restrict__ meta_dev) {
  using R = Ring<D>;
  constexpr int KK = D / 16, NT = D / 8;  // steps of the first product, column tiles of the second
  constexpr bool kThird = Parts<T>::kMore > 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* joined = reinterpret_cast<float*>(smem + R::join);
  float2* joined_stat = reinterpret_cast<float2*>(smem + R::stat);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * R::slots * R::slot;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + R::bars) + warp * R::slots;
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (lane == 0) {
    for (int i = 0; i < R::slots; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  // beside: launched while the call's kernel before works on, whose results are others than
  // what this one reads and writes; it has ended before this one does
  if (!beside) pdl_wait();
  pdl_trigger();

  Walk cur, ahead;
  if constexpr (std::is_same_v<Walk, SharedWalk>)
    cur.locate(cur.begin(meta, n_seg, wide, hkv, hq / hkv, kRows, kLead8, cta, ctas));
  else
    cur.locate(cur.begin(meta, n_seg, wide, selected, n_select, sel_stride, sel_cap, n_tok, hkv, hq / hkv, kRows, kLead8, cta, ctas));
  if (!cur.any()) {
    pdl_wait();
    return;
  }

  // ---- a tile's rows: lane (g, c) holds row g; what they see in common, and at all
  int live, min_hi, max_hi, min_lo, max_lo;
  RowAt at;
  float2 x[KK][2];
  const auto fetch = [&]() {
    live = cur.tile_rows();
    at = RowAt{0, 0, 0, 0x7FFFFFFF};
    if (g < live) at = cur.row(g, hq);
    const float* src = q + (size_t)at.tok * q_stride + (size_t)(at.row - at.tok * hq) * D + 2 * c;
#pragma unroll
    for (int k = 0; k < KK; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[k][j] = make_float2(0.0f, 0.0f);
        if (g < live) x[k][j] = __ldg(reinterpret_cast<const float2*>(src + 16 * k + 8 * j));
      }
    min_hi = at.hi, max_hi = g < live ? at.hi : -1, min_lo = g < live ? at.lo : 0x7FFFFFFF, max_lo = at.lo;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      min_hi = min(min_hi, __shfl_xor_sync(0xFFFFFFFFu, min_hi, o));
      max_hi = max(max_hi, __shfl_xor_sync(0xFFFFFFFFu, max_hi, o));
      min_lo = min(min_lo, __shfl_xor_sync(0xFFFFFFFFu, min_lo, o));
      max_lo = max(max_lo, __shfl_xor_sync(0xFFFFFFFFu, max_lo, o));
    }
  };
  fetch();
  ahead = cur;

  // ---- asking: entry `e` of ahead's run; 32 entries' blocks and pages in the lanes.  Entries
  // of which no row sees a key of this warp are neither asked for nor gone through.
  int e = ahead.i - 1, list_at = ahead.i - 32, list_block = 0, list_page = 0, row0 = 0, filled = 0;
  bool asking = true, value_next = false;
  const auto find = [&]() {  // the next entry to ask for
    for (;;) {
      if (++e == ahead.i_end) {
        if (!ahead.another()) {
          asking = false;
          return;
        }
        ahead.locate(ahead.following());
        e = ahead.i;
        list_at = e - 32;
      }
      if (e - list_at == 32) {
        list_at = e;
        if (e + lane < ahead.n_pages) {
          const int got = ahead.listed(e + lane);
          list_block = ahead.block(e + lane, got);
          if constexpr (std::is_same_v<Walk, SharedWalk>)
            list_page = ahead.page(e + lane);
          else
            list_page = ahead.seen(list_block * kPgKeys, 1) ? ahead.page(got) : 0;
        }
      }
      const int block = __shfl_sync(0xFFFFFFFFu, list_block, e - list_at);
      const int page = __shfl_sync(0xFFFFFFFFu, list_page, e - list_at);
      if (ahead.seen(block * kPgKeys + 32 * warp, 32)) {
        row0 = (page * hkv + ahead.h) * kPgKeys + 32 * warp;
        return;
      }
    }
  };
  // One lane asks for 32 keys of K, or then of V, into the slot that is next.
  const auto ask = [&]() {
    if (!asking) return;
    if (lane == 0) {
      const CUtensorMap* map = value_next ? &tmv : &tmk;
      mbar_arrive_expect_tx(&full[filled], R::slot);
#pragma unroll
      for (int x = 0; x < D / 64; ++x) tma_box(ring + filled * R::slot + x * R::slab, map, 64 * x, row0, &full[filled]);
    }
    if (++filled == R::slots) filled = 0;
    value_next = !value_next;
    if (!value_next) find();
  };
  find();
#pragma unroll 1
  for (int i = 0; i < R::slots; ++i) ask();

  // ldmatrix: lane i points at row i % 8 of matrix i / 8.  K: matrices (keys 0-7, dims
  // 0-7), (keys 0-7, dims 8-15), (keys 8-15, ..); V: (keys 0-7, dims 0-7), (keys 8-15, dims 0-7),
  // (keys 0-7, dims 8-15), ..
  // Piece j of a row of 128 bytes lies at piece j ^ (row % 8): steps of two pieces flip
  // bits 5 and 6 of the address.
  const uint32_t k_at = smem_addr(ring) + ((lane & 7) + (lane >> 4) * 8) * 128 + (((lane >> 3 & 1) ^ (lane & 7)) << 4);
  const uint32_t v_at = smem_addr(ring) + ((lane & 7) + (lane >> 3 & 1) * 8) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
  int slot = 0;
  uint32_t phase = 0;
  const auto next_slot = [&]() {
    fence_proxy_async_smem();  // what the lanes have read or cleared precedes the next copy
    __syncwarp();
    if (++slot == R::slots) slot = 0, phase ^= 1u;
    ask();
  };

  for (;;) {
    // upper and lower parts of dimensions 16 k + 2c, + 1 and 16 k + 8 + 2c, + 1; the third
    uint32_t qa[KK][4], qb[kThird ? KK : 1][2];
    float rs;
    {
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < KK; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) m = fmaxf(m, fmaxf(fabsf(x[k][j].x), fabsf(x[k][j].y)));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      float by;
      row_powers<T>(m, by, rs);
      by *= scale_log2e;
#pragma unroll
      for (int k = 0; k < KK; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x0 = x[k][j].x * by, x1 = x[k][j].y * by;
          qa[k][2 * j] = Parts<T>::take(x0, x1);
          qa[k][2 * j + 1] = Parts<T>::take(x0, x1);
          if constexpr (kThird) qb[k][j] = Parts<T>::take(x0, x1);
        }
    }

    f2 o[NT];  // of row g: dimensions 8 t + 2c, + 1
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t] = 0;
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
      const int key0 = block * kPgKeys + 32 * warp;
      if (!cur.seen(key0, 32)) continue;

      // ---- scores of row g with keys 8 t + 2c, + 1
      float s[4][4], s3[kThird ? 4 : 1][4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          s[t][n] = 0.0f;
          if constexpr (kThird) s3[t][n] = 0.0f;
        }
      if (!mbar_wait(&full[slot], phase)) g_err_attention_pages = 1u;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        uint32_t b[2][4];
        const uint32_t from = ((k_at + slot * R::slot) ^ (32 * (k & 3))) + (k >> 2) * R::slab;
        ldsm(b[0], from);
        ldsm(b[1], from + 16 * 128);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          mma<T>(s[t], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b[t >> 1][2 * (t & 1)], b[t >> 1][2 * (t & 1) + 1]);
          if constexpr (kThird) mma<T>(s3[t], 0u, qb[k][0], 0u, qb[k][1], b[t >> 1][2 * (t & 1)], b[t >> 1][2 * (t & 1) + 1]);
        }
      }
      next_slot();

      float p[8];  // of keys 8 (n >> 1) + 2c + (n & 1)
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        float low = s[n >> 1][2 + (n & 1)];
        if constexpr (kThird) low += s3[n >> 1][2 + (n & 1)];
        p[n] = s[n >> 1][n & 1] + low;
      }
      const bool whole = key0 >= max_lo && key0 + 31 <= min_hi;
      unsigned hidden = 0;
      if (!whole) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int key = key0 + 8 * (n >> 1) + 2 * c + (n & 1);
          hidden |= (unsigned)(key > at.hi || key < at.lo) << n;
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < 8; ++n) top = fmaxf(top, hidden >> n & 1u ? -INFINITY : p[n] * rs);
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const bool grown = top + minus > Parts<T>::kRoom + kSlack;
      if (__any_sync(0xFFFFFFFFu, grown)) {
        const float to_minus = grown ? Parts<T>::kRoom - top : minus, f = exp2_of(to_minus - minus);
        minus = to_minus;
        l *= f;
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] = mul2(o[t], pack(f, f));
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        p[n] = hidden >> n & 1u ? 0.0f : exp2_of(fmaf(p[n], rs, minus));
        if constexpr (kThird) p[n] *= unit;
        l += p[n];
      }

      if (!mbar_wait(&full[slot], phase)) g_err_attention_pages = 1u;
      __syncwarp();
      if (!whole) {
        // Lane i looks after key i.  One that no row sees may hold anything: cleared.  One
        // that some rows see, with an infinity or a NaN: 0 times it is no 0, so it is
        // cleared too, and added to the rows that see it.  (Pieces of a row in an order that
        // turns with the lane: other banks.)
        const int key = key0 + lane;
        const bool none = key > max_hi || key < min_lo;
        bool strange = false;
        uint4* row = reinterpret_cast<uint4*>(ring + slot * R::slot + lane * 128);
        if (min_hi < max_hi || min_lo < max_lo) {
#pragma unroll 4
          for (int x = 0; x < NT; ++x) {
            const uint4 v = row[(x >> 3) * (R::slab / 16) + ((x ^ lane) & 7)];
            strange = strange || odd<T>(v.x) || odd<T>(v.y) || odd<T>(v.z) || odd<T>(v.w);
          }
        }
        if (none || strange) {
#pragma unroll 4
          for (int x = 0; x < NT; ++x) row[(x >> 3) * (R::slab / 16) + ((x ^ lane) & 7)] = make_uint4(0, 0, 0, 0);
        }
        unsigned odd_keys = __ballot_sync(0xFFFFFFFFu, strange && !none);
        if (odd_keys) {
          const int page = [&] {
            if constexpr (std::is_same_v<Walk, SharedWalk>)
              return cur.page(i);
            else
              return cur.page(block);
          }();
          const T* rows = vp + (((size_t)page * hkv + cur.h) * kPgKeys + 32 * warp) * D;
#pragma unroll 1
          for (; odd_keys; odd_keys &= odd_keys - 1) {
            const int k = __ffs(odd_keys) - 1, from_lane = (lane & ~3) | (k >> 1 & 3), n = 2 * (k >> 3) + (k & 1);
            float mine = 0.0f;
#pragma unroll
            for (int m = 0; m < 8; ++m)
              if (m == n) mine = p[m];
            const float w = __shfl_sync(0xFFFFFFFFu, mine, from_lane);
            if (__shfl_sync(0xFFFFFFFFu, hidden, from_lane) >> n & 1u) continue;
#pragma unroll
            for (int t = 0; t < NT; ++t)
              o[t] = fma2(pack(w, w), pack(value<T>(rows[k * D + 8 * t + 2 * c]), value<T>(rows[k * D + 8 * t + 2 * c + 1])), o[t]);
          }
        }
        __syncwarp();
      }
      // ---- output
      uint32_t a[2][4], third[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x0 = p[4 * k + 2 * j], x1 = p[4 * k + 2 * j + 1];
          a[k][2 * j] = Parts<T>::take(x0, x1);
          a[k][2 * j + 1] = Parts<T>::take(x0, x1);
          third[k][j] = Parts<T>::take(x0, x1);
        }
#pragma unroll
      for (int t2 = 0; t2 < NT / 2; ++t2) {
        uint32_t b[2][4];
        const uint32_t from = ((v_at + slot * R::slot) ^ (32 * (t2 & 3))) + (t2 >> 2) * R::slab;
        ldsm_t(b[0], from);
        ldsm_t(b[1], from + 16 * 128);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (kThird) {
            mma<T>(d, 0u, third[0][0], 0u, third[0][1], b[0][2 * t], b[0][2 * t + 1]);
            mma<T>(d, 0u, third[1][0], 0u, third[1][1], b[1][2 * t], b[1][2 * t + 1]);
          }
          mma<T>(d, a[0][0], a[0][1], a[0][2], a[0][3], b[0][2 * t], b[0][2 * t + 1]);
          mma<T>(d, a[1][0], a[1][1], a[1][2], a[1][3], b[1][2 * t], b[1][2 * t + 1]);
          o[2 * t2 + t] = add2(o[2 * t2 + t], add2(pack(d[0], d[1]), pack(d[2], d[3])));
        }
      }
      next_slot();
    }

    // ---- the part's end: the four warps' rows joined
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
    __syncthreads();  // the last part's have been read
    {
      float2* row = reinterpret_cast<float2*>(joined + (warp * kRows + g) * D) + c;
#pragma unroll
      for (int t = 0; t < NT; ++t) row[4 * t] = unpack(o[t]);
      if (c == 0) joined_stat[warp * kRows + g] = make_float2(-minus, l);
    }
    // a thread's share of the rows, and where it goes: to the output where this CTA has all
    // of the run, else to a slot
    const int r = tid >> 4, d0 = (tid & 15) * (D / 16);
    const bool done = cur.alone() && cur.i == 0 && cur.i_end == cur.n_pages;
    float* dst = nullptr;
    float2* stat = nullptr;
    int empty_at = 0, empty = 0;  // slots behind the first part's that the row's parts leave
    if (r < live) {
      const size_t row = (size_t)cur.row(r, hq).row;
      const int part = cur.part(cta);
      const size_t place = row * to.slots + cur.slot_base() + (done ? 0 : part);
      dst = done ? to.out + row * D : to.acc + place * D;
      if (d0 == 0 && !(done && cur.slot_cap() == 1)) {
        stat = to.stat + place;
        if (!done && part == 0) {
          empty_at = cur.parts();
          empty = cur.slot_cap();
        }
      }
    }
    // the next run's rows are on their way meanwhile
    const bool more = cur.another();
    if (more) {
      cur.locate(cur.following());
      fetch();
    }
    __syncthreads();
    if (dst) {
      float2 st[kWarps];
      float ref = -kNoRef;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        st[w] = joined_stat[w * kRows + r];
        ref = fmaxf(ref, st[w].x);
      }
      float sum = 0.0f, y[D / 16];
#pragma unroll
      for (int k = 0; k < D / 16; ++k) y[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_of(st[w].x - ref);
        sum = fmaf(f, st[w].y, sum);
        const float4* src = reinterpret_cast<const float4*>(joined + (w * kRows + r) * D + d0);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const float4 z = src[k];
          y[4 * k] = fmaf(f, z.x, y[4 * k]);
          y[4 * k + 1] = fmaf(f, z.y, y[4 * k + 1]);
          y[4 * k + 2] = fmaf(f, z.z, y[4 * k + 2]);
          y[4 * k + 3] = fmaf(f, z.w, y[4 * k + 3]);
        }
      }
      if (stat) {
        *stat = done ? make_float2(0.0f, -1.0f) : make_float2(ref, sum);
        for (; empty_at < empty; ++empty_at) stat[empty_at] = make_float2(0.0f, 0.0f);
      }
      if (done) {
        const float by = sum == 0.0f ? 0.0f : __frcp_rn(sum);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) y[k] *= by;
      }
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
        reinterpret_cast<float4*>(dst + d0)[k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
    }
    if (!more) break;
  }
  pdl_wait();
}

// The parts' sums of a row at the largest of their references, in slot order, by a warp.  It
// takes one row of a few, and of many up to 32, of which it finds those that are in parts by
// one load: rows beyond what the GPU holds warps would wait their turn to find that there is
// nothing to join (prompts of 160000 rows: 712 us a call with a row to a warp, 683 so).
template <int D, int N>
__global__ void __launch_bounds__(kThreads) attention_join_kernel(int n_seq, int rows, int per, int hq, PartialsOut from,
                                                                  const __grid_constant__ ParamWords<N> words) {
  constexpr int V = D / 32;  // dimensions of a lane
  pdl_wait();
  pdl_trigger();
  const int row0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * per, lane = threadIdx.x & 31;
  if (row0 >= rows) return;
  unsigned todo = 1;
  if (per > 1)
    todo = __ballot_sync(0xFFFFFFFFu, lane < min(per, rows - row0) &&
                                          __ldcg(&from.stat[(size_t)(row0 + lane) * from.slots].y) != -1.0f);
  for (; todo; todo &= todo - 1) {
    const int row = row0 + __ffs(todo) - 1, tok = row / hq;
    int s = 0, hi = n_seq - 1;
    while (s < hi) {
      const int mid = (s + hi + 1) >> 1;
      if (words.w[2 * mid] <= tok)
        s = mid;
      else
        hi = mid - 1;
    }
    const int n = words.w[2 * s + 1];
    if (n == 0) continue;
    const float2* stat = from.stat + (size_t)row * from.slots;
    const float* acc = from.acc + (size_t)row * from.slots * D + lane * V;
    float2 mine = make_float2(0.0f, 0.0f);
    if (lane < n) mine = __ldcg(stat + lane);
    if (__shfl_sync(0xFFFFFFFFu, mine.y, 0) == -1.0f) continue;
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
}

template <int D, typename T, typename Walk, int N>
cudaError_t pages_go(const PageAttnArgs& a, const MetaArg& meta, cudaStream_t st) {
  using R = Ring<D>;
  static_assert(2 * (R::smem + 1024) <= 228 * 1024, "two CTAs an SM");
  auto kern = attention_pages_kernel<D, T, Walk, N>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = allow_smem(kern, R::smem, &ready);
  if (e != cudaSuccess) return e;
  CUtensorMap tmk, tmv;
  if ((e = kv_tensor_map(a.k, a.pool_rows, D, std::is_same_v<T, __half> ? 0 : 1, R::keys, &tmk)) != cudaSuccess) return e;
  if ((e = kv_tensor_map(a.v, a.pool_rows, D, std::is_same_v<T, __half> ? 0 : 1, R::keys, &tmv)) != cudaSuccess) return e;
  ParamWords<N> w;
  fill_words(meta, &w);
  const PartialsOut to{reinterpret_cast<float2*>(a.stat), a.acc, a.out, a.slots};
  return launch_kernel(kern, dim3((unsigned)a.ctas), dim3(kThreads), (size_t)R::smem, st, tmk, tmv, a.q, a.q_stride, a.hq,
                       a.hkv, static_cast<const T*>(a.v), a.n_seg, a.n_tok, a.selected, a.n_select,
                       a.sel_stride, a.sel_cap, (float)(1.4426950408889634 / std::sqrt((double)D)), a.unit, to, a.wide_pages, a.beside, w,
                       meta.dev);
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

unsigned int read_clear_error_attention_pages() {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_attention_pages, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  cudaMemcpyToSymbol(g_err_attention_pages, &z, sizeof z);
  return v;
}

cudaError_t launch_attention_join(const PageAttnArgs& a, int n_seq, int head_dim, const MetaArg& meta, cudaStream_t st) {
  const PartialsOut from{reinterpret_cast<float2*>(a.stat), a.acc, a.out, a.slots};
  const int rows = a.n_tok * a.hq, per = std::min(std::max(rows / 8192, 1), 32);
  const dim3 grid((unsigned)((rows + kWarps * per - 1) / (kWarps * per)));
  const auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    ParamWords<N> w;
    fill_words(meta, &w);
    return head_dim == 128 ? launch_kernel(attention_join_kernel<128, N>, grid, dim3(kThreads), 0, st, n_seq, rows, per, a.hq, from, w)
                           : launch_kernel(attention_join_kernel<64, N>, grid, dim3(kThreads), 0, st, n_seq, rows, per, a.hq, from, w);
  };
  if (meta.n_words <= kParamFew) return go(std::integral_constant<int, kParamFew>{});
  return go(std::integral_constant<int, kParamWords>{});
}

}  // namespace dsbk
