// Decode attention over the paged 4-bit KV cache (sm_103a).
//
// For query row r (token j of the sequence's new ones, head gi of the kv head's
// group) and the keys k it sees (k <= len - new + j, and k > that - window under
// a window), with K_k = z + d (c - 8) and V alike:
//     out = sum_k softmax_k(q . K_k / sqrt D) V_k
//
// The codes enter both products as small integers, exact in fp16, and the scale
// and offset of a key are applied outside them, in float32:
//     q . K_k = d (sum_i q_i (c_i - 8)) + z (sum_i q_i)
//     sum_k p_k V_k = sum_k (p_k d_k) (c_k - 8) + sum_k p_k z_k
// q and the weights w_k = p_k d_k are split into two fp16 (hi + lo: 22 bits), two
// products into one float32 sum.  Both products have the 8 query rows as their
// columns, S^T = K Q^T (keys x rows) and O^T = V^T P^T (dimensions x rows) (up to 4
// rows: hi and lo as columns of one product), so that
// m16n8k16 carries no padding at 8 rows and a warp's output tile is D/4 registers
// a thread; the weights turn from the first product's result layout into the
// second's operand layout by an 8 x 8 transpose in the warp.
//
// Work: a CTA of four warps takes units of a few pages of one (sequence, kv
// head, tile of 4 or 8 query rows); how many pages a unit has depends on the
// sequence alone (its pages, kv heads and rows), so a sequence's rows are bitwise
// the same alone and in a batch.  A warp takes 32 of a page's 128 keys and carries its own
// maximum, sum and output tile through the unit: inside a unit the warps meet at
// no barrier but those of the copies.  The K and V halves of the pages arrive as
// bulk copies, four halves ahead.  The four warps' results are joined at the unit's
// end, the units' by a second kernel in unit order (a sequence of one unit needs
// none).
//
// The running reference of the exponentials is the largest s_k + log d_k (d_k: V's
// scale of the same key) over the keys that the row sees, so that the weights that
// enter the fp16 split are at most 2^14 whatever the scales are; p_k itself and the
// sums over it are float32.
//
// Measured: 4 sequences of 16384 to 65536 keys, 32 kv heads of 128, one row each
// (720 MB of pages): 193 us with the join, 3.7 TB/s, 0.55 of the copy rate.  Bound by
// the latencies of some 640 instructions a warp and page, 290 of them the unpacking of
// the codes, at 16 warps an SM (124 registers; with 8 rows 128), issued in 0.6 of the
// cycles; an eighth of the waiting is at the units' ends.  16 sequences of up to
// 4096 keys, 8 kv heads of 128, 5 rows each (29 MB): 20 us for 2 or 4 pages a CTA.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "attention_q4.cuh"
#include "dsb_kernels.h"
#include "dsb_ptx.cuh"
#include "dsb_q4.cuh"

namespace dsbk {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ unsigned int g_err_attention_q4 = 0;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from an accumulator whose rows hold (c0, c1).
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %10, %11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
// An 8 x 8 tile of 16-bit values, a row of two to each thread, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

constexpr int kSlots = 5;  // half pages (K or V) on their way or in use
constexpr int kAhead = 8;  // items known at a time: a power of two, above the halves' reach of units of a page

template <int D>
struct Q4Smem {
  static constexpr int half = Q4Block<D>::v;                // K codes and numbers; V's are as many bytes
  static constexpr int q = kSlots * half;                   // [D/16][32 lanes] uint4: q as right operand
  static constexpr int rows = q + D / 16 * 512;             // [8] float4: scale, sum, last key, -
  static constexpr int join = rows + 8 * 16;                // [4 warps][D/32][32 lanes] float4
  static constexpr int stat = join + 4 * (D / 32) * 512;    // [4 warps][4] float4: M, M, sum, sum
  static constexpr int bars = stat + 4 * 64;
  static constexpr int cursors = bars + 2 * kSlots * 8;     // the items asked for, and how many those are
  static constexpr int bytes = cursors + kAhead * (int)sizeof(Cursor) + 8;
};

// ROWS, the query rows of an item: 8, or 4, whose hi and lo parts then share a
// product as columns 0 .. 3 and 4 .. 7.
template <int D, int ROWS, int N>
__global__ void __launch_bounds__(kThreads, 4) attention_q4_kernel(
    const float* __restrict__ q, long long q_stride, int hq, int hkv, const uint8_t* __restrict__ pool, int n_seq,
    float scale_log2e, int max_units, float* __restrict__ partials, float* __restrict__ out,
    const __grid_constant__ ParamWords<N> words, const int32_t* __restrict__ meta_dev) {
  using B = Q4Block<D>;
  using S = Q4Smem<D>;
  constexpr int W = D / 32;    // 32-bit words of a thread's piece of a K row, and of a V key pair
  constexpr int NT = D / 16;   // 16-dimension tiles of the output
  constexpr bool kFew = ROWS == 4;
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* qs = reinterpret_cast<uint4*>(smem + S::q);
  float4* rowp = reinterpret_cast<float4*>(smem + S::rows);
  float4* join = reinterpret_cast<float4*>(smem + S::join);
  float4* stat = reinterpret_cast<float4*>(smem + S::stat);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::bars);
  uint64_t* empty = full + kSlots;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int pair = kFew ? c & 1 : c;   // the thread's rows are 2 pair and 2 pair + 1
  const bool first_half = !kFew || c < 2;  // its columns are those of the hi parts
  const int G = hq / hkv;
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // This CTA's items: those that start in its share of the pages.  Thread 0 asks
  // for the half pages, kSlots - 1 ahead: after its warp has left one, for the slot
  // of the one before, which the other warps have left long since.
  Cursor* items = reinterpret_cast<Cursor*>(smem + S::cursors);  // item i of this CTA at i % kAhead
  volatile int* known = reinterpret_cast<volatile int*>(items + kAhead);
  const long long total = meta[n_seq * kQ4SeqWords];
  const int w1 = (int)(total * (blockIdx.x + 1) / gridDim.x);
  int ask_slot = 0, ask_which = 0, ask_item = 0, ask_pg = 0, ask_page = 0;
  uint32_t ask_phase = 1;  // parity of the slot's last release; the first round waits for none
  bool more = false;
  auto ask = [&]() {
    if (!mbar_wait(&empty[ask_slot], ask_phase)) g_err_attention_q4 = 1u;
    Cursor* it = items + (ask_item & (kAhead - 1));
    request<D>(*it, ask_pg, ask_page, ask_which, pool, hkv, smem + ask_slot * S::half, &full[ask_slot]);
    if (++ask_slot == kSlots) ask_slot = 0, ask_phase ^= 1;
    if ((ask_which ^= 1) != 0) return;
    if (++ask_pg == it->pg_end) {
      more = it->end() < w1;
      if (!more) return;
      Cursor* then = items + (++ask_item & (kAhead - 1));
      *then = *it;
      then->next<ROWS>(meta, hkv, G);
      ask_pg = then->pg;
      *known = ask_item + 1;
      it = then;
    }
    ask_page = meta[it->q.pg_at + ask_pg];  // not waited for before the next call
  };
  if (warp == 0) {
    const int w0 = (int)(total * blockIdx.x / gridDim.x);
    Cursor first;
    more = w0 < w1 && first.start<ROWS>(meta, n_seq, hkv, G, w0) && first.at < w1;
    if (lane == 0) {
      *known = more;
      if (more) *items = first;
    }
    ask_pg = first.pg;
    if (more) ask_page = meta[first.q.pg_at + ask_pg];
  }
  __syncthreads();
  if (*known == 0) return;
  if (tid == 0)  // meanwhile warp 1 stages the rows
    for (int i = 0; i < kSlots - 1 && more; ++i) ask();

  int slot = 0;
  uint32_t phase = 0;
  auto release = [&]() {  // this warp is done with the slot
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (++slot == kSlots) slot = 0, phase ^= 1;
  };
  for (int item = 0;; ++item) {
    const Cursor* cur = items + (item & (kAhead - 1));
    const int len = cur->q.len, n_new = cur->q.n_new, window = cur->q.window, row0 = cur->rt * ROWS, R = G * n_new;
    if (cur->fresh) {
      if (warp == 1) {  // column g, dimensions D/4 c ..
        const int r = row0 + (g & (ROWS - 1)), j = r / G, gi = r - j * G;
        const bool live = r < R;
        float x[D / 4];
        const float* src = q + (size_t)(cur->q.tok0 + j) * q_stride + (size_t)(cur->h * G + gi) * D + c * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const float4 v = live ? __ldcg(reinterpret_cast<const float4*>(src) + i) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[4 * i] = v.x * scale_log2e, x[4 * i + 1] = v.y * scale_log2e;
          x[4 * i + 2] = v.z * scale_log2e, x[4 * i + 3] = v.w * scale_log2e;
        }
        // the row over a power of two that brings its largest value to [2^10, 2^11):
        // the split keeps its 22 bits whatever q's size
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) m = fmaxf(m, fabsf(x[i]));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const int e = min(max((int)(__float_as_uint(m) >> 23), 11), 254);
        const float row_scale = __uint_as_float((uint32_t)(e - 10) << 23);  // 2^-10 of that
        const float inv = __uint_as_float((uint32_t)(264 - e) << 23);
        float row_sum = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) {
          x[i] *= inv;
          row_sum += x[i];
        }
        row_sum += __shfl_xor_sync(0xFFFFFFFFu, row_sum, 1);
        row_sum += __shfl_xor_sync(0xFFFFFFFFu, row_sum, 2);
        // a row past the last: q = 0, the keys of the last token; never written
        if (c == 0)
          rowp[g] = make_float4(row_scale, row_sum,
                                           __int_as_float(live ? len - n_new + j : len - 1), 0.0f);
        // word w holds dimensions 8w .. 8w+7 of the piece, paired (n, n + 4)
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint4 v;  // hi of the step's two halves, then lo
            split(pack(x[8 * w + 2 * b], x[8 * w + 2 * b + 4]), v.x, v.z);
            split(pack(x[8 * w + 2 * b + 1], x[8 * w + 2 * b + 5]), v.y, v.w);
            if constexpr (kFew)
              reinterpret_cast<uint2*>(qs)[(2 * w + b) * 32 + lane] = g < 4 ? make_uint2(v.x, v.y) : make_uint2(v.z, v.w);
            else
              qs[(2 * w + b) * 32 + lane] = v;
          }
      }
      __syncthreads();
    }
    // the two rows: the scale taken out of q, sum(q), the last key seen
    f2 scale2, sum2;
    int hi0, hi1;
    {
      const float4 a = rowp[2 * pair], b = rowp[2 * pair + 1];
      scale2 = pack(a.x, b.x);
      sum2 = pack(a.y, b.y);
      hi0 = __float_as_int(a.z), hi1 = __float_as_int(b.z);
    }
    const int back = window > 0 ? window - 1 : 0x7FFFFFFF;  // keys seen before the last
    float o[NT][4];
    float M0, M1;
    f2 lsum, zsum;
    {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.0f;
      M0 = M1 = -INFINITY;
      lsum = zsum = 0;
    }
    // what any row of the item can see, and what every row sees
    const int j0 = row0 / G, j1 = min(row0 + ROWS - 1, R - 1) / G;
    const int first_hi = len - n_new + j0, last_hi = len - n_new + j1;
    const int any_lo = first_hi - back, all_lo = window > 0 ? len - window : 0;

    int key0 = ((cur->q.chunk0 + cur->pg) << 7) + 32 * warp;  // this warp's first key of the page
    for (int left = cur->pg_end - cur->pg; left > 0; --left, key0 += kQ4Page) {
      const bool some = key0 <= last_hi && key0 + 31 >= any_lo;
      const bool whole = key0 + 31 <= first_hi && key0 >= all_lo;  // no row hides a key
      const auto hidden = [&](int key, int last) { return key > last || last - key > back; };
      // ---- scores of 32 keys, two tiles of 16, from centred codes.  (The bare codes,
      // below fp16's normal range, would need no conversion and took 5% off the time
      // at 65536 keys; but the tensor cores drop low bits of such products: the
      // output was off by 4e-6 of its size, against 5e-7.)
      if (!mbar_wait(&full[slot], phase)) g_err_attention_q4 = 1u;
      __syncwarp();
      f2 x[2][2];  // [tile][half]: s of keys 16t + 8h + g and the two rows, over the row's scale
      if (some) {
        const uint8_t* blk = smem + slot * S::half;
        float sc[2][2][4];  // [tile][hi, lo of q; or halves of the sum]: keys g, g, g + 8, g + 8 of columns 2c, 2c + 1
        uint32_t kw[2][2][W];   // [tile][key g, g + 8]
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* kp = blk + (32 * warp + 16 * t + 8 * h + g) * (D / 2) + c * (D / 8);
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(kp);
              kw[t][h][0] = v.x, kw[t][h][1] = v.y, kw[t][h][2] = v.z, kw[t][h][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(kp);
              kw[t][h][0] = v.x, kw[t][h][1] = v.y;
            }
          }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          __half2 u[2][4], v[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) q4_unpack(kw[t][0][w], u[t]), q4_unpack(kw[t][1][w], v[t]);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint4 q4;
            if constexpr (kFew) {
              const uint2 q2 = reinterpret_cast<const uint2*>(qs)[(2 * w + b) * 32 + lane];
              q4 = make_uint4(q2.x, q2.y, 0, 0);
            } else {
              q4 = qs[(2 * w + b) * 32 + lane];
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t a0 = bits(u[t][2 * b]), a1 = bits(v[t][2 * b]), a2 = bits(u[t][2 * b + 1]),
                             a3 = bits(v[t][2 * b + 1]);
              if constexpr (kFew) {
                if (w == 0)
                  mma_from(sc[t][b], a0, a1, a2, a3, q4.x, q4.y, 0.0f, 0.0f);
                else
                  mma(sc[t][b], a0, a1, a2, a3, q4.x, q4.y);
              } else if (w == 0 && b == 0) {
                mma_from(sc[t][0], a0, a1, a2, a3, q4.x, q4.y, 0.0f, 0.0f);
                mma_from(sc[t][1], a0, a1, a2, a3, q4.z, q4.w, 0.0f, 0.0f);
              } else {
                mma(sc[t][0], a0, a1, a2, a3, q4.x, q4.y);
                mma(sc[t][1], a0, a1, a2, a3, q4.z, q4.w);
              }
            }
          }
        }
        // s = d acc + z sum(q)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 dz =
                __half22float2(*reinterpret_cast<const __half2*>(blk + B::kz + (32 * warp + 16 * t + 8 * h + g) * 4));
            f2 acc = add2(pack(sc[t][0][2 * h], sc[t][0][2 * h + 1]), pack(sc[t][1][2 * h], sc[t][1][2 * h + 1]));
            if constexpr (kFew) {  // hi parts' and lo parts' columns
              const float2 v = unpack(acc);
              acc = add2(acc, pack(__shfl_xor_sync(0xFFFFFFFFu, v.x, 2), __shfl_xor_sync(0xFFFFFFFFu, v.y, 2)));
            }
            x[t][h] = fma2(pack(dz.x, dz.x), acc, mul2(pack(dz.y, dz.y), sum2));
          }
      }
      release();
      if (tid == 0 && more) ask();

      if (!mbar_wait(&full[slot], phase)) g_err_attention_q4 = 1u;
      __syncwarp();
      if (some) {
        const uint8_t* blk = smem + slot * S::half;
        __half2 vn[2][2];  // V's numbers of the thread's keys
        {
          // score plus the log of the key's own V scale, for each row over the keys
          // that it sees: what another row sees, or a key without weight, does not
          // move a row's reference
          float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              vn[t][h] = *reinterpret_cast<const __half2*>(blk + B::kz + (32 * warp + 16 * t + 8 * h + g) * 4);
              const float vd_log = lg2(fmaxf(__low2float(vn[t][h]), kLeastScale));
              float2 v = unpack(fma2(scale2, x[t][h], pack(vd_log, vd_log)));
              if (!whole) {
                const int key = key0 + 16 * t + 8 * h + g;
                if (hidden(key, hi0)) v.x = -INFINITY;
                if (hidden(key, hi1)) v.y = -INFINITY;
              }
              top0 = fmaxf(top0, v.x);
              top1 = fmaxf(top1, v.y);
            }
#pragma unroll
          for (int s4 = 4; s4 < 32; s4 <<= 1) {
            top0 = fmaxf(top0, __shfl_xor_sync(0xFFFFFFFFu, top0, s4));
            top1 = fmaxf(top1, __shfl_xor_sync(0xFFFFFFFFu, top1, s4));
          }
          // The reference is set 2^10 below the largest weight times scale and moves only when
          // that has grown to 2^14 of it: fp16 ends at 2^16, and a low part is never
          // coarser than 2^-35 of the largest.
          if (__any_sync(0xFFFFFFFFu, top0 > M0 + 14.0f || top1 > M1 + 14.0f)) {
            const float to0 = top0 > M0 + 14.0f ? top0 - 10.0f : M0;
            const float to1 = top1 > M1 + 14.0f ? top1 - 10.0f : M1;
            if (__any_sync(0xFFFFFFFFu, M0 != -INFINITY || M1 != -INFINITY)) {  // else nothing is summed yet
              const float f0 = M0 == -INFINITY ? 0.0f : ex2(M0 - to0);
              const float f1 = M1 == -INFINITY ? 0.0f : ex2(M1 - to1);
              lsum = mul2(lsum, pack(f0, f1));
              zsum = mul2(zsum, pack(f0, f1));
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                o[t][0] *= f0, o[t][1] *= f1;
                o[t][2] *= f0, o[t][3] *= f1;
              }
            }
            M0 = to0, M1 = to1;
          }
        }
        // ---- weights, and 16 keys at a time their product with V
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t ph[2], pl[2];  // P^T: keys 2c, 2c + 1 of row g, hi and lo, of the tile's halves; of column g
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 dz = __half22float2(vn[t][h]);
            f2 d = pack(dz.x, dz.x), z = pack(dz.y, dz.y);
            const float2 v = unpack(fma2(scale2, x[t][h], pack(-M0, -M1)));
            float2 pr = make_float2(ex2(v.x), ex2(v.y));
            if (!whole) {  // a hidden key's numbers may be anything
              const int key = key0 + 16 * t + 8 * h + g;
              const bool no0 = hidden(key, hi0), no1 = hidden(key, hi1);
              if (no0) pr.x = 0.0f;
              if (no1) pr.y = 0.0f;
              d = pack(no0 ? 0.0f : dz.x, no1 ? 0.0f : dz.x);
              z = pack(no0 ? 0.0f : dz.y, no1 ? 0.0f : dz.y);
            }
            const f2 pp = pack(pr.x, pr.y);
            lsum = add2(lsum, pp);
            zsum = fma2(pp, z, zsum);
            split(mul2(pp, d), ph[h], pl[h]);
            if constexpr (kFew) {
              ph[h] = transpose8(first_half ? ph[h] : pl[h]);
            } else {
              ph[h] = transpose8(ph[h]);
              pl[h] = transpose8(pl[h]);
            }
          }
          uint32_t v0[W], v1[W];
          const uint8_t* vp = blk + (16 * warp + 8 * t + c) * D + g * (D / 8);
          if constexpr (D == 128) {
            const uint4 u0 = *reinterpret_cast<const uint4*>(vp), u1 = *reinterpret_cast<const uint4*>(vp + 4 * D);
            v0[0] = u0.x, v0[1] = u0.y, v0[2] = u0.z, v0[3] = u0.w;
            v1[0] = u1.x, v1[1] = u1.y, v1[2] = u1.z, v1[3] = u1.w;
          } else {
            const uint2 u0 = *reinterpret_cast<const uint2*>(vp), u1 = *reinterpret_cast<const uint2*>(vp + 4 * D);
            v0[0] = u0.x, v0[1] = u0.y;
            v1[0] = u1.x, v1[1] = u1.y;
          }
          // tile j: its rows g and g + 8 are dimensions D/8 g + 2j and + 1
#pragma unroll
          for (int w = 0; w < W; ++w) {
            __half2 h0[4], h1[4];
            q4_unpack(v0[w], h0);
            q4_unpack(v1[w], h1);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              mma(o[2 * w + i], bits(h0[2 * i]), bits(h0[2 * i + 1]), bits(h1[2 * i]), bits(h1[2 * i + 1]),
                  ph[0], ph[1]);
            if constexpr (!kFew) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                mma(o[2 * w + i], bits(h0[2 * i]), bits(h0[2 * i + 1]), bits(h1[2 * i]), bits(h1[2 * i + 1]),
                    pl[0], pl[1]);
            }
          }
        }
      }
      release();
      if (tid == 0 && more) ask();
    }

    // ---- the unit's end.  A thread's rows and dimensions are the same in every
    // warp: warps two apart swap halves of their tiles and add the ones they keep,
    // then neighbours halves of those, so that warp w ends with the sums of the
    // w-th quarter of the tiles.
#pragma unroll
    for (int s4 = 4; s4 < 32; s4 <<= 1) {
      const float2 l = unpack(lsum), z = unpack(zsum);
      lsum = add2(lsum, pack(__shfl_xor_sync(0xFFFFFFFFu, l.x, s4), __shfl_xor_sync(0xFFFFFFFFu, l.y, s4)));
      zsum = add2(zsum, pack(__shfl_xor_sync(0xFFFFFFFFu, z.x, s4), __shfl_xor_sync(0xFFFFFFFFu, z.y, s4)));
    }
    {
      const float2 z = first_half ? unpack(zsum) : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        o[t][0] += z.x, o[t][1] += z.y;
        o[t][2] += z.x, o[t][3] += z.y;
      }
    }
    const bool mine = row0 + 2 * pair < R;  // else the thread's rows are nobody's
    // The region and statistics that a warp reads in one round are the ones it writes
    // in the next, be it the next item's: no other warp reads them, so that the two
    // barriers are enough.  A lane writes the tiles that it has read itself, but the
    // statistics that all lanes have read are written by the first of them: the warp
    // meets before each round's writes.
    const auto swap = [&](auto upper, auto tiles, int to, int from) {
      constexpr int n = decltype(tiles)::value / 2, keep = decltype(upper)::value ? n : 0, give = n - keep;
      float4* dst = join + to * (NT / 2 * 32) + lane;
      __syncwarp();
      if (mine) {
#pragma unroll
        for (int t = 0; t < n; ++t)
          dst[t * 32] = make_float4(o[give + t][0], o[give + t][1], o[give + t][2], o[give + t][3]);
        const float2 l = unpack(lsum);
        if (g == 0) stat[to * 4 + c] = make_float4(M0, M1, l.x, l.y);
      }
      __syncthreads();
      if (mine) {
        const float4* src = join + from * (NT / 2 * 32) + lane;
        const float4 b = stat[from * 4 + c];
        const float2 l = unpack(lsum);
        const float t0 = fmaxf(M0, b.x), t1 = fmaxf(M1, b.y);
        // no maximum: nothing was seen, or only NaN scores, which the sums carry
        const float a0 = M0 == t0 ? 1.0f : ex2(M0 - t0), a1 = M1 == t1 ? 1.0f : ex2(M1 - t1);
        const float b0 = b.x == t0 ? 1.0f : ex2(b.x - t0), b1 = b.y == t1 ? 1.0f : ex2(b.y - t1);
        M0 = t0, M1 = t1;
        lsum = pack(__fadd_rn(__fmul_rn(a0, l.x), __fmul_rn(b0, b.z)), __fadd_rn(__fmul_rn(a1, l.y), __fmul_rn(b1, b.w)));
#pragma unroll
        for (int t = 0; t < n; ++t) {
          const float4 v = src[t * 32];
          o[t][0] = __fmaf_rn(b0, v.x, a0 * o[keep + t][0]);
          o[t][1] = __fmaf_rn(b1, v.y, a1 * o[keep + t][1]);
          o[t][2] = __fmaf_rn(b0, v.z, a0 * o[keep + t][2]);
          o[t][3] = __fmaf_rn(b1, v.w, a1 * o[keep + t][3]);
        }
      }
    };
    const int me = item & 1 ? warp ^ 3 : warp;
    if (warp & 2)
      swap(std::true_type{}, std::integral_constant<int, NT>{}, me, me ^ 2);
    else
      swap(std::false_type{}, std::integral_constant<int, NT>{}, me, me ^ 2);
    // thread 0 may write over the item once it has passed the next barrier
    const int units = cur->units, u = cur->u, tok0 = cur->q.tok0, head0 = cur->h * G;
    if (warp & 1)
      swap(std::true_type{}, std::integral_constant<int, NT / 2>{}, me ^ 2, me ^ 3);
    else
      swap(std::false_type{}, std::integral_constant<int, NT / 2>{}, me ^ 2, me ^ 3);
    {
      constexpr int Q = NT / 4;  // tiles of this warp
      const float2 l = unpack(lsum);
      if constexpr (kFew) {
#pragma unroll
        for (int t = 0; t < Q; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][i] += __shfl_xor_sync(0xFFFFFFFFu, o[t][i], 2);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = row0 + 2 * pair + e;
        if (r >= R || !first_half) continue;
        const int j = r / G, dim = g * (D / 8) + warp * (2 * Q);
        const size_t row = (size_t)(tok0 + j) * hq + head0 + r - j * G;
        const float le = e ? l.y : l.x;
        if (units == 1) {
          float2* dst = reinterpret_cast<float2*>(out + row * D + dim);
#pragma unroll
          for (int t = 0; t < Q; ++t) dst[t] = make_float2(__fdiv_rn(o[t][e], le), __fdiv_rn(o[t][2 + e], le));
        } else {
          float* at = partials + (row * max_units + u) * (D + 2);
          float2* dst = reinterpret_cast<float2*>(at + 2 + dim);
#pragma unroll
          for (int t = 0; t < Q; ++t) dst[t] = make_float2(o[t][e], o[t][2 + e]);
          if (warp == 0 && g == 0) *reinterpret_cast<float2*>(at) = make_float2(e ? M1 : M0, le);
        }
      }
    }
    if (*known <= item + 1) break;  // the last half page was asked for long ago: no more items will be known
  }
}

// One CTA of D threads per (token row, query head): the units' (maximum, sum,
// row) joined in unit order.  Sequences of one unit are done already.  Bound by
// latency: 640 rows of up to 16 units 4.3 us, 128 rows of up to 64 units 7.6 us.
template <int D, int N>
__global__ void __launch_bounds__(D) attention_q4_merge_kernel(const float* __restrict__ partials, int hq, int n_seq,
                                                               int max_units, float* __restrict__ out,
                                                               const __grid_constant__ ParamWords<N> words,
                                                               const int32_t* __restrict__ meta_dev) {
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  const int t = blockIdx.x, head = blockIdx.y, dim = threadIdx.x, lane = dim & 31;
  int lo = 0, hi = n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (meta[mid * kQ4SeqWords + 1] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int32_t* p = meta + lo * kQ4SeqWords;
  const int pages = ((p[3] - 1) >> 7) - p[5] + 1, units = (pages + p[7] - 1) / p[7];
  const bool listed = t >= p[1] && t < p[1] + p[2];  // the launch may be for some of the sequences
  pdl_wait();
  pdl_trigger();
  if (units == 1 || !listed) return;
  const size_t row = (size_t)t * hq + head;
  const float* base = partials + row * max_units * (D + 2);
  // 32 units at a time: their maxima and sums in the lanes, their rows all on the
  // way before the first is used
  constexpr int kBatch = 16;
  float M = -INFINITY, m0 = -INFINITY, l0 = 0.0f, v[kBatch];
  if (lane < units) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(base + (size_t)lane * (D + 2)));
    m0 = ml.x, l0 = ml.y;
  }
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    if (i < units) v[i] = __ldcg(base + (size_t)i * (D + 2) + 2 + dim);
  M = m0;
  for (int u = lane + 32; u < units; u += 32) M = fmaxf(M, __ldcg(base + (size_t)u * (D + 2)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float l = 0.0f, acc = 0.0f;
  for (int u0 = 0; u0 < units; u0 += 32) {
    if (u0 > 0) {
      m0 = -INFINITY, l0 = 0.0f;
      if (u0 + lane < units) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(base + (size_t)(u0 + lane) * (D + 2)));
        m0 = ml.x, l0 = ml.y;
      }
    }
    const float f = m0 == -INFINITY ? (M == -INFINITY ? 1.0f : 0.0f) : ex2(m0 - M);
    l = __fmaf_rn(f, l0, l);
    const int n = min(32, units - u0);
    for (int b = 0; b < n; b += kBatch) {
      if (u0 + b > 0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (b + i < n) v[i] = __ldcg(base + (size_t)(u0 + b + i) * (D + 2) + 2 + dim);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, (b + i) & 31);
        if (b + i < n) acc = __fmaf_rn(w, v[i], acc);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l = __fadd_rn(l, __shfl_xor_sync(0xFFFFFFFFu, l, o));
  out[row * D + dim] = __fdiv_rn(acc, l);
}

template <int D, int ROWS, int N>
cudaError_t attention_go(const Q4AttnArgs& a, const MetaArg& meta, cudaStream_t st) {
  constexpr int smem = Q4Smem<D>::bytes;
  auto kern = attention_q4_kernel<D, ROWS, N>;
  int resident = 0;
  {
    static std::mutex mu;
    static int cache[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64) resident = cache[dev];
    if (resident == 0) {
      int per_sm = 0, sms = 0;
      if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
      if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem)) != cudaSuccess) return e;
      if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
      resident = (per_sm > 0 ? per_sm : 1) * sms;
      if (dev >= 0 && dev < 64) cache[dev] = resident;
    }
  }
  ParamWords<N> w;
  fill_words(meta, &w);
  const unsigned grid = (unsigned)(a.items < resident ? a.items : resident);
  return launch_kernel(kern, dim3(grid), dim3(kThreads), smem, st, a.q, a.q_stride, a.hq, a.hkv,
                       static_cast<const uint8_t*>(a.pool), a.n_seq, (float)(1.4426950408889634 / sqrt((double)D)),
                       a.max_units, a.partials, a.out, w, meta.dev);
}

template <int D, int N>
cudaError_t merge_go(const Q4AttnArgs& a, const MetaArg& meta, cudaStream_t st) {
  ParamWords<N> w;
  fill_words(meta, &w);
  // the join's CTAs may start while the last units run (they wait for them)
  const bool was = pdl();
  set_pdl(true);
  const cudaError_t e =
      launch_kernel(attention_q4_merge_kernel<D, N>, dim3((unsigned)a.n_tok, (unsigned)a.hq), dim3(D), 0, st, a.partials,
                    a.hq, a.n_seq, a.max_units, a.out, w, meta.dev);
  set_pdl(was);
  return e;
}

template <int D>
cudaError_t attention_pick(const Q4AttnArgs& a, const MetaArg& meta, cudaStream_t st) {
  cudaError_t e;
  if (a.tile_rows == 4)
    e = with_words(meta, [&](auto n) { return attention_go<D, 4, decltype(n)::value>(a, meta, st); });
  else if (a.tile_rows == 8)
    e = with_words(meta, [&](auto n) { return attention_go<D, 8, decltype(n)::value>(a, meta, st); });
  else
    e = launch_attention_q4_tc(a, meta, st);
  if (e != cudaSuccess || a.max_units == 1) return e;
  return with_words(meta, [&](auto n) { return merge_go<D, decltype(n)::value>(a, meta, st); });
}

}  // namespace

// Long units cost less joining, short ones fill the GPU with few sequences: the
// sequence alone makes up to 1024 items (heads and row tiles included), of two or
// four pages at least where it has many.  At most eight: the tensor cores' sums
// drop the bits below their last, toward zero, and over units of 16 pages that
// made the output of 65536 keys 1.1e-6 of its size off, over eight 0.9e-6 (191 and
// 193 us).  One unit for up to 8 pages, without a join, is faster for many sequences at
// once (64 of 12 heads: 29 us, not 33) and slower for few (one of 1000 keys: 19, not 13).
// The tcgen05 kernel's units, whose sums are float32's from page to page, have more to
// set up and to add up at their end: up to 128 items, of at most 16 pages (one sequence
// of 32768 keys, 40 rows: 85 us with the 32 pages that makes, 65 with 16).
int q4_unit_pages(int n, int lanes, int tile_rows) {
  const bool tc = tile_rows > 8;
  const long long alone = tc ? 128 : 1024;
  if (n <= 2) return n;
  const int least = tc ? 4 : n <= 4 ? 1 : n <= 64 ? 2 : 4;  // tc: n is more than 16
  const int cap = tc ? 16 : 8, most = n < cap ? n : cap;
  const long long u = ((long long)n * lanes + alone - 1) / alone;
  return u < least ? least : u > most ? most : (int)u;
}

cudaError_t launch_attention_q4(const Q4AttnArgs& a, int head_dim, const MetaArg& meta, cudaStream_t st) {
  if (a.items == 0) return cudaSuccess;
  if (head_dim == 128) return attention_pick<128>(a, meta, st);
  if (head_dim == 64) return attention_pick<64>(a, meta, st);
  return cudaErrorInvalidValue;
}

unsigned int read_clear_error_attention_q4() {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_attention_q4, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  cudaMemcpyToSymbol(g_err_attention_q4, &z, sizeof z);
  return v;
}

}  // namespace dsbk
