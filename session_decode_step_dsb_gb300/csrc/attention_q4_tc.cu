// Decode attention over the paged 4-bit KV cache for many query rows on a kv head
// (more than 16, but for 25 to 32: draft tokens, wide groups) over long sequences, on
// the 5th-generation tensor cores (sm_103a).  The mathematics is that of
// attention_q4.cu; what differs is who
// multiplies.  With many rows the warp-level products there unpack every code
// once for each 8 rows and are bound by instruction issue and the warp-level
// tensor pipe; here a page is unpacked once for up to 24 rows and two MMAs of
// 128 x N x 128 do the rest, N = 2 rows (hi and lo parts of q, and of the weights,
// as columns of their own).
//
// A CTA of 256 threads, two for each key (K, softmax) and each dimension (output),
// which share out the dimensions of K, the keys of V and the rows of the softmax:
//   K codes   the threads' row of 64 bytes becomes 64 columns of tensor memory
//             (A operand), (c - 8) as fp16
//   S^T       128 keys x N in tensor memory: thread k reads its key's scores of
//             half of the rows, applies the key's numbers and the row's reference,
//             and writes the weights' hi and lo parts as B operand of the second
//             product
//   V codes   likewise into shared memory, K-major, eight keys a store
//   O^T       D dimensions x N of one page in tensor memory, then added to float32
//             registers: the tensor core's sums round toward zero, which would tell
//             over a unit's pages
// The unpacking of V runs while the first product does, that of the next K while
// the second does; two CTAs share an SM.
//
// Measured: 8 sequences of 4096 to 16384 keys (77760 in all), 8 kv heads of 128, 40
// rows each: 132 us for two tiles of 24 (85 MB of pages, read twice).  Bound by latency:
// the phases of a page follow one another, some 800 instructions a warp (codes and
// weights to fp16, masks, sums) issued in half of the cycles by 18 warps an SM with 96
// registers a thread (8 bytes spilled); the CTA with the most pages takes a fifth longer
// than the mean.
//
// A row's reference is set 2^10 below its largest weight of the unit's first page;
// a page that brings 2^4 more (any thread sees it) is weighed again with a new one.
//
// Operand layouts (no swizzle, K-major; 8 x 8 core matrices of 8 rows of 16 bytes):
// V and the weights keep their core matrices 144 bytes apart in the direction the
// threads of a store run, so that these hit different banks.
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

constexpr int D = 128;    // head dimension
constexpr int ROWS = 24;  // query rows of an item
using B = Q4Block<D>;
constexpr int kWorkers = 256;
constexpr int kThreads = kWorkers + 32;  // and a warp that asks for the pages and issues the products
constexpr int kRing = 3;  // half pages asked for at a time
constexpr float kNoKey = -0x1.fffffep127f;  // reference of a row that has seen no key: below any score

__device__ unsigned int g_err_attention_q4_tc = 0;

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor, no swizzle: start, distance of core matrices
// along K and along M/N (all >> 4), version 1 at bit 46.
__device__ __forceinline__ uint64_t desc(const void* p, uint32_t along_k, uint32_t along_mn) {
  return (uint64_t)((smem_addr(p) & 0x3FFFFu) >> 4) | ((uint64_t)(along_k >> 4) << 16) |
         ((uint64_t)(along_mn >> 4) << 32) | (1ull << 46);
}
// kind::f16, f16 operands, f32 accumulator, both K-major, M = 128.
__device__ __forceinline__ uint32_t idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (8u << 24); }

__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_sa(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t at, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tm_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_ld4(uint32_t at, float (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tm_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// The workers' barrier; the second form tells whether any of them passed true.
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool meet_or(bool x) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, 1, 256, p;\n selp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void st_b16(uint32_t at, uint32_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"((unsigned short)v) : "memory");
}

struct TcSmem {
  static constexpr int NT = 2 * ROWS;                     // columns at most: hi and lo
  static constexpr int v_k = D / 8 * 144;                 // V: core matrices along the keys, and along the dimensions
  static constexpr int v_m = 144;
  static constexpr int p_k = 144, p_n = 16 * 144;         // weights: along the keys, along the rows
  static constexpr int q_k = 128, q_n = D / 8 * 128;        // q: along the dimensions, the rows
  static constexpr int v = 0, v_bytes = 15 * v_k + 16 * v_m;
  static constexpr int p = v + v_bytes, p_bytes = NT / 8 * p_n;
  static constexpr int q = p + p_bytes, q_bytes = NT / 8 * q_n;
  static constexpr int raw = q + q_bytes;                 // kRing half pages
  static constexpr int pairs = raw + kRing * B::v;        // [ROWS / 2] float4: scales, sums
  static constexpr int minus = pairs + ROWS / 2 * 16;     // [ROWS] -reference
  static constexpr int last = minus + ROWS * 4;           // [ROWS] last key seen
  static constexpr int top = last + ROWS * 4;             // [4][ROWS] maxima, and at the end sums
  static constexpr int top2 = top + 4 * ROWS * 4;         // [4][ROWS] offsets' sums
  static constexpr int fac = top2 + 4 * ROWS * 4;         // [ROWS] factors of a new reference
  static constexpr int where = fac + ROWS * 4;            // [ROWS] token row * query heads + head
  static constexpr int bars = where + ROWS * 4;           // ring, scores, output, keys, weights
  static constexpr int base = bars + (kRing + 4) * 8;     // tensor memory's address
  static constexpr int cursors = base + 8;
  static constexpr int bytes = cursors + 2 * (int)sizeof(Cursor) + 8;
  static constexpr int a_col = 0, s_col = D / 2, o_col = s_col + NT;
  static constexpr int cols = 256;  // a power of two; two CTAs an SM
  static_assert(o_col + NT <= 256, "tensor memory");
  static_assert(v_bytes % 16 == 0 && raw % 128 == 0 && p % 16 == 0 && q % 16 == 0, "operand alignment");
};

// Sums over the 32 lanes of the lane's COUNT values: each step halves the values
// and the lanes that share one.  Lane i ends with value i COUNT / 32.
template <int COUNT>
__device__ __forceinline__ float lane_sums(float (&v)[COUNT], int lane) {
  constexpr int STEPS = 4;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int mask = 16 >> s, n = COUNT >> (s + 1);
    const bool up = lane & mask;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float send = up ? v[j] : v[j + n], keep = up ? v[j + n] : v[j];
      v[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, mask);
    }
  }
#pragma unroll
  for (int mask = 16 >> STEPS; mask > 0; mask >>= 1) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], mask);
  return v[0];
}

template <int N>
__global__ void __launch_bounds__(kThreads, 2) attention_q4_tc_kernel(
    const float* __restrict__ q, long long q_stride, int hq, int hkv, const uint8_t* __restrict__ pool, int n_seq,
    float scale_log2e, int max_units, float* __restrict__ partials, float* __restrict__ out,
    const __grid_constant__ ParamWords<N> words, const int32_t* __restrict__ meta_dev) {
  using S = TcSmem;
  extern __shared__ __align__(128) uint8_t smem[];
  float4* pairs = reinterpret_cast<float4*>(smem + S::pairs);
  float* minus = reinterpret_cast<float*>(smem + S::minus);
  int* last = reinterpret_cast<int*>(smem + S::last);
  float* top = reinterpret_cast<float*>(smem + S::top);
  float* top2 = reinterpret_cast<float*>(smem + S::top2);
  float* fac = reinterpret_cast<float*>(smem + S::fac);
  int* where = reinterpret_cast<int*>(smem + S::where);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::bars);
  uint64_t *scores = full + kRing, *output = scores + 1;  // a product is over
  uint64_t *keys = output + 1, *weights = keys + 1;       // its operand is there
  uint32_t* base = reinterpret_cast<uint32_t*>(smem + S::base);
  Cursor* cur = reinterpret_cast<Cursor*>(smem + S::cursors);
  Cursor* ahead = cur + 1;
  int* done = reinterpret_cast<int*>(cur + 2);
  // quarter: the 32 lanes of tensor memory (keys, dimensions) of this warp; part:
  // which of the two warps on them; at: the thread's key or dimension
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3, part = warp >> 2;
  const int at = 32 * quarter + lane;
  const int G = hq / hkv;
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  if (tid == 0) {
    for (int i = 0; i < kRing + 2; ++i) mbar_init(&full[i], 1);
    mbar_init(keys, kWorkers / 32);
    mbar_init(weights, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(base)), "r"(S::cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *base, mine = tm + ((uint32_t)(32 * quarter) << 16);
  pdl_wait();
  pdl_trigger();

  // This CTA's items: those that start in its share of the pages.
  const long long total = meta[n_seq * kQ4SeqWords];
  const int w1 = (int)(total * (blockIdx.x + 1) / gridDim.x);
  if (warp == 0) {
    const int w0 = (int)(total * blockIdx.x / gridDim.x);
    Cursor first;
    const bool any = w0 < w1 && first.start<ROWS>(meta, n_seq, hkv, G, w0) && first.at < w1;
    if (lane == 0) {
      *done = !any;
      if (any) *cur = *ahead = first;
    }
  }
  __syncthreads();
  if (warp == 8) {
    // ---- the asking and issuing thread.  A half page's place in the ring is free
    // again once the operand made from it is there.
    if (lane == 0 && !*done) {
      int slot = 0, which = 0, asked = 0;
      bool more = true;
      auto ask = [&]() {
        request<D>(*ahead, ahead->pg, meta[ahead->q.pg_at + ahead->pg], which, pool, hkv, smem + S::raw + slot * B::v,
                   &full[slot]);
        ++asked;
        if (++slot == kRing) slot = 0;
        if ((which ^= 1) == 0 && ++ahead->pg == ahead->pg_end) {
          if (ahead->end() < w1)
            ahead->next<ROWS>(meta, hkv, G);
          else
            more = false;
        }
      };
      for (int i = 0; i < kRing && more; ++i) ask();
      const uint32_t id = idesc(2 * ROWS);
      const uint64_t qd = desc(smem + S::q, S::q_k, S::q_n);
      const uint64_t vd = desc(smem + S::v, S::v_k, S::v_m), pd = desc(smem + S::p, S::p_k, S::p_n);
      for (int n = 0; more || 2 * n < asked; ++n) {
        if (!mbar_wait(keys, n & 1)) g_err_attention_q4_tc = 1u;
        fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ta(tm + S::s_col, tm + S::a_col + 8 * k, qd + (uint64_t)(k * (2 * S::q_k >> 4)), id, k > 0);
        commit(scores);
        if (more) ask();
        if (!mbar_wait(weights, n & 1)) g_err_attention_q4_tc = 1u;
        fence_after();
#pragma unroll
        for (int k = 0; k < kQ4Page / 16; ++k)
          mma_sa(tm + S::o_col, vd + (uint64_t)(k * (2 * S::v_k >> 4)), pd + (uint64_t)(k * (2 * S::p_k >> 4)), id, k > 0);
        commit(output);
        if (more) ask();
      }
    }
    __syncwarp();
    __syncthreads();
    return;
  }

  int slot = 0;
  uint32_t phase = 0, s_phase = 0, o_phase = 0;
  bool multiplied = false;  // a second product has been issued that nobody has waited for
  const uint32_t p_key = smem_addr(smem + S::p) + (uint32_t)((at >> 3) * S::p_k + (at & 7) * 2);
  while (!*done) {
    const int len = cur->q.len, n_new = cur->q.n_new, window = cur->q.window, row0 = cur->rt * ROWS, R = G * n_new;
    const int rows = min(ROWS, R - row0);  // rows past them: q = 0, never written
    const bool fresh = cur->fresh;
    if (fresh) {
      // q: eight threads a row, an eighth of its dimensions each
      const int i = tid >> 3, c = tid & 7, r = row0 + i, j = r / G, gi = r - j * G;
      if (i < ROWS) {
        const bool live = i < rows;
        float x[D / 8];
        const float* src = q + (size_t)(cur->q.tok0 + j) * q_stride + (size_t)(cur->h * G + gi) * D + c * (D / 8);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const float4 v = live ? __ldcg(reinterpret_cast<const float4*>(src) + k) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[4 * k] = v.x * scale_log2e, x[4 * k + 1] = v.y * scale_log2e;
          x[4 * k + 2] = v.z * scale_log2e, x[4 * k + 3] = v.w * scale_log2e;
        }
        // the row over a power of two that brings its largest value to [2^10, 2^11):
        // the split keeps its 22 bits whatever q's size
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) m = fmaxf(m, fabsf(x[k]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const int e = min(max((int)(__float_as_uint(m) >> 23), 11), 254);
        const float inv = __uint_as_float((uint32_t)(264 - e) << 23);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          x[k] *= inv;
          sum += x[k];
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        uint8_t* hi = smem + S::q + (i >> 3) * S::q_n + (i & 7) * 16;
        uint8_t* lo = hi + ROWS / 8 * S::q_n;
        if (c == 0) {
          float* to = reinterpret_cast<float*>(&pairs[i >> 1]) + (i & 1);
          to[0] = __uint_as_float((uint32_t)(e - 10) << 23);
          to[2] = sum;
          last[i] = live ? len - n_new + j : len - 1;
          where[i] = (cur->q.tok0 + j) * hq + cur->h * G + gi;
        }
        // eight dimensions in the order of their nibbles, (0, 4), (1, 5), ..
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint4 a, b;
          split(pack(x[8 * w], x[8 * w + 4]), a.x, b.x);
          split(pack(x[8 * w + 1], x[8 * w + 5]), a.y, b.y);
          split(pack(x[8 * w + 2], x[8 * w + 6]), a.z, b.z);
          split(pack(x[8 * w + 3], x[8 * w + 7]), a.w, b.w);
          *reinterpret_cast<uint4*>(hi + (c * (D / 64) + w) * S::q_k) = a;
          *reinterpret_cast<uint4*>(lo + (c * (D / 64) + w) * S::q_k) = b;
        }
      }
      fence_proxy_async_smem();  // q is the first product's operand
      meet();
    }
    // this thread's rows: 8c + 4 part .. + 3 for c < ROWS / 8, two to a pair
    constexpr int PAIRS = ROWS / 4;
    f2 lsum[PAIRS], zsum[PAIRS];
    float acc[2 * PAIRS];  // the output of dimension `at`
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) lsum[i] = zsum[i] = 0, acc[2 * i] = acc[2 * i + 1] = 0.0f;
    // adds the page's output, once its product is over
    auto drain = [&]() {
      if (!mbar_wait(output, o_phase)) g_err_attention_q4_tc = 1u;
      o_phase ^= 1;
      multiplied = false;
      __syncwarp();
      fence_after();
      float hi[ROWS / 8][4], lo[ROWS / 8][4];
#pragma unroll
      for (int c = 0; c < ROWS / 8; ++c) {
        tm_ld4(mine + S::o_col + 8 * c + 4 * part, hi[c]);
        tm_ld4(mine + S::o_col + ROWS + 8 * c + 4 * part, lo[c]);
      }
      tm_ld_wait();
#pragma unroll
      for (int c = 0; c < ROWS / 8; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[4 * c + i] += hi[c][i] + lo[c][i];
      fence_before();
    };
    const int back = window > 0 ? window - 1 : 0x7FFFFFFF;  // keys seen before the last
    const int first_hi = len - n_new + row0 / G, all_lo = window > 0 ? len - window : 0;
    int key0 = ((cur->q.chunk0 + cur->pg) << 7) + 32 * quarter;
    bool first = true;
    for (int left = cur->pg_end - cur->pg; left > 0; --left, key0 += kQ4Page, first = false) {
      const bool whole = key0 + 31 <= first_hi && key0 >= all_lo;  // no row hides a key of this warp
      const int key = key0 + lane;
      // ---- K: half of this thread's key into tensor memory
      if (!mbar_wait(&full[slot], phase)) g_err_attention_q4_tc = 1u;
      __syncwarp();
      f2 kd, kz;
      {
        const uint8_t* raw = smem + S::raw + slot * B::v;
        constexpr int NP = 2;  // 16-byte pieces
        uint4 w[NP];
        // in an order that turns with the lane (so that rows hit other banks), put right by selects
        const int turn = (lane >> 1) & 1;
#pragma unroll
        for (int k = 0; k < NP; ++k)
          w[k] = *reinterpret_cast<const uint4*>(raw + at * (D / 2) + part * (D / 4) + (k ^ turn) * 16);
        const uint4 first_w = w[0], second_w = w[1];
        w[0] = turn ? second_w : first_w;
        w[1] = turn ? first_w : second_w;
        const float2 dz = __half22float2(*reinterpret_cast<const __half2*>(raw + B::kz + at * 4));
        kd = pack(dz.x, dz.x);
        kz = pack(dz.y, dz.y);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          uint32_t c[16];
          const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __half2 h[4];
            q4_unpack(v[i], h);
#pragma unroll
            for (int n = 0; n < 4; ++n) c[4 * i + n] = *reinterpret_cast<const uint32_t*>(&h[n]);
          }
          tm_st16(mine + S::a_col + 16 * (NP * part + k), c);
        }
      }
      tm_st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(keys);
      if (++slot == kRing) slot = 0, phase ^= 1;

      // ---- V: codes less 8 as fp16, eight keys of a dimension together; the product
      // that reads the last page's is over
      if (multiplied) drain();
      if (!mbar_wait(&full[slot], phase)) g_err_attention_q4_tc = 1u;
      __syncwarp();
      float vd, vz;
      {
        const uint8_t* raw = smem + S::raw + slot * B::v;
#pragma unroll
        for (int it = 0; it < 2; ++it) {  // word `lane` of the key pairs of eight keys
          const int kg = warp + 8 * it;
          __half2 h[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q4_unpack(*reinterpret_cast<const uint32_t*>(raw + (4 * kg + j) * D + 4 * lane), h[j]);
          uint8_t* dst = smem + S::v + kg * S::v_k + (lane >> 1) * S::v_m + (lane & 1) * 64;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            uint4 v;
            v.x = *reinterpret_cast<const uint32_t*>(&h[0][n]);
            v.y = *reinterpret_cast<const uint32_t*>(&h[1][n]);
            v.z = *reinterpret_cast<const uint32_t*>(&h[2][n]);
            v.w = *reinterpret_cast<const uint32_t*>(&h[3][n]);
            *reinterpret_cast<uint4*>(dst + n * 16) = v;
          }
        }
        const float2 dz = __half22float2(*reinterpret_cast<const __half2*>(raw + B::kz + at * 4));
        vd = dz.x;
        vz = dz.y;
      }
      const float vd_log = lg2(fmaxf(vd, kLeastScale));

      // ---- the scores
      if (!mbar_wait(scores, s_phase)) g_err_attention_q4_tc = 1u;
      s_phase ^= 1;
      __syncwarp();
      fence_after();
      const auto hidden = [&](int row) {
        const int l = last[row];
        return key > l || l - key > back;
      };
      // s of this thread's rows over the row's scale, then p
      f2 x[PAIRS], p[PAIRS];
      {
        float hi[ROWS / 8][4], lo[ROWS / 8][4];
#pragma unroll
        for (int c = 0; c < ROWS / 8; ++c) {
          tm_ld4(mine + S::s_col + 8 * c + 4 * part, hi[c]);
          tm_ld4(mine + S::s_col + ROWS + 8 * c + 4 * part, lo[c]);
        }
        tm_ld_wait();
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          const int c = i >> 1, e = 2 * (i & 1);
          const float4 pr = pairs[4 * c + 2 * part + (i & 1)];
          x[i] = fma2(kd, add2(pack(hi[c][e], hi[c][e + 1]), pack(lo[c][e], lo[c][e + 1])), mul2(kz, pack(pr.z, pr.w)));
        }
      }
      const float limit = 14.0f - vd_log;
      const f2 vd2 = pack(vd, vd), neg1 = pack(-1.0f, -1.0f);
      const uint32_t p_hi = p_key + (uint32_t)(part * 64), p_lo = p_hi + (uint32_t)(ROWS / 8 * S::p_n);
      // Once, or twice where a row's weights have grown too far for its reference.
      for (int pass = 0;; ++pass) {
        if (first ? pass == 0 : pass > 0) {
          // New references: of every row on the unit's first page, else of those whose
          // weights have grown to 2^14; the sums so far follow.
#pragma unroll
          for (int i = 0; i < PAIRS; ++i) {
            const int row = 8 * (i >> 1) + 4 * part + 2 * (i & 1);
            const float4 pr = pairs[row / 2];
            float2 t = unpack(fma2(pack(pr.x, pr.y), x[i], pack(vd_log, vd_log)));
            if (!whole) {
              if (hidden(row)) t.x = -INFINITY;
              if (hidden(row + 1)) t.y = -INFINITY;
            }
            t.x = warp_max(t.x);
            t.y = warp_max(t.y);
            if (lane == 0) *reinterpret_cast<float2*>(&top[quarter * ROWS + row]) = t;
          }
          meet();
          if (tid < ROWS) {
            const float t = fmaxf(fmaxf(top[tid], top[ROWS + tid]), fmaxf(top[2 * ROWS + tid], top[3 * ROWS + tid]));
            if (first) {
              minus[tid] = t == -INFINITY ? -kNoKey : 10.0f - t;
            } else {
              const float old = -minus[tid], to = t > old + 14.0f ? t - 10.0f : old;
              minus[tid] = -to;
              fac[tid] = ex2(old - to);
            }
          }
          meet();
          if (!first) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
              const int row = 8 * (i >> 1) + 4 * part + 2 * (i & 1);
              const float2 f = *reinterpret_cast<const float2*>(&fac[row]);
              lsum[i] = mul2(lsum[i], pack(f.x, f.y));
              zsum[i] = mul2(zsum[i], pack(f.x, f.y));
              acc[2 * i] *= f.x;
              acc[2 * i + 1] *= f.y;
            }
          }
        }
        // weights of this key into the second product's operand; pages that every row
        // sees whole take a path of their own, free of the masks' predicates
        float most = -INFINITY;
        const auto weigh = [&](auto all) {
#pragma unroll
          for (int i = 0; i < PAIRS; ++i) {
            const int row = 8 * (i >> 1) + 4 * part + 2 * (i & 1);
            const float4 pr = pairs[row / 2];
            const float2 mm = *reinterpret_cast<const float2*>(&minus[row]);
            const float2 a = unpack(fma2(pack(pr.x, pr.y), x[i], pack(mm.x, mm.y)));
            float2 w = make_float2(ex2(a.x), ex2(a.y));
            f2 d = vd2;
            if constexpr (decltype(all)::value) {
              most = fmaxf(most, fmaxf(a.x, a.y));
            } else {  // a hidden key's numbers may be anything
              const bool no0 = hidden(row), no1 = hidden(row + 1);
              most = fmaxf(most, fmaxf(no0 ? -INFINITY : a.x, no1 ? -INFINITY : a.y));
              w = make_float2(no0 ? 0.0f : w.x, no1 ? 0.0f : w.y);
              d = pack(no0 ? 0.0f : vd, no1 ? 0.0f : vd);
            }
            p[i] = pack(w.x, w.y);
            const f2 wd = mul2(p[i], d);
            const float2 v = unpack(wd);
            const __half2 hi = __floats2half2_rn(v.x, v.y);
            const float2 back2 = __half22float2(hi);
            const float2 rest = unpack(fma2(pack(back2.x, back2.y), neg1, wd));
            const __half2 lo = __floats2half2_rn(rest.x, rest.y);
            const uint32_t hb = *reinterpret_cast<const uint32_t*>(&hi), lb = *reinterpret_cast<const uint32_t*>(&lo);
            const uint32_t to = (uint32_t)((i >> 1) * S::p_n + 2 * (i & 1) * 16);
            st_b16(p_hi + to, hb);
            st_b16(p_hi + to + 16, hb >> 16);
            st_b16(p_lo + to, lb);
            st_b16(p_lo + to + 16, lb >> 16);
          }
        };
        if (whole)
          weigh(std::true_type{});
        else
          weigh(std::false_type{});
        fence_proxy_async_smem();  // V and the weights precede the product
        fence_before();
        if (!meet_or(pass == 0 && !first && most > limit)) break;
      }
      if (tid == 0) arrive(weights);
      multiplied = true;
      if (++slot == kRing) slot = 0, phase ^= 1;
      if (whole) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) zsum[i] = fma2(p[i], pack(vz, vz), zsum[i]);
      } else {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          const int row = 8 * (i >> 1) + 4 * part + 2 * (i & 1);
          zsum[i] = fma2(p[i], pack(hidden(row) ? 0.0f : vz, hidden(row + 1) ? 0.0f : vz), zsum[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) lsum[i] = add2(lsum[i], p[i]);
    }

    // ---- the unit's end: sums over the keys, then the output by dimension
    drain();
    {
      constexpr int COUNT = 16;  // two for each pair, rounded up to a power of two
      float l[COUNT], z[COUNT];
#pragma unroll
      for (int i = 0; i < COUNT / 2; ++i) {
        const float2 a = unpack(i < PAIRS ? lsum[i] : 0), b = unpack(i < PAIRS ? zsum[i] : 0);
        l[2 * i] = a.x, l[2 * i + 1] = a.y;
        z[2 * i] = b.x, z[2 * i + 1] = b.y;
      }
      const float ls = lane_sums<COUNT>(l, lane), zs = lane_sums<COUNT>(z, lane);
      constexpr int SHARE = 32 / COUNT;  // lanes with the same sum
      const int i = lane / SHARE, row = 8 * (i >> 2) + 4 * part + (i & 3);
      if (lane % SHARE == 0 && i < 2 * PAIRS) {
        top[quarter * ROWS + row] = ls;
        top2[quarter * ROWS + row] = zs;
      }
    }
    meet();
    {
      const int units = cur->units, u = cur->u;
#pragma unroll
      for (int i = 0; i < 2 * PAIRS; ++i) {
        const int r = 8 * (i >> 2) + 4 * part + (i & 3);
        if (r < rows) {
          const float l = (top[r] + top[ROWS + r]) + (top[2 * ROWS + r] + top[3 * ROWS + r]);
          const float z = (top2[r] + top2[ROWS + r]) + (top2[2 * ROWS + r] + top2[3 * ROWS + r]);
          const size_t row = (size_t)where[r];
          if (units == 1) {
            out[row * D + at] = __fdiv_rn(acc[i] + z, l);
          } else {
            float* to = partials + (row * max_units + u) * (D + 2);
            to[2 + at] = acc[i] + z;
            if (at == 0) *reinterpret_cast<float2*>(to) = make_float2(-minus[r], l);
          }
        }
      }
    }
    fence_before();
    meet();  // every thread has read the item and the output
    if (tid == 0) {
      *done = cur->end() >= w1;
      if (!*done) cur->next<ROWS>(meta, hkv, G);
    }
    meet();
  }
  __syncthreads();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(S::cols) : "memory");
  }
}

template <int N>
cudaError_t tc_go(const Q4AttnArgs& a, const MetaArg& meta, cudaStream_t st) {
  constexpr int smem = TcSmem::bytes;
  static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs an SM");
  auto kern = attention_q4_tc_kernel<N>;
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
      int sms = 0;
      if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
      if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
      resident = 2 * sms;
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

}  // namespace

cudaError_t launch_attention_q4_tc(const Q4AttnArgs& a, const MetaArg& meta, cudaStream_t st) {
  return with_words(meta, [&](auto n) { return tc_go<decltype(n)::value>(a, meta, st); });
}

unsigned int read_clear_error_attention_q4_tc() {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_attention_q4_tc, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  cudaMemcpyToSymbol(g_err_attention_q4_tc, &z, sizeof z);
  return v;
}

}  // namespace dsbk
