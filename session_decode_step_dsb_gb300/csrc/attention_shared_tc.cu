// Decode attention over shared 16-bit pages for many query rows on a kv head (the drafts
// and sessions of a group together, prompts), on the 5th-generation tensor cores
// (sm_103a).  The mathematics is that of attention_shared.cu.
//
// A CTA takes 128 query rows of a kv head through its share of pages, 128 keys at a time:
//   S = Q K^T   128 x 128, Q in parts (fp16: two; bf16: three, so that a product keeps
//               float32's bits) in shared memory, K as it lies in the page
//   P           256 threads, two to a row; weights go back to tensor memory in as many
//               parts, the first two over the scores that they come from
//   O = P V     128 x D of one page, V as it lies in the page; 256 more threads add it to
//               float32 registers (the tensor core's sums round toward zero) and write
//               the rows at the end, while the others begin the next
// The scores of the next page are multiplied while the weights of this one are made:
// S(n + 1) lies between P V(n - 1) and P V(n).  A warp of its own asks for the pages (TMA,
// two of K and two of V), another issues the products.  Bound by the products: 32 (fp16) or 48
// (bf16) of 128 x 128 x 16 for a page of 128-wide heads.
//
// Measured (GB300), 128-wide heads, 40 on 8: prompts of 4 x 1000 tokens behind 4096 keys, bf16,
// 689 us with the join, 0.55 PFLOP/s, in three parts 1.64 (tensor pipe active 0.74 of the
// time); drafts of 32 sessions on 32768 keys, fp16, 97 us on 123 SMs (0.59).  A page takes
// 2800 cycles (fp16) or 4000 (bf16): a product with both operands in shared memory 106, one
// with its left operand in tensor memory 73, which makes 2860 and 4300 one after the other.
// With the fp16 Q in tensor memory too (2340) a page took as long: the weights then do.
// A change of runs takes 5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

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

// Threads that make weights, that add up the output, and a warpgroup of which one warp asks
// for pages and one issues products; and the registers of each (the launch gives 96).
constexpr int kWeighers = 256, kAdders = 256, kIssuers = 128;
constexpr int kThreads = kWeighers + kAdders + kIssuers;
constexpr int kWeigherRegs = 88, kAdderRegs = 112, kIssuerRegs = 80;
static_assert(kWeighers * kWeigherRegs + kAdders * kAdderRegs + kIssuers * kIssuerRegs <= kThreads * 96, "register split");
constexpr int kRows = 128;

__device__ unsigned int g_err_attention_shared_tc = 0;

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle: start, distance of 64-column groups
// (of an operand whose columns run along its rows), distance of groups of eight rows.
__device__ __forceinline__ uint64_t desc(uint32_t at, uint32_t groups, uint32_t eights) {
  return (uint64_t)((at & 0x3FFFFu) >> 4) | ((uint64_t)(groups >> 4) << 16) | ((uint64_t)(eights >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// kind::f16 with float32 sums, M = 128; trans_b: B's rows run along N.
template <typename T>
__device__ __forceinline__ uint32_t idesc(int n, bool trans_b) {
  const uint32_t type = std::is_same_v<T, __half> ? 0u : 1u;
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)trans_b << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// The products are issued by a warp whose lanes stay together (the operands' descriptors
// then live in its uniform registers); `one` is true in one of them.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc), "r"(one)
      : "memory");
}
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.b32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// 32 columns of this thread's row.
__device__ __forceinline__ void tm_ld32(uint32_t at, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t at, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ uint32_t tm_ld1(uint32_t at) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void tm_st8(uint32_t at, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tm_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The two weighing warps of 32 rows; the adders; the weighers; the latter telling whether any
// passed true.
__device__ __forceinline__ void meet_pair(int quarter) { asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory"); }
__device__ __forceinline__ void meet_adders() { asm volatile("bar.sync 6, 256;" ::: "memory"); }
__device__ __forceinline__ void meet() { asm volatile("bar.sync 5, 256;" ::: "memory"); }
__device__ __forceinline__ bool meet_or(bool x) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, 5, 256, p;\n selp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)x)
      : "memory");
  return r != 0;
}

template <typename T>
__device__ __forceinline__ float half_of(uint32_t w, int which) {
  const uint16_t h = (uint16_t)(which ? w >> 16 : w);
  if constexpr (std::is_same_v<T, __half>)
    return __half2float(__ushort_as_half(h));
  else
    return __uint_as_float((uint32_t)h << 16);
}

template <int D, typename T>
struct Smem {
  static constexpr int parts = Parts<T>::kMore + 1;
  static constexpr int slab = 128 * 128;                // 64 columns of 128 rows
  static constexpr int tile = D / 64 * slab;            // a part of Q, a page of K or V
  static constexpr int q = 0;
  static constexpr int k = q + parts * tile;            // two pages
  static constexpr int v = k + 2 * tile;                // two pages
  static constexpr int top = v + 2 * tile;              // [2][128] row maxima of the halves; limits of rows
  static constexpr int stat = top + 2 * 128 * 4;        // [128] -reference, sum of weights
  static constexpr int fac = stat + 128 * 8;            // [3][128] of a page: the sums before it times 2^-fac
  static constexpr int strange = fac + 3 * 128;         // [3] of a page: keys (4 words), whether any
  static constexpr int bars = strange + 64;             // see below
  static constexpr int base = bars + 15 * 8;
  static constexpr int bytes = base + 8;
  // tensor memory: scores and weights of two pages, output, third parts of two pages
  static constexpr int s_col = 0, o_col = 256, t_col = 384;
};

template <int D, typename T, int N>
__global__ void __launch_bounds__(kThreads, 1) attention_shared_tc_kernel(
    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const float* __restrict__ q,
    long long q_stride, int hq, int hkv, const T* __restrict__ vp, int n_seg, float scale_log2e, float unit,
    PartialsOut to, bool wide, bool beside, const __grid_constant__ ParamWords<N> words, const int32_t* __restrict__ meta_dev) {
  using S = Smem<D, T>;
  constexpr int PARTS = S::parts, HD = D / 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* top = reinterpret_cast<float*>(smem + S::top);
  float2* stats = reinterpret_cast<float2*>(smem + S::stat);
  uint8_t* fac = smem + S::fac;
  unsigned* strange = reinterpret_cast<unsigned*>(smem + S::strange);
  // pages of K and of V; scores of a page; V has been read; a page's output; its weights (by
  // the weighers' warps; of two pages, since those of the next may be there before the issuer
  // has seen that these are); the output has been added (the adders'); a run's queries, its
  // statistics (weighers), and these have been read (adders).  No barrier completes a phase
  // before the one ahead of it has been seen by all that wait for it.
  uint64_t* full_k = reinterpret_cast<uint64_t*>(smem + S::bars);
  uint64_t *full_v = full_k + 2, *scores = full_v + 2, *free_v = scores + 2, *output = free_v + 2, *weights = output + 1, *added = weights + 2,
           *queries = added + 1, *stat_full = queries + 1, *stat_free = stat_full + 1;
  uint32_t* base = reinterpret_cast<uint32_t*>(smem + S::base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  const int cta = blockIdx.x, ctas = gridDim.x;
  SharedWalk cur;  // each role finds its runs anew, so that nothing of them is carried through
  int pos = cur.begin(meta, n_seg, wide, hkv, hq / hkv, kRows, kLead128, cta, ctas);
  if (tid == 0) {
    for (int i = 0; i < 9; ++i) mbar_init(&full_k[i], 1);
    mbar_init(&weights[0], kWeighers / 32);
    mbar_init(&weights[1], kWeighers / 32);
    mbar_init(added, kAdders / 32);
    mbar_init(queries, kWeighers / 32);
    mbar_init(stat_full, kWeighers / 32);
    mbar_init(stat_free, kAdders / 32);
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *base;
  if (!beside) pdl_wait();  // as in attention_pages_kernel
  pdl_trigger();
  const auto wait = [&](uint64_t* bar, int parity) {  // tells which barrier it was that did not come
    if (!mbar_wait(bar, (uint32_t)parity)) atomicOr(&g_err_attention_shared_tc, 2u << (int)(bar - full_k));
  };

  if (warp >= (kWeighers + kAdders) / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssuerRegs));
    const uint32_t one = elect();
    if (warp == (kWeighers + kAdders) / 32) {
      // ---- the asking warp: pages in the order of all runs, each place as it becomes free
      const auto ask = [&](int where, const CUtensorMap* map, int row0, uint64_t* bar) {
        if (one) {
          mbar_arrive_expect_tx(bar, S::tile);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) tma_box(smem + where + x * S::slab, map, 64 * x, row0, bar);
        }
        __syncwarp();
      };
      for (int n = 0;; pos = cur.following()) {
        cur.locate(pos);
        if (!cur.any()) break;  // a share without a page
#pragma unroll 1
        for (int i = cur.i; i < cur.i_end; ++i, ++n) {
          const int row0 = (cur.page(i) * hkv + cur.h) * kPgKeys, b = n & 1;
          if (n > 1) wait(&scores[b], (n >> 1) - 1 & 1);
          ask(S::k + b * S::tile, &tmk, row0, &full_k[b]);
          if (n > 1) wait(&free_v[b], (n >> 1) - 1 & 1);
          ask(S::v + b * S::tile, &tmv, row0, &full_v[b]);
        }
        if (!cur.another()) break;
      }
    } else if (warp == (kWeighers + kAdders) / 32 + 1) {
      // ---- the issuing warp; n counts the pages of all its runs.  The tensor core queues a few
      // products, which cover one wait at a time: the waits of a product of pages lie
      // within the one before it.
      const uint32_t id_s = idesc<T>(128, false), id_o = idesc<T>(D, true);
      const uint32_t sq = smem_addr(smem + S::q), sk = smem_addr(smem + S::k), sv = smem_addr(smem + S::v);
      const auto score = [&](int n, int part) {  // one part of the scores of page n
        const uint64_t kd = desc(sk + (n & 1) * S::tile, 0, 1024), qd = desc(sq + part * S::tile, 0, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t step = (uint64_t)((k >> 2) * (S::slab >> 4) + (k & 3) * 2);
          mma_ss(tm + S::s_col + 128 * (n & 1), qd + step, kd + step, id_s, part < PARTS - 1 || k > 0, one);
        }
      };
      const auto weigh = [&](int n, int part) {  // one part of the output of page n
        const uint64_t vd = desc(sv + (n & 1) * S::tile, S::slab, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t a = part == 2 ? tm + S::t_col + 64 * (n & 1) + 8 * k
                                       : tm + S::s_col + 128 * (n & 1) + 16 * part + 32 * (k >> 1) + 8 * (k & 1);
          mma_ts(tm + S::o_col, a, vd + (uint64_t)(k * (2048 >> 4)), id_o, part < PARTS - 1 || k > 0, one);
        }
      };
      int n = 0;
      bool odd_page = false;  // the last page was one
      for (int run = 0;; ++run, pos = cur.following()) {
        cur.locate(pos);
        if (!cur.any()) break;  // a share without a page
        const int end = n + cur.here();
        wait(queries, run & 1);
        wait(&full_k[n & 1], n >> 1 & 1);
        // the first page's scores alone, then those of a page's next with its output
#pragma unroll 1
        for (int m = n - 1; m < end; ++m) {
          const bool next = m + 1 < end, out = m >= n;
          if (next) {
            // the next scores take the place of the last weights, which a page of strange values
            // (see below) needs until it has been added
            if (out && odd_page) wait(added, (m - 1) & 1);
            fence_after();
            score(m + 1, PARTS - 1);
          }
          if (out) wait(&full_v[m & 1], m >> 1 & 1);
          if (next && PARTS > 2) score(m + 1, 1);
          if (out && m > 0) wait(added, (m - 1) & 1);  // the output's place is free
          if (next) {
            score(m + 1, 0);
            if (one) commit(&scores[(m + 1) & 1]);
            __syncwarp();
          }
          if (!out) {
            if (n + 1 < end) wait(&full_k[(n + 1) & 1], (n + 1) >> 1 & 1);
            continue;
          }
          wait(&weights[m & 1], m >> 1 & 1);
          fence_after();
#pragma unroll 1
          for (int part = PARTS - 1; part > 0; --part) weigh(m, part);
          if (m + 2 < end) wait(&full_k[m & 1], (m + 2) >> 1 & 1);  // (the first two pages': above)
          odd_page = strange[5 * (m % 3) + 4];
          weigh(m, 0);
          if (one) {
            commit(output);
            if (next) commit(&free_v[m & 1]);  // the last page's place serves the adders first
          }
          __syncwarp();
        }
        n = end;
        if (!cur.another()) break;
      }
    }
    __syncwarp();
    __syncthreads();
    return;
  }

  const int quarter = warp & 3, row = 32 * quarter + lane;
  const uint32_t mine = tm + ((uint32_t)(32 * quarter) << 16);
  int n = 0;

  if (warp >= kWeighers / 32) {
    // ---- the adders: a thread has half of a row's output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAdderRegs));
    const int d0 = (warp - kWeighers / 32) / 4 * HD;
    for (int run = 0;; ++run, pos = cur.following()) {
      cur.locate(pos);
      if (!cur.any()) break;  // a share without a page
      // where the row goes: to the output where this CTA has all of it, else to a slot
      RowAt at{0, 0, 0, 0x7FFFFFFF};
      float* dst = nullptr;
      float2* stat = nullptr;
      int empty = 0;  // slots behind the first part's that the row's parts leave
      const bool done = cur.alone() && cur.i == 0 && cur.i_end == cur.n_pages;
      if (row < cur.tile_rows()) {
        at = cur.row(row, hq);
        const int part = cur.part(cta);
        const size_t slot = (size_t)at.row * to.slots + cur.slot_base() + (done ? 0 : part);
        dst = done ? to.out + (size_t)at.row * D : to.acc + slot * D;
        if (d0 == 0 && !(done && cur.slot_cap() == 1)) {
          stat = to.stat + slot;
          if (!done && part == 0) empty = cur.slot_cap() - cur.parts();
        }
      }
      float acc[HD];
#pragma unroll
      for (int i = 0; i < HD; ++i) acc[i] = 0.0f;
      for (int i = cur.i; i < cur.i_end; ++i, ++n) {
        wait(output, n & 1);
        __syncwarp();
        fence_after();
        const int down = fac[128 * (n % 3) + row];
        const float f = down > 126 ? 0.0f : __uint_as_float((uint32_t)(127 - down) << 23);
        if (__any_sync(0xFFFFFFFFu, down)) {
#pragma unroll
          for (int k = 0; k < HD; ++k) acc[k] *= f;
        }
#pragma unroll
        for (int x = 0; x < HD / 16; ++x) {
          float o[16];
          tm_ld16(mine + S::o_col + d0 + 16 * x, o);
          tm_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) acc[16 * x + k] += o[k];
        }
        const unsigned* odd_keys = strange + 5 * (n % 3);
        if (odd_keys[4]) {
          const int key0 = cur.block(i, 0) * kPgKeys;
          const T* page = vp + ((size_t)cur.page(i) * hkv + cur.h) * kPgKeys * D;
#pragma unroll 1
          for (int w = 0; w < 4; ++w)
#pragma unroll 1
            for (unsigned left = odd_keys[w]; left; left &= left - 1) {
              const int key = 32 * w + __ffs(left) - 1;
              const uint32_t hi_at = mine + S::s_col + 128 * (n & 1) + 32 * (key >> 5) + (key & 31) / 2;
              // the weight's parts, the smallest first
              uint32_t got[3] = {tm_ld1(hi_at), tm_ld1(hi_at + 16), 0};
              if constexpr (PARTS > 2) got[2] = tm_ld1(mine + S::t_col + 64 * (n & 1) + key / 2);
              tm_ld_wait();
              const float p = (half_of<T>(got[2], key & 1) + half_of<T>(got[1], key & 1)) + half_of<T>(got[0], key & 1);
              if (key0 + key >= at.lo && key0 + key <= at.hi) {
                const uint32_t* v = reinterpret_cast<const uint32_t*>(page + (size_t)key * D + d0);
#pragma unroll
                for (int k = 0; k < HD / 2; ++k) {
                  const uint32_t two = v[k];
                  acc[2 * k] = fmaf(p, half_of<T>(two, 0), acc[2 * k]);
                  acc[2 * k + 1] = fmaf(p, half_of<T>(two, 1), acc[2 * k + 1]);
                }
              }
              __syncwarp();  // rows that see the key and others load the next one's weight together
            }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(added);
      }
      // ---- the part's end.  Rows leave through the place of V's last page, 64 dimensions at
      // a time, so that lanes write along them; the place is free for another page after that.
      wait(stat_full, run & 1);
      const float2 st = stats[row];
      __syncwarp();
      if (lane == 0) arrive(stat_free);
      if (stat) {
        *stat = done ? make_float2(0.0f, -1.0f) : make_float2(-st.x, st.y);
        for (; empty > 0; --empty) stat[empty + cur.parts() - 1] = make_float2(0.0f, 0.0f);
      }
      if (done) {
        const float by = __frcp_rn(st.y);
#pragma unroll
        for (int k = 0; k < HD; ++k) acc[k] *= by;
      }
      {
        const int b = (n - 1) & 1;
        float4* stage = reinterpret_cast<float4*>(smem + S::v + b * S::tile);  // [128][HD / 4], pieces turned by row
        constexpr int P = HD / 4;
        const int r_out = 16 * (d0 != 0) + lane / P;  // the first row that this lane writes, of its quarter
#pragma unroll
        for (int round = 0; round < 2; ++round) {
          if ((d0 != 0) == (round == 1)) {
#pragma unroll
            for (int k = 0; k < P; ++k)
              stage[row * P + (k ^ (row & (P - 1)))] = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
          }
          meet_adders();
#pragma unroll
          for (int k = 0; k < 16; k += 32 / P) {
            const int r = r_out + k, rr = 32 * quarter + r;
            float* out = reinterpret_cast<float*>(__shfl_sync(0xFFFFFFFFu, (unsigned long long)dst, r));
            if (out) reinterpret_cast<float4*>(out + round * HD)[lane % P] = stage[rr * P + ((lane % P) ^ (rr & (P - 1)))];
          }
          fence_proxy_async_smem();  // precedes the next page's copy
          meet_adders();
        }
        if (tid == kWeighers) arrive(&free_v[b]);
      }
      __syncwarp();
      if (!cur.another()) break;
    }
    fence_before();
    __syncthreads();
    return;
  }

  // ---- the weighers: thread (row, part) has half of the row's keys
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWeigherRegs));
  const int part = warp >> 2;
  for (int run = 0;; ++run, pos = cur.following()) {
    cur.locate(pos);
    if (!cur.any()) break;  // a share without a page
    const int live = cur.tile_rows();
    {
      // q: a warp takes 16 rows, lanes along them
      constexpr int LANES = D / 4, ROWS = 32 / LANES;
      const int l = lane % LANES;
      RowAt its{0, 0, 0, 0};
      const int r0 = 16 * warp, mine_q = r0 + lane % 16;
      if (mine_q < live) its = cur.row(mine_q, hq);
      its.row -= its.tok * hq;
      // four loads on their way while four rows are cut into parts
      float4 x[4], y[4];
      const auto load = [&](int j, float4* to) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (j + i) * ROWS + lane / LANES;
          const int tok = __shfl_sync(0xFFFFFFFFu, its.tok, r), head = __shfl_sync(0xFFFFFFFFu, its.row, r);
          to[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r0 + r < live) to[i] = __ldg(reinterpret_cast<const float4*>(q + (size_t)tok * q_stride + (size_t)head * D) + l);
        }
      };
      load(0, x);
#pragma unroll 1
      for (int j = 0; j < 16 / ROWS; j += 4) {
        if (j + 4 < 16 / ROWS) load(j + 4, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + (j + i) * ROWS + lane / LANES;
          float v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
          for (int o = 1; o < LANES; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          float by, after;
          row_powers<T>(m, by, after);
          if (l == 0) top[r] = after;
          by *= scale_log2e;
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] *= by;
          const int piece = l >> 1;
          uint8_t* dst = smem + S::q + (piece >> 3) * S::slab + r * 128 + (((piece & 7) ^ (r & 7)) << 4) + (l & 1) * 8;
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            const uint32_t w0 = Parts<T>::take(v[0], v[1]), w1 = Parts<T>::take(v[2], v[3]);
            *reinterpret_cast<uint2*>(dst + p * S::tile) = make_uint2(w0, w1);
          }
          x[i] = y[i];
        }
      }
    }
    fence_proxy_async_smem();  // q is the first product's operand
    __syncwarp();
    if (lane == 0) arrive(queries);
    RowAt at{0, 0, 0, 0x7FFFFFFF};
    if (row < live) at = cur.row(row, hq);
    // what the tile's rows see in common, and at all
    int all_lo = 0, all_hi = 0x7FFFFFFF, any_lo = 0x7FFFFFFF, any_hi = -1;
    float rs;
    {
      int* lim = reinterpret_cast<int*>(top + 128);  // [4 quarters][4]
      const int a = __reduce_max_sync(0xFFFFFFFFu, at.lo), b = __reduce_min_sync(0xFFFFFFFFu, at.hi);
      const int c = __reduce_min_sync(0xFFFFFFFFu, row < live ? at.lo : 0x7FFFFFFF);
      const int d = __reduce_max_sync(0xFFFFFFFFu, row < live ? at.hi : -1);
      if (lane == 0 && part == 0) *reinterpret_cast<int4*>(lim + 4 * warp) = make_int4(a, b, c, d);
      meet();
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int4 v = *reinterpret_cast<const int4*>(lim + 4 * w);
        all_lo = max(all_lo, v.x), all_hi = min(all_hi, v.y), any_lo = min(any_lo, v.z), any_hi = max(any_hi, v.w);
      }
      rs = top[row];
      meet();
    }

    float minus = kNoRef;
    f2 sum[2] = {0, 0};
    for (int i = cur.i; i < cur.i_end; ++i, ++n) {
      const int key0 = cur.block(i, 0) * kPgKeys;
      const bool whole = key0 >= all_lo && key0 + kPgKeys - 1 <= all_hi;
      const uint32_t s_at = mine + S::s_col + 128 * (n & 1) + 64 * part;
      wait(&scores[n & 1], n >> 1 & 1);
      __syncwarp();
      fence_after();
      // the keys of this half that the row sees, as bits
      unsigned long long seen = ~0ull;
      if (!whole) {
        const int from = max(at.lo - (key0 + 64 * part), 0), upto = min(at.hi - (key0 + 64 * part), 63);
        seen = from > upto ? 0ull : (~0ull >> (63 - upto)) & (~0ull << from);
      }
      const auto load = [&](int c, float* x) {
        tm_ld32(s_at + 32 * c, x);
        tm_ld_wait();
        if (!whole) {
          const uint32_t bits = (uint32_t)(seen >> (32 * c));
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = bits >> k & 1u ? x[k] : -INFINITY;
        }
      };
      float most = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        float x[32];
        load(c, x);
        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int k = 4; k < 32; ++k) m4[k & 3] = fmaxf(m4[k & 3], x[k]);
        most = fmaxf(most, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
      }
      top[part * 128 + row] = most;
      meet_pair(quarter);
      most = fmaxf(most, top[(part ^ 1) * 128 + row]) * rs;
      // references are whole numbers, so that a change of one is an exponent
      int down = 0;
      if (most + minus > Parts<T>::kRoom + kSlack) {
        const float to_minus = rintf(Parts<T>::kRoom - most);
        down = minus - to_minus < 127.0f ? (int)(minus - to_minus) : 127;
        const float f = down > 126 ? 0.0f : __uint_as_float((uint32_t)(127 - down) << 23);
        minus = to_minus;
        sum[0] = mul2(sum[0], pack(f, f));
        sum[1] = mul2(sum[1], pack(f, f));
      }
      if (part == 0) fac[128 * (n % 3) + row] = (uint8_t)down;
      // weights; a hidden key's score is -inf here, its weight 0 whatever rs and minus are
      const f2 rs2 = pack(rs, rs), minus2 = pack(minus, minus), unit2 = pack(unit, unit);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {  // the weights of 32 keys over their scores
        float x[32];
        load(c, x);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t w[PARTS][8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 e = unpack(fma2(pack(x[16 * j + 2 * k], x[16 * j + 2 * k + 1]), rs2, minus2));
            f2 two = pack(exp2_of(e.x), exp2_of(e.y));
            if constexpr (PARTS > 2) two = mul2(two, unit2);
            sum[k & 1] = add2(sum[k & 1], two);
            float p0 = unpack(two).x, p1 = unpack(two).y;
#pragma unroll
            for (int p = 0; p < PARTS; ++p) w[p][k] = Parts<T>::take(p0, p1);
          }
          tm_st8(s_at + 32 * c + 8 * j, w[0]);
          tm_st8(s_at + 32 * c + 16 + 8 * j, w[1]);
          if constexpr (PARTS > 2) tm_st8(mine + S::t_col + 64 * (n & 1) + 32 * part + 16 * c + 8 * j, w[PARTS - 1]);
        }
      }
      unsigned* odd_keys = strange + 5 * (n % 3);
      if (whole) {
        if (tid == 0) odd_keys[4] = 0;
        meet_pair(quarter);  // the maxima have been read
      } else {
        // Two threads to a key of V.  One that no row sees may hold anything: cleared.  One
        // that some rows see, with an infinity or a NaN: 0 times it is no 0, so it is
        // cleared too, and added to the rows that see it.
        wait(&full_v[n & 1], n >> 1 & 1);
        const int key = tid >> 1, half = tid & 1;
        const bool none = key0 + key > any_hi || key0 + key < any_lo;
        bool is = false;
        uint4* vrow = reinterpret_cast<uint4*>(smem + S::v + (n & 1) * S::tile + (D == 128 ? half * S::slab : half * 64) + key * 128);
        // (64-wide heads: a thread's half of the row is four pieces; the swizzle only
        // permutes the pieces of a row)
#pragma unroll
        for (int p = 0; p < D / 16; ++p) {  // (in an order that turns with the key: other banks)
          const uint4 v = vrow[p ^ (key & (D / 16 - 1))];
          is = is || odd<T>(v.x) || odd<T>(v.y) || odd<T>(v.z) || odd<T>(v.w);
        }
        is = __shfl_xor_sync(0xFFFFFFFFu, (int)is, 1) || is;
        if (none || is)
#pragma unroll
          for (int p = 0; p < D / 16; ++p) vrow[p ^ (key & (D / 16 - 1))] = make_uint4(0, 0, 0, 0);
        is = is && !none;
        if (tid < 5) odd_keys[tid] = 0;
        if (meet_or(is)) {
          if (is && half == 0) atomicOr(&odd_keys[key >> 5], 1u << (key & 31));
          if (tid == 0) odd_keys[4] = 1;
        }
        fence_proxy_async_smem();
      }
      tm_st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(&weights[n & 1]);
    }

    // ---- the part's end
    const float2 a = unpack(add2(sum[0], sum[1]));
    const float l = a.x + a.y;
    meet_pair(quarter);
    if (part == 1) top[row] = l;
    meet_pair(quarter);
    if (run > 0) wait(stat_free, (run - 1) & 1);
    if (part == 0) stats[row] = make_float2(minus, l + top[row]);
    __syncwarp();
    if (lane == 0) arrive(stat_full);
    if (!cur.another()) break;
    meet();  // the sums have been read
  }
  __syncthreads();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
    pdl_wait();
  }
}

template <int D, typename T>
cudaError_t tc_go(const PageAttnArgs& a, const MetaArg& meta, cudaStream_t st) {
  using S = Smem<D, T>;
  static_assert(S::bytes <= 227 * 1024, "shared memory");
  CUtensorMap tmk, tmv;
  cudaError_t e = kv_tensor_map(a.k, a.pool_rows, D, std::is_same_v<T, __half> ? 0 : 1, kPgKeys, &tmk);
  if (e == cudaSuccess) e = kv_tensor_map(a.v, a.pool_rows, D, std::is_same_v<T, __half> ? 0 : 1, kPgKeys, &tmv);
  if (e != cudaSuccess) return e;
  return with_words(meta, [&](auto n) {
    constexpr int N = decltype(n)::value;
    auto kern = attention_shared_tc_kernel<D, T, N>;
    static std::atomic<unsigned long long> ready{0};
    const cudaError_t err = allow_smem(kern, S::bytes, &ready);
    if (err != cudaSuccess) return err;
    ParamWords<N> w;
    fill_words(meta, &w);
    const PartialsOut to{reinterpret_cast<float2*>(a.stat), a.acc, a.out, a.slots};
    return launch_kernel(kern, dim3((unsigned)a.ctas), dim3(kThreads), (size_t)S::bytes, st, tmk, tmv, a.q, a.q_stride,
                         a.hq, a.hkv, static_cast<const T*>(a.v), a.n_seg,
                         (float)(1.4426950408889634 / std::sqrt((double)D)), a.unit, to, a.wide_pages, a.beside, w, meta.dev);
  });
}

}  // namespace

cudaError_t launch_attention_shared_tc(const PageAttnArgs& a, int dtype, int head_dim, const MetaArg& meta,
                                       cudaStream_t st) {
  if (head_dim == 128) return dtype == 0 ? tc_go<128, __half>(a, meta, st) : tc_go<128, __nv_bfloat16>(a, meta, st);
  return dtype == 0 ? tc_go<64, __half>(a, meta, st) : tc_go<64, __nv_bfloat16>(a, meta, st);
}

unsigned int read_clear_error_attention_shared_tc() {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_attention_shared_tc, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
  cudaMemcpyToSymbol(g_err_attention_shared_tc, &z, sizeof z);
  return v;
}

}  // namespace dsbk
