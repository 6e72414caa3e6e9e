// Choosing pages for a query without reading their keys (sm_103a).
//
// Bounds of a page: for each kv head and dimension the least and the largest value of its
// keys, exact in the cache's type.  For the query rows r of a head's group
//   sum_r q_r . k <= sum_d a_d hi_d + b_d lo_d,  a_d = sum_r max(q_rd, 0), b_d = sum_r min(q_rd, 0)
// for every key k of the page: one pass over 4 D bytes for a page of 512 D, whatever the
// group's size.  A selection is whole numbers and has one right answer, so the score is
// fully specified: products and sums rounded to float32 one by one, sums pairwise,
// neighbours first.
//
// Bounds: one CTA per (page, kv head), a thread keeps eight dimensions of every 16th (or
// 32nd) key.  Selection: a cluster of up to eight CTAs per (token, kv head) scores the pages, D / 8
// lanes to a page, and leaves the keys of the order in its first CTA's shared memory,
// which finds the n-th largest by its bytes (four histograms) and writes the indices in
// rising order.
//
// Measured (GB300): bounds of 16 sessions' last pages and the selection of 64 pages of their
// 128 to 512 for 8 kv heads of 128: 14 us for 27 MB (4 us at the copy rate).  Latency bounds both: a
// launch each, then loads, sums over lanes, a cluster's barrier and four histograms, one
// behind the other.  (Clusters of eight, page numbers of 32 bits and unrolled sums: 24 us.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "attention_shared.cuh"
#include "dsb_kernels.h"
#include "dsb_ptx.cuh"

namespace dsbk {

namespace {

constexpr int kBoundThreads = 256;
constexpr int kSelThreads = 256;
constexpr int kPageKeys = 128;
// Largest list of scores: a slot of metadata holds 11281 words, two page numbers to one.
constexpr int kMostOrder = 96 * 1024;

template <typename T>
struct Two;
template <>
struct Two<__half> {
  using type = __half2;
  static __device__ __forceinline__ float2 f(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
};
template <>
struct Two<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ float2 f(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
};
// The lesser / the larger of each half; a NaN makes the result NaN.
template <typename T>
__device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
  using V = typename Two<T>::type;
  const V r = __hmin2_nan(*reinterpret_cast<const V*>(&a), *reinterpret_cast<const V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
  using V = typename Two<T>::type;
  const V r = __hmax2_nan(*reinterpret_cast<const V*>(&a), *reinterpret_cast<const V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D, typename T, int N>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const uint4* __restrict__ k, int hkv,
                                                                    uint4* __restrict__ bounds,
                                                                    const __grid_constant__ ParamWords<N> words) {
  constexpr int L = D / 8, ROWS = kBoundThreads / L;  // pieces of a row; rows at a time
  __shared__ uint4 part[2][ROWS][L];
  pdl_wait();
  pdl_trigger();
  const int page = words.w[2 * blockIdx.y], keys = words.w[2 * blockIdx.y + 1];
  const size_t head = (size_t)page * hkv + blockIdx.x;
  const int row = threadIdx.x / L, piece = threadIdx.x % L;
  const uint4* src = k + head * kPageKeys * L + piece;
  // rows past the last repeat row 0, which every page has
  uint4 v[kPageKeys / ROWS];
#pragma unroll
  for (int i = 0; i < kPageKeys / ROWS; ++i) {
    const int r = row + i * ROWS;
    v[i] = __ldg(src + (size_t)(r < keys ? r : 0) * L);
  }
  uint4 lo = v[0], hi = v[0];
#pragma unroll
  for (int i = 1; i < kPageKeys / ROWS; ++i) {
    lo = make_uint4(least<T>(lo.x, v[i].x), least<T>(lo.y, v[i].y), least<T>(lo.z, v[i].z), least<T>(lo.w, v[i].w));
    hi = make_uint4(most<T>(hi.x, v[i].x), most<T>(hi.y, v[i].y), most<T>(hi.z, v[i].z), most<T>(hi.w, v[i].w));
  }
  part[0][row][piece] = lo;
  part[1][row][piece] = hi;
  __syncthreads();
  // a word of eight bytes' dimensions for each of the first 2 D / 2 threads
  if (threadIdx.x < D) {
    const int which = threadIdx.x / (D / 2), word = threadIdx.x % (D / 2);
    const uint32_t* col = reinterpret_cast<const uint32_t*>(&part[which][0][0]) + word;
    uint32_t x = col[0];
#pragma unroll
    for (int r = 1; r < ROWS; ++r) x = which ? most<T>(x, col[r * (D / 2)]) : least<T>(x, col[r * (D / 2)]);
    reinterpret_cast<uint32_t*>(bounds)[head * D + threadIdx.x] = x;
  }
}

// Whole numbers in the order of the scores: NaN above all of them, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xFFFFFFFEu;
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
  return u ^ ((int32_t)u < 0 ? 0xFFFFFFFFu : 0x80000000u);
}
constexpr uint32_t kAlways = 0xFFFFFFFFu;

// Pairwise sum, neighbours first, of values that come eight at a time, as if zeros
// followed up to a power of two.
struct Pairwise {
  float held[14];  // sums of 8, 16, .. values that wait for their neighbours
  int n = 0;       // eights so far
  __device__ __forceinline__ void add(const float (&v)[8]) {
    float x = __fadd_rn(__fadd_rn(__fadd_rn(v[0], v[1]), __fadd_rn(v[2], v[3])),
                        __fadd_rn(__fadd_rn(v[4], v[5]), __fadd_rn(v[6], v[7])));
    int level = 0;
#pragma unroll 1
    for (; n >> level & 1; ++level) x = __fadd_rn(held[level], x);
    held[level] = x;
    ++n;
  }
  __device__ __forceinline__ float sum() const {
    float x = 0.0f;
#pragma unroll 1
    for (int level = 0; n >> level; ++level)
      if (n >> level & 1) x = __fadd_rn(held[level], x);
    return x;
  }
};

template <int D, typename T, int N>
__global__ void __launch_bounds__(kSelThreads, 4) select_pages_kernel(
    const float* __restrict__ q, long long q_stride, int hq, int hkv, const uint4* __restrict__ bounds, int n_seq,
    int n_select, int keep_first, int keep_last, int32_t* __restrict__ selected, bool wide,
    const __grid_constant__ ParamWords<N> words, const int32_t* __restrict__ meta_dev) {
  constexpr int L = D / 8;                // lanes to a page
  constexpr int AT = kSelThreads / L;     // pages at a time
  constexpr int U = 4;                    // and as many again on their way
  constexpr int W = kSelThreads / 32;
  extern __shared__ uint32_t order[];     // [pages], of the cluster's first CTA
  __shared__ float ab[2][D];
  __shared__ int hist[256];
  __shared__ int found[2];
  __shared__ int counts[2][W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_ctarank(), ranks = gridDim.x;
  const int h = blockIdx.y, t = blockIdx.z;
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  pdl_wait();
  pdl_trigger();
  int s = 0;
  {
    int hi = n_seq - 1;
    while (s < hi) {
      const int mid = (s + hi + 1) >> 1;
      if (meta[mid * kSelSeqWords] <= t)
        s = mid;
      else
        hi = mid - 1;
    }
  }
  const int32_t* rec = meta + s * kSelSeqWords;
  const int mine = (rec[2] - rec[1] + (t - rec[0])) / kPageKeys;  // the token's own page
  const int n = mine + 1;                                         // pages that it sees
  const int32_t* pages = meta + rec[3];
  const auto page_of = [&](int j) { return wide ? pages[j] : (int)reinterpret_cast<const uint16_t*>(pages)[j]; };
  int32_t* out = selected + ((size_t)t * hkv + h) * n_select;
  if (n <= n_select) {  // the same in every CTA of the cluster
    if (rank == 0)
      for (int i = tid; i < n_select; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  if (ranks > 1) cluster_sync();  // the first CTA's memory is written from the others
  // ---- the group's rows as two
  const int G = hq / hkv;
  if (tid < D) {
    const float* row = q + (size_t)t * q_stride + (size_t)h * G * D + tid;
    Pairwise a, b;
#pragma unroll 1
    for (int r0 = 0; r0 < G; r0 += 8) {
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = r0 + i < G ? __ldg(row + (size_t)(r0 + i) * D) : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // a NaN stays one in both
        y[i] = x[i] > 0.0f ? 0.0f : x[i];
        x[i] = x[i] < 0.0f ? 0.0f : x[i];
      }
      a.add(x);
      b.add(y);
    }
    ab[0][tid] = a.sum();
    ab[1][tid] = b.sum();
  }
  __syncthreads();
  const int part = tid % L;
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = ab[0][8 * part + i];
    b[i] = ab[1][8 * part + i];
  }
  // ---- scores: D / 8 lanes to a page; a CTA takes every ranks-th group of pages
  const uint32_t first_cta = cluster_map(order, 0);
  for (int j0 = rank * AT * U; j0 < n; j0 += ranks * AT * U) {
    uint4 lo[U], hi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * AT + tid / L;
      if (j < n) {
        const uint4* src = bounds + ((size_t)page_of(j) * hkv + h) * 2 * L + part;
        lo[u] = __ldg(src);
        hi[u] = __ldg(src + L);
      } else {
        lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t lw[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w}, hw[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w};
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 l = Two<T>::f(lw[i]), x = Two<T>::f(hw[i]);
        const float t0 = __fadd_rn(__fmul_rn(a[2 * i], x.x), __fmul_rn(b[2 * i], l.x));
        const float t1 = __fadd_rn(__fmul_rn(a[2 * i + 1], x.y), __fmul_rn(b[2 * i + 1], l.y));
        p[i] = __fadd_rn(t0, t1);
      }
      float sc = __fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3]));
#pragma unroll
      for (int o = 1; o < L; o <<= 1) sc = __fadd_rn(sc, __shfl_xor_sync(0xFFFFFFFFu, sc, o));
      const int j = j0 + u * AT + tid / L;
      if (part == 0 && j < n) {
        const uint32_t key = j < keep_first || j > mine - keep_last ? kAlways : order_of(sc);
        if (ranks == 1)
          order[j] = key;
        else
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(first_cta + 4u * j), "r"(key) : "memory");
      }
    }
  }
  if (ranks > 1) {
    cluster_sync();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  // ---- the n_select-th largest, eight bits at a time
  uint32_t prefix = 0;
  int need = n_select;
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int j = tid; j < n; j += kSelThreads) {
      const uint32_t key = order[j];
      if ((key & mask) == prefix) atomicAdd(&hist[key >> shift & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane i holds the bins 255 - 8 i .. 248 - 8 i
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += x;
      }
      before -= sum;
      if (before < need && need <= before + sum) {
        int i = 0;
        while (before + c[i] < need) before += c[i++];
        found[0] = 255 - 8 * lane - i;
        found[1] = need - before;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    need = found[1];
  }
  // ---- those above it, and the first `need` of those equal to it, in rising order: each
  // warp a run of indices
  const int run = (n + W - 1) / W, j_end = min(n, (warp + 1) * run);
  int above = 0, equal = 0;
  for (int j = warp * run + lane; j - lane < j_end; j += 32) {
    const bool in = j < j_end;
    above += __popc(__ballot_sync(0xFFFFFFFFu, in && order[j] > prefix));
    equal += __popc(__ballot_sync(0xFFFFFFFFu, in && order[j] == prefix));
  }
  if (lane == 0) {
    counts[0][warp] = above;
    counts[1][warp] = equal;
  }
  __syncthreads();
  above = equal = 0;
  for (int w = 0; w < warp; ++w) {
    above += counts[0][w];
    equal += counts[1][w];
  }
  for (int j = warp * run + lane; j - lane < j_end; j += 32) {
    const bool in = j < j_end;
    const bool gt = in && order[j] > prefix, eq = in && order[j] == prefix;
    const unsigned gts = __ballot_sync(0xFFFFFFFFu, gt), eqs = __ballot_sync(0xFFFFFFFFu, eq);
    const unsigned below = (1u << lane) - 1u;
    const int g0 = above + __popc(gts & below), e0 = equal + __popc(eqs & below);
    if (gt || (eq && e0 < need)) out[g0 + min(e0, need)] = j;
    above += __popc(gts);
    equal += __popc(eqs);
  }
}

template <int D, typename T>
cudaError_t select_go(const SelectArgs& a, const MetaArg& meta, cudaStream_t st) {
  return with_words(meta, [&](auto n) {
    constexpr int N = decltype(n)::value;
    ParamWords<N> w;
    fill_words(meta, &w);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.ranks, (unsigned)a.hkv, (unsigned)a.n_tok);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)a.max_pages * 4;
    if (cfg.dynamicSmemBytes > 40 * 1024) {  // past what a launch has without asking (beside 2 KB of static)
      // the same whatever the call needs, so that calls of two threads do not take it from each other
      static std::atomic<unsigned long long> ready{0};
      const cudaError_t e = allow_smem(select_pages_kernel<D, T, N>, kMostOrder, &ready);
      if (e != cudaSuccess) return e;
    }
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_pages_kernel<D, T, N>, a.q, a.q_stride, a.hq, a.hkv,
                              static_cast<const uint4*>(a.bounds), a.n_seq, a.n_select, a.keep_first, a.keep_last,
                              a.selected, a.wide_pages, w, meta.dev);
  });
}

template <int D, typename T>
cudaError_t bounds_go(const void* k, int hkv, int pages, void* bounds, const MetaArg& meta, cudaStream_t st) {
  const auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    ParamWords<N> w;
    fill_words(meta, &w);
    return launch_kernel(page_bounds_kernel<D, T, N>, dim3((unsigned)hkv, (unsigned)pages), dim3(kBoundThreads), 0, st,
                         static_cast<const uint4*>(k), hkv, static_cast<uint4*>(bounds), w);
  };
  if (meta.n_words <= kParamFew) return go(std::integral_constant<int, kParamFew>{});
  return go(std::integral_constant<int, kParamWords>{});
}

}  // namespace

cudaError_t launch_page_bounds(const void* k, int dtype, int hkv, int head_dim, int pages, void* bounds,
                               const MetaArg& meta, cudaStream_t st) {
  if (head_dim == 128)
    return dtype == 0 ? bounds_go<128, __half>(k, hkv, pages, bounds, meta, st)
                      : bounds_go<128, __nv_bfloat16>(k, hkv, pages, bounds, meta, st);
  return dtype == 0 ? bounds_go<64, __half>(k, hkv, pages, bounds, meta, st)
                    : bounds_go<64, __nv_bfloat16>(k, hkv, pages, bounds, meta, st);
}

cudaError_t launch_select_pages(const SelectArgs& a, int dtype, int head_dim, const MetaArg& meta, cudaStream_t st) {
  if (head_dim == 128)
    return dtype == 0 ? select_go<128, __half>(a, meta, st) : select_go<128, __nv_bfloat16>(a, meta, st);
  return dtype == 0 ? select_go<64, __half>(a, meta, st) : select_go<64, __nv_bfloat16>(a, meta, st);
}

}  // namespace dsbk
