// Rows of the paged 4-bit cache as the 16-bit values they stand for (sm_103a):
// to move a session to a 16-bit cache, or for a kernel that reads one.
//
// Bound by its writes: (D + 8) bytes in, 4 D out per key and head.  One CTA per
// (page, kv head); a thread turns eight codes into one 16-byte store.  8 sequences of
// 4096 to 16384 keys of 8 heads of 128 (425 MB): 67 us, 6.3 TB/s, 0.93 of the copy
// rate; 87 us with a head's pages side by side and loads between the stores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dsb_kernels.h"
#include "dsb_ptx.cuh"
#include "dsb_q4.cuh"

namespace dsbk {

namespace {

constexpr int kGatherThreads = 256;

template <typename T>
__device__ __forceinline__ uint32_t two16(float a, float b);
template <>
__device__ __forceinline__ uint32_t two16<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t two16<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float q4_value(uint32_t w, int n, float2 dz) {
  return __fmaf_rn(dz.x, (float)((int)(w >> (4 * n) & 15u) - 8), dz.y);
}

template <typename T>
__device__ __forceinline__ uint4 eight(uint32_t w, float2 dz) {
  return make_uint4(two16<T>(q4_value(w, 0, dz), q4_value(w, 1, dz)), two16<T>(q4_value(w, 2, dz), q4_value(w, 3, dz)),
                    two16<T>(q4_value(w, 4, dz), q4_value(w, 5, dz)), two16<T>(q4_value(w, 6, dz), q4_value(w, 7, dz)));
}

template <int D, typename T, int N>
__global__ void __launch_bounds__(kGatherThreads) gather_q4_kernel(const uint8_t* __restrict__ pool, int hkv, int n_seq,
                                                                   T* __restrict__ k, T* __restrict__ v,
                                                                   const __grid_constant__ ParamWords<N> words,
                                                                   const int32_t* __restrict__ meta_dev) {
  using B = Q4Block<D>;
  pdl_wait();
  pdl_trigger();
  const int32_t* meta = N > 1 ? words.w : meta_dev;
  const int item = blockIdx.y, g = blockIdx.x, tid = threadIdx.x;
  int lo = 0, hi = n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (meta[mid * kQ4SpanWords] <= item)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int32_t* sp = meta + lo * kQ4SpanWords;
  const int first = sp[1], count = sp[2], i = item - sp[0];
  const int page = meta[sp[4] + i];
  const int key0 = ((first >> 7) + i) << 7;                 // position of the page's first key
  const int r0 = max(first - key0, 0), r1 = min(first + count - key0, kQ4Page);
  const uint8_t* blk = pool + ((size_t)page * hkv + g) * B::bytes;
  // row r of the page is output row row0 + key0 + r - first
  const size_t stride = (size_t)hkv * D;
  const long long base = (long long)sp[3] + key0 - first;
  constexpr int W = D / 8;  // words of a K row, and of a V row
  // everything is on its way before the first value is stored
  constexpr int NK = kQ4Page * W / kGatherThreads, NV = NK / 2;
  uint32_t kc[NK];
  uint2 vc[NV], vdz[NV];
  __half2 kdz[NK];
#pragma unroll
  for (int n = 0; n < NK; ++n) {
    const int e = tid + n * kGatherThreads, r = e / W;
    if (r >= r0 && r < r1) {
      kc[n] = __ldcg(reinterpret_cast<const uint32_t*>(blk) + e);
      kdz[n] = __ldg(reinterpret_cast<const __half2*>(blk + B::kz) + r);
    }
  }
#pragma unroll
  for (int n = 0; n < NV; ++n) {  // eight dimensions of a key pair
    const int e = tid + n * kGatherThreads, r = e / W * 2;
    if (r + 1 >= r0 && r < r1) {
      vc[n] = __ldcg(reinterpret_cast<const uint2*>(blk + B::v) + e);
      vdz[n] = __ldg(reinterpret_cast<const uint2*>(blk + B::vz) + (r >> 1));
    }
  }
#pragma unroll
  for (int n = 0; n < NK; ++n) {
    const int e = tid + n * kGatherThreads, r = e / W, w = e % W;
    if (r >= r0 && r < r1)
      *reinterpret_cast<uint4*>(k + (size_t)(base + r) * stride + (size_t)g * D + 8 * w) =
          eight<T>(kc[n], __half22float2(kdz[n]));
  }
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int e = tid + n * kGatherThreads, r = e / W * 2, w = e % W;
    T* dst = v + (size_t)(base + r) * stride + (size_t)g * D + 8 * w;
    if (r >= r0 && r < r1)
      *reinterpret_cast<uint4*>(dst) = eight<T>(__byte_perm(vc[n].x, vc[n].y, 0x5410),
                                                __half22float2(*reinterpret_cast<const __half2*>(&vdz[n].x)));
    if (r + 1 >= r0 && r + 1 < r1)
      *reinterpret_cast<uint4*>(dst + stride) = eight<T>(__byte_perm(vc[n].x, vc[n].y, 0x7632),
                                                         __half22float2(*reinterpret_cast<const __half2*>(&vdz[n].y)));
  }
}

template <int D, typename T>
cudaError_t gather_go(const void* pool, int hkv, int n_seq, long long pages, void* k, void* v, const MetaArg& meta,
                      cudaStream_t st) {
  // the heads of a page side by side: together they write whole rows of the output
  const dim3 grid((unsigned)hkv, (unsigned)pages);
  return with_words(meta, [&](auto n) {
    ParamWords<decltype(n)::value> w;
    fill_words(meta, &w);
    return launch_kernel(gather_q4_kernel<D, T, decltype(n)::value>, grid, dim3(kGatherThreads), 0, st,
                         static_cast<const uint8_t*>(pool), hkv, n_seq, static_cast<T*>(k),
                         static_cast<T*>(v), w, meta.dev);
  });
}

}  // namespace

cudaError_t launch_gather_q4(const void* pool, int hkv, int head_dim, int n_seq, long long pages, int dtype, void* k,
                             void* v, const MetaArg& meta, cudaStream_t st) {
  if (pages == 0) return cudaSuccess;
  if (head_dim == 128)
    return dtype == 0 ? gather_go<128, __half>(pool, hkv, n_seq, pages, k, v, meta, st)
                      : gather_go<128, __nv_bfloat16>(pool, hkv, n_seq, pages, k, v, meta, st);
  if (head_dim == 64)
    return dtype == 0 ? gather_go<64, __half>(pool, hkv, n_seq, pages, k, v, meta, st)
                      : gather_go<64, __nv_bfloat16>(pool, hkv, n_seq, pages, k, v, meta, st);
  return cudaErrorInvalidValue;
}

}  // namespace dsbk
