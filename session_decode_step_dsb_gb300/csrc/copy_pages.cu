// Rows of KV pages into other pages, in every layer's pool at once (sm_103a): a fork
// copies a session's last, partly filled page, a compaction moves whole ones.
//
// Bytes in, bytes out: bound by memory.  One CTA per (copy, plane, kv head), the heads of
// a page side by side; a plane is a pool's K or V pages, or a 4-bit pool.  A thread asks
// for all its 16-byte pieces before it stores the first, so that a CTA has up to 32 KB
// on their way.
//
// Measured (GB300), 40 layers of 8 kv heads of 128: the last pages of 16 forks, bf16, 376 MB
// read and written: 57 us, 0.98 of the copy rate; 50 whole 4-bit pages, 557 MB: 81 us, 1.0.
// A fork of three sessions in two layers: 2 us, a launch.
#include <cuda_runtime.h>

#include <cstdint>

#include "dsb_kernels.h"
#include "dsb_ptx.cuh"
#include "dsb_q4.cuh"

namespace dsbk {

namespace {

constexpr int kCopyThreads = 256;

__device__ __forceinline__ uint8_t* plane_of(const int32_t* words, int plane) {
  return reinterpret_cast<uint8_t*>((unsigned long long)(uint32_t)words[2 * plane] |
                                    (unsigned long long)(uint32_t)words[2 * plane + 1] << 32);
}

// HEAD_BYTES: of a page of one kv head, 128 keys.
template <int HEAD_BYTES, int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(int planes, int hkv,
                                                                  const __grid_constant__ ParamWords<N> words) {
  constexpr int P = HEAD_BYTES / 16 / kCopyThreads;
  pdl_wait();
  pdl_trigger();
  const int32_t* one = words.w + 2 * planes + 3 * blockIdx.y;
  uint8_t* plane = plane_of(words.w, blockIdx.z);
  const uint4* src = reinterpret_cast<const uint4*>(plane + ((size_t)one[0] * hkv + blockIdx.x) * HEAD_BYTES);
  uint4* dst = reinterpret_cast<uint4*>(plane + ((size_t)one[1] * hkv + blockIdx.x) * HEAD_BYTES);
  const int pieces = one[2] * (HEAD_BYTES / 16 / kQ4Page);
  uint4 v[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int at = threadIdx.x + i * kCopyThreads;
    if (at < pieces) v[i] = __ldcg(src + at);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int at = threadIdx.x + i * kCopyThreads;
    if (at < pieces) __stcg(dst + at, v[i]);
  }
}

// A 4-bit page's block of one head: K codes, K numbers, V codes in key pairs, V numbers.
// Only the keys that are copied are written: a piece of four keys' numbers by words, the
// codes of a pair whose second key stays by the first key's halves.
template <int D, int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_q4_kernel(int planes, int hkv,
                                                                     const __grid_constant__ ParamWords<N> words) {
  using B = Q4Block<D>;
  constexpr int PIECES = B::bytes / 16, P = (PIECES + kCopyThreads - 1) / kCopyThreads;
  pdl_wait();
  pdl_trigger();
  const int32_t* one = words.w + 2 * planes + 3 * blockIdx.y;
  uint8_t* plane = plane_of(words.w, blockIdx.z);
  const uint4* src = reinterpret_cast<const uint4*>(plane + ((size_t)one[0] * hkv + blockIdx.x) * B::bytes);
  uint4* dst = reinterpret_cast<uint4*>(plane + ((size_t)one[1] * hkv + blockIdx.x) * B::bytes);
  const int keys = one[2];
  // keys of piece `at` from its first one on, and how many a whole piece has
  const auto held = [&](int at, int& whole) {
    const bool v = at >= B::v / 16;
    const int in = v ? at - B::v / 16 : at;
    if (in >= B::kz / 16) {
      whole = 4;
      return keys - (in - B::kz / 16) * 4;
    }
    whole = v ? 2 : 1;
    return keys - (v ? in / (D / 16) * 2 : in / (D / 32));
  };
  uint4 v[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int at = threadIdx.x + i * kCopyThreads;
    int whole;
    if (at < PIECES && held(at, whole) > 0) v[i] = __ldcg(src + at);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int at = threadIdx.x + i * kCopyThreads;
    int whole;
    const int have = at < PIECES ? held(at, whole) : 0;
    if (have <= 0) continue;
    if (have >= whole) {
      __stcg(dst + at, v[i]);
    } else if (whole == 4) {
      uint32_t* to = reinterpret_cast<uint32_t*>(dst + at);
      to[0] = v[i].x;
      if (have > 1) to[1] = v[i].y;
      if (have > 2) to[2] = v[i].z;
    } else {
      uint16_t* to = reinterpret_cast<uint16_t*>(dst + at);
      to[0] = (uint16_t)v[i].x;
      to[2] = (uint16_t)v[i].y;
      to[4] = (uint16_t)v[i].z;
      to[6] = (uint16_t)v[i].w;
    }
  }
}

}  // namespace

cudaError_t launch_copy_pages(int planes, int copies, int hkv, int head_dim, bool q4, const MetaArg& meta, cudaStream_t st) {
  const dim3 grid((unsigned)hkv, (unsigned)copies, (unsigned)planes);
  const auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    ParamWords<N> w;
    fill_words(meta, &w);
    auto kern = q4 ? (head_dim == 128 ? copy_pages_q4_kernel<128, N> : copy_pages_q4_kernel<64, N>)
                   : (head_dim == 128 ? copy_pages_kernel<128 * 128 * 2, N> : copy_pages_kernel<128 * 64 * 2, N>);
    return launch_kernel(kern, grid, dim3(kCopyThreads), 0, st, planes, hkv, w);
  };
  if (meta.n_words <= kParamFew) return go(std::integral_constant<int, kParamFew>{});
  return go(std::integral_constant<int, kParamWords>{});
}

}  // namespace dsbk
