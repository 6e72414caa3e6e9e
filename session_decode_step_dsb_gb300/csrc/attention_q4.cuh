// What the two kernels of the attention over 4-bit pages share: a CTA's walk over
// its work items and the requests for the half pages they need.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dsb_kernels.h"
#include "dsb_ptx.cuh"
#include "dsb_q4.cuh"

namespace dsbk {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a V scale counts as at least in a row's reference.  Scales are fp16, 2^-24 or
// more, or 0: then the weight p_k d_k is 0 and needs no room in fp16, only a p_k (at
// most 2^14 over this) whose sums, of p_k z_k too, stay within float32.
constexpr float kLeastScale = 0x1p-60f;

// Two float32 at once.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// x0, x1 as hi + lo fp16 pairs.
__device__ __forceinline__ void split(f2 x, uint32_t& hi, uint32_t& lo) {
  const float2 v = unpack(x);
  const __half2 h = __floats2half2_rn(v.x, v.y);
  const float2 f = __half22float2(h);
  const float2 t = unpack(add2(x, pack(-f.x, -f.y)));
  const __half2 r = __floats2half2_rn(t.x, t.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}

// Where a CTA is in its list of items: one unit of one (sequence, kv head, row
// tile), and the page inside it.  Divides once, at its start; then it counts.
// Kept in shared memory by thread 0; the others read what they need of it.
struct Cursor {
  int fresh;  // another sequence, head or row tile than the item before
  int at;  // pages of work before this item
  int s, h, rt, u, units, tiles, pages, pg, pg_end;
  Q4Seq q;

  template <int ROWS>
  __device__ __forceinline__ void load(const int32_t* meta, int G) {
    const int32_t* p = meta + s * kQ4SeqWords;
    q.work_off = p[0];
    q.tok0 = p[1];
    q.n_new = p[2];
    q.len = p[3];
    q.window = p[4];
    q.chunk0 = p[5];
    q.pg_at = p[6];
    q.u_pages = p[7];
    pages = ((q.len - 1) >> 7) - q.chunk0 + 1;
    units = (pages + q.u_pages - 1) / q.u_pages;
    tiles = (G * q.n_new + ROWS - 1) / ROWS;
  }
  __device__ __forceinline__ void place() {
    pg = u * q.u_pages;
    pg_end = min(pg + q.u_pages, pages);
  }
  // The first item that starts at or after `from` pages of work; false if none.  The
  // 32 lanes of a warp call it alike: they search 32 sequences at once (a search by
  // halves waits for one word after the other).
  template <int ROWS>
  __device__ __forceinline__ bool start(const int32_t* meta, int n_seq, int hkv, int G, int from) {
    const int lane = threadIdx.x & 31;
    s = -1;
    for (int i = lane; i - lane < n_seq; i += 32) {
      const unsigned before = __ballot_sync(0xFFFFFFFFu, i < n_seq && meta[i * kQ4SeqWords] <= from);
      s += __popc(before);
      if (before != 0xFFFFFFFFu) break;
    }
    load<ROWS>(meta, G);
    const int rel = from - q.work_off;
    int x = rel / pages;
    u = (rel - x * pages + q.u_pages - 1) / q.u_pages;
    if (u == units) u = 0, ++x;
    h = x / tiles;
    rt = x - h * tiles;
    if (h == hkv) {
      if (++s == n_seq) return false;
      h = 0;
      load<ROWS>(meta, G);
    }
    place();
    at = q.work_off + (h * tiles + rt) * pages + pg;
    fresh = 1;
    return true;
  }
  // The next item (one that exists).
  template <int ROWS>
  __device__ __forceinline__ void next(const int32_t* meta, int hkv, int G) {
    at += pg_end - u * q.u_pages;
    fresh = 0;
    if (++u == units) {
      u = 0;
      fresh = 1;
      if (++rt == tiles) {
        rt = 0;
        if (++h == hkv) {
          h = 0;
          ++s;
          load<ROWS>(meta, G);
        }
      }
    }
    place();
  }
  __device__ __forceinline__ int end() const { return at + pg_end - u * q.u_pages; }  // pages before the next item
};

// One thread requests the K (which = 0) or V half of page pg of the cursor's unit,
// page `page` of the pool:
// codes and numbers up to the sequence's last key (rounded up to four keys:
// 16-byte pieces), or, where the page is full, the half in one piece.
template <int D>
__device__ __forceinline__ void request(const Cursor& c, int pg, int page, int which, const uint8_t* pool, int hkv,
                                        uint8_t* dst, uint64_t* bar) {
  using B = Q4Block<D>;
  const uint8_t* src = pool + ((size_t)page * hkv + c.h) * B::bytes + (which ? B::v : 0);
  const int keys = min(kQ4Page, (c.q.len - ((c.q.chunk0 + pg) << 7) + 3) & ~3);
  if (keys == kQ4Page) {
    mbar_arrive_expect_tx(bar, B::v);
    bulk_g2s(dst, src, B::v, bar);
  } else {
    const uint32_t codes = keys * (D / 2), nums = keys * 4;
    mbar_arrive_expect_tx(bar, codes + nums);
    bulk_g2s(dst, src, codes, bar);
    bulk_g2s(dst + B::kz, src + B::kz, nums, bar);
  }
}

}  // namespace dsbk
