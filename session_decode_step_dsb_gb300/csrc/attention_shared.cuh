// What the kernels of the attention over shared and over selected pages have in common:
// the plan that the host lays down and a CTA's walk over it.
//
// A plan is a list of segments.  A segment is a run of pages that one or more sequences
// read: the leading pages that several have in common, or those of one alone.  Its rows
// are its sequences' query rows on a kv head, one sequence after the other (of some of
// their tokens, where all would not fit a launch); they are cut into tiles, and a (segment, kv head, tile) is a run of pages to go through.  The runs
// lie behind each other, counted in pages, with a lead before each that stands for what it
// takes to begin and to end one.  Each CTA takes an even share of all that, and of the runs
// the pages that lie in it: a run has as many parts as CTAs reach into its pages, and
// every part leaves its rows' sums in a slot of its own.  The join adds the slots of a
// row, in order.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "dsb_f32x2.cuh"
#include "dsb_kernels.h"
#include "dsb_ptx.cuh"

namespace dsbk {

// Lets a kernel have so much dynamic shared memory, once on each device.
template <typename Kern>
inline cudaError_t allow_smem(Kern kern, int bytes, std::atomic<unsigned long long>* ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (ready->load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready->fetch_or(bit);
  return e;
}

constexpr int kPgKeys = 128;
// minus the reference of a row that has seen no key: the reference lies below any score
constexpr float kNoRef = 0x1.fffffep127f;
// A row's weights are exp2(score - reference), the reference 2^kRoom (of Parts) below its largest
// score so far; a score that brings 2^kSlack more moves it.
constexpr float kSlack = 4.0f;

__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A box of a tensor map (64 columns of some keys) into shared memory; bar counts its bytes.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
// Whether a pair of 16-bit values holds an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool odd(uint32_t w) {
  constexpr uint32_t e = std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u;
  return (w & e) == e || (w & e << 16) == e << 16;
}

// A float32 pair as pairs of the 16-bit type that add up to it, largest first: two of fp16
// hold 22 bits (of values scaled into its range), two of bf16 only 16, three 24.  kMore:
// products of the warp-level kernel, which holds two parts in one.  kRoom: the largest weights
// are 2^10 in fp16, whose range that uses; values up to 2^16 then add up to 2^60 at most.  In
// bf16 they are 1 times the call's unit, by which weighted values of the type's largest
// size add up to less than that (see PageAttnArgs).
template <typename T>
struct Parts;
template <>
struct Parts<__half> {
  static constexpr int kMore = 1;
  static constexpr float kRoom = 10.0f;
  static __device__ __forceinline__ uint32_t take(float& x, float& y) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    x -= f.x;
    y -= f.y;
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Parts<__nv_bfloat16> {
  static constexpr int kMore = 2;
  static constexpr float kRoom = 0.0f;
  static __device__ __forceinline__ uint32_t take(float& x, float& y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
    // (both at once: the tcgen05 kernel's weights hold its products up; prompts 706 -> 688 us)
    const float2 left = unpack(fma2(pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)),
                                    pack(-1.0f, -1.0f), pack(x, y)));
    x = left.x;
    y = left.y;
    return w;
  }
};

// The powers of two that a query row, with m its largest value, is multiplied by before it
// is cut into parts, and its scores after.  fp16: m goes to [2^13, 2^14), and with the
// scores' factor to [2^10, 2^12): the parts keep their bits whatever q's size, and no key makes
// more than 2^35.  bf16 has float32's range, and its keys too: a row stays as it is, and its
// products are finite where float32's own are.  Only one below 2^-60, whose third parts could
// lie below the type's least value, is lifted there.
template <typename T>
__device__ __forceinline__ void row_powers(float m, float& before, float& after) {
  const int ex = (int)(__float_as_uint(m) >> 23);
  const int to = std::is_same_v<T, __half> ? 140 : 67;
  const int up = to - (std::is_same_v<T, __half> ? min(max(ex, 14), 254) : min(max(ex, 1), 67));
  before = __uint_as_float((uint32_t)(127 + up) << 23);
  after = __uint_as_float((uint32_t)(127 - up) << 23);
}

// Where sums go: statistics (-reference, sum of weights) and sums of weighted values of
// [row][slot]; out where a row has one part.  A sum of weights of -1: the row is done.
struct PartialsOut {
  float2* stat;
  float* acc;
  float* out;
  int slots;  // of a row
};

// Page e of a list: 32-bit numbers, or where the pool has no more than 2^16 pages two to
// a word.
__device__ __forceinline__ int page_at(const int32_t* list, int e, bool wide) {
  return wide ? list[e] : (int)reinterpret_cast<const uint16_t*>(list)[e];
}

// One row of a tile: its place in q, in out, and the keys that it sees.
struct RowAt {
  int tok, row, lo, hi;  // row: token * query heads + head
};

// The CTAs' shares of the work, the first `rest` of them one larger.
struct Shares {
  int share, rest;

  __device__ __forceinline__ void cut(int total, int ctas) {
    share = total / ctas;
    rest = total - share * ctas;
  }
  __device__ __forceinline__ int start(int cta) const { return cta * share + min(cta, rest); }
  __device__ __forceinline__ int cta_of(int at) const {
    const int large = rest * (share + 1);
    return at < large ? at / (share + 1) : rest + (at - large) / share;
  }
};

// Walk over the segments of a plan (all fields alike in the threads that share it).
struct SharedWalk {
  const int32_t* meta;
  int n_seg, hkv, G, rows, lead;  // rows of a tile
  bool wide;
  Shares shares;
  // the segment
  int seg, n_rows, mem_at, n_mem, chunk0, pg_at, slot0, cap, first, last;
  // the run, and this CTA's part of it
  int h, tile, at;     // at: work before the run's pages
  int page0, n_pages;  // its first page in the segment's, and how many
  int i, i_end;        // pages of the run
  int stop;            // end of this CTA's share

  // This CTA's share; returns its start.
  __device__ __forceinline__ int begin(const int32_t* m, int n, bool wide_pages, int kv_heads, int group, int tile_rows,
                                       int run_lead, int cta, int ctas) {
    meta = m;
    n_seg = n;
    wide = wide_pages;
    hkv = kv_heads;
    G = group;
    rows = tile_rows;
    lead = run_lead;
    shares.cut(m[n * kSharedSegWords], ctas);
    stop = shares.start(cta + 1);
    return shares.start(cta);
  }
  // The run that place `pos` of the work lies in, from there on.  Found anew for each run:
  // what a run needs of the plan is not carried through its pages.
  __device__ __forceinline__ void locate(int pos) {
    int lo = 0, hi = n_seg - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (meta[mid * kSharedSegWords] <= pos)
        lo = mid;
      else
        hi = mid - 1;
    }
    seg = lo;
    const int32_t* p = meta + seg * kSharedSegWords;
    n_rows = p[1];
    mem_at = p[2];
    n_mem = p[3];
    chunk0 = p[4];
    n_pages = p[5];
    pg_at = p[6];
    slot0 = p[7];
    cap = p[8];
    first = p[9];
    last = p[10];
    const int tiles_at = p[12], tiles = (n_rows + rows - 1) / rows;
    page0 = 0;
    int rel = pos - p[0];
    if (tiles_at) {  // tiles that see only some of the pages
      const int32_t* t = meta + tiles_at;
      const int per_head = t[2 * tiles];
      h = rel / per_head;
      rel -= h * per_head;
      lo = 0, hi = tiles - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t[2 * mid] <= rel)
          lo = mid;
        else
          hi = mid - 1;
      }
      tile = lo;
      rel -= t[2 * tile];
      page0 = t[2 * tile + 1];
      n_pages = t[2 * tile + 2] - t[2 * tile] - lead;
    } else {
      const int run = rel / (n_pages + lead);
      rel -= run * (n_pages + lead);
      h = run / tiles;
      tile = run - h * tiles;
    }
    at = pos - rel + lead;
    i = max(rel - lead, 0);
    i_end = min(n_pages, stop - at);
  }
  // Whether any page lies in the share; whether this CTA has a part of another run, and
  // where that begins.
  __device__ __forceinline__ bool any() const { return i < i_end; }
  __device__ __forceinline__ bool another() const { return at + n_pages + lead < stop; }
  __device__ __forceinline__ int following() const { return at + n_pages; }
  __device__ __forceinline__ int here() const { return i_end - i; }  // pages of this CTA's part
  __device__ __forceinline__ int page(int e) const { return page_at(meta + pg_at, page0 + e, wide); }
  __device__ __forceinline__ int block(int e, int) const { return chunk0 + page0 + e; }
  __device__ __forceinline__ int listed(int) const { return 0; }
  // whether keys key0 .. key0 + n - 1 can be seen by any row of the segment
  __device__ __forceinline__ bool seen(int key0, int n) const { return key0 <= last && key0 + n > first; }
  // Parts of this run before this CTA's, and in all.
  __device__ __forceinline__ int part(int cta) const { return cta - shares.cta_of(at); }
  __device__ __forceinline__ int parts() const { return shares.cta_of(at + n_pages - 1) - shares.cta_of(at) + 1; }
  __device__ __forceinline__ int slot_base() const { return slot0; }
  __device__ __forceinline__ int slot_cap() const { return cap; }
  __device__ __forceinline__ bool alone() const { return slot0 == 0 && meta[seg * kSharedSegWords + 11] == cap; }
  __device__ __forceinline__ int tile_rows() const { return min(rows, n_rows - tile * rows); }
  __device__ __forceinline__ RowAt row(int r, int hq) const {
    r += tile * rows;
    int lo = 0, hi = n_mem - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (meta[mem_at + mid * kSharedMemWords] <= r)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int32_t* m = meta + mem_at + lo * kSharedMemWords;
    const int rel = r - m[0], j = rel / G, gi = rel - j * G;
    RowAt a;
    a.tok = m[1] + j;
    a.row = a.tok * hq + h * G + gi;
    a.hi = m[3] - m[2] + j;
    a.lo = m[4] > 0 ? max(0, a.hi - m[4] + 1) : 0;
    return a;
  }
};

// Walk over the selected pages: a run is the list of a (token, kv head, tile of its group).
struct SelectedWalk {
  const int32_t* meta;
  const int32_t* sel;
  int n_seg, hkv, G, rows, lead, stride, cap, tiles;
  bool wide;
  Shares shares;
  int tok, pg_at, h, tile, at, i, i_end, stop, last;
  int n_pages;  // entries of a run

  __device__ __forceinline__ int begin(const int32_t* m, int n, bool wide_pages, const int32_t* selected, int n_select,
                                       int list_stride, int slots, int n_tok, int kv_heads, int group, int tile_rows, int run_lead,
                                       int cta, int ctas) {
    meta = m;
    wide = wide_pages;
    sel = selected;
    n_seg = n;
    hkv = kv_heads;
    G = group;
    rows = tile_rows;
    lead = run_lead;
    n_pages = n_select;
    stride = list_stride;
    cap = slots;
    tiles = (G + rows - 1) / rows;
    shares.cut(n_tok * hkv * tiles * (n_pages + lead), ctas);
    stop = shares.start(cta + 1);
    return shares.start(cta);
  }
  __device__ __forceinline__ void locate(int pos) {
    const int run = pos / (n_pages + lead), th = run / tiles, rel = pos - run * (n_pages + lead);
    tile = run - th * tiles;
    tok = th / hkv;
    h = th - tok * hkv;
    at = pos - rel + lead;
    i = max(rel - lead, 0);
    i_end = min(n_pages, stop - at);
    int lo = 0, hi = n_seg - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (meta[mid * kSelSeqWords] <= tok)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int32_t* p = meta + lo * kSelSeqWords;
    last = p[2] - p[1] + (tok - p[0]);  // the token's position
    pg_at = p[3];
  }
  __device__ __forceinline__ bool any() const { return i < i_end; }
  __device__ __forceinline__ bool another() const { return at + n_pages + lead < stop; }
  __device__ __forceinline__ int following() const { return at + n_pages; }
  // The block of entry e; one that the token does not see becomes a block behind its last.
  __device__ __forceinline__ int listed(int e) const {
    const int b = __ldg(sel + ((size_t)tok * hkv + h) * stride + e);
    return b >= 0 && b <= last / kPgKeys ? b : last / kPgKeys + 1;
  }
  __device__ __forceinline__ int page(int b) const { return page_at(meta + pg_at, b, wide); }
  __device__ __forceinline__ int block(int, int got) const { return got; }
  __device__ __forceinline__ bool seen(int key0, int) const { return key0 <= last; }
  __device__ __forceinline__ int part(int cta) const { return cta - shares.cta_of(at); }
  __device__ __forceinline__ int parts() const { return shares.cta_of(at + n_pages - 1) - shares.cta_of(at) + 1; }
  __device__ __forceinline__ int slot_base() const { return 0; }
  __device__ __forceinline__ int slot_cap() const { return cap; }
  __device__ __forceinline__ bool alone() const { return true; }
  __device__ __forceinline__ int tile_rows() const { return min(rows, G - tile * rows); }
  __device__ __forceinline__ RowAt row(int r, int hq) const {
    RowAt a;
    a.tok = tok;
    a.row = tok * hq + h * G + tile * rows + r;
    a.hi = last;
    a.lo = 0;
    return a;
  }
};

}  // namespace dsbk
