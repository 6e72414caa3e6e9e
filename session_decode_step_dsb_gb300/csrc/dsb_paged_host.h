// Host-side checks and the metadata path that the calls on paged batches share.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <new>
#include <vector>

#include "dsb.h"
#include "dsb_host.h"
#include "dsb_kernels.h"

namespace dsbh {

constexpr int kMaxLen = 1 << 30;   // keys of a sequence

// Runs an entry point's body: no exception leaves the C boundary.
template <typename F>
inline dsb_status guarded(F&& body) {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return fail(DSB_ERR_INVALID_ARG, "out of host memory");
  } catch (...) {
    return fail(DSB_ERR_INVALID_ARG, "unexpected host error");
  }
}

// Whether two ranges of device memory share a byte.
inline bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// Whether n rows of `width` floats, a stride apart, and a range share a byte.
inline bool rows_touch(const float* a, int64_t stride, int64_t width, int n, const void* b, size_t bytes) {
  if (!overlap(a, ((n - 1) * stride + width) * sizeof(float), b, bytes)) return false;
  const int64_t step = stride * (int64_t)sizeof(float);
  const int64_t off = ((reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) % step + step) % step;
  return off < width * (int64_t)sizeof(float) || off + (int64_t)bytes > step;
}

inline dsb_status check_workspace(const dsb_workspace* ws) {
  if (!ws) return fail(DSB_ERR_WORKSPACE, "workspace is NULL");
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != ws->device)
    return fail(DSB_ERR_INVALID_ARG, "workspace of device %d used with device %d current", ws->device, dev);
  return DSB_OK;
}

// Whether words of metadata can reach a launch on the stream: staged words are
// overwritten by later calls, so a captured launch cannot use them.
inline dsb_status check_capture(size_t most_words, cudaStream_t st) {
  if (most_words <= (size_t)dsbk::kParamWords) return DSB_OK;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(st, &cap);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
  if (cap != cudaStreamCaptureStatusNone)
    return fail(DSB_ERR_UNSUPPORTED, "a captured call holds at most %d words of metadata (this one: %zu)",
                dsbk::kParamWords, most_words);
  return DSB_OK;
}

inline dsb_status meta_arg(dsb_workspace* ws, const std::vector<int32_t>& words, cudaStream_t st, dsbk::MetaArg* out) {
  out->n_words = (int)words.size();
  if (words.size() <= (size_t)dsbk::kParamWords) {
    out->host = words.data();
    return DSB_OK;
  }
  return stage(ws, words, st, &out->dev);
}

inline dsb_status check_q4_pages(const dsb_kv_q4_pages* kv) {
  if (!kv) return fail(DSB_ERR_INVALID_ARG, "kv is NULL");
  if (!kv->blocks || !aligned16(kv->blocks)) return fail(DSB_ERR_INVALID_ARG, "kv->blocks is NULL or not 16-byte aligned");
  if (kv->n_pages < 1 || kv->n_kv_heads < 1) return fail(DSB_ERR_INVALID_ARG, "n_pages / n_kv_heads < 1");
  if (kv->n_kv_heads > 65535 || (long long)kv->n_pages * kv->n_kv_heads > INT_MAX)
    return fail(DSB_ERR_UNSUPPORTED, "a pool of %d pages x %d kv heads", kv->n_pages, kv->n_kv_heads);
  if (kv->head_dim != 64 && kv->head_dim != 128)
    return fail(DSB_ERR_UNSUPPORTED, "head_dim=%d: 4-bit pages serve 64 and 128", kv->head_dim);
  return DSB_OK;
}

inline size_t pool_bytes(const dsb_kv_q4_pages* kv) {
  return (size_t)kv->n_pages * kv->n_kv_heads * DSB_KV_PAGE * (kv->head_dim + 8);
}

// The batch's tables against a pool of n_pages; *n_tok: its new token rows.
inline dsb_status check_paged_batch(const dsb_paged_batch* b, int n_pages, int max_len, int* n_tok) {
  if (!b) return fail(DSB_ERR_INVALID_ARG, "batch is NULL");
  if (b->n_seq < 1 || b->n_seq > DSB_MAX_SEQS) return fail(DSB_ERR_INVALID_ARG, "n_seq=%d out of [1, %d]", b->n_seq, DSB_MAX_SEQS);
  if (b->max_blocks < 1) return fail(DSB_ERR_INVALID_ARG, "max_blocks=%d < 1", b->max_blocks);
  if (!b->block_table || !b->n_blocks || !b->window || !b->new_tokens || !b->seq_lens)
    return fail(DSB_ERR_INVALID_ARG, "block_table / n_blocks / window / new_tokens / seq_lens is NULL");
  long long tokens = 0;
  for (int s = 0; s < b->n_seq; ++s) {
    const int nb = b->n_blocks[s], w = b->window[s], len = b->seq_lens[s], n = b->new_tokens[s];
    if (len < 0 || len > max_len) return fail(DSB_ERR_INVALID_ARG, "seq_lens[%d]=%d out of [0, %d]", s, len, max_len);
    if (n < 0 || n > len) return fail(DSB_ERR_INVALID_ARG, "new_tokens[%d]=%d out of [0, seq_lens=%d]", s, n, len);
    if (nb < 0 || nb > b->max_blocks) return fail(DSB_ERR_INVALID_ARG, "n_blocks[%d]=%d out of [0, %d]", s, nb, b->max_blocks);
    if (w < 0) return fail(DSB_ERR_INVALID_ARG, "window[%d]=%d < 0", s, w);
    if (w == 0 && ((long long)len + DSB_KV_PAGE - 1) / DSB_KV_PAGE > nb)
      return fail(DSB_ERR_INVALID_ARG, "sequence %d: %d blocks do not cover %d keys", s, nb, len);
    if (w > 0 && len > 0 && (nb < 1 || (long long)nb * DSB_KV_PAGE < (long long)w + n - 1))
      return fail(DSB_ERR_INVALID_ARG, "sequence %d: a ring of %d pages cannot hold window %d beside %d new tokens", s, nb, w, n);
    const int32_t* row = b->block_table + (size_t)s * b->max_blocks;
    for (int i = 0; i < nb; ++i)
      if (row[i] < 0 || row[i] >= n_pages)
        return fail(DSB_ERR_INVALID_ARG, "block_table[%d][%d]=%d out of [0, %d)", s, i, row[i], n_pages);
    tokens += n;
  }
  if (tokens > DSB_MAX_TOKENS) return fail(DSB_ERR_INVALID_ARG, "%lld new tokens exceed %d", tokens, DSB_MAX_TOKENS);
  *n_tok = (int)tokens;
  return DSB_OK;
}

// The page of sequence s's 128-key block i (counted from position 0).
inline int page_of(const dsb_paged_batch* b, int s, int i) {
  if (b->window[s] > 0) i %= b->n_blocks[s];
  return b->block_table[(size_t)s * b->max_blocks + i];
}

}  // namespace dsbh
