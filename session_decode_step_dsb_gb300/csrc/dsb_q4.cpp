// C ABI of the rotary layouts, the paged append, and the 4-bit KV cache's
// attention and read-back (declared in include/dsb.h).  As in dsb.cpp, all
// arguments are checked on the host before any CUDA call.  A call's metadata
// rides in its kernel's parameters where it fits, else it goes through the
// workspace's staging ring; tables that exceed a staging slot are cut between
// sequences into several launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "dsb.h"
#include "dsb_host.h"
#include "dsb_kernels.h"
#include "dsb_paged_host.h"

using namespace dsbh;

namespace {

constexpr int kMaxPos = 1 << 24;   // positions a rotation serves

dsb_status check_rotary(const dsb_rotary* r, int head_dim) {
  if (!r) return fail(DSB_ERR_INVALID_ARG, "rotary is NULL");
  if (check_rope(&r->rope) != DSB_OK) return DSB_ERR_INVALID_ARG;
  const int rd = r->rotary_dim == 0 ? head_dim : r->rotary_dim;
  if (rd < 2 || rd % 2 || rd > head_dim)
    return fail(DSB_ERR_INVALID_ARG, "rotary_dim=%d must be even in [2, head_dim=%d], or 0", r->rotary_dim, head_dim);
  if (r->interleaved != 0 && r->interleaved != 1) return fail(DSB_ERR_INVALID_ARG, "interleaved=%d must be 0 or 1", r->interleaved);
  if (r->scaling < DSB_ROPE_UNSCALED || r->scaling > DSB_ROPE_BANDS)
    return fail(DSB_ERR_INVALID_ARG, "scaling=%d is not a dsb_rope_scaling", r->scaling);
  if (r->scaling == DSB_ROPE_UNSCALED) return DSB_OK;
  if (r->rope.yarn_factor > 1.0f) return fail(DSB_ERR_INVALID_ARG, "scaling=%d together with yarn_factor > 1", r->scaling);
  if (!(r->scale_factor >= 1.0f) || !std::isfinite(r->scale_factor))
    return fail(DSB_ERR_INVALID_ARG, "scale_factor must be finite and >= 1");
  if (r->scaling == DSB_ROPE_NTK && rd == 2) return fail(DSB_ERR_INVALID_ARG, "DSB_ROPE_NTK needs rotary_dim > 2");
  if (r->scaling == DSB_ROPE_BANDS) {
    if (r->scale_orig_ctx < 1) return fail(DSB_ERR_INVALID_ARG, "scale_orig_ctx=%d < 1", r->scale_orig_ctx);
    if (!(r->scale_low > 0.0f) || !(r->scale_high > r->scale_low) || !std::isfinite(r->scale_high))
      return fail(DSB_ERR_INVALID_ARG, "bands must satisfy 0 < scale_low < scale_high, finite");
  }
  return DSB_OK;
}

void build_rotary(const dsb_rotary& r, int head_dim, dsbk::RotaryTable* out) {
  const int rd = r.rotary_dim == 0 ? head_dim : r.rotary_dim;
  const double s = (double)r.scale_factor;
  double theta = (double)r.rope.theta;
  if (r.scaling == DSB_ROPE_NTK) theta *= std::pow(s, (double)rd / (rd - 2));
  dsbk::RopeFreqs f;
  if (r.rope.yarn_factor > 1.0f)
    dsbk::rope_freqs(theta, rd, &f, (double)r.rope.yarn_factor, r.rope.yarn_orig_ctx, (double)r.rope.yarn_beta_fast,
                     (double)r.rope.yarn_beta_slow);
  else
    dsbk::rope_freqs(theta, rd, &f);
  for (int i = 0; i < rd / 2; ++i) {
    if (r.scaling == DSB_ROPE_LINEAR) f.f[i] /= s;
    if (r.scaling == DSB_ROPE_BANDS) {
      const double turns = r.scale_orig_ctx * f.f[i] / 6.283185307179586;
      const double keep =
          std::min(1.0, std::max(0.0, (turns - r.scale_low) / ((double)r.scale_high - r.scale_low)));
      f.f[i] = f.f[i] * keep + f.f[i] / s * (1.0 - keep);
    }
  }
  const double gain = r.rope.yarn_factor > 1.0f ? 0.1 * std::log((double)r.rope.yarn_factor) + 1.0 : 1.0;
  dsbk::rotary_table(f.f, rd, r.interleaved != 0, gain, out);
}

// The same of n rows of `width` floats each, a stride apart; rows of two strides in
// one range count as shared.
bool rows_overlap(const float* a, int64_t a_stride, int64_t a_width, const float* b, int64_t b_stride, int64_t b_width,
                  int n) {
  if (!overlap(a, ((n - 1) * a_stride + a_width) * sizeof(float), b, ((n - 1) * b_stride + b_width) * sizeof(float)))
    return false;
  if (a_stride != b_stride) return true;
  const int64_t bytes = a_stride * (int64_t)sizeof(float);
  const int64_t off = ((reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) % bytes + bytes) % bytes;
  return off < a_width * (int64_t)sizeof(float) || off + b_width * (int64_t)sizeof(float) > bytes;
}

// The page rows that the batch's new tokens go to, as one range per touched
// block: two tokens on one row would race.
dsb_status check_writes(const dsb_paged_batch* b) {
  struct Range {
    int page, lo, hi, s;
  };
  std::vector<Range> r;
  for (int s = 0; s < b->n_seq; ++s) {
    if (b->new_tokens[s] == 0) continue;
    const int p0 = b->seq_lens[s] - b->new_tokens[s], p1 = b->seq_lens[s] - 1;
    for (int i = p0 / DSB_KV_PAGE; i <= p1 / DSB_KV_PAGE; ++i)
      r.push_back(Range{page_of(b, s, i), std::max(p0 - i * DSB_KV_PAGE, 0), std::min(p1 - i * DSB_KV_PAGE, DSB_KV_PAGE - 1), s});
  }
  std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.page != y.page ? x.page < y.page : x.lo < y.lo; });
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].page == r[i - 1].page && r[i].lo <= r[i - 1].hi)
      return fail(DSB_ERR_INVALID_ARG, "two tokens of the call write row %d of page %d (sequences %d and %d)", r[i].lo,
                  r[i].page, r[i - 1].s, r[i].s);
  return DSB_OK;
}

// Sequences [s0, s1) whose metadata makes one launch.
struct Group {
  int s0, s1;
  std::vector<int32_t> words;
};

// Cuts the sequences into groups of at most kMetaWords words: fixed +
// per_seq + pages(s) each.
template <typename Pages>
dsb_status cut_groups(int n_seq, size_t fixed, size_t per_seq, Pages pages, std::vector<Group>* out) {
  size_t have = 0;
  for (int s = 0; s < n_seq; ++s) {
    const size_t need = per_seq + (size_t)pages(s);
    if (fixed + need > kMetaWords) return fail(DSB_ERR_UNSUPPORTED, "sequence %d's block table exceeds the staging slot", s);
    if (out->empty() || have + need > kMetaWords) {
      out->push_back(Group{s, s, {}});
      have = fixed;
    }
    have += need;
    out->back().s1 = s + 1;
  }
  return DSB_OK;
}

// vc: NULL where kc is the pool of both.
dsb_status append_common(float* qkv, int64_t row_stride, int n_q_heads, int n_pages, int n_kv_heads, int head_dim,
                         void* kc, void* vc, size_t pool_bytes, dsbk::KvStore store, const dsb_paged_batch* b, const dsb_rotary* rotary,
                         const float* q_norm, const float* k_norm, float eps, dsb_workspace* ws, void* stream) {
  if (n_q_heads < 0 || n_q_heads > 65535 || n_kv_heads > 65535)
    return fail(DSB_ERR_INVALID_ARG, "n_q_heads=%d / n_kv_heads=%d out of range", n_q_heads, n_kv_heads);
  int n_tok = 0;
  dsb_status st = check_paged_batch(b, n_pages, kMaxPos, &n_tok);
  if (st != DSB_OK) return st;
  if ((st = check_rotary(rotary, head_dim)) != DSB_OK) return st;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(DSB_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (q_norm && !aligned16(q_norm)) return fail(DSB_ERR_INVALID_ARG, "q_norm not 16-byte aligned");
  if (k_norm && !aligned16(k_norm)) return fail(DSB_ERR_INVALID_ARG, "k_norm not 16-byte aligned");
  const int64_t width = ((int64_t)n_q_heads + 2 * n_kv_heads) * head_dim;
  if (row_stride < width || row_stride % 4 || row_stride > (1LL << 40))
    return fail(DSB_ERR_INVALID_ARG, "row_stride=%lld must be a multiple of 4, at least %lld", (long long)row_stride,
                (long long)width);
  if (!ws) return fail(DSB_ERR_WORKSPACE, "workspace is NULL");
  if ((st = check_writes(b)) != DSB_OK) return st;
  if (n_tok == 0) return DSB_OK;
  if (!qkv || !aligned16(qkv)) return fail(DSB_ERR_INVALID_ARG, "qkv is NULL or not 16-byte aligned");
  if (vc && overlap(kc, pool_bytes, vc, pool_bytes)) return fail(DSB_ERR_INVALID_ARG, "the pools of K and V overlap");
  for (const void* pool : {kc, vc})
    if (pool && rows_touch(qkv, row_stride, width, n_tok, pool, pool_bytes))
      return fail(DSB_ERR_INVALID_ARG, "qkv and a page pool overlap");
  for (const float* w : {q_norm, k_norm})
    if (w && rows_touch(qkv, row_stride, width, n_tok, w, head_dim * sizeof(float)))
      return fail(DSB_ERR_INVALID_ARG, "qkv and the weights of a norm overlap");
  // tok_off[n + 1] | pos0[n] | pg_off[n + 1] | pages, of the sequences with new tokens.
  // A sequence of n touches at most (n - 2) / DSB_KV_PAGE + 2 pages, so that any call
  // fits a staging slot.
  static_assert(5 * (size_t)DSB_MAX_SEQS + 2 + DSB_MAX_TOKENS / DSB_KV_PAGE <= kMetaWords, "append metadata");
  std::vector<int32_t> words, pos0, pg_off, list;
  int tok = 0;
  for (int s = 0; s < b->n_seq; ++s) {
    if (b->new_tokens[s] == 0) continue;
    words.push_back(tok);
    pos0.push_back(b->seq_lens[s] - b->new_tokens[s]);
    pg_off.push_back((int32_t)list.size());
    for (int i = pos0.back() / DSB_KV_PAGE; i <= (b->seq_lens[s] - 1) / DSB_KV_PAGE; ++i) list.push_back(page_of(b, s, i));
    tok += b->new_tokens[s];
  }
  const int live = (int)pos0.size();
  words.push_back(tok);
  pg_off.push_back((int32_t)list.size());
  words.insert(words.end(), pos0.begin(), pos0.end());
  words.insert(words.end(), pg_off.begin(), pg_off.end());
  words.insert(words.end(), list.begin(), list.end());
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if ((st = check_workspace(ws)) != DSB_OK) return st;
  if ((st = check_capture(words.size(), cs)) != DSB_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != DSB_OK) return st;
  dsbk::RotaryTable rot;
  build_rotary(*rotary, head_dim, &rot);
  dsbk::MetaArg meta;
  if ((st = meta_arg(ws, words, cs, &meta)) != DSB_OK) return st;
  const dsbk::AppendArgs a{qkv, row_stride, n_q_heads, n_kv_heads, kc, vc, q_norm, k_norm, eps, live, n_tok,
                           dev.sms};
  const cudaError_t e = dsbk::launch_kv_append(a, head_dim, store, rot, meta, cs);
  return e == cudaSuccess ? DSB_OK : cuda_fail(e, "kv_append launch");
}

}  // namespace

extern "C" {

dsb_status dsb_rope_rotary(float* q, int64_t q_stride, int n_q_heads, float* k, int64_t k_stride, int n_kv_heads,
                           int head_dim, int n_tok, const int32_t* pos, const dsb_rotary* rotary, dsb_workspace* ws,
                           void* stream) {
  return guarded([&]() -> dsb_status {
    if (n_tok < 0 || n_tok > DSB_MAX_TOKENS) return fail(DSB_ERR_INVALID_ARG, "n_tok=%d out of [0, %d]", n_tok, DSB_MAX_TOKENS);
    if (head_dim < 2 || head_dim % 2 || head_dim > 1024)
      return fail(DSB_ERR_INVALID_ARG, "head_dim=%d must be even in [2, 1024]", head_dim);
    if (n_q_heads < 1 || n_q_heads > 65535 || n_kv_heads < 0 || n_kv_heads > 65535)
      return fail(DSB_ERR_INVALID_ARG, "n_q_heads=%d / n_kv_heads=%d out of range", n_q_heads, n_kv_heads);
    if ((n_kv_heads == 0) != (k == nullptr)) return fail(DSB_ERR_INVALID_ARG, "k must be NULL exactly when n_kv_heads == 0");
    if (q_stride < (int64_t)n_q_heads * head_dim || q_stride > (1LL << 40) ||
        (k && (k_stride < (int64_t)n_kv_heads * head_dim || k_stride > (1LL << 40))))
      return fail(DSB_ERR_INVALID_ARG, "q_stride=%lld / k_stride=%lld below the row's width", (long long)q_stride,
                  (long long)k_stride);
    dsb_status st = check_rotary(rotary, head_dim);
    if (st != DSB_OK) return st;
    if (!ws) return fail(DSB_ERR_WORKSPACE, "workspace is NULL");
    if (n_tok == 0) return DSB_OK;
    if (!q || !pos) return fail(DSB_ERR_INVALID_ARG, "q / pos is NULL");
    if (!aligned16(q) || (k && !aligned16(k))) return fail(DSB_ERR_INVALID_ARG, "q / k not 16-byte aligned");
    for (int t = 0; t < n_tok; ++t)
      if (pos[t] < 0 || pos[t] >= kMaxPos) return fail(DSB_ERR_INVALID_ARG, "pos[%d]=%d out of [0, 2^24)", t, pos[t]);
    if (k && rows_overlap(q, q_stride, (int64_t)n_q_heads * head_dim, k, k_stride, (int64_t)n_kv_heads * head_dim, n_tok))
      return fail(DSB_ERR_INVALID_ARG, "q and k share values: they would be rotated twice");
    if ((st = check_workspace(ws)) != DSB_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    // runs of consecutive positions (a prompt is one), or the positions themselves
    // where they are fewer words
    std::vector<int32_t> words, first;
    for (int t = 0; t < n_tok; ++t)
      if (t == 0 || pos[t] != pos[t - 1] + 1) {
        words.push_back(t);
        first.push_back(pos[t]);
      }
    int runs = (int)first.size();
    words.insert(words.end(), first.begin(), first.end());
    if (words.size() > (size_t)n_tok) {
      runs = 0;
      words.assign(pos, pos + n_tok);
    }
    if ((st = check_capture(words.size(), cs)) != DSB_OK) return st;
    dsbk::RotaryTable rot;
    build_rotary(*rotary, head_dim, &rot);
    dsbk::MetaArg meta;
    if ((st = meta_arg(ws, words, cs, &meta)) != DSB_OK) return st;
    const cudaError_t e =
        dsbk::launch_rope_rotary(q, q_stride, n_q_heads, k, k ? k_stride : 0, n_kv_heads, head_dim, n_tok, rot, runs, meta, cs);
    return e == cudaSuccess ? DSB_OK : cuda_fail(e, "rope_rotary launch");
  });
}

dsb_status dsb_kv_append_paged(float* qkv, int64_t row_stride, int n_q_heads, const dsb_kv_pages* kv,
                               const dsb_paged_batch* batch, const dsb_rotary* rotary, const float* q_norm,
                               const float* k_norm, float eps, dsb_workspace* ws, void* stream) {
  return guarded([&]() -> dsb_status {
    if (!kv) return fail(DSB_ERR_INVALID_ARG, "kv is NULL");
    if (!kv->k || !kv->v) return fail(DSB_ERR_INVALID_ARG, "kv->k / kv->v is NULL");
    if (!aligned16(kv->k) || !aligned16(kv->v)) return fail(DSB_ERR_INVALID_ARG, "page pools not 16-byte aligned");
    if (kv->dtype != DSB_F16 && kv->dtype != DSB_BF16) return fail(DSB_ERR_INVALID_ARG, "dtype must be DSB_F16 or DSB_BF16");
    if (kv->n_pages < 1 || kv->n_kv_heads < 1) return fail(DSB_ERR_INVALID_ARG, "n_pages / n_kv_heads < 1");
    if (kv->head_dim != 64 && kv->head_dim != 128)
      return fail(DSB_ERR_UNSUPPORTED, "head_dim=%d: the paged append serves 64 and 128", kv->head_dim);
    return append_common(qkv, row_stride, n_q_heads, kv->n_pages, kv->n_kv_heads, kv->head_dim, kv->k, kv->v,
                         (size_t)kv->n_pages * kv->n_kv_heads * DSB_KV_PAGE * kv->head_dim * 2, kv->dtype == DSB_F16 ? dsbk::KvStore::kF16 : dsbk::KvStore::kBF16, batch, rotary, q_norm, k_norm,
                         eps, ws, stream);
  });
}

size_t dsb_kv_q4_page_bytes(int n_kv_heads, int head_dim) {
  if (n_kv_heads < 1 || (head_dim != 64 && head_dim != 128)) return 0;
  return (size_t)n_kv_heads * DSB_KV_PAGE * (head_dim + 8);
}

dsb_status dsb_kv_append_q4(float* qkv, int64_t row_stride, int n_q_heads, const dsb_kv_q4_pages* kv,
                            const dsb_paged_batch* batch, const dsb_rotary* rotary, const float* q_norm,
                            const float* k_norm, float eps, dsb_workspace* ws, void* stream) {
  return guarded([&]() -> dsb_status {
    const dsb_status st = check_q4_pages(kv);
    if (st != DSB_OK) return st;
    return append_common(qkv, row_stride, n_q_heads, kv->n_pages, kv->n_kv_heads, kv->head_dim, kv->blocks, nullptr, pool_bytes(kv),
                         dsbk::KvStore::kQ4, batch, rotary, q_norm, k_norm, eps, ws, stream);
  });
}

dsb_status dsb_attention_decode_q4(const float* q, int64_t q_stride, int n_q_heads, const dsb_kv_q4_pages* kv,
                                   const dsb_paged_batch* b, float* out, dsb_workspace* ws, void* stream) {
  return guarded([&]() -> dsb_status {
    dsb_status st = check_q4_pages(kv);
    if (st != DSB_OK) return st;
    if (n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % kv->n_kv_heads)
      return fail(DSB_ERR_INVALID_ARG, "n_q_heads=%d is not a positive multiple of n_kv_heads=%d", n_q_heads, kv->n_kv_heads);
    int n_tok = 0;
    if ((st = check_paged_batch(b, kv->n_pages, kMaxLen, &n_tok)) != DSB_OK) return st;
    if (q_stride < (int64_t)n_q_heads * kv->head_dim || q_stride % 4 || q_stride > (1LL << 40))
      return fail(DSB_ERR_INVALID_ARG, "q_stride=%lld must be a multiple of 4, at least %lld", (long long)q_stride,
                  (long long)n_q_heads * kv->head_dim);
    if (!ws) return fail(DSB_ERR_WORKSPACE, "workspace is NULL");
    if (n_tok == 0) return DSB_OK;
    if (!q || !out) return fail(DSB_ERR_INVALID_ARG, "q / out is NULL");
    if (!aligned16(q) || !aligned16(out)) return fail(DSB_ERR_INVALID_ARG, "q / out not 16-byte aligned");
    const int G = n_q_heads / kv->n_kv_heads, D = kv->head_dim;
    auto chunk0 = [&](int s) {
      const int w = b->window[s];
      return w > 0 ? std::max(0, b->seq_lens[s] - b->new_tokens[s] + 1 - w) / DSB_KV_PAGE : 0;
    };
    auto pages = [&](int s) { return b->new_tokens[s] == 0 ? 0 : (b->seq_lens[s] - 1) / DSB_KV_PAGE - chunk0(s) + 1; };
    std::vector<Group> groups;
    if ((st = cut_groups(b->n_seq, 1, dsbk::kQ4SeqWords, pages, &groups)) != DSB_OK) return st;
    // One launch for each group and height of the row tiles: that, like the units,
    // depends on a sequence's own rows, not on its neighbours.
    struct Plan {
      std::vector<int32_t> words;
      int live = 0, max_units = 1, tok0 = 0, n_tok = 0, tile_rows = 8;
      long long items = 0, work = 0;
    };
    std::vector<Plan> plans;
    int tok0 = 0;
    size_t most = 0, need = 0;
    for (const Group& g : groups) {
      int tok1 = tok0;
      for (const int rows : {4, 8, 24}) {
        Plan p;
        std::vector<int32_t> list;
        p.tok0 = tok0;
        p.tile_rows = rows;
        auto mine = [&](int s) {
          return b->new_tokens[s] > 0 && dsbk::q4_tile_rows((long long)G * b->new_tokens[s], pages(s), D) == rows;
        };
        for (int s = g.s0; s < g.s1; ++s) p.live += mine(s);
        int tok = 0;
        for (int s = g.s0; s < g.s1; tok += b->new_tokens[s], ++s) {
          if (!mine(s)) continue;
          const int n = b->new_tokens[s], np = pages(s);
          const int tiles = (int)(((long long)G * n + rows - 1) / rows);
          const int u = dsbk::q4_unit_pages(np, kv->n_kv_heads * tiles, rows), units = (np + u - 1) / u;
          const int32_t rec[dsbk::kQ4SeqWords] = {(int32_t)p.work,
                                                  tok,
                                                  n,
                                                  b->seq_lens[s],
                                                  b->window[s],
                                                  chunk0(s),
                                                  (int32_t)((size_t)p.live * dsbk::kQ4SeqWords + 1 + list.size()),
                                                  u};
          p.words.insert(p.words.end(), rec, rec + dsbk::kQ4SeqWords);
          for (int i = 0; i < np; ++i) list.push_back(page_of(b, s, chunk0(s) + i));
          p.items += (long long)kv->n_kv_heads * tiles * units;
          p.work += (long long)kv->n_kv_heads * tiles * np;
          p.max_units = std::max(p.max_units, units);
          p.n_tok = tok + n;
          if (p.work > INT_MAX) return fail(DSB_ERR_UNSUPPORTED, "too many attention items");
        }
        tok1 = tok0 + tok;
        if (p.live == 0) continue;
        p.words.push_back((int32_t)p.work);
        p.words.insert(p.words.end(), list.begin(), list.end());
        most = std::max(most, p.words.size());
        if (p.max_units > 1) need = std::max(need, (size_t)p.n_tok * n_q_heads * p.max_units * (D + 2) * sizeof(float));
        plans.push_back(std::move(p));
      }
      tok0 = tok1;
    }
    if (need > partial_capacity(ws))
      return fail(DSB_ERR_WORKSPACE, "attention needs %zu workspace bytes for partials, have %zu", need, partial_capacity(ws));
    const int64_t width = (int64_t)n_q_heads * D;
    if (overlap(q, ((n_tok - 1) * q_stride + width) * sizeof(float), out, n_tok * width * sizeof(float)))
      return fail(DSB_ERR_INVALID_ARG, "out overlaps the rows of q");
    if (overlap(kv->blocks, pool_bytes(kv), out, n_tok * width * sizeof(float)))
      return fail(DSB_ERR_INVALID_ARG, "out overlaps the page pool");
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if ((st = check_workspace(ws)) != DSB_OK) return st;
    if ((st = check_capture(most, cs)) != DSB_OK) return st;
    for (const Plan& p : plans) {
      dsbk::MetaArg meta;
      if ((st = meta_arg(ws, p.words, cs, &meta)) != DSB_OK) return st;
      const dsbk::Q4AttnArgs a{q + (size_t)p.tok0 * q_stride,
                               q_stride,
                               n_q_heads,
                               kv->n_kv_heads,
                               kv->blocks,
                               p.live,
                               p.n_tok,
                               p.tile_rows,
                               p.items,
                               p.max_units,
                               reinterpret_cast<float*>(partial_base(ws)),
                               out + (size_t)p.tok0 * n_q_heads * D};
      const cudaError_t e = dsbk::launch_attention_q4(a, D, meta, cs);
      if (e != cudaSuccess) return cuda_fail(e, "attention_decode_q4 launch");
    }
    return DSB_OK;
  });
}

dsb_status dsb_kv_gather_q4(const dsb_kv_q4_pages* kv, const dsb_paged_batch* b, const int32_t* first,
                            const int32_t* count, int dtype, void* k_out, void* v_out, dsb_workspace* ws, void* stream) {
  return guarded([&]() -> dsb_status {
    dsb_status st = check_q4_pages(kv);
    if (st != DSB_OK) return st;
    int n_tok = 0;
    if ((st = check_paged_batch(b, kv->n_pages, kMaxLen, &n_tok)) != DSB_OK) return st;
    if (dtype != DSB_F16 && dtype != DSB_BF16) return fail(DSB_ERR_INVALID_ARG, "dtype=%d must be DSB_F16 or DSB_BF16", dtype);
    if (!first || !count) return fail(DSB_ERR_INVALID_ARG, "first / count is NULL");
    long long rows = 0;
    for (int s = 0; s < b->n_seq; ++s) {
      if (first[s] < 0 || count[s] < 0 || (long long)first[s] + count[s] > b->seq_lens[s])
        return fail(DSB_ERR_INVALID_ARG, "sequence %d: keys %d .. +%d out of its %d", s, first[s], count[s], b->seq_lens[s]);
      if (count[s] > 0 && b->window[s] > 0 &&
          first[s] < (long long)b->seq_lens[s] - (long long)b->n_blocks[s] * DSB_KV_PAGE)
        return fail(DSB_ERR_INVALID_ARG, "sequence %d: key %d is no longer in its ring of %d pages", s, first[s], b->n_blocks[s]);
      rows += count[s];
    }
    if (rows > INT_MAX) return fail(DSB_ERR_UNSUPPORTED, "%lld rows", rows);
    if (!ws) return fail(DSB_ERR_WORKSPACE, "workspace is NULL");
    if (rows == 0) return DSB_OK;
    if (!k_out || !v_out) return fail(DSB_ERR_INVALID_ARG, "k_out / v_out is NULL");
    if (!aligned16(k_out) || !aligned16(v_out)) return fail(DSB_ERR_INVALID_ARG, "k_out / v_out not 16-byte aligned");
    auto pages = [&](int s) {
      return count[s] == 0 ? 0 : (first[s] + count[s] - 1) / DSB_KV_PAGE - first[s] / DSB_KV_PAGE + 1;
    };
    std::vector<Group> groups;
    if ((st = cut_groups(b->n_seq, 1, dsbk::kQ4SpanWords, pages, &groups)) != DSB_OK) return st;
    std::vector<int> live(groups.size(), 0), total(groups.size(), 0);
    size_t most = 0;
    long long row0 = 0;
    for (size_t gi = 0; gi < groups.size(); ++gi) {
      Group& g = groups[gi];
      std::vector<int32_t> list;
      for (int s = g.s0; s < g.s1; ++s) live[gi] += count[s] > 0;
      for (int s = g.s0; s < g.s1; ++s) {
        if (count[s] == 0) continue;
        const int32_t rec[dsbk::kQ4SpanWords] = {(int32_t)list.size(), first[s], count[s], (int32_t)row0,
                                                 (int32_t)((size_t)live[gi] * dsbk::kQ4SpanWords + 1 + list.size())};
        g.words.insert(g.words.end(), rec, rec + dsbk::kQ4SpanWords);
        for (int i = 0; i < pages(s); ++i) list.push_back(page_of(b, s, first[s] / DSB_KV_PAGE + i));
        row0 += count[s];
      }
      total[gi] = (int)list.size();
      g.words.push_back((int32_t)list.size());
      g.words.insert(g.words.end(), list.begin(), list.end());
      most = std::max(most, g.words.size());
    }
    const size_t out_bytes = (size_t)rows * kv->n_kv_heads * kv->head_dim * 2;
    if (overlap(k_out, out_bytes, v_out, out_bytes)) return fail(DSB_ERR_INVALID_ARG, "k_out and v_out overlap");
    for (const void* o : {k_out, v_out})
      if (overlap(kv->blocks, pool_bytes(kv), o, out_bytes))
        return fail(DSB_ERR_INVALID_ARG, "k_out / v_out and the page pool overlap");
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if ((st = check_workspace(ws)) != DSB_OK) return st;
    if ((st = check_capture(most, cs)) != DSB_OK) return st;
    for (size_t gi = 0; gi < groups.size(); ++gi) {
      if (total[gi] == 0) continue;
      dsbk::MetaArg meta;
      if ((st = meta_arg(ws, groups[gi].words, cs, &meta)) != DSB_OK) return st;
      const cudaError_t e = dsbk::launch_gather_q4(kv->blocks, kv->n_kv_heads, kv->head_dim, live[gi], total[gi], dtype,
                                                   k_out, v_out, meta, cs);
      if (e != cudaSuccess) return cuda_fail(e, "kv_gather_q4 launch");
    }
    return DSB_OK;
  });
}

}  // extern "C"
