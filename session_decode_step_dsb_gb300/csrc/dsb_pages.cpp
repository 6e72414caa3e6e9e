// C ABI of the calls on whole KV pages (declared in include/dsb.h): copies, bounds and
// selection, attention over pages that sequences share and over selected pages.  As in
// dsb.cpp, all arguments are checked on the host before any CUDA call.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>
#include <numeric>
#include <vector>

#include "dsb.h"
#include "dsb_host.h"
#include "dsb_kernels.h"
#include "dsb_paged_host.h"

using namespace dsbh;

namespace {
dsb_status check_pages16(const dsb_kv_pages* kv) {
  if (!kv) return fail(DSB_ERR_INVALID_ARG, "kv is NULL");
  if (!kv->k || !kv->v) return fail(DSB_ERR_INVALID_ARG, "kv->k / kv->v is NULL");
  if (!aligned16(kv->k) || !aligned16(kv->v)) return fail(DSB_ERR_INVALID_ARG, "page pools not 16-byte aligned");
  if (kv->dtype != DSB_F16 && kv->dtype != DSB_BF16) return fail(DSB_ERR_INVALID_ARG, "dtype must be DSB_F16 or DSB_BF16");
  if (kv->n_pages < 1 || kv->n_kv_heads < 1) return fail(DSB_ERR_INVALID_ARG, "n_pages / n_kv_heads < 1");
  if (kv->head_dim != 64 && kv->head_dim != 128)
    return fail(DSB_ERR_UNSUPPORTED, "head_dim=%d: these calls serve 64 and 128", kv->head_dim);
  if (kv->n_kv_heads > 65535 || (long long)kv->n_pages * kv->n_kv_heads > (INT_MAX - 128) / DSB_KV_PAGE)
    return fail(DSB_ERR_UNSUPPORTED, "a pool of %d pages x %d kv heads", kv->n_pages, kv->n_kv_heads);
  return DSB_OK;
}

size_t pool16_bytes(const dsb_kv_pages* kv) {
  return (size_t)kv->n_pages * kv->n_kv_heads * DSB_KV_PAGE * kv->head_dim * 2;
}

dsb_status check_linear(const dsb_paged_batch* b) {
  for (int s = 0; s < b->n_seq; ++s)
    if (b->window[s] != 0) return fail(DSB_ERR_UNSUPPORTED, "sequence %d: pages are selected from linear tables, not rings", s);
  return DSB_OK;
}

dsb_status check_q(const float* q, int64_t q_stride, int n_q_heads, const dsb_kv_pages* kv) {
  if (n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % kv->n_kv_heads)
    return fail(DSB_ERR_INVALID_ARG, "n_q_heads=%d is not a positive multiple of n_kv_heads=%d", n_q_heads, kv->n_kv_heads);
  if (q_stride < (int64_t)n_q_heads * kv->head_dim || q_stride % 4 || q_stride > (1LL << 40))
    return fail(DSB_ERR_INVALID_ARG, "q_stride=%lld must be a multiple of 4, at least %lld", (long long)q_stride,
                (long long)n_q_heads * kv->head_dim);
  return DSB_OK;
}

// out[n_tok][width] of an attention call, apart from what it reads.
dsb_status check_out(const float* q, int64_t q_stride, int64_t width, int n_tok, const dsb_kv_pages* kv, const float* out) {
  const size_t bytes = n_tok * width * sizeof(float);
  if (overlap(q, ((n_tok - 1) * q_stride + width) * sizeof(float), out, bytes))
    return fail(DSB_ERR_INVALID_ARG, "out overlaps the rows of q");
  for (const void* pool : {kv->k, kv->v})
    if (overlap(pool, pool16_bytes(kv), out, bytes)) return fail(DSB_ERR_INVALID_ARG, "out overlaps the page pools");
  return DSB_OK;
}

// Copies within every plane: the sources and destinations of n_copies, one launch for as
// many as the parameters hold.
dsb_status copy_common(const std::vector<void*>& planes, size_t plane_bytes, int n_pages, int n_kv_heads, int head_dim,
                       bool q4, const int32_t* src, const int32_t* dst, const int32_t* keys, int n_copies, void* stream) {
  if (n_copies < 0) return fail(DSB_ERR_INVALID_ARG, "n_copies=%d < 0", n_copies);
  if (n_copies > 0 && (!src || !dst || !keys)) return fail(DSB_ERR_INVALID_ARG, "src / dst / keys is NULL");
  std::vector<void*> sorted(planes);
  std::sort(sorted.begin(), sorted.end());
  for (size_t i = 1; i < sorted.size(); ++i)
    if (overlap(sorted[i - 1], plane_bytes, sorted[i], plane_bytes))
      return fail(DSB_ERR_INVALID_ARG, "two page pools of the call overlap");
  std::vector<int> live;
  std::vector<std::pair<int, int>> used;  // page, copy (destinations), or page, -1 (sources)
  for (int i = 0; i < n_copies; ++i) {
    if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages)
      return fail(DSB_ERR_INVALID_ARG, "copy %d: pages %d -> %d out of [0, %d)", i, src[i], dst[i], n_pages);
    if (keys[i] < 0 || keys[i] > DSB_KV_PAGE)
      return fail(DSB_ERR_INVALID_ARG, "keys[%d]=%d out of [0, %d]", i, keys[i], DSB_KV_PAGE);
    if (keys[i] == 0) continue;
    live.push_back(i);
    used.emplace_back(src[i], -1);
    used.emplace_back(dst[i], i);
  }
  std::sort(used.begin(), used.end());
  for (size_t i = 1; i < used.size(); ++i)
    if (used[i].first == used[i - 1].first && used[i].second >= 0)
      return fail(DSB_ERR_INVALID_ARG, "page %d is written by copy %d and %s", used[i].first, used[i].second,
                  used[i - 1].second < 0 ? "read by the same call" : "another one");
  const size_t head = 2 * planes.size(), room = ((size_t)dsbk::kParamWords - head) / 3;
  std::vector<int32_t> words;
  for (size_t at = 0; at < live.size(); at += room) {
    const size_t n = std::min(room, live.size() - at);
    words.clear();
    for (void* p : planes) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(p);
      words.push_back((int32_t)(uint32_t)a);
      words.push_back((int32_t)(uint32_t)((uint64_t)a >> 32));
    }
    for (size_t i = at; i < at + n; ++i) words.insert(words.end(), {src[live[i]], dst[live[i]], keys[live[i]]});
    dsbk::MetaArg meta;
    meta.host = words.data();
    meta.n_words = (int)words.size();
    const cudaError_t e = dsbk::launch_copy_pages((int)planes.size(), (int)n, n_kv_heads, head_dim, q4, meta,
                                                  static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "copy_pages launch");
  }
  return DSB_OK;
}

constexpr int kMaxPools = 512;

// Lists of page numbers take a word each, or where the pool's have 16 bits half of one.
bool wide_pages(const dsb_kv_pages* kv) { return kv->n_pages > 1 << 16; }
size_t page_words(int n, bool wide) { return wide ? (size_t)n : ((size_t)n + 1) / 2; }
template <typename Page>
void put_pages(std::vector<int32_t>* words, int n, bool wide, Page page) {
  const size_t at = words->size();
  words->resize(at + page_words(n, wide));
  if (wide) {
    for (int i = 0; i < n; ++i) (*words)[at + i] = page(i);
  } else {
    uint16_t* to = reinterpret_cast<uint16_t*>(words->data() + at);
    for (int i = 0; i < n; ++i) to[i] = (uint16_t)page(i);
  }
}

// Work of a launch, in pages, counts in 32 bits.
constexpr int kMostWork = INT_MAX / 2;

// ---- the plan of an attention over shared pages -------------------------------------

// Where a segment's metadata or work would not fit a launch, its sequences' tokens are
// divided between several, a group: beside each other in Tree::segs, of the same pages,
// sequences and slots.
struct Segment {
  int parent;     // a segment of the pages before these (any of a group), or -1
  int group;      // the first one of its group
  int m0, m1;     // the group's sequences in Tree::order
  int t0, t1;     // its own of their new tokens, counted one sequence after the other
  int members;    // sequences that it has tokens of
  int b0, n;      // first block, pages
  int rows;       // query rows on a kv head
  int tile;       // of them go through the pages together
  int slot0 = 0, cap = 0;
  std::vector<int32_t> table;  // of its tiles, where they see only some of its pages

  int tiles() const { return (rows + tile - 1) / tile; }
  static int lead_of(int tile) { return tile == 8 ? dsbk::kLead8 : dsbk::kLead128; }
  int lead() const { return lead_of(tile); }
  long long work_a_head() const { return table.empty() ? (long long)tiles() * (n + lead()) : table.back(); }
};

struct Tree {
  const dsb_paged_batch* b;
  int G, hkv;
  bool wide_numbers;       // of pages
  bool wide;               // tiles of 128 rows are taken where they cost less
  std::vector<int> order;  // sequences with new tokens; a segment's are side by side
  std::vector<Segment> segs;
  std::vector<int> end;    // last segment of a sequence's path
  bool divided = false;    // a segment does not fit a launch

  const int32_t* table(int s) const { return b->block_table + (size_t)s * b->max_blocks; }
  int pages(int s) const { return (b->seq_lens[s] - 1) / DSB_KV_PAGE + 1; }
  int first_block(int s) const {
    const int w = b->window[s];
    return w > 0 ? std::max(0, b->seq_lens[s] - b->new_tokens[s] + 1 - w) / DSB_KV_PAGE : 0;
  }
  int tokens_of(int m0, int m1) const {
    int n = 0;
    for (int m = m0; m < m1; ++m) n += b->new_tokens[order[m]];
    return n;
  }
  // What n pages cost a segment of so many rows.
  int tile_of(int rows, int n) const { return wide ? dsbk::shared_tile_rows(rows, n) : 8; }
  long long cost(int rows, int n) const { return dsbk::shared_tile_cost(rows, n, tile_of(rows, n)); }

  // Whether pages that m1 - m0 sequences have in common are worth a segment: they save the
  // sequences' own tiles, but a tile that ends there begins once more behind them, which
  // takes as long as some pages.
  bool worth(int m0, int m1, int n) const {
    if (n <= 0) return false;
    long long apart = 0;
    for (int m = m0; m < m1; ++m) apart += cost(G * b->new_tokens[order[m]], n);
    const int rows = G * tokens_of(m0, m1);
    return apart > cost(rows, n) + cost(rows, 3);
  }

  // Pages that each tile of a sequence's rows sees of its segment, where that is not all:
  // (work of the tiles before, first page) of each, and the work of all.
  void cut_tiles(Segment* g) const {
    const int s = order[g->m0], pos0 = b->seq_lens[s] - b->new_tokens[s] + g->t0, w = b->window[s];
    int sum = 0;
    bool cut = false;
    for (int r = 0; r < g->rows; r += g->tile) {
      const int lo = pos0 + r / G, hi = pos0 + (std::min(r + g->tile, g->rows) - 1) / G;
      const int from = w > 0 ? std::max(0, lo - w + 1) / DSB_KV_PAGE : 0;
      int a = std::max(from - g->b0, 0), z = std::min(hi / DSB_KV_PAGE - g->b0, g->n - 1);
      if (a > z) a = z = 0;  // none of them: one page, all hidden
      g->table.insert(g->table.end(), {sum, a});
      sum += z - a + 1 + g->lead();
      cut = cut || z - a + 1 < g->n;
    }
    g->table.push_back(sum);
    if (!cut) g->table.clear();
  }

  // Words that a launch's parameters have for a segment's sequences and its tiles' table, beside
  // its pages; and of how many tiles such a table holds.
  int room_of(int n) const { return dsbk::kParamWords - 1 - dsbk::kSharedSegWords - (int)page_words(n, wide_numbers); }
  int places_of(int n) const { return (room_of(n) - dsbk::kSharedMemWords - 1) / 2; }

  int add(int parent, int m0, int m1, int b0, int b1) {
    const int tokens = tokens_of(m0, m1);
    for (constexpr int kMost = 2048; b0 < b1; b0 += kMost) {  // pages of a segment
      Segment g{parent,       (int)segs.size(), m0, m1, 0, tokens, m1 - m0, b0, std::min(kMost, b1 - b0),
                G * tokens, tile_of(G * tokens, b1 - b0)};
      if (g.members == 1 && g.tiles() > 1 && g.tiles() <= places_of(g.n)) cut_tiles(&g);
      divided = divided || !fits(g);
      parent = g.group;
      segs.push_back(std::move(g));
    }
    return parent;
  }

  bool fits(const Segment& g) const {
    if ((long long)hkv * g.tiles() * (g.n + g.lead()) > kMostWork) return false;
    return g.members == 1 ? g.tiles() <= places_of(g.n) : g.members <= room_of(g.n) / dsbk::kSharedMemWords;
  }

  // Groups of segments for those that do not fit a launch (once all sequences have their places
  // in `order`).
  void divide() {
    std::vector<Segment> out;
    std::vector<int> to(segs.size());
    for (size_t i = 0; i < segs.size(); ++i) {
      Segment& whole = segs[i];
      if (whole.parent >= 0) whole.parent = to[whole.parent];
      whole.group = to[i] = (int)out.size();
      if (fits(whole)) {
        out.push_back(std::move(whole));
        continue;
      }
      // tokens of a segment: whose work counts, and whose tiles a table holds
      const int tokens = whole.t1, places = places_of(whole.n), most_members = room_of(whole.n) / dsbk::kSharedMemWords;
      long long most = kMostWork / ((long long)hkv * (whole.n + whole.lead())) * whole.tile / G;
      if (whole.members == 1) most = std::min(most, std::max(1LL, (long long)places * whole.tile / G));
      const int parts = (int)((tokens + most - 1) / most), share = (tokens + parts - 1) / parts;
      for (int t0 = 0, m = whole.m0, m_end = 0; t0 < tokens;) {  // m_end: of the tokens of sequences before m
        Segment g = whole;
        g.t0 = g.t1 = t0;
        g.members = 0;
        g.table.clear();
        while (g.t1 < std::min(t0 + share, tokens) && g.members < most_members) {
          while (m_end <= g.t1) m_end += b->new_tokens[order[m++]];
          g.t1 = std::min({t0 + share, tokens, m_end});
          ++g.members;
        }
        g.rows = G * (g.t1 - t0);
        // (more tiles than that are one token's, which see the same)
        if (whole.members == 1 && g.tiles() > 1 && g.tiles() <= places) cut_tiles(&g);
        t0 = g.t1;
        out.push_back(std::move(g));
      }
    }
    for (int& e : end)
      if (e >= 0) e = to[e];
    segs.swap(out);
  }

  // Segments of order[m0, m1), which have blocks 0 .. known - 1 in common and those before
  // `from` in segments already (the last of them `parent`).
  void split(int m0, int m1, int from, int known, int parent) {
    if (m1 - m0 == 1) {
      const int s = order[m0];
      end[s] = add(parent, m0, m1, std::max(from, first_block(s)), pages(s));
      return;
    }
    const int32_t* lead = table(order[m0]);
    int e = pages(order[m0]);
    for (int m = m0 + 1; m < m1; ++m) {
      const int32_t* t = table(order[m]);
      const int most = std::min(e, pages(order[m]));
      e = (int)(std::mismatch(lead + known, lead + most, t + known).first - lead);
    }
    if (worth(m0, m1, e - from)) {
      parent = add(parent, m0, m1, from, e);
      from = e;
    }
    // by the page behind the common ones; sequences that end there come first
    const auto key = [&](int s) { return pages(s) > e ? table(s)[e] : -1; };
    std::stable_sort(order.begin() + m0, order.begin() + m1, [&](int x, int y) { return key(x) < key(y); });
    for (int a = m0; a < m1;) {
      int z = a + 1;
      const int k = key(order[a]);
      while (z < m1 && key(order[z]) == k) ++z;
      if (k >= 0) {
        split(a, z, from, e, parent);
      } else {
        for (; a < z; ++a) end[order[a]] = from < e ? add(parent, a, a + 1, from, e) : parent;
      }
      a = z;
    }
  }

  // Cuts segments of several tiles of 128 rows into pieces of about a CTA's share of the
  // work: CTAs side by side then take the tiles through the same pages at the same time,
  // which come from memory once (a CTA that goes through all pages of a tile, and others at
  // other places of theirs, read 134 MB of pages three times).
  void cut_shares(int ctas) {
    long long work = 0;
    for (const Segment& g : segs)
      if (g.tile == 128) work += hkv * g.work_a_head();
    const int share = std::max(16, (int)((work + ctas - 1) / ctas));  // (shorter pieces would be mostly ends)
    std::vector<Segment> out;
    out.reserve(2 * segs.size());
    std::vector<int> last(segs.size());
    for (size_t i = 0, z; i < segs.size(); i = z) {  // a group alike
      bool cut = true;
      for (z = i; z < segs.size() && segs[z].group == (int)i; ++z)
        cut = cut && segs[z].tile == 128 && segs[z].tiles() > 1 && segs[z].table.empty();
      const int n = segs[i].n, pieces = cut ? std::max(1, (n + share / 2) / share) : 1;
      int parent = segs[i].parent >= 0 ? last[segs[i].parent] : -1;
      for (int k = 0; k < pieces; ++k) {
        const int group = (int)out.size(), from = (int)((long long)n * k / pieces), upto = (int)((long long)n * (k + 1) / pieces);
        for (size_t g = i; g < z; ++g) {
          Segment p = k + 1 < pieces ? segs[g] : std::move(segs[g]);
          p.parent = parent;
          p.group = group;
          p.b0 += from;
          p.n = upto - from;
          out.push_back(std::move(p));
        }
        parent = group;
      }
      last[i] = parent;  // (a group's first one is what others name)
    }
    for (int& e : end)
      if (e >= 0) e = last[e];
    segs.swap(out);
  }

  // SMs for the tiles of 128 rows: all, or where there are tiles of 8 rows too, as many as let
  // the two kernels end at the same time beside each other (one after the other on all SMs,
  // each with its beginning and its end: 64 samples 50 us for 46, a document's drafts 109 for
  // 103).  In units of 0.1 us: a page of a tile 1.4 and 0.7, and 2 us more for the tcgen05 kernel to
  // begin.
  int wide_sms(int sms) const {
    long long cost[2] = {0, 0};
    for (const Segment& g : segs) cost[g.tile == 128] += hkv * g.work_a_head() * (g.tile == 128 ? 14 : 7);
    if (cost[0] == 0 || cost[1] == 0) return sms;
    int best = 1;
    long long least = LLONG_MAX;
    for (int n = 1; n < sms; ++n) {
      const long long t = std::max(cost[1] / n + 20, cost[0] / (sms - n));
      if (t < least) least = t, best = n;
    }
    return best;
  }

  void build() {
    end.assign(b->n_seq, -1);
    segs.reserve(2 * b->n_seq);
    for (int pass = 0; pass < 2; ++pass)
      for (int s = 0; s < b->n_seq; ++s)
        if (b->new_tokens[s] > 0 && (b->window[s] > 0) == (pass == 1)) order.push_back(s);
    int linear = 0;
    while (linear < (int)order.size() && b->window[order[linear]] == 0) ++linear;
    if (linear > 0) {
      // sequences without a first page in common go apart at once
      const auto key = [&](int s) { return table(s)[0]; };
      std::stable_sort(order.begin(), order.begin() + linear, [&](int x, int y) { return key(x) < key(y); });
      for (int a = 0, z; a < linear; a = z) {
        for (z = a + 1; z < linear && key(order[z]) == key(order[a]);) ++z;
        split(a, z, 0, z - a > 1 ? 1 : 0, -1);
      }
    }
    for (int m = linear; m < (int)order.size(); ++m) split(m, m + 1, 0, 0, -1);
    if (divided) divide();
  }
};

// The largest number of parts that a run of n pages has, where every CTA takes at least
// `share` pages of work.
int most_parts(int n, long long share) {
  return n == 1 ? 1 : (int)std::min<long long>(n, (n - 2) / share + 2);
}

// While it lives, launches may start before the stream's kernel before them has ended
// (they wait for it themselves).
struct Overlap {
  const bool was = dsbk::pdl();
  explicit Overlap(bool on) { dsbk::set_pdl(on || was); }
  ~Overlap() { dsbk::set_pdl(was); }
};

// Segments of one launch, all of one height of tiles.
struct Launch {
  int tile;
  std::vector<int> segs;
  size_t n_words = 1;
  long long work = 0;
  int ctas = 1;
};

// A launch of a call on selected pages: sequences, or tokens of them, whose metadata it holds.
struct SelLaunch {
  std::vector<int32_t> words;
  int n_seq = 0, tok0 = 0, n_tok = 0, most = 0;
};

// most_tok: new tokens of a launch; a sequence with more of them is cut.
dsb_status selection_launches(const dsb_paged_batch* b, bool wide, int most_tok, cudaStream_t cs,
                              std::vector<SelLaunch>* out) {
  const auto pages = [&](int s) { return b->new_tokens[s] == 0 ? 0 : (b->seq_lens[s] - 1) / DSB_KV_PAGE + 1; };
  size_t all = 0;
  for (int s = 0; s < b->n_seq; ++s) all += dsbk::kSelSeqWords + page_words(pages(s), wide);
  size_t room = kMetaWords;
  if (all > (size_t)dsbk::kParamWords) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    const cudaError_t e = cudaStreamIsCapturing(cs, &cap);
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
    if (cap != cudaStreamCaptureStatusNone) room = dsbk::kParamWords;
  }
  struct Tokens {
    int s, n, len;  // sequence, new tokens, keys up to the last of them
  };
  std::vector<Tokens> mine;
  size_t have = 0;
  int tok = 0, taken = 0;
  const auto close = [&]() {
    SelLaunch l;
    l.n_seq = (int)mine.size();
    l.tok0 = tok;
    int at = l.n_seq * dsbk::kSelSeqWords;
    for (const Tokens& t : mine) {
      l.words.insert(l.words.end(), {l.n_tok, t.n, t.len, at});
      l.n_tok += t.n;
      l.most = std::max(l.most, pages(t.s));
      at += (int)page_words(pages(t.s), wide);
    }
    for (const Tokens& t : mine) put_pages(&l.words, pages(t.s), wide, [&](int i) { return page_of(b, t.s, i); });
    tok += l.n_tok;
    out->push_back(std::move(l));
    mine.clear();
    have = 0;
    taken = 0;
  };
  for (int s = 0; s < b->n_seq; ++s) {
    const size_t need = dsbk::kSelSeqWords + page_words(pages(s), wide);
    if (b->new_tokens[s] > 0 && need > room)
      return fail(DSB_ERR_UNSUPPORTED, "sequence %d: a call holds at most %zu words of metadata", s, room);
    for (int j = 0, n; j < b->new_tokens[s]; j += n) {
      if (have + need > room || taken == most_tok) close();
      n = std::min(b->new_tokens[s] - j, most_tok - taken);
      mine.push_back({s, n, b->seq_lens[s] - b->new_tokens[s] + j + n});
      have += need;
      taken += n;
    }
  }
  if (!mine.empty()) close();
  return DSB_OK;
}

}  // namespace

extern "C" {

dsb_status dsb_kv_copy_pages(const dsb_kv_pages* pools, int n_pools, const int32_t* src, const int32_t* dst,
                             const int32_t* keys, int n_copies, void* stream) {
  return guarded([&]() -> dsb_status {
    if (!pools) return fail(DSB_ERR_INVALID_ARG, "pools is NULL");
    if (n_pools < 1 || n_pools > kMaxPools) return fail(DSB_ERR_INVALID_ARG, "n_pools=%d out of [1, %d]", n_pools, kMaxPools);
    std::vector<void*> planes;
    for (int i = 0; i < n_pools; ++i) {
      const dsb_kv_pages& p = pools[i];
      const dsb_status st = check_pages16(&p);
      if (st != DSB_OK) return st;
      if (p.dtype != pools->dtype || p.n_pages != pools->n_pages || p.n_kv_heads != pools->n_kv_heads ||
          p.head_dim != pools->head_dim)
        return fail(DSB_ERR_INVALID_ARG, "pool %d differs from the first in dtype, pages, heads or head_dim", i);
      planes.push_back(p.k);
      planes.push_back(p.v);
    }
    return copy_common(planes, pool16_bytes(pools), pools->n_pages, pools->n_kv_heads, pools->head_dim, false, src, dst,
                       keys, n_copies, stream);
  });
}

dsb_status dsb_kv_copy_pages_q4(const dsb_kv_q4_pages* pools, int n_pools, const int32_t* src, const int32_t* dst,
                                const int32_t* keys, int n_copies, void* stream) {
  return guarded([&]() -> dsb_status {
    if (!pools) return fail(DSB_ERR_INVALID_ARG, "pools is NULL");
    if (n_pools < 1 || n_pools > kMaxPools) return fail(DSB_ERR_INVALID_ARG, "n_pools=%d out of [1, %d]", n_pools, kMaxPools);
    std::vector<void*> planes;
    for (int i = 0; i < n_pools; ++i) {
      const dsb_kv_q4_pages& p = pools[i];
      const dsb_status st = check_q4_pages(&p);
      if (st != DSB_OK) return st;
      if (p.n_pages != pools->n_pages || p.n_kv_heads != pools->n_kv_heads || p.head_dim != pools->head_dim)
        return fail(DSB_ERR_INVALID_ARG, "pool %d differs from the first in pages, heads or head_dim", i);
      planes.push_back(p.blocks);
    }
    return copy_common(planes, pool_bytes(pools), pools->n_pages, pools->n_kv_heads, pools->head_dim, true, src, dst,
                       keys, n_copies, stream);
  });
}

dsb_status dsb_attention_decode_shared(const float* q, int64_t q_stride, int n_q_heads, const dsb_kv_pages* kv,
                                       const dsb_paged_batch* b, float* out, dsb_workspace* ws, void* stream) {
  return guarded([&]() -> dsb_status {
    dsb_status st = check_pages16(kv);
    if (st != DSB_OK) return st;
    if ((st = check_q(q, q_stride, n_q_heads, kv)) != DSB_OK) return st;
    int n_tok = 0;
    if ((st = check_paged_batch(b, kv->n_pages, kMaxLen, &n_tok)) != DSB_OK) return st;
    if (!ws) return fail(DSB_ERR_WORKSPACE, "workspace is NULL");
    if (n_tok == 0) return DSB_OK;
    if (!q || !out) return fail(DSB_ERR_INVALID_ARG, "q / out is NULL");
    if (!aligned16(q) || !aligned16(out)) return fail(DSB_ERR_INVALID_ARG, "q / out not 16-byte aligned");
    const int hkv = kv->n_kv_heads, D = kv->head_dim;
    if ((st = check_out(q, q_stride, (int64_t)n_q_heads * D, n_tok, kv, out)) != DSB_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if ((st = check_workspace(ws)) != DSB_OK) return st;

    DeviceInfo dev;
    if ((st = device_info(&dev)) != DSB_OK) return st;
    const bool wide = wide_pages(kv);
    Tree tree{b, n_q_heads / hkv, hkv, wide, true, {}, {}, {}};
    tree.build();
    // the tcgen05 kernel's launch has to save what it takes
    long long saved = 0;
    for (const Segment& g : tree.segs)
      saved += dsbk::shared_tile_cost(g.rows, g.n, 8) - dsbk::shared_tile_cost(g.rows, g.n, g.tile);
    if (saved > 0 && saved * hkv < (long long)dsbk::kWideCost * dev.sms) {
      tree = Tree{b, n_q_heads / hkv, hkv, wide, false, {}, {}, {}};
      tree.build();
    }
    const int wide_sms = tree.wide_sms(dev.sms), sms8 = wide_sms < dev.sms ? dev.sms - wide_sms : dev.sms;
    tree.cut_shares(wide_sms);
    std::vector<int> tok0(b->n_seq);
    for (int s = 0, t = 0; s < b->n_seq; t += b->new_tokens[s], ++s) tok0[s] = t;
    const auto words_of = [&](const Segment& g) {
      return (size_t)dsbk::kSharedSegWords + (size_t)g.members * dsbk::kSharedMemWords + page_words(g.n, wide) +
             g.table.size();
    };

    // launches: what a captured call keeps has to ride in its parameters
    size_t all = 1;
    for (const Segment& g : tree.segs) all += words_of(g);
    size_t room = kMetaWords;
    if (all > (size_t)dsbk::kParamWords) {
      cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
      const cudaError_t e = cudaStreamIsCapturing(cs, &cap);
      if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
      if (cap != cudaStreamCaptureStatusNone) room = dsbk::kParamWords;
    }
    std::vector<Launch> launches;
    for (const int tile : {128, 8}) {
      bool open = false;
      for (size_t i = 0; i < tree.segs.size(); ++i) {
        const Segment& g = tree.segs[i];
        if (g.tile != tile) continue;
        const size_t n = words_of(g);
        const long long work = hkv * g.work_a_head();
        if (!open || launches.back().n_words + n > room || launches.back().work + work > kMostWork) {
          launches.emplace_back();
          launches.back().tile = tile;
          open = true;
        }
        launches.back().segs.push_back((int)i);
        launches.back().n_words += n;
        launches.back().work += work;
      }
    }
    int slots = 0;
    for (Launch& l : launches) {
      l.ctas = (int)std::min<long long>(l.tile == 8 ? dsbk::page_attn_resident(sms8) : wide_sms, l.work);
      for (int i : l.segs) tree.segs[i].cap = most_parts(tree.segs[i].n, l.work / l.ctas);
    }
    for (Segment& g : tree.segs) tree.segs[g.group].cap = std::max(tree.segs[g.group].cap, g.cap);
    for (Segment& g : tree.segs) {  // a parent comes before its children
      g.cap = tree.segs[g.group].cap;
      if (g.parent >= 0) g.slot0 = tree.segs[g.parent].slot0 + tree.segs[g.parent].cap;
      slots = std::max(slots, g.slot0 + g.cap);
    }
    const auto slots_of = [&](int s) { return tree.segs[tree.end[s]].slot0 + tree.segs[tree.end[s]].cap; };
    const size_t rows = (size_t)n_tok * n_q_heads;
    if (slots > 1 && rows * slots * (D + 2) * sizeof(float) > partial_capacity(ws))
      return fail(DSB_ERR_WORKSPACE, "attention needs %zu workspace bytes for partials, have %zu",
                  rows * slots * (D + 2) * sizeof(float), partial_capacity(ws));

    dsbk::PageAttnArgs a = {};
    a.q = q;
    a.q_stride = q_stride;
    a.hq = n_q_heads;
    a.hkv = hkv;
    a.k = kv->k;
    a.v = kv->v;
    a.pool_rows = (long long)kv->n_pages * hkv * DSB_KV_PAGE;
    a.n_tok = n_tok;
    a.acc = reinterpret_cast<float*>(partial_base(ws));
    a.stat = a.acc + rows * slots * D;
    a.out = out;
    a.slots = slots;
    a.unit = dsbk::weight_unit(*std::max_element(b->seq_lens, b->seq_lens + b->n_seq));
    a.wide_pages = wide;
    // Metadata before the launches, as many as there are places for staged ones: a copy
    // between two would keep them apart.
    std::vector<std::vector<int32_t>> metas(launches.size());
    std::vector<dsbk::MetaArg> args(launches.size());
    const auto lay_out = [&](size_t li) {
      const Launch& l = launches[li];
      std::vector<int32_t>& words = metas[li];
      words.assign(l.segs.size() * dsbk::kSharedSegWords + 1, 0);
      words.reserve(l.n_words);
      long long work = 0;
      for (size_t i = 0; i < l.segs.size(); ++i) {
        const Segment& g = tree.segs[l.segs[i]];
        int first = INT_MAX, last = 0, most = 0;
        const int mem_at = (int)words.size();
        for (int m = g.m0, row = 0, at = 0; m < g.m1; at += b->new_tokens[tree.order[m++]]) {
          const int s = tree.order[m], pos0 = b->seq_lens[s] - b->new_tokens[s], w = b->window[s];
          most = std::max(most, slots_of(s));
          const int j = std::max(g.t0 - at, 0), j_end = std::min(g.t1 - at, b->new_tokens[s]);
          if (j >= j_end) continue;  // another segment's of the group
          words.insert(words.end(), {row, tok0[s] + j, j_end - j, pos0 + j_end, w});
          row += tree.G * (j_end - j);
          first = std::min(first, w > 0 ? std::max(0, pos0 + j + 1 - w) : 0);
          last = std::max(last, pos0 + j_end - 1);
        }
        const int pg_at = (int)words.size();
        put_pages(&words, g.n, wide, [&](int p) { return page_of(b, tree.order[g.m0], g.b0 + p); });
        const int table_at = g.table.empty() ? 0 : (int)words.size();
        words.insert(words.end(), g.table.begin(), g.table.end());
        const int32_t rec[dsbk::kSharedSegWords] = {(int32_t)work, g.rows, mem_at, g.members, g.b0, g.n, pg_at,
                                                    g.slot0,       g.cap,  first,  last,        most, table_at};
        std::copy(rec, rec + dsbk::kSharedSegWords, words.begin() + i * dsbk::kSharedSegWords);
        work += hkv * g.work_a_head();
      }
      words[l.segs.size() * dsbk::kSharedSegWords] = (int32_t)work;
      return meta_arg(ws, words, cs, &args[li]);
    };
    for (size_t li = 0; li < launches.size(); ++li) {
      if (li % kSlots == 0)
        for (size_t i = li; i < std::min(li + kSlots, launches.size()); ++i)
          if ((st = lay_out(i)) != DSB_OK) return st;
      const Launch& l = launches[li];
      a.n_seg = (int)l.segs.size();
      a.ctas = l.ctas;
      a.beside = li % kSlots > 0;  // no kernel of the call reads or writes what another one writes
      const Overlap overlap(a.beside);
      const cudaError_t e = l.tile == 8 ? dsbk::launch_attention_pages(a, kv->dtype == DSB_F16 ? 0 : 1, D, args[li], cs)
                                        : dsbk::launch_attention_shared_tc(a, kv->dtype == DSB_F16 ? 0 : 1, D, args[li], cs);
      if (e != cudaSuccess) return cuda_fail(e, "attention_decode_shared launch");
    }
    // the join, where a row's sums lie in parts
    std::vector<int32_t> words;
    bool join = false;
    for (int s = 0; s < b->n_seq; ++s) {
      if (b->new_tokens[s] == 0) continue;
      const Segment& g = tree.segs[tree.end[s]];
      int alone = g.parent < 0 && g.cap == 1;  // written by its one part ..
      for (int m = g.m0; m < g.m1 && alone; ++m) alone = slots_of(tree.order[m]) == 1;  // .. which serves no longer one
      words.insert(words.end(), {tok0[s], alone ? 0 : slots_of(s)});
      join = join || !alone;
    }
    if (!join) return DSB_OK;
    static_assert(2 * DSB_MAX_SEQS <= dsbk::kParamWords, "join metadata");
    dsbk::MetaArg meta;
    meta.host = words.data();
    meta.n_words = (int)words.size();
    const Overlap overlap(true);
    const cudaError_t e = dsbk::launch_attention_join(a, (int)words.size() / 2, D, meta, cs);
    return e == cudaSuccess ? DSB_OK : cuda_fail(e, "attention_decode_shared join");
  });
}

dsb_status dsb_kv_page_bounds(const dsb_kv_pages* kv, const dsb_paged_batch* b, void* bounds, void* stream) {
  return guarded([&]() -> dsb_status {
    dsb_status st = check_pages16(kv);
    if (st != DSB_OK) return st;
    int n_tok = 0;
    if ((st = check_paged_batch(b, kv->n_pages, kMaxLen, &n_tok)) != DSB_OK) return st;
    if ((st = check_linear(b)) != DSB_OK) return st;
    if (!bounds || !aligned16(bounds)) return fail(DSB_ERR_INVALID_ARG, "bounds is NULL or not 16-byte aligned");
    const size_t bytes = (size_t)kv->n_pages * kv->n_kv_heads * 2 * kv->head_dim * 2;
    for (const void* pool : {kv->k, kv->v})
      if (overlap(pool, pool16_bytes(kv), bounds, bytes)) return fail(DSB_ERR_INVALID_ARG, "bounds overlaps the page pools");
    std::vector<int32_t> words;
    std::vector<int> touched;
    for (int s = 0; s < b->n_seq; ++s) {
      const int len = b->seq_lens[s], n = b->new_tokens[s];
      for (int i = (len - n) / DSB_KV_PAGE; n > 0 && i * DSB_KV_PAGE < len; ++i) {
        words.insert(words.end(), {page_of(b, s, i), std::min(DSB_KV_PAGE, len - i * DSB_KV_PAGE)});
        touched.push_back(words[words.size() - 2]);
      }
    }
    std::sort(touched.begin(), touched.end());
    const auto twice = std::adjacent_find(touched.begin(), touched.end());
    if (twice != touched.end()) return fail(DSB_ERR_INVALID_ARG, "new tokens of the call lie twice on page %d", *twice);
    for (size_t at = 0; at < words.size(); at += dsbk::kParamWords) {
      static_assert(dsbk::kParamWords % 2 == 0, "pairs of words");
      dsbk::MetaArg meta;
      meta.host = words.data() + at;
      meta.n_words = (int)std::min<size_t>(dsbk::kParamWords, words.size() - at);
      const cudaError_t e = dsbk::launch_page_bounds(kv->k, kv->dtype == DSB_F16 ? 0 : 1, kv->n_kv_heads, kv->head_dim,
                                                     meta.n_words / 2, bounds, meta, static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return cuda_fail(e, "kv_page_bounds launch");
    }
    return DSB_OK;
  });
}

dsb_status dsb_kv_select_pages(const float* q, int64_t q_stride, int n_q_heads, const dsb_kv_pages* kv,
                               const void* bounds, const dsb_paged_batch* b, int n_select, int keep_first, int keep_last,
                               int32_t* selected, dsb_workspace* ws, void* stream) {
  return guarded([&]() -> dsb_status {
    dsb_status st = check_pages16(kv);
    if (st != DSB_OK) return st;
    if ((st = check_q(q, q_stride, n_q_heads, kv)) != DSB_OK) return st;
    int n_tok = 0;
    if ((st = check_paged_batch(b, kv->n_pages, kMaxLen, &n_tok)) != DSB_OK) return st;
    if ((st = check_linear(b)) != DSB_OK) return st;
    if (keep_first < 0 || keep_last < 1 || keep_first > n_select || keep_last > n_select - keep_first)
      return fail(DSB_ERR_INVALID_ARG, "keep_first=%d >= 0 and keep_last=%d >= 1 must fit n_select=%d", keep_first, keep_last,
                  n_select);
    if (n_select > kMaxLen / DSB_KV_PAGE) return fail(DSB_ERR_INVALID_ARG, "n_select=%d", n_select);
    if (!ws) return fail(DSB_ERR_WORKSPACE, "workspace is NULL");
    if (n_tok == 0) return DSB_OK;
    if (!q || !bounds || !selected) return fail(DSB_ERR_INVALID_ARG, "q / bounds / selected is NULL");
    if (!aligned16(q) || !aligned16(bounds) || !aligned16(selected))
      return fail(DSB_ERR_INVALID_ARG, "q / bounds / selected not 16-byte aligned");
    const int hkv = kv->n_kv_heads, D = kv->head_dim;
    const size_t out_bytes = (size_t)n_tok * hkv * n_select * sizeof(int32_t);
    if (overlap(q, ((n_tok - 1) * q_stride + (int64_t)n_q_heads * D) * sizeof(float), selected, out_bytes) ||
        overlap(bounds, (size_t)kv->n_pages * hkv * 2 * D * 2, selected, out_bytes))
      return fail(DSB_ERR_INVALID_ARG, "selected overlaps q or bounds");
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if ((st = check_workspace(ws)) != DSB_OK) return st;
    DeviceInfo dev;
    if ((st = device_info(&dev)) != DSB_OK) return st;
    std::vector<SelLaunch> launches;
    if ((st = selection_launches(b, wide_pages(kv), n_tok, cs, &launches)) != DSB_OK) return st;
    for (const SelLaunch& l : launches) {
      dsbk::MetaArg meta;
      if ((st = meta_arg(ws, l.words, cs, &meta)) != DSB_OK) return st;
      // CTAs of a cluster: while they find SMs and each has a round of pages of its own
      int ranks = 1;
      while (ranks < 8 && (long long)l.n_tok * hkv * ranks * 2 <= 4 * dev.sms && ranks * 128 < l.most) ranks *= 2;
      const dsbk::SelectArgs a{q + (size_t)l.tok0 * q_stride,
                               q_stride,
                               n_q_heads,
                               hkv,
                               bounds,
                               l.n_seq,
                               l.n_tok,
                               n_select,
                               keep_first,
                               keep_last,
                               selected + (size_t)l.tok0 * hkv * n_select,
                               ranks,
                               l.most,
                               wide_pages(kv)};
      const cudaError_t e = dsbk::launch_select_pages(a, kv->dtype == DSB_F16 ? 0 : 1, D, meta, cs);
      if (e != cudaSuccess) return cuda_fail(e, "kv_select_pages launch");
    }
    return DSB_OK;
  });
}

dsb_status dsb_attention_decode_selected(const float* q, int64_t q_stride, int n_q_heads, const dsb_kv_pages* kv,
                                         const dsb_paged_batch* b, const int32_t* selected, int n_select, float* out,
                                         dsb_workspace* ws, void* stream) {
  return guarded([&]() -> dsb_status {
    dsb_status st = check_pages16(kv);
    if (st != DSB_OK) return st;
    if ((st = check_q(q, q_stride, n_q_heads, kv)) != DSB_OK) return st;
    int n_tok = 0;
    if ((st = check_paged_batch(b, kv->n_pages, kMaxLen, &n_tok)) != DSB_OK) return st;
    if ((st = check_linear(b)) != DSB_OK) return st;
    if (n_select < 1 || n_select > kMaxLen / DSB_KV_PAGE) return fail(DSB_ERR_INVALID_ARG, "n_select=%d", n_select);
    if (!ws) return fail(DSB_ERR_WORKSPACE, "workspace is NULL");
    if (n_tok == 0) return DSB_OK;
    if (!q || !selected || !out) return fail(DSB_ERR_INVALID_ARG, "q / selected / out is NULL");
    if (!aligned16(q) || !aligned16(selected) || !aligned16(out))
      return fail(DSB_ERR_INVALID_ARG, "q / selected / out not 16-byte aligned");
    const int hkv = kv->n_kv_heads, D = kv->head_dim;
    const int64_t width = (int64_t)n_q_heads * D;
    if ((st = check_out(q, q_stride, width, n_tok, kv, out)) != DSB_OK) return st;
    if (overlap(selected, (size_t)n_tok * hkv * n_select * sizeof(int32_t), out, n_tok * width * sizeof(float)))
      return fail(DSB_ERR_INVALID_ARG, "out overlaps selected");
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if ((st = check_workspace(ws)) != DSB_OK) return st;
    DeviceInfo dev;
    if ((st = device_info(&dev)) != DSB_OK) return st;
    const int tiles = (n_q_heads / hkv + 7) / 8, resident = dsbk::page_attn_resident(dev.sms);
    // entries read of every list: of the call, however it is cut into launches
    const int longest = *std::max_element(b->seq_lens, b->seq_lens + b->n_seq);
    const int read = std::min(n_select, (longest - 1) / DSB_KV_PAGE + 1);
    const long long work_a_token = (long long)hkv * tiles * (read + dsbk::kLead8);
    if (work_a_token > kMostWork) return fail(DSB_ERR_UNSUPPORTED, "%d listed pages for %d query heads", read, n_q_heads);
    std::vector<SelLaunch> launches;
    const int most_tok = (int)std::min<long long>(n_tok, kMostWork / work_a_token);
    if ((st = selection_launches(b, wide_pages(kv), most_tok, cs, &launches)) != DSB_OK) return st;
    std::vector<dsbk::PageAttnArgs> args;
    for (const SelLaunch& l : launches) {
      dsbk::PageAttnArgs a = {};
      a.n_select = read;
      const long long work = l.n_tok * work_a_token;
      a.ctas = (int)std::min<long long>(resident, work);
      a.sel_cap = a.slots = most_parts(a.n_select, work / a.ctas);
      const size_t need = (size_t)l.n_tok * n_q_heads * a.slots * (D + 2) * sizeof(float);
      if (a.slots > 1 && need > partial_capacity(ws))
        return fail(DSB_ERR_WORKSPACE, "attention needs %zu workspace bytes for partials, have %zu", need, partial_capacity(ws));
      a.q = q + (size_t)l.tok0 * q_stride;
      a.q_stride = q_stride;
      a.hq = n_q_heads;
      a.hkv = hkv;
      a.k = kv->k;
      a.v = kv->v;
      a.pool_rows = (long long)kv->n_pages * hkv * DSB_KV_PAGE;
      a.n_seg = l.n_seq;
      a.n_tok = l.n_tok;
      a.selected = selected + (size_t)l.tok0 * hkv * n_select;
      a.sel_stride = n_select;
      a.acc = reinterpret_cast<float*>(partial_base(ws));
      a.stat = a.acc + (size_t)l.n_tok * n_q_heads * a.slots * D;
      a.out = out + (size_t)l.tok0 * width;
      a.unit = dsbk::weight_unit((long long)read * DSB_KV_PAGE);
      a.wide_pages = wide_pages(kv);
      args.push_back(a);
    }
    for (size_t i = 0; i < launches.size(); ++i) {
      const dsbk::PageAttnArgs& a = args[i];
      dsbk::MetaArg meta;
      if ((st = meta_arg(ws, launches[i].words, cs, &meta)) != DSB_OK) return st;
      cudaError_t e = dsbk::launch_attention_pages(a, kv->dtype == DSB_F16 ? 0 : 1, D, meta, cs);
      if (e != cudaSuccess) return cuda_fail(e, "attention_decode_selected launch");
      if (a.slots == 1) continue;
      const int32_t words[2] = {0, a.slots};
      dsbk::MetaArg one;
      one.host = words;
      one.n_words = 2;
      const Overlap overlap(true);
      e = dsbk::launch_attention_join(a, 1, D, one, cs);
      if (e != cudaSuccess) return cuda_fail(e, "attention_decode_selected join");
    }
    return DSB_OK;
  });
}

}  // extern "C"
