// kv_pool.cu -- the host side of the paged cache: which pages hold which sequence.  Pages
// carry reference counts, so that a fork shares its parent's pages until one of them writes
// to the last, partly filled one; the pages to copy then go to kv_copy_pages.  Host code
// only: no device access, no C++ exception crosses the entry points.
#include <algorithm>
#include <functional>
#include <mutex>
#include <new>
#include <queue>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <vector>
#include "launch.h"
#include "qgemm.h"

namespace {

struct Seq {
  std::vector<int> pages;
  int len = 0;
  bool live = false;
};

int bad(int code, const char *fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return qw::set_last_error(code, msg);
}

}  // namespace

struct kv_pool {
  std::mutex mu;
  int page = 0;
  std::vector<int> ref;                  // references of each page
  std::vector<int> heap;                 // free pages, a min-heap: the lowest is handed out first
  std::vector<Seq> seqs;
  std::vector<int> idle;                 // sequence ids that can be used again

  Seq *find(int s) {
    return s >= 0 && s < (int)seqs.size() && seqs[s].live ? &seqs[s] : nullptr;
  }
  int take() {                           // the lowest free page (the heap is not empty)
    std::pop_heap(heap.begin(), heap.end(), std::greater<int>());
    const int p = heap.back();
    heap.pop_back();
    ref[p] = 1;
    return p;
  }
  void drop(int p) {                     // heap's capacity is num_pages: no allocation
    if (--ref[p] == 0) {
      heap.push_back(p);
      std::push_heap(heap.begin(), heap.end(), std::greater<int>());
    }
  }
};

namespace {
template <typename F>
int guarded(kv_pool_t *pool, F f) {
  if (!pool) return bad(QW_ERR_INVALID_ARG, "null pool");
  try {
    std::lock_guard<std::mutex> lk(pool->mu);
    return f(*pool);
  } catch (const std::bad_alloc &) {
    return bad(QW_ERR_HOST_MEMORY, "out of host memory");
  } catch (...) {
    return bad(QW_ERR_HOST_MEMORY, "host failure");
  }
}
int no_seq(int s) { return bad(QW_ERR_INVALID_ARG, "no sequence %d", s); }

int new_seq(kv_pool &p) {                // an id with room made for it, not yet live
  if (!p.idle.empty()) return p.idle.back();
  p.seqs.emplace_back();
  p.idle.reserve(p.seqs.size());
  p.idle.push_back((int)p.seqs.size() - 1);
  return p.idle.back();
}
}  // namespace

extern "C" {

int kv_pool_create(int num_pages, int page, kv_pool_t **out) {
  if (!out) return bad(QW_ERR_INVALID_ARG, "null output");
  *out = nullptr;
  if (num_pages < 0 || page < 1 || page > (1 << 20)) return bad(QW_ERR_INVALID_ARG, "num_pages >= 0, 1 <= page <= 2^20");
  kv_pool *p = nullptr;
  try {
    p = new kv_pool;
    p->page = page;
    p->ref.assign(num_pages, 0);
    p->heap.resize(num_pages);
    for (int i = 0; i < num_pages; ++i) p->heap[i] = i;        // ascending: a min-heap
  } catch (...) {
    delete p;
    return bad(QW_ERR_HOST_MEMORY, "out of host memory");
  }
  *out = p;
  return QW_OK;
}

void kv_pool_destroy(kv_pool_t *pool) { delete pool; }

int kv_pool_add(kv_pool_t *pool, int *seq) {
  return guarded(pool, [&](kv_pool &p) {
    if (!seq) return bad(QW_ERR_INVALID_ARG, "null output");
    const int s = new_seq(p);
    p.idle.pop_back();
    p.seqs[s].live = true;
    p.seqs[s].len = 0;
    *seq = s;
    return (int)QW_OK;
  });
}

int kv_pool_extend(kv_pool_t *pool, int seq, int n_tokens, int32_t *pair, int *n_pairs) {
  return guarded(pool, [&](kv_pool &p) {
    Seq *s = p.find(seq);
    if (!s) return no_seq(seq);
    if (n_tokens < 0 || !pair || !n_pairs) return bad(QW_ERR_INVALID_ARG, "bad argument");
    *n_pairs = 0;
    if (n_tokens == 0) return (int)QW_OK;
    if (n_tokens > 0x7fffffff - p.page - s->len) return bad(QW_ERR_UNSUPPORTED_SHAPE, "length above 2^31 - 1");
    const int have = (int)s->pages.size(), want = (s->len + n_tokens + p.page - 1) / p.page;
    const bool shared = s->len % p.page != 0 && p.ref[s->pages.back()] > 1;
    if ((size_t)(want - have) + (shared ? 1 : 0) > p.heap.size())
      return bad(QW_ERR_NO_PAGES, "%d pages needed, %zu free", want - have + (shared ? 1 : 0), p.heap.size());
    s->pages.reserve(want);
    if (shared) {                        // the last page is written to: a copy of its own
      const int from = s->pages.back(), to = p.take();
      p.drop(from);
      s->pages.back() = to;
      pair[0] = from;
      pair[1] = to;
      *n_pairs = 1;
    }
    for (int i = have; i < want; ++i) s->pages.push_back(p.take());
    s->len += n_tokens;
    return (int)QW_OK;
  });
}

int kv_pool_truncate(kv_pool_t *pool, int seq, int len) {
  return guarded(pool, [&](kv_pool &p) {
    Seq *s = p.find(seq);
    if (!s) return no_seq(seq);
    if (len < 0 || len > s->len) return bad(QW_ERR_INVALID_ARG, "length %d outside 0..%d", len, s->len);
    const size_t keep = ((size_t)len + p.page - 1) / p.page;
    while (s->pages.size() > keep) {
      p.drop(s->pages.back());
      s->pages.pop_back();
    }
    s->len = len;
    return (int)QW_OK;
  });
}

int kv_pool_fork(kv_pool_t *pool, int seq, int *child) {
  return guarded(pool, [&](kv_pool &p) {
    if (!p.find(seq)) return no_seq(seq);
    if (!child) return bad(QW_ERR_INVALID_ARG, "null output");
    const int c = new_seq(p);            // may move p.seqs
    p.seqs[c].pages = p.seqs[seq].pages;
    p.seqs[c].len = p.seqs[seq].len;
    p.seqs[c].live = true;
    p.idle.pop_back();
    for (int q : p.seqs[c].pages) ++p.ref[q];
    *child = c;
    return (int)QW_OK;
  });
}

int kv_pool_free(kv_pool_t *pool, int seq) {
  return guarded(pool, [&](kv_pool &p) {
    Seq *s = p.find(seq);
    if (!s) return no_seq(seq);
    p.idle.reserve(p.seqs.size());
    for (int q : s->pages) p.drop(q);
    s->pages.clear();
    s->len = 0;
    s->live = false;
    p.idle.push_back(seq);
    return (int)QW_OK;
  });
}

int kv_pool_compact(kv_pool_t *pool, int32_t *pairs, int cap, int *n_pairs) {
  return guarded(pool, [&](kv_pool &p) {
    if (cap < 0 || !n_pairs || (cap > 0 && !pairs)) return bad(QW_ERR_INVALID_ARG, "bad argument");
    *n_pairs = 0;
    const int total = (int)p.ref.size(), live = total - (int)p.heap.size();
    std::vector<int> to(total, -1);
    std::vector<int> heap;
    heap.reserve(total);                 // keeps the capacity that drop() relies on
    int n = 0, hole = 0;
    for (int q = live; q < total && n < cap; ++q) {      // live pages past the first `live`
      if (p.ref[q] == 0) continue;
      while (p.ref[hole] != 0 || to[hole] >= 0) ++hole;  // there are as many holes below `live`
      to[q] = hole;
      pairs[2 * n] = q;
      pairs[2 * n + 1] = hole;
      ++n;
      ++hole;
    }
    for (int i = 0; i < n; ++i) {
      p.ref[pairs[2 * i + 1]] = p.ref[pairs[2 * i]];
      p.ref[pairs[2 * i]] = 0;
    }
    for (Seq &s : p.seqs)
      for (int &q : s.pages)
        if (to[q] >= 0) q = to[q];
    for (int q = 0; q < total; ++q)
      if (p.ref[q] == 0) heap.push_back(q);              // ascending: a min-heap
    p.heap.swap(heap);
    *n_pairs = n;
    return (int)QW_OK;
  });
}

int kv_pool_table(kv_pool_t *pool, const int32_t *seqs, int B, int max_pages, int32_t *table, int32_t *lens) {
  return guarded(pool, [&](kv_pool &p) {
    if (B < 0 || max_pages < 0 || (B > 0 && (!seqs || !lens || (max_pages > 0 && !table))))
      return bad(QW_ERR_INVALID_ARG, "bad argument");
    for (int b = 0; b < B; ++b) {
      const Seq *s = p.find(seqs[b]);
      if (!s) return no_seq(seqs[b]);
      if ((int)s->pages.size() > max_pages)
        return bad(QW_ERR_UNSUPPORTED_SHAPE, "sequence %d has %zu pages, the table %d", seqs[b], s->pages.size(), max_pages);
    }
    for (int b = 0; b < B; ++b) {
      const Seq &s = p.seqs[seqs[b]];
      int32_t *row = table + (size_t)b * max_pages;
      std::copy(s.pages.begin(), s.pages.end(), row);
      std::fill(row + s.pages.size(), row + max_pages, 0);
      lens[b] = s.len;
    }
    return (int)QW_OK;
  });
}

int kv_pool_pages(kv_pool_t *pool, int seq, int *len, int *pages) {
  return guarded(pool, [&](kv_pool &p) {
    const Seq *s = p.find(seq);
    if (!s) return no_seq(seq);
    if (len) *len = s->len;
    if (pages) *pages = (int)s->pages.size();
    return (int)QW_OK;
  });
}

int kv_pool_free_pages(kv_pool_t *pool) {
  return guarded(pool, [](kv_pool &p) { return (int)p.heap.size(); });
}

}  // extern "C"
