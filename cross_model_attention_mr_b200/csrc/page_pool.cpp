// Host-side page pool of the paged cache (MapFlow section 6, "PagedAttention"): which pages each sequence
// holds, with reference counts so that forked sequences share pages until one of them writes.
// Host code only.  Every function changes nothing when it reports an error: what can throw (host memory)
// happens before the first change.
#include <stdint.h>

#include <algorithm>
#include <functional>
#include <mutex>
#include <new>
#include <unordered_map>
#include <vector>

#include "../../include/mr.h"

namespace {

struct Seq {
  std::vector<int32_t> pages;  // -1: given up by mr_pp_slide
  int rows = 0;
  int window = 0, sinks = 0;   // of the last mr_pp_slide (window 0: none)
};

}  // namespace

struct mr_page_pool {
  int n_pages = 0, page_rows = 0;
  int64_t next_id = 0;
  std::vector<int32_t> refs;   // per page
  std::vector<int32_t> free_;  // a heap with the lowest page first, capacity n_pages
  std::unordered_map<int64_t, Seq> seqs;
  std::mutex mu;

  void put_free(int32_t page) {  // never allocates: the capacity is there from the start
    free_.push_back(page);
    std::push_heap(free_.begin(), free_.end(), std::greater<int32_t>());
  }
  int32_t take_free() {
    std::pop_heap(free_.begin(), free_.end(), std::greater<int32_t>());
    const int32_t page = free_.back();
    free_.pop_back();
    refs[page] = 1;
    return page;
  }
  void drop(int32_t page) {
    if (page >= 0 && --refs[page] == 0) put_free(page);
  }
  // whether `s` can be cut to `rows`: no page was given up that the next query (position `rows` or later, under the
  // last slide's window and sinks) sees, nor the page of the last remaining row (so a page that new rows continue in
  // is always there)
  bool can_end_at(const Seq& s, int rows) const {
    if (rows > s.rows) return false;
    if (rows == 0 || rows == s.rows) return true;
    const int last = (rows - 1) / page_rows;
    if (s.pages[last] < 0) return false;
    const int64_t first = (int64_t)rows - s.window + 1;  // of the window
    for (int i = 0; i < last; ++i)
      if (s.pages[i] < 0 && ((int64_t)(i + 1) * page_rows > first || (int64_t)i * page_rows < s.sinks)) return false;
    return true;
  }
  int pages_for(int64_t rows) const { return (int)((rows + page_rows - 1) / page_rows); }
};

// Runs f under the pool's lock.  Nothing it throws (host memory ran out) crosses the C-ABI.
template <typename R, typename F>
static R guarded(mr_page_pool* pp, R failed, F f) {
  try {
    std::lock_guard<std::mutex> lk(pp->mu);
    return f();
  } catch (...) {
    return failed;
  }
}

extern "C" {

mr_page_pool* mr_pp_create(int n_pages, int page_rows) {
  if (n_pages < 1 || page_rows < 1) return nullptr;
  mr_page_pool* pp = nullptr;
  try {
    pp = new mr_page_pool();
    pp->n_pages = n_pages;
    pp->page_rows = page_rows;
    pp->refs.assign(n_pages, 0);
    pp->free_.resize(n_pages);
    for (int i = 0; i < n_pages; ++i) pp->free_[i] = i;  // ascending: a heap already
    return pp;
  } catch (...) {
    delete pp;
    return nullptr;
  }
}

void mr_pp_destroy(mr_page_pool* pp) { delete pp; }

int64_t mr_pp_open(mr_page_pool* pp) {
  if (!pp) return -(int64_t)MR_ERR_INVALID_ARG;
  return guarded<int64_t>(pp, -(int64_t)MR_ERR_CAPACITY, [&]() -> int64_t {
    const int64_t id = pp->next_id;
    pp->seqs.emplace(id, Seq());
    ++pp->next_id;
    return id;
  });
}

int64_t mr_pp_fork(mr_page_pool* pp, int64_t seq, int rows) {
  if (!pp || rows < 0) return -(int64_t)MR_ERR_INVALID_ARG;
  return guarded<int64_t>(pp, -(int64_t)MR_ERR_CAPACITY, [&]() -> int64_t {
    auto it = pp->seqs.find(seq);
    if (it == pp->seqs.end() || !pp->can_end_at(it->second, rows)) return -(int64_t)MR_ERR_INVALID_ARG;
    Seq s;
    s.rows = rows;
    s.window = it->second.window;
    s.sinks = it->second.sinks;
    s.pages.assign(it->second.pages.begin(), it->second.pages.begin() + pp->pages_for(rows));
    const int64_t id = pp->next_id;
    Seq& kept = pp->seqs.emplace(id, std::move(s)).first->second;
    ++pp->next_id;
    for (int32_t p : kept.pages)
      if (p >= 0) ++pp->refs[p];
    return id;
  });
}

int mr_pp_extend(mr_page_pool* pp, int64_t seq, int rows, int32_t* pair) {
  if (!pp || !pair || rows < 0) return -(int)MR_ERR_INVALID_ARG;
  return guarded<int>(pp, -(int)MR_ERR_CAPACITY, [&]() -> int {
    auto it = pp->seqs.find(seq);
    if (it == pp->seqs.end()) return -(int)MR_ERR_INVALID_ARG;
    Seq& s = it->second;
    const int64_t want = (int64_t)s.rows + rows;
    if (want > INT32_MAX) return -(int)MR_ERR_INVALID_ARG;
    const int have = (int)s.pages.size(), need = pp->pages_for(want) - have;
    // the page that the new rows begin in, when it holds rows already
    const int last = rows > 0 && s.rows % pp->page_rows ? s.rows / pp->page_rows : -1;
    const bool shared = last >= 0 && pp->refs[s.pages[last]] > 1;
    if (need + (shared ? 1 : 0) > (int)pp->free_.size()) return -(int)MR_ERR_CAPACITY;
    s.pages.reserve(have + std::max(0, need));
    int n = 0;
    if (shared) {
      pair[0] = s.pages[last];
      pair[1] = pp->take_free();
      --pp->refs[pair[0]];
      s.pages[last] = pair[1];
      n = 1;
    }
    for (int i = 0; i < need; ++i) s.pages.push_back(pp->take_free());
    s.rows = (int)want;
    return n;
  });
}

mr_status mr_pp_truncate(mr_page_pool* pp, int64_t seq, int rows) {
  if (!pp || rows < 0) return MR_ERR_INVALID_ARG;
  return guarded<mr_status>(pp, MR_ERR_CAPACITY, [&]() -> mr_status {
    auto it = pp->seqs.find(seq);
    if (it == pp->seqs.end() || !pp->can_end_at(it->second, rows)) return MR_ERR_INVALID_ARG;
    Seq& s = it->second;
    const int keep = pp->pages_for(rows);
    while ((int)s.pages.size() > keep) {
      pp->drop(s.pages.back());
      s.pages.pop_back();
    }
    s.rows = rows;
    return MR_OK;
  });
}

int mr_pp_slide(mr_page_pool* pp, int64_t seq, int window, int sinks) {
  if (!pp || window < 1 || sinks < 0) return -(int)MR_ERR_INVALID_ARG;
  return guarded<int>(pp, -(int)MR_ERR_CAPACITY, [&]() -> int {
    auto it = pp->seqs.find(seq);
    if (it == pp->seqs.end()) return -(int)MR_ERR_INVALID_ARG;
    Seq& s = it->second;
    // a query at position >= rows sees rows from rows - window + 1 on, and the sinks
    const int64_t first = (int64_t)s.rows - window + 1;
    int n = 0;
    for (int i = pp->pages_for(sinks); i < (int)s.pages.size() && (int64_t)(i + 1) * pp->page_rows <= first; ++i) {
      if (s.pages[i] < 0) continue;
      pp->drop(s.pages[i]);
      s.pages[i] = -1;
      ++n;
    }
    s.window = window;
    s.sinks = sinks;
    return n;
  });
}

mr_status mr_pp_close(mr_page_pool* pp, int64_t seq) {
  if (!pp) return MR_ERR_INVALID_ARG;
  return guarded<mr_status>(pp, MR_ERR_CAPACITY, [&]() -> mr_status {
    auto it = pp->seqs.find(seq);
    if (it == pp->seqs.end()) return MR_ERR_INVALID_ARG;
    for (int32_t p : it->second.pages) pp->drop(p);
    pp->seqs.erase(it);
    return MR_OK;
  });
}

int mr_pp_compact(mr_page_pool* pp, int32_t* pairs, int max_pairs) {
  if (!pp || max_pairs < 0 || (max_pairs > 0 && !pairs)) return -(int)MR_ERR_INVALID_ARG;
  return guarded<int>(pp, -(int)MR_ERR_CAPACITY, [&]() -> int {
    // pages in use at or behind the number of pages in use move into the free ones in front of it
    const int used = pp->n_pages - (int)pp->free_.size();
    std::vector<int32_t> to(pp->n_pages, -1);
    int n = 0, hole = 0;
    for (int p = pp->n_pages - 1; p >= used && n < max_pairs; --p) {
      if (pp->refs[p] == 0) continue;
      while (pp->refs[hole] != 0) ++hole;
      to[p] = hole;
      pairs[2 * n] = p;
      pairs[2 * n + 1] = hole++;
      ++n;
    }
    for (int i = 0; i < n; ++i) {
      pp->refs[pairs[2 * i + 1]] = pp->refs[pairs[2 * i]];
      pp->refs[pairs[2 * i]] = 0;
    }
    for (auto& kv : pp->seqs)
      for (int32_t& p : kv.second.pages)
        if (p >= 0 && to[p] >= 0) p = to[p];
    pp->free_.clear();
    for (int p = 0; p < pp->n_pages; ++p)
      if (pp->refs[p] == 0) pp->free_.push_back(p);
    return n;
  });
}

int mr_pp_table(mr_page_pool* pp, int64_t seq, int32_t* pages, int max_pages, int* rows) {
  if (!pp || max_pages < 0 || (max_pages > 0 && !pages)) return -(int)MR_ERR_INVALID_ARG;
  return guarded<int>(pp, -(int)MR_ERR_CAPACITY, [&]() -> int {
    auto it = pp->seqs.find(seq);
    if (it == pp->seqs.end()) return -(int)MR_ERR_INVALID_ARG;
    const Seq& s = it->second;
    if ((int)s.pages.size() > max_pages) return -(int)MR_ERR_CAPACITY;
    std::fill(std::copy(s.pages.begin(), s.pages.end(), pages), pages + max_pages, -1);
    if (rows) *rows = s.rows;
    return (int)s.pages.size();
  });
}

mr_status mr_pp_stats(mr_page_pool* pp, int64_t* out) {
  if (!pp || !out) return MR_ERR_INVALID_ARG;
  return guarded<mr_status>(pp, MR_ERR_CAPACITY, [&]() -> mr_status {
    out[0] = pp->n_pages;
    out[1] = (int64_t)pp->free_.size();
    out[2] = (int64_t)pp->seqs.size();
    out[3] = std::count_if(pp->refs.begin(), pp->refs.end(), [](int32_t r) { return r > 1; });
    return MR_OK;
  });
}

}  // extern "C"
