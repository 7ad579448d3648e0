// Host page allocator [HBM-layout page, section 三: allocate_blocks takes
// ceil(tokens / block_size) blocks from a free list and fails (None) when the
// list is short; free_sequence returns a sequence's blocks to the list].
// Pages leave the free list from the front and return to its back, so the
// allocation order is deterministic.
//
// A page may belong to several sequences (fork); `refs` counts its owners, and
// it returns to the free list when the last of them lets go. What a call needs
// is allocated before anything changes, so a call that fails (no pages, no host
// memory) leaves the allocator as it was.
#include <algorithm>
#include <deque>
#include <unordered_map>
#include <vector>

#include "pkv.h"

struct pkv_allocator {
  int32_t num_pages = 0;
  std::deque<int32_t> free_list;
  std::unordered_map<int64_t, std::vector<int32_t>> owned;
  std::vector<int32_t> refs;   // owners of each page
};

namespace {

// C entry points let no exception out; the standard containers only throw for
// lack of memory.
template <class F>
pkv_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return PKV_ERR_HOST_MEMORY;
  }
}

void write_row(const std::vector<int32_t>& pages, int32_t* row, int32_t max_pages) {
  for (int32_t i = 0; i < max_pages; ++i) row[i] = i < (int32_t)pages.size() ? pages[i] : -1;
}

}  // namespace

extern "C" {

pkv_status pkv_alloc_create(int32_t num_pages, pkv_allocator** out) {
  if (!out || num_pages < 0) return PKV_ERR_INVALID_ARG;
  pkv_allocator* a = nullptr;
  const pkv_status st = guarded([&] {
    a = new pkv_allocator();
    a->num_pages = num_pages;
    a->refs.assign(num_pages, 0);
    for (int32_t i = 0; i < num_pages; ++i) a->free_list.push_back(i);
    return PKV_OK;
  });
  if (st != PKV_OK) {
    delete a;
    return st;
  }
  *out = a;
  return PKV_OK;
}

void pkv_alloc_destroy(pkv_allocator* a) { delete a; }

pkv_status pkv_alloc_reserve(pkv_allocator* a, int64_t seq_id, int32_t total_tokens,
                             int32_t page_size, int32_t* block_table_row, int32_t max_pages) {
  if (!a || total_tokens < 0 || page_size <= 0 || max_pages < 0) return PKV_ERR_INVALID_ARG;
  if (max_pages > 0 && !block_table_row) return PKV_ERR_INVALID_ARG;
  const int64_t need = ((int64_t)total_tokens + page_size - 1) / page_size;
  if (need > max_pages) return PKV_ERR_INVALID_ARG;
  return guarded([&] {
    auto it = a->owned.find(seq_id);
    const int64_t have = it == a->owned.end() ? 0 : (int64_t)it->second.size();
    const int64_t extra = need > have ? need - have : 0;
    if (extra > (int64_t)a->free_list.size()) return PKV_ERR_OUT_OF_PAGES;
    const bool is_new = it == a->owned.end();
    if (is_new) it = a->owned.emplace(seq_id, std::vector<int32_t>()).first;
    std::vector<int32_t>& pages = it->second;
    try {
      if (extra > 0 && pages.capacity() < (size_t)need)
        pages.reserve(std::max((size_t)need, 2 * pages.capacity()));
    } catch (...) {
      if (is_new) a->owned.erase(it);
      throw;
    }
    for (int64_t i = 0; i < extra; ++i) {
      pages.push_back(a->free_list.front());
      a->free_list.pop_front();
      a->refs[pages.back()] = 1;
    }
    write_row(pages, block_table_row, max_pages);
    return PKV_OK;
  });
}

pkv_status pkv_alloc_fork(pkv_allocator* a, int64_t parent, int64_t child, int32_t tokens, int32_t page_size,
                          int32_t* block_table_row, int32_t max_pages) {
  if (!a || tokens < 0 || page_size <= 0 || max_pages < 0) return PKV_ERR_INVALID_ARG;
  if (max_pages > 0 && !block_table_row) return PKV_ERR_INVALID_ARG;
  const int64_t need = ((int64_t)tokens + page_size - 1) / page_size;
  if (need > max_pages) return PKV_ERR_INVALID_ARG;
  return guarded([&] {
    auto it = a->owned.find(parent);
    if (it == a->owned.end() || (int64_t)it->second.size() < need) return PKV_ERR_INVALID_ARG;
    if (a->owned.count(child)) return PKV_ERR_INVALID_ARG;
    std::vector<int32_t> pages(it->second.begin(), it->second.begin() + need);
    std::vector<int32_t>& mine = a->owned[child];   // may move the parent's node: `it` is not used after
    mine.swap(pages);
    for (int32_t pg : mine) ++a->refs[pg];
    write_row(mine, block_table_row, max_pages);
    return PKV_OK;
  });
}

pkv_status pkv_alloc_unshare(pkv_allocator* a, int64_t seq_id, int32_t first_token, int32_t page_size,
                             int32_t max_copies, int32_t* src_pages, int32_t* dst_pages, int32_t* num_copies,
                             int32_t* block_table_row, int32_t max_pages) {
  if (!a || !num_copies || first_token < 0 || page_size <= 0 || max_copies < 0 || max_pages < 0)
    return PKV_ERR_INVALID_ARG;
  if (max_copies > 0 && (!src_pages || !dst_pages)) return PKV_ERR_INVALID_ARG;
  if (max_pages > 0 && !block_table_row) return PKV_ERR_INVALID_ARG;
  auto it = a->owned.find(seq_id);
  if (it == a->owned.end()) return PKV_ERR_INVALID_ARG;
  std::vector<int32_t>& pages = it->second;
  if ((int64_t)pages.size() > max_pages) return PKV_ERR_INVALID_ARG;
  int64_t n = 0;
  const size_t first = (size_t)(first_token / page_size);
  for (size_t i = first; i < pages.size(); ++i) n += a->refs[pages[i]] > 1;
  if (n > max_copies) return PKV_ERR_INVALID_ARG;
  if (n > (int64_t)a->free_list.size()) return PKV_ERR_OUT_OF_PAGES;
  n = 0;
  for (size_t i = first; i < pages.size(); ++i) {
    if (a->refs[pages[i]] <= 1) continue;
    src_pages[n] = pages[i];
    dst_pages[n] = a->free_list.front();
    a->free_list.pop_front();
    --a->refs[pages[i]];
    pages[i] = dst_pages[n++];
    a->refs[pages[i]] = 1;
  }
  *num_copies = (int32_t)n;
  write_row(pages, block_table_row, max_pages);
  return PKV_OK;
}

pkv_status pkv_alloc_compact(pkv_allocator* a, int32_t max_moves, int32_t* src_pages, int32_t* dst_pages,
                             int32_t* num_moves) {
  if (!a || !num_moves || max_moves < 0) return PKV_ERR_INVALID_ARG;
  if (max_moves > 0 && (!src_pages || !dst_pages)) return PKV_ERR_INVALID_ARG;
  return guarded([&] {
    std::vector<int32_t> to(a->num_pages);   // where each page goes
    for (int32_t p = 0; p < a->num_pages; ++p) to[p] = p;
    std::vector<uint8_t> taken(a->num_pages, 0);
    int32_t n = 0, lo = 0, hi = a->num_pages - 1;
    while (n < max_moves) {
      while (lo < hi && a->refs[lo] > 0) ++lo;
      while (lo < hi && a->refs[hi] == 0) --hi;
      if (lo >= hi) break;
      src_pages[n] = hi;
      dst_pages[n++] = lo;
      to[hi--] = lo;
      taken[lo++] = 1;
    }
    // the free list keeps its order without the pages taken; the pages left
    // go to its back
    std::deque<int32_t> rest;
    for (int32_t pg : a->free_list)
      if (!taken[pg]) rest.push_back(pg);
    for (int32_t i = 0; i < n; ++i) rest.push_back(src_pages[i]);
    a->free_list.swap(rest);
    for (int32_t i = 0; i < n; ++i) {
      a->refs[dst_pages[i]] = a->refs[src_pages[i]];
      a->refs[src_pages[i]] = 0;
    }
    for (auto& kv : a->owned)
      for (int32_t& pg : kv.second) pg = to[pg];
    *num_moves = n;
    return PKV_OK;
  });
}

pkv_status pkv_alloc_table(const pkv_allocator* a, int64_t seq_id, int32_t* block_table_row, int32_t max_pages) {
  if (!a || max_pages < 0 || (max_pages > 0 && !block_table_row)) return PKV_ERR_INVALID_ARG;
  auto it = a->owned.find(seq_id);
  if (it == a->owned.end() || (int64_t)it->second.size() > max_pages) return PKV_ERR_INVALID_ARG;
  write_row(it->second, block_table_row, max_pages);
  return PKV_OK;
}

pkv_status pkv_alloc_free(pkv_allocator* a, int64_t seq_id) {
  if (!a) return PKV_ERR_INVALID_ARG;
  auto it = a->owned.find(seq_id);
  if (it == a->owned.end()) return PKV_ERR_INVALID_ARG;
  return guarded([&] {
    // from the first page on: the order in which they return to the list
    const size_t before = a->free_list.size();
    try {
      for (int32_t pg : it->second)
        if (a->refs[pg] == 1) a->free_list.push_back(pg);
    } catch (...) {
      while (a->free_list.size() > before) a->free_list.pop_back();
      throw;
    }
    for (int32_t pg : it->second) --a->refs[pg];
    a->owned.erase(it);
    return PKV_OK;
  });
}

int32_t pkv_alloc_num_free(const pkv_allocator* a) { return a ? (int32_t)a->free_list.size() : 0; }

int32_t pkv_alloc_seq_pages(const pkv_allocator* a, int64_t seq_id) {
  if (!a) return 0;
  auto it = a->owned.find(seq_id);
  return it == a->owned.end() ? 0 : (int32_t)it->second.size();
}

int32_t pkv_alloc_page_refs(const pkv_allocator* a, int32_t page) {
  if (!a || page < 0 || page >= a->num_pages) return 0;
  return a->refs[page];
}

int32_t pkv_alloc_check(const pkv_allocator* a) {
  if (!a) return 0;
  int32_t bad = 0;
  const pkv_status st = guarded([&] {
    std::vector<int32_t> listed(a->num_pages, 0), owners(a->num_pages, 0);
    auto mark = [&](std::vector<int32_t>& count, int32_t pg) {
      if (pg < 0 || pg >= a->num_pages) ++bad;
      else ++count[pg];
    };
    for (int32_t pg : a->free_list) mark(listed, pg);
    for (const auto& kv : a->owned)
      for (int32_t pg : kv.second) mark(owners, pg);
    for (int32_t p = 0; p < a->num_pages; ++p)
      bad += owners[p] != a->refs[p] || listed[p] != (owners[p] == 0 ? 1 : 0);
    return PKV_OK;
  });
  return st == PKV_OK ? bad : -1;
}

}  // extern "C"
