// The page allocator with a memory that runs out at its n-th request, for every n: each call either
// succeeds or leaves the allocator as it was. Prints the number of refused calls.
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <new>
#include <vector>

#include "allocator.cpp"

static long left = -1;   // requests that still succeed; -1: all

void* operator new(std::size_t n) {
  if (left == 0) throw std::bad_alloc();
  if (left > 0) --left;
  if (void* p = std::malloc(n)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

constexpr int kPages = 1500, kWidth = 1200;

struct State {
  std::vector<int32_t> v;
  explicit State(pkv_allocator* a) {
    v.reserve(8 * kWidth + kPages);
    for (int64_t s = 0; s < 8; ++s) {
      std::vector<int32_t> row(kWidth, -2);
      pkv_alloc_table(a, s, row.data(), kWidth);
      v.insert(v.end(), row.begin(), row.end());
      v.push_back(pkv_alloc_seq_pages(a, s));
    }
    for (int32_t p = 0; p < kPages; ++p) v.push_back(pkv_alloc_page_refs(a, p));
    v.push_back(pkv_alloc_num_free(a));
    v.insert(v.end(), a->free_list.begin(), a->free_list.end());
  }
};

#define NEED(c) \
  if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); }

int main() {
  std::vector<int32_t> row(kWidth), src(kPages), dst(kPages);
  int32_t n = 0;
  // sequences 0 (1000 pages), 1 (a fork of 700 of them), 2 (300 pages)
  auto make = [&] {
    pkv_allocator* a = nullptr;
    NEED(pkv_alloc_create(kPages, &a) == PKV_OK);
    NEED(pkv_alloc_reserve(a, 0, 16000, 16, row.data(), kWidth) == PKV_OK);
    NEED(pkv_alloc_reserve(a, 2, 4800, 16, row.data(), kWidth) == PKV_OK);
    NEED(pkv_alloc_fork(a, 0, 1, 11200, 16, row.data(), kWidth) == PKV_OK);
    return a;
  };
  const std::vector<std::function<pkv_status(pkv_allocator*)>> calls = {
      [&](pkv_allocator* a) { return pkv_alloc_reserve(a, 5, 3000, 16, row.data(), kWidth); },
      [&](pkv_allocator* a) { return pkv_alloc_reserve(a, 2, 7000, 16, row.data(), kWidth); },
      [&](pkv_allocator* a) { return pkv_alloc_fork(a, 0, 6, 16000, 16, row.data(), kWidth); },
      [&](pkv_allocator* a) { return pkv_alloc_unshare(a, 1, 9600, 16, kPages, src.data(), dst.data(), &n, row.data(), kWidth); },
      [&](pkv_allocator* a) { return pkv_alloc_compact(a, kPages, src.data(), dst.data(), &n); },
      [&](pkv_allocator* a) { return pkv_alloc_free(a, 0); },
      [&](pkv_allocator* a) { return pkv_alloc_free(a, 2); },
  };
  int refused = 0;
  for (size_t c = 0; c < calls.size(); ++c) {
    for (long k = 0;; ++k) {
      pkv_allocator* a = make();
      const State before(a);
      left = k;
      const pkv_status st = calls[c](a);
      left = -1;
      NEED(pkv_alloc_check(a) == 0);
      const bool same = State(a).v == before.v;
      pkv_alloc_destroy(a);
      if (st == PKV_OK) break;
      NEED(st == PKV_ERR_HOST_MEMORY);
      if (!same) std::printf("call %zu, request %ld: the allocator has changed\n", c, k);
      NEED(same);
      ++refused;
      NEED(k < 100000);
    }
  }
  left = 0;
  pkv_allocator* a = nullptr;
  NEED(pkv_alloc_create(kPages, &a) == PKV_ERR_HOST_MEMORY && !a);
  left = -1;
  std::printf("refused %d\n", refused);
}
