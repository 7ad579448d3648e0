// Copying pages inside a cache and renaming them in block tables: what a forked
// sequence needs before it writes into a page it shares, and what moving a
// pool's pages together needs.
//
// The page lists are host arrays, checked here as a whole (ranges, a page
// written twice, a page both read and written) before anything is launched,
// and handed to the kernels by value as launch parameters: no device list, no
// host-to-device copy whose buffer would have to outlive the call, and nothing
// the kernels could find wrong.
#include <vector>

#include "pkv_internal.h"

namespace pkv {
namespace {

// A launch's (source, destination) pairs. Launch parameters hold at most
// 32764 bytes; short lists take the small form (their launch carries less).
constexpr int kSmallPairs = 64, kLargePairs = 4000;
template <int N>
struct PairList {
  int32_t src[N], dst[N];
};

struct CopyParams {
  // [0..3]: K pages, V pages, scales, boxes; [4]: the open groups' originals
  uint8_t* base[5];
  uint32_t bytes[5];       // of one page (or row) of each; 0: not kept
  uint32_t pieces[5];      // kPiece-sized pieces of each
  uint32_t page_pieces;    // of a page over all its parts
  uint32_t num_pairs, num_rows;   // list entries [0, num_pairs) are pages, the next num_rows rows
};

constexpr uint32_t kPiece = 16384;
constexpr int kCopyThreads = 256;

template <int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams p,
                                                                  const __grid_constant__ PairList<N> list) {
  pdl_wait();
  pdl_launch_dependents();
  uint32_t e, part = 0, piece;
  const uint32_t page_items = p.num_pairs * p.page_pieces;
  if (blockIdx.x < page_items) {
    e = blockIdx.x / p.page_pieces;
    piece = blockIdx.x - e * p.page_pieces;
    while (piece >= p.pieces[part]) piece -= p.pieces[part++];
  } else {
    part = 4;
    const uint32_t x = blockIdx.x - page_items;
    e = x / p.pieces[4];
    piece = x - e * p.pieces[4];
    e += p.num_pairs;
  }
  const size_t size = p.bytes[part], off = (size_t)piece * kPiece;
  const uint8_t* src = p.base[part] + (size_t)list.src[e] * size + off;
  uint8_t* dst = p.base[part] + (size_t)list.dst[e] * size + off;
  const uint32_t n = (uint32_t)min((size_t)kPiece, size - off) / 16;
  constexpr int U = kPiece / 16 / kCopyThreads;
  uint4 v[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t j = i * kCopyThreads + threadIdx.x;
    if (j < n) v[i] = __ldcs(reinterpret_cast<const uint4*>(src) + j);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t j = i * kCopyThreads + threadIdx.x;
    if (j < n) __stcs(reinterpret_cast<uint4*>(dst) + j, v[i]);
  }
}

// Table entries that equal a source become its destination. Each block puts
// the pairs into a hash table in shared memory (open addressing, at most half
// full), then looks up a share of the entries. Sources are distinct and no
// destination is a source (checked on the host), so neither the order of the
// insertions nor that of several launches matters.
constexpr int kRemapThreads = 256;

template <int N>
__global__ void __launch_bounds__(kRemapThreads) remap_kernel(int32_t* __restrict__ table, long long entries, int n,
                                                              const __grid_constant__ PairList<N> list) {
  constexpr int SLOTS = N <= kSmallPairs ? 128 : 8192;   // a power of two, >= 2 N
  extern __shared__ int32_t slots[];   // keys, then values
  int32_t* val = slots + SLOTS;
  for (int i = threadIdx.x; i < SLOTS; i += kRemapThreads) slots[i] = -1;
  __syncthreads();
  auto hash = [](int32_t x) { return (int)(((uint32_t)x * 2654435761u) >> 16) & (SLOTS - 1); };
  for (int i = threadIdx.x; i < n; i += kRemapThreads) {
    int h = hash(list.src[i]);
    while (atomicCAS(&slots[h], -1, list.src[i]) != -1) h = (h + 1) & (SLOTS - 1);
    val[h] = list.dst[i];
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const long long step = (long long)gridDim.x * kRemapThreads;
  for (long long i = (long long)blockIdx.x * kRemapThreads + threadIdx.x; i < entries; i += step) {
    const int32_t t = table[i];
    if (t < 0) continue;
    for (int h = hash(t); slots[h] != -1; h = (h + 1) & (SLOTS - 1)) {
      if (slots[h] == t) {
        table[i] = val[h];
        break;
      }
    }
  }
}

// A set of small whole numbers with an O(1) clear of what was added; kept per
// thread, so a call allocates only when a larger pool is seen.
class Marks {
 public:
  bool reserve(size_t n) {
    try {
      if (bits_.size() < (n + 63) / 64) bits_.resize((n + 63) / 64, 0);
    } catch (...) {
      return false;
    }
    return true;
  }
  bool add(uint32_t x) {   // false: was there
    const uint64_t m = 1ull << (x & 63);
    const bool had = bits_[x >> 6] & m;
    bits_[x >> 6] |= m;
    return !had;
  }
  bool has(uint32_t x) const { return bits_[x >> 6] >> (x & 63) & 1; }
  void remove(uint32_t x) { bits_[x >> 6] &= ~(1ull << (x & 63)); }

 private:
  std::vector<uint64_t> bits_;
};

// All entries of both lists in [0, limit), `once` without repeats, and none of
// it in `other`.
pkv_status check_lists(int32_t n, const int32_t* once, const int32_t* other, int32_t limit) {
  if (n < 0 || (n > 0 && (!once || !other))) return PKV_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (once[i] < 0 || once[i] >= limit || other[i] < 0 || other[i] >= limit) return PKV_ERR_INVALID_ARG;
  if (n == 0) return PKV_OK;
  static thread_local Marks marks;
  if (!marks.reserve((size_t)limit)) return PKV_ERR_HOST_MEMORY;
  pkv_status st = PKV_OK;
  int32_t added = 0;
  while (added < n && marks.add((uint32_t)once[added])) ++added;
  if (added < n) st = PKV_ERR_INVALID_ARG;
  for (int32_t i = 0; st == PKV_OK && i < n; ++i)
    if (marks.has((uint32_t)other[i])) st = PKV_ERR_INVALID_ARG;
  for (int32_t i = 0; i < added; ++i) marks.remove((uint32_t)once[i]);
  return st;
}

template <int N>
pkv_status launch_copy(CopyParams p, const int32_t* src, const int32_t* dst, const int32_t* src_rows,
                       const int32_t* dst_rows, cudaStream_t st) {
  PairList<N> list;
  const int np = (int)p.num_pairs, nr = (int)p.num_rows;
  for (int i = 0; i < np; ++i) {
    list.src[i] = src[i];
    list.dst[i] = dst[i];
  }
  for (int i = 0; i < nr; ++i) {
    list.src[np + i] = src_rows[i];
    list.dst[np + i] = dst_rows[i];
  }
  const unsigned grid = p.num_pairs * p.page_pieces + p.num_rows * p.pieces[4];
  void* args[] = {&p, &list};
  const void* fn = reinterpret_cast<const void*>(&copy_pages_kernel<N>);
  return launch_pdl(fn, dim3(grid), dim3(kCopyThreads), 0, st, args) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int N>
pkv_status launch_remap(int32_t* table, long long entries, int n, const int32_t* src, const int32_t* dst,
                        cudaStream_t st) {
  PairList<N> list;
  for (int i = 0; i < n; ++i) {
    list.src[i] = src[i];
    list.dst[i] = dst[i];
  }
  constexpr size_t smem = (N <= kSmallPairs ? 128 : 8192) * 2 * sizeof(int32_t);
  const void* fn = reinterpret_cast<const void*>(&remap_kernel<N>);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return PKV_ERR_CUDA;
  const long long blocks = (entries + kRemapThreads - 1) / kRemapThreads;
  void* args[] = {&table, &entries, &n, &list};
  return launch_pdl(fn, dim3((unsigned)(blocks < 304 ? blocks : 304)), dim3(kRemapThreads), smem, st, args) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // namespace

pkv_status copy_pages(const pkv_cache* c, int32_t n, const int32_t* src, const int32_t* dst, int32_t n_rows,
                      const int32_t* src_rows, const int32_t* dst_rows, cudaStream_t stream) {
  pkv_status st = check_lists(n, dst, src, c->num_pages);
  if (st != PKV_OK) return st;
  if (n_rows != 0 && (c->quant != PKV_QUANT_PER_GROUP64 || !c->tail)) return PKV_ERR_INVALID_ARG;
  if (n_rows > 0 && (reinterpret_cast<uintptr_t>(c->tail) & 15u)) return PKV_ERR_INVALID_ARG;
  st = check_lists(n_rows, dst_rows, src_rows, c->tail_rows);
  if (st != PKV_OK) return st;
  const uint64_t rows = (uint64_t)c->num_kv_heads * c->page_size;
  const uint64_t row = c->kv_dtype == PKV_U4 ? c->head_dim / 2 : (c->kv_dtype == PKV_I8 ? c->head_dim : 2 * c->head_dim);
  const uint64_t gran = c->quant == PKV_QUANT_PER_GROUP64 ? 64 : 1;
  const uint64_t bytes[5] = {rows * row, rows * row, c->quant == PKV_QUANT_NONE ? 0 : rows / gran * 16,
                             c->page_meta ? (uint64_t)c->num_kv_heads * 2 * c->head_dim * 4 : 0,
                             (uint64_t)c->num_kv_heads * 2 * 2 * 64 * c->head_dim * 4};
  CopyParams p = {};
  void* base[5] = {c->k_pages, c->v_pages, c->kv_sz, c->page_meta, c->tail};
  for (int i = 0; i < 5; ++i) {
    if (bytes[i] > (1u << 30)) return PKV_ERR_UNSUPPORTED;   // one page of one pool
    p.base[i] = static_cast<uint8_t*>(base[i]);
    p.bytes[i] = (uint32_t)bytes[i];
    p.pieces[i] = (uint32_t)((bytes[i] + kPiece - 1) / kPiece);
    if (i < 4) p.page_pieces += p.pieces[i];
  }
  const int64_t total = (int64_t)n + n_rows;
  if (total == 0) return PKV_OK;
  // as many pairs a launch as its parameters and its grid (below 2^31 blocks) hold
  int64_t cap = total <= kSmallPairs ? kSmallPairs : kLargePairs;
  const int64_t widest = p.page_pieces > p.pieces[4] ? p.page_pieces : p.pieces[4];
  if (cap * widest >= (1ll << 31)) cap = ((1ll << 31) - 1) / widest;
  for (int64_t at = 0; at < total; at += cap) {
    const int64_t end = at + cap < total ? at + cap : total;
    const int64_t p0 = at < n ? at : n, p1 = end < n ? end : n;        // pages [p0, p1)
    const int64_t r0 = at > n ? at - n : 0, r1 = end > n ? end - n : 0;   // rows [r0, r1)
    p.num_pairs = (uint32_t)(p1 - p0);
    p.num_rows = (uint32_t)(r1 - r0);
    auto go = cap <= kSmallPairs ? &launch_copy<kSmallPairs> : &launch_copy<kLargePairs>;
    st = go(p, src + p0, dst + p0, src_rows + r0, dst_rows + r0, stream);
    if (st != PKV_OK) return st;
  }
  return PKV_OK;
}

pkv_status remap_block_table(int32_t* table, long long entries, int32_t num_pages, int32_t n, const int32_t* src,
                             const int32_t* dst, cudaStream_t stream) {
  pkv_status st = check_lists(n, src, dst, num_pages);
  if (st != PKV_OK || n == 0 || entries == 0) return st;
  for (int32_t at = 0; at < n; at += kLargePairs) {
    const int m = n - at < kLargePairs ? n - at : kLargePairs;
    auto go = m <= kSmallPairs ? &launch_remap<kSmallPairs> : &launch_remap<kLargePairs>;
    st = go(table, entries, m, src + at, dst + at, stream);
    if (st != PKV_OK) return st;
  }
  return PKV_OK;
}

}  // namespace pkv
