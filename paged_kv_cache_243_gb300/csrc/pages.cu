// Copying pages inside a cache and renaming them in block tables: what a forked
// sequence needs before it writes into a page it shares, and what moving a
// pool's pages together needs.
//
// The page lists are host arrays, checked here as a whole (ranges, a page
// written twice, a page both read and written) before anything is launched,
// and handed to the kernels by value as launch parameters: no device list, no
// host-to-device copy whose buffer would have to outlive the call, and nothing
// the kernels could find wrong.
#include <type_traits>
#include <vector>

#include "pkv_internal.h"

namespace pkv {
namespace {

// A launch's (source, destination) pairs. Launch parameters hold at most
// 32764 bytes; short lists take the small form (their launch carries less), and ids
// below 65536 are passed in 16 bits.
constexpr int kSmallPairs = 64;
template <class T>
constexpr int kLargePairs = 16000 / (int)sizeof(T);
template <class T, int N>
struct PairList {
  T src[N], dst[N];
};

struct CopyParams {
  // [0..3]: K pages, V pages, scales, boxes; [4]: the open groups' originals
  uint8_t* base[5];
  uint32_t bytes[5];       // of one page (or row) of each; 0: not kept
  uint32_t pieces[5];      // kPiece-sized pieces of each
  uint32_t page_pieces;    // of a page over all its parts
  uint32_t num_pairs, num_rows;   // list entries [0, num_pairs) are pages, the next num_rows rows
};

// dst page := src page in every part, byte for byte. Bound by memory: each byte is read and
// written once, past the caches' retention (streaming loads and stores: it comes back no
// sooner than a step later). A block moves one 16 KB piece, four 16-byte loads in flight
// per thread before the first store; pieces of all pages and parts are one grid, so that one
// page of K and V (64 KB) is four blocks and 1024 pages are 16384. 1024 pages of 32 kv heads
// x 16 x 128 bf16: 78.9 us, 6.8 TB/s, the rate of a plain copy; one page of 8 kv heads: 2 us,
// the launch.
constexpr uint32_t kPiece = 16384;
constexpr int kCopyThreads = 256;

template <class T, int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams p,
                                                                  const __grid_constant__ PairList<T, N> list) {
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

// Table entries that equal a source become its destination. Block (x, y) puts
// the y-th kRemapChunk pairs into a hash table in shared memory (open
// addressing, at most half full, source and destination in one word), then looks up a
// share of the entries. Sources are distinct and no destination is a source (checked on
// the host), so an entry is changed by one block at most, whatever the order of the
// blocks, insertions or launches. Bound by building the tables, not by the entries
// (4 bytes read each): pairs are split over blocks, 1024 to a table. 3635 pairs over
// 48 x 512 and over 48 x 4096 entries: 10 and 26 us with 512 pairs to a table read through the
// constant cache, 4.3 and 12 read as below, 5.0 and 8.6 with 1024, 7.9 and 9.6 with 2048;
// one table of all of them took 22 us and more.
constexpr int kRemapThreads = 256, kRemapChunk = 1024, kRemapSlots = 2 * kRemapChunk;
template <class T>
using RemapSlot = std::conditional_t<sizeof(T) == 2, unsigned int, unsigned long long>;

template <class T, int N>
__global__ void __launch_bounds__(kRemapThreads) remap_kernel(int32_t* __restrict__ table, long long entries, int n,
                                                              const __grid_constant__ PairList<T, N> list) {
  using Slot = RemapSlot<T>;
  constexpr int BITS = 8 * (int)sizeof(T);
  constexpr Slot kNone = ~(Slot)0;   // no pair: a page is not moved onto itself
  __shared__ Slot slots[kRemapSlots];
  for (int i = threadIdx.x; i < kRemapSlots; i += kRemapThreads) slots[i] = kNone;
  __syncthreads();
  auto hash = [](uint32_t x) { return (int)((x * 2654435761u) >> 16) & (kRemapSlots - 1); };
  const int first = blockIdx.y * kRemapChunk, end = min(n, first + kRemapChunk);
  // (as ordinary memory: by way of the constant cache the lanes of a warp, which read at different
  // places, would be served one after the other)
  const T *src = list.src, *dst = list.dst;
  asm("" : "+l"(src), "+l"(dst));
  for (int i = first + threadIdx.x; i < end; i += kRemapThreads) {
    const uint32_t key = (uint32_t)src[i];
    const Slot pair = (Slot)key << BITS | (Slot)(uint32_t)dst[i];
    int h = hash(key);
    while (atomicCAS(&slots[h], kNone, pair) != kNone) h = (h + 1) & (kRemapSlots - 1);
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const long long step = (long long)gridDim.x * kRemapThreads;
  for (long long i = (long long)blockIdx.x * kRemapThreads + threadIdx.x; i < entries; i += step) {
    const int32_t t = table[i];
    if (t < 0 || (BITS == 16 && t > 0xFFFF)) continue;
    for (int h = hash((uint32_t)t); slots[h] != kNone; h = (h + 1) & (kRemapSlots - 1)) {
      if ((uint32_t)(slots[h] >> BITS) == (uint32_t)t) {
        table[i] = (int32_t)(slots[h] & (((Slot)1 << BITS) - 1));
        break;
      }
    }
  }
}

// All entries of both lists in [0, limit), `once` without repeats, and none of
// it in `other`. The marks are kept per thread and left clear, so a call
// allocates only when a larger pool is seen.
pkv_status check_lists(int32_t n, const int32_t* once, const int32_t* other, int32_t limit) {
  if (n < 0 || (n > 0 && (!once || !other))) return PKV_ERR_INVALID_ARG;
  if (n == 0) return PKV_OK;
  uint32_t over = 0;
  for (int32_t i = 0; i < n; ++i)
    over |= (uint32_t)((uint32_t)once[i] >= (uint32_t)limit) | (uint32_t)((uint32_t)other[i] >= (uint32_t)limit);
  if (over) return PKV_ERR_INVALID_ARG;
  static thread_local std::vector<uint8_t> marks;
  try {
    if (marks.size() < (size_t)limit) marks.resize((size_t)limit, 0);
  } catch (...) {
    return PKV_ERR_HOST_MEMORY;
  }
  uint8_t* const seen = marks.data();
  uint32_t bad = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t x = once[i];
    bad |= seen[x];
    seen[x] = 1;
  }
  for (int32_t i = 0; i < n; ++i) bad |= seen[other[i]];
  for (int32_t i = 0; i < n; ++i) seen[once[i]] = 0;
  return bad ? PKV_ERR_INVALID_ARG : PKV_OK;
}

template <class T, int N>
pkv_status launch_copy(CopyParams p, const int32_t* src, const int32_t* dst, const int32_t* src_rows,
                       const int32_t* dst_rows, cudaStream_t st) {
  PairList<T, N> list;
  const int np = (int)p.num_pairs, nr = (int)p.num_rows;
  for (int i = 0; i < np; ++i) list.src[i] = (T)src[i];
  for (int i = 0; i < np; ++i) list.dst[i] = (T)dst[i];
  for (int i = 0; i < nr; ++i) {
    list.src[np + i] = (T)src_rows[i];
    list.dst[np + i] = (T)dst_rows[i];
  }
  const unsigned grid = p.num_pairs * p.page_pieces + p.num_rows * p.pieces[4];
  void* args[] = {&p, &list};
  const void* fn = reinterpret_cast<const void*>(&copy_pages_kernel<T, N>);
  return launch_pdl(fn, dim3(grid), dim3(kCopyThreads), 0, st, args) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <class T, int N>
pkv_status launch_remap(int32_t* table, long long entries, int n, const int32_t* src, const int32_t* dst,
                        cudaStream_t st) {
  PairList<T, N> list;
  for (int i = 0; i < n; ++i) list.src[i] = (T)src[i];
  for (int i = 0; i < n; ++i) list.dst[i] = (T)dst[i];
  const void* fn = reinterpret_cast<const void*>(&remap_kernel<T, N>);
  const long long blocks = (entries + kRemapThreads - 1) / kRemapThreads;
  void* args[] = {&table, &entries, &n, &list};
  const dim3 grid((unsigned)(blocks < 304 ? blocks : 304), (unsigned)((n + kRemapChunk - 1) / kRemapChunk));
  return launch_pdl(fn, grid, dim3(kRemapThreads), 0, st, args) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // namespace

pkv_status copy_pages(const pkv_cache* c, int32_t n, const int32_t* src, const int32_t* dst, int32_t n_rows,
                      const int32_t* src_rows, const int32_t* dst_rows, cudaStream_t stream) {
  // (no pool of this many pages fits a device: 1280 bytes is the smallest page's)
  if (c->num_pages > (1 << 28) || c->tail_rows > (1 << 28)) return PKV_ERR_UNSUPPORTED;
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
  const bool narrow = c->num_pages <= 65536 && (n_rows == 0 || c->tail_rows <= 65536);
  const auto go = total <= kSmallPairs ? &launch_copy<int32_t, kSmallPairs>
                  : narrow             ? &launch_copy<uint16_t, kLargePairs<uint16_t>>
                                       : &launch_copy<int32_t, kLargePairs<int32_t>>;
  int64_t cap = total <= kSmallPairs ? kSmallPairs : narrow ? kLargePairs<uint16_t> : kLargePairs<int32_t>;
  const int64_t widest = p.page_pieces > p.pieces[4] ? p.page_pieces : p.pieces[4];
  if (cap * widest >= (1ll << 31)) cap = ((1ll << 31) - 1) / widest;
  for (int64_t at = 0; at < total; at += cap) {
    const int64_t end = at + cap < total ? at + cap : total;
    const int64_t p0 = at < n ? at : n, p1 = end < n ? end : n;        // pages [p0, p1)
    const int64_t r0 = at > n ? at - n : 0, r1 = end > n ? end - n : 0;   // rows [r0, r1)
    p.num_pairs = (uint32_t)(p1 - p0);
    p.num_rows = (uint32_t)(r1 - r0);
    st = go(p, src + p0, dst + p0, src_rows + r0, dst_rows + r0, stream);
    if (st != PKV_OK) return st;
  }
  return PKV_OK;
}

pkv_status remap_block_table(int32_t* table, long long entries, int32_t num_pages, int32_t n, const int32_t* src,
                             const int32_t* dst, cudaStream_t stream) {
  if (num_pages > (1 << 28)) return PKV_ERR_UNSUPPORTED;
  pkv_status st = check_lists(n, src, dst, num_pages);
  if (st != PKV_OK || n == 0 || entries == 0) return st;
  const bool narrow = num_pages <= 65536;
  const int cap = narrow ? kLargePairs<uint16_t> : kLargePairs<int32_t>;
  for (int64_t at = 0; at < n; at += cap) {
    const int m = n - at < cap ? (int)(n - at) : cap;
    const auto go = m <= kSmallPairs ? &launch_remap<int32_t, kSmallPairs>
                    : narrow         ? &launch_remap<uint16_t, kLargePairs<uint16_t>>
                                     : &launch_remap<int32_t, kLargePairs<int32_t>>;
    st = go(table, entries, m, src + at, dst + at, stream);
    if (st != PKV_OK) return st;
  }
  return PKV_OK;
}

}  // namespace pkv
