// Shared-prefix attention, and attention for trees of drafts: launch plans of the kernels in
// shared_kernel.cuh.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <set>
#include <utility>

#include "shared_kernel.cuh"

namespace pkv {

const void* shared_kernel_f16(int D);
const void* shared_kernel_bf16(int D);
const void* shared_kernel_i8t(int D, bool bf);
const void* shared_kernel_i8g(int D, bool bf);
const void* shared_kernel_u4t(int D, bool bf);
const void* tree_kernel_f16(int D, bool few);
const void* tree_kernel_bf16(int D, bool few);
const void* tree_kernel_i8t(int D, bool bf, bool few);
const void* tree_kernel_i8g(int D, bool bf, bool few);
const void* tree_kernel_u4t(int D, bool bf, bool few);

namespace {

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct Device {
  int index = 0, sms = 0, smem = 0;
};

// The current device; its numbers are asked for once.
pkv_status device(Device& d) {
  constexpr int kMost = 64;
  static std::mutex mu;
  static Device known[kMost];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  if (dev < 0 || dev >= kMost) return PKV_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev].sms == 0) {
    Device n;
    n.index = dev;
    if (cudaDeviceGetAttribute(&n.smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return PKV_ERR_CUDA;
    known[dev] = n;
  }
  d = known[dev];
  return PKV_OK;
}

// Let a kernel have the device's shared memory; once per device and kernel.
pkv_status allow_smem(const void* fn, const Device& d) {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  try {
    std::lock_guard<std::mutex> lk(mu);
    const auto key = std::make_pair(d.index, fn);
    if (done.count(key)) return PKV_OK;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem) != cudaSuccess)
      return PKV_ERR_CUDA;
    done.insert(key);
    return PKV_OK;
  } catch (...) {
    return PKV_ERR_HOST_MEMORY;
  }
}

// Workspace: each row's place in the plan, (m, l) by record row, accumulators.
// Record rows: one per query row, segment kind and stream for the block where the
// segment begins, and 256 per block for the segment that it continues.
struct Work {
  size_t ml, acc, total;
};
Work layout(const pkv_cache* c, int batch, int hq, int ctas) {
  const size_t rows = 4 * (size_t)batch * hq + (size_t)ctas * 2 * kTile;
  Work w;
  w.ml = align256((size_t)batch * c->num_kv_heads * 3 * sizeof(int4));
  w.acc = w.ml + align256(rows * sizeof(float2));
  w.total = w.acc + align256(rows * c->head_dim * sizeof(float)) + 256;
  return w;
}

// For trees: each pair of row tiles' place, and besides the blocks' 256 one record row per query row of each sequence's kv head,
// rounded up to 32; where rows are few (16 at most) one of each stream. (Counted as the latter up to 64 rows: a workspace
// for some drafts serves fewer, too.)
size_t tree_record_rows(const pkv_cache* c, int sequences, int drafts, int group, int ctas) {
  return (size_t)sequences * c->num_kv_heads * std::max(64, (drafts * group + 31) / 32 * 32) + (size_t)(ctas + 1) * 2 * kTile;
}
// Their values are counted in 32 bits.
bool tree_records_fit(const pkv_cache* c, int sequences, int drafts, int group, int ctas) {
  return tree_record_rows(c, sequences, drafts, group, ctas) * c->head_dim < (1ull << 31);
}
Work tree_layout(const pkv_cache* c, int sequences, int drafts, int group, int ctas) {
  const size_t recs = tree_record_rows(c, sequences, drafts, group, ctas), heads = (size_t)sequences * c->num_kv_heads;
  const size_t pairs = (drafts * group + 2 * kTile - 1) / (2 * kTile);
  Work w;
  w.ml = align256(heads * pairs * sizeof(int4));
  w.acc = w.ml + align256(recs * sizeof(float2));
  w.total = w.acc + align256(recs * c->head_dim * sizeof(float)) + 256;
  return w;
}
int tree_pairs(int drafts, int group) { return (drafts * group + 2 * kTile - 1) / (2 * kTile); }

using EncodeTiledFn = PFN_cuTensorMapEncodeTiled_v12000;
EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// A 16-bit pool as [rows][d], copied in boxes of 16 rows x 64 channels.
bool pool_map(void* base, uint64_t rows, int d, bool bf, CUtensorMap& m) {
  const EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d, rows}, strides[1] = {(cuuint64_t)d * 2};
  const cuuint32_t box[2] = {64, 16}, step[2] = {1, 1};
  return enc(&m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, dims, strides, box,
             step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [rows][heads][d] in boxes of 64 channels x a group's heads x `drafts` rows.
bool query_map(const void* q, uint64_t rows, int heads, int group, int d, int drafts, bool bf, CUtensorMap& m) {
  const EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, rows}, strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)drafts}, step[3] = {1, 1, 1};
  return enc(&m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(q), dims,
             strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int kind_of(const pkv_cache* c) {
  return c->kv_dtype == PKV_F16 ? KV_F16 : c->kv_dtype == PKV_BF16 ? KV_BF16 : c->kv_dtype == PKV_U4 ? KV_U4T
         : c->quant == PKV_QUANT_PER_TOKEN ? KV_I8T : KV_I8G;
}

template <int D, int KV>
void sizes(int& threads, int& smem, int& entries, SharedLayout& lay, int avail, int batch, int groups, bool tree) {
  using G = SharedGeom<D, KV, true>;   // operand types have the same sizes
  threads = G::THREADS;
  entries = kMaxEntries;
  while (entries > 1 && 1024 + shared_layout<G>(entries, batch, groups, tree).total > avail) --entries;
  lay = shared_layout<G>(entries, batch, groups, tree);
  smem = 1024 + lay.total;
}

// Block and shared memory of the attention kernel, and its parameters from the cache.
pkv_status cache_params(const pkv_cache* c, const Device& dev, const void* fn, int rows, int groups, bool tree,
                        SharedParams& p, int& threads, int& smem) {
  const int D = c->head_dim, kind = kind_of(c);
#define PKV_SIZES(d, kv) \
  if (D == d && kind == kv) sizes<d, kv>(threads, smem, p.entries, p.lay, dev.smem, rows, groups, tree);
  PKV_SIZES(64, KV_F16) PKV_SIZES(64, KV_BF16) PKV_SIZES(64, KV_I8T) PKV_SIZES(64, KV_I8G) PKV_SIZES(64, KV_U4T)
  PKV_SIZES(128, KV_F16) PKV_SIZES(128, KV_BF16) PKV_SIZES(128, KV_I8T) PKV_SIZES(128, KV_I8G) PKV_SIZES(128, KV_U4T)
#undef PKV_SIZES
  if (smem > dev.smem) return PKV_ERR_UNSUPPORTED;
  const pkv_status st = allow_smem(fn, dev);
  if (st != PKV_OK) return st;
  if (kind == KV_F16 || kind == KV_BF16) {
    const uint64_t n = (uint64_t)c->num_pages * c->num_kv_heads * c->page_size;
    if (!pool_map(c->k_pages, n, D, kind == KV_BF16, p.tmap_k) || !pool_map(c->v_pages, n, D, kind == KV_BF16, p.tmap_v))
      return PKV_ERR_CUDA;
  }
  p.k_pages = static_cast<const uint8_t*>(c->k_pages);
  p.v_pages = static_cast<const uint8_t*>(c->v_pages);
  p.kv_sz = c->kv_sz;
  p.num_pages = c->num_pages;
  p.page_size = c->page_size;
  p.num_kv_heads = c->num_kv_heads;
  p.kv_kind = kind;
  return PKV_OK;
}

template <int D>
const void* merge_kernel(int warps) {
  return warps == 4 ? reinterpret_cast<const void*>(&shared_merge_kernel<D, 4>)
                    : reinterpret_cast<const void*>(&shared_merge_kernel<D, 1>);
}

template <int D>
const void* tree_merge(int warps) {
  return warps == 4 ? reinterpret_cast<const void*>(&tree_merge_kernel<D, 4>)
                    : reinterpret_cast<const void*>(&tree_merge_kernel<D, 1>);
}

}  // namespace

pkv_status shared_workspace_bytes(const pkv_cache* c, int batch, int num_q_heads, int num_splits, size_t& bytes) {
  Device dev;
  if (num_splits == 0) {
    const pkv_status st = device(dev);
    if (st != PKV_OK) return st;
  }
  bytes = layout(c, batch, num_q_heads, num_splits ? num_splits : dev.sms).total;
  return PKV_OK;
}

pkv_status launch_shared(const SharedArgs& a) {
  const pkv_cache* c = a.cache;
  Device dev;
  pkv_status st = device(dev);
  if (st != PKV_OK) return st;
  const int D = c->head_dim, group = a.num_q_heads / c->num_kv_heads, kind = kind_of(c);
  // visits are counted in 32 bits: rows and prefixes at the table's full width
  const long long tiles = ((long long)a.max_pages * c->page_size + kTile - 1) / kTile;
  const int ctas = a.num_splits ? a.num_splits : dev.sms;
  if (c->num_kv_heads * tiles * (2ll * a.batch + (long long)a.batch * group / (2 * kTile)) >= (1ll << 31) ||
      (4ll * a.batch * a.num_q_heads + 512ll * ctas) * D >= (1ll << 31))
    return PKV_ERR_UNSUPPORTED;
  const Work w = layout(c, a.batch, a.num_q_heads, ctas);
  if (!a.workspace || (reinterpret_cast<uintptr_t>(a.workspace) & 255u) || a.workspace_bytes < w.total)
    return PKV_ERR_WORKSPACE;

  SharedParams p = {};
  const bool bf = a.q_dtype == PKV_BF16;
  const void* fn = kind == KV_F16    ? shared_kernel_f16(D)
                   : kind == KV_BF16 ? shared_kernel_bf16(D)
                   : kind == KV_I8T  ? shared_kernel_i8t(D, bf)
                   : kind == KV_I8G  ? shared_kernel_i8g(D, bf)
                                     : shared_kernel_u4t(D, bf);
  int threads = 0, smem = 0;
  st = cache_params(c, dev, fn, a.batch, a.num_groups, false, p, threads, smem);
  if (st != PKV_OK) return st;
  p.q = static_cast<const uint8_t*>(a.q);
  p.out = a.out;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.prefix_group = a.prefix_group;
  p.prefix_lens = a.prefix_lens;
  p.dev_status = a.dev_status;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.ws_info = reinterpret_cast<int4*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(ws + w.ml);
  p.ws_acc = reinterpret_cast<float*>(ws + w.acc);
  p.num_q_heads = a.num_q_heads;
  p.group = group;
  p.batch = a.batch;
  p.max_pages = a.max_pages;
  p.num_groups = a.num_groups;
  p.num_ctas = ctas;
  p.round_to = kind == KV_I8G ? 64 : 16;
  p.q_dtype = a.q_dtype;
  p.out_dtype = a.out_dtype;
  p.two_terms = a.out_dtype == PKV_F32;
  p.scale = a.sm_scale * 1.4426950408889634f;
  void* args[] = {&p};
  if (launch_pdl(fn, dim3(ctas), dim3(threads), smem, a.stream, args) != cudaSuccess) return PKV_ERR_CUDA;
  const long long outs = (long long)a.batch * a.num_q_heads * D, units = (outs + 127) / 128;
  // Few outputs have many records each, and four warps apiece do not fill the device; more of them
  // are better off with a warp each. One warp against four, us a call: 8 units (2 short rows) 10.8 and
  // 11.2, 64 (2 rows x 64K) 59 and 51, INT8 65 and 56, 512 (16 rows x 32K) 94 and 91, 768 (24 rows x
  // 16K, 4-bit) 45.6 and 42.5, 1024 (32 rows x 2K) 23.3 and 25.1, 2048 (64 rows x 16K) 49.4 and 48.1,
  // (64 rows x 8K, INT8) 58.1 and 59.9, 3904 (5 groups x 5K) 46.6 and 57.6, 8192 (256 rows x 8K) 83 and 104.
  const int wpw = units < 6 * dev.sms ? 4 : 1;
  const void* merge = D == 64 ? merge_kernel<64>(wpw) : merge_kernel<128>(wpw);
  const int per = 4 / wpw;
  return launch_pdl(merge, dim3((unsigned)((units + per - 1) / per)), dim3(kMergeThreads), 0, a.stream, args) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

pkv_status tree_workspace_bytes(const pkv_cache* c, int batch, int drafts, int num_q_heads, int num_splits,
                                size_t& bytes) {
  Device dev;
  if (num_splits == 0) {
    const pkv_status st = device(dev);
    if (st != PKV_OK) return st;
  }
  const int group = num_q_heads / c->num_kv_heads, ctas = num_splits ? num_splits : dev.sms;
  if (!tree_records_fit(c, batch, drafts, group, ctas)) return PKV_ERR_UNSUPPORTED;
  bytes = tree_layout(c, batch, drafts, group, ctas).total;
  return PKV_OK;
}

pkv_status launch_tree(const TreeArgs& a) {
  const pkv_cache* c = a.cache;
  Device dev;
  pkv_status st = device(dev);
  if (st != PKV_OK) return st;
  const int D = c->head_dim, group = a.num_q_heads / c->num_kv_heads, kind = kind_of(c);
  const int rows = a.batch * a.drafts, pairs = tree_pairs(a.drafts, group);
  // visits, two units each at most, are counted in 32 bits
  static_assert(SharedGeom<64, KV_F16, false>::FEW <= 32, "few rows: records of two streams within 64");
  const long long tiles = ((long long)a.max_pages * c->page_size + kTile - 1) / kTile;
  const int ctas = a.num_splits ? a.num_splits : dev.sms;
  if (2 * (tiles + 4) >= (1ll << 31) / ((long long)c->num_kv_heads * a.batch * pairs) ||
      !tree_records_fit(c, a.batch, a.drafts, group, ctas))
    return PKV_ERR_UNSUPPORTED;
  const Work w = tree_layout(c, a.batch, a.drafts, group, ctas);
  if (!a.workspace || (reinterpret_cast<uintptr_t>(a.workspace) & 255u) || a.workspace_bytes < w.total)
    return PKV_ERR_WORKSPACE;
  SharedParams p = {};
  const bool bf = a.q_dtype == PKV_BF16;
  const bool few = a.drafts * group <= (kind == KV_F16 || kind == KV_BF16 ? SharedGeom<64, KV_F16, false>::FEW
                                                                         : SharedGeom<64, KV_I8T, false>::FEW);
  const void* fn = kind == KV_F16    ? tree_kernel_f16(D, few)
                   : kind == KV_BF16 ? tree_kernel_bf16(D, few)
                   : kind == KV_I8T  ? tree_kernel_i8t(D, bf, few)
                   : kind == KV_I8G  ? tree_kernel_i8g(D, bf, few)
                                     : tree_kernel_u4t(D, bf, few);
  int threads = 0, smem = 0;
  st = cache_params(c, dev, fn, 0, a.batch, true, p, threads, smem);
  if (st != PKV_OK) return st;
  p.q = static_cast<const uint8_t*>(a.q);
  p.out = a.out;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.dev_status = a.dev_status;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.ws_info = reinterpret_cast<int4*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(ws + w.ml);
  p.ws_acc = reinterpret_cast<float*>(ws + w.acc);
  p.num_q_heads = a.num_q_heads;
  p.group = group;
  p.batch = rows;
  p.max_pages = a.max_pages;
  p.num_groups = a.batch;
  p.num_ctas = ctas;
  p.q_dtype = a.q_dtype;
  p.out_dtype = a.out_dtype;
  p.two_terms = a.out_dtype == PKV_F32;
  p.scale = a.sm_scale * 1.4426950408889634f;
  p.draft_lens = a.draft_lens;
  p.tree_mask = reinterpret_cast<const uint64_t*>(a.tree_mask);
  p.drafts = a.drafts;
  p.mask_words = (a.drafts + 63) / 64;
  p.mask_stride = a.mask_shared ? 0 : (long long)a.drafts * p.mask_words;
  p.pairs = pairs;
  p.rec_rows = (a.drafts * group + 31) / 32 * 32;
  // Row tiles that end between two drafts are copied as boxes; the others are gathered. (24 x ~6K, 64 drafts of 4 heads:
  // a segment's 256 rows by one warp took 8 us, which nothing hides.)
  p.q_box = kTile % group != 0 ? 0 : std::min(a.drafts, kTile / group);
  if (p.q_box && !query_map(a.q, (uint64_t)rows, a.num_q_heads, group, D, p.q_box, bf, p.tmap_q)) return PKV_ERR_CUDA;
  void* args[] = {&p};
  if (launch_pdl(fn, dim3(ctas), dim3(threads), smem, a.stream, args) != cudaSuccess) return PKV_ERR_CUDA;
  const long long items = (long long)a.batch * c->num_kv_heads * (p.rec_rows / 32) * (D / 16);
  // Where the warps are few, a block's four share an item's records, which come from memory one after the other. (Four and
  // one, with 1024 items: 8 x ~3K with 16 drafts of 4 heads 30.8 and 34.5 us, 4 x ~27K with 13 drafts of 32 kv heads 265.6 and 268.9. With
  // many more they only wait for one another: 12288, 24 x ~6K with 64 drafts, 162.0 and 151.8; 24576, 48 x ~770 with 64, 117.7 and
  // 96.5. In between they are within 2 us: 1536 39.9 and 41.4, 2048 34.9 and 37.0, 4096 50.4 and 48.4.)
  const int wpw = items < 8ll * dev.sms ? 4 : 1, per = 4 / wpw;
  const void* merge = D == 64 ? tree_merge<64>(wpw) : tree_merge<128>(wpw);
  return launch_pdl(merge, dim3((unsigned)((items + per - 1) / per)), dim3(kMergeThreads), 0, a.stream, args) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // namespace pkv
