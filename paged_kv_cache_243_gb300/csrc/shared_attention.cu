// Decode attention over shared prefixes, in its plainest form: one warp per
// query row walks the row's tokens through the block table, 32 lanes over the
// channels, with a running maximum and sum.
#include "pkv_internal.h"
#include "quant.cuh"

namespace pkv {
namespace {

struct SharedParams {
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const float* kv_sz;
  const void* q;
  void* out;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* prefix_group;
  const int32_t* prefix_lens;
  int32_t* dev_status;
  int num_pages, page_size, num_kv_heads, num_q_heads, head_dim, max_pages, num_groups;
  int kind, q_dtype, out_dtype;
  float scale;
};

__device__ float restored(const SharedParams& p, const uint8_t* pool, int which, size_t row, size_t szrow, int i) {
  const int D = p.head_dim;
  if (p.kind == KV_F16) return __half2float(reinterpret_cast<const __half*>(pool)[row * D + i]);
  if (p.kind == KV_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(pool)[row * D + i]);
  const float s = p.kv_sz[szrow * 4 + which], z = p.kv_sz[szrow * 4 + which + 1];
  const uint32_t u = p.kind == KV_U4T ? pool[(row * D + i) / 2] >> (4 * (i & 1)) & 15u : pool[row * D + i];
  return fmaf((float)u, s, z);
}

__global__ void shared_plain_kernel(const SharedParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, h = blockIdx.x, lane = threadIdx.x, D = p.head_dim;
  const int kvh = h / (p.num_q_heads / p.num_kv_heads);
  const long long cap = (long long)p.max_pages * p.page_size;
  int L = p.seq_lens[b];
  if (L < 0 || L > cap) {
    if (lane == 0 && h == 0) flag_status(p.dev_status, PKV_DEV_BAD_POSITION);
    L = L < 0 ? 0 : (int)cap;
  }
  const int g = p.prefix_group[b];
  if (h == 0 && lane == 0 && (g < -1 || g >= p.num_groups || (g >= 0 && p.prefix_lens[g] < 0)))
    flag_status(p.dev_status, PKV_DEV_BAD_GROUP);
  const size_t qo = ((size_t)b * p.num_q_heads + h) * D;
  float m = -INFINITY, l = 0.f, acc[4] = {}, q[4] = {};
  for (int j = 0; j * 32 < D; ++j) q[j] = load_q_elem(p.q, p.q_dtype, qo + j * 32 + lane) * p.scale;
  for (int t = 0; t < L; ++t) {
    const int page = p.block_table[(size_t)b * p.max_pages + t / p.page_size];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) flag_status(p.dev_status, PKV_DEV_BAD_PAGE);
      continue;
    }
    const size_t row = ((size_t)page * p.num_kv_heads + kvh) * p.page_size + t % p.page_size;
    const size_t szrow = p.kind == KV_I8G ? row / 64 : row;
    float s = 0.f;
    for (int j = 0; j * 32 < D; ++j) s = fmaf(q[j], restored(p, p.k_pages, 0, row, szrow, j * 32 + lane), s);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    const float mn = fmaxf(m, s), a = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - mn);
    l = fmaf(l, a, w);
    for (int j = 0; j * 32 < D; ++j)
      acc[j] = fmaf(acc[j], a, w * restored(p, p.v_pages, 2, row, szrow, j * 32 + lane));
    m = mn;
  }
  for (int j = 0; j * 32 < D; ++j)
    store_out_elem(p.out, p.out_dtype, qo + j * 32 + lane, l > 0.f ? acc[j] / l : 0.f);
}

}  // namespace

pkv_status shared_workspace_bytes(const pkv_cache*, int, int, int, size_t& bytes) {
  bytes = 256;
  return PKV_OK;
}

pkv_status launch_shared(const SharedArgs& a) {
  const pkv_cache* c = a.cache;
  if (!a.workspace || (reinterpret_cast<uintptr_t>(a.workspace) & 255u) || a.workspace_bytes < 256)
    return PKV_ERR_WORKSPACE;
  SharedParams p = {};
  p.k_pages = static_cast<const uint8_t*>(c->k_pages);
  p.v_pages = static_cast<const uint8_t*>(c->v_pages);
  p.kv_sz = c->kv_sz;
  p.q = a.q;
  p.out = a.out;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.prefix_group = a.prefix_group;
  p.prefix_lens = a.prefix_lens;
  p.dev_status = a.dev_status;
  p.num_pages = c->num_pages;
  p.page_size = c->page_size;
  p.num_kv_heads = c->num_kv_heads;
  p.num_q_heads = a.num_q_heads;
  p.head_dim = c->head_dim;
  p.max_pages = a.max_pages;
  p.num_groups = a.num_groups;
  p.kind = c->kv_dtype == PKV_F16 ? KV_F16 : c->kv_dtype == PKV_BF16 ? KV_BF16 : c->kv_dtype == PKV_U4 ? KV_U4T
           : c->quant == PKV_QUANT_PER_TOKEN ? KV_I8T : KV_I8G;
  p.q_dtype = a.q_dtype;
  p.out_dtype = a.out_dtype;
  p.scale = a.sm_scale * 1.4426950408889634f;
  void* args[] = {&p};
  return launch_pdl(reinterpret_cast<const void*>(&shared_plain_kernel), dim3(a.num_q_heads, a.batch), dim3(32), 0,
                    a.stream, args) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // namespace pkv
