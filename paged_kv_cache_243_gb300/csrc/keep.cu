// keep_tokens: what verifying drafts leaves. The tokens of one path of a sequence's tree, somewhere among
// its drafts, move to the places right behind the tokens that were there before:
//   token first + keep[j] -> token first + j,  keep strictly ascending.
// With keep[j] >= j no token is overwritten before it is read, so long as a run of tokens is
// read as a whole before it is written: a block does that for one kv head, K, V and scales, as
// many tokens at a time as its threads hold. Boxes of the pages from the last old token's on are made
// anew by the same block.
//
// What bounds it: latency (lists, block table, rows, stores), a few KB a row. One launch: a second
// one for the boxes would cost as much again.
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kKeepThreads = 256;
constexpr int kHeld = 4;          // 16-byte pieces that a thread holds
constexpr int kKeepTokens = 128;  // tokens whose places are looked up at a time

// Channels [0, C) of the lane's block of a stored key row, as attention and the boxes see them:
// fl32(fl32(u s) + z) for codes (the packed forms of these could be contracted; scalar ones are not).
template <int C, int KV>
__device__ __forceinline__ void key_channels(const uint8_t* row, float2 sz, float (&x)[C]) {
  if constexpr (KV == KV_I8T) {
    uint32_t w[C / 4];
#pragma unroll
    for (int i = 0; i < C / 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(row)[i];
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = __fadd_rn(__fmul_rn(u8_as_float(w[c / 4], c % 4), sz.x), sz.y);
  } else if constexpr (KV == KV_U4T) {
    const uint32_t w = C == 8 ? *reinterpret_cast<const uint32_t*>(row) : *reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = __fadd_rn(__fmul_rn((float)(w >> (4 * c) & 15), sz.x), sz.y);
  } else {
#pragma unroll
    for (int c = 0; c < C; c += 2) unpack2<KV>(reinterpret_cast<const uint32_t*>(row)[c / 2], x[c], x[c + 1]);
  }
}

// grid (kv head and row). 256 threads.
template <int D, int KV>
__global__ void __launch_bounds__(kKeepThreads) keep_tokens_kernel(const KeepParams p) {
  constexpr bool QUANT = KV == KV_I8T || KV == KV_U4T;
  constexpr int ROW = KV == KV_U4T ? D / 2 : QUANT ? D : 2 * D;
  constexpr int PIECES = 2 * (ROW / 16) + QUANT;   // of a token: K, V, scales
  constexpr int RUN = kKeepThreads * kHeld / PIECES < kKeepTokens ? kKeepThreads * kHeld / PIECES : kKeepTokens;
  __shared__ long long from[kKeepTokens], to[kKeepTokens];   // pool rows, -1: none
  __shared__ float box[kKeepThreads / 32][2][D];
  pdl_wait();
  pdl_launch_dependents();
  const pkv_cache& c = p.cache;
  const int H = c.num_kv_heads, ps = c.page_size, b = blockIdx.x / H, g = blockIdx.x - b * H;
  const int32_t* table = p.block_table + (size_t)b * p.max_pages;
  const long long cap = (long long)p.max_pages * ps;
  const int first = p.first[b], n = p.keep_lens ? p.keep_lens[b] : p.max_keep;
  const int32_t* keep = p.keep + (size_t)b * p.max_keep;
  // the whole list before anything moves: ascending from 0 on, and within the table
  bool wrong = first < 0 || n < 0 || n > p.max_keep || (long long)first + n > cap;
  if (!wrong)
    for (int j = threadIdx.x; j < n; j += kKeepThreads) {
      const int k = keep[j];
      wrong |= k <= (j ? keep[j - 1] : -1) || (long long)first + k >= cap;
    }
  if (__syncthreads_or(wrong)) {
    if (threadIdx.x == 0) flag_status(p.dev_status, PKV_DEV_BAD_POSITION);
    return;
  }
  auto pool_row = [&](int tok) -> long long {
    const int page = table[tok / ps];
    if (page < 0 || page >= c.num_pages) {
      flag_status(p.dev_status, PKV_DEV_BAD_PAGE);
      return -1;
    }
    return ((long long)page * H + g) * ps + tok % ps;
  };
  uint8_t* const kp = static_cast<uint8_t*>(c.k_pages);
  uint8_t* const vp = static_cast<uint8_t*>(c.v_pages);
  auto piece = [&](long long row, int i) -> uint4* {
    uint8_t* at = i < ROW / 16 ? kp + row * ROW + i * 16
                  : i < 2 * (ROW / 16) ? vp + row * ROW + (i - ROW / 16) * 16
                                       : reinterpret_cast<uint8_t*>(c.kv_sz + row * 4);
    return reinterpret_cast<uint4*>(at);
  };
  for (int j0 = 0; j0 < n; j0 += RUN) {
    const int m = min(RUN, n - j0);
    if ((int)threadIdx.x < m) {
      const int j = j0 + threadIdx.x, k = keep[j];
      const long long d = k == j ? -1 : pool_row(first + j), s = k == j ? -1 : pool_row(first + k);
      from[threadIdx.x] = s;
      to[threadIdx.x] = s < 0 ? -1 : d;
    }
    __syncthreads();
    uint4 held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int x = threadIdx.x + i * kKeepThreads, j = x / PIECES;
      if (j < m && to[j] >= 0) held[i] = *piece(from[j], x - j * PIECES);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int x = threadIdx.x + i * kKeepThreads, j = x / PIECES;
      if (j < m && to[j] >= 0) *piece(to[j], x - j * PIECES) = held[i];
    }
    __syncthreads();
  }
  if (!c.page_meta) return;
  // sixteen lanes a row, a pass over sixteen rows at a time
  constexpr int C = D / 16;
  const int part = threadIdx.x & 15, slot = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int end = first + n;
  for (int lp = max(0, first - 1) / ps; lp * (long long)ps < end; ++lp) {
    const int page = table[lp];   // (the same for the whole block)
    if (page < 0 || page >= c.num_pages) {
      if (threadIdx.x == 0) flag_status(p.dev_status, PKV_DEV_BAD_PAGE);
      continue;
    }
    const int tokens = min(ps, end - lp * ps);
    const size_t row0 = ((size_t)page * H + g) * ps;
    float mn[C], mx[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      mn[i] = INFINITY;
      mx[i] = -INFINITY;
    }
#pragma unroll 4
    for (int t = slot; t < tokens; t += kKeepThreads / 16) {
      float x[C];
      const float2 sz = QUANT ? *reinterpret_cast<const float2*>(c.kv_sz + (row0 + t) * 4) : make_float2(0.f, 0.f);
      key_channels<C, KV>(kp + (row0 + t) * ROW + part * (ROW / 16), sz, x);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        mn[i] = fminf(mn[i], x[i]);
        mx[i] = fmaxf(mx[i], x[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      mn[i] = fminf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], 16));
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 16));
      if ((slot & 1) == 0) {
        box[warp][0][part * C + i] = mn[i];
        box[warp][1][part * C + i] = mx[i];
      }
    }
    __syncthreads();
    if ((int)threadIdx.x < 2 * D) {
      const int r = threadIdx.x / D, ch = threadIdx.x % D;
      float v = box[0][r][ch];
#pragma unroll
      for (int w = 1; w < kKeepThreads / 32; ++w) v = r ? fmaxf(v, box[w][1][ch]) : fminf(v, box[w][0][ch]);
      c.page_meta[(((size_t)page * H + g) * 2 + r) * D + ch] = v;
    }
    __syncthreads();
  }
}

}  // namespace

pkv_status launch_keep(const KeepParams& p, cudaStream_t st) {
  const pkv_cache& c = p.cache;
  const int kv = c.kv_dtype == PKV_F16 ? KV_F16 : c.kv_dtype == PKV_BF16 ? KV_BF16 : c.kv_dtype == PKV_U4 ? KV_U4T : KV_I8T;
  const void* fn = nullptr;
#define PKV_KEEP(d, k) \
  if (c.head_dim == d && kv == k) fn = reinterpret_cast<const void*>(&keep_tokens_kernel<d, k>);
  PKV_KEEP(64, KV_F16) PKV_KEEP(64, KV_BF16) PKV_KEEP(64, KV_I8T) PKV_KEEP(64, KV_U4T)
  PKV_KEEP(128, KV_F16) PKV_KEEP(128, KV_BF16) PKV_KEEP(128, KV_I8T) PKV_KEEP(128, KV_U4T)
#undef PKV_KEEP
  KeepParams q = p;
  void* args[] = {&q};
  return launch_pdl(fn, dim3((unsigned)(p.batch * c.num_kv_heads)), dim3(kKeepThreads), 0, st, args) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // namespace pkv
