// keep_tokens: what verifying drafts leaves. The tokens of one path of a sequence's tree, somewhere among
// its drafts, move to the places right behind the tokens that were there before:
//   token first + keep[j] -> token first + j,  keep strictly ascending.
// With keep[j] >= j no token is overwritten before it is read, so long as a run of tokens is
// read as a whole before it is written: a block does that for one kv head, K, V and scales, as
// many tokens at a time as its threads hold. Boxes of the pages from the last old token's on are made
// anew by the same block, from the places where the tokens still are.
//
// What bounds it: latency, a few KB a row: lists, block table, rows and stores follow one another, and nothing
// else does (128 rows of 8 heads with boxes: 5.6 us; with the boxes read back behind the stores 9.4).
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kKeepThreads = 256;
constexpr int kHeld = 4;          // 16-byte pieces that a thread holds
constexpr int kKeepTokens = 256;  // at most, one a thread

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

// Boxes: none, a page's by a warp (pages of up to 32 tokens), or by the block.
enum KeepBoxes { kNoBoxes = 0, kByWarp = 1, kByBlock = 2 };

// grid (kv head and row). 256 threads. Seven blocks an SM with boxes by warps: 128 rows of 8 heads are then one wave
// (10.5 us as the compiler likes it, four an SM 7.6, six 6.4, seven 5.6).
template <int D, int KV, int BOXES>
__global__ void __launch_bounds__(kKeepThreads, BOXES == kNoBoxes ? 8 : BOXES == kByWarp ? 7 : 4) keep_tokens_kernel(const KeepParams p) {
  constexpr bool QUANT = KV == KV_I8T || KV == KV_U4T, BLOCK = BOXES == kByBlock;
  constexpr int ROW = KV == KV_U4T ? D / 2 : QUANT ? D : 2 * D;
  constexpr int PIECES = 2 * (ROW / 16) + QUANT;             // of a token: K, V, scales
  constexpr int RUN = kKeepThreads * kHeld / PIECES;         // tokens that the block holds
  __shared__ int from[kKeepTokens], to[kKeepTokens];         // pool rows (of the tokens as they are; -1: it stays)
  __shared__ float box[BLOCK ? 2 : 1][BLOCK ? kKeepThreads / 32 : 1][2][D];
  pdl_wait();
  pdl_launch_dependents();
  const pkv_cache& c = p.cache;
  const int H = c.num_kv_heads, ps = c.page_size, b = blockIdx.x / H, g = blockIdx.x - b * H;
  const int32_t* table = p.block_table + (size_t)b * p.max_pages;
  const long long cap = (long long)p.max_pages * ps;
  const int j = threadIdx.x;
  const int32_t* keep = p.keep + (size_t)b * p.max_keep;
  // (all of the lists at once: the thread's place, and the one before)
  const int first = p.first[b], n = p.keep_lens ? p.keep_lens[b] : p.max_keep;
  const int k = j < p.max_keep ? keep[j] : 0, k0 = j > 0 && j < p.max_keep ? keep[j - 1] : -1;
  // the whole list before anything moves: ascending from 0 on, and within the table
  bool wrong = first < 0 || n < 0 || n > p.max_keep || (long long)first + n > cap;
  if (!wrong && j < n) wrong = k <= k0 || (long long)first + k >= cap;
  if (__syncthreads_or(wrong)) {
    if (j == 0) flag_status(p.dev_status, PKV_DEV_BAD_POSITION);
    return;
  }
  auto page_of = [&](int lp) {
    const int page = table[lp];
    return page >= 0 && page < c.num_pages ? page : -1;
  };
  // (the host keeps pool rows below 2^31)
  if (j < n) {
    const int d = first + j, s = first + k;
    const int dp = page_of(d / ps), sp = k == j ? dp : page_of(s / ps);
    const int here = dp < 0 ? -1 : (dp * H + g) * ps + d % ps;
    if (dp < 0 || sp < 0) flag_status(p.dev_status, PKV_DEV_BAD_PAGE);
    const bool moves = k != j && dp >= 0 && sp >= 0;
    from[j] = moves ? (sp * H + g) * ps + s % ps : here;
    to[j] = moves ? here : -1;
  }
  __syncthreads();
  uint8_t* const kp = static_cast<uint8_t*>(c.k_pages);
  uint8_t* const vp = static_cast<uint8_t*>(c.v_pages);
  auto piece = [&](int row, int i) -> uint4* {
    uint8_t* at = i < ROW / 16 ? kp + (size_t)row * ROW + i * 16
                  : i < 2 * (ROW / 16) ? vp + (size_t)row * ROW + (i - ROW / 16) * 16
                                       : reinterpret_cast<uint8_t*>(c.kv_sz + (size_t)row * 4);
    return reinterpret_cast<uint4*>(at);
  };
  uint4 held[kHeld];
  auto load = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int x = threadIdx.x + i * kKeepThreads, t = j0 + x / PIECES;
      if (t < min(n, j0 + RUN) && to[t] >= 0) held[i] = *piece(from[t], x % PIECES);
    }
  };
  load(0);   // on their way while the boxes are made
  if constexpr (BOXES != kNoBoxes) {
    // sixteen lanes a row: a warp, or the block, takes as many rows a pass as it has lanes for
    constexpr int C = D / 16, ROWS = BLOCK ? kKeepThreads / 16 : 2;
    const int part = threadIdx.x & 15, warp = threadIdx.x >> 5, slot = (int)(threadIdx.x >> 4) & (ROWS - 1);
    const int end = first + n;
    int turn = 0;
    for (int lp = max(0, first - 1) / ps + (BLOCK ? 0 : warp); lp * (long long)ps < end; lp += BLOCK ? 1 : kKeepThreads / 32) {
      const int page = page_of(lp);   // (the same for the whole warp, or block)
      if (page < 0) {
        if ((threadIdx.x & 31) == 0) flag_status(p.dev_status, PKV_DEV_BAD_PAGE);
        continue;
      }
      const int tokens = min(ps, end - lp * ps), row0 = (page * H + g) * ps, old = first - lp * ps;   // the first `old` of them
      float mn[C], mx[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        mn[i] = INFINITY;
        mx[i] = -INFINITY;
      }
      constexpr int AHEAD = BLOCK ? 4 : 2;
#pragma unroll AHEAD
      for (int t = slot; t < tokens; t += ROWS) {
        float x[C];
        const size_t row = t < old ? row0 + t : from[t - old];
        const float2 sz = QUANT ? *reinterpret_cast<const float2*>(c.kv_sz + row * 4) : make_float2(0.f, 0.f);
        key_channels<C, KV>(kp + row * ROW + part * (ROW / 16), sz, x);
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
      }
      float* meta = c.page_meta + ((size_t)page * H + g) * 2 * D;
      if constexpr (!BLOCK) {
        if (slot == 0) {
#pragma unroll
          for (int i = 0; i < C; i += 4) {
            *reinterpret_cast<float4*>(meta + part * C + i) = make_float4(mn[i], mn[i + 1], mn[i + 2], mn[i + 3]);
            *reinterpret_cast<float4*>(meta + D + part * C + i) = make_float4(mx[i], mx[i + 1], mx[i + 2], mx[i + 3]);
          }
        }
      } else {
        if ((slot & 1) == 0) {
#pragma unroll
          for (int i = 0; i < C; ++i) {
            box[turn][warp][0][part * C + i] = mn[i];
            box[turn][warp][1][part * C + i] = mx[i];
          }
        }
        __syncthreads();   // (two buffers: the one of two pages ago is read before this)
        if ((int)threadIdx.x < 2 * D) {
          const int r = threadIdx.x / D, ch = threadIdx.x % D;
          float v = box[turn][0][r][ch];
#pragma unroll
          for (int w = 1; w < kKeepThreads / 32; ++w) v = r ? fmaxf(v, box[turn][w][1][ch]) : fminf(v, box[turn][w][0][ch]);
          meta[r * D + ch] = v;
        }
        turn ^= 1;
      }
    }
  }
  for (int j0 = 0; j0 < n; j0 += RUN) {
    if (j0 > 0) load(j0);
    __syncthreads();   // every token of the run, and every one that a box needs, is read
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int x = threadIdx.x + i * kKeepThreads, t = j0 + x / PIECES;
      if (t < min(n, j0 + RUN) && to[t] >= 0) *piece(to[t], x % PIECES) = held[i];
    }
  }
}

}  // namespace

pkv_status launch_keep(const KeepParams& p, cudaStream_t st) {
  const pkv_cache& c = p.cache;
  const int kv = c.kv_dtype == PKV_F16 ? KV_F16 : c.kv_dtype == PKV_BF16 ? KV_BF16 : c.kv_dtype == PKV_U4 ? KV_U4T : KV_I8T;
  const void* fn = nullptr;
  const int boxes = !c.page_meta ? kNoBoxes : c.page_size > 32 ? kByBlock : kByWarp;
#define PKV_KEEP(d, k)                                                                                     \
  if (c.head_dim == d && kv == k)                                                                          \
    fn = boxes == kNoBoxes  ? reinterpret_cast<const void*>(&keep_tokens_kernel<d, k, kNoBoxes>)           \
         : boxes == kByWarp ? reinterpret_cast<const void*>(&keep_tokens_kernel<d, k, kByWarp>)            \
                            : reinterpret_cast<const void*>(&keep_tokens_kernel<d, k, kByBlock>);
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
