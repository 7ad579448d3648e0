// Rotary positions on the way into the cache: new keys are rotated and appended, new values
// appended, and the queries of the same tokens rotated, in one launch.
//
// The channels of a head's first rot_dim are paired, (i, i + rot_dim / 2) or (2 i, 2 i + 1), and pair
// i of a token at position m turned by the angle m w_i:
//   y1 = fl(fl(x1 c) - fl(x2 s)),  y2 = fl(fl(x2 c) + fl(x1 s)),  c, s = table[m][i], table[m][rot_dim / 2 + i],
// each step one fp32 rounding (no fused multiply-add), so that the values, and the codes that the
// quantisers make of them, are the same as any other IEEE implementation's. The table holds
// cosines and sines of angles worked out in 64 bits: at position 100000 an fp32 angle is off by 0.004.
//
// What bounds it: bytes; for a few tokens the latency of what follows one another, the positions,
// the table's row and the block table's entry, the stores. A token's 16 cosines and sines stay in
// registers for all the heads of a task, so the table is read once for them, and four heads' loads are in
// flight before the position is known.
//
// Measured (32 + 2 x 8 heads of 128, bf16): 4 x 8192 tokens 124 us, 6.6 TB/s, 0.99 of the copy rate; 4 tokens 2.1 us,
// 61 x 11 tokens (28 + 2 x 4 heads of 64) 3.1 us. Into per-token INT8 179, 3.2, 6.1 us, 4-bit 175, 3.2, 6.1: the quantisers'
// arithmetic; per-group INT8 301, 4.9, 8.0: every group in 32 bits, each key read twice and the table for every head.
// Boxes are one more launch, which reads the keys back: 2.5 to 3 us, 9 to 11 on 4 x 8192.
#include <cmath>

#include "pkv_internal.h"
#include "quant.cuh"

namespace pkv {

namespace {

constexpr int kRotaryThreads = 128;
constexpr int kAhead = 4;   // heads whose loads are in flight together

template <bool BF>
__device__ __forceinline__ void widen8(uint4 w, float* x) {
  const float4 a = widen4_t<BF>(make_uint2(w.x, w.y)), b = widen4_t<BF>(make_uint2(w.z, w.w));
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <bool BF>
__device__ __forceinline__ uint4 narrow8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    else
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A task: 32 / (D / 16) tokens and a run of their heads (queries', keys', values', in this order); a
// warp each. D / 16 lanes have a token, each 16 channels: both members of eight pairs.
template <int D, int KV, bool BF, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads) rotary_append_kernel(const RotaryParams p) {
  constexpr int LANES = D / 16, TOKENS = 32 / LANES;
  constexpr bool QUANT = KV == KV_I8T || KV == KV_U4T;
  constexpr bool SAME = !QUANT && (KV == KV_BF16) == BF;   // rows are stored as they come
  pdl_wait();
  pdl_launch_dependents();
  const AppendParams& a = p.a;
  const int lane = threadIdx.x & 31, j = lane % LANES;
  const int task = blockIdx.x * (kRotaryThreads / 32) + (threadIdx.x >> 5);
  if (task >= p.tasks) return;   // a whole warp
  const int run = task / p.token_tasks, n = (task - run * p.token_tasks) * TOKENS + lane / LANES;
  const int Hq = p.num_q_heads, H = a.num_kv_heads;
  const int h0 = run * p.heads_per_task, h1 = min(Hq + 2 * H, h0 + p.heads_per_task);
  const bool there = n < a.batch * a.t_new;
  const int nn = there ? n : 0, b = nn / a.t_new, t = nn - b * a.t_new;
  // the lane's two pieces of eight channels, and whether they turn
  const int half = a.rot_dim / 16;
  const bool turns = j < half;
  const int pa = INTERLEAVED ? 2 * j : turns ? j : 2 * j, pb = INTERLEAVED || !turns ? 2 * j + 1 : j + half;
  auto source = [&](int h) {
    const uint16_t* s = h < Hq       ? static_cast<const uint16_t*>(p.q) + nn * p.q_stride + h * D
                        : h < Hq + H ? static_cast<const uint16_t*>(a.k_new) + nn * a.k_stride + (h - Hq) * D
                                     : static_cast<const uint16_t*>(a.v_new) + nn * a.v_stride + (h - Hq - H) * D;
    return reinterpret_cast<const uint4*>(s);
  };
  uint4 raw[kAhead][2];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint4* s = source(min(h + i, h1 - 1));
      raw[i][0] = s[pa];
      raw[i][1] = s[pb];
    }
  };
  load(h0);   // before the position is known

  int pos = a.positions[b];
  const int count = a.new_lens ? a.new_lens[b] : a.t_new;
  const int at = a.rotary_positions ? a.rotary_positions[nn] : 0;
  bool on = there && t < count;
  if (count > a.t_new || count < 0 || pos < 0 || (long long)pos + count > (long long)a.max_pages * a.page_size) {
    if (there && j == 0) flag_status(a.dev_status, PKV_DEV_BAD_POSITION);
    on = false;
  }
  pos = on ? pos + t : 0;
  int m = a.rotary_positions ? at : pos;
  if (m < 0 || m >= a.table_positions) {
    if (on && j == 0) flag_status(a.dev_status, PKV_DEV_BAD_POSITION);
    m = m < 0 ? 0 : a.table_positions - 1;
  }
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    if (turns) {
      const float* row = a.cos_sin + (size_t)m * a.rot_dim + 8 * j + i;
      const float4 x = *reinterpret_cast<const float4*>(row), y = *reinterpret_cast<const float4*>(row + a.rot_dim / 2);
      c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
      s[i] = y.x; s[i + 1] = y.y; s[i + 2] = y.z; s[i + 3] = y.w;
    }
  }
  size_t place = 0;   // row of kv head 0 in the pools
  bool stored = on && h1 > Hq;
  if (stored) {
    const int page = a.block_table[(size_t)b * a.max_pages + (a.ps_shift >= 0 ? pos >> a.ps_shift : pos / a.page_size)];
    if (page < 0 || page >= a.num_pages) {
      if (j == 0) flag_status(a.dev_status, PKV_DEV_BAD_PAGE);
      stored = false;
    }
    place = (size_t)page * H * a.page_size + (a.ps_shift >= 0 ? pos & (a.page_size - 1) : pos % a.page_size);
  }

  // both pieces in 32 bits: a pair's members lie at i and 8 + i, or beside each other
  auto turn = [&](float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& u = x[INTERLEAVED ? 2 * i : i];
      float& v = x[INTERLEAVED ? 2 * i + 1 : i + 8];
      const float u1 = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(v, s[i]));
      v = __fadd_rn(__fmul_rn(v, c[i]), __fmul_rn(u, s[i]));
      u = u1;
    }
  };
  for (int hb = h0; hb < h1; hb += kAhead) {   // (the same heads for the whole warp)
    if (hb > h0) load(hb);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = hb + i;
      if (h >= h1) break;
      if (h < Hq) {
        uint4 w[2] = {raw[i][0], raw[i][1]};
        if (turns) {
          float x[16];
          widen8<BF>(w[0], x);
          widen8<BF>(w[1], x + 8);
          turn(x);
          w[0] = narrow8<BF>(x);
          w[1] = narrow8<BF>(x + 8);
        }
        if (on) {
          uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + ((size_t)nn * Hq + h) * D);
          out[pa] = w[0];
          out[pb] = w[1];
        }
        continue;
      }
      const bool isv = h >= Hq + H;
      const size_t row = place + (size_t)(h - Hq - (isv ? H : 0)) * a.page_size;
      uint8_t* pool = static_cast<uint8_t*>(isv ? a.v_pages : a.k_pages);
      float x[16];
      widen8<BF>(raw[i][0], x);
      widen8<BF>(raw[i][1], x + 8);
      if (!isv && turns) turn(x);
      if constexpr (QUANT) {
        float mn = x[0], mx = x[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) {
          mn = fminf(mn, x[e]);
          mx = fmaxf(mx, x[e]);
        }
#pragma unroll
        for (int off = LANES / 2; off > 0; off >>= 1) {
          mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        }
        const float sc = __fdiv_rn(__fsub_rn(mx, mn), KV == KV_U4T ? 15.f : 255.f), rs = quant_recip(sc);
        if (stored) {
          if constexpr (KV == KV_U4T) {
            uint32_t w[2];
            quant_nibbles<16>(x, sc, mn, rs, w);
            uint32_t* dst = reinterpret_cast<uint32_t*>(pool + row * (D / 2));
            dst[pa] = w[0];
            dst[pb] = w[1];
          } else {
            uint32_t w[4];
            quant_words<16>(x, sc, mn, rs, w);
            uint2* dst = reinterpret_cast<uint2*>(pool + row * D);
            dst[pa] = make_uint2(w[0], w[1]);
            dst[pb] = make_uint2(w[2], w[3]);
          }
          if (j == 0) *reinterpret_cast<float2*>(a.kv_sz + row * 4 + (isv ? 2 : 0)) = make_float2(sc, mn);
        }
      } else if (stored) {
        const bool as_is = SAME && (isv || !turns);
        uint4* dst = reinterpret_cast<uint4*>(pool + row * (2 * D));
        dst[pa] = as_is ? raw[i][0] : narrow8<KV == KV_BF16>(x);
        dst[pb] = as_is ? raw[i][1] : narrow8<KV == KV_BF16>(x + 8);
      }
    }
  }
}

// Cosines and sines of m w_i in 64 bits. grid (rows, up to 65535 at a time), a thread a pair.
struct TableParams {
  float* cos_sin;
  int positions, half;
  double scale, w[64];
};
__global__ void __launch_bounds__(64) rotary_table_kernel(const TableParams p) {
  pdl_wait();
  pdl_launch_dependents();
  if ((int)threadIdx.x >= p.half) return;
  for (int m = blockIdx.x; m < p.positions; m += gridDim.x) {
    double s, c;
    sincos(m * p.w[threadIdx.x], &s, &c);
    float* row = p.cos_sin + (size_t)m * 2 * p.half + threadIdx.x;
    row[0] = (float)(c * p.scale);
    row[p.half] = (float)(s * p.scale);
  }
}

template <int D, bool INTERLEAVED>
const void* kernel_of(int kv, bool bf) {
#define PKV_ROT(k, s) \
  if (kv == k && bf == s) return reinterpret_cast<const void*>(&rotary_append_kernel<D, k, s, INTERLEAVED>);
  PKV_ROT(KV_F16, false) PKV_ROT(KV_F16, true) PKV_ROT(KV_BF16, false) PKV_ROT(KV_BF16, true)
  PKV_ROT(KV_I8T, false) PKV_ROT(KV_I8T, true) PKV_ROT(KV_U4T, false) PKV_ROT(KV_U4T, true)
#undef PKV_ROT
  return nullptr;
}

}  // namespace

pkv_status launch_rotary_append(RotaryParams p, cudaStream_t st) {
  const AppendParams& a = p.a;
  const bool groups = a.quant == PKV_QUANT_PER_GROUP64;
  const int kv = groups || a.kv_dtype == PKV_F16 ? KV_F16 : a.kv_dtype == PKV_BF16 ? KV_BF16
                 : a.kv_dtype == PKV_U4 ? KV_U4T : KV_I8T;
  const bool bf = a.src_dtype == PKV_BF16;
  RotaryParams r = p;
  if (groups) r.a.num_kv_heads = 0;   // their keys and values go group by group, below
  const int heads = p.num_q_heads + 2 * r.a.num_kv_heads;
  cudaError_t e = cudaSuccess;
  if (heads > 0) {
    const int D = a.head_dim, per = 512 / D;   // tokens of a task
    r.token_tasks = (a.batch * a.t_new + per - 1) / per;
    // One head a task while the device has room for more warps, then up to 16 of them.
    const long long all = (long long)heads * r.token_tasks;
    r.heads_per_task = (int)(all / 4096 < 1 ? 1 : all / 4096 > 16 ? 16 : all / 4096);
    const long long tasks = (long long)r.token_tasks * ((heads + r.heads_per_task - 1) / r.heads_per_task);
    if (tasks > INT32_MAX / 2) return PKV_ERR_UNSUPPORTED;
    r.tasks = (int)tasks;
    const void* fn = D == 128 ? (a.interleaved ? kernel_of<128, true>(kv, bf) : kernel_of<128, false>(kv, bf))
                              : (a.interleaved ? kernel_of<64, true>(kv, bf) : kernel_of<64, false>(kv, bf));
    void* args[] = {&r};
    const int warps = kRotaryThreads / 32;
    e = launch_pdl(fn, dim3((r.tasks + warps - 1) / warps), dim3(kRotaryThreads), 0, st, args);
  }
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  if (groups) {
    const pkv_status s = launch_append_rotated_groups(a, st);
    if (s != PKV_OK) return s;
  }
  return a.page_meta ? launch_append_boxes(a, st) : PKV_OK;
}

pkv_status launch_rotary_table(float* cos_sin, int positions, int rot_dim, const double* inv_freq, double scale,
                               cudaStream_t st) {
  TableParams p = {};
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.half = rot_dim / 2;
  p.scale = scale;
  for (int i = 0; i < p.half; ++i) p.w[i] = inv_freq[i];
  void* args[] = {&p};
  const int grid = positions < 65535 ? positions : 65535;
  return launch_pdl(reinterpret_cast<const void*>(&rotary_table_kernel), dim3(grid), dim3(64), 0, st, args) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

// Frequencies w_i = base^(-2 i / rot_dim), and what long contexts make of them.
pkv_status rotary_frequencies(int rot_dim, double base, int scaling, double factor, double low, double high,
                              double original, double* inv_freq, double* scale) {
  constexpr double kTwoPi = 6.283185307179586476925;
  if (rot_dim <= 0 || !inv_freq || !scale || !(base > 1.0) || !std::isfinite(base)) return PKV_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0 || rot_dim > 128) return PKV_ERR_UNSUPPORTED;
  if (scaling < PKV_ROTARY_PLAIN || scaling > PKV_ROTARY_RAMP) return PKV_ERR_INVALID_ARG;
  if (scaling != PKV_ROTARY_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return PKV_ERR_INVALID_ARG;
  const bool banded = scaling == PKV_ROTARY_BANDS, ramp = scaling == PKV_ROTARY_RAMP;
  if ((banded || ramp) && !(low > 0.0 && high > low && std::isfinite(high) && original > 0.0 && std::isfinite(original)))
    return PKV_ERR_INVALID_ARG;
  if (scaling == PKV_ROTARY_BASE) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  // ramp: the (whole) pair indexes whose waves turn `high` and `low` times in the original length
  double first = 0.0, last = 0.0;
  if (ramp) {
    auto index = [&](double turns) { return rot_dim * std::log(original / (turns * kTwoPi)) / (2.0 * std::log(base)); };
    first = std::fmax(std::floor(index(high)), 0.0);
    last = std::fmin(std::ceil(index(low)), rot_dim - 1.0);
    if (last <= first) last = first + 0.001;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double w = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == PKV_ROTARY_LINEAR) {
      inv_freq[i] = w / factor;
    } else if (banded || ramp) {
      // how much of the frequency is kept: by the turns in the original length, or by index
      double keep = banded ? (original * w / kTwoPi - low) / (high - low) : 1.0 - (i - first) / (last - first);
      keep = std::fmin(std::fmax(keep, 0.0), 1.0);
      inv_freq[i] = keep * w + (1.0 - keep) * (w / factor);
    } else {
      inv_freq[i] = w;
    }
  }
  *scale = ramp ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return PKV_OK;
}

}  // namespace pkv
