// Decode attention over shared prefixes on the tensor cores (tcgen05).
//
// What it computes. For query head h of row b, out = softmax(sm q . K^T) V over
// tokens [0, len_b). The rows of a group have tokens [0, P) in common, so
//   state over [0, P):    all query heads of all the group's rows at once, as
//                         [rows x G] x d times d x P products, K/V read once
//   state over [P, len):  the G heads of one row
// and the two states merge like any split of a softmax: with m the running
// maximum (log2 domain), l the sum of 2^(s - m), a = sum 2^(s - m) v,
//   M = max m_i,  out = sum 2^(m_i - M) a_i / sum 2^(m_i - M) l_i.
// P is the group's prefix rounded down to 16 tokens (64 for per-group scales,
// whose open group depends on what follows); the rest is read with the row.
//
// Work decomposition. A segment is one of the products above for one kv head:
// up to 256 query rows over a token range. It is cut into tiles of 128 tokens; one
// visit is one tile for all of the segment's rows. Visits of all segments are
// laid end to end (prefixes first) and block c of N takes visits [c W / N,
// (c + 1) W / N): every SM streams the same number of K/V tiles whatever the
// lengths are. A block that covers part of a segment leaves a partial state; the
// second launch merges them.
//
// Inside a block (one per SM, TMEM fully used: two score tiles of 128 columns and two
// accumulators of d columns):
//   loader warp   TMA copies of K and V tiles, 16 tokens a box (a page may end every
//                 16), into a ring; block-table entries one visit ahead
//   MMA thread    S = Q K^T (both operands in shared memory, 128-byte swizzle), O += P V
//                 (P in TMEM, over the scores it was made from; V as stored, MN-major)
//   Q warp        gathers the rows' queries into the swizzled operand tile, a segment ahead
//   2 x 4 softmax warps, one per stream; thread = query row
// Two streams keep the tensor cores busy while the exponentials of the other are
// computed: with more than 128 rows each stream has its own 128 rows and
// both use every tile; otherwise the tiles alternate between the streams, which
// merge when the segment ends.
// The running maximum follows the true one only when that is over 2^8 above it:
// weights then stay below 2^8, and the accumulator in TMEM is rarely rescaled.
//
// INT8 and 4-bit caches: the codes enter the products as exact small integers, u - c
// with c the middle code, made by four converter warps from the staged bytes;
// scales and zero points are applied in fp32:
//   q . k = ks (q . (u - c)) + (kz + c ks) sum q
//   sum p v = sum (p vs) (u - c) + sum p (vz + c vs)
// p vs is divided by a power of two near the largest vs, so that it stays inside
// fp16's range; the accumulator is rescaled when a later tile's scales outgrow it.
#pragma once

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kTile = 128;        // tokens of a visit, query rows of a tile
constexpr int kHdrs = 8;          // visit headers kept (more than the visits the ring holds)
constexpr int kScaleSlots = 4;    // visits whose scales are kept for the softmax
constexpr int kQSums = 8;
constexpr int kMaxEntries = 12;   // ring entries: at most 2 (kHdrs - 2)

struct SharedParams {
  CUtensorMap tmap_k, tmap_v;   // 16-bit pools as [rows][d], boxes of 16 rows x 64 channels
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const float* kv_sz;
  const uint8_t* q;
  void* out;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* prefix_group;
  const int32_t* prefix_lens;
  int32_t* dev_status;
  // workspace: (m, l) and accumulators by record row, and each row's place in the plan
  float2* ws_ml;
  float* ws_acc;
  int4* ws_info;
  int num_pages, page_size, num_kv_heads, num_q_heads, group, batch, max_pages, num_groups;
  int num_ctas, entries, round_to, q_dtype, out_dtype, two_terms, rows_per_warp_group;
  float scale;   // sm_scale * log2(e)
};

template <int D, int KV, bool BF>
struct SharedGeom {
  static constexpr bool QUANT = KV == KV_I8T || KV == KV_I8G || KV == KV_U4T;
  static constexpr int HALVES = D / 64;
  static constexpr int OPERAND = HALVES * 16384;   // 128 rows x d 16-bit values, [half][row][128 bytes]
  static constexpr int ROW = KV == KV_U4T ? D / 2 : (QUANT ? D : 2 * D);
  static constexpr int ENTRY = QUANT ? kTile * ROW : OPERAND;
  static constexpr int RAW_SCALES = QUANT ? (KV == KV_I8G ? 128 : kTile * 16) : 0;
  static constexpr int SCALES = QUANT ? 4 * kTile * 4 : 0;   // ks, kz', vs, vz' of a visit
  static constexpr int THREADS = QUANT ? 512 : 384;
  static constexpr float CENTRE = KV == KV_U4T ? 8.f : 128.f;
};

// Shared memory by offset from a 1024-byte boundary.
struct SharedLayout {
  int q, kop, vop, ring, raw, scales, bars, hdr, ml, qsum, vmax, misc, lens, skip, bpre, gpre, gp, moff, members, rank;
  int total;
};
enum SharedBars {   // mbarriers, 8 bytes each
  kBarFull = 0, kBarEmpty = kMaxEntries, kBarHdr = 2 * kMaxEntries, kBarQFull = kBarHdr + kHdrs,
  kBarQEmpty = kBarQFull + 2, kBarS = kBarQEmpty + 2, kBarP = kBarS + 2, kBarO = kBarP + 2,
  kBarKop = kBarO + 2, kBarVop = kBarKop + 2, kBarPair = kBarVop + 2, kBarEnd = kBarPair + 4, kBarCount = kBarEnd + 1
};

template <class G>
__host__ __device__ inline SharedLayout shared_layout(int entries, int batch, int groups) {
  SharedLayout o;
  int at = 0;
  auto put = [&](int bytes) {
    const int r = at;
    at += (bytes + 127) / 128 * 128;
    return r;
  };
  o.q = put(2 * G::OPERAND);
  o.kop = put(G::QUANT ? G::OPERAND : 0);
  o.vop = put(G::QUANT ? G::OPERAND : 0);
  o.ring = put(entries * G::ENTRY);
  o.raw = put(entries / 2 * G::RAW_SCALES);
  o.scales = put(kScaleSlots * G::SCALES);
  o.bars = put(kBarCount * 8);
  o.hdr = put(kHdrs * 8);
  o.ml = put(2 * kTile * 16);
  o.qsum = put(G::QUANT ? kQSums * kTile * 4 : 0);
  o.vmax = put(G::QUANT ? kScaleSlots * 16 : 0);
  o.misc = put(40 * 4);
  o.lens = put(batch * 4);
  o.skip = put(batch * 4);
  o.bpre = put((batch + 1) * 4);
  o.gpre = put((groups + 1) * 4);
  o.gp = put(groups * 4);
  o.moff = put((groups + 1) * 4);
  o.members = put(batch * 2);
  o.rank = put(batch * 2);
  o.total = at;
  return o;
}

// Blocks' shares of W visits.
__device__ __forceinline__ int share_lo(long long c, long long W, long long N) { return (int)(c * W / N); }
// The block that holds visit x: the largest c with floor(c W / N) <= x.
__device__ __forceinline__ int share_of(long long x, long long W, long long N) {
  return (int)(((x + 1) * N + W - 1) / W - 1);
}

// ------------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle: start address, leading and
// stride byte offsets in 16-byte units, descriptor version 1.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 |
         2ull << 61;
}

// D[tmem] (+)= A[smem] B[smem], or A in TMEM.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// 32 columns of this warp's 32 TMEM lanes: lane i of the warp holds row i.
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (BF)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF>
__device__ __forceinline__ float low16(uint32_t w) {
  return BF ? bf16_lo(w) : f16_lo(w);
}
template <bool BF>
__device__ __forceinline__ float high16(uint32_t w) {
  return BF ? bf16_hi(w) : f16_hi(w);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// ---------------------------------------------------------------------- plan
struct SharedPlan {
  const int *lens, *skip, *bpre, *gpre, *gp, *moff;
  const uint16_t* members;
  int batch, groups, heads, group, W, Wp;   // Wp: visits of prefix segments
};

// The segment that visit x belongs to.
struct Seg {
  int begin, end;     // its visits inside the block's range
  int tile0, tiles;   // tile of visit `begin`, and tiles of the whole segment
  int first_tok, end_tok;
  int row, head;      // block-table row to read through, kv head
  int rows;           // query rows
  int q0;             // prefix: first query row within the group; suffix: 0
  int mem0;           // prefix: first member; suffix: -1
  int rec;            // record row of query row 0 (whole-segment region)
};

__device__ __forceinline__ int upper(const int* pre, int n, int x) {   // largest i with pre[i] <= x
  int a = 0, b = n;
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (pre[m] <= x) a = m;
    else b = m;
  }
  return a;
}

__device__ __forceinline__ Seg locate(const SharedPlan& p, int x, int hi) {
  Seg s;
  int rem;
  if (x < p.Wp) {
    const int g = upper(p.gpre, p.groups, x);
    const int T = (p.gp[g] + kTile - 1) / kTile;
    const int total = (p.moff[g + 1] - p.moff[g]) * p.group;
    const int pairs = (total + 2 * kTile - 1) / (2 * kTile);
    rem = x - p.gpre[g];
    const int hp = rem / T;
    rem -= hp * T;
    s.head = hp / pairs;
    s.q0 = (hp - s.head * pairs) * 2 * kTile;
    s.rows = min(2 * kTile, total - s.q0);
    s.tiles = T;
    s.first_tok = 0;
    s.end_tok = p.gp[g];
    s.mem0 = p.moff[g];
    s.row = p.members[s.mem0];
    s.rec = s.head * p.batch * p.group + s.mem0 * p.group + s.q0;
  } else {
    const int b = upper(p.bpre, p.batch, x);
    s.first_tok = p.skip[b];
    s.end_tok = p.lens[b];
    s.tiles = (s.end_tok - s.first_tok + kTile - 1) / kTile;
    rem = x - p.bpre[b];
    s.head = rem / s.tiles;
    rem -= s.head * s.tiles;
    s.rows = p.group;
    s.q0 = 0;
    s.mem0 = -1;
    s.row = b;
    s.rec = ((p.heads + s.head) * p.batch + b) * p.group;
  }
  s.tile0 = rem;
  s.begin = x;
  s.end = min(hi, x + s.tiles - rem);
  return s;
}

// Exclusive prefix sums of val(i), i < n, into pre[0 .. n]; every thread of the block.
template <class F>
__device__ __forceinline__ void block_scan(int* pre, int n, int base, int threads, int* scratch, F&& val) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + threads - 1) / threads;
  const int a = min(n, tid * per), b = min(n, a + per);
  int sum = 0;
  for (int i = a; i < b; ++i) sum += val(i);
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int run = base + incl - sum;
  for (int w = 0; w < warp; ++w) run += scratch[w];
  for (int i = a; i < b; ++i) {
    pre[i] = run;
    run += val(i);
  }
  if (tid == threads - 1) pre[n] = run;
  __syncthreads();
}

// --------------------------------------------------------------- code -> value
// Codes of 16 channels as 8 packed pairs u - c of the operand type, exactly.
template <bool BF>
__device__ __forceinline__ uint32_t pair_of_bytes(uint32_t w, int i) {   // bytes i, i + 1
  if constexpr (!BF) {
    // 0x6400 | u is 1024 + u; 1152 = 1024 + 128
    const uint32_t t = __byte_perm(w, 0x64646464u, 0x4040u + (uint32_t)(i * 0x0001 + (i + 1) * 0x0100));
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(0xE480E480u));
    return r;
  } else {
    // bf16 holds 8 bits: through fp32, 2^23 + u
    const float a = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u + (uint32_t)i)) - 8388736.0f;
    const float b = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u + (uint32_t)(i + 1))) - 8388736.0f;
    return pack16<true>(a, b);
  }
}
template <bool BF>
__device__ __forceinline__ uint32_t pair_of_nibbles(uint32_t w, uint32_t w4, int i) {   // byte i: its two codes
  // low half: byte i of w, high half: byte i of w >> 4, each with a byte of no interest above it
  const uint32_t v = __byte_perm(w, w4, (uint32_t)i | (uint32_t)i << 4 | (uint32_t)(i + 4) << 8 | (uint32_t)(i + 4) << 12);
  uint32_t r;
  if constexpr (!BF) {
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"((v & 0x000F000Fu) | 0x64006400u), "r"(0xE408E408u));   // - 1032
  } else {
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"((v & 0x000F000Fu) | 0x43004300u), "r"(0xC308C308u));   // - 136
  }
  return r;
}

// A staged tile of codes [128][ROW] to an operand tile [half][128][128 bytes], swizzled: 16-byte
// piece j of row r of a half sits at j ^ (r % 8). 128 threads.
template <int D, int KV, bool BF>
__device__ __forceinline__ void convert_tile(const uint8_t* src, uint8_t* dst, int t) {
  if constexpr (KV == KV_U4T) {
    constexpr int PER = D / 32;   // 16-byte pieces of codes per row, 32 channels each
#pragma unroll
    for (int it = 0; it < PER; ++it) {
      const int i = it * 128 + t, r = i / PER, c = i % PER;
      const uint4 v = *reinterpret_cast<const uint4*>(src + (size_t)i * 16);
      uint8_t* row = dst + (c >> 1) * 16384 + r * 128;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w4 = w[k] >> 4;
        const uint4 o = make_uint4(pair_of_nibbles<BF>(w[k], w4, 0), pair_of_nibbles<BF>(w[k], w4, 1),
                                   pair_of_nibbles<BF>(w[k], w4, 2), pair_of_nibbles<BF>(w[k], w4, 3));
        *reinterpret_cast<uint4*>(row + ((((c & 1) * 4 + k) ^ (r & 7)) << 4)) = o;
      }
    }
  } else {
    constexpr int PER = D / 16;
#pragma unroll 4
    for (int it = 0; it < PER; ++it) {
      const int i = it * 128 + t, r = i / PER, c = i % PER;
      const uint4 v = *reinterpret_cast<const uint4*>(src + (size_t)i * 16);
      uint8_t* row = dst + (c >> 2) * 16384 + r * 128;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 o = make_uint4(pair_of_bytes<BF>(w[2 * k], 0), pair_of_bytes<BF>(w[2 * k], 2),
                                   pair_of_bytes<BF>(w[2 * k + 1], 0), pair_of_bytes<BF>(w[2 * k + 1], 2));
        *reinterpret_cast<uint4*>(row + ((((c & 3) * 2 + k) ^ (r & 7)) << 4)) = o;
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel
template <int D, int KV, bool BF>
__global__ void __launch_bounds__(SharedGeom<D, KV, BF>::THREADS, 1)
    shared_attention_kernel(const __grid_constant__ SharedParams p) {
  using G = SharedGeom<D, KV, BF>;
  constexpr bool QUANT = G::QUANT;
  constexpr int NT = G::THREADS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const SharedLayout lay = shared_layout<G>(p.entries, p.batch, p.num_groups);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bars = smem_u32(smem + lay.bars);
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  volatile int* misc = reinterpret_cast<volatile int*>(smem + lay.misc);   // [0] TMEM base, [1] gave up
  int* scratch = const_cast<int*>(misc) + 4;
  int* lens = reinterpret_cast<int*>(smem + lay.lens);
  int* skip = reinterpret_cast<int*>(smem + lay.skip);
  int* bpre = reinterpret_cast<int*>(smem + lay.bpre);
  int* gpre = reinterpret_cast<int*>(smem + lay.gpre);
  int* gp = reinterpret_cast<int*>(smem + lay.gp);
  int* moff = reinterpret_cast<int*>(smem + lay.moff);
  uint16_t* members = reinterpret_cast<uint16_t*>(smem + lay.members);
  uint16_t* rank = reinterpret_cast<uint16_t*>(smem + lay.rank);
  const int S = p.entries, B = p.batch, NG = p.num_groups, Gq = p.group;

  if (tid == 0) {
    for (int i = 0; i < kMaxEntries; ++i) {
      mbar_init(bar(kBarFull + i), 1);
      mbar_init(bar(kBarEmpty + i), QUANT ? 4 : 1);
    }
    for (int i = 0; i < kHdrs; ++i) mbar_init(bar(kBarHdr + i), QUANT ? 4 : 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarQFull + i), 1);
      mbar_init(bar(kBarQEmpty + i), 1);
      mbar_init(bar(kBarS + i), 1);
      mbar_init(bar(kBarP + i), 4);
      mbar_init(bar(kBarO + i), 1);
    }
    mbar_init(bar(kBarKop), 4);        // converted K ready / free again
    mbar_init(bar(kBarKop + 1), 1);
    mbar_init(bar(kBarVop), 4);
    mbar_init(bar(kBarVop + 1), 1);
    for (int i = 0; i < 4; ++i) mbar_init(bar(kBarPair + i), 2);
    mbar_init(bar(kBarEnd), 1);
    misc[1] = 0;
  }
  fence_mbar_init();
  pdl_wait();
  pdl_launch_dependents();

  // ---- plan: lengths, who shares, visits before each segment
  const long long cap = (long long)p.max_pages * p.page_size;
  for (int g = tid; g < NG; g += NT) {
    const int P = p.prefix_lens[g];
    if (P < 0 && blockIdx.x == 0) flag_status(p.dev_status, PKV_DEV_BAD_GROUP);
    gp[g] = P < 0 ? 0 : P;
    moff[g] = 0;
  }
  __syncthreads();
  for (int b = tid; b < B; b += NT) {
    int L = p.seq_lens[b], g = p.prefix_group[b];
    if (L < 0 || L > cap) {
      if (blockIdx.x == 0) flag_status(p.dev_status, PKV_DEV_BAD_POSITION);
      L = L < 0 ? 0 : (int)cap;
    }
    if (g < -1 || g >= NG) {
      if (blockIdx.x == 0) flag_status(p.dev_status, PKV_DEV_BAD_GROUP);
      g = -1;
    }
    // a row shares its group's prefix if it has all of it
    const int P = g >= 0 ? gp[g] / p.round_to * p.round_to : 0;
    if (g >= 0 && (P == 0 || L < gp[g])) g = -1;
    lens[b] = L;
    skip[b] = g >= 0 ? P : 0;
    members[b] = (uint16_t)g;   // the group for now
  }
  __syncthreads();
  if (warp == 0) {   // each row's place among its group's rows
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + lane;
      const int g = b < B ? (int)(int16_t)members[b] : -1;
      const unsigned same = __match_any_sync(0xffffffffu, g);
      const int base = g >= 0 ? moff[g] : 0;
      __syncwarp();
      if (g >= 0 && lane == __ffs(same) - 1) moff[g] = base + __popc(same);
      __syncwarp();
      if (b < B) rank[b] = (uint16_t)(base + __popc(same & ((1u << lane) - 1)));
    }
  }
  __syncthreads();
  // visits of a group's prefix: kv heads x pairs of row tiles x tiles of tokens
  for (int g = tid; g < NG; g += NT) gp[g] = gp[g] / p.round_to * p.round_to;
  __syncthreads();
  block_scan(gpre, NG, 0, NT, scratch, [&](int g) {
    const int rows = moff[g] * Gq;
    return rows == 0 ? 0 : p.num_kv_heads * ((rows + 2 * kTile - 1) / (2 * kTile)) * ((gp[g] + kTile - 1) / kTile);
  });
  {   // members before each group, in place of their counts
    const int per = (NG + NT - 1) / NT;   // <= 3: up to 1024 groups, 384 threads and more
    const int a = min(NG, tid * per), e = min(NG, a + per);
    int c[3], sum = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      c[i] = a + i < e ? moff[a + i] : 0;
      sum += c[i];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += scratch[w];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (a + i < e) moff[a + i] = run;
      run += c[i];
    }
    if (tid == NT - 1) moff[NG] = run;
    __syncthreads();
  }
  const int Wp = gpre[NG];
  block_scan(bpre, B, Wp, NT, scratch,
             [&](int b) { return p.num_kv_heads * ((lens[b] - skip[b] + kTile - 1) / kTile); });
  const int W = bpre[B];
  // members by group; the group of row b is still in members[b], so each thread reads its rows' first
  {
    int16_t mine[4];
    constexpr int PER = (1024 + NT - 1) / NT;
    static_assert(PER <= 4, "rows per thread");
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = tid + i * NT;
      mine[i] = b < B ? (int16_t)members[b] : (int16_t)-1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = tid + i * NT;
      if (b >= B) continue;
      const int g = mine[i];
      if (g >= 0) members[moff[g] + rank[b]] = (uint16_t)b;
      if (b % (int)gridDim.x == (int)blockIdx.x) {   // for the merge: where row b's segments are
        const int rows = g >= 0 ? (moff[g + 1] - moff[g]) * Gq : 0;
        p.ws_info[2 * b] = make_int4(g >= 0 ? moff[g] * Gq : 0, g >= 0 ? rank[b] : 0, g >= 0 ? gpre[g] : 0,
                                     (rows + 2 * kTile - 1) / (2 * kTile));
        p.ws_info[2 * b + 1] = make_int4(g >= 0 ? (gp[g] + kTile - 1) / kTile : 0, bpre[b],
                                         (lens[b] - skip[b] + kTile - 1) / kTile, W);
      }
    }
  }
  const SharedPlan plan = {lens, skip, bpre, gpre, gp, moff, members, B, NG, p.num_kv_heads, Gq, W, Wp};
  const int lo = W > 0 ? share_lo(blockIdx.x, W, p.num_ctas) : 0;
  const int hi = W > 0 ? share_lo(blockIdx.x + 1, W, p.num_ctas) : 0;
  if (lo >= hi) return;   // uniform over the block

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(smem + lay.misc))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = (uint32_t)misc[0];
  const uint32_t tm_s[2] = {tmem, tmem + 128}, tm_o[2] = {tmem + 256, tmem + 256 + D};

  // Bounded wait; the first warp to give up reports it and everyone stops.
  auto wait = [&](int i, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(i), parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar(i), parity)) {
      if (misc[1]) return false;
      if (clock64() - t0 > (1ll << 31)) {
        misc[1] = 1;
        flag_status(p.dev_status, PKV_DEV_TIMEOUT);
        return false;
      }
    }
    return true;
  };

  // for a whole warp: every lane goes on, or none does
  auto wait_warp = [&](int i, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(i, parity)); };

  if (warp == 8) {
    // ================================================================ loader
    const uint64_t pol = policy_evict_first();
    // lanes 0-15 copy K, 16-31 V; within them piece (16 tokens) and half of the channels
    constexpr int PARTS = QUANT ? 1 : G::HALVES;
    const int isv = lane >> 4, piece = (lane & 15) / PARTS, half = (lane & 15) % PARTS;
    const bool lane_on = piece < 8;
    int v = 0;
    bool ok = true;
    // page of this lane's piece, one visit ahead
    Seg s = locate(plan, lo, hi);
    auto lookup = [&](const Seg& sg, int x) -> int {
      const int tok = sg.first_tok + (sg.tile0 + x - sg.begin) * kTile + 16 * piece;
      if (!lane_on || tok >= sg.end_tok) return -2;   // nothing to copy
      return p.block_table[(size_t)sg.row * p.max_pages + tok / p.page_size];
    };
    int page = lookup(s, lo);
    for (int x = lo; x < hi && ok; ++x, ++v) {
      const Seg cs = s;
      const int tok = cs.first_tok + (cs.tile0 + x - cs.begin) * kTile + 16 * piece;
      const int pg = page;
      if (x + 1 < hi) {
        if (x + 1 == s.end) s = locate(plan, x + 1, hi);
        page = lookup(s, x + 1);
      }
      const bool bad = pg != -2 && (pg < 0 || pg >= p.num_pages);
      if (bad && isv == 0 && half == 0) flag_status(p.dev_status, PKV_DEV_BAD_PAGE);
      const bool copy = pg != -2 && !bad;
      const unsigned has = __ballot_sync(0xffffffffu, copy && half == 0);
      // bit i: piece i was copied (from the K lanes; the V lanes have the same)
      unsigned mask = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mask |= (has >> (i * PARTS) & 1u) << i;
      const int e = 2 * v + isv, slot = e % S, use = e / S;
      ok = use == 0 || wait(kBarEmpty + slot, (use - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t fb = bar(kBarFull + slot);
      if ((lane & 15) == 0) {
        if (isv == 0) {
          const int n = min(kTile, cs.end_tok - (cs.first_tok + (cs.tile0 + x - cs.begin) * kTile));
          *reinterpret_cast<int2*>(smem + lay.hdr + (v % kHdrs) * 8) = make_int2(n, (int)mask);
        }
        uint32_t bytes = (uint32_t)__popc(mask) * 16u * G::ROW;
        if constexpr (KV == KV_I8T || KV == KV_U4T) bytes += isv == 0 ? (uint32_t)__popc(mask) * 256u : 0u;
        if constexpr (KV == KV_I8G) bytes += isv == 0 ? (uint32_t)((mask & 0xF ? 16 : 0) + (mask & 0xF0 ? 16 : 0)) : 0u;
        if (bytes)
          mbar_arrive_expect_tx(fb, bytes);
        else
          mbar_arrive(fb);
        if (!QUANT && isv == 0) mbar_arrive(bar(kBarHdr + v % kHdrs));
      }
      __syncwarp();
      if (copy) {
        const size_t row = ((size_t)pg * p.num_kv_heads + cs.head) * p.page_size + tok % p.page_size;
        uint8_t* dst = smem + lay.ring + (size_t)slot * G::ENTRY;
        if constexpr (!QUANT) {
          tma_load_2d(smem_u32(dst + half * 16384 + piece * 2048), isv ? &p.tmap_v : &p.tmap_k, half * 64, (int)row,
                      fb, pol);
        } else {
          bulk_g2s(smem_u32(dst + piece * 16 * G::ROW), (isv ? p.v_pages : p.k_pages) + row * G::ROW, 16 * G::ROW, fb,
                   pol);
          if (isv == 0) {
            uint8_t* raw = smem + lay.raw + (size_t)(v % (S / 2)) * G::RAW_SCALES;
            if constexpr (KV != KV_I8G) {
              bulk_g2s(smem_u32(raw + piece * 256), p.kv_sz + row * 4, 256, fb, pol);
            } else if ((mask & ((1u << piece) - 1) & (piece < 4 ? 0xFu : 0xF0u)) == 0) {
              // the first copied piece of a 64-token group brings its scales
              bulk_g2s(smem_u32(raw + (piece >> 2) * 16), p.kv_sz + row / 64 * 4, 16, fb, pol);
            }
          }
        }
      }
      __syncwarp();
    }
    // every issued copy lands before the block can end
    if (lane == 0) {
      const int n = 2 * v;
      for (int e = n > S ? n - S : 0; e < n; ++e)
        if (!mbar_wait_bounded(bar(kBarFull + e % S), (e / S) & 1)) break;
    }
  } else if (warp == 9) {
    // =================================================================== MMA
    if (lane == 0) {
      constexpr uint32_t kType = BF ? (1u << 7 | 1u << 10) : 0u;
      constexpr uint32_t idesc_s = 1u << 4 | kType | (uint32_t)(kTile / 8) << 17 | 8u << 24;
      constexpr uint32_t idesc_o = 1u << 4 | kType | 1u << 16 | (uint32_t)(D / 8) << 17 | 8u << 24;
      const uint32_t qb = smem_u32(smem + lay.q), ring = smem_u32(smem + lay.ring);
      const uint32_t kop = smem_u32(smem + lay.kop), vop = smem_u32(smem + lay.vop);
      int qc = 0, v = 0;
      uint32_t pn[2] = {0, 0};   // events so far on each stream
      bool ok = true;
      // the event whose P V product is still to be issued
      struct { int st, v, steps; bool on, fresh, last_use, seg_end; } pend = {};
      auto issue_pv = [&]() -> bool {
        const int st = pend.st, e = 2 * pend.v + 1;
        if (!wait(kBarP + st, (pn[st] - 1) & 1)) return false;
        uint32_t vb;
        if constexpr (QUANT) {
          if (!wait(kBarVop, pend.v & 1)) return false;
          vb = vop;
        } else {
          if (!wait(kBarFull + e % S, (e / S) & 1)) return false;
          vb = ring + (uint32_t)(e % S) * G::ENTRY;
        }
        tc_after();
        for (int j = 0; j < pend.steps; ++j) {
          const uint64_t vd = operand_desc(vb + j * 2048, 16384, 1024);
          const uint32_t a = tm_s[st] + 32 * (j >> 1) + 8 * (j & 1);
          mma_ts(tm_o[st], a, vd, idesc_o, !(pend.fresh && j == 0));
          if (p.two_terms) mma_ts(tm_o[st], a + 16, vd, idesc_o, 1);
        }
        if (pend.last_use) tc_commit(QUANT ? bar(kBarVop + 1) : bar(kBarEmpty + e % S));
        if (pend.seg_end) tc_commit(bar(kBarO + st));
        pend.on = false;
        return true;
      };
      for (int x = lo; x < hi && ok;) {
        const Seg s = locate(plan, x, hi);
        const bool two = s.rows > kTile;
        const int n = s.end - s.begin;
        for (int i = 0; i < n && ok; ++i, ++v) {
          const int e = 2 * v, slot = e % S;
          ok = QUANT ? wait(kBarKop, v & 1) : wait(kBarFull + slot, (e / S) & 1);
          if (!ok) break;
          const int ntok = *reinterpret_cast<const volatile int*>(smem + lay.hdr + (v % kHdrs) * 8);
          const uint32_t kb = QUANT ? kop : ring + (uint32_t)slot * G::ENTRY;
          for (int u = 0; u < (two ? 2 : 1) && ok; ++u) {
            const int st = two ? u : v & 1, qs = (qc + (two ? u : 0)) & 1;
            // normally the streams alternate; a score tile is never overwritten
            // before the weights in it are used
            if (pend.on && pend.st == st) ok = issue_pv();
            if (!ok) break;
            if (i == 0) ok = wait(kBarQFull + qs, ((qc + (two ? u : 0)) >> 1) & 1);
            if (!ok) break;
            tc_after();
            const uint32_t q = qb + (uint32_t)qs * G::OPERAND;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (uint32_t)(k >> 2) * 16384 + (uint32_t)(k & 3) * 32;
              mma_ss(tm_s[st], operand_desc(q + off, 16, 1024), operand_desc(kb + off, 16, 1024), idesc_s, k > 0);
            }
            tc_commit(bar(kBarS + st));
            const bool last_s = u == (two ? 1 : 0);
            if (last_s) tc_commit(QUANT ? bar(kBarKop + 1) : bar(kBarEmpty + slot));
            if (i == n - 1) tc_commit(bar(kBarQEmpty + qs));
            if (pend.on) ok = issue_pv();
            ++pn[st];
            pend.st = st;
            pend.v = v;
            pend.steps = (ntok + 15) >> 4;
            pend.on = true;
            pend.fresh = two ? i == 0 : i < 2;
            pend.last_use = last_s;
            pend.seg_end = two ? i == n - 1 : i >= n - 2;
          }
        }
        qc += two ? 2 : 1;
        x = s.end;
      }
      if (ok && pend.on) ok = issue_pv();
      // nothing of the tensor cores is in flight past this point
      tc_commit(bar(kBarEnd));
      if (!mbar_wait_bounded(bar(kBarEnd), 0)) flag_status(p.dev_status, PKV_DEV_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ============================================================== Q gather
    constexpr int CH = D / 8;   // 16-byte pieces of a query row
    int qc = 0;
    bool ok = true;
    for (int x = lo; x < hi && ok;) {
      const Seg s = locate(plan, x, hi);
      const int tiles = s.rows > kTile ? 2 : 1;
      for (int u = 0; u < tiles && ok; ++u, ++qc) {
        const int qs = qc & 1;
        if (qc >= 2) ok = wait_warp(kBarQEmpty + qs, ((qc >> 1) - 1) & 1);
        if (!ok) break;
        uint8_t* dst = smem + lay.q + (size_t)qs * G::OPERAND;
        const int rows = min(kTile, s.rows - u * kTile);
        for (int i = lane; i < rows * CH; i += 32) {
          const int r = i / CH, c = i - r * CH;
          const int R = s.q0 + u * kTile + r;
          int b = s.row, gq = R;
          if (s.mem0 >= 0) {
            const int m = R / Gq;
            b = members[s.mem0 + m];
            gq = R - m * Gq;
          }
          const uint8_t* src = p.q + (((size_t)b * p.num_q_heads + s.head * Gq + gq) * D + c * 8) * 2;
          cp_async16(smem_u32(dst + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)), src);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        if constexpr (QUANT) {   // sum of each row's query, for the zero points
          float* qsum = reinterpret_cast<float*>(smem + lay.qsum) + (qc % kQSums) * kTile;
          for (int r = lane; r < rows; r += 32) {
            float t = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const uint4 w = *reinterpret_cast<const uint4*>(dst + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
              t += (low16<BF>(w.x) + high16<BF>(w.x)) + (low16<BF>(w.y) + high16<BF>(w.y)) +
                   ((low16<BF>(w.z) + high16<BF>(w.z)) + (low16<BF>(w.w) + high16<BF>(w.w)));
            }
            qsum[r] = t;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarQFull + qs));
      }
      x = s.end;
    }
  } else if (warp >= 12) {
    // ============================================================ converters
    if constexpr (QUANT) {
      const int t = tid - 384;
      for (int v = 0; v < hi - lo; ++v) {
        const int ek = 2 * v, ev = ek + 1;
        if (!wait_warp(kBarFull + ek % S, (ek / S) & 1)) break;
        if (v > 0 && !wait_warp(kBarKop + 1, (v - 1) & 1)) break;   // the previous visit's scores are done
        convert_tile<D, KV, BF>(smem + lay.ring + (size_t)(ek % S) * G::ENTRY, smem + lay.kop, t);
        // scales of token t, with the middle code's part in the zero points
        const int2 hd = *reinterpret_cast<const int2*>(smem + lay.hdr + (v % kHdrs) * 8);
        const bool valid = t < hd.x && (hd.y >> (t >> 4) & 1);
        const float4 z = *reinterpret_cast<const float4*>(smem + lay.raw + (size_t)(v % (S / 2)) * G::RAW_SCALES +
                                                          (KV == KV_I8G ? t >> 6 : t) * 16);
        float* sc = reinterpret_cast<float*>(smem + lay.scales + (v % kScaleSlots) * G::SCALES);
        sc[t] = valid ? z.x : 0.f;
        sc[kTile + t] = valid ? fmaf(G::CENTRE, z.x, z.y) : 0.f;
        sc[2 * kTile + t] = valid ? z.z : 0.f;
        sc[3 * kTile + t] = valid ? fmaf(G::CENTRE, z.z, z.w) : 0.f;
        float vm = valid ? z.z : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
        if (lane == 0) reinterpret_cast<float*>(smem + lay.vmax + (v % kScaleSlots) * 16)[warp - 12] = vm;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kBarKop));
          mbar_arrive(bar(kBarHdr + v % kHdrs));
          mbar_arrive(bar(kBarEmpty + ek % S));
        }
        if (!wait_warp(kBarFull + ev % S, (ev / S) & 1)) break;
        if (v > 0 && !wait_warp(kBarVop + 1, (v - 1) & 1)) break;
        convert_tile<D, KV, BF>(smem + lay.ring + (size_t)(ev % S) * G::ENTRY, smem + lay.vop, t);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kBarVop));
          mbar_arrive(bar(kBarEmpty + ev % S));
        }
      }
    }
  } else if (warp < 8) {
    // =============================================================== softmax
    const int st = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t ts = tm_s[st] + lanes, to = tm_o[st] + lanes;
    float4* mls = reinterpret_cast<float4*>(smem + lay.ml);
    int qc = 0, v = 0;
    uint32_t n_ev = 0, n_seg = 0, n_pair = 0;   // events and segments seen on this stream, meetings
    bool ok = true;
    for (int x = lo; x < hi && ok;) {
      const Seg s = locate(plan, x, hi);
      const bool two = s.rows > kTile;
      const int n = s.end - s.begin;
      const int my_rows = two ? min(kTile, s.rows - st * kTile) : s.rows;
      const bool active = quad * 32 < my_rows;   // this warp has query rows
      float m = -INFINITY, l = 0.f, zs = 0.f, vref = 0.f, qs = 0.f;
      bool have = false;
      for (int i = 0; i < n && ok; ++i, ++v) {
        if (!two && (v & 1) != st) continue;
        ok = wait_warp(kBarHdr + v % kHdrs, (v / kHdrs) & 1);
        if (ok) ok = wait_warp(kBarS + st, n_ev & 1);
        if (!ok) break;
        ++n_ev;
        const int2 hd = *reinterpret_cast<const int2*>(smem + lay.hdr + (v % kHdrs) * 8);
        const int ntok = hd.x;
        const bool partial = ntok < kTile || hd.y != 0xFF;
        if constexpr (!QUANT) {
          if (partial) {
            // rows of V that hold no token of this segment may hold anything, NaN
            // too, and a weight of 0 would not clear it
            const int e = 2 * v + 1;
            ok = wait_warp(kBarFull + e % S, (e / S) & 1);
            if (!ok) break;
            if (row < (ntok + 15) / 16 * 16 && (row >= ntok || !(hd.y >> (row >> 4) & 1))) {
              uint8_t* vr = smem + lay.ring + (size_t)(e % S) * G::ENTRY + row * 128;
#pragma unroll
              for (int h = 0; h < G::HALVES; ++h)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  *reinterpret_cast<uint4*>(vr + h * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
        }
        if (active) {
          tc_after();
          float a[kTile];
          uint32_t* ar = reinterpret_cast<uint32_t*>(a);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, ar + 32 * c);
          tc_wait_ld();
          const float* sc = reinterpret_cast<const float*>(smem + lay.scales + (v % kScaleSlots) * G::SCALES);
          if constexpr (QUANT) {
            if (!have)
              qs = reinterpret_cast<const float*>(smem + lay.qsum)[((qc + (two ? st : 0)) % kQSums) * kTile + row];
#pragma unroll
            for (int j = 0; j < kTile; j += 4) {
              const float4 ks = *reinterpret_cast<const float4*>(sc + j);
              const float4 kz = *reinterpret_cast<const float4*>(sc + kTile + j);
              a[j] = fmaf(ks.x, a[j], kz.x * qs);
              a[j + 1] = fmaf(ks.y, a[j + 1], kz.y * qs);
              a[j + 2] = fmaf(ks.z, a[j + 2], kz.z * qs);
              a[j + 3] = fmaf(ks.w, a[j + 3], kz.w * qs);
            }
          }
          if (partial) {
#pragma unroll
            for (int j = 0; j < kTile; ++j)
              if (j >= ntok || !(hd.y >> (j >> 4) & 1)) a[j] = -INFINITY;
          }
          float mx[4] = {a[0], a[1], a[2], a[3]};
#pragma unroll
          for (int j = 4; j < kTile; ++j) mx[j & 3] = fmaxf(mx[j & 3], a[j]);
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale;
          float alpha = 1.f;
          if (mt > m + 8.f) {
            alpha = m == -INFINITY ? 0.f : fast_exp2(m - mt);
            m = mt;
            l *= alpha;
            zs *= alpha;
          }
          float rv = 0.f;
          if constexpr (QUANT) {
            const float4 vm4 = *reinterpret_cast<const float4*>(smem + lay.vmax + (v % kScaleSlots) * 16);
            const float vm = fmaxf(fmaxf(vm4.x, vm4.y), fmaxf(vm4.z, vm4.w));
            if (vm > 64.f * vref) {   // uniform: the next power of two, within 2^-100 .. 2^100
              const uint32_t up = (__float_as_uint(vm) + 0x7FFFFFu) & 0x7F800000u;
              const float nv = __uint_as_float(min(max(up, 27u << 23), 227u << 23));
              alpha *= vref / nv;
              vref = nv;
            }
            rv = vref > 0.f ? __uint_as_float((254u << 23) - __float_as_uint(vref)) : 0.f;
          }
          if (have && __any_sync(0xffffffffu, alpha != 1.f)) {
            // S of this event is complete, so every earlier product of this stream is
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(to + 32 * c, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st32(to + 32 * c, o);
            }
          }
          const float mref = m == -INFINITY ? 0.f : m;
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (32 * c < ntok) {
              uint32_t hi16[16], lo16[16];
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                float w0 = fast_exp2(fmaf(a[32 * c + j], p.scale, -mref));
                float w1 = fast_exp2(fmaf(a[32 * c + j + 1], p.scale, -mref));
                ls[j & 2] += w0;
                ls[(j & 2) + 1] += w1;
                if constexpr (QUANT) {
                  const float2 vs = *reinterpret_cast<const float2*>(sc + 2 * kTile + 32 * c + j);
                  const float2 vz = *reinterpret_cast<const float2*>(sc + 3 * kTile + 32 * c + j);
                  zs = fmaf(w0, vz.x, zs);
                  zs = fmaf(w1, vz.y, zs);
                  w0 *= vs.x * rv;
                  w1 *= vs.y * rv;
                }
                // the weights' one rounding to the operand type; a second term
                // holds what it left where the output keeps more bits
                hi16[j / 2] = pack16<BF>(w0, w1);
                if (p.two_terms)
                  lo16[j / 2] = pack16<BF>(w0 - low16<BF>(hi16[j / 2]), w1 - high16<BF>(hi16[j / 2]));
              }
              tmem_st16(ts + 32 * c, hi16);
              if (p.two_terms) tmem_st16(ts + 32 * c + 16, lo16);
            }
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
          tc_wait_st();
          tc_before();
        }
        have = true;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarP + st));
      }
      if (!ok) break;
      // ---- end of the block's part of the segment: one record per query row
      const bool part = s.tile0 > 0;   // the segment began in an earlier block
      const int tile_row = two ? st * kTile + row : row;
      const size_t rec = part ? (size_t)2 * p.num_kv_heads * B * Gq + (size_t)blockIdx.x * 2 * kTile + tile_row
                              : (size_t)s.rec + tile_row;
      float* acc = p.ws_acc + rec * D;
      const bool both = !two && n > 1;
      if (have) {
        ok = wait_warp(kBarO + st, n_seg & 1);
        if (!ok) break;
        ++n_seg;
      }
      if (active && !both) {
        if (have) {
          tc_after();
          if (row < my_rows) p.ws_ml[rec] = make_float2(m, l);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(to + 32 * c, o);
            tc_wait_ld();
            if (row < my_rows) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                float4 f = make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]), __uint_as_float(o[j + 2]),
                                       __uint_as_float(o[j + 3]));
                if constexpr (QUANT) {
                  f.x = fmaf(f.x, vref, zs);
                  f.y = fmaf(f.y, vref, zs);
                  f.z = fmaf(f.z, vref, zs);
                  f.w = fmaf(f.w, vref, zs);
                }
                *reinterpret_cast<float4*>(acc + 32 * c + j) = f;
              }
            }
          }
          tc_before();
        }
      } else if (active) {
        // the two streams' states of each row meet: each stream's warp merges
        // half of the channels of both accumulators
        mls[st * kTile + row] = make_float4(m, l, zs, vref);
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPair + quad));
        ok = wait_warp(kBarPair + quad, n_pair++ & 1);
        if (!ok) break;
        tc_after();
        const float4 other = mls[(st ^ 1) * kTile + row];
        const float M = fmaxf(m, other.x);
        float f0 = m == -INFINITY ? 0.f : fast_exp2(m - M), f1 = other.x == -INFINITY ? 0.f : fast_exp2(other.x - M);
        if (row < my_rows && st == 0) p.ws_ml[rec] = make_float2(M, fmaf(l, f0, other.y * f1));
        const float z = fmaf(zs, f0, other.z * f1);
        if constexpr (QUANT) {
          f0 *= vref;
          f1 *= other.w;
        }
        const uint32_t to2 = tm_o[st ^ 1] + lanes;
#pragma unroll 1
        for (int c = st * (D / 64); c < (st + 1) * (D / 64); ++c) {
          uint32_t o[32], o2[32];
          tmem_ld32(to + 32 * c, o);
          tmem_ld32(to2 + 32 * c, o2);
          tc_wait_ld();
          if (row < my_rows) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              float4 f = make_float4(fmaf(__uint_as_float(o[j]), f0, __uint_as_float(o2[j]) * f1),
                                     fmaf(__uint_as_float(o[j + 1]), f0, __uint_as_float(o2[j + 1]) * f1),
                                     fmaf(__uint_as_float(o[j + 2]), f0, __uint_as_float(o2[j + 2]) * f1),
                                     fmaf(__uint_as_float(o[j + 3]), f0, __uint_as_float(o2[j + 3]) * f1));
              if constexpr (QUANT) {
                f.x += z;
                f.y += z;
                f.z += z;
                f.w += z;
              }
              *reinterpret_cast<float4*>(acc + 32 * c + j) = f;
            }
          }
        }
        tc_before();   // neither accumulator is overwritten before both are read
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPair + quad));
        ok = wait_warp(kBarPair + quad, n_pair++ & 1);
        if (!ok) break;
      }
      qc += two ? 2 : 1;
      x = s.end;
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------ the merge
// Folds a query row's records (from the block where each of its two segments begins
// and from the blocks that continue them): WPR warps per row, each lane 4 channels of
// every WPR-th record (two records at a time at 64 channels).
constexpr int kMergeThreads = 128;

template <int D, int WPR>
__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const __grid_constant__ SharedParams p) {
  constexpr int LPR = D / 4, SUB = 32 / LPR;       // lanes per record, records side by side in a warp
  constexpr int STREAMS = WPR * SUB, BATCH = 4;
  __shared__ float part[4][WPR > 1 ? D + 2 : 1];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.x * (4 / WPR) + warp / WPR, w = warp % WPR;
  pdl_wait();
  if (item >= p.batch * p.num_q_heads) return;   // uniform over a row's warps
  const int b = item / p.num_q_heads, hq = item - b * p.num_q_heads;
  const int h = hq / p.group, gq = hq - h * p.group;
  const int4 i0 = __ldcg(p.ws_info + 2 * b), i1 = __ldcg(p.ws_info + 2 * b + 1);
  const long long W = i1.w, N = p.num_ctas;
  const int base2 = 2 * p.num_kv_heads * p.batch * p.group;
  // prefix records, then the row's own
  int c0[2] = {0, 0}, n[2] = {0, 0}, rec[2], sub[2];
  {
    const int R = i0.y * p.group + gq;             // query row within the group
    rec[0] = h * p.batch * p.group + i0.x + R;
    sub[0] = R % (2 * kTile);
    if (i1.x > 0) {
      const int s0 = i0.z + (h * i0.w + R / (2 * kTile)) * i1.x;
      c0[0] = share_of(s0, W, N);
      n[0] = share_of(s0 + i1.x - 1, W, N) - c0[0] + 1;
    }
    rec[1] = ((p.num_kv_heads + h) * p.batch + b) * p.group + gq;
    sub[1] = gq;
    if (i1.z > 0) {
      const int s0 = i1.y + h * i1.z;
      c0[1] = share_of(s0, W, N);
      n[1] = share_of(s0 + i1.z - 1, W, N) - c0[1] + 1;
    }
  }
  const int total = n[0] + n[1];
  const int my = w * SUB + lane / LPR, ch = (lane % LPR) * 4;
  float M = -INFINITY, L = 0.f;
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = my; j0 < total; j0 += STREAMS * BATCH) {
    float2 ml[BATCH];
    float4 a[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      int j = j0 + i * STREAMS;
      const int k = j >= n[0];
      bool on = j < total;
      if (k) j -= n[0];
      const int c = c0[k] + j;
      // a block without visits (fewer visits than blocks) has no record
      if (on && j > 0) on = share_lo(c, W, N) < share_lo(c + 1, W, N);
      const size_t r = on ? (j == 0 ? (size_t)rec[k] : (size_t)base2 + (size_t)c * 2 * kTile + sub[k]) : 0;
      ml[i] = on ? __ldcg(p.ws_ml + r) : make_float2(-INFINITY, 0.f);
      a[i] = on ? __ldcg(reinterpret_cast<const float4*>(p.ws_acc + r * D + ch)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float Mn = M;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) Mn = fmaxf(Mn, ml[i].x);
    if (Mn == -INFINITY) continue;
    const float f0 = M == -INFINITY ? 0.f : exp2f(M - Mn);
    L *= f0;
    A.x *= f0; A.y *= f0; A.z *= f0; A.w *= f0;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (ml[i].x == -INFINITY) continue;   // no token: its accumulator means nothing
      const float f = exp2f(ml[i].x - Mn);
      L = fmaf(f, ml[i].y, L);
      A.x = fmaf(f, a[i].x, A.x);
      A.y = fmaf(f, a[i].y, A.y);
      A.z = fmaf(f, a[i].z, A.z);
      A.w = fmaf(f, a[i].w, A.w);
    }
    M = Mn;
  }
  auto join = [&](float M2, float L2, float4 A2) {
    const float Mn = fmaxf(M, M2);
    if (Mn == -INFINITY) return;
    const float f = M == -INFINITY ? 0.f : exp2f(M - Mn), f2 = M2 == -INFINITY ? 0.f : exp2f(M2 - Mn);
    L = L * f + L2 * f2;
    A.x = A.x * f + A2.x * f2;
    A.y = A.y * f + A2.y * f2;
    A.z = A.z * f + A2.z * f2;
    A.w = A.w * f + A2.w * f2;
    M = Mn;
  };
  if constexpr (SUB == 2) {
    const float M2 = __shfl_xor_sync(0xffffffffu, M, 16), L2 = __shfl_xor_sync(0xffffffffu, L, 16);
    const float4 A2 = make_float4(__shfl_xor_sync(0xffffffffu, A.x, 16), __shfl_xor_sync(0xffffffffu, A.y, 16),
                                  __shfl_xor_sync(0xffffffffu, A.z, 16), __shfl_xor_sync(0xffffffffu, A.w, 16));
    if (lane < 16) join(M2, L2, A2);
  }
  if constexpr (WPR > 1) {
    if (lane < LPR) {
      *reinterpret_cast<float2*>(&part[w][ch]) = make_float2(A.x, A.y);
      *reinterpret_cast<float2*>(&part[w][ch + 2]) = make_float2(A.z, A.w);
      if (lane == 0) {
        part[w][D] = M;
        part[w][D + 1] = L;
      }
    }
    __syncthreads();
    if (w != 0 || lane >= LPR) return;
#pragma unroll
    for (int o = 1; o < WPR; ++o)
      join(part[o][D], part[o][D + 1],
           make_float4(part[o][ch], part[o][ch + 1], part[o][ch + 2], part[o][ch + 3]));
  }
  if (lane >= LPR) return;
  // no token at all: zeros (L is 0 only then; a NaN stays one)
  const float r = L == 0.f ? 0.f : 1.f / L;
  const size_t o = (size_t)item * D + ch;
  const float4 f = make_float4(A.x * r, A.y * r, A.z * r, A.w * r);
  if (p.out_dtype == PKV_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = f;
  } else {
    const uint2 v = p.out_dtype == PKV_BF16 ? make_uint2(pack16<true>(f.x, f.y), pack16<true>(f.z, f.w))
                                            : make_uint2(pack16<false>(f.x, f.y), pack16<false>(f.z, f.w));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o) = v;
  }
}

}  // namespace pkv
