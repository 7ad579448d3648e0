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
// What bounds it. Bytes of K and V where a prefix serves few query rows, 4 d operations per
// query row and token where it serves many; in between and for short calls the latency of
// what follows one another: scores, softmax, P V.
//
// Work decomposition. A segment is one of the products above for one kv head:
// up to 256 query rows over a token range. It is cut into tiles of 128 tokens; one
// visit is one tile for all of the segment's rows. The visits of all segments are
// laid end to end and each block takes an equal share of them (see Shares), whatever the
// lengths are. A block that covers part of a segment leaves a partial state; the
// second launch merges them. Every block makes the plan for itself from the lengths: with a
// launch of its own it would cost more than the 1.3 us that it takes.
//
// Inside a block (one per SM, TMEM fully used: two score tiles of 128 columns and two
// accumulators of d columns):
//   warps 0-7    softmax, four for each of two streams
//   warps 8, 11  K and V tiles into a ring each, 16 tokens a copy (a page may end every 16);
//                block-table entries of four visits a load, a batch ahead
//   warp 9       the products: S of the next event, then P V of the one before
//   warp 10      the next segment's queries into the swizzled operand tile; descriptions of
//                the visits to come; for the merge, where the records will be
//   12-15, 16-19 quantised caches: codes of K and of V into operand tiles
// An event is a visit's scores for one row tile. Two streams keep the tensor cores busy
// while the exponentials of the other are computed: with more than 128 rows each has its own
// 128 rows and both use every tile; otherwise the tiles alternate between the streams,
// whose states meet when the segment ends.
//   Few rows (16, quantised caches 8): transposed, S^T = K Q^T and O^T = V^T P^T, a thread has
//     a token, so that a tile costs 8 or 16 exponentials a thread and not 128. The weights'
//     two terms are two halves of one operand.
//   More: a thread has a query row. P lies in TMEM over the scores it was made from.
// V enters as stored (MN-major); Q and K with 128-byte swizzle.
//
// Weights are 2^(s - r) with a reference r that follows the running maximum, less kWeightBits,
// only when that is over 8 above it: the largest weight then lies in [2^7, 2^15], in the upper part
// of fp16's range (2^-24 to 65504), so that the smallest still count, and the accumulator in TMEM
// is rarely rescaled. Maxima, sums and accumulators are fp32.
//
// INT8 and 4-bit caches: the codes enter the products as exact small integers, u - c
// with c the middle code, made by four converter warps from the staged bytes;
// scales and zero points are applied in fp32:
//   q . k = ks (q . (u - c)) + (kz + c ks) sum q
//   sum p v = sum (p vs) (u - c) + sum p (vz + c vs)
// There r follows the largest of score + log2(that token's value size), so that p vs stays inside
// fp16's range and a large value of no weight costs the others no bits: few rows token by
// token, more rows by the tile's largest score and largest size as long as the sizes in
// the tile are within 2^kEvenBits of one another. (Scales folded into the codes would round every key
// to 11 bits, or 8.)
//
// Measured, both launches, back to back (peaks 6.78 TB/s, 1.91 PFLOP/s; d = 128):
//   2 rows x 64K, 32 heads over 8, bf16      50 us, 5.3 TB/s; INT8 56 us, 4-bit 59 us
//   64 rows alone x ~2K, bf16                87 us, 6.2 TB/s
//   16 rows x 32K, 32 kv heads, bf16         90 us, 6.1 TB/s
//   64 rows x 16K, 32 heads over 8, bf16     50 us, 0.34 PFLOP/s; INT8 74 us
// Counters of 256 rows x 8K: tensor pipe active 23 % of the cycles, issue slots 25 %, DRAM
// 32 %: bound by the chain of an event (softmax 1600 cycles, then P V and S of 520 each
// with 200-700 cycles of hand-over each), twice which is a visit's period of 4600.
// INT8: softmax 6000 cycles (two reads of the scales, 96 registers).
//
// Trees of drafts (kFewDrafts, kDraftRows) are segments of another kind: all drafts' query rows of a sequence, over its
// whole cache, with a mask over the last tokens, the drafts. Sequences take the place of groups; nothing else is planned.
//   Masks: a tile that holds drafts gets 128 bits for each query row (or, transposed, a row's bits for each token), read
//     from the caller's words while the scores are on their way; scores of tokens that a row does not
//     attend to become -inf in the pass that looks for the maximum.
//   A value of 0 weight still makes NaN of an infinity or NaN. Such values of drafts are taken out of the operand tile
//     (or their scales of the scales), rows that do attend to them are marked in the sign of their sum, and
//     the merge adds what was taken out.
//   Queries come as boxes of a tensor map, where a group's heads divide 128.
//   Records are laid out for 32 rows at a time, channel by channel, so that a thread that has a row writes, and the
//     merge reads, 128 bytes together.
//   Measured (both launches, d = 128, back to back, 16-bit outputs): 4 sequences of 20K to 32K, 13 drafts, 32 kv heads, f16
//     262 to 267 us, 6.6 to 6.7 TB/s; 24 of 4K to 8K, 64 drafts of 32 heads over 8, bf16 152 to 160 us, 1.0 PFLOP/s; 8 of 2K to 4K,
//     16 drafts 30 us; 16 x 8192, 24 drafts, bf16 95, INT8 133, 4-bit 127 us. With 32-bit outputs, whose weights are two terms and whose
//     products are not issued in the inner loop, 262, 210, 33, 104, 158, 151 us. A visit of two row tiles takes 3970 cycles, of
//     which the products are 2050: the chain of an event is maximum 500, reference 150, weights 1070, then P V and S and their
//     hand-over 1470 to 2000. Shared memory is wanted for 2050 as well: S takes 128 bytes a cycle of operands, all there is, P V
//     half as much, and copies 64 KB. INT8's event: 2740, 240 and 2540, the latency of the scales' loads (1024 of shared
//     memory's 3700 cycles a visit).
//
// Code size is a cost of its own: the two SMs of a pair share an instruction cache, and
// 155 KB of code took 16 rows x 32K from 97 to 117 us. So loops stay loops, waits and plans
// are out of line, and each product is written once.
#pragma once

#include <type_traits>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

// A place in a ring, and the parity of its use.
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1;
    }
  }
};

constexpr int kTile = 128;        // tokens of a visit, query rows of a tile
// Visit headers kept. The K loader writes header v once entry v - S is free, i.e. its codes are
// converted; then the scores of v - S - 1 are done, and with them the softmax of
// v - S - 3 (16-bit caches: one visit later in each step). kMaxEntries + 3 are in use.
constexpr int kHdrs = 16;
// Visits whose scales are kept: written for v once the scores of v - 1, and so the
// softmax of v - 3, are done.
constexpr int kScaleSlots = 3;
// Query tiles whose sums are kept: tile t is gathered once the last scores of tile t - 2
// are done, when at most the last two events are still to be read, of tiles from t - 4 on.
constexpr int kQSums = 6;
constexpr int kMaxEntries = 6;    // ring entries of K, and of V
// The largest weight (times its value's size) is stored as at least 2^kWeightBits, and 2^8 times as
// much at most: 2^15 with sizes of at most 1.
constexpr float kWeightBits = 7.f;
// Value sizes of a tile that differ by more are looked at token by token: what the tile's largest
// one costs the others stays below this many bits.
constexpr int kEvenBits = 4;
constexpr int kVisits = 64;      // visits described in shared memory, refilled by halves
// Visits whose values that are no numbers are marked: the two streams are less than three visits apart.
constexpr int kBadSlots = 4;

// Shared memory by offset from a 1024-byte boundary.
struct SharedLayout {
  int q, kop, vop, ring, raw, pt, xch, scales, bars, hdr, ml, qsum, vmax, bad, misc, visits, bpre, gpre, lpre, moff, hseg, lseg, members, lens, skip, gp, rank, rowg;
  int total;
};
struct SharedParams {
  CUtensorMap tmap_k, tmap_v;   // 16-bit pools as [rows][d], boxes of 16 rows x 64 channels
  CUtensorMap tmap_q;           // trees: the queries as [drafts][heads][d], see q_box
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
  int4* ws_info;   // three for each row and kv head
  int num_pages, page_size, num_kv_heads, num_q_heads, group, batch, max_pages, num_groups;
  int num_ctas, entries /* of K, and of V */, round_to, q_dtype, out_dtype, two_terms;
  float scale;   // sm_scale * log2(e)
  // trees of drafts: the groups are the sequences, each row of the batch a draft
  const int32_t* draft_lens;   // drafts of each sequence, or NULL: `drafts` of each
  const uint64_t* tree_mask;   // [sequences][drafts][mask_words], or NULL: each after the one before
  int drafts, mask_words, pairs, kv_kind;
  int rec_rows;   // record rows of a sequence's kv head: its query rows, rounded up to 32
  int q_box;   // drafts of a box of queries (64 channels of a group's heads of each), 0: they are gathered
  long long mask_stride;       // words from one sequence's masks to the next's (0: the same)
  SharedLayout lay;
};

template <int D, int KV, bool BF>
struct SharedGeom {
  static constexpr bool QUANT = KV == KV_I8T || KV == KV_I8G || KV == KV_U4T;
  static constexpr int HALVES = D / 64;
  static constexpr int OPERAND = HALVES * 16384;   // 128 rows x d 16-bit values, [half][row][128 bytes]
  static constexpr int ROW = KV == KV_U4T ? D / 2 : (QUANT ? D : 2 * D);
  static constexpr int ENTRY = QUANT ? kTile * ROW : OPERAND;
  static constexpr int RAW_SCALES = QUANT ? (KV == KV_I8G ? 128 : kTile * 16) : 0;
  // scales of a visit: by pairs of tokens (ks, ks, kz', kz'), then (vs, vs, vz', vz')
  static constexpr int SCALES = QUANT ? 4 * kTile * 4 : 0;
  // Segments of at most FEW query rows run transposed; PT: a stream's weights of them, two
  // terms each. 16 against 8 on 16-bit caches: 16 rows x 32K 90.5 and 93.0 us, 32 rows x 2K
  // 25.7 and 26.6, 256 rows x 8K 82.8 and 84.5, but 256 rows x ~128 alone, four query rows
  // each, 44 and 41. Quantised caches have no room for 16 beside their converted tiles.
  static constexpr int FEW = QUANT ? 8 : 16, PT = FEW * 2 * kTile * 2;
  static constexpr int THREADS = QUANT ? 640 : 384;
  static constexpr float CENTRE = KV == KV_U4T ? 8.f : 128.f;
};

enum SharedBars {   // mbarriers, 8 bytes each
  kBarKFull = 0, kBarVFull = kMaxEntries, kBarKEmpty = 2 * kMaxEntries, kBarVEmpty = 3 * kMaxEntries,
  kBarHdr = 4 * kMaxEntries, kBarQFull = kBarHdr + kHdrs, kBarQEmpty = kBarQFull + 2, kBarS = kBarQEmpty + 2,
  kBarP = kBarS + 2, kBarO = kBarP + 2, kBarKop = kBarO + 2, kBarVop = kBarKop + 2,
  kBarPair = kBarVop + 2, kBarVisits = kBarPair + 4, kBarPassed = kBarVisits + 2, kBarEnd = kBarPassed + 2,
  kBarQLoad = kBarEnd + 1 /* copied queries whose sums are still to be taken */, kBarCount = kBarQLoad + 2
};

template <class G>
__host__ __device__ inline SharedLayout shared_layout(int entries, int batch, int groups, bool tree = false) {
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
  o.ring = put(2 * entries * G::ENTRY);
  o.raw = put(entries * G::RAW_SCALES);
  o.pt = put(2 * G::PT);
  o.xch = put(2 * 2 * 4 * 32 * 4);
  o.scales = put(kScaleSlots * G::SCALES);
  o.bars = put(kBarCount * 8);
  o.hdr = put(kHdrs * 8);
  o.ml = put(2 * kTile * 16);
  o.qsum = put(G::QUANT ? kQSums * kTile * 4 : 0);
  o.vmax = put(G::QUANT ? kScaleSlots * 32 : 0);
  o.bad = put(tree ? (G::QUANT ? kHdrs * 16 : kBadSlots * kTile * 4) : 0);
  o.misc = put(21 * 16);
  o.visits = put(kVisits * 32);
  o.bpre = put((batch + 1) * 4);
  o.gpre = put((groups + 1) * 4);
  o.lpre = put((groups + 1) * 4);
  o.moff = put((groups + 1) * 4);
  o.members = put(batch * 2);
  if (tree) {
    o.gp = put(groups * 4);
    o.hseg = put((groups + 1) * 4);
    o.lseg = put((groups + 1) * 4);
  }
  o.total = at;
  // the plan's other arrays are needed only while the ring is still empty
  at = o.ring;
  o.lens = put(batch * 4);
  o.skip = put(batch * 4);
  if (!tree) o.gp = put(groups * 4);
  o.rank = put(batch * 2);
  o.rowg = put(batch * 2);
  if (at > o.total) o.total = at;
  return o;
}

// Shares of the work. Visits are numbered: prefixes of more than one row tile first
// (`heavy` of them), then the other prefixes, then the rows' own tokens. A heavy visit
// counts as two units: it has twice the products and exponentials. (256 rows x 8K bf16,
// 256 tokens of their own, with a ratio of 1, 1.5, 2, 3: 103, 92, 83, 95 us; INT8 with 1, 2,
// 2.5, 3: 77, 60, 65, 67 us.) Block c of `blocks` gets the visits that start in its
// share of the units; every share holds at least one.
struct Shares {
  int heavy, blocks, q, r;   // units = blocks q + r
  __host__ __device__ __forceinline__ Shares() {}
  __device__ __forceinline__ Shares(int heavy_visits, int visits, int ctas) {
    heavy = heavy_visits;
    const int units = visits + heavy;
    blocks = min(ctas, max(1, units >> 1));
    q = units / blocks;
    r = units - q * blocks;
  }
  // first visit of block c (c <= blocks)
  __device__ __forceinline__ int first(int c) const {
    const int unit = c * q + min(c, r);
    return unit < 2 * heavy ? (unit + 1) >> 1 : unit - heavy;
  }
  // the block of visit x
  __device__ __forceinline__ int block_of(int x) const {
    const int unit = x < heavy ? 2 * x : x + heavy, k = r * (q + 1);
    return unit < k ? unit / (q + 1) : r + (unit - k) / q;
  }
};

// ------------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The instructions below are issued by the one lane with `on` set, in code that the
// whole warp runs: their operands then live in uniform registers (issued from
// code of a single lane, each took about 110 cycles to set up).
__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t on) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.u32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(r));
  return r;
}

// Shared-memory operand descriptor, 128-byte swizzle: start address, leading and
// stride byte offsets in 16-byte units, descriptor version 1.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 |
         2ull << 61;
}

// D[tmem] (+)= A[smem] B[smem], or A in TMEM.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t on) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t on) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)
      : "memory");
}

// N columns of this warp's 32 TMEM lanes: lane i of the warp holds row i.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t* r);
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t* r);
template <>
__device__ __forceinline__ void tmem_ld<8>(uint32_t t, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t t, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(t));
}
template <>
__device__ __forceinline__ void tmem_ld<32>(uint32_t t, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(t));
}
template <>
__device__ __forceinline__ void tmem_st<8>(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
template <>
__device__ __forceinline__ void tmem_st<16>(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
template <>
__device__ __forceinline__ void tmem_st<32>(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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
  const int *gpre, *lpre, *bpre;   // visits before each group's prefix (heavy, other), each row's own tokens
  const int* moff;                 // members before each group
  const uint16_t* members;
  const int *lens, *skip, *gp;     // shared memory (while planning), or NULL: from the inputs again (trees: gp stays)
  int lo, hi;                      // the block's visits
  // trees: moff has each sequence's drafts, and the segments before each, of two row tiles and of fewer rows
  const int *hseg, *lseg;
};

// One visit: a tile of a segment.
struct Visit {
  int tok0;     // its first token
  int flags;    // its tokens (1 .. 128), and the bits below
  int row;      // block-table row to read through
  int head;     // kv head
  int rows;     // query rows of the segment (up to 256)
  int q0;       // prefix: the first of them within the group
  int mem0;     // prefix: the group's first member; a row's own tokens: -1
  int rec;      // record row of the first query row
  __device__ __forceinline__ int tokens() const { return flags & 0xFF; }
  __device__ __forceinline__ bool is(int bit) const { return flags & bit; }
};
enum VisitBits {   // place in the block's part of the segment
  kFirst = 0x100, kLast = 0x200, kEarly = 0x400 /* one of the first two */, kLate = 0x800 /* of the last two */,
  kMany = 0x1000 /* the part has several */, kContinued = 0x2000 /* the segment began in an earlier block */,
  kTwo = 0x4000 /* two row tiles */,
  kDrafts = 0x8000 /* some of its tokens are drafts, which some rows do not attend to */
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

// Length of row b within the table, and the tokens it has in common with its
// group (0: it attends on its own); g: its group, -1 without.
struct RowPlan {
  int len, skip, group, bad;
};
template <class F>
__device__ __forceinline__ RowPlan row_plan(const SharedParams& p, int L, int g, F&& prefix_len) {
  RowPlan r;
  const long long cap = (long long)p.max_pages * p.page_size;
  r.bad = 0;
  if (L < 0 || L > cap) {
    r.bad |= PKV_DEV_BAD_POSITION;
    L = L < 0 ? 0 : (int)cap;
  }
  if (g < -1 || g >= p.num_groups) {
    r.bad |= PKV_DEV_BAD_GROUP;
    g = -1;
  }
  const int P = prefix_len(g);   // 0 for -1
  if (P < p.round_to || L < P) g = -1;
  r.len = L;
  r.group = g;
  r.skip = g >= 0 ? P & -p.round_to : 0;
  return r;
}

// Trees: a sequence's kv head has segments of two row tiles, and one of what is left where that is one tile. The end
// of a segment costs a block as much as some visits: in the shares every segment has that many more. (Of two row tiles with 0, 1, 2, 3, 4:
// 40 calls of 24 to 357 us drawn over types, heads and sizes take 1.008, 0.977, 0.980, 1, 1.016 times as long as with 3, by their geometric mean;
// for a single call, where a border falls makes up to a tenth either way. Of fewer rows with 0, 2, 3, 4: 8 x ~3K of 16 drafts 32.0, 29.3,
// 29.6, 29.9 us.)
constexpr int kEndHeavy = 1, kEndLight = 2;
__host__ __device__ __forceinline__ int heavy_pairs(int rows) { return (rows + kTile - 1) / (2 * kTile); }
__host__ __device__ __forceinline__ int light_pairs(int rows) { return (rows + 2 * kTile - 1) / (2 * kTile) - heavy_pairs(rows); }

// Trees of drafts: the tokens of sequence g within the table, the last `drafts` of which are drafts.
struct TreePlan {
  int len, drafts, bad;
};
__device__ __forceinline__ TreePlan tree_plan(const SharedParams& p, int g) {
  TreePlan r;
  const long long cap = (long long)p.max_pages * p.page_size;
  int L = p.seq_lens[g], n = p.draft_lens ? p.draft_lens[g] : p.drafts;
  r.bad = L < 0 || L > cap || n < 0 || n > p.drafts || n > L ? PKV_DEV_BAD_POSITION : 0;
  L = L < 0 ? 0 : (int)(L > cap ? cap : L);
  r.drafts = max(0, min(n, min(p.drafts, L)));
  r.len = r.drafts ? L : 0;   // without a draft there is nothing to do
  return r;
}

// Which of 32 tokens draft t attends to, the first of them draft j0 of its sequence (below 0: tokens
// before the drafts, to which all attend). Bits of drafts that do not exist mean nothing.
__device__ __forceinline__ uint32_t tree_bits(const SharedParams& p, const uint64_t* words, int t, int j0) {
  if (j0 <= -32) return 0xffffffffu;
  if (!words) {   // drafts up to t
    const int n = t + 1 - j0;
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  }
  const int at = max(j0, 0), w = at >> 6, s = at & 63;
  uint64_t x = w < p.mask_words ? __ldg(words + w) >> s : 0;
  if (s > 32 && w + 1 < p.mask_words) x |= __ldg(words + w + 1) << (64 - s);
  return j0 >= 0 ? (uint32_t)x : (uint32_t)x << -j0 | ((1u << -j0) - 1u);
}
__device__ __forceinline__ const uint64_t* tree_words(const SharedParams& p, int g, int t) {
  return p.tree_mask ? p.tree_mask + g * p.mask_stride + (size_t)t * p.mask_words : nullptr;
}

// The four words of a tile's 128 tokens for draft t of sequence g; the tile's first token is draft j0.
static __device__ __noinline__ uint4 tree_window(const SharedParams& p, int g, int t, int j0) {
  const uint64_t* w = tree_words(p, g, t);
  return make_uint4(tree_bits(p, w, t, j0), tree_bits(p, w, t, j0 + 32), tree_bits(p, w, t, j0 + 64),
                    tree_bits(p, w, t, j0 + 96));
}

// Which of a segment's few query rows attend to draft j of the sequence (below 0: a token before the drafts).
static __device__ __noinline__ uint32_t tree_rows(const SharedParams& p, const Visit& s, int j) {
  if (j < 0) return 0xffffffffu;
  uint32_t rows = 0;
#pragma unroll 4
  for (int i = 0; i < s.rows; ++i) {
    const int t = (s.q0 + i) / p.group;
    rows |= (tree_bits(p, tree_words(p, s.row, t), t, j) & 1u) << i;
  }
  return rows;
}

template <bool TREE>
static __device__ __noinline__ void describe_visit(const SharedParams& p, const SharedPlan& pl, int x, int4* out) {
  Visit s;
  int tile, tiles, end_tok, first_tok;
  [[maybe_unused]] int drafts = 0;
  if (TREE || x < pl.lpre[p.num_groups]) {
    const int* pre = x < pl.gpre[p.num_groups] ? pl.gpre : pl.lpre;
    const int g = upper(pre, p.num_groups, x);
    if constexpr (TREE) {
      end_tok = pl.gp[g];
      drafts = pl.moff[g];
    } else {
      end_tok = pl.gp ? pl.gp[g] : p.prefix_lens[g] & -p.round_to;
    }
    first_tok = 0;
    tiles = (end_tok + kTile - 1) / kTile;
    const int total = (TREE ? drafts : pl.moff[g + 1] - pl.moff[g]) * p.group;
    const int before = TREE && pre == pl.lpre ? heavy_pairs(total) : 0;   // pairs that are numbered elsewhere
    const int pairs = TREE ? (before || pre == pl.lpre ? 1 : heavy_pairs(total)) : (total + 2 * kTile - 1) / (2 * kTile);
    const int rem = x - pre[g], hp = rem / tiles;
    tile = rem - hp * tiles;
    s.head = hp / pairs;
    s.q0 = (hp - s.head * pairs + before) * 2 * kTile;
    s.rows = min(2 * kTile, total - s.q0);
    s.mem0 = TREE ? 0 : pl.moff[g];
    s.row = TREE ? g : pl.members[s.mem0];
    s.rec = TREE ? (g * p.num_kv_heads + s.head) * p.rec_rows + s.q0
                 : s.head * p.batch * p.group + s.mem0 * p.group + s.q0;
  } else {
    const int b = upper(pl.bpre, p.batch, x);
    if (pl.lens) {
      first_tok = pl.skip[b];
      end_tok = pl.lens[b];
    } else {
      const RowPlan r = row_plan(p, p.seq_lens[b], p.prefix_group[b], [&](int g) { return g < 0 ? 0 : p.prefix_lens[g]; });
      first_tok = r.skip;
      end_tok = r.len;
    }
    tiles = (end_tok - first_tok + kTile - 1) / kTile;
    const int rem = x - pl.bpre[b];
    s.head = rem / tiles;
    tile = rem - s.head * tiles;
    s.rows = p.group;
    s.q0 = 0;
    s.mem0 = -1;
    s.row = b;
    s.rec = ((p.num_kv_heads + s.head) * p.batch + b) * p.group;
  }
  s.tok0 = first_tok + tile * kTile;
  const int whole0 = x - tile, x0 = max(pl.lo, whole0), x1 = min(pl.hi, whole0 + tiles);
  s.flags = min(kTile, end_tok - s.tok0) | (x == x0 ? kFirst : 0) | (x == x1 - 1 ? kLast : 0) |
            (x < x0 + 2 ? kEarly : 0) | (x >= x1 - 2 ? kLate : 0) | (x1 - x0 > 1 ? kMany : 0) |
            (x0 > whole0 ? kContinued : 0) | (s.rows > kTile ? kTwo : 0);
  if (TREE && s.tok0 + kTile > end_tok - drafts) s.flags |= kDrafts;
  out[0] = make_int4(s.tok0, s.flags, s.row, s.head);
  out[1] = make_int4(s.rows, s.q0, s.mem0, s.rec);
}

// Exclusive prefix sums over the block's threads of four values (in place), and their totals.
__device__ __forceinline__ int4 block_scan4(int4& x, int threads, int4* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int4 i = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int4 y = make_int4(__shfl_up_sync(0xffffffffu, i.x, off), __shfl_up_sync(0xffffffffu, i.y, off),
                             __shfl_up_sync(0xffffffffu, i.z, off), __shfl_up_sync(0xffffffffu, i.w, off));
    if (lane >= off) i = make_int4(i.x + y.x, i.y + y.y, i.z + y.z, i.w + y.w);
  }
  if (lane == 31) scratch[warp] = i;
  __syncthreads();
  const int4 t = lane < threads / 32 ? scratch[lane] : make_int4(0, 0, 0, 0);
  const int4 b = lane < warp ? t : make_int4(0, 0, 0, 0);
  auto sum = [](int v) { return (int)__reduce_add_sync(0xffffffffu, v); };
  x = make_int4(i.x - x.x + sum(b.x), i.y - x.y + sum(b.y), i.z - x.z + sum(b.z), i.w - x.w + sum(b.w));
  return make_int4(sum(t.x), sum(t.y), sum(t.z), sum(t.w));
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
      const bool h = c >> 1;   // (see below)
      const uint32_t w[4] = {h ? v.z : v.x, h ? v.w : v.y, h ? v.x : v.z, h ? v.y : v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w4 = w[k] >> 4;
        const uint4 o = make_uint4(pair_of_nibbles<BF>(w[k], w4, 0), pair_of_nibbles<BF>(w[k], w4, 1),
                                   pair_of_nibbles<BF>(w[k], w4, 2), pair_of_nibbles<BF>(w[k], w4, 3));
        *reinterpret_cast<uint4*>(row + ((((c & 1) * 4 + (k ^ h * 2)) ^ (r & 7)) << 4)) = o;
      }
    }
  } else {
    constexpr int PER = D / 16;
#pragma unroll 4
    for (int it = 0; it < PER; ++it) {
      const int i = it * 128 + t, r = i / PER, c = i % PER;
      const uint4 v = *reinterpret_cast<const uint4*>(src + (size_t)i * 16);
      uint8_t* row = dst + (c >> 2) * 16384 + r * 128;
      // Lanes of the second half write their pieces in another order, so that eight
      // lanes reach all banks at once.
      const bool h = c >> 2;
      const uint32_t w[4] = {h ? v.z : v.x, h ? v.w : v.y, h ? v.x : v.z, h ? v.y : v.w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 o = make_uint4(pair_of_bytes<BF>(w[2 * k], 0), pair_of_bytes<BF>(w[2 * k], 2),
                                   pair_of_bytes<BF>(w[2 * k + 1], 0), pair_of_bytes<BF>(w[2 * k + 1], 2));
        *reinterpret_cast<uint4*>(row + ((((c & 3) * 2 + (k ^ h)) ^ (r & 7)) << 4)) = o;
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel
// Sum over the warp of each of v[0 .. 7], by exchanging halves: a lane ends with the
// total of one of them, `j`. Overwrites v.
__device__ __forceinline__ float scatter_sum8(float* v, int lane, int& j) {
  j = 0;
#pragma unroll
  for (int n = 4, off = 16; n > 0; n >>= 1, off >>= 1) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
    j += up ? n : 0;
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Log2 of the size of a quantised token's values, to the next whole number. Their size is that of a
// step of the codes, or of the codes' middle, where that is far above it (the codes matter less
// then). Within [-80, 122], so that weights, up to 2^15 / size, and their sums stay in fp32's range.
__device__ __forceinline__ float value_size(float step, float middle) { return fmaxf(fabsf(step), fabsf(middle) * (1.f / 128.f)); }
__device__ __forceinline__ int size_exponent(float size) {
  return min(max((int)((__float_as_uint(size) + 0x7FFFFFu) >> 23), 47), 249) - 127;
}

// Whether a phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Rest of a whole warp's bounded wait; the first warp to give up reports it
// and everyone stops. Out of line: the kernel waits in dozens of places, and its
// code has to stay small (see the softmax).
static __device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, volatile int* misc, int32_t* status) {
  const long long t0 = clock64();
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, misc[1] != 0)) return false;
    if (__any_sync(0xffffffffu, clock64() - t0 > (1ll << 31))) {
      if ((threadIdx.x & 31) == 0) {
        misc[1] = 1;
        flag_status(status, PKV_DEV_TIMEOUT);
      }
      return false;
    }
  }
}

// Queries of tile u of a segment into an operand tile (swizzled), by `warps` warps.
template <int D, bool TREE>
static __device__ __noinline__ void gather_queries(const SharedParams& p, const Visit& s, const uint16_t* members, int u,
                                                   uint32_t dst, int w, int warps) {
  constexpr int CH = D / 8, RPI = 32 / CH;   // 16-byte pieces of a row, rows an instruction
  const int lane = threadIdx.x & 31;
  const int rows = min(kTile, s.rows - u * kTile);
  if (!TREE && s.mem0 < 0) {   // one row's heads: its queries lie together
    const uint8_t* src = p.q + ((size_t)s.row * p.num_q_heads + s.head * p.group) * D * 2;
#pragma unroll 2
    for (int i = 32 * w + lane; i < rows * CH; i += 32 * warps) {
      const int r = i / CH, c = i % CH;
      cp_async16(dst + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4), src + (size_t)i * 16);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  for (int r0 = 32 * w; r0 < rows; r0 += 32 * warps) {
    // lane i finds row r0 + i
    const int R = s.q0 + u * kTile + r0 + lane, m = R / p.group, gq = R - m * p.group;
    int b = 0;
    if (r0 + lane < rows) b = TREE ? s.row * p.drafts + m : members[s.mem0 + m];
    const int qrow = b * p.num_q_heads + s.head * p.group + gq;
    const int n = min(32, rows - r0), c = lane % CH;
#pragma unroll 8
    for (int i = 0; i < 32; i += RPI) {
      if (i >= n) break;
      const int r = i + lane / CH;
      const int from = __shfl_sync(0xffffffffu, qrow, r & 31);
      if (r < n)
        cp_async16(dst + (c >> 3) * 16384 + (r0 + r) * 128 + (((c & 7) ^ (r & 7)) << 4),
                   p.q + ((size_t)from * D + c * 8) * 2);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Sums of the queries of a gathered tile, for the zero points; a warp.
template <int D, bool BF>
static __device__ __noinline__ void sum_queries(const uint8_t* src, float* qsum, int rows) {
  for (int r = threadIdx.x & 31; r < rows; r += 32) {
    float t = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const uint4 w = *reinterpret_cast<const uint4*>(src + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
      t += (low16<BF>(w.x) + high16<BF>(w.x)) + (low16<BF>(w.y) + high16<BF>(w.y)) +
           ((low16<BF>(w.z) + high16<BF>(w.z)) + (low16<BF>(w.w) + high16<BF>(w.w)));
    }
    qsum[r] = t;
  }
}

// Infinities and NaNs of a tile's row of 16-bit values become 0, the row marked (before that: another
// warp that finds the 0 finds the mark, too).
template <int HALVES, bool BF>
static __device__ __noinline__ void clear_no_numbers(uint8_t* tile, int row, volatile int* mark, int v) {
  constexpr uint32_t E = BF ? 0x7F80u : 0x7C00u;
  constexpr int HELD = 8;
  auto piece = [&](int i) {
    return reinterpret_cast<uint4*>(tile + (i >> 3) * 16384 + row * 128 + ((i & 7) ^ (row & 7)) * 16);
  };
  auto none = [](uint32_t w) { return ((w & E) == E ? 0xFFFFu : 0u) | ((w >> 16 & E) == E ? 0xFFFF0000u : 0u); };
#pragma unroll 1
  for (int i = 0; i < HALVES * 8; i += HELD) {
    uint4 x[HELD];
    bool found = false;
#pragma unroll
    for (int j = 0; j < HELD; ++j) x[j] = *piece(i + j);
#pragma unroll
    for (int j = 0; j < HELD; ++j) {   // (carries out of the exponents' places: those of none but ones)
      auto some = [](uint32_t w) { return (((w & 0x7FFF7FFFu) + ((0x8000u - E) * 0x10001u)) & 0x80008000u) != 0; };
      found |= some(x[j].x) || some(x[j].y) || some(x[j].z) || some(x[j].w);
    }
    if (!found) continue;
    *mark = v;
    __threadfence_block();
#pragma unroll 1
    for (int j = 0; j < HELD; ++j) {
      uint4* at = piece(i + j);
      const uint4 y = *at;
      *at = make_uint4(y.x & ~none(y.x), y.y & ~none(y.y), y.z & ~none(y.z), y.w & ~none(y.w));
    }
  }
  __threadfence_block();
}

// For the merge: where the records of the rows' kv heads are (the block's share of
// them), from the plan and the inputs; one warp.
static __device__ __noinline__ void place_records(const SharedParams& p, const SharedPlan& pl, int few_max) {
  const int lane = threadIdx.x & 31, Gq = p.group, B = p.batch, whole = 2 * B * p.num_q_heads;
  const Shares shares(pl.gpre[p.num_groups], pl.bpre[B], p.num_ctas);
#pragma unroll 1
  for (int i = blockIdx.x + gridDim.x * lane; i < B * p.num_kv_heads; i += gridDim.x * 32) {
    const int b = i / p.num_kv_heads, h = i - b * p.num_kv_heads;
    const RowPlan r = row_plan(p, p.seq_lens[b], p.prefix_group[b], [&](int g) { return g < 0 ? 0 : p.prefix_lens[g]; });
    auto tiles_of = [](int tokens) { return (uint32_t)(tokens + kTile - 1) / kTile; };
    // a segment's visits [x, x + n), its rows from query row `row` of its record rows `rec` on
    auto place = [&](int x, uint32_t n, int rec, int row, bool few) {
      const int c = shares.block_of(x);
      return make_int4(rec, 2 * whole + (c + 1) * 2 * kTile + row, shares.block_of(x + n - 1) - c + 1, few);
    };
    int4 own = make_int4(0, 0, 0, 0), pre = own, pre2 = own;
    uint32_t n = tiles_of(r.len - r.skip);
    if (n > 0) own = place(pl.bpre[b] + h * n, n, ((p.num_kv_heads + h) * B + b) * Gq, 0, Gq <= few_max);
    if (r.group >= 0) {
      const int g = r.group, m0 = pl.moff[g], m1 = pl.moff[g + 1], rows = (m1 - m0) * Gq;
      int lo = m0, hi = m1;   // the row among the members, which are in ascending order
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pl.members[mid] <= b) lo = mid;
        else hi = mid;
      }
      const int R = (lo - m0) * Gq, pairs = (uint32_t)(rows + 2 * kTile - 1) / (2 * kTile);
      n = tiles_of(r.skip);
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {   // a row's heads may lie in two pairs of row tiles
        const int pair = (uint32_t)(R + k * (Gq - 1)) / (2 * kTile);
        pre2 = place((rows > kTile ? pl.gpre : pl.lpre)[g] + (h * pairs + pair) * n, n, h * B * Gq + m0 * Gq + R,
                     R - pair * 2 * kTile, rows - pair * 2 * kTile <= few_max);
        if (k == 0) pre = pre2;
      }
      pre.w |= (2 * kTile - R % (2 * kTile)) << 1;   // the head from which on the second holds
    }
    p.ws_info[3 * i] = own;
    p.ws_info[3 * i + 1] = pre;
    p.ws_info[3 * i + 2] = pre2;
  }
}

// Trees: record rows of one stream, in all sequences (only few rows have records of both). An accumulator's place is [32 rows][channel][row], so that
// 32 lanes that have a row each write and read a channel together.
__host__ __device__ __forceinline__ int tree_records(const SharedParams& p) {
  return p.num_groups * p.num_kv_heads * p.rec_rows;
}

// Their shares: visits and segments' ends.
__device__ __forceinline__ Shares tree_shares(const SharedPlan& pl, int NG, int ctas) {
  const int heavy = pl.gpre[NG] + kEndHeavy * pl.hseg[NG];
  return Shares(heavy, heavy + pl.lpre[NG] - pl.gpre[NG] + kEndLight * pl.lseg[NG], ctas);
}

// The same for trees of drafts: for each sequence, kv head and pair of row tiles its record rows (of the
// first block, of those that continue it), parts and query rows, and whether both streams have a record.
static __device__ __noinline__ void place_tree_records(const SharedParams& p, const SharedPlan& pl, bool few) {
  const int lane = threadIdx.x & 31, whole = tree_records(p) << few, NG = p.num_groups;
  const Shares shares = tree_shares(pl, NG, p.num_ctas);
#pragma unroll 1
  for (int i = blockIdx.x + gridDim.x * lane; i < NG * p.num_kv_heads * p.pairs; i += gridDim.x * 32) {
    const int gh = i / p.pairs, pair = i - gh * p.pairs, g = gh / p.num_kv_heads, h = gh - g * p.num_kv_heads;
    const int rows = pl.moff[g] * p.group, heavy = heavy_pairs(rows);
    const int n = (int)((uint32_t)(pl.gp[g] + kTile - 1) / kTile), mine = min(2 * kTile, rows - pair * 2 * kTile);
    int4 info = make_int4(0, 0, 0, 0);
    if (mine > 0) {
      // the segment's first visit, counted with the segments' ends
      const int x = pair < heavy ? pl.gpre[g] + kEndHeavy * pl.hseg[g] + (h * heavy + pair) * (n + kEndHeavy)
                                 : pl.lpre[g] + kEndHeavy * pl.hseg[NG] + kEndLight * pl.lseg[g] + h * (n + kEndLight);
      const int c = shares.block_of(x);
      info = make_int4(gh * p.rec_rows + pair * 2 * kTile, whole + (c + 1) * 2 * kTile,
                       (shares.block_of(x + n - 1) - c + 1) | mine << 16, few);
    }
    p.ws_info[i] = info;
  }
}

// What a kernel serves. Trees have one for calls of few query rows, where a segment's rows never exceed FEW, and
// one for the others: half the code and fewer registers (one for both: 8 x ~3K of 16 drafts 32 us, 24 x ~6K of 64 157, the tree of
// 5 x ~800 in 4 bits 16; two: 29, 152, 11).
enum SharedMode { kPrefixes = 0, kFewDrafts = 1, kDraftRows = 2 };

template <int D, int KV, bool BF, int MODE>
__global__ void __launch_bounds__(SharedGeom<D, KV, BF>::THREADS, 1)
    shared_attention_kernel(const __grid_constant__ SharedParams p) {
  using G = SharedGeom<D, KV, BF>;
  constexpr bool QUANT = G::QUANT, TREE = MODE != kPrefixes;
  constexpr int NT = G::THREADS, COLS = QUANT ? 32 : 64;   // columns of a pass over the scores
  constexpr int FEW = G::FEW;
  // whether a segment of so many rows runs transposed, and whether it has two row tiles
  auto is_few = [](int rows) { return MODE == kFewDrafts || (MODE == kPrefixes && rows <= FEW); };
  auto is_two = [](int rows) { return MODE != kFewDrafts && rows > kTile; };
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const SharedLayout& lay = p.lay;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bars = smem_u32(smem + lay.bars);
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  volatile int* misc = reinterpret_cast<volatile int*>(smem + lay.misc);   // [0] TMEM base, [1] gave up
  int4* scratch = reinterpret_cast<int4*>(smem + lay.misc) + 1;
  int* lens = reinterpret_cast<int*>(smem + lay.lens);
  int* skip = reinterpret_cast<int*>(smem + lay.skip);
  int4* visits = reinterpret_cast<int4*>(smem + lay.visits);
  int* bpre = reinterpret_cast<int*>(smem + lay.bpre);
  int* gpre = reinterpret_cast<int*>(smem + lay.gpre);
  int* gp = reinterpret_cast<int*>(smem + lay.gp);
  int* moff = reinterpret_cast<int*>(smem + lay.moff);
  uint16_t* members = reinterpret_cast<uint16_t*>(smem + lay.members);
  int* lpre = reinterpret_cast<int*>(smem + lay.lpre);
  [[maybe_unused]] int* hseg = reinterpret_cast<int*>(smem + lay.hseg);   // trees
  [[maybe_unused]] int* lseg = reinterpret_cast<int*>(smem + lay.lseg);
  uint16_t* rank = reinterpret_cast<uint16_t*>(smem + lay.rank);
  int16_t* rowg = reinterpret_cast<int16_t*>(smem + lay.rowg);
  // (trees of drafts: the groups are all there is)
  const int S = p.entries, B = TREE ? 0 : p.batch, NG = p.num_groups, Gq = p.group;

  if (tid == 0) {
    for (int i = 0; i < kMaxEntries; ++i) {
      mbar_init(bar(kBarKFull + i), 1);
      mbar_init(bar(kBarVFull + i), 1);
      mbar_init(bar(kBarKEmpty + i), QUANT ? 4 : 1);
      mbar_init(bar(kBarVEmpty + i), QUANT ? 4 : 1);
    }
    for (int i = 0; i < kHdrs; ++i) mbar_init(bar(kBarHdr + i), QUANT ? 4 : 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarQFull + i), 1);
      mbar_init(bar(kBarQEmpty + i), 1);
      mbar_init(bar(kBarQLoad + i), 1);
      mbar_init(bar(kBarS + i), 1);
      mbar_init(bar(kBarP + i), 4);
      mbar_init(bar(kBarO + i), 1);
    }
    mbar_init(bar(kBarKop), 4);        // converted K ready / free again
    mbar_init(bar(kBarKop + 1), 1);
    mbar_init(bar(kBarVop), 4);
    mbar_init(bar(kBarVop + 1), 1);
    for (int i = 0; i < 4; ++i) mbar_init(bar(kBarPair + i), 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarVisits + i), 1);
      mbar_init(bar(kBarPassed + i), QUANT ? 19 : 11);   // loaders, MMA, softmax, converters
    }
    mbar_init(bar(kBarEnd), 1);
    misc[1] = 0;
  }
  fence_mbar_init();
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(smem + lay.misc))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  for (int g = tid; g < NG; g += NT) moff[g] = 0;
  pdl_wait();
  pdl_launch_dependents();

  // ---- plan: lengths, who shares, visits before each segment. (Its loops stay
  // loops: this code is fetched anew by every call.)
  SharedPlan plan = {gpre, lpre, bpre, moff, members, lens, skip, gp, 0, 0, hseg, lseg};
  auto tiles_of = [](int tokens) { return (uint32_t)(tokens + kTile - 1) / kTile; };
  int lo = 0, hi = 0;
  // trees: a sequence's segments of fewer rows, visits of two row tiles, other visits, segments of two row tiles
  [[maybe_unused]] auto tree_counts = [&](int rows, int tiles) {
    const int h = tiles ? p.num_kv_heads * heavy_pairs(rows) : 0, l = tiles ? p.num_kv_heads * light_pairs(rows) : 0;
    return make_int4(l, h * tiles, l * tiles, h);
  };
  // the visit at a border of the shares that lies among `n` segments, `at` from their first; -1: it lies elsewhere
  [[maybe_unused]] auto visit_at = [](int at, int n, int tiles, int end, int first) {
    return at >= 0 && at < n * (tiles + end) ? first + at / (tiles + end) * tiles + min(at % (tiles + end), tiles) : -1;
  };
  if constexpr (TREE && !QUANT) {   // no visit's marks
    for (int i = tid; i < kBadSlots * kTile; i += NT) reinterpret_cast<int*>(smem + lay.bad)[i] = -1;
  }
  if (TREE && NG <= 32) {
    // few sequences: a lane each, in every warp, without a wait in between
    TreePlan r = {0, 0, 0};
    if (lane < NG) r = tree_plan(p, lane);
    const int tiles = tiles_of(r.len);
    const int4 mine = tree_counts(r.drafts * Gq, tiles);
    int4 e = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int4 y = make_int4(__shfl_up_sync(0xffffffffu, e.x, off), __shfl_up_sync(0xffffffffu, e.y, off),
                               __shfl_up_sync(0xffffffffu, e.z, off), __shfl_up_sync(0xffffffffu, e.w, off));
      if (lane >= off) e = make_int4(e.x + y.x, e.y + y.y, e.z + y.z, e.w + y.w);
    }
    const int4 all = make_int4(__shfl_sync(0xffffffffu, e.x, 31), __shfl_sync(0xffffffffu, e.y, 31),
                               __shfl_sync(0xffffffffu, e.z, 31), __shfl_sync(0xffffffffu, e.w, 31));
    e = make_int4(e.x - mine.x, e.y - mine.y, e.z - mine.z, e.w - mine.w);
    if (warp == 0) {
      if (r.bad && blockIdx.x == 0) flag_status(p.dev_status, r.bad);
      if (lane < NG) {
        moff[lane] = r.drafts;
        gp[lane] = r.len;
        gpre[lane] = e.y;
        lpre[lane] = all.y + e.z;
        hseg[lane] = e.w;
        lseg[lane] = e.x;
      }
      if (lane == 0) {
        gpre[NG] = all.y;
        lpre[NG] = all.y + all.z;
        hseg[NG] = all.w;
        lseg[NG] = all.x;
      }
    }
    const int heavy = all.y + kEndHeavy * all.w, total = all.y + all.z;
    const Shares shares(heavy, heavy + all.z + kEndLight * all.x, p.num_ctas);
    auto border = [&](int c) {
      const int x = shares.first(c);
      const int v = __reduce_max_sync(0xffffffffu, max(visit_at(x - e.y - kEndHeavy * e.w, mine.w, tiles, kEndHeavy, e.y),
                                                       visit_at(x - heavy - e.z - kEndLight * e.x, mine.x, tiles, kEndLight,
                                                                all.y + e.z)));
      return v < 0 ? total : v;
    };
    if ((int)blockIdx.x < shares.blocks && total > 0) {
      lo = border(blockIdx.x);
      hi = border(blockIdx.x + 1);
    }
    __syncthreads();
  } else {
  if constexpr (TREE) {
#pragma unroll 1
    for (int g = tid; g < NG; g += NT) {
      const TreePlan r = tree_plan(p, g);
      if (r.bad && blockIdx.x == 0) flag_status(p.dev_status, r.bad);
      moff[g] = r.drafts;
      gp[g] = r.len;
    }
    __syncthreads();
  } else {
    const int lens32 = lane < NG ? p.prefix_lens[lane] : 0;   // of the first 32 groups
#pragma unroll 1
    for (int b0 = warp * 32; b0 < B; b0 += NT) {
      const int b = b0 + lane;
      const RowPlan r = row_plan(p, b < B ? p.seq_lens[b] : 0, b < B ? p.prefix_group[b] : -1, [&](int g) {
        if (NG > 32) return g < 0 ? 0 : p.prefix_lens[g];
        const int P = __shfl_sync(0xffffffffu, lens32, g & 31);
        return g < 0 ? 0 : P;
      });
      if (b >= B) continue;
      if (r.bad && blockIdx.x == 0) flag_status(p.dev_status, r.bad);
      lens[b] = r.len;
      skip[b] = r.skip;
      rowg[b] = (int16_t)r.group;
    }
#pragma unroll 1
    for (int g = tid; g < NG; g += NT) {
      const int P = g < 32 ? lens32 : p.prefix_lens[g];
      if (P < 0 && blockIdx.x == 0) flag_status(p.dev_status, PKV_DEV_BAD_GROUP);
      gp[g] = max(P, 0) & -p.round_to;
    }
    __syncthreads();
    if (warp == 0 && NG > 0) {   // each row's place among its group's rows
#pragma unroll 1
      for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane, g = b < B ? rowg[b] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, g);
        const int base = g >= 0 ? moff[g] : 0;
        __syncwarp();
        if (g >= 0 && lane == __ffs(same) - 1) moff[g] = base + __popc(same);
        __syncwarp();
        if (b < B) rank[b] = (uint16_t)(base + __popc(same & ((1u << lane) - 1)));
      }
    }
    __syncthreads();
  }
  // kv heads x pairs of row tiles x tiles of tokens
  auto prefix_visits = [&](int g) {
    return moff[g] == 0 ? 0 : (int)(p.num_kv_heads * ((uint32_t)(moff[g] * Gq + 2 * kTile - 1) / (2 * kTile)) * tiles_of(gp[g]));
  };
  // each thread's share of the groups and rows: members, heavy visits, other
  // prefix visits, visits of the rows' own tokens
  const int per_g = (NG + NT - 1) / NT, per_b = (B + NT - 1) / NT;
  const int ga = min(NG, tid * per_g), ge = min(NG, ga + per_g), ba = min(B, tid * per_b), be = min(B, ba + per_b);
  int4 run = make_int4(0, 0, 0, 0);
  [[maybe_unused]] auto count_tree = [&](int g) {
    const int4 n = tree_counts(moff[g] * Gq, tiles_of(gp[g]));
    run = make_int4(run.x + n.x, run.y + n.y, run.z + n.z, run.w + n.w);
  };
#pragma unroll 1
  for (int g = ga; g < ge; ++g) {
    if constexpr (TREE) {
      count_tree(g);
      continue;
    }
    const int n = prefix_visits(g);
    run.x += moff[g];
    (moff[g] * Gq > kTile ? run.y : run.z) += n;
  }
#pragma unroll 1
  for (int b = ba; b < be; ++b) run.w += p.num_kv_heads * tiles_of(lens[b] - skip[b]);
  const int4 all = block_scan4(run, NT, scratch);
#pragma unroll 1
  for (int g = ga; g < ge; ++g) {
    gpre[g] = run.y;
    lpre[g] = all.y + run.z;
    if constexpr (TREE) {
      hseg[g] = run.w;
      lseg[g] = run.x;
      count_tree(g);
      continue;
    }
    const int n = prefix_visits(g), c = moff[g];
    moff[g] = run.x;
    run.x += c;
    (c * Gq > kTile ? run.y : run.z) += n;
  }
#pragma unroll 1
  for (int b = ba; b < be; ++b) {
    bpre[b] = all.y + all.z + run.w;
    run.w += p.num_kv_heads * tiles_of(lens[b] - skip[b]);
  }
  if (tid == 0) {
    gpre[NG] = all.y;
    lpre[NG] = all.y + all.z;
    if constexpr (TREE) {
      hseg[NG] = all.w;
      lseg[NG] = all.x;
    } else {
      moff[NG] = all.x;
      bpre[B] = all.y + all.z + all.w;
    }
  }
  __syncthreads();
  const int total = all.y + all.z + (TREE ? 0 : all.w);   // visits
  const Shares shares = TREE ? tree_shares(plan, NG, p.num_ctas) : Shares(all.y, total, p.num_ctas);
#pragma unroll 1
  for (int b = tid; b < B; b += NT)
    if (rowg[b] >= 0) members[moff[rowg[b]] + rank[b]] = (uint16_t)b;
  const bool idle = (int)blockIdx.x >= shares.blocks || total == 0;
  lo = idle ? 0 : shares.first(blockIdx.x);
  hi = idle ? 0 : shares.first(blockIdx.x + 1);
  if constexpr (TREE) {
    // from the count with the segments' ends to that of the visits: the sequence within which a border lies finds it
    volatile int* range = reinterpret_cast<volatile int*>(scratch);
    if (tid < 2) range[tid] = idle ? 0 : total;   // (where no sequence does)
    __syncthreads();
#pragma unroll 1
    for (int g = tid; g < NG; g += NT) {
      const int tiles = tiles_of(gp[g]), hl = hseg[NG] * kEndHeavy;
#pragma unroll 1
      for (int i = 0; i < 4 && !idle && tiles; ++i) {
        const bool light = i & 1;
        const int end = light ? kEndLight : kEndHeavy, seg = light ? lseg[g] : hseg[g];
        const int n = (light ? lseg[g + 1] : hseg[g + 1]) - seg, real = light ? lpre[g] : gpre[g];
        const int v = visit_at((i < 2 ? lo : hi) - (real + (light ? hl : 0) + end * seg), n, tiles, end, real);
        if (v >= 0) range[i >> 1] = v;
      }
    }
    __syncthreads();
    lo = range[0];
    hi = range[1];
  }
  __syncthreads();
  }
  const int nv = hi - lo;
  plan.lo = lo;
  plan.hi = hi;
  if (tid < min(nv, kVisits)) describe_visit<TREE>(p, plan, lo + tid, visits + 2 * tid);
  plan.lens = plan.skip = nullptr;
  if constexpr (!TREE) plan.gp = nullptr;
  fence_proxy_async_smem();   // the ring, so far the plan's, is the copies' from here on
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, (uint32_t)misc[0], 0);
  auto records = [&]() {
    if constexpr (TREE) place_tree_records(p, plan, MODE == kFewDrafts);
    else place_records(p, plan, FEW);
  };
  if (nv <= 0) {   // uniform over the block
    if (warp == 8) records();
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    return;
  }
  // a stream's scores (and weights over them), and its accumulator
  auto tm_s = [&](int st) { return tmem + 128u * (uint32_t)st; };
  auto tm_o = [&](int st) { return tmem + 256u + (uint32_t)(D * st); };

  // for a whole warp: every lane goes on, or none does
  auto wait_warp = [&](int i, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar(i), parity))) return true;
    return wait_longer(bar(i), parity, misc, p.dev_status);
  };
  // visit v of the block; its description may have to be waited for
  auto described = [&](int v) -> bool {
    return v < kVisits || (v & (kVisits / 2 - 1)) != 0 ||
           wait_warp(kBarVisits + (v / (kVisits / 2) & 1), (v / kVisits - 1) & 1);
  };
  auto visit = [&](int v, Visit& d) -> bool {
    if (!described(v)) return false;
    const int4 a = visits[2 * (v & (kVisits - 1))], b = visits[2 * (v & (kVisits - 1)) + 1];
    d = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    return true;
  };
  auto flags_of = [&](int v) { return visits[2 * (v & (kVisits - 1))].y; };
  // this warp needs visit v and those before it no more
  auto passed = [&](int v) {
    if ((v & (kVisits / 2 - 1)) == kVisits / 2 - 1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarPassed + (v / (kVisits / 2) & 1)));
    }
  };
  auto gather_q = [&](const Visit& s, int u, int qs, int w, int warps) {
    gather_queries<D, TREE>(p, s, members, u, smem_u32(smem + lay.q) + (uint32_t)qs * G::OPERAND, w, warps);
  };
  auto sum_q = [&](const Visit& s, int u, int qs, int slot) {
    sum_queries<D, BF>(smem + lay.q + (size_t)qs * G::OPERAND,
                       reinterpret_cast<float*>(smem + lay.qsum) + slot * kTile, min(kTile, s.rows - u * kTile));
  };

  // the first segment's queries, by the warps that have nothing else to do yet
  Visit first;
  visit(0, first);
  const int first_tiles = first.rows > kTile ? 2 : 1;
  const bool copied_q = TREE && p.q_box;   // queries come by tensor copies, issued by warp 10
  if (copied_q) {
  } else if (warp < 8) {
    for (int u = 0; u < first_tiles; ++u) gather_q(first, u, u, warp, 8);
    fence_proxy_async_smem();
    named_bar_sync(1, 288);
  } else if (warp == 10) {
    named_bar_sync(1, 288);
    if constexpr (QUANT) {
      for (int u = 0; u < first_tiles; ++u) sum_q(first, u, u, u);
      __syncwarp();
    }
    if (lane == 0)
      for (int u = 0; u < first_tiles; ++u) mbar_arrive(bar(kBarQFull + u));
  }

  if (warp == 8 || warp == 11) {
    // =============================================== loaders: K (8) and V (11)
    const bool isv = warp == 11;
    const uint64_t pol = policy_evict_first();
    constexpr int PARTS = QUANT ? 1 : G::HALVES;   // boxes side by side in a row
    const int piece = lane / PARTS, half = lane % PARTS;
    const int fulls = isv ? kBarVFull : kBarKFull, empties = isv ? kBarVEmpty : kBarKEmpty;
    uint8_t* ring = smem + lay.ring + (isv ? (size_t)S * G::ENTRY : 0);
    const uint8_t* pool = isv ? p.v_pages : p.k_pages;
    const void* map = isv ? &p.tmap_v : &p.tmap_k;
    // Block-table entries of four visits at a time, a batch ahead: lane 8 j + i has piece
    // i (16 tokens) of visit j of the batch. Its pool row, or -1 for none.
    int page = 0, base = 0, tok = 0;   // of the next batch, the load on its way
    auto fetch = [&](int v0) -> bool {
      if (v0 < nv && !described(v0)) return false;
      const int v = v0 + (lane >> 3), i = lane & 7;
      page = -2;
      if (v < nv) {
        const int4 d = visits[2 * (v & (kVisits - 1))];
        if (16 * i < (d.y & 0xFF)) {
          tok = d.x + 16 * i;
          base = d.w;
          page = p.block_table[(size_t)d.z * p.max_pages + tok / p.page_size];
        }
      }
      return true;
    };
    int v = 0;
    bool ok = fetch(0);
    RingPos pos;
    for (int v0 = 0; v0 < nv && ok; v0 += 4) {
      const bool good = page >= 0 && page < p.num_pages;
      if (page != -2 && !good && !isv) flag_status(p.dev_status, PKV_DEV_BAD_PAGE);
      // (the host keeps pool rows below 2^31)
      const int rows4 = good ? (page * p.num_kv_heads + base) * p.page_size + tok % p.page_size : -1;
      const unsigned have = __ballot_sync(0xffffffffu, good);
      const int n = min(4, nv - v0);
      // descriptions of the next four visits may themselves still be on their
      // way behind these
      const bool wait_later = ((v0 + 4) & (kVisits / 2 - 1)) == 0;
      int lens4 = 0;
      if (!isv && lane < n) lens4 = visits[2 * ((v0 + lane) & (kVisits - 1))].y & 0xFF;
      if (wait_later) passed(v0 + 3);
      if (!wait_later) fetch(v0 + 4);
      for (int j = 0; j < n; ++j, ++v, pos.next(S)) {
        const uint32_t mask = have >> (8 * j) & 0xFFu;   // bit i: piece i is copied
        const int row = __shfl_sync(0xffffffffu, rows4, 8 * j + (piece & 7));
        const int ntok = __shfl_sync(0xffffffffu, lens4, j);
        const int slot = pos.slot;
        ok = v < S || wait_warp(empties + slot, pos.phase ^ 1);
        if (!ok) break;
        const uint32_t fb = bar(fulls + slot);
        if (lane == 0) {
          if (!isv) *reinterpret_cast<int2*>(smem + lay.hdr + (v % kHdrs) * 8) = make_int2(ntok, (int)mask);
          uint32_t bytes = (uint32_t)__popc(mask) * 16u * G::ROW;
          if constexpr (KV == KV_I8T || KV == KV_U4T) bytes += !isv ? (uint32_t)__popc(mask) * 256u : 0u;
          if constexpr (KV == KV_I8G) bytes += !isv ? (uint32_t)((mask & 0xF ? 16 : 0) + (mask & 0xF0 ? 16 : 0)) : 0u;
          if (bytes)
            mbar_arrive_expect_tx(fb, bytes);
          else
            mbar_arrive(fb);
          if (!QUANT && !isv) mbar_arrive(bar(kBarHdr + v % kHdrs));
        }
        __syncwarp();
        if (piece < 8 && row >= 0) {
          uint8_t* dst = ring + (size_t)slot * G::ENTRY;
          if constexpr (!QUANT) {
            tma_load_2d(smem_u32(dst + half * 16384 + piece * 2048), map, half * 64, row, fb, pol);
          } else {
            bulk_g2s(smem_u32(dst + piece * 16 * G::ROW), pool + (size_t)row * G::ROW, 16 * G::ROW, fb, pol);
            if (!isv) {
              uint8_t* raw = smem + lay.raw + (size_t)slot * G::RAW_SCALES;
              if constexpr (KV != KV_I8G) {
                bulk_g2s(smem_u32(raw + piece * 256), p.kv_sz + (size_t)row * 4, 256, fb, pol);
              } else if ((mask & ((1u << piece) - 1) & (piece < 4 ? 0xFu : 0xF0u)) == 0) {
                // the first copied piece of a 64-token group brings its scales
                bulk_g2s(smem_u32(raw + (piece >> 2) * 16), p.kv_sz + (size_t)(row / 64) * 4, 16, fb, pol);
              }
            }
          }
        }
        __syncwarp();
      }
      if (ok && wait_later) ok = fetch(v0 + 4);
    }
    // every issued copy lands before the block can end
    if (lane == 0)
      for (int e = v > S ? v - S : 0; e < v; ++e)
        if (!mbar_wait_bounded(bar(fulls + e % S), (e / S) & 1)) break;
    __syncwarp();
  } else if (warp == 9) {
    // =================================================================== MMA
    {
      const uint32_t on = elect_one();
      auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      constexpr uint32_t kType = 1u << 4 | (BF ? (1u << 7 | 1u << 10) : 0u) | 8u << 24;   // fp32 sums, M = 128
      const uint64_t kmajor = operand_desc(0, 16, 1024), vmajor = operand_desc(0, D == 128 ? 16384 : 0, 1024);
      const uint64_t pmajor = (uint64_t)(128 >> 4) << 16 | (uint64_t)(2048 >> 4) << 32 | 1ull << 46;   // no swizzle
      auto at = [](uint64_t d, uint32_t addr) { return d | (uint64_t)(addr >> 4); };
      const uint32_t qb = smem_u32(smem + lay.q), ring = smem_u32(smem + lay.ring), pt = smem_u32(smem + lay.pt);
      const uint32_t kop = smem_u32(smem + lay.kop), vop = smem_u32(smem + lay.vop);
      uint32_t odd = 0;         // bit st: parity of the events so far on stream st
      uint32_t vop_phase = 0;   // uses of the converted V tile
      int qc = 0, v = 0, u = 0;
      RingPos pos;
      // the event whose P V product is still to be issued
      struct { int st, steps; RingPos at; bool on, few, fresh, last_use, seg_end; } pend = {};
      const int end = uni(nv);
      bool ok = true, begun = false;
      int rows = 0, flags = 0;
      // Each pass issues the scores of the next event (visit v, row tile u),
      // then the P V product of the one before. Normally the streams
      // alternate; where they do not, the scores wait for a pass of their own,
      // so that none is overwritten before the weights in it are used.
      while (ok && (v < end || pend.on)) {
        if (v < end && !begun) {
          Visit d;
          ok = visit(v, d);
          if (!ok) break;
          rows = uni(d.rows);
          flags = uni(d.flags);
          if constexpr (MODE == kDraftRows) {
            // Whole tiles within a segment, without what its ends need. The order is that of the passes below, but
            // a pass is P V of an event and S of the stream's next one: between the weights' arrival and the next
            // scores lie just these products, everything else is done behind them or while the weights
            // are being made. (This warp's instructions are slow, fetched anew between those of the softmax.)
            // With one row tile the scores of v go out before V of v - 2 is given back, which a ring of a single entry does not
            // allow: the softmax takes the scores of v as the sign that it is (see begin below).
            const bool two = is_two(rows);
            const int inside = (two ? kFirst | kLast : kEarly | kLate) | 0xFF;
            if ((QUANT || S > 1) && pend.on && !p.two_terms && (flags & inside) == kTile) {
              const uint32_t hi_k = (uint32_t)(kmajor >> 32), hi_v = (uint32_t)(vmajor >> 32), lo_v = (uint32_t)vmajor;
              constexpr uint32_t is = kType | (uint32_t)(kTile / 8) << 17, io = kType | 1u << 16 | (uint32_t)(D / 8) << 17;
              auto desc = [](uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; };
              auto k_there = [&]() { return QUANT ? wait_warp(kBarKop, v & 1) : wait_warp(kBarKFull + pos.slot, pos.phase); };
              uint32_t acc = !pend.fresh;                // of the first P V to come
              RingPos last = pend.at, before_last = {};  // of the visits before v
              bool pv = false, more = true;
              ok = k_there();
              while (ok) {
                const int ms = two ? u : v & 1;
                if (pv) {
                  const RingPos at = two ? last : before_last;
                  if (!two || ms == 0) {   // (otherwise V is known to be there)
                    ok = QUANT ? wait_warp(kBarVop, vop_phase) : wait_warp(kBarVFull + at.slot, at.phase);
                    if (!ok) break;
                  }
                  const uint32_t vlo = lo_v | (QUANT ? vop : ring + (uint32_t)(S + at.slot) * G::ENTRY) >> 4;
                  ok = wait_warp(kBarP + ms, ~(odd >> ms) & 1);
                  if (!ok) break;
                  tc_after();
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    mma_ts(tm_o(ms), tm_s(ms) + 32 * (j >> 1) + 8 * (j & 1), desc(vlo + j * 128, hi_v), io, j > 0 ? 1 : acc, on);
                  acc = 1;
                }
                if (more) {
                  if (QUANT && u == 0 && pv) {   // (the next K is converted once the last S is done: not before P V)
                    ok = k_there();
                    if (!ok) break;
                  }
                  const uint32_t klo = (uint32_t)kmajor | (QUANT ? kop : ring + (uint32_t)pos.slot * G::ENTRY) >> 4;
                  const uint32_t qlo = (uint32_t)kmajor | (qb + (uint32_t)((qc + u) & 1) * G::OPERAND) >> 4;
                  tc_after();
#pragma unroll
                  for (int k = 0; k < D / 16; ++k)
                    mma_ss(tm_s(ms), desc(qlo + (k >> 2) * 1024 + (k & 3) * 2, hi_k),
                           desc(klo + (k >> 2) * 1024 + (k & 3) * 2, hi_k), is, k > 0, on);
                  tc_commit(bar(kBarS + ms), on);
                }
                if (pv && (!two || ms == 1)) {
                  tc_commit(QUANT ? bar(kBarVop + 1) : bar(kBarVEmpty + (two ? last : before_last).slot), on);
                  vop_phase ^= 1;
                }
                if (!more) break;
                pv = true;
                odd ^= 1u << ms;
                if (two && u == 0) {
                  u = 1;
                  continue;
                }
                tc_commit(QUANT ? bar(kBarKop + 1) : bar(kBarKEmpty + pos.slot), on);
                u = 0;
                before_last = last;
                last = pos;
                passed(v);
                ++v;
                pos.next(S);
                ok = described(v);
                if (!ok) break;
                flags = uni(flags_of(v));
                more = (flags & inside) == kTile;
                if (more && !QUANT) ok = k_there();
              }
              if (!ok) break;
              pend.st = two ? 1 : (v - 1) & 1;
              pend.at = last;
              pend.fresh = false;
            }
          }
          ok = QUANT ? wait_warp(kBarKop, v & 1) : wait_warp(kBarKFull + pos.slot, pos.phase);
          if (!ok) break;
          begun = true;
        }
        const bool two = is_two(rows);
        const int st = two ? u : v & 1;
        const int qt = qc + (two ? u : 0), qs = qt & 1;
        // queries still on their way hold up no product that could go ahead
        const bool scores =
            v < end && !(pend.on && (pend.st == st || (flags & kFirst &&
                                                       !__all_sync(0xffffffffu, mbar_test(bar(kBarQFull + qs), (qt >> 1) & 1)))));
        const bool few = is_few(rows);
        const bool last_s = !two || u == 1;
        if (scores) {
          if (flags & kFirst) ok = wait_warp(kBarQFull + qs, (qt >> 1) & 1);
          if (!ok) break;
          tc_after();
          const uint64_t kd = at(kmajor, QUANT ? kop : ring + (uint32_t)pos.slot * G::ENTRY);
          const uint64_t qd = at(kmajor, qb + (uint32_t)qs * G::OPERAND);
          // S = Q K^T, rows x tokens; few rows: S^T = K Q^T, tokens x rows
          const uint64_t ad = few ? kd : qd, bd = few ? qd : kd;
          const uint32_t idesc = kType | (uint32_t)(few ? 16 / 8 : kTile / 8) << 17;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tm_s(st), ad + (k >> 2) * 1024 + (k & 3) * 2, bd + (k >> 2) * 1024 + (k & 3) * 2, idesc, k > 0, on);
          tc_commit(bar(kBarS + st), on);
          if (last_s) tc_commit(QUANT ? bar(kBarKop + 1) : bar(kBarKEmpty + pos.slot), on);
          if (flags & kLast) tc_commit(bar(kBarQEmpty + qs), on);
        }
        if (pend.on) {
          const int ps = pend.st, slot = pend.at.slot;
          ok = wait_warp(kBarP + ps, ~(odd >> ps) & 1);
          if (!ok) break;
          ok = QUANT ? wait_warp(kBarVop, vop_phase) : wait_warp(kBarVFull + slot, pend.at.phase);
          if (!ok) break;
          tc_after();
          const uint64_t vd = at(vmajor, QUANT ? vop : ring + (uint32_t)(S + slot) * G::ENTRY);
          const uint32_t o = tm_o(ps);
          uint32_t acc = !pend.fresh;
          if (MODE == kFewDrafts || (MODE == kPrefixes && pend.few)) {
            // O^T (+)= V^T [P1^T | P2^T]: channels x rows, first and second terms of
            // the weights side by side
            constexpr uint32_t idesc = kType | 1u << 15 | 1u << 16 | (uint32_t)(2 * FEW / 8) << 17;
            const uint64_t pd = at(pmajor, pt + (uint32_t)ps * G::PT);
            // (without a condition in between: with one, the products went out 100 cycles apart)
            auto step = [&](int j) { mma_ss(o, vd + j * 128, pd + j * 16, idesc, acc, on); };
            if (pend.steps == 8) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                step(j);
                acc = 1;
              }
            } else {
#pragma unroll 1
              for (int j = 0; j < pend.steps; ++j) {
                step(j);
                acc = 1;
              }
            }
          } else {
            constexpr uint32_t idesc = kType | 1u << 16 | (uint32_t)(D / 8) << 17;
            auto step = [&](uint32_t a, int j) { mma_ts(o, a + 32 * (j >> 1) + 8 * (j & 1), vd + j * 128, idesc, acc, on); };
#pragma unroll 1
            for (uint32_t a = tm_s(ps), last = a + (p.two_terms ? 16 : 0); a <= last; a += 16) {
              if (pend.steps == 8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  step(a, j);
                  acc = 1;
                }
              } else {
#pragma unroll 1
                for (int j = 0; j < pend.steps; ++j) {
                  step(a, j);
                  acc = 1;
                }
              }
            }
          }
          if (pend.last_use) {
            tc_commit(QUANT ? bar(kBarVop + 1) : bar(kBarVEmpty + slot), on);
            vop_phase ^= 1;
          }
          if (pend.seg_end) tc_commit(bar(kBarO + ps), on);
          pend.on = false;
        }
        if (scores) {
          odd ^= 1u << st;
          pend.st = st;
          pend.at = pos;
          pend.steps = ((flags & 0xFF) + 15) >> 4;
          pend.few = few;
          pend.on = true;
          pend.fresh = flags & (two ? kFirst : kEarly);
          pend.last_use = last_s;
          pend.seg_end = flags & (two ? kLast : kLate);
          if (last_s) {
            if (flags & kLast) qc += two ? 2 : 1;
            passed(v);
            ++v;
            pos.next(S);
            u = 0;
            begun = false;
          } else {
            u = 1;
          }
        }
      }
      // nothing of the tensor cores is in flight past this point
      tc_commit(bar(kBarEnd), on);
      if (!mbar_wait_bounded(bar(kBarEnd), 0) && lane == 0) flag_status(p.dev_status, PKV_DEV_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ============================== Q gather, from the second segment on (copies: from the first)
    int qc = copied_q ? 0 : first_tiles;
    bool ok = true, placed = false;
    for (int v = copied_q ? 0 : 1; v < nv && ok; ++v) {
      if (v >= kVisits && (v & (kVisits / 2 - 1)) == 0) {
        // the next half of the visits' descriptions, once the last use of their place is over
        const int h = v / (kVisits / 2) & 1;
        ok = wait_warp(kBarPassed + h, (v / kVisits - 1) & 1);
        if (!ok) break;
        for (int i = v + lane; i < min(nv, v + kVisits / 2); i += 32)
          describe_visit<TREE>(p, plan, lo + i, visits + 2 * (i & (kVisits - 1)));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarVisits + h));
      }
      const int4 a = visits[2 * (v & (kVisits - 1))], b = visits[2 * (v & (kVisits - 1)) + 1];
      const Visit s = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      if (!s.is(kFirst)) continue;
      const int tiles = s.rows > kTile ? 2 : 1;
      for (int u = 0; u < tiles && ok; ++u, ++qc) {
        const int qs = qc & 1;
        if (qc >= 2 && !placed) {   // both tiles are in use: time for this
          records();
          placed = true;
        }
        if (qc >= 2) ok = wait_warp(kBarQEmpty + qs, ((qc >> 1) - 1) & 1);
        if (!ok) break;
        if (copied_q) {
          const uint32_t full = bar((QUANT ? kBarQLoad : kBarQFull) + qs);
          if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(G::HALVES * 128 * Gq) * (uint32_t)p.q_box);
          __syncwarp();
          if (lane < G::HALVES)
            tma_load_3d(smem_u32(smem + lay.q) + (uint32_t)qs * G::OPERAND + (uint32_t)lane * 16384u, &p.tmap_q, lane * 64,
                        s.head * Gq, s.row * p.drafts + (s.q0 + u * kTile) / Gq, full);
          __syncwarp();
          if constexpr (QUANT) {
            ok = wait_warp(kBarQLoad + qs, (qc >> 1) & 1);
            if (!ok) break;
            sum_q(s, u, qs, qc % kQSums);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarQFull + qs));
          }
          continue;
        }
        gather_q(s, u, qs, 0, 1);
        __syncwarp();
        if constexpr (QUANT) sum_q(s, u, qs, qc % kQSums);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarQFull + qs));
      }
    }
    // every issued copy lands before the block can end
    if (copied_q && lane == 0)
      for (int e = qc > 2 ? qc - 2 : 0; e < qc; ++e)
        if (!mbar_wait_bounded(bar((QUANT ? kBarQLoad : kBarQFull) + (e & 1)), (e >> 1) & 1)) break;
    __syncwarp();
    if (!placed) records();
  } else if (warp >= 12) {
    // ============================ converters: K (12-15) and V (16-19)
    if constexpr (QUANT) {
      const int t = tid & 127;
      const bool isv = warp >= 16;
      const int fulls = isv ? kBarVFull : kBarKFull, empties = isv ? kBarVEmpty : kBarKEmpty;
      const int ops = isv ? kBarVop : kBarKop;
      const uint8_t* ring = smem + lay.ring + (isv ? (size_t)S * G::ENTRY : 0);
      uint8_t* op = smem + (isv ? lay.vop : lay.kop);
      RingPos pos;
      for (int v = 0; v < nv; ++v, pos.next(S)) {
        const int slot = pos.slot;
        if (!wait_warp(fulls + slot, pos.phase)) break;
        // the products with the previous visit's tile are done
        if (v > 0 && !wait_warp(ops + 1, (v - 1) & 1)) break;
        convert_tile<D, KV, BF>(ring + (size_t)slot * G::ENTRY, op, t);
        if (!isv) {
          // scales of token t, with the middle code's part in the zero points
          const int2 hd = *reinterpret_cast<const int2*>(smem + lay.hdr + (v % kHdrs) * 8);
          const bool valid = t < hd.x && (hd.y >> (t >> 4) & 1);
          float4 z = *reinterpret_cast<const float4*>(smem + lay.raw + (size_t)slot * G::RAW_SCALES +
                                                      (KV == KV_I8G ? t >> 6 : t) * 16);
          bool counts = valid;   // among the values' sizes
          if constexpr (TREE) {
            // A draft whose values are no numbers must not reach the rows that do not attend to
            // it: its values are taken out here, and the merge gives them to the rows that do.
            bool bad = false;
            const int4 d = visits[2 * (v & (kVisits - 1))];   // first token, flags, sequence
            if (d.y & kDrafts && d.x + t >= gp[d.z] - moff[d.z]) {
              bad = valid && !(fabsf(z.z) < INFINITY && fabsf(fmaf(G::CENTRE, z.z, z.w)) < INFINITY);
              if (bad) z.z = z.w = 0.f;
              counts = valid && !bad;
            }
            const uint32_t bads = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) reinterpret_cast<uint32_t*>(smem + lay.bad)[(v % kHdrs) * 4 + (warp - 12)] = bads;
          }
          float* sc = reinterpret_cast<float*>(smem + lay.scales + (v % kScaleSlots) * G::SCALES);
          // (scores come out in the log2 domain; one without a token is -inf, see the softmax)
          const float vz = fmaf(G::CENTRE, z.z, z.w);
          sc += (t >> 1) * 4 + (t & 1);
          sc[0] = valid ? z.x * p.scale : 1.f;
          sc[2] = valid ? fmaf(G::CENTRE, z.x, z.y) * p.scale : 0.f;
          sc[2 * kTile] = valid ? z.z : 0.f;
          sc[2 * kTile + 2] = valid ? vz : 0.f;
          // the largest of the values' sizes, and the smallest
          const float size = value_size(z.z, vz);
          const float most = warp_max(counts ? size : 0.f), least = -warp_max(counts ? -size : -INFINITY);
          if (lane == 0) {
            float* vm = reinterpret_cast<float*>(smem + lay.vmax + (v % kScaleSlots) * 32) + (warp - 12);
            vm[0] = most;
            vm[4] = least;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(ops));
          if (!isv) mbar_arrive(bar(kBarHdr + v % kHdrs));
          mbar_arrive(bar(empties + slot));
        }
        passed(v);
      }
    }
  } else if (warp < 8) {
    // =============================================================== softmax
    const int st = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t ts = tm_s(st) + lanes, to = tm_o(st) + lanes;
    const size_t whole = TREE ? tree_records(p) : (size_t)2 * p.batch * p.num_q_heads;   // record rows of segments by stream
    int qc = 0, v = 0;
    uint32_t n_ev = 0, n_seg = 0, n_pair = 0, n_x = 0;   // events, segments, meetings so far
    auto meet = [&](int b, uint32_t& n) -> bool {   // two warps of the same rows
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
      return wait_warp(b, n++ & 1);
    };
    // The stream's four warps. A warp that has given up has arrived here once
    // more (below), so that this ends, and the others see that it has.
    auto meet_all = [&]() -> bool {
      named_bar_sync(2 + st, 128);
      return misc[1] == 0;
    };
    // trees: the tokens of sequence g before its drafts
    [[maybe_unused]] auto before = [&](int g) { return gp[g] - moff[g]; };
    // the stream's next event: the scores of visit v are there
    int ntok = 0, mask = 0;
    bool valid = false;   // token `row` of the tile
    const float* sc = nullptr;
    float lv = 0.f;
    bool even = true;
    // trees of drafts: whether the tile has some, and which of its tokens' values are no numbers
    [[maybe_unused]] bool drafts = false;
    [[maybe_unused]] uint32_t bads[4] = {0, 0, 0, 0};
    auto begin = [&]() -> bool {
      if (!wait_warp(kBarHdr + v % kHdrs, (v / kHdrs) & 1)) return false;
      // Trees look at a tile's drafts while its scores are on their way, but only in the ring's first round: the scores
      // of v are the sign that V of v - S is done with, without which the parity of V's barrier says nothing.
      const bool early = TREE && !QUANT && v < S;
      if (!early && !wait_warp(kBarS + st, n_ev++ & 1)) return false;
      const int2 hd = *reinterpret_cast<const int2*>(smem + lay.hdr + (v % kHdrs) * 8);
      ntok = hd.x;
      mask = hd.y;
      valid = row < ntok && (mask >> (row >> 4) & 1);
      if constexpr (TREE) drafts = flags_of(v) & kDrafts;
      if constexpr (TREE && QUANT) {
        if (drafts) {
          const uint4 b = *reinterpret_cast<const uint4*>(smem + lay.bad + (v % kHdrs) * 16);
          bads[0] = b.x, bads[1] = b.y, bads[2] = b.z, bads[3] = b.w;
        }
      }
      if constexpr (QUANT) {
        sc = reinterpret_cast<const float*>(smem + lay.scales + (v % kScaleSlots) * G::SCALES);
        const float4* vm = reinterpret_cast<const float4*>(smem + lay.vmax + (v % kScaleSlots) * 32);
        const int most = size_exponent(fmaxf(fmaxf(vm[0].x, vm[0].y), fmaxf(vm[0].z, vm[0].w)));
        even = most - size_exponent(fminf(fminf(vm[1].x, vm[1].y), fminf(vm[1].z, vm[1].w))) <= kEvenBits;
        lv = (float)most;
      } else if (ntok < kTile || mask != 0xFF || (TREE && drafts)) {
        // rows of V that hold no token of this segment may hold anything, NaN
        // too, and a weight of 0 would not clear it
        const int slot = v % S;
        // (A slot's parity tells its last two uses apart. With two slots and more the scores of v were issued behind
        // the products of V of v - S at the latest. With a single slot they were issued behind V of v - 2 was
        // given back, and V of v - 1 has to be, too: that barrier's parity then means v - 1, not v - 3.)
        if (S == 1 && v > 0 && !wait_warp(kBarVEmpty, (v - 1) & 1)) return false;
        if (!wait_warp(kBarVFull + slot, (v / S) & 1)) return false;
        if (row < (ntok + 15) / 16 * 16 && !valid) {
          uint8_t* vr = smem + lay.ring + (size_t)(S + slot) * G::ENTRY + row * 128;
#pragma unroll 4
          for (int i = 0; i < G::HALVES * 8; ++i)
            *reinterpret_cast<uint4*>(vr + (i >> 3) * 16384 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        if constexpr (TREE) {
          if (drafts) {   // (see the converters)
            int* marks = reinterpret_cast<int*>(smem + lay.bad) + (v % kBadSlots) * kTile;
            const Visit& d = *reinterpret_cast<const Visit*>(visits + 2 * (v & (kVisits - 1)));
            if (valid && d.tok0 + row >= before(d.row))
              clear_no_numbers<G::HALVES, BF>(smem + lay.ring + (size_t)(S + slot) * G::ENTRY, row, marks + row, v);
            if (!meet_all()) return false;
#pragma unroll
            for (int i = 0; i < 4; ++i) bads[i] = __ballot_sync(0xffffffffu, *(volatile int*)(marks + 32 * i + lane) == v);
          }
        }
        fence_proxy_async_smem();   // before the products read them
      }
      if (early && !wait_warp(kBarS + st, n_ev++ & 1)) return false;
      tc_after();
      return true;
    };
    auto end_event = [&]() {   // the weights are written
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarP + st));
    };
    // Weights are 2^(score - r), for each query row with a reference r that follows the largest
    // score (quantised caches: score + log2 of the token's value size) less kWeightBits, only
    // once that is more than 8 above it: a weight (times a value's scale) stays within fp16's
    // range, and the accumulator is rarely rescaled.

    bool ok = true;
    while (v < nv && ok) {
      Visit s;
      ok = visit(v, s);
      if (!ok) break;
      const bool two = MODE != kFewDrafts && s.is(kTwo), few = is_few(s.rows);
      constexpr int STREAMS = MODE == kDraftRows ? 1 : 2;   // that write records of their own
      const size_t rec0 = s.is(kContinued) ? STREAMS * whole + (size_t)blockIdx.x * 2 * kTile + (few ? st * kTile : 0)
                                           : (few ? st * whole : 0) + s.rec;
      const float* qsum = reinterpret_cast<const float*>(smem + lay.qsum) + ((qc + (two ? st : 0)) % kQSums) * kTile;
      qc += two ? 2 : 1;
      bool have = false;
      if (few) {
        // ---- up to 16 query rows: thread = token for the scores, channel for the values;
        // rows in blocks of eight, of which the second may be empty. Lane j of every
        // warp holds row j's reference, each thread its token's part of the rows' sums.
        float* xch = reinterpret_cast<float*>(smem + lay.xch) + st * (2 * 4 * 32);
        uint8_t* pt = smem + lay.pt + st * G::PT;
        const bool wide = s.rows > 8;
        [[maybe_unused]] uint32_t poison = 0;   // rows that attend to values that are no numbers
        float r = -INFINITY, l[FEW];
        [[maybe_unused]] float zs[FEW];
        int flags = s.flags;
        for (;;) {
          if ((v & 1) == st) {
            [[maybe_unused]] uint32_t sees = 0xffffffffu;   // rows that attend to the thread's token
            if constexpr (TREE) {   // (known before the scores are there)
              if (flags & kDrafts) sees = tree_rows(p, s, visits[2 * (v & (kVisits - 1))].x + row - before(s.row));
            }
            ok = begin();
            if (!ok) break;
            if (!have) {
#pragma unroll
              for (int j = 0; j < FEW; ++j) {
                l[j] = 0.f;
                if constexpr (QUANT) zs[j] = 0.f;
              }
            }
            float a[FEW];
            if constexpr (TREE) {
              if (!valid) sees = 0;
              if (drafts && (bads[quad] >> lane & 1)) poison |= sees;
            }
            const int at = (row >> 1) * 4 + (row & 1);
            const float ks = QUANT ? sc[at] : p.scale;
            const float kz = QUANT ? sc[at + 2] : 0.f, vs = QUANT ? sc[2 * kTile + at] : 1.f;
            [[maybe_unused]] const float vz = QUANT ? sc[2 * kTile + at + 2] : 0.f;
            [[maybe_unused]] const float lt = QUANT ? (float)size_exponent(value_size(vs, vz)) : 0.f;
            float* xb = xch + (n_x++ & 1) * (4 * 32);
            float keep = -INFINITY;
#pragma unroll
            for (int e = 0; e < FEW; e += 8) {
              if (e > 0 && !wide) break;
              tmem_ld<8>(ts + e, reinterpret_cast<uint32_t*>(a + e));
              float4 q4[2] = {};
              if constexpr (QUANT) {
                q4[0] = *reinterpret_cast<const float4*>(qsum + e);
                q4[1] = *reinterpret_cast<const float4*>(qsum + e + 4);
              }
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                a[e + j] = QUANT ? fmaf(ks, a[e + j], kz * reinterpret_cast<const float*>(q4)[j]) : a[e + j] * ks;
                if (TREE ? !(sees >> (e + j) & 1) : !valid) a[e + j] = -INFINITY;
                const float w = warp_max(QUANT ? a[e + j] + lt : a[e + j]);
                if (lane == e + j) keep = w;
              }
            }
            if (lane < FEW) xb[quad * 32 + lane] = keep;
            ok = meet_all();
            if (!ok) break;
            // lane j: the largest of row j over the tile's tokens
            xb += lane & (FEW - 1);
            const float t = fmaxf(fmaxf(xb[0], xb[32]), fmaxf(xb[64], xb[96])) - kWeightBits;
            float alpha = 1.f;
            if (t > r + 8.f) {
              alpha = fast_exp2(r - t);   // 0 from -inf
              r = t;
            }
            if (have && __any_sync(0xffffffffu, alpha != 1.f)) {   // the same for the whole stream
#pragma unroll
              for (int e = 0; e < FEW; e += 8) {
                if (e > 0 && !wide) break;
                uint32_t o[16];
                tmem_ld<8>(to + e, o);
                tmem_ld<8>(to + FEW + e, o + 8);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float f = __shfl_sync(0xffffffffu, alpha, e + j);
                  l[e + j] *= f;
                  if constexpr (QUANT) zs[e + j] *= f;
                  o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                  o[8 + j] = __float_as_uint(__uint_as_float(o[8 + j]) * f);
                }
                tmem_st<8>(to + e, o);
                tmem_st<8>(to + FEW + e, o + 8);
              }
              tc_wait_st();
            }
            const float ref = r == -INFINITY ? 0.f : r;
#pragma unroll
            for (int e = 0; e < FEW; e += 8) {
              if (e > 0 && !wide) break;
              // weights of token `row`, first terms and what their rounding left, as
              // [8-row block][token][8]
              uint32_t hi16[4], lo16[4];
#pragma unroll
              for (int k = 0; k < 8; k += 2) {
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int j = e + k + i;
                  w[i] = fast_exp2(a[j] - __shfl_sync(0xffffffffu, ref, j));
                  l[j] += w[i];
                  if constexpr (QUANT) {
                    zs[j] = fmaf(w[i], vz, zs[j]);
                    w[i] *= vs;
                  }
                }
                hi16[k / 2] = pack16<BF>(w[0], w[1]);
                lo16[k / 2] = pack16<BF>(w[0] - low16<BF>(hi16[k / 2]), w[1] - high16<BF>(hi16[k / 2]));
              }
              *reinterpret_cast<uint4*>(pt + e * 256 + row * 16) = make_uint4(hi16[0], hi16[1], hi16[2], hi16[3]);
              *reinterpret_cast<uint4*>(pt + (FEW + e) * 256 + row * 16) = make_uint4(lo16[0], lo16[1], lo16[2], lo16[3]);
            }
            fence_proxy_async_smem();
            have = true;
            end_event();
          }
          passed(v++);
          if (flags & kLast) break;
          ok = described(v);
          if (!ok) break;
          flags = flags_of(v);
        }
        if (!ok || !have) continue;   // !have: a part of one visit, the other stream's
        // ---- the stream's record of each row
        float* xb = xch + (n_x++ & 1) * (4 * 32);
#pragma unroll
        for (int e = 0; e < FEW; e += 8) {
          if (e > 0 && !wide) break;
          int j;
          const float ls = scatter_sum8(l + e, lane, j);
          xb[quad * 32 + e + j] = ls;
          if constexpr (QUANT) xb[quad * 32 + FEW + e + j] = scatter_sum8(zs + e, lane, j);
        }
        if constexpr (TREE) xb[quad * 32 + 31] = __uint_as_float(__reduce_or_sync(0xffffffffu, poison));
        ok = meet_all();
        if (!ok) break;
        auto total = [&](int i) { return (xb[i] + xb[32 + i]) + (xb[64 + i] + xb[96 + i]); };
        if (row < s.rows) {
          float ls = total(row);
          if constexpr (TREE) {   // a sum with a sign: values were left out, see the merge
            const uint32_t rows = __float_as_uint(xb[31]) | __float_as_uint(xb[63]) | __float_as_uint(xb[95]) |
                                  __float_as_uint(xb[127]);
            if (rows >> row & 1) ls = -ls;
          }
          p.ws_ml[rec0 + row] = make_float2(r, ls);
          if (!s.is(kMany)) {   // a part of one visit: the other stream has nothing
            const size_t other = s.is(kContinued) ? rec0 + (st ? -kTile : kTile) : st ? s.rec : whole + s.rec;
            p.ws_ml[other + row] = make_float2(-INFINITY, 0.f);
          }
        }
        ok = wait_warp(kBarO + st, n_seg++ & 1);
        if (!ok) break;
        tc_after();
        if (quad * 32 < D) {
#pragma unroll 1
          for (int e = 0; e < s.rows; e += 8) {
            uint32_t o[16];
            tmem_ld<8>(to + e, o);
            tmem_ld<8>(to + FEW + e, o + 8);
            tc_wait_ld();
            if constexpr (TREE) {   // (rows up to the next multiple of 32 are the record's own)
              float f[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                f[k] = __uint_as_float(o[k]) + __uint_as_float(o[8 + k]);
                if constexpr (QUANT) f[k] += total(FEW + e + k);
              }
              float4* at = reinterpret_cast<float4*>(p.ws_acc + rec0 * D + row * 32 + e);
              at[0] = make_float4(f[0], f[1], f[2], f[3]);
              at[1] = make_float4(f[4], f[5], f[6], f[7]);
              continue;
            }
            float* acc = p.ws_acc + (rec0 + e) * D + row;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (e + k >= s.rows) break;
              float f = __uint_as_float(o[k]) + __uint_as_float(o[8 + k]);
              if constexpr (QUANT) f += total(FEW + e + k);
              acc[k * D] = f;
            }
          }
        }
        tc_before();
        continue;
      }

      // ---- more rows: thread = query row. Scores are read twice, COLS columns at a time in
      // loops that stay loops: with all 128 in registers and the code unrolled, the warps
      // waited for instructions. Quantised caches: the first time they are scaled and written
      // back (INT8, 64 rows x 8K: 58.3 -> 57.0 us against reading the scales again).
      const int my_rows = two ? min(kTile, s.rows - st * kTile) : s.rows;
      const bool active = quad * 32 < my_rows;   // this warp has query rows
      float r = -INFINITY, l = 0.f;
      [[maybe_unused]] float zs = 0.f, qs = 0.f;
      [[maybe_unused]] bool poison = false;   // the row attends to values that are no numbers
      for (;;) {
        if (two || (v & 1) == st) {
          [[maybe_unused]] uint4 sees = make_uint4(~0u, ~0u, ~0u, ~0u);   // tokens that the row attends to
          if constexpr (TREE) {
            if (s.is(kDrafts) && row < my_rows)
              sees = tree_window(p, s.row, (s.q0 + (two ? st * kTile : 0) + row) / Gq,
                                 visits[2 * (v & (kVisits - 1))].x - before(s.row));
            __syncwarp();
          }
          ok = begin();
          if (!ok) break;
          if (active) {
            if (QUANT && !have) qs = qsum[row];
            const uint64_t qs2 = pack2f(qs, qs), scale2 = pack2f(p.scale, p.scale);
            const bool partial = ntok < kTile || mask != 0xFF;
            if constexpr (TREE) {
              if (drafts && row < my_rows)
                poison |= (sees.x & bads[0]) | (sees.y & bads[1]) | (sees.z & bads[2]) | (sees.w & bads[3]);
            }
            // tokens [c, c + 32) of the tile that the row attends to
            [[maybe_unused]] auto sees32 = [&](int c) {
              uint32_t on = c < 64 ? (c < 32 ? sees.x : sees.y) : (c < 96 ? sees.z : sees.w);
              if (ntok - c < 32) on &= (1u << max(ntok - c, 0)) - 1u;
              const int pieces = mask >> (c >> 4);
              return on & ((pieces & 1 ? 0xFFFFu : 0u) | (pieces & 2 ? 0xFFFF0000u : 0u));
            };
            if (!TREE && partial) {   // columns without a token (trees: left out in the pass below)
#pragma unroll 1
              for (int c = 0; c < kTile; c += 16) {
                const int left = mask >> (c >> 4) & 1 ? ntok - c : 0;
                if (left >= 16) continue;
                float a[16];
                tmem_ld<16>(ts + c, reinterpret_cast<uint32_t*>(a));
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (j >= left) a[j] = -INFINITY;
                tmem_st<16>(ts + c, reinterpret_cast<uint32_t*>(a));
              }
              tc_wait_st();
            }
            float mx = -INFINITY;
            // Scales of 8 tokens are loaded while the scores, or those before, are on their way. (A step of 16 x ~6K INT8 with 24
            // drafts, 4, 8, 16 tokens ahead: 116, 105, 106 us; more of them do not fit 96 registers.)
            constexpr int PRE = 4;
            [[maybe_unused]] ulonglong2 k2[PRE];
            [[maybe_unused]] auto scales = [&](int at) {
#pragma unroll
              for (int j = 0; j < PRE; ++j) k2[j] = *reinterpret_cast<const ulonglong2*>(sc + 2 * at + 4 * j);
            };
            if constexpr (QUANT) scales(0);
#pragma unroll 1
            for (int c = 0; c < ntok; c += COLS) {
              float a[COLS];
              tmem_ld<32>(ts + c, reinterpret_cast<uint32_t*>(a));
              if constexpr (COLS == 64) tmem_ld<32>(ts + c + 32, reinterpret_cast<uint32_t*>(a + 32));
              tc_wait_ld();
              if constexpr (QUANT) {
#pragma unroll
                for (int h = 0; h < COLS; h += 2 * PRE) {
#pragma unroll
                  for (int j = 0; j < 2 * PRE; j += 2)
                    unpack2f(ffma2(pack2f(a[h + j], a[h + j + 1]), k2[j / 2].x, fmul2(k2[j / 2].y, qs2)), a[h + j],
                             a[h + j + 1]);
                  scales(min(c + h + 2 * PRE, kTile - 2 * PRE));
                }
              }
              if constexpr (TREE) {
                if (drafts || partial) {
#pragma unroll
                  for (int h = 0; h < COLS; h += 32) {
                    const uint32_t on = sees32(c + h);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                      if (!(on >> j & 1)) a[h + j] = -INFINITY;
                    if constexpr (!QUANT) tmem_st<32>(ts + c + h, reinterpret_cast<uint32_t*>(a + h));
                  }
                }
              }
              if constexpr (QUANT) tmem_st<32>(ts + c, reinterpret_cast<uint32_t*>(a));
              float m4[4] = {mx, a[0], a[1], a[2]};
#pragma unroll
              for (int j = 3; j < COLS - 1; j += 2) m4[j >> 1 & 3] = max3(m4[j >> 1 & 3], a[j], a[j + 1]);
              mx = max3(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]), a[COLS - 1]);
            }
            if constexpr (QUANT || TREE) tc_wait_st();
            if constexpr (QUANT) {
              if (!even) {   // uniform over the block
                mx = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < ntok; c += 8) {
                  float a[8];
                  tmem_ld<8>(ts + c, reinterpret_cast<uint32_t*>(a));
                  tc_wait_ld();
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const float* v2 = sc + 2 * kTile + 2 * (c + (j & -2)) + (j & 1);
                    mx = fmaxf(mx, a[j] + (float)size_exponent(value_size(v2[0], v2[2])));
                  }
                }
              } else {
                mx += lv;
              }
            } else {
              mx *= p.scale;
            }
            const float t = mx - kWeightBits;
            float alpha = 1.f;
            if (t > r + 8.f) {
              alpha = fast_exp2(r - t);   // 0 from -inf
              r = t;
              l *= alpha;
              if constexpr (QUANT) zs *= alpha;
            }
            if (have && __any_sync(0xffffffffu, alpha != 1.f)) {
              // S of this event is complete, so every earlier product of this stream is
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld<32>(to + c, o);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                tmem_st<32>(to + c, o);
              }
            }
            const float ref = r == -INFINITY ? 0.f : r;
            const uint64_t ref2 = pack2f(-ref, -ref);
            uint64_t ls0 = 0, ls1 = 0, z2 = 0;
            if constexpr (QUANT) scales(kTile);
#pragma unroll 1
            for (int c = 0; c < ntok; c += COLS) {
              float a[COLS];
              tmem_ld<32>(ts + c, reinterpret_cast<uint32_t*>(a));
              if constexpr (COLS == 64) tmem_ld<32>(ts + c + 32, reinterpret_cast<uint32_t*>(a + 32));
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < COLS; j += 2) {
                float x, y;
                if constexpr (QUANT)
                  unpack2f(fadd2(pack2f(a[j], a[j + 1]), ref2), x, y);
                else
                  unpack2f(ffma2(pack2f(a[j], a[j + 1]), scale2, ref2), x, y);
                a[j] = fast_exp2(x);
                a[j + 1] = fast_exp2(y);
                const uint64_t w2 = pack2f(a[j], a[j + 1]);
                (j & 2 ? ls1 : ls0) = fadd2(j & 2 ? ls1 : ls0, w2);
                if constexpr (QUANT) {
                  const ulonglong2 v2 = k2[j / 2 % PRE];
                  z2 = ffma2(w2, v2.y, z2);
                  unpack2f(fmul2(w2, v2.x), a[j], a[j + 1]);
                  if (j % (2 * PRE) == 2 * PRE - 2) scales(kTile + min(c + j + 2, kTile - 2 * PRE));
                }
              }
              // The weights' one rounding to the operand type. They take the
              // place of their scores: 16 columns for 32 tokens, and 16 more of
              // second terms, which hold what the rounding left, where the output
              // keeps more bits.
#pragma unroll
              for (int e = 0; e < COLS; e += 32) {
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j] = pack16<BF>(a[e + 2 * j], a[e + 2 * j + 1]);
                tmem_st<16>(ts + c + e, w);
                if (p.two_terms) {
#pragma unroll
                  for (int j = 0; j < 16; ++j)
                    w[j] = pack16<BF>(a[e + 2 * j] - low16<BF>(w[j]), a[e + 2 * j + 1] - high16<BF>(w[j]));
                  tmem_st<16>(ts + c + e + 16, w);
                }
              }
            }
            l += hsum2(fadd2(ls0, ls1));
            if constexpr (QUANT) zs += hsum2(z2);
            tc_wait_st();
          }
          have = true;
          end_event();
        }
        passed(v++);
        if (s.is(kLast)) break;
        ok = described(v);
        if (!ok) break;
        s.flags = flags_of(v);
      }
      if (!ok || !have) continue;
      // ---- one record per query row; where both streams have tiles of the same
      // rows, their states meet and each writes half of the channels of their sum
      const bool both = !two && s.is(kMany);
      const int tile_row = two ? st * kTile + row : row;
      ok = wait_warp(kBarO + st, n_seg++ & 1);
      if (!ok) break;
      tc_after();
      if (active) {
        float R = r, L = l, z = QUANT ? zs : 0.f, f0 = 1.f, f1 = 0.f;
        int from = 0, to_c = D;
        if (both) {
          float4* mls = reinterpret_cast<float4*>(smem + lay.ml);
          mls[st * kTile + row] = make_float4(r, l, z, TREE && poison ? 1.f : 0.f);
          tc_before();
          ok = meet(kBarPair + quad, n_pair);
          if (!ok) break;
          tc_after();
          const float4 other = mls[(st ^ 1) * kTile + row];
          R = fmaxf(r, other.x);
          const float Rr = R == -INFINITY ? 0.f : R;
          f0 = fast_exp2(r - Rr);
          f1 = fast_exp2(other.x - Rr);
          L = fmaf(l, f0, other.y * f1);
          z = fmaf(z, f0, other.z * f1);
          if constexpr (TREE) poison |= other.w != 0.f;
          from = st * (D / 2);
          to_c = from + D / 2;
        }
        if constexpr (TREE) L = poison ? -L : L;
        if (row < my_rows && from == 0) p.ws_ml[rec0 + tile_row] = make_float2(R, L);
        // CHUNK channels at a time through shared memory (the stream's place for transposed
        // weights), so that a row's 64 (32) bytes are written together
        const uint32_t to2 = tm_o(st ^ 1) + lanes;
        if constexpr (TREE) {
          constexpr int PASS = QUANT ? 8 : 32;
          float* out = p.ws_acc + (rec0 + tile_row - lane) * D + lane;
#pragma unroll 1
          for (int c = from; c < to_c; c += PASS) {
            uint32_t o[PASS], o2[PASS];
            tmem_ld<PASS>(to + c, o);
            if (both) tmem_ld<PASS>(to2 + c, o2);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < PASS; ++j) {
              float f = __uint_as_float(o[j]);
              if (both) f = fmaf(__uint_as_float(o2[j]), f1, f * f0);
              if constexpr (QUANT) f += z;
              out[(c + j) * 32] = f;
            }
          }
        } else {
        constexpr int CHUNK = G::PT / 512, PARTS4 = CHUNK / 4;   // 16 or 8
        uint8_t* stage = smem + lay.pt + st * G::PT + quad * (32 * CHUNK * 4);
        const int live = min(32, my_rows - quad * 32);   // the warp's query rows
        float* out = p.ws_acc + (rec0 + tile_row - lane) * D + (lane & (PARTS4 - 1)) * 4;
#pragma unroll 1
        for (int c = from; c < to_c; c += CHUNK) {
          uint32_t o[CHUNK], o2[CHUNK];
          tmem_ld<CHUNK>(to + c, o);
          if (both) tmem_ld<CHUNK>(to2 + c, o2);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < CHUNK; j += 4) {
            float f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              f[k] = __uint_as_float(o[j + k]);
              if (both) f[k] = fmaf(__uint_as_float(o2[j + k]), f1, f[k] * f0);
              if constexpr (QUANT) f[k] += z;
            }
            *reinterpret_cast<float4*>(stage + (lane * PARTS4 + (j >> 2 ^ lane / (8 / PARTS4) & (PARTS4 - 1))) * 16) =
                make_float4(f[0], f[1], f[2], f[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32; i += 32 / PARTS4) {
            const int q = i + lane / PARTS4, j = lane & (PARTS4 - 1);
            const float4 f =
                *reinterpret_cast<const float4*>(stage + (q * PARTS4 + (j ^ q / (8 / PARTS4) & (PARTS4 - 1))) * 16);
            if (q < live) *reinterpret_cast<float4*>(out + (size_t)q * D + c) = f;
          }
          __syncwarp();
        }
        }
        if (both) {   // neither accumulator is overwritten before both are read
          tc_before();
          ok = meet(kBarPair + quad, n_pair);
          if (!ok) break;
        }
      }
      tc_before();
    }
    // given up: the stream's other warps may be waiting for this one
    if (!ok) asm volatile("bar.arrive %0, 128;" ::"r"(2 + st) : "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------ the merge
// out = sum 2^(m_i - M) a_i / sum 2^(m_i - M) l_i over the records of 128 outputs (a query
// row, or two of 64 channels), from the blocks of its prefix segment and of its own
// tokens: WPW warps each take every WPW-th record, a lane 4 channels. Bound by latency
// (records come from L2, four at a time in flight per warp): 3 to 6 us a call, of which about 2
// are the launch. Where the records are has been worked out by the attention kernel: this
// kernel is short, as its code is fetched anew by every call.
constexpr int kMergeThreads = 128;

// Four outputs, rounded once.
__device__ __forceinline__ void store_out4(const SharedParams& p, size_t at, float4 f) {
  if (p.out_dtype == PKV_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = f;
  } else {
    const uint2 v = p.out_dtype == PKV_BF16 ? make_uint2(pack16<true>(f.x, f.y), pack16<true>(f.z, f.w))
                                            : make_uint2(pack16<false>(f.x, f.y), pack16<false>(f.z, f.w));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = v;
  }
}

// The attention kernel takes infinities and NaNs out of the drafts' values (0 times one of them would be
// one, in rows that do not attend to it) and marks the records of the rows that do attend to them:
// the sum of those of a row's four channels, for its output.
static __device__ __noinline__ float4 no_numbers(const SharedParams& p, int b, int t, int h, int ch, int D) {
  const TreePlan r = tree_plan(p, b);
  const uint64_t* words = tree_words(p, b, t);
  float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int j = 0; j < r.drafts; ++j) {
    if (!(tree_bits(p, words, t, j) & 1)) continue;
    const int tok = r.len - r.drafts + j, page = p.block_table[(size_t)b * p.max_pages + tok / p.page_size];
    if (page < 0 || page >= p.num_pages) continue;
    const size_t row = ((size_t)page * p.num_kv_heads + h) * p.page_size + tok % p.page_size;
    float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.kv_kind >= KV_I8T) z = *reinterpret_cast<const float4*>(p.kv_sz + (p.kv_kind == KV_I8G ? row / 64 : row) * 4);
    for (int i = 0; i < 4; ++i) {
      const size_t at = row * D + ch + i;
      const float v = p.kv_kind == KV_F16    ? __half2float(reinterpret_cast<const __half*>(p.v_pages)[at])
                      : p.kv_kind == KV_BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v_pages)[at])
                      : p.kv_kind == KV_U4T  ? fmaf((float)(p.v_pages[at / 2] >> (at & 1) * 4 & 15), z.z, z.w)
                                             : fmaf((float)p.v_pages[at], z.z, z.w);
      if (!(fabsf(v) < INFINITY)) x[i] += v;
    }
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}

template <int D, int WPW>
__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const __grid_constant__ SharedParams p) {
  constexpr int BATCH = 4;
  __shared__ float4 part_a[WPW > 1 ? WPW : 1][32];
  __shared__ float2 part_ml[WPW > 1 ? WPW : 1][32];
  const int lane = threadIdx.x & 31, w = WPW > 1 ? threadIdx.x >> 5 : 0;
  const int at = ((int)blockIdx.x * (4 / WPW) + (WPW > 1 ? 0 : (int)threadIdx.x >> 5)) * 128 + lane * 4;   // output
  const int item = at / D;   // row and query head
  pdl_wait();
  if (at >= p.batch * p.num_q_heads * D) return;
  const int kvi = item / p.group, gq = item - kvi * p.group;   // row and kv head
  const int4 own = __ldcg(p.ws_info + 3 * kvi);
  int4 pre = __ldcg(p.ws_info + 3 * kvi + 1);
  const int4 pre2 = __ldcg(p.ws_info + 3 * kvi + 2);
  if (gq >= pre.w >> 1) pre = pre2;   // in the next pair of row tiles
  pre.w &= 1;
  const int ch = at % D, whole = 2 * p.batch * p.num_q_heads;
  const int n0 = pre.z << pre.w, n1 = own.z << own.w;
  float M = -INFINITY, L = 0.f;
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int j0 = w; j0 < n0 + n1; j0 += WPW * BATCH) {
    float2 ml[BATCH];
    float4 a[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      int j = j0 + i * WPW;
      const bool on = j < n0 + n1;
      int4 seg = pre;
      if (j >= n0) {
        seg = own;
        j -= n0;
      }
      // stream and part; a block's first part, where it continues the segment,
      // has its place by block
      const int st = j & seg.w, k = j >> seg.w;
      int r = k == 0 ? seg.x + st * whole : seg.y + (k - 1) * 2 * kTile + st * kTile;
      r = on ? r + gq : 0;
      ml[i] = __ldcg(p.ws_ml + r);
      if (!on) ml[i] = make_float2(-INFINITY, 0.f);
      a[i] = __ldcg(reinterpret_cast<const float4*>(p.ws_acc + (size_t)r * D + ch));
    }
    float Mn = M;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) Mn = fmaxf(Mn, ml[i].x);
    const float Mr = Mn == -INFINITY ? 0.f : Mn, f0 = fast_exp2(M - Mr);
    M = Mn;
    L *= f0;
    A = make_float4(A.x * f0, A.y * f0, A.z * f0, A.w * f0);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      // no token: its accumulator means nothing. (Maxima pass over NaN scores, so a record of
      // nothing else has m = -inf too; its l is NaN, and so is what becomes of it.)
      if (ml[i].x == -INFINITY && ml[i].y == 0.f) continue;
      const float f = fast_exp2(ml[i].x - Mr);
      L = fmaf(f, ml[i].y, L);
      A = make_float4(fmaf(f, a[i].x, A.x), fmaf(f, a[i].y, A.y), fmaf(f, a[i].z, A.z), fmaf(f, a[i].w, A.w));
    }
  }
  if constexpr (WPW > 1) {
    part_a[w][lane] = A;
    part_ml[w][lane] = make_float2(M, L);
    __syncthreads();
    if (w != 0) return;
#pragma unroll 1
    for (int o = 1; o < WPW; ++o) {
      const float2 ml = part_ml[o][lane];
      const float4 a = part_a[o][lane];
      const float Mn = fmaxf(M, ml.x), Mr = Mn == -INFINITY ? 0.f : Mn, f = fast_exp2(M - Mr), f2 = fast_exp2(ml.x - Mr);
      L = L * f + ml.y * f2;
      A = make_float4(A.x * f + a.x * f2, A.y * f + a.y * f2, A.z * f + a.z * f2, A.w * f + a.w * f2);
      M = Mn;
    }
  }
  // no token at all: zeros (L is 0 only then, or where every score is -inf; a NaN stays one)
  const float r = L == 0.f ? 0.f : 1.f / L;
  const float4 f = make_float4(A.x * r, A.y * r, A.z * r, A.w * r);
  store_out4(p, at, f);
}

// The same for trees: a warp (WPW of them, each every WPW-th record) has 16 channels of 32 query rows of a
// segment, a row a lane. The rows' records lie together, so each load brings a channel of all 32, and
// a record's 16 loads, and the next one's, are in flight at once.
template <int D, int WPW>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ SharedParams p) {
  constexpr int CH = 16, SLICES = D / CH;
  __shared__ float part[WPW > 1 ? WPW - 1 : 1][CH + 2][32];
  const int lane = threadIdx.x & 31, w = WPW > 1 ? threadIdx.x >> 5 : 0;
  const int item = (int)blockIdx.x * (4 / WPW) + (WPW > 1 ? 0 : (int)threadIdx.x >> 5);
  const int each = p.drafts * p.group, blocks = (each + 31) / 32;   // query rows of a sequence's kv head
  const int sb = item / SLICES, slice = item - sb * SLICES, sh = sb / blocks, r0 = (sb - sh * blocks) * 32, pair = r0 / (2 * kTile);
  pdl_wait();
  if (sh >= p.num_groups * p.num_kv_heads) return;
  const int4 seg = __ldcg(p.ws_info + (size_t)sh * p.pairs + pair);
  const int first = r0 - pair * 2 * kTile, live = (seg.z >> 16) - first;   // the segment's rows from r0 on
  const int n = live > 0 ? (seg.z & 0xFFFF) << seg.w : 0, whole = tree_records(p);
  float M = -INFINITY, L = 0.f, A[CH];
  bool marked = false;   // some of the row's records leave values out
#pragma unroll
  for (int c = 0; c < CH; ++c) A[c] = 0.f;
  auto join = [&](float2 ml, const float* a) {
    marked |= signbit(ml.y);
    const float l = fabsf(ml.y), Mn = fmaxf(M, ml.x), Mr = Mn == -INFINITY ? 0.f : Mn, f0 = fast_exp2(M - Mr);
    // no token: its accumulator means nothing (see above)
    const bool none = ml.x == -INFINITY && l == 0.f;
    const float f = fast_exp2(ml.x - Mr);
    M = Mn;
    L = none ? L * f0 : fmaf(f, l, L * f0);
#pragma unroll
    for (int c = 0; c < CH; ++c) A[c] = none ? A[c] * f0 : fmaf(f, a[c], A[c] * f0);
  };
#pragma unroll 2
  for (int j = w; j < n; j += WPW) {
    // stream and part; a block's first part, where it continues the segment, has its place by block
    const int st = j & seg.w, k = j >> seg.w;
    const size_t rec = (size_t)(k == 0 ? seg.x + st * whole : seg.y + (k - 1) * 2 * kTile + st * kTile) + first;
    const float* acc = p.ws_acc + rec * D + slice * CH * 32 + lane;
    float a[CH];
    float2 ml = __ldcg(p.ws_ml + rec + min(lane, live - 1));
#pragma unroll
    for (int c = 0; c < CH; ++c) a[c] = __ldcg(acc + c * 32);
    join(ml, a);
  }
  if constexpr (WPW > 1) {
    if (w > 0) {
      part[w - 1][0][lane] = M;
      part[w - 1][1][lane] = marked ? -L : L;
#pragma unroll
      for (int c = 0; c < CH; ++c) part[w - 1][2 + c][lane] = A[c];
    }
    __syncthreads();
    if (w != 0) return;
#pragma unroll 1
    for (int o = 0; o < WPW - 1; ++o) {
      float a[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) a[c] = part[o][2 + c][lane];
      join(make_float2(part[o][0][lane], part[o][1][lane]), a);
    }
  }
  const int R = r0 + lane, seq = sh / p.num_kv_heads, head = sh - seq * p.num_kv_heads, t = R / p.group;
  if (R >= each) return;
  // no token at all: zeros (L is 0 only then, or where every score is -inf; a NaN stays one)
  const float r = lane >= live || L == 0.f ? 0.f : 1.f / L;
  const size_t at = (((size_t)seq * p.drafts + t) * p.num_q_heads + head * p.group + (R - t * p.group)) * D + slice * CH;
#pragma unroll
  for (int c = 0; c < CH; c += 4) {
    float4 f = make_float4(A[c] * r, A[c + 1] * r, A[c + 2] * r, A[c + 3] * r);
    if (lane >= live) f = make_float4(0.f, 0.f, 0.f, 0.f);
    else if (marked) {
      const float4 x = no_numbers(p, seq, t, head, slice * CH + c, D);
      f = make_float4(f.x + x.x, f.y + x.y, f.z + x.z, f.w + x.w);
    }
    store_out4(p, at + c, f);
  }
}

}  // namespace pkv
