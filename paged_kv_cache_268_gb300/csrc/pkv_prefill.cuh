// Prompt-side attention on the 5th-generation tensor cores (tcgen05, TMEM),
// warp-specialised and persistent: softmax(q . K^T scale) . V of many rows a
// sequence, over the paged cache or over packed keys and values.
//
// The query rows of one key head are taken together: row r of a tile of 128 is
// token r / G, head r % G of its group, so grouped heads share every key tile
// that is read, and a few new tokens of many heads still fill a tile (tiles
// hold whole tokens: 128 / G of them).  An item is up to two row tiles of one
// (sequence, key head), over the keys that its rows see, or a piece of them.
// The CTAs, one an SM, share the items' keys out evenly among them.
//
//   softmax     eight warps a row tile: a thread has a row and half of the keys
//   producer    a warp: Q by TMA, K and V tiles into a ring of slots
//   issuer      a warp that issues the matrix products
//   scheduler   a warp that finds the CTA's next items, up to four of them
//   values      a warp that looks V tiles over which hide something (below)
//
// S = Q K^T (both K-major in shared memory) goes to TMEM; a softmax thread
// reads its half row, p = 2^(s c - m c), and writes P over S in 16 bits, from where
// it is the first operand of O += P V (V read MN-major from its tile).  While
// one row tile is in softmax, the tensor cores work on the other: P0 V, S0 of
// the next keys, P1 V, S1 of the next keys.  With a single row tile the two S
// buffers take the key tiles in turn instead, S one tile ahead of P.
// m follows the row's running maximum only where that grows by more than 2^8;
// then O and the sum are rescaled (rare: the first key tile sets it).  P is held
// in the inputs' type, as the tensor cores want both operands alike; that adds
// half a step of the type to each weight (the whole result of bfloat16 rows is
// then off by 1.4 times the store's own rounding, in the mean).  A second product
// with the rest of P would cost long rows half of their rate.  For few rows, which
// bytes bound, it was tried in items of one row tile whose keys no other item
// reads: bfloat16 rows then round only in the store (2.3e-3 to 1.7e-3), as the
// decode kernels' do, but 4 x 8 tokens after 32760 take 89.4 us instead of 87.0,
// all other calls 1 to 3% more for the longer loop (binary16 25%: the registers).
// P in binary16 is scaled by 2^7 so that weights of down to 2^-21 of the largest
// keep all their bits; the largest, 2^15, is still in range.  In bfloat16 it is
// scaled by 2^-8: the largest is 1, and O in FP32 holds what a plain softmax's
// sums hold of values near the type's end.  The sums are of P in FP32, before
// its rounding.
//
// Hidden keys: P is zero there, but 0 times an infinity or NaN is not.  In key
// tiles that hide something from some row, values past the sequence's end are
// cleared, and those that are no numbers as well (and kept in mind: at the
// end they are added for the rows that see them, whose weights are positive).
// A warp does so as the tiles land, before their products.
//
// What bounds it.  Long rows: 128 keys of 2 x 128 rows are 2048 cycles of matrix
// products (128 channels) and take about 2650, of which no part of the softmax
// alone is worth more than 3% (its exponentials, its maximum or its meeting
// left out one at a time); an item costs 5500 cycles besides (first scores, O to
// memory), a call 5 us until its first loads and the reduce after it.  Few rows:
// the cache's bytes.  Measured on one GB300, graph-timed, bfloat16, 32 heads of 128
// on 8: a prompt of 8192 tokens 328 us, 1675 TFLOP/s, 0.86 of the library's
// 8192^3 product; 2048 tokens after 8192 in blocks of 16 190 us, 1630; 4 x 8 tokens of
// 64/8 heads after 32760 each 88 us, 6.1 TB/s, 0.90 of a copy; without a mask,
// 4096 tokens, head_dim 64 / 128 / 256: 1010, 1630, 1505 TFLOP/s (at 64 no unit is
// full: issue slots 59%, exponentials and tensor pipe 44% each; it is the chain from
// scores to weights to products of the two row tiles).
// On the way (a prompt of 8192): 729 us with one issuing lane that worked out its
// descriptors, 501 with descriptors in uniform registers, 411 with two threads a
// row, 371 with items cut evenly over the CTAs, V looked over by a warp of its
// own and O exchanged between lanes, 352 with the next item's scores early, 344 with
// two barriers asked at once, 337 with an issuer that does not sleep.  32 prompts
// of 1-2048 tokens, 32 heads of 128: 371 us, 365 with items told of further ahead,
// 354 with masks against constants and a quicker look at the values, 348 with
// output stores that pass L1 by, 351 since logits of any size are taken.
// Tried and slower: P beside S with scores that need not wait for it (head_dim 64,
// 138 to 160 us); four output warps (80 registers for the softmax, 337 to 367);
// a quarter of the exponentials by polynomial (175 to 200 of 4096 tokens); the
// exponents before the two warps of a row agree on the maximum (2% slower); an
// item's output after the next one's first weights (none to 2% slower); the row
// tiles' order by which is through first (one-to-one heads end a key tile apart;
// the choice costs the issuer 2%, which is what it saves).
//
// Every wait is bounded; a role that gives up leaves, the others follow, and
// the device error word is set.
#pragma once

#include "pkv_prefill.h"
#include "pkv_prefill_line.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr uint32_t kFullMask = 0xffffffffu;

template <int D>
struct PrefillLayout {
  static constexpr int NQ = prefill_row_tiles(D);
  static constexpr int BN = prefill_key_tile(D);
  static constexpr int PANELS = D / 64;             // 128-byte columns of a row
  static constexpr int SOFT = 8 * NQ;               // softmax warps
  static constexpr int THREADS = (SOFT + 4) * 32;
  static constexpr int Q_TILE = 128 * D * 2;
  static constexpr int KV_TILE = BN * D * 2;
  static constexpr int STAGES = D == 64 ? 8 : 5;
  // Items that the scheduler has told of and that are not through: with two, the
  // producer had none to load while short items ended (2% of such a batch).
  static constexpr int ITEMS_LOG2 = 2, ITEMS = 1 << ITEMS_LOG2;
  static constexpr int OFF_KV = NQ * Q_TILE;
  static constexpr int OFF_BAR = OFF_KV + STAGES * KV_TILE;
  static constexpr int KV_FULL = 0, KV_EMPTY = STAGES, Q_FULL = 2 * STAGES, Q_EMPTY = Q_FULL + 2,
                       S_FULL = Q_EMPTY + 2, P_FULL = S_FULL + 3, O_DONE = P_FULL + 6,
                       O_LAST = O_DONE + 2, O_FREE = O_LAST + 2, I_FULL = O_FREE + 2,
                       I_EMPTY = I_FULL + ITEMS, V_HERE = I_EMPTY + ITEMS, V_CLEAN = V_HERE + 2,
                       NBAR = V_CLEAN + 2;
  static constexpr int OFF_ITEM = OFF_BAR + NBAR * 8;
  static constexpr int OFF_TMEM = OFF_ITEM + ITEMS * 80;
  static constexpr int OFF_XCH = OFF_TMEM + 16;     // [NQ][2][128] floats
  static constexpr int BYTES = OFF_XCH + NQ * 1024;
  // S buffer 0, 1: of row tile 0, 1; 2: buffer 1 with a single row tile (a
  // barrier of its own, so that each has one group of softmax warps only)
  static constexpr int S_COL(int s) { return s > 0 ? BN : 0; }
  static constexpr int O_COL(int x) { return 256 + x * D; }
  // P of keys 16 kk .. 16 kk + 15: each half of the keys over its own half of S
  static constexpr int P_COL(int kk) { return kk < BN / 32 ? kk * 8 : BN / 2 + (kk - BN / 32) * 8; }
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

struct PrefillItem {
  int work;                      // 0: no more items
  int seq, kvh;
  int q_row, ntok;               // its rows: tokens [q_row, q_row + ntok)
  int two;                       // both row tiles are used
  int L;                         // keys of the sequence
  int off;                       // position of the first token
  int t0;                        // first key tile
  int n0, n1;                    // key tiles that row tile 0, 1 sees from there
  int hidden;                    // of these, from here on some hide something from some row
  int key_base;                  // packed: row of the first key
  int once;                      // no other item reads these keys
  int piece;                     // of partial rows that the item's rows go to, or -1: whole
  int bad_values;                // values that are no numbers were cleared
};
static_assert(sizeof(PrefillItem) <= 80, "item slot");

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Values that a tmem_ld32 brings may be used from here on (after tmem_wait_ld).
__device__ __forceinline__ void tmem_ready32(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                 "+f"(v[15]));
  asm volatile(""
               : "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// mbar_wait in few instructions: a try sleeps for up to a microsecond, and after
// four million of them the wait gives up.  Some waits are as long as an item (of
// the warps that are told of items ahead, that look values over or that have the
// second row tile): one of the longest sequence, 2^24 keys, takes 0.1 to 0.4
// seconds (1500 to 2700 cycles for 128 keys, or their bytes at an SM's share).
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 0;\n\t"
      "TRY:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 q, n, 4000000;\n\t"
      "@q bra TRY;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000)
      : "memory");
  return ok != 0;
}

// A wait of the warp that the others wait for: asks without a pause (an answer
// takes a third of the time that a try's does), 160 million times at most.
__device__ __forceinline__ bool mbar_wait_spin(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 0;\n\t"
      "TRY:\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 q, n, 160000000;\n\t"
      "@q bra TRY;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Whether both phases have ended; asked at once.
__device__ __forceinline__ bool mbar_try_both(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1) {
  uint32_t r0, r1;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%2], %3;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%4], %5;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tselp.u32 %1, 1, 0, q;\n\t}"
      : "=r"(r0), "=r"(r1)
      : "r"(b0), "r"(p0), "r"(b1), "r"(p1)
      : "memory");
  return (r0 & r1) != 0;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Matrix products that the whole warp reaches and the lane with `leader` issues:
// without a branch, the descriptors stay in uniform registers.  A descriptor is
// its low word (address, leading offset) and a constant high word.
//   D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                        uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
//   D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                        uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint32_t bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}

// TMA loads that the whole warp reaches and the lane with `leader` issues.
__device__ __forceinline__ void tma_2d_if(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                          uint64_t policy, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tma_3d_if(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                          uint64_t policy, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %7, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy), "r"(leader)
      : "memory");
}

// 32 bytes to global memory, which nobody here reads again.  Rows of the output: to
// an address that is `wide`, aligned to them, in one piece that passes L1 by (1-3%
// of the kernel's time) and is the first to leave L2; else in two plain ones.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.L1::no_allocate.L2::evict_first.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
// The same for partial rows, which the reduce finds in L2.
__device__ __forceinline__ void store32_part(float* p, const float* v) {
  asm volatile("st.global.L1::no_allocate.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Pairs of floats in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\tmov.b64 z, {%5, %6};\n\t"
      "fma.rn.f32x2 %0, x, y, z;\n\t}"
      : "=l"(d)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
      "mul.rn.f32x2 %0, x, y;\n\t}"
      : "=l"(d)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
      "add.rn.f32x2 %0, x, y;\n\t}"
      : "=l"(d)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}

// Queries and keys of sequence b: rows [q0, q0 + n) attend over L keys, whose
// first is key row k0 (packed).  n = 0 where the arrays hold no valid range;
// `code` then says what is wrong.  I: the scheduler's integers (with 32 bits no
// sequence can be too long).
struct PrefillSeq {
  int q0, n, k0, L, code;
  bool falls;                    // its rows end before they begin: rows may be several sequences'
};
template <typename I>
__device__ __forceinline__ PrefillSeq prefill_seq(const PrefillArgs& a, int b) {
  // (all loads at once)
  const int i = min(b, a.B - 1);
  const int q0 = a.query_starts[i], q1 = a.query_starts[i + 1];
  const bool packed = a.key_starts != nullptr;
  const int32_t* keys = packed ? a.key_starts : a.context_lens;
  const int k0 = packed ? keys[i] : 0, k1 = keys[packed ? i + 1 : i];
  const bool rows = q0 >= 0 && q1 >= q0 && q1 <= a.T, cols = k0 >= 0 && k1 >= k0 && k1 <= a.max_keys &&
                    (sizeof(I) == 4 || k1 - k0 <= kPrefillMostKeys);
  const bool fine = rows && cols && b < a.B;
  PrefillSeq s;
  s.q0 = q0;
  s.n = fine ? q1 - q0 : 0;
  s.k0 = k0;
  s.L = fine ? k1 - k0 : 0;
  s.falls = b < a.B && q1 < q0;
  s.code = b >= a.B || fine ? 0 : (rows && !packed ? kDevBadContext : kDevBadStarts);
  return s;
}

template <bool BF, int D>
__global__ void __launch_bounds__(PrefillLayout<D>::THREADS, 1)
    prefill_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using LY = PrefillLayout<D>;
  constexpr int BN = LY::BN, ST = LY::STAGES, PANELS = LY::PANELS;
  constexpr int SOFT = LY::SOFT;
  extern __shared__ __align__(1024) uint8_t smem[];   // swizzle atoms are 1024 bytes
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + LY::OFF_BAR + 8 * i; };
  auto i_full = [&](int i) { return LY::I_FULL + (i & (LY::ITEMS - 1)); };
  auto i_empty = [&](int i) { return LY::I_EMPTY + (i & (LY::ITEMS - 1)); };
  auto i_phase = [&](int i) { return static_cast<uint32_t>(i >> LY::ITEMS_LOG2) & 1; };
  auto item_at = [&](int i) { return reinterpret_cast<PrefillItem*>(smem + LY::OFF_ITEM + (i & (LY::ITEMS - 1)) * 80); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + LY::OFF_TMEM);
  const int tid = threadIdx.x, warp = __shfl_sync(kFullMask, tid >> 5, 0), lane = tid & 31;
  const int TPT = 128 / a.G;                       // tokens of a row tile
  // A V tile lies in runs of keys, all panels of a run one after the other: a
  // run is a block (paged) or the tile.
  const int run_log2 = a.key_starts == nullptr ? a.bs_log2 : (BN == 128 ? 7 : 6);

  if (tid < LY::NBAR) {
    int count = 1;
    if (tid >= LY::P_FULL && tid < LY::P_FULL + 6) count = 8;
    if (tid >= LY::O_FREE && tid < LY::O_FREE + 2) count = 8;
    if (tid >= LY::I_EMPTY && tid < LY::I_EMPTY + LY::ITEMS) count = SOFT + 3;
    mbar_init(bar(tid), count);
  }
  if (sb & 1023) {                                 // (never: the array is aligned)
    if (tid == 0) record_error(a.err, kDevTimeout);
    return;
  }
  if (warp == SOFT && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), 512);
  __syncwarp();
  if (tid < LY::NBAR) fence_mbar_init();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the stream's previous kernel may still have been running until here
  pdl_wait();
  pdl_launch_dependents();
  bool fail = false;

  if (warp >= SOFT) {
    if (warp == SOFT + 2) {
      // -------------------------------------------------------- next item
      // The lines of all sequences and key heads, one after the other, are cut
      // into equal lengths, one a CTA; every CTA finds its own from the lengths
      // on the device.  An item that a cut goes through is done in pieces, which
      // the reduce joins (where there is no workspace for that, cuts move to the items' ends).
      // Sequences are looked at 32 at a time, a lane each.
      const int per_item = TPT * LY::NQ;            // tokens
      const int least = a.cuts != nullptr ? a.min_part : 0x3fffffff;
      auto schedule = [&](auto zero) {
      using I = decltype(zero);
      PrefillSeq s;
      I mine = 0, upto = 0;                 // length of the lane's sequence, all key heads; to its end
      auto length_of = [&](const PrefillSeq& q) {
        return PrefillLine<I>(q.n, q.L, per_item, TPT, a.causal).length() * a.Hkv;
      };
      auto look = [&](int b) {
        s = prefill_seq<I>(a, b + lane);
        upto = mine = length_of(s);
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
          const I u = __shfl_up_sync(kFullMask, upto, i);
          if (lane >= i) upto += u;
        }
      };
      look(0);
      if (s.code != 0 && blockIdx.x == 0) record_error(a.err, s.code);
      I total = __shfl_sync(kFullMask, upto, 31);
      bool falls = s.falls;
      if (a.B > 32) {
        I more = 0;
#pragma unroll 4
        for (int b = 32 + lane; b < a.B; b += 32) {
          const PrefillSeq q = prefill_seq<I>(a, b);
          if (q.code != 0 && blockIdx.x == 0) record_error(a.err, q.code);
          falls |= q.falls;
          more += length_of(q);
        }
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) more += __shfl_xor_sync(kFullMask, more, i);
        total += more;
      }
      const PrefillShares<I> shares(total, static_cast<int>(gridDim.x));
      auto cut_at = [&](int c) { return shares.begin(c); };
      const I x0 = cut_at(blockIdx.x), x1 = cut_at(blockIdx.x + 1);

      // sequences [chunk, chunk + 32) are looked at; their line begins at `before`
      int chunk = 0;
      I before = 0;
      auto next_chunk = [&] {
        before += __shfl_sync(kFullMask, upto, 31);
        chunk += 32;
        if (chunk < a.B) look(chunk);
        return chunk < a.B;
      };
      int published = 0;
      // (without a fall the sequences' rows are T at most, which bounds the total)
      bool more = !__any_sync(kFullMask, falls) && x1 > x0;
      while (more && before + __shfl_sync(kFullMask, upto, 31) <= x0) more = next_chunk();
      PrefillCut cut{};
      if (more) {
        // the item that x0 is in: sequence, key head, item of the head's line
        int seq = __ffs(__ballot_sync(kFullMask, before + upto > x0)) - 1;
        const I start = before + __shfl_sync(kFullMask, upto - mine, seq);
        PrefillLine<I> line(__shfl_sync(kFullMask, s.n, seq), __shfl_sync(kFullMask, s.L, seq), per_item, TPT, a.causal);
        const I head_length = line.length();
        int kvh = min(a.Hkv - 1, __float2int_rz(static_cast<float>(x0 - start) / static_cast<float>(head_length)));
        while (start + kvh * head_length > x0) --kvh;         // (the quotient was rounded)
        while (kvh + 1 < a.Hkv && start + (kvh + 1) * head_length <= x0) ++kvh;
        I at = start + kvh * head_length;           // where the item begins
        int tile = 0, step = line.tiles;
        while (step > 1) {                          // the last one that begins at or before x0
          step = (step + 31) / 32;
          const int t = tile + lane * step;
          tile += (__popc(__ballot_sync(kFullMask, t < line.tiles && at + line.begin(t) <= x0)) - 1) * step;
        }
        at += line.begin(tile);
        while (at < x1) {
          const I cost = line.cost(tile);
          const int keys = line.keys(tile), tiles = (keys + BN - 1) / BN;
          const bool one = line.one(tile);
          auto cut_in = [&](I x) {
            return prefill_cut<BN>(x - at, cost, one, one ? line.item1 : line.item, tiles, least);
          };
          const int from = cut_in(x0), to = cut_in(x1);
          if (from < to || (tiles == 0 && at >= x0)) {
            PrefillItem it;
            it.work = 1;
            it.seq = chunk + seq;
            it.kvh = kvh;
            it.L = line.L;
            it.key_base = __shfl_sync(kFullMask, s.k0, seq);
            it.once = line.tiles == 1;
            it.q_row = __shfl_sync(kFullMask, s.q0, seq) + tile * per_item;
            it.ntok = min(per_item, line.n - tile * per_item);
            it.two = it.ntok > TPT;
            it.off = line.L - line.n + tile * per_item;
            it.t0 = from;
            const int last0 = a.causal ? it.off + min(TPT, it.ntok) - 1 : line.L - 1;
            it.n0 = max(0, min(to, last0 < 0 ? 0 : last0 / BN + 1) - from);
            it.n1 = it.two ? to - from : 0;
            it.hidden = max(0, (a.causal ? it.off + 1 : it.L) / BN - from);
            const int cta = blockIdx.x;
            it.piece = from > 0 ? 2 * cta : (to < tiles ? 2 * cta + 1 : -1);
            it.bad_values = 0;
            if (from > 0) {                         // another CTA has the keys before
              int c = blockIdx.x - 1;
              while (cut_in(cut_at(c)) == from) --c;
              const bool first = cut_in(cut_at(c)) == 0;
              cut = PrefillCut{first ? 2 : 1, c, to == tiles, kvh, it.q_row, it.ntok};
            }
            if (published >= LY::ITEMS &&
                !__all_sync(kFullMask, mbar_wait_short(bar(i_empty(published)), i_phase(published) ^ 1))) {
              fail = true;
              break;
            }
            if (lane == 0) {
              *item_at(published) = it;
              mbar_arrive(bar(i_full(published)));
            }
            ++published;
          }
          at += cost;
          if (++tile == line.tiles) {
            tile = 0;
            if (++kvh == a.Hkv) {
              kvh = 0;
              uint32_t rest = seq < 31 ? __ballot_sync(kFullMask, mine > 0) >> (seq + 1) << (seq + 1) : 0;
              while (rest == 0 && next_chunk()) rest = __ballot_sync(kFullMask, mine > 0);
              if (rest == 0) break;
              seq = __ffs(rest) - 1;
              line = PrefillLine<I>(__shfl_sync(kFullMask, s.n, seq), __shfl_sync(kFullMask, s.L, seq), per_item, TPT, a.causal);
            }
          }
        }
      }
      if (a.cuts != nullptr && lane == 0) a.cuts[blockIdx.x] = cut;
      if (!fail) {
        if (published >= LY::ITEMS &&
            !__all_sync(kFullMask, mbar_wait_short(bar(i_empty(published)), i_phase(published) ^ 1)))
          fail = true;
        if (!fail && lane == 0) {
          item_at(published)->work = 0;
          mbar_arrive(bar(i_full(published)));
        }
      }
      };
      if (a.small) schedule(0); else schedule(0ll);
    } else if (warp == SOFT) {
      // -------------------------------------------------------- producer
      const uint32_t leader = elect_lane();
      const uint64_t stream_policy = l2_policy_evict_first();
      uint64_t keep_policy;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep_policy));
      const bool paged = a.key_starts == nullptr;
      const int past = paged ? static_cast<int>((static_cast<long long>(a.NB) * a.Hkv) << a.bs_log2) : 0;
      int at = 0, loaded = 0;                       // slot, tiles so far
      uint32_t phase = 0, qs0 = 0, qs1 = 0;         // of the slot; row tiles' loads so far
      auto wait = [&](int b, uint32_t parity) {
        if (!__all_sync(kFullMask, mbar_wait_short(bar(b), parity))) fail = true;
      };
      for (int slot = 0; !fail; ++slot) {
        wait(i_full(slot), i_phase(slot));
        if (fail) break;
        const PrefillItem it = *item_at(slot);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i_empty(slot)));
        if (!it.work) break;
        const int n = max(it.n0, it.n1);
        if (n == 0) continue;
        const uint64_t policy = it.once ? stream_policy : keep_policy;
        // paged: lane l knows where block l of a key tile is
        const int bs = 1 << a.bs_log2, per_tile = BN >> a.bs_log2, blocks = (it.L + bs - 1) >> a.bs_log2;
        const int32_t* table = paged ? a.block_tables + static_cast<size_t>(it.seq) * a.MB : nullptr;
        auto row_of = [&](int t) {                  // cache row of the lane's block in key tile t
          const int j = t * per_tile + lane;
          if (lane >= per_tile || j >= blocks) return past;    // past the end: reads as zero
          const int id = __ldg(table + j);
          if (id < 0 || id >= a.NB) {
            record_error(a.err, kDevBadBlock);
            return past;
          }
          return (id * a.Hkv + it.kvh) << a.bs_log2;
        };
        int y = paged ? row_of(it.t0) : 0;
        for (int i = 0; i < n; ++i) {
          const int y_next = paged && i + 1 < n ? row_of(it.t0 + i + 1) : 0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            wait(LY::KV_EMPTY + at, phase ^ 1);     // (a slot's first use does not wait)
            if (fail) break;
            const CUtensorMap* map = kv ? &tmV : &tmK;
            const uint32_t full = bar(LY::KV_FULL + at), dst = sb + LY::OFF_KV + at * LY::KV_TILE;
            if (leader) mbar_arrive_expect_tx(full, LY::KV_TILE);
            __syncwarp();
            if (paged && kv == 0) {
              // 64 channels of a block a load: a tile's panels keep all its keys together
#pragma unroll 4
              for (int b = 0; b < per_tile; ++b) {
                const int row = __shfl_sync(kFullMask, y, b);
#pragma unroll
                for (int c = 0; c < PANELS; ++c)
                  tma_2d_if(dst + c * (BN * 128) + (b << a.bs_log2) * 128, map, c * 64, row, full, policy, leader);
              }
            } else if (paged) {
              // a block a load: its panels one after the other
#pragma unroll 4
              for (int b = 0; b < per_tile; ++b)
                tma_3d_if(dst + (b << a.bs_log2) * (D * 2), map, 0, __shfl_sync(kFullMask, y, b), 0, full, policy, leader);
            } else {
#pragma unroll
              for (int c = 0; c < PANELS; ++c)
                tma_3d_if(dst + c * (BN * 128), map, c * 64, it.kvh, it.key_base + (it.t0 + i) * BN, full, policy, leader);
            }
            ++loaded;
            if (++at == ST) {
              at = 0;
              phase ^= 1;
            }
            if (i == 0 && (kv == 0 || it.two)) {    // row tile 0 after the first keys, 1 after their values
              uint32_t& uses = kv ? qs1 : qs0;
              wait(LY::Q_EMPTY + kv, (uses & 1) ^ 1);
              ++uses;
              if (fail) break;
              if (leader) mbar_arrive_expect_tx(bar(LY::Q_FULL + kv), PANELS * TPT * a.G * 128);
              __syncwarp();
#pragma unroll
              for (int c = 0; c < PANELS; ++c)
                tma_3d_if(sb + kv * LY::Q_TILE + c * 16384, &tmQ, c * 64, it.kvh * a.G, it.q_row + kv * TPT,
                          bar(LY::Q_FULL + kv), stream_policy, leader);
            }
          }
          if (fail) break;
          y = y_next;
        }
      }
      // Nothing may land or arrive in this CTA's shared memory after it has
      // left: every slot's last load was read and its release has come.
      for (int r = max(0, loaded - ST); r < loaded; ++r) {
        const bool landed = mbar_wait(bar(LY::KV_FULL + r % ST), (r / ST) & 1, 100000000ull);
        if (!fail && landed) mbar_wait(bar(LY::KV_EMPTY + r % ST), (r / ST) & 1, 100000000ull);
      }
      for (int x = 0; x < 2; ++x) {
        const uint32_t uses = x ? qs1 : qs0;
        if (uses == 0) continue;
        mbar_wait(bar(LY::Q_FULL + x), (uses - 1) & 1, 100000000ull);
        if (!fail) mbar_wait(bar(LY::Q_EMPTY + x), (uses - 1) & 1, 100000000ull);
      }
    } else if (warp == SOFT + 1) {
      // -------------------------------------------------------- matrix products
      const uint32_t leader = elect_lane();
      // (a negative scale: S of -Q, bit 13)
      const uint32_t idesc_qk = umma_idesc_f16(BF, 0, 0, BN, 128) | (a.negative ? 1u << 13 : 0u);
      const uint32_t idesc_pv = umma_idesc_f16(BF, 0, 1, D, 128);
      // descriptors: eight rows of 128 bytes an atom (stride 1024), version 1,
      // 128-byte swizzle; V's leading offset is from one 64-channel panel to the next
      constexpr uint32_t kHi = (1024 >> 4) | 1u << 14 | 2u << 29;
      const uint32_t q_lo = (sb >> 4) | 1u << 16, k_lo = ((sb + LY::OFF_KV) >> 4) | 1u << 16;
      const uint32_t v_lo = ((sb + LY::OFF_KV) >> 4) | (128u << run_log2 >> 4) << 16;
      uint32_t v_step[BN / 16];                     // where 16 keys begin in a V tile
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        v_step[kk] = ((kk >> (run_log2 - 4)) * (D * 2u << run_log2) + (kk & ((1 << (run_log2 - 4)) - 1)) * 2048u) >> 4;
      auto qk = [&](int s, int x, int at) {         // S buffer s = Q tile x . K of slot `at`
        tc_fence_after();
        const uint32_t a_lo = q_lo + x * (LY::Q_TILE >> 4), b_lo = k_lo + at * (LY::KV_TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss(tmem + LY::S_COL(s), a_lo + (kk >> 2) * (16384 >> 4) + (kk & 3) * 2,
                  b_lo + (kk >> 2) * (BN * 128 >> 4) + (kk & 3) * 2, kHi, idesc_qk, kk > 0, leader);
        umma_commit_if(bar(LY::S_FULL + s), leader);
      };
      auto pv = [&](int s, int x, int at, uint32_t parity, bool first, bool last) {   // O tile x += P of buffer s . V of slot `at`
        tc_fence_after();
        const uint32_t b_lo = v_lo + at * (LY::KV_TILE >> 4);
        constexpr int PARTS = BN / 64, PER = 2;     // of P; groups of 16 keys of a part, in each half
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          if (q > 0) {
            if (!__all_sync(kFullMask, mbar_wait_spin(bar(LY::P_FULL + s + q * 3), parity))) fail = true;
            tc_fence_after();
          }
#pragma unroll
          for (int g = 0; g < 2 * PER; ++g) {
            const int kk = (g / PER) * (BN / 32) + q * PER + g % PER;
            umma_ts(tmem + LY::O_COL(x), tmem + LY::S_COL(s) + LY::P_COL(kk), b_lo + v_step[kk], kHi, idesc_pv,
                    !first || g > 0 || q > 0, leader);
          }
        }
        umma_commit_if(bar(LY::O_DONE + x), leader);
        if (last) umma_commit_if(bar(LY::O_LAST + x), leader);
      };
      // The ring's tiles come K(0) V(0) K(1) V(1) ...; slots and phases of the
      // next tile that is waited for and of the next to be released.
      int at = 0;
      uint32_t phase = 0;
      auto landed = [&] {
        if (!__all_sync(kFullMask, mbar_wait_spin(bar(LY::KV_FULL + at), phase))) fail = true;
        const int slot = at;
        if (++at == ST) {
          at = 0;
          phase ^= 1;
        }
        return slot;
      };
      // Two tiles in turn: their barriers are asked at once, as an answer takes long.
      auto landed_two = [&](int& v, int& k) {
        v = at;
        k = at + 1 == ST ? 0 : at + 1;
        const uint32_t next = at + 1 == ST ? phase ^ 1 : phase;
        const bool both = mbar_try_both(bar(LY::KV_FULL + v), phase, bar(LY::KV_FULL + k), next);
        if (!__all_sync(kFullMask, both)) {
          landed();
          landed();
          return;
        }
        at = k + 1 == ST ? 0 : k + 1;
        phase = k + 1 == ST ? next ^ 1 : next;
      };
      uint32_t qs0 = 0, qs1 = 0, su0 = 0, su1 = 0, su2 = 0, ou0 = 0, ou1 = 0;   // uses so far: Q, S buffers, O tiles
      auto have_p = [&](int s, uint32_t& uses) {    // P of S buffer s has been written
        if (!__all_sync(kFullMask, mbar_wait_spin(bar(LY::P_FULL + s), uses & 1))) fail = true;
        ++uses;
      };
      // V tiles that hide something: the values warp is told of tile i when K(i)
      // is there (then it may wait for V(i): all tiles before have landed).  That
      // may be while it works on the one before, hence two barriers each.
      uint32_t told = 0, cleaned = 0;
      auto tell = [&](bool some) {
        if (!some) return;
        if (lane == 0) mbar_arrive(bar(LY::V_HERE + (told & 1)));
        ++told;
      };
      auto clean = [&] {                            // the V tile's values have been looked over
        if (!__all_sync(kFullMask, mbar_wait_spin(bar(LY::V_CLEAN + (cleaned & 1)), (cleaned >> 1) & 1))) fail = true;
        ++cleaned;
      };
      auto have_o = [&](int x, uint32_t& uses) {    // O tile x has been read by the item before
        if (uses > 0 && !__all_sync(kFullMask, mbar_wait_spin(bar(LY::O_FREE + x), (uses - 1) & 1))) fail = true;
        ++uses;
      };
      auto have_q = [&](int x, uint32_t& uses) {
        if (!__all_sync(kFullMask, mbar_wait_spin(bar(LY::Q_FULL + x), uses & 1))) fail = true;
        ++uses;
      };
      uint32_t ring = 0;                            // tiles of the items before
      bool ahead = false;                           // S0 of the item's first keys is under way already
      for (int slot = 0; !fail; ++slot) {
        if (!__all_sync(kFullMask, mbar_wait_spin(bar(i_full(slot)), i_phase(slot)))) {
          fail = true;
          break;
        }
        const PrefillItem* item = item_at(slot);
        const int work = item->work, two = item->two, n0 = item->n0, n1 = item->n1, n = max(n0, n1);
        const int hidden = item->hidden;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i_empty(slot)));
        if (!work) break;
        if (n == 0) continue;
        int k = landed();
        tell(hidden == 0);
        if (!ahead) {
          have_q(0, qs0);
          if (fail) break;
          if (n0 > 0) qk(0, 0, k);
        }
        if (n0 <= 1) umma_commit_if(bar(LY::Q_EMPTY), leader);
        if (LY::NQ == 2 && two) {
          have_q(1, qs1);
          if (fail) break;
          qk(1, 1, k);
          if (n1 == 1) umma_commit_if(bar(LY::Q_EMPTY + 1), leader);
        }
        umma_commit_if(bar(LY::KV_EMPTY + k), leader);
        ahead = false;
        if (LY::NQ == 2 && two) {
          for (int i = 0; i < n; ++i) {
            int v;
            if (i + 1 < n) {
              landed_two(v, k);
              tell(i + 1 >= hidden);
            } else {
              v = landed();
            }
            if (i >= hidden) clean();
            if (i < n0) {
              have_p(0, su0);
              if (i == 0) have_o(0, ou0);
              if (fail) break;
              pv(0, 0, v, (su0 - 1) & 1, i == 0, i + 1 == n0);
            }
            if (fail) break;
            if (i + 1 < n0) {
              qk(0, 0, k);
              if (i + 2 == n0) umma_commit_if(bar(LY::Q_EMPTY), leader);
            } else if (i + 2 >= n && !ahead) {
              // Row tile 0 is through: on to the next item's first keys, if they
              // and its row tile are there.  (Every ring tile but the last two
              // or three of this item has landed, so the slot of those keys is
              // at their phase or the one before.)
              const uint32_t next = ring + 2 * n;
              const PrefillItem* then = item_at(slot + 1);
              bool go = mbar_test_wait(bar(i_full(slot + 1)), i_phase(slot + 1)) && then->work &&
                        then->n0 > 0 && mbar_test_wait(bar(LY::Q_FULL), qs0 & 1) &&
                        mbar_test_wait(bar(LY::KV_FULL + next % ST), (next / ST) & 1);
              go = __all_sync(kFullMask, go);
              if (go) {
                ++qs0;
                ahead = true;
                qk(0, 0, next % ST);
              }
            }
            if (i < n1) {
              have_p(1, su1);
              if (i == 0) have_o(1, ou1);
              if (fail) break;
              pv(1, 1, v, (su1 - 1) & 1, i == 0, i + 1 == n1);
            }
            umma_commit_if(bar(LY::KV_EMPTY + v), leader);
            if (i + 1 < n1) {
              qk(1, 1, k);
              if (i + 2 == n1) umma_commit_if(bar(LY::Q_EMPTY + 1), leader);
            }
            if (i + 1 < n) umma_commit_if(bar(LY::KV_EMPTY + k), leader);
          }
        } else {
          for (int i = 0; i < n; ++i) {
            int v;
            if (i + 1 == n) {
              v = landed();
            } else {
              landed_two(v, k);
              tell(i + 1 >= hidden);
              if (fail) break;
              qk(i & 1 ? 0 : 2, 0, k);
              if (i + 2 == n) umma_commit_if(bar(LY::Q_EMPTY), leader);
              umma_commit_if(bar(LY::KV_EMPTY + k), leader);
            }
            if (i >= hidden) clean();
            if (i & 1) have_p(2, su2); else have_p(0, su0);
            if (i == 0) have_o(0, ou0);
            if (fail) break;
            pv(i & 1 ? 2 : 0, 0, v, (i & 1 ? su2 - 1 : su0 - 1) & 1, i == 0, i + 1 == n);
            umma_commit_if(bar(LY::KV_EMPTY + v), leader);
          }
        }
        ring += 2 * n;
      }
    } else {
      // -------------------------------------------------------- values
      int ring = 0;
      uint32_t here = 0;
      for (int slot = 0; !fail; ++slot) {
        if (!__all_sync(kFullMask, mbar_wait_short(bar(i_full(slot)), i_phase(slot)))) {
          fail = true;
          break;
        }
        PrefillItem* item = item_at(slot);
        if (!item->work) break;
        const int n = max(item->n0, item->n1), L = item->L, t0 = item->t0;
        const int seen = a.causal ? min(L, item->off + 1) : L;   // keys that every row sees
        for (int i = item->hidden; i < n; ++i) {
          const int rv = ring + 2 * i + 1;
          if (!__all_sync(kFullMask, mbar_wait_short(bar(LY::V_HERE + (here & 1)), (here >> 1) & 1) &&
                                         mbar_wait_short(bar(LY::KV_FULL + rv % ST), (rv / ST) & 1))) {
            fail = true;
            break;
          }
          const uint32_t tile = sb + LY::OFF_KV + (rv % ST) * LY::KV_TILE;
          const int key0 = (t0 + i) * BN, first = max(0, seen - key0), end = min(BN, L - key0);
          // rows [first, end): a product with zero is no number where the value is none
          uint32_t odd[4] = {0, 0, 0, 0};
          // (four rows at a time; rows past either end are read as the last one there)
#pragma unroll 4
          for (int r0 = first < end ? first & ~3 : end; r0 < end; r0 += 4) {
            const int vr = min(max(r0 + (lane >> 3), first), end - 1);
            const uint32_t from = tile + (vr >> run_log2) * (D * 2 << run_log2) + (vr & ((1 << run_log2) - 1)) * 128 + (lane & 7) * 16;
#pragma unroll
            for (int c = 0; c < PANELS; ++c) {
              uint32_t d[4];
              asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                           : "r"(from + (c << run_log2) * 128));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if constexpr (BF)
                  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(odd[e]) : "r"(d[e]), "r"(0));
                else
                  asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(odd[e]) : "r"(d[e]), "r"(0));
              }
            }
          }
          const uint32_t any = (odd[0] | odd[1] | odd[2] | odd[3]) & 0x7fff7fffu;   // (zeros of either sign are fine)
          const bool bad = __any_sync(kFullMask, any != 0);
          if (bad || end < BN) {
            for (int u = (bad ? first : end) * (D / 8) + lane; u < BN * (D / 8); u += 32) {
              const int vr = u / (D / 8), ch = u % (D / 8);
              const uint32_t at = tile + (vr >> run_log2) * (D * 2 << run_log2) + ((ch >> 3) << run_log2) * 128 +
                                  (vr & ((1 << run_log2) - 1)) * 128 + (ch & 7) * 16;
              uint32_t d[4] = {0, 0, 0, 0};
              if (vr < end) {
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                             : "r"(at));
                constexpr uint32_t kExp = BF ? 0x7f807f80u : 0x7c007c00u, kOne = BF ? 0x00800080u : 0x04000400u;
#pragma unroll
                for (int e = 0; e < 4; ++e)         // a half whose exponent is all ones becomes zero
                  d[e] &= ~(((((d[e] & kExp) + kOne) & 0x80008000u) >> 15) * 0xffffu);
              }
              asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(d[0]), "r"(d[1]), "r"(d[2]),
                           "r"(d[3])
                           : "memory");
            }
            if (bad && lane == 0) item->bad_values = 1;
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(LY::V_CLEAN + (here & 1)));
          ++here;
        }
        if (lane == 0) mbar_arrive(bar(i_empty(slot)));
        ring += 2 * n;
      }
    }
  } else {
    // ---------------------------------------------------------- softmax
    // Warps w and w + 4 of a row tile have the same rows and a half of the keys
    // each (and of the output's channels); they meet at a barrier of their own.
    // So none of them leaves an item early: after a failed wait a warp skips its
    // later waits and runs on with whatever is there, and before the next item
    // the two leave together.
    constexpr float kShift = BF ? -8.f : 7.f;       // P is 2^kShift times the weight relative to m
    constexpr int HN = BN / 2, HD = D / 2;
    const int w = warp >> 3, h = (warp >> 2) & 1, pair = 1 + w * 4 + (warp & 3);
    const int r = (warp & 3) * 32 + lane;           // row of the tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float* xch = reinterpret_cast<float*>(smem + LY::OFF_XCH) + w * 256;
    float *own = xch + h * 128 + r, *others = xch + (h ^ 1) * 128 + r;
    const int tl = r / a.G;                         // token of the row within its tile
    const bool has_token = tl < TPT;
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    const float c = a.scale_log2;
    // S buffers' uses, own O tile's products and its items so far
    int su = 0, su2 = 0, od = 0, outs = 0;
    auto wait = [&](int b, uint32_t parity) {
      if (!fail && !__all_sync(kFullMask, mbar_wait_short(bar(b), parity))) fail = true;
    };
    for (int slot = 0;; ++slot) {
      wait(i_full(slot), i_phase(slot));
      if (named_bar_or(pair, 64, fail)) {
        fail = true;
        break;
      }
      PrefillItem* item = item_at(slot);
      if (!item->work) break;
      const int two = item->two, L = item->L, off = item->off, t0 = item->t0;
      const int n = w == 0 ? item->n0 : item->n1;
      const int j = w * TPT + tl;                   // token of the row within the item
      const bool valid = has_token && j < item->ntok && (w == 0 || two);
      const int lim = a.causal ? off + j : L - 1;   // last key that the row sees
      const int all_see = __reduce_min_sync(kFullMask, valid ? lim : 0x7fffffff);   // last key that all of the warp's rows see
      // The row's reference.  m c is rounded, by up to 2^-24 of it, and all of the
      // row's weights are off by one factor.  So that this stays small, far from
      // zero the reference is held apart, m is as in a row that has seen nothing,
      // which raises the reference at every key tile, and the scores take it off
      // before they are scaled.
      float m = -INFINITY, held = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      bool raised = true;                           // by the last key tile (or the item before used the exchange)
      for (int i = 0; i < n; ++i) {
        const int s = two ? w : (i & 1 ? 2 : 0);
        wait(LY::S_FULL + s, (s == 2 ? su2 : su) & 1);
        s == 2 ? ++su2 : ++su;
        tc_fence_after();
        const uint32_t mine = lanes + LY::S_COL(s) + h * HN;
        float x[HN];
#pragma unroll
        for (int q = 0; q < HN / 32; ++q) tmem_ld32(mine + q * 32, x + q * 32);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < HN / 32; ++q) tmem_ready32(x + q * 32);
        const int col0 = (t0 + i) * BN + h * HN;
        if (col0 + HN - 1 > all_see) {
          const int sees = lim - col0;              // (then a comparison has a constant: 2% of short prompts)
#pragma unroll
          for (int e = 0; e < HN; ++e) x[e] = e <= sees ? x[e] : -INFINITY;
        }
        float top[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) top[q] = fmaxf(x[q], x[4 + q]);
#pragma unroll
        for (int e = 8; e < HN; e += 8) {
#pragma unroll
          for (int q = 0; q < 4; ++q) top[q] = fmaxf(top[q], fmaxf(x[e + q], x[e + 4 + q]));
        }
        const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // (rows of no token have no say: they hold other sequences' queries or what
        // was in shared memory, and the item's rows would be rounded differently)
        raised = named_bar_or(pair, 64, i == 0 || (valid && (mt - m) * c > 8.f));
        if (raised) {
          // raise the reference to the whole row's maximum
          *own = mt;
          named_bar_sync(pair, 64);
          const float was = m == -INFINITY ? held : m, up = fmaxf(was, fmaxf(mt, *others));
          const float keep = was == -INFINITY ? 0.f : fast_exp2((was - up) * c);
          if (i > 0) {
            // O holds the products up to the last tile's.  (That barrier is at
            // this phase or the next: the one before had ended when S was
            // there, the one after waits for this tile's P.)
            wait(LY::O_DONE + w, (od + i - 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < HD / 16; ++q) {
              float o[16];
              tmem_ld16(lanes + LY::O_COL(w) + h * HD + q * 16, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= keep;
              tmem_st16(lanes + LY::O_COL(w) + h * HD + q * 16, o);
            }
          }
          l2.x *= keep;
          l2.y *= keep;
          const bool far = valid && up != -INFINITY && fabsf(up * c) > kPrefillFar;
          if (__any_sync(kFullMask, far)) {
            // (in pairs, as what skips this pays for its length)
            const float less = far ? -up : 0.f;
#pragma unroll
            for (int e = 0; e < HN; e += 2) {
              const float2 y = add2(make_float2(x[e], x[e + 1]), make_float2(less, less));
              x[e] = y.x;
              x[e + 1] = y.y;
            }
          }
          m = far ? -INFINITY : up;
          held = far ? up : -INFINITY;
        }
        const float mc = (m == -INFINITY ? 0.f : m * c) - kShift;
        const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
        float2 sum[2] = {l2, make_float2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < HN / 32; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 p = fma2(make_float2(x[q * 32 + 2 * e], x[q * 32 + 2 * e + 1]), c2, mc2);
            p.x = fast_exp2(p.x);
            p.y = fast_exp2(p.y);
            sum[e & 1] = add2(sum[e & 1], p);
            pk[e] = pack2<BF>(p.x, p.y);
          }
          tmem_st16u(mine + q * 16, pk);
          // (a part at a time, so that the products with the first one begin)
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(LY::P_FULL + s + q * 3));
        }
        l2 = add2(sum[0], sum[1]);
      }
      // -------------------------------------------------------- the item's rows out
      // (while the last products are under way)
      if (raised) named_bar_sync(pair, 64);         // the last maximum has been read
      float l = l2.x + l2.y;
      *own = l;
      named_bar_sync(pair, 64);
      l += *others;
      const int kvh = item->kvh, piece = item->piece, head = r - tl * a.G;
      const size_t row = static_cast<size_t>(item->q_row + j) * a.Hq + kvh * a.G + head;
      const size_t prow = static_cast<size_t>(max(piece, 0)) * a.rows + j * a.G + head;
      const float inv = piece >= 0 ? 1.f : (l > 0.f ? 1.f / l : 0.f);
      // CW channels at a time.  So that a warp's stores fill whole sectors of few
      // lines, NC lanes exchange their rows' 32-byte chunks first: lane l of them
      // then has chunk l of each of their rows, that of the row of lane l ^ e as its e-th.
      constexpr int CW = HD < 64 ? HD : 64, NC = CW / 16;
      const int sub = lane % NC;
      uint32_t rows_at[NC];                         // (fewer than 2^32 - 1 rows of 128 bytes or more fit into the memory)
#pragma unroll
      for (int e = 0; e < NC; ++e)
        rows_at[e] = __shfl_xor_sync(kFullMask, valid ? static_cast<uint32_t>(row) : 0xffffffffu, e);
      if (n > 0) {
        wait(LY::O_LAST + w, outs & 1);
        ++outs;
        tc_fence_after();
      }
#pragma unroll 1
      for (int q = 0; q < HD / CW; ++q) {
        const int ch0 = h * HD + q * CW;            // first channel
        float o[CW];
        if (n > 0) {
#pragma unroll
          for (int g = 0; g < CW / 32; ++g) tmem_ld32(lanes + LY::O_COL(w) + ch0 + g * 32, o + g * 32);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < CW / 32; ++g) tmem_ready32(o + g * 32);
          if (q + 1 == HD / CW) {                   // the next item's products may go there
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(LY::O_FREE + w));
          }
#pragma unroll
          for (int e = 0; e < CW; e += 2) {
            const float2 y = mul2(make_float2(o[e], o[e + 1]), make_float2(inv, inv));
            o[e] = y.x;
            o[e + 1] = y.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < CW; ++e) o[e] = 0.f;
        }
        if (piece >= 0) {
          if (valid) {
            float* dst = a.part_o + prow * D + ch0;
#pragma unroll
            for (int e = 0; e < CW; e += 8) store32_part(dst + e, o + e);
          }
        } else {
          uint32_t pk[NC][8];
#pragma unroll
          for (int e = 0; e < CW / 2; ++e) pk[e / 8][e % 8] = pack2<BF>(o[2 * e], o[2 * e + 1]);
#pragma unroll
          for (int st = 1; st < NC; st <<= 1) {     // chunk sub ^ e to the e-th place
            const bool up = sub & st;
#pragma unroll
            for (int g = 0; g < NC; ++g) {
              if (g & st) continue;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t lo = pk[g][e], hi = pk[g | st][e];
                pk[g][e] = up ? hi : lo;
                pk[g | st][e] = up ? lo : hi;
              }
            }
          }
#pragma unroll
          for (int g = 0; g < NC; ++g) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (g > 0) pk[g][e] = __shfl_xor_sync(kFullMask, pk[g][e], g);
            if (rows_at[g] != 0xffffffffu)
              store32(a.out + static_cast<size_t>(rows_at[g]) * D + ch0 + sub * 16, pk[g], wide);
          }
        }
      }
      if (n > 0 && item->bad_values) {
        // values that were cleared, for the rows that see them
        __syncwarp();                               // (the row may have been stored by another lane)
        const int to = valid ? min(min(lim, L - 1), (t0 + n) * BN - 1) : -1;
        for (int key = max(max(off + 1, 0), t0 * BN); key <= to; ++key) {
          const uint16_t* v;
          if (a.key_starts != nullptr) {
            v = a.v + (item->key_base + key) * a.v_stride + static_cast<size_t>(kvh) * D;
          } else {
            const int id = a.block_tables[static_cast<size_t>(item->seq) * a.MB + (key >> a.bs_log2)];
            if (id < 0 || id >= a.NB) continue;
            v = a.v + (((static_cast<size_t>(id) * a.Hkv + kvh) << a.bs_log2) + (key & ((1 << a.bs_log2) - 1))) * D;
          }
#pragma unroll 1
          for (int ch = h * HD; ch < h * HD + HD; ++ch) {
            const float y = unpack2<BF>(v[ch]).x;
            if (fabsf(y) <= 3.402823466e38f) continue;
            if (piece >= 0) {
              a.part_o[prow * D + ch] += y;
            } else {
              uint16_t* at = a.out + row * D + ch;
              *at = to_elem<BF>(unpack2<BF>(*at).x + y);
            }
          }
        }
      }
      if (piece >= 0 && valid && h == 0)
        a.part_ml[prow] = make_float2(l == 0.f ? -INFINITY : (m == -INFINITY ? held : m), l);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(i_empty(slot)));
      }
      od += n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
  if (fail && lane == 0) record_error(a.err, kDevTimeout);
}

}  // namespace pkv
