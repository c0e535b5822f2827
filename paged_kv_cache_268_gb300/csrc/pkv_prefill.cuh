// Prompt-side attention on the 5th-generation tensor cores (tcgen05, TMEM),
// warp-specialised and persistent: softmax(q . K^T scale) . V of many rows a
// sequence, over the paged cache or over packed keys and values.
//
// The query rows of one key head are taken together: row r of a tile of 128 is
// token r / G, head r % G of its group, so grouped heads share every key tile
// that is read, and a few new tokens of many heads still fill a tile (tiles
// hold whole tokens: 128 / G of them).  An item is up to two row tiles of one
// (sequence, key head), over the keys that its rows see, or a partition of
// them.  The CTAs, one an SM, take the items in turn.
//
//   warps 0-3, 4-7  softmax of row tile 0 and 1; a thread owns a row
//   warp 8          producer: Q by TMA, K and V tiles into a ring of slots
//   warp 9          issues the matrix products
//   warp 10         finds the CTA's next item, one ahead
//
// S = Q K^T (both K-major in shared memory) goes to TMEM; a softmax thread
// reads its row, p = 2^(s c - m c), and writes P over S in 16 bits, from where
// it is the first operand of O += P V (V read MN-major from its tile).  While
// one row tile is in softmax, the tensor cores work on the other: P0 V, S0 of
// the next keys, P1 V, S1 of the next keys.  With a single row tile the two S
// buffers take the key tiles in turn instead, S one tile ahead of P.
// m follows the row's running maximum only where that grows by more than 2^8;
// then O and the sum are rescaled (rare: the first key tile sets it).  P in
// binary16 is scaled by 2^7 so that weights of down to 2^-21 of the largest
// keep all their bits; the largest, 2^15, is still in range.  The sums are of
// P in FP32, before its rounding.
//
// Hidden keys: P is zero there, but 0 times an infinity or NaN is not.  In key
// tiles that hide something from some row, values past the sequence's end are
// cleared, and those that are no numbers as well (and kept in mind: at the
// end they are added for the rows that see them, whose weights are positive).
//
// Every wait is bounded; a role that gives up leaves, the others follow, and
// the device error word is set.
#pragma once

#include "pkv_prefill.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr uint32_t kFullMask = 0xffffffffu;

template <int D>
struct PrefillLayout {
  static constexpr int NQ = prefill_row_tiles(D);
  static constexpr int BN = prefill_key_tile(D);
  static constexpr int PANELS = D / 64;             // 128-byte columns of a row
  static constexpr int Q_TILE = 128 * D * 2;
  static constexpr int KV_TILE = BN * D * 2;
  static constexpr int STAGES = D == 64 ? 8 : 5;
  static constexpr int OFF_KV = NQ * Q_TILE;
  static constexpr int OFF_BAR = OFF_KV + STAGES * KV_TILE;
  static constexpr int KV_FULL = 0, KV_EMPTY = STAGES, Q_FULL = 2 * STAGES, Q_EMPTY = Q_FULL + 1,
                       S_FULL = Q_FULL + 2, P_FULL = S_FULL + 3, O_DONE = P_FULL + 3,
                       O_FREE = O_DONE + 2, I_FULL = O_FREE + 2, I_EMPTY = I_FULL + 2,
                       NBAR = I_EMPTY + 2;
  static constexpr int OFF_ITEM = OFF_BAR + NBAR * 8;
  static constexpr int OFF_TMEM = OFF_ITEM + 2 * 80;
  static constexpr int BYTES = OFF_TMEM + 16 + 1024;
  // S buffer 0, 1: of row tile 0, 1; 2: buffer 1 with a single row tile (a
  // barrier of its own, so that each has one group of softmax warps only)
  static constexpr int S_COL(int s) { return s > 0 ? BN : 0; }
  static constexpr int O_COL(int x) { return 256 + x * D; }
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

constexpr int kPrefillThreads = 384;
constexpr int kPrefillRegs = 168;     // a thread's at launch, which setmaxnreg shares out anew

struct PrefillItem {
  int work;                      // 0: no more items
  int seq, kvh;
  int q_row, ntok;               // its rows: tokens [q_row, q_row + ntok)
  int two;                       // both row tiles are used
  int L;                         // keys of the sequence
  int off;                       // position of the first token
  int t0;                        // first key tile
  int n0, n1;                    // key tiles that row tile 0, 1 sees from there
  int key_base;                  // packed: row of the first key
  int once;                      // no other item reads these keys
  int parts, part;
  int bad_values;                // values that are no numbers were cleared
  long long row;                 // partial row of the sequence's first row
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

// D[tmem] (+)= A[tmem] * B[smem], one elected thread.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
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
// `code` then says what is wrong.
struct PrefillSeq {
  int q0, n, k0, L, code;
};
__device__ __forceinline__ PrefillSeq prefill_seq(const PrefillArgs& a, int b) {
  PrefillSeq s{0, 0, 0, 0, 0};
  if (b >= a.B) return s;
  s.q0 = a.query_starts[b];
  const int q1 = a.query_starts[b + 1];
  if (s.q0 < 0 || q1 < s.q0 || q1 > a.T) {
    s.code = kDevBadStarts;
    return s;
  }
  int L;
  if (a.key_starts != nullptr) {
    s.k0 = a.key_starts[b];
    const int k1 = a.key_starts[b + 1];
    if (s.k0 < 0 || k1 < s.k0 || k1 > a.max_keys) {
      s.code = kDevBadStarts;
      return s;
    }
    L = k1 - s.k0;
  } else {
    L = a.context_lens[b];
    if (L < 0 || L > a.max_keys) {
      s.code = kDevBadContext;
      return s;
    }
  }
  s.L = L;
  s.n = q1 - s.q0;
  return s;
}

// Partitions of a sequence of `rows` rows a key head and `tiles` key tiles:
// (count, tiles of each).  `total` is the key tiles of all items, `unit` keys
// in tiles that make the smallest partition.  Items that are longer than a
// half of a CTA's share of the work (a quarter where they have few rows, whose
// partial results cost little) are cut to that length.
__device__ __forceinline__ int2 prefill_parts(const PrefillArgs& a, long long total, int rows, int tiles,
                                              int unit) {
  if (a.plan == nullptr || rows == 0 || tiles == 0) return make_int2(1, max(tiles, 1));
  long long most = a.part_tiles;
  if (most == 0) {
    const int units = a.ctas * (rows <= kPrefillFewRows ? kPrefillFewUnits : kPrefillUnits);
    most = max(static_cast<long long>(unit), (total + units - 1) / units);
  }
  if (tiles <= most) return make_int2(1, tiles);
  const int parts = static_cast<int>((tiles + most - 1) / most);
  const int per = (tiles + parts - 1) / parts;
  return make_int2((tiles + per - 1) / per, per);
}

template <bool BF, int D>
__global__ void __launch_bounds__(kPrefillThreads, 1)
    prefill_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using LY = PrefillLayout<D>;
  constexpr int BN = LY::BN, ST = LY::STAGES, PANELS = LY::PANELS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + LY::OFF_BAR + 8 * i; };
  auto item_at = [&](int i) { return reinterpret_cast<PrefillItem*>(smem + LY::OFF_ITEM + (i & 1) * 80); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + LY::OFF_TMEM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int TPT = 128 / a.G;                       // tokens of a row tile

  if (tid < LY::NBAR) {
    int count = 1;
    if (tid >= LY::P_FULL && tid < LY::P_FULL + 3) count = 4;
    if (tid >= LY::O_FREE && tid < LY::O_FREE + 2) count = 4;
    if (tid >= LY::I_EMPTY && tid < LY::I_EMPTY + 2) count = 10;
    mbar_init(bar(tid), count);
  }
  if (warp == 8 && lane == 0) {
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

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 10) {
      // -------------------------------------------------------- next item
      // Sequences are looked at 32 at a time, a lane each.  Within a sequence
      // the last rows, which see most, come first.
      const int unit = max(1, kPrefillMinPart / BN);
      const int per_item = TPT * LY::NQ;            // tokens
      long long total = 0;
      auto tiles_of = [&](const PrefillSeq& s) { return (s.L + BN - 1) / BN; };
      if (a.plan != nullptr && a.part_tiles == 0) {
        for (int b = lane; b < a.B; b += 32) {
          const PrefillSeq s = prefill_seq(a, b);
          total += static_cast<long long>((s.n + per_item - 1) / per_item) * a.Hkv * tiles_of(s);
        }
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) total += __shfl_xor_sync(kFullMask, total, i);
      }
      int chunk = 0;
      long long before = 0, rows_before = 0;        // items and partial rows of the chunks before
      PrefillSeq s;
      int2 cut;
      long long mine, upto, row;                    // items of the lane's sequence, up to its end; its partial row
      auto look = [&](int b0) {
        s = prefill_seq(a, b0 + lane);
        if (s.code != 0 && blockIdx.x == 0) record_error(a.err, s.code);
        cut = prefill_parts(a, total, s.n * a.G, tiles_of(s), unit);
        mine = static_cast<long long>((s.n + per_item - 1) / per_item) * a.Hkv * cut.x;
        const long long rows = cut.x > 1 ? static_cast<long long>(s.n) * a.Hq * cut.x : 0;
        upto = mine;
        row = rows;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
          const long long u = __shfl_up_sync(kFullMask, upto, i), r = __shfl_up_sync(kFullMask, row, i);
          if (lane >= i) {
            upto += u;
            row += r;
          }
        }
        row += rows_before - rows;
      };
      if (a.plan != nullptr && blockIdx.x == 0) {   // for the reduce
        for (int b0 = 0; b0 < a.B; b0 += 32) {
          look(b0);
          if (b0 + lane < a.B) a.plan[b0 + lane] = PrefillPlan{cut.x, cut.y, row};
          rows_before = __shfl_sync(kFullMask, row + (cut.x > 1 ? static_cast<long long>(s.n) * a.Hq * cut.x : 0), 31);
        }
        rows_before = 0;
      }
      look(0);
      int slot = 0;
      for (long long id = blockIdx.x;; id += gridDim.x) {
        long long all = __shfl_sync(kFullMask, upto, 31);
        while (chunk < a.B && id >= before + all) {
          before += all;
          rows_before = __shfl_sync(kFullMask, row + (cut.x > 1 ? static_cast<long long>(s.n) * a.Hq * cut.x : 0), 31);
          chunk += 32;
          if (chunk >= a.B) break;
          look(chunk);
          all = __shfl_sync(kFullMask, upto, 31);
        }
        PrefillItem it;
        it.work = chunk < a.B;
        if (it.work) {
          const int from = __ffs(__ballot_sync(kFullMask, upto > id - before)) - 1;
          long long r = id - before - (upto - mine);
          r = __shfl_sync(kFullMask, r, from);
          it.seq = chunk + from;
          const int n = __shfl_sync(kFullMask, s.n, from), q0 = __shfl_sync(kFullMask, s.q0, from);
          it.L = __shfl_sync(kFullMask, s.L, from);
          it.key_base = __shfl_sync(kFullMask, s.k0, from);
          it.parts = __shfl_sync(kFullMask, cut.x, from);
          const int per = __shfl_sync(kFullMask, cut.y, from);
          it.row = __shfl_sync(kFullMask, row, from);
          const int tiles = (n + per_item - 1) / per_item;
          const int rem = static_cast<int>(r % (static_cast<long long>(a.Hkv) * it.parts));
          const int tile = tiles - 1 - static_cast<int>(r / (static_cast<long long>(a.Hkv) * it.parts));
          it.part = rem / a.Hkv;
          it.kvh = rem % a.Hkv;
          it.once = tiles == 1;
          it.q_row = q0 + tile * per_item;
          it.ntok = min(per_item, n - tile * per_item);
          it.two = it.ntok > TPT;
          it.off = it.L - n + tile * per_item;
          const int last0 = a.causal ? it.off + min(TPT, it.ntok) - 1 : it.L - 1;
          const int last1 = a.causal ? it.off + it.ntok - 1 : it.L - 1;
          it.t0 = it.part * per;
          const int end = it.t0 + per;
          it.n0 = max(0, min(end, last0 < 0 ? 0 : last0 / BN + 1) - it.t0);
          it.n1 = it.two ? max(0, min(end, last1 < 0 ? 0 : last1 / BN + 1) - it.t0) : 0;
          it.bad_values = 0;
          if (it.parts > 1 && it.n0 + it.n1 == 0) continue;   // no row sees this partition
        }
        if (slot >= 2 && !__all_sync(kFullMask, mbar_wait(bar(LY::I_EMPTY + (slot & 1)), ((slot >> 1) - 1) & 1))) {
          fail = true;
          break;
        }
        if (lane == 0) {
          *item_at(slot) = it;
          mbar_arrive(bar(LY::I_FULL + (slot & 1)));
        }
        ++slot;
        if (!it.work) break;
      }
    } else if (warp == 8) {
      // -------------------------------------------------------- producer
      const uint64_t stream_policy = l2_policy_evict_first();
      uint64_t keep_policy;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep_policy));
      const bool paged = a.key_starts == nullptr;
      const int past = paged ? static_cast<int>((static_cast<long long>(a.NB) * a.Hkv) << a.bs_log2) : 0;
      int ring = 0, qs = 0;                         // tiles and queries loaded so far
      for (int slot = 0;; ++slot) {
        if (!__all_sync(kFullMask, mbar_wait(bar(LY::I_FULL + (slot & 1)), (slot >> 1) & 1))) {
          fail = true;
          break;
        }
        const PrefillItem it = *item_at(slot);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(LY::I_EMPTY + (slot & 1)));
        if (!it.work) break;
        const int n = max(it.n0, it.n1);
        if (n == 0) continue;
        const uint64_t policy = it.once ? stream_policy : keep_policy;
        // paged: lane l brings 64 columns (l % PANELS) of block l / PANELS of the tile
        const int bs = 1 << a.bs_log2, per_tile = BN >> a.bs_log2, blocks = (it.L + bs - 1) >> a.bs_log2;
        const int panel = lane % PANELS, blk = lane / PANELS;
        const int32_t* table = paged ? a.block_tables + static_cast<size_t>(it.seq) * a.MB : nullptr;
        auto row_of = [&](int t) {                  // cache row of the lane's block in key tile t
          const int j = t * per_tile + blk;
          if (blk >= per_tile || j >= blocks) return past;     // past the end: reads as zero
          const int id = __ldg(table + j);
          if (id < 0 || id >= a.NB) {
            record_error(a.err, kDevBadBlock);
            return past;
          }
          return (id * a.Hkv + it.kvh) << a.bs_log2;
        };
        int y = paged ? row_of(it.t0) : 0;
        for (int i = 0; i < n && !fail; ++i) {
          const int y_next = paged && i + 1 < n ? row_of(it.t0 + i + 1) : 0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int sl = ring % ST;
            if (ring >= ST && !__all_sync(kFullMask, mbar_wait(bar(LY::KV_EMPTY + sl), ((ring / ST) - 1) & 1))) {
              fail = true;
              break;
            }
            const CUtensorMap* map = kv ? &tmV : &tmK;
            const uint32_t full = bar(LY::KV_FULL + sl), dst = sb + LY::OFF_KV + sl * LY::KV_TILE;
            if (lane == 0) mbar_arrive_expect_tx(full, LY::KV_TILE);
            __syncwarp();
            if (paged) {
              if (blk < per_tile)
                tma_load_2d(dst + panel * (BN * 128) + (blk << a.bs_log2) * 128, map, panel * 64, y, full, policy);
            } else if (lane < PANELS) {
              tma_load_3d(dst + lane * (BN * 128), map, lane * 64, it.kvh, it.key_base + (it.t0 + i) * BN, full, policy);
            }
            ++ring;
            if (i == 0 && kv == 0) {
              const int tiles = it.two ? 2 : 1;
              if (qs > 0 && !__all_sync(kFullMask, mbar_wait(bar(LY::Q_EMPTY), (qs - 1) & 1))) {
                fail = true;
                break;
              }
              if (lane == 0) mbar_arrive_expect_tx(bar(LY::Q_FULL), tiles * PANELS * TPT * a.G * 128);
              __syncwarp();
              if (lane < tiles * PANELS) {
                const int x = lane / PANELS, c = lane % PANELS;
                tma_load_3d(sb + x * LY::Q_TILE + c * 16384, &tmQ, c * 64, it.kvh * a.G, it.q_row + x * TPT,
                            bar(LY::Q_FULL), stream_policy);
              }
              ++qs;
            }
          }
          y = y_next;
        }
        if (fail) break;
      }
      // Nothing may land or arrive in this CTA's shared memory after it has
      // left: every slot's last load was read and its release has come.
      for (int r = max(0, ring - ST); r < ring; ++r) {
        const bool landed = mbar_wait(bar(LY::KV_FULL + r % ST), (r / ST) & 1, 100000000ull);
        if (!fail && landed) mbar_wait(bar(LY::KV_EMPTY + r % ST), (r / ST) & 1, 100000000ull);
      }
      if (qs > 0) {
        mbar_wait(bar(LY::Q_FULL), (qs - 1) & 1, 100000000ull);
        if (!fail) mbar_wait(bar(LY::Q_EMPTY), (qs - 1) & 1, 100000000ull);
      }
    } else if (warp == 9) {
      // -------------------------------------------------------- matrix products
      if (lane == 0) {
        const uint32_t idesc_qk = umma_idesc_f16(BF, 0, 0, BN, 128);
        const uint32_t idesc_pv = umma_idesc_f16(BF, 0, 1, D, 128);
        auto slot_of = [&](int r) { return sb + LY::OFF_KV + (r % ST) * LY::KV_TILE; };
        auto landed = [&](int r) {
          if (!mbar_wait(bar(LY::KV_FULL + r % ST), (r / ST) & 1)) fail = true;
          return !fail;
        };
        auto qk = [&](int s, int x, int r) {        // S buffer s = Q tile x . K of ring tile r
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t ad = umma_desc_sw128(sb + x * LY::Q_TILE + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024);
            const uint64_t bd = umma_desc_sw128(slot_of(r) + (kk >> 2) * (BN * 128) + (kk & 3) * 32, 16, 1024);
            umma_f16(tmem + LY::S_COL(s), ad, bd, idesc_qk, kk > 0 ? 1u : 0u);
          }
          umma_commit(bar(LY::S_FULL + s));
        };
        auto pv = [&](int s, int x, int r, bool first) {   // O tile x += P of buffer s . V of ring tile r
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            const uint64_t bd = umma_desc_sw128(slot_of(r) + kk * 2048, BN * 128, 1024);
            umma_f16_ts(tmem + LY::O_COL(x), tmem + LY::S_COL(s) + kk * 8, bd, idesc_pv, !first || kk > 0 ? 1u : 0u);
          }
          umma_commit(bar(LY::O_DONE + x));
        };
        int ring = 0, qs = 0, su[3] = {0, 0, 0}, ou[2] = {0, 0};   // S buffers' and O tiles' uses so far
        auto have_p = [&](int s, int x, bool first) {
          // P of S buffer s has been written; before the first product of an item O must be free
          if (!mbar_wait(bar(LY::P_FULL + s), su[s] & 1)) fail = true;
          ++su[s];
          if (!fail && first) {
            if (ou[x] > 0 && !mbar_wait(bar(LY::O_FREE + x), (ou[x] - 1) & 1)) fail = true;
            ++ou[x];
          }
          return !fail;
        };
        for (int slot = 0; !fail; ++slot) {
          if (!mbar_wait(bar(LY::I_FULL + (slot & 1)), (slot >> 1) & 1)) {
            fail = true;
            break;
          }
          const PrefillItem it = *item_at(slot);
          mbar_arrive(bar(LY::I_EMPTY + (slot & 1)));
          if (!it.work) break;
          const int n0 = it.n0, n1 = it.n1, n = max(n0, n1);
          if (n == 0) continue;
          if (!mbar_wait(bar(LY::Q_FULL), qs & 1)) {
            fail = true;
            break;
          }
          ++qs;
          // ring tile of K(i) is ring + 2 i, of V(i) the one after
          if (!landed(ring)) break;
          if (it.two) {
            if (n0 > 0) qk(0, 0, ring);
            if (n1 > 0) qk(1, 1, ring);
          } else {
            qk(0, 0, ring);
          }
          umma_commit(bar(LY::KV_EMPTY + ring % ST));
          if (n == 1) umma_commit(bar(LY::Q_EMPTY));
          for (int i = 0; i < n; ++i) {
            const int rv = ring + 2 * i + 1, rk = rv + 1;
            const bool more = i + 1 < n;
            if (it.two) {
              if (!landed(rv)) break;
              if (i < n0) {
                if (!have_p(0, 0, i == 0)) break;
                pv(0, 0, rv, i == 0);
              }
              if (more && !landed(rk)) break;
              if (i + 1 < n0) qk(0, 0, rk);
              if (i < n1) {
                if (!have_p(1, 1, i == 0)) break;
                pv(1, 1, rv, i == 0);
              }
              umma_commit(bar(LY::KV_EMPTY + rv % ST));
              if (i + 1 < n1) qk(1, 1, rk);
              if (more) umma_commit(bar(LY::KV_EMPTY + rk % ST));
            } else {
              if (more) {
                if (!landed(rk)) break;
                qk(i & 1 ? 0 : 2, 0, rk);
                umma_commit(bar(LY::KV_EMPTY + rk % ST));
              }
              const int sp = i & 1 ? 2 : 0;
              if (!landed(rv) || !have_p(sp, 0, i == 0)) break;
              pv(sp, 0, rv, i == 0);
              umma_commit(bar(LY::KV_EMPTY + rv % ST));
            }
            if (i + 2 == n) umma_commit(bar(LY::Q_EMPTY));
          }
          ring += 2 * n;
        }
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    constexpr float kShift = BF ? 0.f : 7.f;        // P is 2^kShift times the weight
    const int w = warp >> 2, r = tid & 127;         // row tile, row
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int tl = r / a.G;                         // token of the row within its tile
    const bool has_token = tl < TPT;
    const float c = a.scale_log2;
    int ring = 0, su = 0, su2 = 0, od = 0;          // ring tiles, S buffers' uses, own O tile's products so far
    for (int slot = 0; !fail; ++slot) {
      if (!__all_sync(kFullMask, mbar_wait(bar(LY::I_FULL + (slot & 1)), (slot >> 1) & 1))) {
        fail = true;
        break;
      }
      PrefillItem* item = item_at(slot);
      if (!item->work) break;
      const int two = item->two, L = item->L, off = item->off, t0 = item->t0;
      const int n0 = item->n0, n1 = item->n1, n = w == 0 ? n0 : n1;
      const int j = w * TPT + tl;                   // token of the row within the item
      const bool valid = has_token && j < item->ntok && (w == 0 || two);
      const int lim = a.causal ? off + j : L - 1;   // last key that the row sees
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int i = 0; i < n; ++i) {
        const int s = two ? w : (i & 1 ? 2 : 0);
        if (!__all_sync(kFullMask, mbar_wait(bar(LY::S_FULL + s), (s == 2 ? su2 : su) & 1))) {
          fail = true;
          break;
        }
        s == 2 ? ++su2 : ++su;
        tc_fence_after();
        float x[BN];
#pragma unroll
        for (int q = 0; q < BN / 32; ++q) tmem_ld32(lanes + LY::S_COL(s) + q * 32, x + q * 32);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < BN / 32; ++q) tmem_ready32(x + q * 32);
        const int key0 = (t0 + i) * BN;
        if (a.negative) {
#pragma unroll
          for (int e = 0; e < BN; ++e) x[e] = -x[e];
        }
        if (__any_sync(kFullMask, valid && key0 + BN - 1 > lim)) {
#pragma unroll
          for (int e = 0; e < BN; ++e) x[e] = key0 + e <= lim ? x[e] : -INFINITY;
        }
        // values that some row must not see (the first softmax warps to work on the tile)
        if ((w == 0 || i >= n0) && key0 + BN > (a.causal ? min(L, off + 1) : L)) {
          const int rv = ring + 2 * i + 1;
          if (!__all_sync(kFullMask, mbar_wait(bar(LY::KV_FULL + rv % ST), (rv / ST) & 1))) {
            fail = true;
            break;
          }
          const uint32_t tile = sb + LY::OFF_KV + (rv % ST) * LY::KV_TILE;
          const int first = max(0, (a.causal ? min(L, off + 1) : L) - key0), end = L - key0;
          for (int u = first * (D / 8) + r; u < BN * (D / 8); u += 128) {
            const int vr = u / (D / 8), ch = u % (D / 8);
            const uint32_t at = tile + (ch >> 3) * (BN * 128) + vr * 128 + (ch & 7) * 16;
            uint32_t d[4] = {0, 0, 0, 0};
            bool store = vr >= end;
            if (!store) {
              asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                           : "r"(at));
              constexpr uint32_t kExp = BF ? 0x7f807f80u : 0x7c007c00u, kOne = BF ? 0x00800080u : 0x04000400u;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t odd = ((d[e] & kExp) + kOne) & 0x80008000u;   // a half's exponent is all ones
                if (odd) {
                  d[e] &= ~((odd >> 15) * 0xffffu);
                  store = true;
                  item->bad_values = 1;
                }
              }
            }
            if (store)
              asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(d[0]), "r"(d[1]), "r"(d[2]),
                           "r"(d[3])
                           : "memory");
          }
          fence_proxy_async_smem();
        }
        float top[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) top[q] = x[q];
#pragma unroll
        for (int e = 4; e < BN; e += 8) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (e + 4 + q < BN)
              top[q] = fmaxf(top[q], fmaxf(x[e + q], x[e + 4 + q]));
            else
              top[q] = fmaxf(top[q], x[e + q]);
          }
        }
        const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if (i == 0) {
          m = mt;
        } else if (__any_sync(kFullMask, (mt - m) * c > 8.f)) {
          // raise the reference: O holds the products up to the last tile's
          const float up = fmaxf(m, mt), keep = m == -INFINITY ? 0.f : fast_exp2((m - up) * c);
          if (!__all_sync(kFullMask, mbar_wait(bar(LY::O_DONE + w), (od + i - 1) & 1))) {
            fail = true;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < D / 16; ++q) {
            float o[16];
            tmem_ld16(lanes + LY::O_COL(w) + q * 16, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= keep;
            tmem_st16(lanes + LY::O_COL(w) + q * 16, o);
          }
          l2.x *= keep;
          l2.y *= keep;
          m = up;
        }
        const float mc = (m == -INFINITY ? 0.f : m * c) - kShift;
        const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
        float2 sum[2] = {l2, make_float2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < BN / 32; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 p = fma2(make_float2(x[q * 32 + 2 * e], x[q * 32 + 2 * e + 1]), c2, mc2);
            p.x = fast_exp2(p.x);
            p.y = fast_exp2(p.y);
            sum[e & 1] = add2(sum[e & 1], p);
            pk[e] = pack2<BF>(p.x, p.y);
          }
          tmem_st16u(lanes + LY::S_COL(s) + q * 16, pk);
        }
        l2 = add2(sum[0], sum[1]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(LY::P_FULL + s));
      }
      if (fail) break;
      // -------------------------------------------------------- the item's rows out
      const float l = l2.x + l2.y;
      if (n > 0) {
        // (the last but one product may be under way as well where S runs ahead
        // of it; a barrier must not be asked for a phase that is not its next)
        if ((n > 1 && !__all_sync(kFullMask, mbar_wait(bar(LY::O_DONE + w), (od + n - 2) & 1))) ||
            !__all_sync(kFullMask, mbar_wait(bar(LY::O_DONE + w), (od + n - 1) & 1))) {
          fail = true;
          break;
        }
        tc_fence_after();
      }
      const int kvh = item->kvh, parts = item->parts;
      const size_t row = (static_cast<size_t>(item->q_row + j) * a.Hq + kvh * a.G + (r - tl * a.G));
      size_t prow = 0;
      if (parts > 1)
        prow = static_cast<size_t>(item->row) +
               (row - static_cast<size_t>(a.query_starts[item->seq]) * a.Hq) * parts + item->part;
      const float inv = parts > 1 ? 1.f : (l > 0.f ? 1.f / l : 0.f);
      const bool bad_values = n > 0 && item->bad_values;
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        if (n > 0) {
          tmem_ld32(lanes + LY::O_COL(w) + q * 32, o);
          tmem_wait_ld();
          tmem_ready32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
          if (bad_values && valid) {
            // cleared values that this row sees
            const int to = min(min(lim, L - 1), (t0 + n) * BN - 1);
            for (int key = max(max(off + 1, 0), t0 * BN); key <= to; ++key) {
              const uint16_t* v;
              if (a.key_starts != nullptr) {
                v = a.v + (item->key_base + key) * a.v_stride + static_cast<size_t>(kvh) * D;
              } else {
                const int id = a.block_tables[static_cast<size_t>(item->seq) * a.MB + (key >> a.bs_log2)];
                if (id < 0 || id >= a.NB) continue;
                v = a.v + (((static_cast<size_t>(id) * a.Hkv + kvh) << a.bs_log2) + (key & ((1 << a.bs_log2) - 1))) * D;
              }
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 y = unpack2<BF>(*reinterpret_cast<const uint32_t*>(v + q * 32 + e));
                if (!(fabsf(y.x) <= 3.402823466e38f)) o[e] += y.x;
                if (!(fabsf(y.y) <= 3.402823466e38f)) o[e + 1] += y.y;
              }
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (valid) {
          if (parts > 1) {
            float* dst = a.part_o + prow * D + q * 32;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(dst + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else {
            uint16_t* dst = a.out + row * D + q * 32;
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(dst + e) =
                  make_uint4(pack2<BF>(o[e], o[e + 1]), pack2<BF>(o[e + 2], o[e + 3]),
                             pack2<BF>(o[e + 4], o[e + 5]), pack2<BF>(o[e + 6], o[e + 7]));
          }
        }
      }
      if (parts > 1 && valid)
        a.part_ml[prow] = make_float2(l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * c) - kShift, l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (n > 0) mbar_arrive(bar(LY::O_FREE + w));
        mbar_arrive(bar(LY::I_EMPTY + (slot & 1)));
      }
      od += n;
      ring += 2 * max(n0, n1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
  if (fail && lane == 0) record_error(a.err, kDevTimeout);
}

}  // namespace pkv
