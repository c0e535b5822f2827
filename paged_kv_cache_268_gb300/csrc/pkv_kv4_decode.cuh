// Paged single-token decode attention over the 4-bit cache, on mma.sync.
//
// With k = s (n + z) in every group g of 32 channels (n the 4-bit codes),
//   q . k_t = sum_g s_tg (sum_{d in g} q_d n_td  +  z_tg sum_{d in g} q_d)
//   out_d   = sum_t (p_t s_tg) (n_td + z_tg)          (p the softmax weights)
// so the matrix instructions multiply the CODES, and the scales and zeros are
// applied per (token, group): to the FP32 accumulators of q . n for the keys,
// to the weights for the values.  Nothing is dequantised element by element.
//
// Codes as operands: a nibble masked into the low bits of a binary16 is the
// subnormal n * 2^-24 (0x000f) or n * 2^-20 (0x00f0), exactly, and the tensor
// cores multiply subnormals exactly and at full rate.  One 32-bit word of codes
// thus becomes four operand registers with a shift and four ANDs, and the
// powers of two come out of the results: for the keys through q (each head's
// row scaled by the power of two that brings its largest element into [2^14,
// 2^15), the odd nibbles' channels by another 2^-4), for the values at the very
// end (even and odd nibbles are different output rows).  (A code in the low
// half of a byte is also n * 2^-9 in e4m3, one AND for four; but this machine
// has no such mma.sync, the compiler converts every operand: 1.2x slower.)
//
// Columns: an operand tile has 8 columns.  Where the CTA's query heads HC are
// fewer, GS = 8 / HC channel groups share it: column (j, h) holds head h, for
// keys only in the channels of the j-th group (so one accumulator collects
// the sums of GS groups side by side), for values with that group's scales.
// A lane then applies one group's parameters instead of GS of them.
//
// One CTA handles one (sequence, kv head, chunk of query heads, partition).
// Each warp owns a ring of stages of 32 tokens (two 16-token blocks or one of
// 32), each block's tile a contiguous run of bytes fetched with one untiled
// bulk copy for K and one for V.  Per 16 tokens:
//   S[16 tok x 8 columns]: ldmatrix gives a lane one word (8 channels) of each
//     of two tokens; two k16 steps per group.
//   P' = P s in binary16, per column (a weight's rounding, 2^-11 of it at most
//     where it is a normal number, and its product's are the only ones below
//     FP32; P is binary16 for bfloat16 inputs too, which have fewer bits).
//   O^T[32 ch x 8 columns] += codes^T P': ldmatrix.trans puts two neighbouring
//     tokens' words side by side; two m16 tiles per group.
//   z^T P' with the pairs (s, z) as they lie in the cache for the A operand:
//     rows 8 on give the zero-point sums (one m16 tile per GS groups).
// P is scaled by 2^12, as the running sum is, so that weights down to 2^-26 of
// the largest are normal numbers.  The reference follows the running maximum
// only when that is more than a factor of 2 ahead, which spares the rescalings
// for small gains: P stays at most 2^13.  It is subtracted where a logit's sum
// begins, in the logit's own units: the exponents that are left are small, so
// that logits past 2^24, whose products with the scale are rounded to more
// than one, still give weights of at most 2^13.
// P' is below 2^14 and, for the largest weight, a normal number where the
// scales are usual ones: below 2, and of 2^-13 or more in some token of each
// channel group's 32.  A group whose scales are not has them multiplied by a
// power of two in shared memory as its stages come, and its sums by what brings
// them in line (`follow`).  So a token's share in a group of channels gets lost
// only below max(2^-24 S, 2^-51) (n + z) of the largest weight, S the largest
// scale of the group in the 32 tokens: small values keep their weights, beside
// large ones of other channels or tokens too.  The look for unusual scales costs ordinary values 0.2-0.7% (64 x
// 512-4096 tokens, 32 kv heads, 117.7 us, 117.2 without; 256 x 1-2048, 69.5 and
// 69.1; up to 2% at head_dim 256), unusual ones more (256 x 1-2048 with values
// of 1e-5, 78.2 us).
// (Following at once makes the largest weight a power of two, which rounds to
// itself: binary16 results are then off by 2.7e-4 of their size in all, 2.8e-4
// as it is, 3.3e-4 at a factor of 32; their own rounding is 2.1e-4.  Measured
// on a form of the kernel before the finer last partitions: 64 sequences of
// 512-4096 tokens 123 us in all three; 256 of 1-2048, four query heads a key
// head, 72.9, 71.7 and 71 us.)
// What bounds it (one GB300, graph-timed; floor: K and V bytes at the measured
// copy rate): 128 sequences of 8192 tokens, 32/8 heads, 207 us of a 201 us
// floor in partitions of one size, so in the steady state memory does.  A
// tile's instructions alone (no loads) take nearly as long as its bytes (64 x
// 512-4096 tokens, 32/32 heads: 96 us and 108; both together 118, floor 111),
// so what start-up and the tail of unequal lengths leave idle is not caught up:
// 256 x 1-2048 69.5 us of 54, 128 log-normal 56 of 40, 4 x 32768 36.5 of 25.
// Half of the instructions are the shift and ANDs of the codes, at two cycles
// each per SM quarter.  Groups of 8 query heads are bound by them (64 x 8192
// tokens: 129 us of 100), wider ones take a multiple (16 heads 211, 32 heads
// 413, whose tiles are fetched twice too).
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "pkv_geometry.h"
#include "pkv_internal.h"
#include "pkv_kv4.cuh"
#include "pkv_ptx.cuh"

namespace pkv {

struct Kv4Args {
  DecodeArgs d;
  const uint8_t* k;     // [NB, Hkv, tile]
  const uint8_t* v;
  int chunks;           // query-head chunks per kv head
  // The sequences from `late` on, dispatched last, are cut into partitions of
  // P2 tokens, S2 of them (d.P and d.S for those before): see the host's rule.
  int late, P2, S2;
  int early_ctas;       // CTAs of the sequences before `late`
  size_t late_part;     // partials of those sequences
};

constexpr int kKv4Warps = 4;
constexpr int kKv4Tokens = 32;   // per stage

// Stages per warp: 40 KB of ring per CTA, 80 KB at head_dim 256.
constexpr int kv4_stages(int D) { return D == 64 ? 4 : 2; }
// Resident CTAs per SM that the registers are budgeted for.
constexpr int kv4_ctas(int D, int HC, int NT) {
  return D * NT == 64 || (D * NT == 128 && HC < 8) ? 4 : (D * NT == 128 ? 3 : 2);
}
// Query heads that share the 8 columns of a tile (HC), and tiles per CTA (NT),
// for a group of G query heads: as few columns as the group needs; from 9 heads
// on two tiles (head_dim 256: one, whose accumulators fill the registers).
constexpr int kv4_columns(int D, int G) { return G <= 2 && D > 64 ? 2 : (G <= 4 ? 4 : 8); }
constexpr int kv4_tiles(int D, int G) { return D <= 128 && G > 8 ? 2 : 1; }
constexpr int kv4_stage_bytes(int D) { return 2 * kv4_tile_bytes(D, kKv4Tokens); }
constexpr int kv4_ring_bytes(int D) { return kKv4Warps * kv4_stages(D) * kv4_stage_bytes(D); }
// The warps' merge reuses the ring: per warp and head the accumulator row
// (padded by 8 floats against bank conflicts), the maximum and the sum.
constexpr int kv4_row(int D) { return D + 8; }
constexpr int kv4_merge_bytes(int D, int NT) { return kKv4Warps * 8 * NT * (kv4_row(D) + 2) * 4; }
// Query fragments, per-group sums and maxima, scales.
constexpr int kv4_query_bytes(int D, int NT) { return (D / 32) * NT * 512 + (2 * (D / 32) + 1) * 8 * NT * 4; }
constexpr int kv4_tail(int D, int NT) {
  return ((kv4_ring_bytes(D) > kv4_merge_bytes(D, NT) ? kv4_ring_bytes(D) : kv4_merge_bytes(D, NT)) + 127) & ~127;
}
constexpr int kv4_smem(int D, int NT) {
  return kv4_tail(D, NT) + kv4_query_bytes(D, NT) + kKv4Warps * kv4_stages(D) * 8 + kMaxBlocksPerCta * 4 + 128;
}

// for (i = 0; i < N; ++i) f(i) with i a constant, so that offsets can be
// immediates of the shared-memory instructions.
template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

template <int OFF, int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(w[0]) : "r"(addr), "n"(OFF));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2+%3];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr), "n"(OFF));
  } else {
    static_for<N / 4>([&](auto j) {
      constexpr int i = 4 * j;
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4+%5];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(addr), "n"(OFF + 4 * i));
    });
  }
}

template <int OFF>
__device__ __forceinline__ void lds_pair(uint32_t addr, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2+%3];" : "=r"(a), "=r"(b) : "r"(addr), "n"(OFF));
}

template <int OFF, bool TRANS>
__device__ __forceinline__ void ldm_x4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFF));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr), "n"(OFF));
}

// d += A B, binary16 operands, FP32 accumulators (registers only: free to be
// scheduled between the loads).
__device__ __forceinline__ void mma_codes(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// One warp's running state over its tokens and its work on one stage.
template <bool BF, int D, int BS, int HC, int NT>
struct Kv4Compute {
  static constexpr int NG = D / 32;        // channel groups
  static constexpr int GS = 8 / HC;        // groups side by side in a tile's columns
  static constexpr int NS = NG / GS;       // sets of such groups: group j * NS + i is set i, place j
  static constexpr int NH = HC * NT;       // heads this warp produces
  static constexpr int TILE = kv4_tile_bytes(D, BS);
  static constexpr int PER = kKv4Tokens / BS;   // blocks per stage
  // Query fragments in registers, or read from shared memory for every stage:
  // at head_dim 128 the registers serve the schedule better (64 x 512-4096
  // tokens, before the finer last partitions: 121 us, 123 with fragments in
  // registers).
  static constexpr bool QREG = D * NT < 128;
  static constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u;
  static constexpr float kShift = 12.f, kSlack = 1.f;
  static_assert(NG % GS == 0 && (NT == 1 || HC == 8), "columns");

  // Columns 2c and 2c + 1 (c = lane % 4) are two heads of one group place.
  uint32_t qf[QREG ? NG : 1][NT][4];       // B fragments: k16 step 0 (b0, b1), step 1 (b0, b1)
  uint32_t qaddr;                          // or where this lane's lie
  float qs[NS][NT][2];                     // 2^-24 sum of the group's q
  float sc[NT][2];                         // to log2 units, not negative
  float o[2 * NG][NT][4];                  // codes^T P'
  float oz[NS][NT][4];                     // (s, z)^T P': elements 2 and 3 are z's
  float m[NT][2], l[NT][2];                // reference, in the logits' units before sc; sum
                                           // (m only in the lanes of group place 0, else 0)
  int down;                                // value scales of group lane % NG count 2^-down times,
                                           // down in bits 0 .. 4; bit 14 where it is not 0;
                                           // negative before the first stage

  static __device__ __forceinline__ int place(int column) { return column / HC; }   // j of a column

  // The queries of the CTA's heads as B fragments, prepared once: warp w does
  // the channel groups w, w + 4, ... and every warp reads all of them back from
  // `qsm`.  A negative softmax scale goes into the sign of q.
  __device__ __forceinline__ void load_q(const uint16_t* qg, int heads, float scale_log2, uint8_t* qsm,
                                         int warp, int lane) {
    constexpr int NW = kKv4Warps, PG = (NG + NW - 1) / NW;
    uint4* frag = reinterpret_cast<uint4*>(qsm);                       // [NG][NT][32]
    float* sums = reinterpret_cast<float*>(qsm + NG * NT * 512);       // [NG][NH]
    float* tops = sums + NG * NH;                                      // [NG][NH]
    float* scales = tops + NG * NH;                                    // [NH]
    const int c = lane & 3, n = lane >> 2;
    uint4 u[PG][NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + n % HC;
#pragma unroll
      for (int i = 0; i < PG; ++i) {
        const int g = warp + i * NW;
        if (g >= NG) break;
        const bool mine = place(n) == g / NS;
        u[i][nt] = make_uint4(0, 0, 0, 0);
        if (mine && h < heads) u[i][nt] = __ldg(reinterpret_cast<const uint4*>(qg + h * D + g * 32 + c * 8));
        const uint32_t x[4] = {u[i][nt].x, u[i][nt].y, u[i][nt].z, u[i][nt].w};
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = unpack2<BF>(x[k]);
          top = max_nan(top, max_nan(fabsf(f.x), fabsf(f.y)));
        }
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (mine && c == 0) tops[g * NH + h] = top;
      }
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + n % HC;
      float top = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) top = max_nan(top, tops[g * NH + h]);
      int e = 14 + 127 - static_cast<int>(__float_as_uint(top) >> 23);
      e = top > 0.f ? min(e, 120) : 0;
      float f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      if (warp == 0 && n < HC && c == 0) {
        // Queries near bfloat16's largest would take this past FP32's.  The sums
        // that it multiplies are whole multiples of 2^-96, so from 2^127 on every
        // difference between two decides alone, as it does for the true factor.
        const int up = min(24 - e, 127);
        const float by = fabsf(scale_log2) * power_of_two(up) * power_of_two(24 - e - up);
        // an infinite or NaN query gives NaN
        scales[h] = top < INFINITY ? (by > 0x1p127f ? 0x1p127f : by) : __uint_as_float(0x7fc00000u);
      }
      if (scale_log2 < 0.f) f = -f;
#pragma unroll
      for (int i = 0; i < PG; ++i) {
        const int g = warp + i * NW;
        if (g >= NG) break;
        const float2 x01 = unpack2<BF>(u[i][nt].x), x23 = unpack2<BF>(u[i][nt].y),
                     x45 = unpack2<BF>(u[i][nt].z), x67 = unpack2<BF>(u[i][nt].w);
        const float fo = f * 0.0625f;
        // k index 2c + {0, 1} of step 0: channels 0 and 4 of the lane's eight,
        // then 2 and 6; of step 1: 1 and 5, then 3 and 7 (16 times their code)
        const uint32_t r0 = pack2<false>(x01.x * f, x45.x * f), r1 = pack2<false>(x23.x * f, x67.x * f);
        const uint32_t r2 = pack2<false>(x01.y * fo, x45.y * fo), r3 = pack2<false>(x23.y * fo, x67.y * fo);
        frag[(g * NT + nt) * 32 + lane] = make_uint4(r0, r1, r2, r3);
        const float2 s0 = unpack2<false>(r0), s1 = unpack2<false>(r1), s2 = unpack2<false>(r2),
                     s3 = unpack2<false>(r3);
        float sum = ((s0.x + s0.y) + (s1.x + s1.y)) * 0x1p-24f + ((s2.x + s2.y) + (s3.x + s3.y)) * 0x1p-20f;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (place(n) == g / NS && c == 0) sums[g * NH + h] = sum;
      }
    }
    __syncthreads();
    const int h0 = 2 * c % HC, j = place(2 * c);
    qaddr = smem_u32(frag + lane);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 x = *reinterpret_cast<const float2*>(scales + nt * 8 + h0);
      sc[nt][0] = x.x;
      sc[nt][1] = x.y;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float2 y = *reinterpret_cast<const float2*>(sums + (j * NS + i) * NH + nt * 8 + h0);
        qs[i][nt][0] = y.x;
        qs[i][nt][1] = y.y;
      }
      if constexpr (QREG) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint4 v = frag[(g * NT + nt) * 32 + lane];
          qf[g][nt][0] = v.x; qf[g][nt][1] = v.y; qf[g][nt][2] = v.z; qf[g][nt][3] = v.w;
        }
      }
    }
  }

  __device__ __forceinline__ void reset() {
    down = static_cast<int>(0x80000000u);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) o[i][nt][e] = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) oz[i][nt][e] = 0.f;
      }
    }
  }

  // Offset of the 16-token half `mt` in a stage's K or V: its block, and its row there.
  static __host__ __device__ constexpr int block_of(int mt) { return PER == 2 ? mt * TILE : 0; }
  static __host__ __device__ constexpr int row_of(int mt) { return PER == 2 ? 0 : mt * 16; }
  static constexpr int VT = PER * TILE;           // V behind K
  static constexpr int PAR = BS * (D / 2);        // parameters behind a tile's codes

  // Clear the parameters of the tokens from `valid` on, so that whatever bytes
  // lie behind a sequence's end (NaN scales among them) count for nothing.
  static __device__ __forceinline__ void clear_tail(uint32_t kt, int valid, int lane) {
    for (int i = lane; i < kKv4Tokens * NG; i += 32) {
      const int t = i / NG, g = i % NG;
      if (t < valid) continue;
      const int mt = t / 16, r = row_of(mt) + t % 16;
      const uint32_t kp = kt + block_of(mt) + kv4_k_par_off<D>(BS, r, g);
      const uint32_t vp = kt + VT + block_of(mt) + kv4_v_par_off<D>(BS, r, g);
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(kp), "r"(0) : "memory");
      asm volatile("st.shared.b16 [%0], %1;" ::"r"(vp), "h"(static_cast<short>(0)) : "memory");
      asm volatile("st.shared.b16 [%0], %1;" ::"r"(vp + 4), "h"(static_cast<short>(0)) : "memory");
    }
    __syncwarp();
  }

  // Address of this lane's share i of the stage's value scales: pair i * 32 +
  // lane of (two tokens, group), which is one of group lane % NG.
  static __device__ __forceinline__ uint32_t scale_pair(uint32_t kt, int i, int lane) {
    const int k = i * 32 + lane, half = k / (8 * NG), rest = k % (8 * NG);
    return kt + VT + PAR + (half ? block_of(1) + row_of(1) / 2 * NG * 8 : 0) + rest * 8;
  }

  static __device__ __forceinline__ float power_of_two(int e) {
    return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  }

  static __device__ __forceinline__ int down_of(int down) { return static_cast<int>(static_cast<uint32_t>(down) << 27) >> 27; }

  // Some group's value scales are not usual ones, of 2^-13 to 2, or were not
  // before.  Where a group's largest is not, its scales in the stage are
  // multiplied by the power of two that brings it to [1, 2) (2^15 at most),
  // and its sums, so far of other multiples, by the one between the two; both
  // are exact, but where large scales make small ones subnormal.  The power
  // stays while the largest is between 1/2 and 2.
  __device__ __forceinline__ void follow(uint32_t kt, int lane) {
    uint32_t x[NG / 2];
    int most = 0;                          // the group's largest, its binary16 bits
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) {
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[i]) : "r"(scale_pair(kt, i, lane)));
      const int a = x[i] & 0xffff, b = x[i] >> 16;
      most = max(most, max(a > 0x7bff ? 0 : a, b > 0x7bff ? 0 : b));   // a NaN counts for none
    }
#pragma unroll
    for (int m = NG; m < 32; m <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, m));
    const int old = down_of(down), e = most >> 10;   // 2^(e - 15) <= most < 2^(e - 14)
    int now = max(min(e - 15, 14), -15);
    if (e >= 2 && e < 16) now = 0;
    if ((old != 0 && (e == old + 15 || e == old + 14)) || most == 0) now = old;
    if (now != 0) {
      const uint32_t f = static_cast<uint32_t>(15 - now) * 0x04000400u;   // 2^-now, twice
#pragma unroll
      for (int i = 0; i < NG / 2; ++i)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(scale_pair(kt, i, lane)), "r"(hmul2_bits(x[i], f)) : "memory");
    }
    down = now == 0 ? 0 : 0x4000 | (now & 31);
    __syncwarp();
    if (!__any_sync(0xffffffffu, now != old)) return;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float f = power_of_two(__shfl_sync(0xffffffffu, old - now, g));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          o[2 * g][nt][e4] *= f;
          o[2 * g + 1][nt][e4] *= f;
        }
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {         // columns 2c and 2c + 1
      const float f = power_of_two(__shfl_sync(0xffffffffu, old - now, place(2 * (lane & 3)) * NS + i));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) oz[i][nt][e4] *= f;
    }
  }

  // The first stage, or its maximum (`top`, above the reference) is past the
  // slack: it becomes the reference, and the sums and the stage's logits follow.
  __device__ __forceinline__ void catch_up(const float (&top)[NT][2], float (&s)[2][NT][4], bool first, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float by[2], more[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float gain = top[nt][j] * sc[nt][j];
        const bool go = first || gain > kSlack;
        by[j] = first ? 0.f : (go ? fast_exp2(-gain) : 1.f);
        more[j] = go ? top[nt][j] : 0.f;
        if (place(2 * (lane & 3)) == 0) m[nt][j] += more[j];
        l[nt][j] *= by[j];
      }
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        s[0][nt][e4] -= more[e4 & 1];
        s[1][nt][e4] -= more[e4 & 1];
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) o[i][nt][e4] *= by[e4 & 1];
#pragma unroll
        for (int i = 0; i < NS; ++i) oz[i][nt][e4] *= by[e4 & 1];
      }
    }
  }

  // 32 tokens at `kt` (K) and `kt + VT` (V); RAGGED: only the first `valid` of
  // them are real.  `lrow[i]`: the lane's ldmatrix row of the group pair i,
  // relative to codes.  Apart from one rare branch this is straight code, so
  // that loads, logic, matrix and exponential instructions can be interleaved.
  template <bool RAGGED>
  __device__ __forceinline__ void stage(uint32_t kt, int valid, const uint32_t (&lrow)[NG / 2], int lane) {
    if constexpr (RAGGED) clear_tail(kt, valid, lane);
    // Is a value scale of 2 or more among the stage's, or none of 2^-13 or more
    // among a lane's share of them, all of group lane % NG?
    uint32_t scales = 0;
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) {
      uint32_t x;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(scale_pair(kt, i, lane)));
      scales |= x;
    }
    uint32_t at[NG / 2];
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) at[i] = kt + lrow[i];
    // the lane's parameters: keys of tokens lane / 4 and 8 on for the group
    // place of its columns 2c, 2c + 1; values of tokens 2c, 2c + 1 and 8 on for
    // that of column lane / 4
    const uint32_t kpar = kt + ((lane >> 2) * NG + place(2 * (lane & 3)) * NS) * 4;
    const uint32_t vpar = kt + ((lane & 3) * NG + place(lane >> 2) * NS) * 8;

    // Logits.  Both halves go side by side, so that one's matrix instructions
    // fill the other's latency.
    float s[2][NT][4];
    uint32_t plo[2][NS], phi[2][NS], r[2][NG / 2][4];
    static_for<2>([&](auto mt) {
      constexpr int KP = block_of(mt) + PAR + row_of(mt) * NG * 4;
      lds_words<KP>(kpar, plo[mt]);
      lds_words<KP + 8 * NG * 4>(kpar, phi[mt]);
    });
    static_for<NG / 2>([&](auto gp) {
      static_for<2>([&](auto mt) {
        constexpr int KB = block_of(mt) + row_of(mt) * (D / 2);
        ldm_x4<KB, false>(at[gp], r[mt][gp]);
      });
    });
    static_for<NS>([&](auto i) {
      float acc[2][NT][4];
      static_for<GS>([&](auto j) {
        constexpr int g = j * NS + i;
        static_for<2>([&](auto mt) {
          const uint32_t a = r[mt][g / 2][2 * (g & 1)], b = r[mt][g / 2][2 * (g & 1) + 1];
          const uint32_t a8 = a >> 8, b8 = b >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (j == 0) {
              const float zl = __high2float(*reinterpret_cast<const __half2*>(&plo[mt][i]));
              const float zu = __high2float(*reinterpret_cast<const __half2*>(&phi[mt][i]));
              acc[mt][nt][0] = zl * qs[i][nt][0];
              acc[mt][nt][1] = zl * qs[i][nt][1];
              acc[mt][nt][2] = zu * qs[i][nt][0];
              acc[mt][nt][3] = zu * qs[i][nt][1];
            }
            uint32_t q[4];
            if constexpr (QREG) {
#pragma unroll
              for (int k = 0; k < 4; ++k) q[k] = qf[g][nt][k];
            } else {
              lds_words<g * NT * 512>(qaddr + nt * 512, q);
            }
            mma_codes(acc[mt][nt], a & M0, b & M0, a8 & M0, b8 & M0, q[0], q[1]);
            mma_codes(acc[mt][nt], a & M1, b & M1, a8 & M1, b8 & M1, q[2], q[3]);
          }
        });
      });
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float sl = __low2float(*reinterpret_cast<const __half2*>(&plo[mt][i]));
        const float su = __low2float(*reinterpret_cast<const __half2*>(&phi[mt][i]));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float by = e < 2 ? sl : su;
            s[mt][nt][e] = fmaf(by, acc[mt][nt][e], i == 0 ? -m[nt][e & 1] : s[mt][nt][e]);
          }
      }
    });
    // the group places of a head lie in lanes 4 / GS apart
#pragma unroll
    for (int m = 4 / GS; m < 4; m <<= 1)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] += __shfl_xor_sync(0xffffffffu, s[mt][nt][e], m);

    // The stage's maximum; s stays in its own units (sc is not negative), above
    // the reference: subtracted first, so that the exponents of large logits
    // have no rounding that the reference has not.
    float top[NT][2];
    // (bits of the exponent; a share past a sequence's end is all zeros)
    const bool unusual = (scales & 0x40004000u) != 0 || ((scales & 0x38003800u) == 0 && !(RAGGED && scales == 0));
    bool rare = unusual || down != 0;
    if constexpr (RAGGED) {   // out of the maximum past the end
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (mt * 16 + (e >> 1) * 8 + (lane >> 2) >= valid) s[mt][nt][e] = -INFINITY;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = fmaxf(fmaxf(s[0][nt][j], s[0][nt][2 + j]), fmaxf(s[1][nt][j], s[1][nt][2 + j]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        top[nt][j] = v;
        rare |= v * sc[nt][j] > kSlack;
      }
    }
    if (__any_sync(0xffffffffu, rare)) {
      const bool first = down < 0;
      if (first) down = 0;
      if (__any_sync(0xffffffffu, unusual || down != 0)) follow(kt, lane);
      catch_up(top, s, first, lane);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p = fast_exp2(fmaf(s[mt][nt][e], sc[nt][e & 1], kShift));
          // (a scale of zero times minus infinity is no number)
          if (RAGGED && mt * 16 + (e >> 1) * 8 + (lane >> 2) >= valid) p = 0.f;
          s[mt][nt][e] = p;
          l[nt][e & 1] += p;
        }

    static_for<2>([&](auto mt) {
      constexpr int VB = VT + block_of(mt) + row_of(mt) * (D / 2);
      constexpr int VP = VT + block_of(mt) + PAR + row_of(mt) / 2 * NG * 8;
      // (s, s), (z, z) of tokens 2c, 2c + 1, then of 8 + 2c, 9 + 2c, per set
      uint32_t w[NS][4];
      static_for<NS>([&](auto i) {
        lds_pair<VP + i * 8>(vpar, w[i][0], w[i][1]);
        lds_pair<VP + (4 * NG + i) * 8>(vpar, w[i][2], w[i][3]);
      });
      // P^T as B operands: tokens 2c, 2c + 1 (b0) and 8 on (b1) of column lane / 4
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        b0[nt] = movmatrix_trans(pack2<false>(s[mt][nt][0], s[mt][nt][1]));
        b1[nt] = movmatrix_trans(pack2<false>(s[mt][nt][2], s[mt][nt][3]));
      }
      uint32_t p0[NS][NT], p1[NS][NT];
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          p0[i][nt] = hmul2_bits(b0[nt], w[i][0]);
          p1[i][nt] = hmul2_bits(b1[nt], w[i][2]);
          mma_codes(oz[i][nt], w[i][0], w[i][1], w[i][2], w[i][3], p0[i][nt], p1[i][nt]);
        }
      static_for<NG / 2>([&](auto gp) {
        uint32_t r[4];
        ldm_x4<VB, true>(at[gp], r);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const int g = 2 * gp + gg;
          const uint32_t a = r[2 * gg], b = r[2 * gg + 1], a8 = a >> 8, b8 = b >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_codes(o[2 * g][nt], a & M0, a & M1, b & M0, b & M1, p0[g % NS][nt], p1[g % NS][nt]);
            mma_codes(o[2 * g + 1][nt], a8 & M0, a8 & M1, b8 & M0, b8 & M1, p0[g % NS][nt],
                      p1[g % NS][nt]);
          }
        }
      });
    });
  }

  // Leave each head's (m, l, o) for the CTA merge.  Rows lane / 4 of tile
  // (g, a) are channels 32 g + 4 (lane / 4) + 2 a, rows 8 on the next channel;
  // columns 2c, 2c + 1 hold group g only where it has their place.
  __device__ __forceinline__ void publish(float* cm, float* cl, float* co, int lane) {
    const int c = lane & 3, j = place(2 * c), h0 = 2 * c % HC;
    float back[NG];   // takes the groups' powers of two out
#pragma unroll
    for (int g = 0; g < NG; ++g) back[g] = power_of_two(down_of(__shfl_sync(0xffffffffu, down, g)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float lt = l[nt][k];
        lt += __shfl_xor_sync(0xffffffffu, lt, 4);
        lt += __shfl_xor_sync(0xffffffffu, lt, 8);
        lt += __shfl_xor_sync(0xffffffffu, lt, 16);
        const int h = nt * 8 + h0 + k;
        if (lane < HC / 2) {
          cm[h] = down < 0 ? -INFINITY : fmaf(m[nt][k], sc[nt][k], -kShift);   // in log2 units
          cl[h] = lt;
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          // the zero-point sum of this place's group lies in its own rows
          const float z = __shfl_sync(0xffffffffu, oz[i][nt][2 + k], j * HC * 4 + c);
#pragma unroll
          for (int x = 0; x < GS; ++x) {
            if (x != j) continue;
            const int g = x * NS + i;
            const float f = back[g];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int d = 32 * g + 4 * (lane >> 2) + 2 * t;
              *reinterpret_cast<float2*>(co + h * kv4_row(D) + d) =
                  make_float2(f * fmaf(o[2 * g + t][nt][k], 0x1p24f, z), f * fmaf(o[2 * g + t][nt][2 + k], 0x1p20f, z));
            }
          }
        }
      }
    }
  }
};

// First partial of output row `row` (sequence seq).
__device__ __forceinline__ size_t kv4_partial(const Kv4Args& p, int seq, size_t row) {
  return seq < p.late ? row * p.d.S
                      : p.late_part + (row - static_cast<size_t>(p.late) * p.d.Hq) * p.S2;
}

template <bool BF, int D, int BS, int HC, int NT>
__global__ void __launch_bounds__(kKv4Warps * 32, kv4_ctas(D, HC, NT)) kv4_decode_kernel(const __grid_constant__ Kv4Args p) {
  using Compute = Kv4Compute<BF, D, BS, HC, NT>;
  constexpr int NW = kKv4Warps, NS = kv4_stages(D), NH = Compute::NH;
  constexpr int TILE = Compute::TILE, PER = Compute::PER, STAGE = kv4_stage_bytes(D);
  static_assert(STAGE == 2 * PER * TILE, "stage");
  const DecodeArgs& a = p.d;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint8_t* qsm = smem + kv4_tail(D, NT);
  uint64_t* bars = reinterpret_cast<uint64_t*>(qsm + kv4_query_bytes(D, NT));
  int* ids = reinterpret_cast<int*>(bars + NW * NS);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int idx = blockIdx.x;
  const bool late = idx >= p.early_ctas;
  if (late) idx -= p.early_ctas;
  const int P = late ? p.P2 : a.P, S = late ? p.S2 : a.S;
  const int split = idx % S;
  idx /= S;
  const int chunk = idx % p.chunks;
  idx /= p.chunks;
  const int kvh = idx % a.Hkv;
  const int seq = idx / a.Hkv + (late ? p.late : 0);
  const int heads = min(NH, a.G - chunk * NH);          // of this CTA
  const int h0 = kvh * a.G + chunk * NH;                // the first of them
  // resident before the stream's previous kernel is done; nothing is read before it is
  pdl_wait();
  pdl_launch_dependents();

  // block ids of the partition, range-checked; the first partition's are
  // loaded together with the length (it is empty only for padding rows)
  const int t0 = split * P, j0 = t0 / BS;
  const int32_t* trow = a.block_tables + static_cast<size_t>(seq) * a.MB + j0;
  const int L = a.context_lens[seq];
  if (split == 0)
    for (int k = threadIdx.x; k < min(P / BS, a.MB - j0); k += NW * 32) ids[k] = __ldg(trow + k);
  if (L < 0 || L > a.max_ctx) {
    if (threadIdx.x == 0 && split == 0 && kvh == 0 && chunk == 0) record_error(a.err, kDevBadContext);
    return;
  }
  if (L == 0) {   // a padding row
    if (split == 0)
      for (int i = threadIdx.x; i < heads * D / 2; i += NW * 32)
        reinterpret_cast<uint32_t*>(a.out + (static_cast<size_t>(seq) * a.Hq + h0) * D)[i] = 0;
    return;
  }
  if (t0 >= L) return;
  const int t1 = L - t0 < P ? L : t0 + P;
  const int nblk = (t1 - t0 + BS - 1) / BS;
  bool bad = false;
  for (int k = threadIdx.x; k < nblk; k += NW * 32) {
    const int id = split == 0 ? ids[k] : __ldg(trow + k);   // ids[k]: this thread's own store
    bad |= (id < 0) | (id >= a.NB);
    ids[k] = id;
  }
  if (threadIdx.x < NW * NS) mbar_init(smem_u32(&bars[threadIdx.x]), 1);
  if (threadIdx.x == 0) fence_mbar_init();
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) record_error(a.err, kDevBadBlock);
    return;
  }

  const int nst = (nblk + PER - 1) / PER;               // stages of the partition
  const int my_n = nst > warp ? (nst - warp + NW - 1) / NW : 0;
  const uint32_t wbuf = smem_u32(smem + warp * NS * STAGE);
  const uint32_t wbar = smem_u32(&bars[warp * NS]);
  const uint64_t policy = l2_policy_evict_first();      // the cache is read once
  // Stage k of this warp: lane 0 announces the bytes, lane 2b + {0, 1} fetches
  // block b's K or V tile.
  const uint8_t* src = ((lane & 1) ? p.v : p.k) + static_cast<size_t>(kvh) * TILE;
  const size_t pitch = static_cast<size_t>(a.Hkv) * TILE;
  const uint32_t dst0 = wbuf + ((lane & 1) * PER + (lane >> 1)) * TILE;
  auto issue = [&](int k, int st) {
    const int b0 = (warp + NW * k) * PER;
    const uint32_t bar = wbar + 8 * st;
    if (lane == 0) mbar_arrive_expect_tx(bar, min(PER, nblk - b0) * 2 * TILE);
    __syncwarp();
    if (lane < 2 * PER && b0 + (lane >> 1) < nblk)
      bulk_load(dst0 + st * STAGE, src + ids[b0 + (lane >> 1)] * pitch, TILE, bar, policy);
  };
  const int pro = my_n < NS ? my_n : NS;
  for (int k = 0; k < pro; ++k) issue(k, k);

  Compute cs;
  cs.load_q(a.q + (static_cast<size_t>(seq) * a.Hq + h0) * D, heads, a.scale_log2, qsm, warp, lane);
  cs.reset();
  uint32_t lrow[Compute::NG / 2];
#pragma unroll
  for (int i = 0; i < Compute::NG / 2; ++i)
    lrow[i] = kv4_code_off<D>(lane & 15, 2 * i + (lane >> 4));
  bool ok = true;
  int k = 0, st = 0;
  uint32_t phase = 0;
  for (; k < my_n; ++k) {
    const bool done = mbar_wait(wbar + 8 * st, phase);
    if (!__all_sync(0xffffffffu, done)) { ok = false; break; }
    const int left = t1 - t0 - (warp + NW * k) * kKv4Tokens;
    if (left >= kKv4Tokens)
      cs.template stage<false>(wbuf + st * STAGE, kKv4Tokens, lrow, lane);
    else
      cs.template stage<true>(wbuf + st * STAGE, left, lrow, lane);
    __syncwarp();
    if (k + NS < my_n) {
      fence_proxy_async_smem();
      issue(k + NS, st);
    }
    if (++st == NS) {
      st = 0;
      phase ^= 1;
    }
  }
  if (!ok) {
    // every load in flight gets a bounded chance to land before the CTA ends
    const int hi = min(k + NS, my_n);
    for (int kk = k; kk < hi; ++kk) mbar_wait(wbar + 8 * (kk % NS), (kk / NS) & 1, 100000000ull);
    if (lane == 0) record_error(a.err, kDevTimeout);
  }
  if (__syncthreads_or(!ok)) return;   // the ring may still be filling: no result

  float* co = reinterpret_cast<float*>(smem);
  float* cm = co + NW * NH * kv4_row(D);
  float* cl = cm + NW * NH;
  cs.publish(cm + warp * NH, cl + warp * NH, co + warp * NH * kv4_row(D), lane);
  __syncthreads();
  const bool single = L <= P;
  for (int i = threadIdx.x; i < heads * (D / 4); i += NW * 32) {
    const int h = i / (D / 4), d = i % (D / 4) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, cm[w * NH + h]);
    float x[4] = {0.f, 0.f, 0.f, 0.f}, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = fast_exp2(cm[w * NH + h] - M);
      const float4 v = *reinterpret_cast<const float4*>(co + (w * NH + h) * kv4_row(D) + d);
      x[0] = fmaf(f, v.x, x[0]);
      x[1] = fmaf(f, v.y, x[1]);
      x[2] = fmaf(f, v.z, x[2]);
      x[3] = fmaf(f, v.w, x[3]);
      lsum = fmaf(f, cl[w * NH + h], lsum);
    }
    const size_t row = static_cast<size_t>(seq) * a.Hq + h0 + h;
    if (single) {
      const float r = 1.f / lsum;
      *reinterpret_cast<uint2*>(a.out + row * D + d) =
          make_uint2(pack2<BF>(x[0] * r, x[1] * r), pack2<BF>(x[2] * r, x[3] * r));
    } else {
      const size_t pr = kv4_partial(p, seq, row) + split;
      *reinterpret_cast<float4*>(a.part_o + pr * D + d) = make_float4(x[0], x[1], x[2], x[3]);
      if (d == 0) a.part_ml[pr] = make_float2(M, lsum);
    }
  }
}

// Cross-split reduce: one warp per output row of more than one partition; rows
// of sequences that all have one are not in the grid.  M = max m, w = 2^(m - M),
// out = sum w o / sum w l in the order of the partitions.  A lane owns D / 32
// elements and has the loads of eight partials in flight, the first of them
// together with those of m.
template <bool BF, int D>
__global__ void __launch_bounds__(128) kv4_reduce_kernel(const __grid_constant__ Kv4Args p, int row0) {
  constexpr int OPL = D / 32, J = 8;
  pdl_launch_dependents();
  const DecodeArgs& a = p.d;
  const int lane = threadIdx.x & 31;
  const long long row = row0 + blockIdx.x * 4ll + (threadIdx.x >> 5);
  int n = 0, seq = 0;
  if (row < static_cast<long long>(a.B) * a.Hq) {
    seq = static_cast<int>(row / a.Hq);
    const int L = a.context_lens[seq];   // written before the decode grid began
    const int P = seq < p.late ? a.P : p.P2;
    if (L >= 1 && L <= a.max_ctx) n = (L - 1) / P + 1;
  }
  pdl_wait();
  if (n <= 1) return;
  const size_t first = kv4_partial(p, seq, row);
  const float2* ml = a.part_ml + first;
  const float* po = a.part_o + first * D + lane * OPL;
  float x[J][OPL], acc[OPL], lsum = 0.f;
  float2 y[J];
  auto load = [&](int j0) {
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (j0 + j < n) {
        y[j] = __ldcg(ml + j0 + j);
#pragma unroll
        for (int e = 0; e < OPL; e += 2) {
          const float2 t = __ldcg(reinterpret_cast<const float2*>(po + static_cast<size_t>(j0 + j) * D + e));
          x[j][e] = t.x;
          x[j][e + 1] = t.y;
        }
      }
  };
  load(0);
  float M = -INFINITY;
  for (int j = lane; j < n; j += 32) M = fmaxf(M, __ldcg(ml + j).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
  for (int e = 0; e < OPL; ++e) acc[e] = 0.f;
  for (int j0 = 0; j0 < n; j0 += J) {
    if (j0 > 0) load(j0);
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (j0 + j < n) {
        const float w = fast_exp2(y[j].x - M);
        lsum = fmaf(w, y[j].y, lsum);
#pragma unroll
        for (int e = 0; e < OPL; ++e) acc[e] = fmaf(w, x[j][e], acc[e]);
      }
  }
  const float r = 1.f / lsum;
  uint16_t* out = a.out + static_cast<size_t>(row) * D + lane * OPL;
#pragma unroll
  for (int e = 0; e < OPL; e += 2) *reinterpret_cast<uint32_t*>(out + e) = pack2<BF>(acc[e] * r, acc[e + 1] * r);
}

// Launch for one element type (pkv_kv4_inst.cu, compiled once per type).
// With `reduce`, the cross-split reduce behind it.
cudaError_t launch_kv4_f16(const Kv4Args&, int head_dim, int block_size, unsigned grid, bool reduce, cudaStream_t);
cudaError_t launch_kv4_bf16(const Kv4Args&, int head_dim, int block_size, unsigned grid, bool reduce, cudaStream_t);

}  // namespace pkv
