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
// cores multiply subnormals exactly.  One 32-bit word of codes thus becomes
// four operand registers with a shift and four ANDs, and the powers of two
// come out of the results: for the keys through q (scaled to each head's
// largest element, the odd nibbles' channels by another 2^-4), for the values
// at the very end (even and odd nibbles are different output rows).
//
// One CTA handles one (sequence, kv head, up to 8 NT query heads, partition).
// Each warp owns a ring of NS stages of 32 tokens (two 16-token blocks or one
// of 32), each block's tile a contiguous run of bytes that lane 0 fetches with
// one untiled bulk copy per block for K and for V.  Per 16 tokens:
//   S[16 tok x 8 heads]: ldmatrix gives a lane one word (8 channels) of each of
//     two tokens; two k16 steps per group.
//   P' = P s in binary16, per group (a weight's rounding, 2^-12 of it at most,
//     and its product's are the only ones below FP32; P is binary16 for
//     bfloat16 inputs too, which have fewer bits).
//   O^T[32 ch x 8 heads] += codes^T P': ldmatrix.trans puts two neighbouring
//     tokens' words side by side; two m16 tiles per group.
//   z^T P' with the pairs (s, z) as they lie in the cache for the A operand:
//     rows 8 on give the group's zero-point sum for each head, in the same
//     lanes as O^T (one more m16 tile; its other rows are not used).
// P is scaled by 2^(9-E), E >= 0 from the largest value scale so far, so that
// neither small weights nor small scales fall out of binary16; the running sum
// carries the same factor.  The running maximum follows the true one only when
// that is more than 2^5 ahead, which spares most rescalings of the
// accumulators: P stays at most 2^14 and P' below 2^15.
#pragma once

#include <cuda_fp16.h>

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
};

constexpr int kKv4Warps = 4;
constexpr int kKv4Tokens = 32;   // per stage

// Stages per warp: about 40-60 KB of ring per CTA.
constexpr int kv4_stages(int D) { return D == 64 ? 4 : 2; }
// Resident CTAs per SM that the registers are budgeted for.
constexpr int kv4_ctas(int D, int NT) { return NT == 1 && D <= 128 ? 4 : (D == 64 ? 3 : 2); }
constexpr int kv4_stage_bytes(int D) { return 2 * kv4_tile_bytes(D, kKv4Tokens); }
constexpr int kv4_merge_bytes(int D, int NT) { return kKv4Warps * 8 * NT * (D + 2) * 4; }
constexpr int kv4_ring_bytes(int D) { return kKv4Warps * kv4_stages(D) * kv4_stage_bytes(D); }
constexpr int kv4_tail(int D, int NT) {
  return ((kv4_ring_bytes(D) > kv4_merge_bytes(D, NT) ? kv4_ring_bytes(D) : kv4_merge_bytes(D, NT)) + 127) & ~127;
}
constexpr int kv4_smem(int D, int NT) {
  return kv4_tail(D, NT) + kKv4Warps * kv4_stages(D) * 8 + kMaxBlocksPerCta * 4 + 128;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], "
      "%2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(addr + i * 4));
  }
}

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// One warp's running state over its tokens and its work on one stage.
template <bool BF, int D, int BS, int NT>
struct Kv4Compute {
  static constexpr int NG = D / 32;        // channel groups
  static constexpr int NH = 8 * NT;        // heads this warp produces
  static constexpr int TILE = kv4_tile_bytes(D, BS);
  static constexpr int PER = kKv4Tokens / BS;   // blocks per stage
  static constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u;
  static constexpr float kShift = 9.f, kSlack = 5.f;

  uint32_t qf[NG][NT][4];                  // B fragments: k16 step 0 (b0, b1), step 1 (b0, b1)
  float qs[NG][NT][2];                     // 2^-24 sum of the group's q, heads 2c and 2c + 1
  float sc[NT][2];                         // to log2 units, heads 2c and 2c + 1
  float o[2 * NG][NT][4];                  // codes^T P'
  float oz[NG][NT][4];                     // (s, z)^T P': elements 2 and 3 are z's
  float ref[NT][2], l[NT][2];              // running maximum less shift; sum
  float shift;                             // kShift - E

  // Heads g0 + nt * 8 + lane / 4 of the group's q rows at `qg` (zeros past G).
  // A head's row is scaled by the power of two that brings its largest element
  // into [2^14, 2^15): exact in binary16 for either type, but for elements
  // 2^-28 times the largest or less.
  __device__ __forceinline__ void load_q(const uint16_t* qg, int heads, float scale_log2, int lane) {
    const int c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + (lane >> 2);
      float x[NG][8];
      float top = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (h < heads) u = __ldg(reinterpret_cast<const uint4*>(qg + h * D + g * 32 + c * 8));
        const float2 f0 = unpack2<BF>(u.x), f1 = unpack2<BF>(u.y), f2 = unpack2<BF>(u.z),
                     f3 = unpack2<BF>(u.w);
        x[g][0] = f0.x; x[g][1] = f0.y; x[g][2] = f1.x; x[g][3] = f1.y;
        x[g][4] = f2.x; x[g][5] = f2.y; x[g][6] = f3.x; x[g][7] = f3.y;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[g][i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = 14 + 127 - static_cast<int>(__float_as_uint(top) >> 23);   // infinity: a finite factor
      e = top > 0.f ? min(e, 120) : 0;
      const float f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      const float back = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * 0x1p24f;
      sc[nt][0] = __shfl_sync(0xffffffffu, back, 8 * c);
      sc[nt][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[g][i] *= f;
          if (i & 1) x[g][i] *= 0.0625f;
        }
        // k index 2c + {0, 1} of step 0: channels 0 and 4 of the lane's eight,
        // then 2 and 6; of step 1: 1 and 5, then 3 and 7 (16 times their code)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int i = (b & 1) * 2 + (b >> 1);
          qf[g][nt][b] = pack2<false>(x[g][i], x[g][i + 4]);
          const float2 r = unpack2<false>(qf[g][nt][b]);
          sum += (r.x + r.y) * (b >> 1 ? 0x1p-20f : 0x1p-24f);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        qs[g][nt][0] = __shfl_sync(0xffffffffu, sum, 8 * c);
        qs[g][nt][1] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
      }
    }
  }

  __device__ __forceinline__ void reset() {
    shift = kShift;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ref[nt][0] = ref[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) o[i][nt][e] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) oz[g][nt][e] = 0.f;
      }
    }
  }

  __device__ __forceinline__ void rescale(const float (&by)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) l[nt][j] *= by[nt][j];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) o[i][nt][e] *= by[nt][e & 1];
#pragma unroll
        for (int g = 0; g < NG; ++g) oz[g][nt][e] *= by[nt][e & 1];
      }
    }
  }

  // Address of the 16-token half `mt` of a stage's K or V (block base and row).
  static __device__ __forceinline__ uint32_t block_of(uint32_t base, int mt) {
    return PER == 2 ? base + mt * TILE : base;
  }
  static constexpr int row_of(int mt) { return PER == 2 ? 0 : mt * 16; }

  // Clear the parameters of the tokens from `valid` on, so that whatever bytes
  // lie behind a sequence's end (NaN scales among them) count for nothing.
  static __device__ __forceinline__ void clear_tail(uint32_t kt, int valid, int lane) {
    const uint32_t vt = kt + PER * TILE;
    for (int i = lane; i < kKv4Tokens * NG; i += 32) {
      const int t = i / NG, g = i % NG;
      if (t < valid) continue;
      const int mt = t / 16, r = row_of(mt) + t % 16;
      const uint32_t kp = block_of(kt, mt) + kv4_k_par_off<D>(BS, r, g);
      const uint32_t vp = block_of(vt, mt) + kv4_v_par_off<D>(BS, r, g);
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(kp), "r"(0) : "memory");
      asm volatile("st.shared.b16 [%0], %1;" ::"r"(vp), "h"(static_cast<short>(0)) : "memory");
      asm volatile("st.shared.b16 [%0], %1;" ::"r"(vp + 4), "h"(static_cast<short>(0)) : "memory");
    }
    __syncwarp();
  }

  // The shift with which weights times a value scale of `top` stay in binary16.
  static __device__ __forceinline__ float lowered(float top, float shift) {
    const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;   // top < 2^(e + 1)
    return fminf(shift, kShift - static_cast<float>(min(max(e, 0), 17)));
  }

  // 32 tokens at `kt` (K) and `kt + PER * TILE` (V), the first `valid` of them real.
  __device__ __forceinline__ void stage(uint32_t kt, int valid, int lane) {
    const uint32_t vt = kt + PER * TILE;
    const int rr = lane & 7, half = (lane >> 3) & 1, hi = lane >> 4;
    // codes of (row half * 8 + rr, group hi of a pair): the lane's ldmatrix row
    const uint32_t lrow = (half * 8 + rr) * (D / 2);
    const int sw = rr * NG / 8;
    // added to the logits of the lane's tokens: minus infinity past the end
    float bias[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    if (valid < kKv4Tokens) {
      clear_tail(kt, valid, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        bias[i >> 1][i & 1] = i * 8 + (lane >> 2) < valid ? 0.f : -INFINITY;
    }

    float s[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t kb = block_of(kt, mt);
      uint32_t plo[NG], phi[NG];
      const uint32_t par = kb + BS * (D / 2) + (row_of(mt) + (lane >> 2)) * NG * 4;
      lds_words(par, plo);
      lds_words(par + 8 * NG * 4, phi);
#pragma unroll
      for (int g0 = 0; g0 < NG; g0 += 2) {
        uint32_t r[4];
        ldmatrix_x4(kb + row_of(mt) * (D / 2) + lrow + (((g0 + hi) ^ sw) << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const int g = g0 + gg;
          const uint32_t a = r[2 * gg], b = r[2 * gg + 1], a8 = a >> 8, b8 = b >> 8;
          const float2 lo = unpack2<false>(plo[g]), up = unpack2<false>(phi[g]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4] = {lo.y * qs[g][nt][0], lo.y * qs[g][nt][1], up.y * qs[g][nt][0],
                            up.y * qs[g][nt][1]};
            mma_16816<false>(acc, a & M0, b & M0, a8 & M0, b8 & M0, qf[g][nt][0], qf[g][nt][1]);
            mma_16816<false>(acc, a & M1, b & M1, a8 & M1, b8 & M1, qf[g][nt][2], qf[g][nt][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float by = e < 2 ? lo.x : up.x;
              s[mt][nt][e] = g == 0 ? by * acc[e] : fmaf(by, acc[e], s[mt][nt][e]);
            }
          }
        }
      }
    }

    // running maximum and sum
    float alpha[NT][2];
    bool grew = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[mt][nt][e] = fmaf(s[mt][nt][e], sc[nt][e & 1], bias[mt][e >> 1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = fmaxf(fmaxf(s[0][nt][j], s[0][nt][2 + j]), fmaxf(s[1][nt][j], s[1][nt][2 + j]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16)) - shift;
        const bool up = v > ref[nt][j] + kSlack;
        alpha[nt][j] = up ? fast_exp2(ref[nt][j] - v) : 1.f;
        ref[nt][j] = up ? v : ref[nt][j];
        grew |= up;
      }
    }
    if (__any_sync(0xffffffffu, grew)) rescale(alpha);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = fast_exp2(s[mt][nt][e] - ref[nt][e & 1]);
          s[mt][nt][e] = p;
          l[nt][e & 1] += p;
        }

#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t vb = block_of(vt, mt);
      // (s, s), (z, z) of tokens 2c, 2c + 1, then of 8 + 2c, 9 + 2c, per group
      uint32_t w[NG][4];
      const uint32_t par = vb + BS * (D / 2) + (row_of(mt) / 2 + (lane & 3)) * NG * 8;
      uint32_t large = 0;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[g][0]), "=r"(w[g][1]) : "r"(par + g * 8));
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                     : "=r"(w[g][2]), "=r"(w[g][3])
                     : "r"(par + 4 * NG * 8 + g * 8));
        large |= w[g][0] | w[g][2];
      }
      if (__any_sync(0xffffffffu, (large & 0x40004000u) != 0)) {   // rare
        float top = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float2 x = unpack2<false>(w[g][0]), y = unpack2<false>(w[g][2]);
          top = fmaxf(fmaxf(top, fmaxf(x.x, x.y)), fmaxf(y.x, y.y));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float now = lowered(top, shift);
        if (now < shift) {
          const float down = fast_exp2(now - shift);
          float by[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              by[nt][j] = down;
              ref[nt][j] += shift - now;
            }
#pragma unroll
            for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
              for (int x = 0; x < 4; ++x) s[m2][nt][x] *= down;
          }
          rescale(by);
          shift = now;
        }
      }
      // P^T as B operands: tokens 2c, 2c + 1 (b0) and 8 on (b1) of head lane / 4
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        b0[nt] = movmatrix_trans(pack2<false>(s[mt][nt][0], s[mt][nt][1]));
        b1[nt] = movmatrix_trans(pack2<false>(s[mt][nt][2], s[mt][nt][3]));
      }
#pragma unroll
      for (int g0 = 0; g0 < NG; g0 += 2) {
        uint32_t r[4];
        ldmatrix_x4_trans(vb + row_of(mt) * (D / 2) + lrow + (((g0 + hi) ^ sw) << 4), r[0], r[1], r[2],
                          r[3]);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const int g = g0 + gg;
          const uint32_t a = r[2 * gg], b = r[2 * gg + 1], a8 = a >> 8, b8 = b >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t p0 = hmul2_bits(b0[nt], w[g][0]), p1 = hmul2_bits(b1[nt], w[g][2]);
            mma_16816<false>(o[2 * g][nt], a & M0, a & M1, b & M0, b & M1, p0, p1);
            mma_16816<false>(o[2 * g + 1][nt], a8 & M0, a8 & M1, b8 & M0, b8 & M1, p0, p1);
            mma_16816<false>(oz[g][nt], w[g][0], w[g][1], w[g][2], w[g][3], p0, p1);
          }
        }
      }
    }
  }

  // Leave each head's (m, l, o) for the CTA merge.  Rows lane / 4 of tile
  // (g, a) are channels 32 g + 4 (lane / 4) + 2 a, rows 8 on the next channel.
  __device__ __forceinline__ void publish(float* cm, float* cl, float* co, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float lt = l[nt][j];
        lt += __shfl_xor_sync(0xffffffffu, lt, 4);
        lt += __shfl_xor_sync(0xffffffffu, lt, 8);
        lt += __shfl_xor_sync(0xffffffffu, lt, 16);
        const int h = nt * 8 + 2 * (lane & 3) + j;
        if (lane < 4) {
          cm[h] = ref[nt][j];
          cl[h] = lt;
        }
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) {
          const int d = 32 * (i >> 1) + 4 * (lane >> 2) + 2 * (i & 1);
          const float z = oz[i >> 1][nt][2 + j];
          *reinterpret_cast<float2*>(co + h * D + d) =
              make_float2(fmaf(o[i][nt][j], 0x1p24f, z), fmaf(o[i][nt][2 + j], 0x1p20f, z));
        }
      }
    }
  }
};

template <bool BF, int D, int BS, int NT>
__global__ void __launch_bounds__(kKv4Warps * 32, kv4_ctas(D, NT)) kv4_decode_kernel(const __grid_constant__ Kv4Args p) {
  using Compute = Kv4Compute<BF, D, BS, NT>;
  constexpr int NW = kKv4Warps, NS = kv4_stages(D), NH = Compute::NH;
  constexpr int TILE = Compute::TILE, PER = Compute::PER, STAGE = kv4_stage_bytes(D);
  static_assert(STAGE == 2 * PER * TILE, "stage");
  const DecodeArgs& a = p.d;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kv4_tail(D, NT));
  int* ids = reinterpret_cast<int*>(bars + NW * NS);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int idx = blockIdx.x;
  const int split = idx % a.S;
  idx /= a.S;
  const int chunk = idx % p.chunks;
  idx /= p.chunks;
  const int kvh = idx % a.Hkv;
  const int seq = idx / a.Hkv;
  const int heads = min(NH, a.G - chunk * NH);          // of this CTA
  const int h0 = kvh * a.G + chunk * NH;                // the first of them
  // resident before the stream's previous kernel is done; nothing is read before it is
  pdl_wait();
  pdl_launch_dependents();

  // block ids of the partition, range-checked; the first partition's are
  // loaded together with the length (it is empty only for padding rows)
  const int t0 = split * a.P, j0 = t0 / BS;
  const int32_t* trow = a.block_tables + static_cast<size_t>(seq) * a.MB + j0;
  const int L = a.context_lens[seq];
  if (split == 0)
    for (int k = threadIdx.x; k < min(a.P / BS, a.MB - j0); k += NW * 32) ids[k] = __ldg(trow + k);
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
  const int t1 = min(t0 + a.P, L);
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
  cs.load_q(a.q + (static_cast<size_t>(seq) * a.Hq + h0) * D, heads, a.scale_log2, lane);
  cs.reset();
  bool ok = true;
  int k = 0, st = 0;
  uint32_t phase = 0;
  for (; k < my_n; ++k) {
    const bool done = mbar_wait(wbar + 8 * st, phase);
    if (!__all_sync(0xffffffffu, done)) { ok = false; break; }
    const int left = t1 - t0 - (warp + NW * k) * kKv4Tokens;
    cs.stage(wbuf + st * STAGE, min(left, kKv4Tokens), lane);
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

  float* cm = reinterpret_cast<float*>(smem);
  float* cl = cm + NW * NH;
  float* co = cl + NW * NH;
  cs.publish(cm + warp * NH, cl + warp * NH, co + warp * NH * D, lane);
  __syncthreads();
  const bool single = (L + a.P - 1) / a.P == 1;
  for (int i = threadIdx.x; i < heads * D; i += NW * 32) {
    const int h = i / D, d = i - h * D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, cm[w * NH + h]);
    float acc = 0.f, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = fast_exp2(cm[w * NH + h] - M);
      acc = fmaf(f, co[(w * NH + h) * D + d], acc);
      lsum = fmaf(f, cl[w * NH + h], lsum);
    }
    const size_t row = static_cast<size_t>(seq) * a.Hq + h0 + h;
    if (single) {
      a.out[row * D + d] = to_elem<BF>(acc / lsum);
    } else {
      const size_t pr = row * a.S + split;
      a.part_o[pr * D + d] = acc;
      if (d == 0) a.part_ml[pr] = make_float2(M, lsum);
    }
  }
}

// Launch for one element type (pkv_kv4_inst.cu, compiled once per type).
cudaError_t launch_kv4_f16(const Kv4Args&, int head_dim, int block_size, int nt, unsigned grid, cudaStream_t);
cudaError_t launch_kv4_bf16(const Kv4Args&, int head_dim, int block_size, int nt, unsigned grid, cudaStream_t);

}  // namespace pkv
