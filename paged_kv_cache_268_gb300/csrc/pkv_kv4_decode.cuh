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
//   z^T P' with z in every row of the A operand: the group's zero-point sum
//     for each head, in the same lanes as O^T (one more m16 tile).
// P is scaled by 2^(15-E), E >= 0 the binary exponent of the largest value
// scale so far, so that neither small weights nor small scales fall out of
// binary16 and P' stays below 2^15; the running sum carries the same factor.
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
constexpr int kv4_stages(int D) { return D == 64 ? 4 : (D == 128 ? 3 : 2); }
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

  uint32_t qf[NG][NT][4];                  // B fragments: k16 step 0 (b0, b1), step 1 (b0, b1)
  float qs[NG][NT][2];                     // 2^-24 sum of the group's q, heads 2c and 2c + 1
  float sc[NT][2];                         // to log2 units, heads 2c and 2c + 1
  float o[2 * NG][NT][4];                  // codes^T P'
  float oz[NG][NT][4];                     // z^T P' (every row the same)
  float ref[NT][2], l[NT][2];              // running maximum less shift; sum
  float shift;                             // 15 - E

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
    shift = 15.f;
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

  // 32 tokens at `kt` (K) and `kt + PER * TILE` (V), the first `valid` of them real.
  __device__ __forceinline__ void stage(uint32_t kt, int valid, int lane) {
    const uint32_t vt = kt + PER * TILE;
    const int rr = lane & 7, half = (lane >> 3) & 1, hi = lane >> 4;
    // codes of (row half * 8 + rr, group hi of a pair): the lane's ldmatrix row
    const uint32_t lrow = (half * 8 + rr) * (D / 2);
    const int sw = rr * NG / 8;
    const bool ragged = valid < kKv4Tokens;

    float s[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t kb = block_of(kt, mt);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
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
            s[mt][nt][0] = fmaf(lo.x, acc[0], s[mt][nt][0]);
            s[mt][nt][1] = fmaf(lo.x, acc[1], s[mt][nt][1]);
            s[mt][nt][2] = fmaf(up.x, acc[2], s[mt][nt][2]);
            s[mt][nt][3] = fmaf(up.x, acc[3], s[mt][nt][3]);
          }
        }
      }
    }

    // running maximum and sum; tokens past the end are masked
    float alpha[NT][2];
    bool grew = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[mt][nt][e] * sc[nt][e & 1];
          if (ragged && mt * 16 + (lane >> 2) + ((e >> 1) << 3) >= valid) x = -INFINITY;
          s[mt][nt][e] = x;
          mx[e & 1] = fmaxf(mx[e & 1], x);
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = mx[j];
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        const float now = fmaxf(ref[nt][j], v - shift);
        alpha[nt][j] = fast_exp2(ref[nt][j] - now);
        grew |= now != ref[nt][j];
        ref[nt][j] = now;
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
      // parameters of tokens 2c, 2c + 1 and 8 + 2c, 9 + 2c: (s, s), (z, z) per group
      uint32_t w0[2 * NG], w1[2 * NG];
      const uint32_t par = vb + BS * (D / 2) + (row_of(mt) / 2 + (lane & 3)) * NG * 8;
      lds_words(par, w0);
      lds_words(par + 4 * NG * 8, w1);
      if (ragged) {
        const int t = mt * 16 + 2 * (lane & 3);
        const uint32_t m0 = (t < valid ? 0xffffu : 0u) | (t + 1 < valid ? 0xffff0000u : 0u);
        const uint32_t m1 = (t + 8 < valid ? 0xffffu : 0u) | (t + 9 < valid ? 0xffff0000u : 0u);
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) {
          w0[i] &= m0;
          w1[i] &= m1;
        }
      }
      // a value scale of 2^E or more: lower the shift (rare)
      __half2 most = *reinterpret_cast<__half2*>(&w0[0]);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        most = __hmax2(most, *reinterpret_cast<__half2*>(&w0[2 * g]));
        most = __hmax2(most, *reinterpret_cast<__half2*>(&w1[2 * g]));
      }
      float top = fmaxf(__low2float(most), __high2float(most));
      if (__any_sync(0xffffffffu, top * __int_as_float(static_cast<int>(112.f + shift) << 23) > 1.f)) {
        // 2^-E = 2^(shift - 15); new E: the exponent above the largest scale
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = static_cast<int>(__float_as_uint(top) >> 23) - 126;
        const float now = 15.f - static_cast<float>(min(e, 17));
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
            const uint32_t p0 = hmul2_bits(b0[nt], w0[2 * g]), p1 = hmul2_bits(b1[nt], w1[2 * g]);
            mma_16816<false>(o[2 * g][nt], a & M0, a & M1, b & M0, b & M1, p0, p1);
            mma_16816<false>(o[2 * g + 1][nt], a8 & M0, a8 & M1, b8 & M0, b8 & M1, p0, p1);
            mma_16816<false>(oz[g][nt], w0[2 * g + 1], w0[2 * g + 1], w1[2 * g + 1], w1[2 * g + 1], p0, p1);
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
          const float z = oz[i >> 1][nt][j];
          *reinterpret_cast<float2*>(co + h * D + d) =
              make_float2(fmaf(o[i][nt][j], 0x1p24f, z), fmaf(o[i][nt][2 + j], 0x1p20f, z));
        }
      }
    }
  }
};

template <bool BF, int D, int BS, int NT>
__global__ void __launch_bounds__(kKv4Warps * 32) kv4_decode_kernel(const __grid_constant__ Kv4Args p) {
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
  auto issue = [&](int k) {
    const int st = k % NS, b0 = (warp + NW * k) * PER;
    const int nb = min(PER, nblk - b0);
    const uint32_t bar = wbar + 8 * st, dst = wbuf + st * STAGE;
    mbar_arrive_expect_tx(bar, nb * 2 * TILE);
    for (int b = 0; b < nb; ++b) {
      const size_t at = (static_cast<size_t>(ids[b0 + b]) * a.Hkv + kvh) * TILE;
      bulk_load(dst + b * TILE, p.k + at, TILE, bar, policy);
      bulk_load(dst + (PER + b) * TILE, p.v + at, TILE, bar, policy);
    }
  };
  if (lane == 0) {
    const int pro = my_n < NS ? my_n : NS;
    for (int k = 0; k < pro; ++k) issue(k);
  }

  Compute cs;
  cs.load_q(a.q + (static_cast<size_t>(seq) * a.Hq + h0) * D, heads, a.scale_log2, lane);
  cs.reset();
  bool ok = true;
  int k = 0;
  for (; k < my_n; ++k) {
    const int st = k % NS;
    const bool done = mbar_wait(wbar + 8 * st, (k / NS) & 1);
    if (!__all_sync(0xffffffffu, done)) { ok = false; break; }
    const int left = t1 - t0 - (warp + NW * k) * kKv4Tokens;
    cs.stage(wbuf + st * STAGE, min(left, kKv4Tokens), lane);
    __syncwarp();
    if (lane == 0 && k + NS < my_n) {
      fence_proxy_async_smem();
      issue(k + NS);
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
