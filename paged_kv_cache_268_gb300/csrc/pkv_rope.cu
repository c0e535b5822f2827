// Rotation and append of a step's queries, keys and values: into the 16-bit
// paged cache (pkv_rope_append) and into the 4-bit one (pkv_kv4_append), and
// the read-back of 4-bit rows (pkv_kv4_gather).  Contracts in include/pkv.h.
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>

#include "pkv.h"
#include "pkv_internal.h"
#include "pkv_kv4.cuh"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;

struct RopeArgs {
  const uint16_t* q;            // [T, Hq, D] with a token stride, or null
  const uint16_t* k;            // [T, Hkv, D] with a token stride
  const uint16_t* v;
  const int32_t* positions;     // [T], or null when rot_dim is 0
  const float* cos_sin;         // [max_position, rot_dim]: cosines, then sines
  const int32_t* slots;         // [T]
  uint16_t* q_out;              // [T, Hq, D]
  void* k_cache;
  void* v_cache;
  int* err;
  long long q_stride, k_stride, v_stride;   // elements between tokens
  int T, Hq, Hkv, bs, bs_log2, NB;
  int rows;                                 // head rows of one slice
  int rot, inter, max_pos;
};

template <bool BF>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const float2 a = unpack2<BF>(u.x), b = unpack2<BF>(u.y), c = unpack2<BF>(u.z),
               d = unpack2<BF>(u.w);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}
template <bool BF>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<BF>(x[0], x[1]), pack2<BF>(x[2], x[3]), pack2<BF>(x[4], x[5]),
                    pack2<BF>(x[6], x[7]));
}

// The IEEE quotient a / b for b with at most 11 significant bits, y = 1 / b to
// within 2^-23 of it.  q = a y, corrected by its exact remainder (Markstein's
// correction): before its last rounding the result is within 2^-22 half-steps
// of a / b.  That decides the rounding, as a / b is never that near a border
// between two floats: the border c has 25 bits, a - b c is a multiple of 2^-36
// of a, and not zero, so a / b is at least 2^-12 steps away from c.  (Quotients
// below 2^-70 may be off by more: their remainder is not exact.  They are never
// told from zero.)
__device__ __forceinline__ float quotient(float a, float b, float y) {
  const float q = __fmul_rn(a, y);
  return fmaf(fmaf(-q, b, a), y, q);
}

// Scale and zero point of the 32 channels that four neighbouring lanes hold
// eight each of, and this lane's eight codes (channel i in bits 4i .. 4i + 3).
// Quotients are true ones: 16-bit inputs often fall exactly on a border
// between two codes, where a product with a reciprocal would decide by its own
// rounding.  The scale is rounded up so that 15 steps always span the group,
// and is at least 1/1024 of its largest magnitude so that the zero point keeps
// a fraction of a step in binary16.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], __half* scale, __half* zero) {
  float lo = min_nan(min_nan(x[0], x[1], x[2]), min_nan(x[3], x[4], x[5]), min_nan(x[6], x[7]));
  float hi = max_nan(max_nan(x[0], x[1], x[2]), max_nan(x[3], x[4], x[5]), max_nan(x[6], x[7]));
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  const bool finite = lo >= -FLT_MAX && hi <= FLT_MAX;
  // (a span past FLT_MAX gives no number here, and the magnitude decides)
  const float span = quotient(__fsub_rn(hi, lo), 15.f, 1.f / 15.f);
  const float want =
      fmaxf(fmaxf(span, __fmul_rn(fmaxf(fabsf(lo), fabsf(hi)), 0x1p-10f)), 0x1p-24f);
  const __half h = __hmin(__float2half_ru(want), __ushort_as_half(0x7bff));   // at most 65504
  const float s = __half2float(h);
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  y = fmaf(fmaf(-s, y, 1.f), y, y);
  const float low = quotient(lo, s, y);
  const __half z = __float2half_rn(fminf(fmaxf(low, -65504.f), 65504.f));
  const float zf = __half2float(z);
  // 1.5 * 2^23 more rounds to a whole number, ties to even, in the low bits.
  // The codes' order is the values', so where lo's and hi's are within 0 .. 15
  // all are; the scale and zero point see to that but where z is large and
  // rounded by up to half a step, or the scale is at its end.
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __fsub_rn(quotient(x[i], s, y), zf);
  const bool within = __fsub_rn(low, zf) >= -0.5f && __fsub_rn(quotient(hi, s, y), zf) < 15.5f;
  if (__any_sync(0xffffffffu, !within)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], 0.f), 15.f);
  }
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) w = w * 16u + __float_as_uint(__fadd_rn(v[i], 12582912.f));
  w -= 0x3f400000u;   // the sum of 0x4b400000 * 16^i, which the eight roundings brought with them
  *scale = finite ? h : __ushort_as_half(0x7e00);   // an infinity or NaN: the group reads as NaN
  *zero = finite ? z : __ushort_as_half(0x7e00);
  return finite ? w : 0u;
}

// Rotation and append.  Work is (token, slice of its head rows); a CTA walks
// tokens blockIdx.x, + gridDim.x, ... of slice blockIdx.y.  Thread 0 stages a
// token's rows of the slice (a contiguous run each of q, k and v) and its
// table row in shared memory with bulk copies, kStages tokens ahead, so that
// the memory system always has tens of KB per SM to fetch and the lanes spend
// no instructions on it; bound by memory.  A lane owns one 16-byte chunk (eight
// channels) of a head row, the D/8 lanes of a row the whole row; it keeps the
// cosines and sines of its chunk for every head of the token and reads the
// half-split partner chunk from shared memory (so queries may be rotated in
// place).  The four lanes of 32 channels agree on the scale by shuffles.
// Measured on one GB300, 8192 tokens of 32 + 2 x 8 bfloat16 heads of 128 (206 MB
// in and out): 33.5 us, 6.1 TB/s, 0.91 of a copy; lanes that fetched their own
// chunks (16-byte asynchronous copies, six ahead) took 50 us and 210
// instructions a chunk, against 116.  Three CTAs per SM 34.6 us, half of the
// threads 40, slices of 8 KB 49.  Into the 4-bit cache, 2047 tokens of 32 + 2 x
// 32 binary16 heads (78 MB): 22.6 us, 0.51 of a copy, bound by the instructions
// of the codes (two thirds of the issue slots) and by 2047 tokens on 608 CTAs;
// 24.5 with slices of 16 KB, 29.6 with a division per channel in place of
// `quotient`.  A warp of its own for the fetching, with barriers both ways:
// 34.3 and 22.6 us, and 0.1-0.2 us more for a few tokens.
constexpr int kStages = 2;

constexpr int kSliceBytes = 24576;   // a slice's rows at most
constexpr int kAppendCtas = 4;       // per SM

struct TokenMeta {
  int slot;    // where k and v go, -1: nowhere
  int known;   // the position has a table row
};

template <bool BF, int D, bool KV4>
__global__ void __launch_bounds__(kThreads, kAppendCtas) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 8;              // lanes per row
  constexpr int R = kThreads / LPR;       // rows per pass
  constexpr int ROW = D * 2;              // bytes
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kStages];
  __shared__ TokenMeta meta[kStages];
  const int all = a.Hq + 2 * a.Hkv;
  const int ua = a.rows * blockIdx.y, n = min(a.rows, all - ua);   // rows of the slice
  const int stage_bytes = a.rows * ROW + a.rot * 4;
  const uint32_t base = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&bars[i]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();

  // Thread 0: stage token `t`, whose position and slot are given.
  auto issue = [&](int t, int pos, int slot, int st) {
    const uint32_t bar = smem_u32(&bars[st]);
    const bool known = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
    const bool beyond = slot >= 0 && static_cast<long long>(slot) >= static_cast<long long>(a.NB) * a.bs;
    if (blockIdx.y == 0) {
      if (!known) record_error(a.err, kDevBadPosition);
      else if (beyond) record_error(a.err, kDevBadSlot);
    }
    meta[st].slot = beyond || slot < 0 ? -1 : slot;
    meta[st].known = known;
    if (!known) {
      mbar_arrive(bar);
      return;
    }
    const int end = meta[st].slot >= 0 ? ua + n : min(ua + n, a.Hq);   // rows to fetch: [ua, end)
    mbar_arrive_expect_tx(bar, max(end - ua, 0) * ROW + a.rot * 4);
    const uint32_t dst = base + st * stage_bytes;
    // rows [from, to) of one tensor whose first row is row `zero` of the token
    auto rows = [&](const uint16_t* x, long long stride, int zero, int heads) {
      const int from = max(ua, zero), to = min(end, zero + heads);
      if (from < to)
        bulk_load(dst + (from - ua) * ROW, x + t * stride + (from - zero) * D, (to - from) * ROW, bar);
    };
    rows(a.q, a.q_stride, 0, a.Hq);
    rows(a.k, a.k_stride, a.Hq, a.Hkv);
    rows(a.v, a.v_stride, a.Hq + a.Hkv, a.Hkv);
    if (a.rot > 0)
      bulk_load(dst + a.rows * ROW, a.cos_sin + static_cast<size_t>(pos) * a.rot, a.rot * 4, bar);
  };
  const int gx = gridDim.x;
  int npos = 0, nslot = 0;                // of the next token to stage (thread 0)
  auto look = [&](int t) {
    if (t < a.T) {
      npos = a.rot > 0 ? a.positions[t] : 0;
      nslot = a.slots[t];
    }
  };
  if (threadIdx.x == 0) {
    look(blockIdx.x);
    for (int i = 0; i < kStages; ++i) {
      const int t = blockIdx.x + i * gx;
      if (t >= a.T) break;
      const int pos = npos, slot = nslot;
      look(t + gx);
      issue(t, pos, slot, i);
    }
  }

  const int c = threadIdx.x % LPR;
  const bool turned = c * 8 < a.rot, first = c * 16 < a.rot;       // in the rotated part; in its first half
  const int partner = (first ? c * 8 + a.rot / 2 : c * 8 - a.rot / 2) * 2;   // byte of the other half's chunk
  const int i0 = a.inter ? c * 4 : (first ? c * 8 : c * 8 - a.rot / 2);
  const int g = c >> 2;
  int st = 0;
  uint32_t phase = 0;
  bool failed = false;
  for (int t = blockIdx.x; t < a.T; t += gx) {
    const bool ok = mbar_wait(smem_u32(&bars[st]), phase);
    if (ok && meta[st].known) {
      const uint8_t* stage = smem + st * stage_bytes;
      const int slot = meta[st].slot;
      const int units = slot >= 0 ? n : min(n, a.Hq - ua);         // rows to work on
      const uint32_t block = slot >= 0 ? static_cast<uint32_t>(slot >> a.bs_log2) * a.Hkv : 0;   // first tile
      const int r = slot & (a.bs - 1);
      float cs[8], sn[8];
      if (turned) {
        const float* row = reinterpret_cast<const float*>(stage + a.rows * ROW) + i0;
        const float4 c0 = *reinterpret_cast<const float4*>(row);
        const float4 s0 = *reinterpret_cast<const float4*>(row + a.rot / 2);
        cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
        sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
        if (!a.inter) {
          const float4 c1 = *reinterpret_cast<const float4*>(row + 4);
          const float4 s1 = *reinterpret_cast<const float4*>(row + a.rot / 2 + 4);
          cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
          sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
        }
      }
      uint16_t* q_out = a.q_out + static_cast<size_t>(t) * a.Hq * D + c * 8;
      // the same number of rounds for every lane of a warp (its shuffles want whole warps)
      for (int b = 0; b < units; b += R) {
        const int i = b + threadIdx.x / LPR, u = ua + i;
        const bool live = i < units;
        const bool is_q = u < a.Hq, is_v = u >= a.Hq + a.Hkv;
        const uint8_t* row = stage + (live ? i : 0) * ROW;
        const uint4 raw = *reinterpret_cast<const uint4*>(row + c * 16);
        float x[8];
        unpack8<BF>(raw, x);
        if (turned && !is_v) {
          if (a.inter) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float p0 = x[2 * j], p1 = x[2 * j + 1];
              x[2 * j] = __fsub_rn(__fmul_rn(p0, cs[j]), __fmul_rn(p1, sn[j]));
              x[2 * j + 1] = __fadd_rn(__fmul_rn(p1, cs[j]), __fmul_rn(p0, sn[j]));
            }
          } else {
            float y[8];
            unpack8<BF>(*reinterpret_cast<const uint4*>(row + partner), y);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float p0 = __fmul_rn(x[j], cs[j]), p1 = __fmul_rn(y[j], sn[j]);
              x[j] = first ? __fsub_rn(p0, p1) : __fadd_rn(p0, p1);
            }
          }
        }
        __half s, z;
        uint32_t w = 0;
        if constexpr (KV4) {   // not where all rows are queries
          if (__any_sync(0xffffffffu, live && !is_q)) w = quantise8(x, &s, &z);
        }
        if (!live) continue;
        if (is_q) {
          *reinterpret_cast<uint4*>(q_out + u * D) = pack8<BF>(x);
          continue;
        }
        const int h = u - a.Hq - (is_v ? a.Hkv : 0);
        if constexpr (KV4) {
          uint8_t* tile = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + static_cast<size_t>(block + h) * static_cast<uint32_t>(kv4_tile_bytes(D, a.bs));
          *reinterpret_cast<uint32_t*>(tile + kv4_code_off<D>(r, g) + (c & 3) * 4) = w;
          if ((c & 3) == 0) {
            if (is_v) {
              uint8_t* par = tile + kv4_v_par_off<D>(a.bs, r, g);
              *reinterpret_cast<__half*>(par) = s;
              *reinterpret_cast<__half*>(par + 4) = z;
            } else {
              *reinterpret_cast<__half2*>(tile + kv4_k_par_off<D>(a.bs, r, g)) = __halves2half2(s, z);
            }
          }
        } else {
          uint16_t* dst = static_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) + (static_cast<size_t>(block + h) * a.bs + r) * D + c * 8;
          *reinterpret_cast<uint4*>(dst) = is_v ? raw : pack8<BF>(x);
        }
      }
    }
    failed = __syncthreads_or(!ok);       // every lane is done with the stage
    if (failed) break;
    if (threadIdx.x == 0) {
      const int next = t + kStages * gx;
      if (next < a.T) {
        const int pos = npos, slot = nslot;
        look(next + gx);
        fence_proxy_async_smem();
        issue(next, pos, slot, st);
      }
    }
    if (++st == kStages) {
      st = 0;
      phase ^= 1;
    }
  }
  if (failed && threadIdx.x == 0) {
    // a copy did not come in time: give all that are in flight a bounded chance to land
    for (int i = 0; i < kStages; ++i) mbar_wait(smem_u32(&bars[i]), i >= st ? phase : phase ^ 1, 100000000ull);
    record_error(a.err, kDevTimeout);
  }
}

// Rows of the 4-bit cache back in 16 bits.  value = scale * code + scale * zero:
// both products are exact in FP32 (15 and 22 bits), so the value is rounded once
// there, and once at the store.  Rows of a negative or
// bad slot become zeros.  The D/8 lanes of a row hold one chunk each; a CTA
// takes TOK tokens and LOOPS passes over their head rows, all of whose bytes
// it asks for before it works on the first.  Bound by memory: three of its four
// bytes are written.  Measured on one GB300, 32768 rows of 8 bfloat16 heads of
// 128 (176 MB in and out): 29.4 us, 6.0 TB/s, 0.89 of a copy, with four tokens
// and one pass (31.2 with two and two, 33.7 when a pass waited for the one
// before, 58 with 64-bit divisions and one load at a time; 256 threads 35.4,
// 64 30.1, eight tokens 30.5).  Small calls want more CTAs: 1999 rows 3.3 us
// with two tokens, 3.4 with four; 128 rows of 32 + 32 heads 1.9 and 2.3.
constexpr int kGatherThreads = 128;

template <bool BF, int D, int BS, int TOK, int LOOPS>
__global__ void __launch_bounds__(kGatherThreads)
    kv4_gather_kernel(const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
                      const int32_t* __restrict__ slots, uint16_t* __restrict__ k,
                      uint16_t* __restrict__ v, int T, int Hkv, int NB, int* err) {
  constexpr int LPR = D / 8;
  constexpr int R = kGatherThreads / LPR;
  constexpr uint32_t TILE = kv4_tile_bytes(D, BS);
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = blockIdx.x * TOK;
  const int c = threadIdx.x % LPR, g = c >> 2;
  uint32_t block[TOK];   // first tile of the slot's block
  int row[TOK];
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    row[i] = -1;
    if (t0 + i < T) {
      const int slot = __ldg(slots + t0 + i);
      if (slot >= 0 && static_cast<long long>(slot) < static_cast<long long>(NB) * BS) {
        block[i] = static_cast<uint32_t>(slot / BS) * Hkv;
        row[i] = slot % BS;
      } else if (slot >= 0 && threadIdx.x == 0 && blockIdx.y == 0) {
        record_error(err, kDevBadSlot);
      }
    }
  }
  const int last = min(2 * Hkv, R * LOOPS * static_cast<int>(blockIdx.y + 1));
  const int u0 = R * LOOPS * blockIdx.y + threadIdx.x / LPR;
  // all of the CTA's bytes first, so that their latencies overlap
  uint32_t w[LOOPS][TOK], par[LOOPS][TOK];
#pragma unroll
  for (int j = 0; j < LOOPS; ++j) {
    const int u = u0 + j * R;
    const bool is_v = u >= Hkv;
    const int h = is_v ? u - Hkv : u;
    const uint8_t* cache = is_v ? v_cache : k_cache;
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      w[j][i] = par[j][i] = 0;                   // a padding row: scale 0, all zeros
      if (row[i] < 0 || u >= last) continue;
      const uint8_t* base = cache + static_cast<size_t>(block[i] + h) * TILE;
      w[j][i] = __ldg(reinterpret_cast<const uint32_t*>(base + kv4_code_off<D>(row[i], g) + (c & 3) * 4));
      if (is_v) {
        const uint8_t* p = base + kv4_v_par_off<D>(BS, row[i], g);
        par[j][i] = __ldg(reinterpret_cast<const uint16_t*>(p)) |
                    static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p + 4))) << 16;
      } else {
        par[j][i] = __ldg(reinterpret_cast<const uint32_t*>(base + kv4_k_par_off<D>(BS, row[i], g)));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < LOOPS; ++j) {
    const int u = u0 + j * R;
    if (u >= last) break;
    const bool is_v = u >= Hkv;
    uint16_t* dst = (is_v ? v : k) + (static_cast<size_t>(t0) * Hkv + (is_v ? u - Hkv : u)) * D + c * 8;
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      if (t0 + i >= T) break;
      const float2 p = unpack2<false>(par[j][i]);
      const float scale = p.x * 0x1p24f, low = p.x * p.y;
      float x[8];
      // nibbles e and e + 4 as binary16 subnormals, n * 2^-24
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 n = unpack2<false>((w[j][i] >> (4 * e)) & 0x000f000fu);
        x[e] = fmaf(n.x, scale, low);
        x[e + 4] = fmaf(n.y, scale, low);
      }
      *reinterpret_cast<uint4*>(dst + static_cast<size_t>(i) * Hkv * D) = pack8<BF>(x);
    }
  }
}

template <int TOK, int LOOPS, bool BF, int D>
auto gather_kernel(int bs) {
  return bs == 32 ? kv4_gather_kernel<BF, D, 32, TOK, LOOPS> : kv4_gather_kernel<BF, D, 16, TOK, LOOPS>;
}
template <int TOK, int LOOPS>
auto gather_kernel(bool bf, int D, int bs) {
  auto kern = bf ? gather_kernel<TOK, LOOPS, true, 64>(bs) : gather_kernel<TOK, LOOPS, false, 64>(bs);
  if (D == 128) kern = bf ? gather_kernel<TOK, LOOPS, true, 128>(bs) : gather_kernel<TOK, LOOPS, false, 128>(bs);
  if (D == 256) kern = bf ? gather_kernel<TOK, LOOPS, true, 256>(bs) : gather_kernel<TOK, LOOPS, false, 256>(bs);
  return kern;
}

// The kernels' shared-memory limit, raised once per device and kernel (threads
// that race here set the same attribute).
cudaError_t raise_smem(const void* kern, bool kv4, bool bf, int D) {
  static std::atomic<unsigned> masks[12];
  std::atomic<unsigned>& mask = masks[(D == 64 ? 0 : (D == 128 ? 1 : 2)) * 4 + kv4 * 2 + bf];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned bit = dev < 32 ? 1u << dev : 0u;
  if (bit != 0 && (mask.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * (kSliceBytes + 1024));
  if (e == cudaSuccess) mask.fetch_or(bit, std::memory_order_release);
  return e;
}

template <bool KV4>
int append(const pkv_shape* s, const pkv_rope* rope, const void* q, const void* k, const void* v,
           const int32_t* positions, const float* cos_sin, const int32_t* slots, int32_t num_tokens,
           void* q_out, void* k_cache, void* v_cache, pkv_stream_t stream) {
  if (!s || !rope) return PKV_ERR_NULL;
  int rc = check_cache_shape(s);
  if (rc != PKV_OK) return rc;
  if (num_tokens < 0 || rope->rot_dim < 0 || rope->rot_dim > s->head_dim ||
      (rope->rot_dim > 0 && rope->max_position < 1) || (q && s->num_q_heads < 1))
    return PKV_ERR_INVALID;
  if (rope->rot_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
  const int D = s->head_dim;
  const long long qd = static_cast<long long>(s->num_q_heads) * D;
  const long long kd = static_cast<long long>(s->num_kv_heads) * D;
  RopeArgs a{};
  a.q_stride = rope->q_stride ? rope->q_stride : qd;
  a.k_stride = rope->k_stride ? rope->k_stride : kd;
  a.v_stride = rope->v_stride ? rope->v_stride : kd;
  if ((q && a.q_stride < qd) || a.k_stride < kd || a.v_stride < kd) return PKV_ERR_INVALID;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slots || !k_cache || !v_cache || (q && !q_out) ||
      (rope->rot_dim > 0 && (!positions || !cos_sin)))
    return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(cos_sin, 16) ||
      !aligned(slots, 4) || !aligned(positions, 4) || a.q_stride % 8 || a.k_stride % 8 || a.v_stride % 8)
    return PKV_ERR_ALIGN;
  // in place only row for row: a strided q has its rows elsewhere than q_out's
  if (q && q == q_out && a.q_stride != qd) return PKV_ERR_INVALID;
  // tokens and rows are counted in 32 bits, with room for the walkers' steps
  if (num_tokens > (1 << 30) || static_cast<long long>(s->num_q_heads) + 2ll * s->num_kv_heads > (1ll << 30))
    return PKV_ERR_UNSUPPORTED;
  a.err = device_error_word();
  if (!a.err) return PKV_ERR_CUDA;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.slots = slots;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.T = num_tokens;
  a.Hq = q ? s->num_q_heads : 0;
  a.Hkv = s->num_kv_heads;
  a.bs = s->block_size;
  a.bs_log2 = s->block_size == 32 ? 5 : 4;
  a.NB = s->num_blocks;
  a.rot = rope->rot_dim;
  a.inter = rope->interleaved != 0;
  a.max_pos = rope->max_position;
  const bool bf = s->dtype == PKV_BF16;
  void (*kern)(RopeArgs) = nullptr;
  if (D == 64) kern = bf ? rope_append_kernel<true, 64, KV4> : rope_append_kernel<false, 64, KV4>;
  if (D == 128) kern = bf ? rope_append_kernel<true, 128, KV4> : rope_append_kernel<false, 128, KV4>;
  if (D == 256) kern = bf ? rope_append_kernel<true, 256, KV4> : rope_append_kernel<false, 256, KV4>;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc != PKV_OK) return rc;
  // kAppendCtas CTAs per SM walk the tokens.  A slice has at most 24 KB of rows
  // (the CTAs' stages fit an SM's shared memory), and fewer where there are
  // not tokens enough for every CTA: down to one pass of the CTA's threads.
  const int pass = kThreads / (D / 8), all = a.Hq + 2 * a.Hkv, most = kSliceBytes / (D * 2);
  const int resident = kAppendCtas * sms;
  long long slices = (all + most - 1) / most;
  if (num_tokens * slices < resident) {
    slices = resident / num_tokens;
    if (slices > (all + pass - 1) / pass) slices = (all + pass - 1) / pass;
  }
  a.rows = static_cast<int>((all + slices - 1) / slices);
  a.rows = (a.rows + pass - 1) / pass * pass;
  if (a.rows > most) a.rows = most;
  slices = (all + a.rows - 1) / a.rows;
  if (slices > 65535) return PKV_ERR_UNSUPPORTED;
  long long walkers = resident / slices;
  if (walkers < 1) walkers = 1;
  const dim3 grid(static_cast<unsigned>(num_tokens < walkers ? num_tokens : walkers),
                  static_cast<unsigned>(slices));
  const size_t smem = static_cast<size_t>(kStages) * (static_cast<size_t>(a.rows) * D * 2 + a.rot * 4);
  cudaError_t e = raise_smem(reinterpret_cast<const void*>(kern), KV4, bf, D);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  e = launch_pdl(kern, grid, kThreads, smem, reinterpret_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launch();
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_rope_append(const pkv_shape* s, const pkv_rope* rope, const void* q, const void* k,
                               const void* v, const int32_t* positions, const float* cos_sin,
                               const int32_t* slot_mapping, int32_t num_tokens, void* q_out,
                               void* k_cache, void* v_cache, pkv_stream_t stream) {
  return append<false>(s, rope, q, k, v, positions, cos_sin, slot_mapping, num_tokens, q_out,
                       k_cache, v_cache, stream);
}

extern "C" int pkv_kv4_append(const pkv_shape* s, const pkv_rope* rope, const void* q, const void* k,
                              const void* v, const int32_t* positions, const float* cos_sin,
                              const int32_t* slot_mapping, int32_t num_tokens, void* q_out,
                              void* k_cache, void* v_cache, pkv_stream_t stream) {
  return append<true>(s, rope, q, k, v, positions, cos_sin, slot_mapping, num_tokens, q_out,
                      k_cache, v_cache, stream);
}

extern "C" int pkv_kv4_gather(const pkv_shape* s, const void* k_cache, const void* v_cache,
                              const int32_t* slot_mapping, int32_t num_tokens, void* k, void* v,
                              pkv_stream_t stream) {
  int rc = check_cache_shape(s);
  if (rc != PKV_OK) return rc;
  if (num_tokens < 0) return PKV_ERR_INVALID;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_mapping, 4))
    return PKV_ERR_ALIGN;
  const int D = s->head_dim;
  const int rows = kGatherThreads / (D / 8);             // of a pass
  const long long passes = (2ll * s->num_kv_heads - 1) / rows + 1;
  if (num_tokens > (1 << 30) || passes > 65535) return PKV_ERR_UNSUPPORTED;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc != PKV_OK) return rc;
  // Four tokens a CTA where that leaves 32 CTAs for every SM, two resident
  // waves (measured equal at 27, 2047 rows of 32 heads: 10.7 us both; figures
  // beyond and below at the kernel).
  const bool many = (num_tokens / 4) * passes >= 32ll * sms;
  const int tokens = many ? 4 : 2, loops = many ? 1 : 2;
  const dim3 grid(static_cast<unsigned>((num_tokens - 1) / tokens + 1),
                  static_cast<unsigned>((passes + loops - 1) / loops));
  int* err = device_error_word();
  if (!err) return PKV_ERR_CUDA;
  const bool bf = s->dtype == PKV_BF16;
  auto kern = many ? gather_kernel<4, 1>(bf, D, s->block_size) : gather_kernel<2, 2>(bf, D, s->block_size);
  cudaError_t e = launch_pdl(kern, grid, kGatherThreads, 0,
                             reinterpret_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(k_cache),
                             static_cast<const uint8_t*>(v_cache), slot_mapping,
                             static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), num_tokens,
                             s->num_kv_heads, s->num_blocks, err);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launch();
  return PKV_OK;
}
