// Rotation and append of a step's queries, keys and values: into the 16-bit
// paged cache (pkv_rope_append) and into the 4-bit one (pkv_kv4_append), and
// the read-back of 4-bit rows (pkv_kv4_gather).  Contracts in include/pkv.h.
#include <cuda_fp16.h>

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
  int Hq, Hkv, bs, NB;
  int rot, inter, max_pos;
};

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

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

// Scale and zero point of the 32 channels that four neighbouring lanes hold
// eight each of, and this lane's eight codes (channel i in bits 4i .. 4i + 3).
// Every quotient is a true division: 16-bit inputs often fall exactly on a
// border between two codes, where a product with a reciprocal would decide by
// its own rounding.  The scale is rounded up so that 15 steps always span the
// group, and is at least 1/1024 of its largest magnitude so that the zero
// point keeps a fraction of a step in binary16.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], __half* scale, __half* zero) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  if (!(lo >= -FLT_MAX && hi <= FLT_MAX)) {   // an infinity or NaN: the group reads as NaN
    *scale = *zero = __ushort_as_half(0x7e00);
    return 0;
  }
  const float want = fmaxf(fmaxf(__fdiv_rn(__fsub_rn(hi, lo), 15.f),
                                 __fmul_rn(fmaxf(fabsf(lo), fabsf(hi)), 0x1p-10f)),
                           0x1p-24f);
  __half h = __float2half_ru(want);
  float s = __half2float(h);
  if (s > 65504.f) {
    s = 65504.f;
    h = __float2half_rn(s);
  }
  const __half z = __float2half_rn(fminf(fmaxf(__fdiv_rn(lo, s), -65504.f), 65504.f));
  const float zf = __half2float(z);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = fminf(fmaxf(rintf(__fsub_rn(__fdiv_rn(x[i], s), zf)), 0.f), 15.f);
    w |= static_cast<uint32_t>(n) << (4 * i);
  }
  *scale = h;
  *zero = z;
  return w;
}

// One CTA per token (and slice of its heads).  A lane owns one 16-byte chunk
// (eight channels) of a head row, the D/8 lanes of a row the whole row; the
// lane keeps the cosines and sines of its chunk in registers for every head
// that it visits.  The half-split partner of a chunk comes from the lane that
// holds it, so queries may be rotated in place.  The four lanes of 32
// channels agree on the scale by shuffles.  Bound by memory: a lane asks for
// its chunks of up to kAhead heads before it works on the first.
constexpr int kAhead = 3;

template <bool BF, int D, bool KV4>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 8;              // lanes per row
  constexpr int R = kThreads / LPR;       // rows per pass
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x;
  const int c = threadIdx.x % LPR;
  const int lane = threadIdx.x & 31;
  const int all = a.Hq + 2 * a.Hkv, step = R * gridDim.y;
  int u = R * blockIdx.y + threadIdx.x / LPR;
  auto load = [&](int v) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (v < all) {
      const uint16_t* row = v < a.Hq ? a.q + t * a.q_stride + v * D
                                     : (v < a.Hq + a.Hkv ? a.k + t * a.k_stride + (v - a.Hq) * D
                                                         : a.v + t * a.v_stride + (v - a.Hq - a.Hkv) * D);
      x = *reinterpret_cast<const uint4*>(row + c * 8);
    }
    return x;
  };
  uint4 raw[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) raw[i] = load(u + i * step);

  int slot = a.slots[t];
  const bool turned = c * 8 < a.rot;
  float cs[8], sn[8];
  if (a.rot > 0) {
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.max_pos) {
      if (threadIdx.x == 0 && blockIdx.y == 0) record_error(a.err, kDevBadPosition);
      return;
    }
    const float* row = a.cos_sin + static_cast<size_t>(pos) * a.rot;
    const int half = a.rot / 2;
    if (turned) {
      const int i0 = a.inter ? c * 4 : (c * 8 < half ? c * 8 : c * 8 - half);
      const int n = a.inter ? 4 : 8;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        if (i < n) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
          const float4 y = __ldg(reinterpret_cast<const float4*>(row + half + i0 + i));
          cs[i] = x.x; cs[i + 1] = x.y; cs[i + 2] = x.z; cs[i + 3] = x.w;
          sn[i] = y.x; sn[i + 1] = y.y; sn[i + 2] = y.z; sn[i + 3] = y.w;
        }
      }
    }
  }
  if (slot >= 0 && static_cast<long long>(slot) >= static_cast<long long>(a.NB) * a.bs) {
    if (threadIdx.x == 0 && blockIdx.y == 0) record_error(a.err, kDevBadSlot);
    slot = -1;
  }
  const int units = slot >= 0 ? all : a.Hq;
  const size_t block = slot >= 0 ? static_cast<size_t>(slot / a.bs) * a.Hkv : 0;
  const int r = slot >= 0 ? slot % a.bs : 0;
  const bool first = c * 16 < a.rot;                       // chunk of the first half
  const int partner = a.inter || !turned ? lane : (first ? lane + a.rot / 16 : lane - a.rot / 16);

  auto work = [&](int v, const uint4& raw) {
    const bool live = v < units;
    const bool is_q = v < a.Hq, is_v = v >= a.Hq + a.Hkv;
    const int h = is_q ? v : (is_v ? v - a.Hq - a.Hkv : v - a.Hq);
    float x[8];
    unpack8<BF>(raw, x);
    if (a.rot > 0) {
      if (a.inter) {
        if (turned && !is_v) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(p, cs[i]), __fmul_rn(q, sn[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(q, cs[i]), __fmul_rn(p, sn[i]));
          }
        }
      } else {
        uint4 other;
        other.x = __shfl_sync(0xffffffffu, raw.x, partner);
        other.y = __shfl_sync(0xffffffffu, raw.y, partner);
        other.z = __shfl_sync(0xffffffffu, raw.z, partner);
        other.w = __shfl_sync(0xffffffffu, raw.w, partner);
        float y[8];
        unpack8<BF>(other, y);
        if (turned && !is_v) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float p = __fmul_rn(x[i], cs[i]), q = __fmul_rn(y[i], sn[i]);
            x[i] = first ? __fsub_rn(p, q) : __fadd_rn(p, q);
          }
        }
      }
    }
    __half s, z;
    uint32_t w = 0;
    if constexpr (KV4) {   // whole warps: the shuffles want them; none where all rows are queries
      if (__any_sync(0xffffffffu, live && !is_q)) w = quantise8(x, &s, &z);
    }
    if (!live) return;
    if (is_q) {
      *reinterpret_cast<uint4*>(a.q_out + (static_cast<size_t>(t) * a.Hq + h) * D + c * 8) = pack8<BF>(x);
      return;
    }
    if constexpr (KV4) {
      uint8_t* base = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (block + h) * kv4_tile_bytes(D, a.bs);
      const int g = c >> 2;
      *reinterpret_cast<uint32_t*>(base + kv4_code_off<D>(r, g) + (c & 3) * 4) = w;
      if ((c & 3) == 0) {
        if (is_v) {
          uint8_t* p = base + kv4_v_par_off<D>(a.bs, r, g);
          *reinterpret_cast<__half*>(p) = s;
          *reinterpret_cast<__half*>(p + 4) = z;
        } else {
          *reinterpret_cast<__half2*>(base + kv4_k_par_off<D>(a.bs, r, g)) = __halves2half2(s, z);
        }
      }
    } else {
      uint16_t* dst = static_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) + ((block + h) * a.bs + r) * D + c * 8;
      *reinterpret_cast<uint4*>(dst) = is_v ? raw : pack8<BF>(x);
    }
  };

  // the same number of rounds for every lane of a warp
  for (int base = R * blockIdx.y; base < units; base += kAhead * step, u += kAhead * step) {
    uint4 now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) now[i] = raw[i];
    if (base + kAhead * step < units) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) raw[i] = load(u + (kAhead + i) * step);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (base + i * step < units) work(u + i * step, now[i]);
  }
}

// Rows of the 4-bit cache back in 16 bits: the D/8 lanes of a row hold one
// chunk each.  value = scale * (code + zero) in FP32 (the sum is exact), one
// rounding at the store.  Rows of a negative or bad slot become zeros.  A CTA
// takes kTokens tokens; a lane asks for the same head's chunk of all of them
// before it works on the first (bound by memory: three of its four bytes are
// written).
constexpr int kTokens = 4;

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads)
    kv4_gather_kernel(const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
                      const int32_t* __restrict__ slots, uint16_t* __restrict__ k,
                      uint16_t* __restrict__ v, int T, int Hkv, int bs, int NB, int* err) {
  constexpr int LPR = D / 8;
  constexpr int R = kThreads / LPR;
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = blockIdx.x * kTokens;
  const int c = threadIdx.x % LPR, g = c >> 2;
  size_t block[kTokens];
  int row[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    row[i] = -1;
    if (t0 + i < T) {
      const int slot = slots[t0 + i];
      if (slot >= 0 && static_cast<long long>(slot) < static_cast<long long>(NB) * bs) {
        block[i] = static_cast<size_t>(slot / bs) * Hkv;
        row[i] = slot % bs;
      } else if (slot >= 0 && threadIdx.x == 0 && blockIdx.y == 0) {
        record_error(err, kDevBadSlot);
      }
    }
  }
  for (int u = R * blockIdx.y + threadIdx.x / LPR; u < 2 * Hkv; u += R * gridDim.y) {
    const bool is_v = u >= Hkv;
    const int h = is_v ? u - Hkv : u;
    uint32_t w[kTokens], par[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      w[i] = par[i] = 0;
      if (row[i] < 0) continue;
      const uint8_t* base = (is_v ? v_cache : k_cache) + (block[i] + h) * kv4_tile_bytes(D, bs);
      w[i] = *reinterpret_cast<const uint32_t*>(base + kv4_code_off<D>(row[i], g) + (c & 3) * 4);
      if (is_v) {
        const uint8_t* p = base + kv4_v_par_off<D>(bs, row[i], g);
        par[i] = *reinterpret_cast<const uint16_t*>(p) |
                 static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + 4)) << 16;
      } else {
        par[i] = *reinterpret_cast<const uint32_t*>(base + kv4_k_par_off<D>(bs, row[i], g));
      }
    }
    uint16_t* dst = (is_v ? v : k) + (static_cast<size_t>(t0) * Hkv + h) * D + c * 8;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (t0 + i >= T) break;
      const float2 p = unpack2<false>(par[i]);   // a padding row: scale 0, all zeros
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = p.x * (static_cast<float>((w[i] >> (4 * j)) & 15u) + p.y);
      *reinterpret_cast<uint4*>(dst + static_cast<size_t>(i) * Hkv * D) = pack8<BF>(x);
    }
  }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

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
  if (static_cast<long long>(s->num_q_heads) + 2ll * s->num_kv_heads > (1ll << 30))
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
  a.Hq = q ? s->num_q_heads : 0;
  a.Hkv = s->num_kv_heads;
  a.bs = s->block_size;
  a.NB = s->num_blocks;
  a.rot = rope->rot_dim;
  a.inter = rope->interleaved != 0;
  a.max_pos = rope->max_position;
  const bool bf = s->dtype == PKV_BF16;
  void (*kern)(RopeArgs) = nullptr;
  if (D == 64) kern = bf ? rope_append_kernel<true, 64, KV4> : rope_append_kernel<false, 64, KV4>;
  if (D == 128) kern = bf ? rope_append_kernel<true, 128, KV4> : rope_append_kernel<false, 128, KV4>;
  if (D == 256) kern = bf ? rope_append_kernel<true, 256, KV4> : rope_append_kernel<false, 256, KV4>;
  const int rows = kThreads / (D / 8);
  const int passes = (a.Hq + 2 * a.Hkv + rows - 1) / rows;
  const dim3 grid(static_cast<unsigned>(num_tokens), static_cast<unsigned>(num_tokens < 1024 ? (passes < 65535 ? passes : 65535) : 1));
  cudaError_t e = launch_pdl(kern, grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream), a);
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
  const int D = s->head_dim, rows = kThreads / (D / 8);
  if (s->num_kv_heads > (1 << 29)) return PKV_ERR_UNSUPPORTED;
  const int tiles = (num_tokens - 1) / kTokens + 1, passes = (2 * s->num_kv_heads - 1) / rows + 1;
  // few tokens: the heads' passes on CTAs of their own
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(tiles < 1024 ? (passes < 65535 ? passes : 65535) : 1));
  int* err = device_error_word();
  if (!err) return PKV_ERR_CUDA;
  const bool bf = s->dtype == PKV_BF16;
  auto kern = kv4_gather_kernel<false, 64>;
  if (D == 64) kern = bf ? kv4_gather_kernel<true, 64> : kv4_gather_kernel<false, 64>;
  if (D == 128) kern = bf ? kv4_gather_kernel<true, 128> : kv4_gather_kernel<false, 128>;
  if (D == 256) kern = bf ? kv4_gather_kernel<true, 256> : kv4_gather_kernel<false, 256>;
  cudaError_t e = launch_pdl(kern, grid, kThreads, 0,
                             reinterpret_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(k_cache),
                             static_cast<const uint8_t*>(v_cache), slot_mapping,
                             static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), num_tokens,
                             s->num_kv_heads, s->block_size, s->num_blocks, err);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launch();
  return PKV_OK;
}
