// Paged single-token decode attention over the 4-bit cache
// (pkv_kv4_attn_decode, contract in include/pkv.h).
#include <cuda_fp16.h>

#include "pkv.h"
#include "pkv_internal.h"
#include "pkv_kv4.cuh"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

struct Kv4Args {
  DecodeArgs d;
  const uint8_t* k;
  const uint8_t* v;
  int bs;
};

// One warp per (sequence, query head): lane l owns channels [l * D/32, ...)
// and the warp walks the tokens one by one with a running maximum and sum.
template <bool BF, int D>
__global__ void __launch_bounds__(32) kv4_decode_kernel(const __grid_constant__ Kv4Args p) {
  constexpr int C = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const DecodeArgs& a = p.d;
  const int seq = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, lane = threadIdx.x;
  const int L = a.context_lens[seq];
  const size_t row = static_cast<size_t>(blockIdx.x) * D + lane * C;
  if (L < 0 || L > a.max_ctx) {
    if (lane == 0 && h == 0) record_error(a.err, kDevBadContext);
    return;
  }
  float q[C], o[C] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < C; i += 2) {
    const float2 f = unpack2<BF>(*reinterpret_cast<const uint32_t*>(a.q + row + i));
    q[i] = f.x * a.scale_log2;
    q[i + 1] = f.y * a.scale_log2;
  }
  const int g = lane * C / 32, ch = lane * C % 32;
  for (int t = 0; t < L; ++t) {
    const int blk = a.block_tables[static_cast<size_t>(seq) * a.MB + t / p.bs], r = t % p.bs;
    if (blk < 0 || blk >= a.NB) {
      if (lane == 0) record_error(a.err, kDevBadBlock);
      return;
    }
    const size_t tile = (static_cast<size_t>(blk) * a.Hkv + h / a.G) * kv4_tile_bytes(D, p.bs);
    const float2 kp = __half22float2(*reinterpret_cast<const __half2*>(p.k + tile + kv4_k_par_off<D>(p.bs, r, g)));
    const uint8_t* vp = p.v + tile + kv4_v_par_off<D>(p.bs, r, g);
    const float vs = __half2float(*reinterpret_cast<const __half*>(vp));
    const float vz = __half2float(*reinterpret_cast<const __half*>(vp + 4));
    const uint8_t* kc = p.k + tile + kv4_code_off<D>(r, g) + ch / 2;
    const uint8_t* vc = p.v + tile + kv4_code_off<D>(r, g) + ch / 2;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i)
      s = fmaf(q[i], kp.x * (static_cast<float>((kc[i / 2] >> (4 * (i & 1))) & 15) + kp.y), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), alpha = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * alpha + w;
#pragma unroll
    for (int i = 0; i < C; ++i)
      o[i] = fmaf(w, vs * (static_cast<float>((vc[i / 2] >> (4 * (i & 1))) & 15) + vz), o[i] * alpha);
  }
  const float inv = L > 0 ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < C; i += 2)
    *reinterpret_cast<uint32_t*>(a.out + row + i) = pack2<BF>(o[i] * inv, o[i + 1] * inv);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int kv4_plan(const pkv_shape* s, int sms, pkv_plan* plan) {
  if (s->kernel != 0) return PKV_ERR_UNSUPPORTED;
  *plan = pkv_plan{};
  plan->variant = 3;
  plan->split_tokens = s->max_context_len;
  plan->num_splits = 1;
  plan->warps_per_cta = 1;
  const long long grid = static_cast<long long>(s->num_seqs) * s->num_q_heads;
  if (grid > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  plan->grid_ctas = static_cast<int32_t>(grid);
  (void)sms;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_kv4_decode_plan(const pkv_shape* s, int32_t num_sms, pkv_plan* plan) {
  if (!s || !plan) return PKV_ERR_NULL;
  if (num_sms < 0) return PKV_ERR_INVALID;
  int rc = check_decode_shape(s);
  if (rc != PKV_OK) return rc;
  if (s->kernel != 0) return PKV_ERR_UNSUPPORTED;
  int sms = num_sms;
  if (sms == 0) {
    rc = device_sms(&sms);
    if (rc != PKV_OK) return rc;
  }
  return kv4_plan(s, sms, plan);
}

extern "C" int pkv_kv4_workspace_bytes(const pkv_shape* s, size_t* bytes) {
  if (!bytes) return PKV_ERR_NULL;
  pkv_plan plan{};
  const int rc = pkv_kv4_decode_plan(s, 0, &plan);
  if (rc == PKV_OK) *bytes = plan.workspace_bytes;
  return rc;
}

extern "C" int pkv_kv4_attn_decode(const pkv_shape* s, const void* q, const void* k_cache,
                                   const void* v_cache, const int32_t* block_tables,
                                   const int32_t* context_lens, float scale, void* out,
                                   void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  int rc = check_decode_shape(s);
  if (rc != PKV_OK) return rc;
  if (s->kernel != 0) return PKV_ERR_UNSUPPORTED;
  if (s->num_seqs == 0) return PKV_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out) return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4))
    return PKV_ERR_ALIGN;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc != PKV_OK) return rc;
  pkv_plan plan{};
  rc = kv4_plan(s, sms, &plan);
  if (rc != PKV_OK) return rc;
  if (plan.workspace_bytes > 0) {
    if (!workspace) {
      rc = device_workspace(&workspace, &workspace_bytes);
      if (rc != PKV_OK) return rc;
    }
    if (!workspace || workspace_bytes < plan.workspace_bytes || !aligned(workspace, 16))
      return PKV_ERR_WORKSPACE;
  }
  Kv4Args a{};
  a.d.q = static_cast<const uint16_t*>(q);
  a.d.block_tables = block_tables;
  a.d.context_lens = context_lens;
  a.d.out = static_cast<uint16_t*>(out);
  a.d.err = device_error_word();
  a.d.B = s->num_seqs;
  a.d.Hq = s->num_q_heads;
  a.d.Hkv = s->num_kv_heads;
  a.d.G = s->num_q_heads / s->num_kv_heads;
  a.d.MB = s->max_blocks_per_seq;
  a.d.NB = s->num_blocks;
  a.d.S = plan.num_splits;
  a.d.P = plan.split_tokens;
  a.d.max_ctx = s->max_context_len;
  a.d.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
  a.k = static_cast<const uint8_t*>(k_cache);
  a.v = static_cast<const uint8_t*>(v_cache);
  a.bs = s->block_size;
  const bool bf = s->dtype == PKV_BF16;
  const int D = s->head_dim;
  void (*kern)(Kv4Args) = nullptr;
  if (D == 64) kern = bf ? kv4_decode_kernel<true, 64> : kv4_decode_kernel<false, 64>;
  if (D == 128) kern = bf ? kv4_decode_kernel<true, 128> : kv4_decode_kernel<false, 128>;
  if (D == 256) kern = bf ? kv4_decode_kernel<true, 256> : kv4_decode_kernel<false, 256>;
  if (launch_pdl(kern, dim3(static_cast<unsigned>(plan.grid_ctas)), 32, 0,
                 reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
    return PKV_ERR_CUDA;
  count_launch();
  return PKV_OK;
}
