// Prompt-side attention: a chunk of new tokens over the paged cache
// (pkv_paged_attn_chunk) and packed prompts (pkv_prompt_attn).  Contracts in
// include/pkv.h.
#include "pkv.h"
#include "pkv_prefill.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

// One warp a (token, query head) row: softmax(q . K^T scale) . V key by key,
// with the running maximum and sum; a lane holds D / 32 channels.
template <bool BF, int D>
__global__ void __launch_bounds__(256) prefill_rows_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(a.T) * a.Hq) return;
  const int t = static_cast<int>(row / a.Hq), h = static_cast<int>(row % a.Hq), kvh = h / a.G;
  int lo = 0, hi = a.B;                    // the last sequence that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.query_starts[mid] <= t) lo = mid; else hi = mid;
  }
  int q0, n, k0, L, code;
  if (!prefill_seq(a, lo, q0, n, k0, L, code)) {
    if (lane == 0) record_error(a.err, code);
    return;
  }
  if (t < q0 || t >= q0 + n) return;
  const int end = a.causal ? min(L, L - n + (t - q0) + 1) : L;
  float q[C], o[C] = {};
  for (int c = 0; c < C; c += 2) {
    const float2 x = unpack2<BF>(*reinterpret_cast<const uint32_t*>(a.q + t * a.q_stride + static_cast<long long>(h) * D + lane * C + c));
    q[c] = x.x;
    q[c + 1] = x.y;
  }
  float m = -INFINITY, l = 0.f;
  for (int s = 0; s < end; ++s) {
    const uint16_t *k, *v;
    if (a.key_starts != nullptr) {
      k = a.k + (k0 + s) * a.k_stride + static_cast<long long>(kvh) * D;
      v = a.v + (k0 + s) * a.v_stride + static_cast<long long>(kvh) * D;
    } else {
      const int block = a.block_tables[static_cast<size_t>(lo) * a.MB + (s >> a.bs_log2)];
      if (block < 0 || block >= a.NB) {
        if (lane == 0) record_error(a.err, kDevBadBlock);
        continue;
      }
      const size_t at = (((static_cast<size_t>(block) * a.Hkv + kvh) << a.bs_log2) + (s & ((1 << a.bs_log2) - 1))) * D;
      k = a.k + at;
      v = a.v + at;
    }
    float x = 0.f;
    for (int c = 0; c < C; c += 2) {
      const float2 y = unpack2<BF>(*reinterpret_cast<const uint32_t*>(k + lane * C + c));
      x = fmaf(q[c], y.x, fmaf(q[c + 1], y.y, x));
    }
    for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
    x *= a.scale;
    const float top = fmaxf(m, x), keep = m == top ? 1.f : expf(m - top), p = expf(x - top);
    m = top;
    l = l * keep + p;
    for (int c = 0; c < C; c += 2) {
      const float2 y = unpack2<BF>(*reinterpret_cast<const uint32_t*>(v + lane * C + c));
      o[c] = fmaf(o[c], keep, p * y.x);
      o[c + 1] = fmaf(o[c + 1], keep, p * y.y);
    }
  }
  for (int c = 0; c < C; c += 2) {
    const float y0 = end > 0 ? o[c] / l : 0.f, y1 = end > 0 ? o[c + 1] / l : 0.f;
    *reinterpret_cast<uint32_t*>(a.out + row * D + lane * C + c) = pack2<BF>(y0, y1);
  }
}

int launch(const PrefillArgs& a, bool bf, int D, cudaStream_t stream) {
  const long long grid = (static_cast<long long>(a.T) * a.Hq + 7) / 8;
  if (grid > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  void (*kern)(PrefillArgs) = nullptr;
  if (D == 64) kern = bf ? prefill_rows_kernel<true, 64> : prefill_rows_kernel<false, 64>;
  if (D == 128) kern = bf ? prefill_rows_kernel<true, 128> : prefill_rows_kernel<false, 128>;
  if (D == 256) kern = bf ? prefill_rows_kernel<true, 256> : prefill_rows_kernel<false, 256>;
  kern<<<static_cast<unsigned>(grid), 256, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  count_launch();
  return PKV_OK;
}

// What both entry points check of a batch's sizes.
int check_sizes(int64_t q_stride, int D, int Hq, int num_tokens) {
  if (num_tokens < 0 || (q_stride != 0 && q_stride < static_cast<int64_t>(Hq) * D)) return PKV_ERR_INVALID;
  if (num_tokens > (1 << 30)) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

int check_prompt(const pkv_prompt* p) {
  if (!p) return PKV_ERR_NULL;
  if (p->num_seqs < 0 || p->num_q_heads < 1 || p->num_kv_heads < 1 || p->num_keys < 0 ||
      p->split_tokens < 0 || p->num_q_heads % p->num_kv_heads != 0)
    return PKV_ERR_INVALID;
  if (p->dtype != PKV_F16 && p->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return PKV_ERR_UNSUPPORTED;
  if (p->num_q_heads / p->num_kv_heads > 32 || p->num_keys > (1 << 30)) return PKV_ERR_UNSUPPORTED;
  const int64_t kd = static_cast<int64_t>(p->num_kv_heads) * p->head_dim;
  if ((p->k_stride != 0 && p->k_stride < kd) || (p->v_stride != 0 && p->v_stride < kd)) return PKV_ERR_INVALID;
  return check_sizes(p->q_stride, p->head_dim, p->num_q_heads, p->num_tokens);
}

int check_chunk(const pkv_shape* s, int64_t q_stride, int num_tokens) {
  const int rc = check_decode_shape(s);
  if (rc != PKV_OK) return rc;
  if (s->kernel != 0) return PKV_ERR_UNSUPPORTED;
  return check_sizes(q_stride, s->head_dim, s->num_q_heads, num_tokens);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_chunk_workspace_bytes(const pkv_shape* s, int32_t num_tokens, size_t* bytes) {
  if (!bytes) return PKV_ERR_NULL;
  const int rc = check_chunk(s, 0, num_tokens);
  if (rc != PKV_OK) return rc;
  *bytes = 0;
  return PKV_OK;
}

extern "C" int pkv_prompt_workspace_bytes(const pkv_prompt* p, size_t* bytes) {
  if (!bytes) return PKV_ERR_NULL;
  const int rc = check_prompt(p);
  if (rc != PKV_OK) return rc;
  *bytes = 0;
  return PKV_OK;
}

extern "C" int pkv_paged_attn_chunk(const pkv_shape* s, const void* q, int64_t q_stride,
                                    int32_t num_tokens, const int32_t* query_starts,
                                    const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, const int32_t* context_lens,
                                    float scale, void* out, void* workspace, size_t workspace_bytes,
                                    pkv_stream_t stream) {
  const int rc = check_chunk(s, q_stride, num_tokens);
  if (rc != PKV_OK) return rc;
  if (s->num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!q || !query_starts || !k_cache || !v_cache || !block_tables || !context_lens || !out)
    return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(query_starts, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) || q_stride % 8)
    return PKV_ERR_ALIGN;
  PrefillArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k_cache);
  a.v = static_cast<const uint16_t*>(v_cache);
  a.query_starts = query_starts;
  a.context_lens = context_lens;
  a.block_tables = block_tables;
  a.out = static_cast<uint16_t*>(out);
  a.err = device_error_word();
  if (!a.err) return PKV_ERR_CUDA;
  a.q_stride = q_stride ? q_stride : static_cast<long long>(s->num_q_heads) * s->head_dim;
  a.B = s->num_seqs;
  a.T = num_tokens;
  a.Hq = s->num_q_heads;
  a.Hkv = s->num_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.max_keys = s->max_context_len;
  a.MB = s->max_blocks_per_seq;
  a.NB = s->num_blocks;
  a.bs_log2 = s->block_size == 32 ? 5 : 4;
  a.causal = 1;
  a.scale = scale;
  return launch(a, s->dtype == PKV_BF16, s->head_dim, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int pkv_prompt_attn(const pkv_prompt* p, const void* q, const void* k, const void* v,
                               const int32_t* query_starts, const int32_t* key_starts, float scale,
                               void* out, void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  const int rc = check_prompt(p);
  if (rc != PKV_OK) return rc;
  if (p->num_seqs == 0 || p->num_tokens == 0) return PKV_OK;
  if (!q || !query_starts || !key_starts || !out || (p->num_keys > 0 && (!k || !v))) return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(query_starts, 4) || !aligned(key_starts, 4) || p->q_stride % 8 || p->k_stride % 8 ||
      p->v_stride % 8)
    return PKV_ERR_ALIGN;
  PrefillArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.query_starts = query_starts;
  a.key_starts = key_starts;
  a.out = static_cast<uint16_t*>(out);
  a.err = device_error_word();
  if (!a.err) return PKV_ERR_CUDA;
  const long long kd = static_cast<long long>(p->num_kv_heads) * p->head_dim;
  a.q_stride = p->q_stride ? p->q_stride : static_cast<long long>(p->num_q_heads) * p->head_dim;
  a.k_stride = p->k_stride ? p->k_stride : kd;
  a.v_stride = p->v_stride ? p->v_stride : kd;
  a.B = p->num_seqs;
  a.T = p->num_tokens;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.max_keys = p->num_keys;
  a.causal = p->causal != 0;
  a.scale = scale;
  return launch(a, p->dtype == PKV_BF16, p->head_dim, reinterpret_cast<cudaStream_t>(stream));
}
