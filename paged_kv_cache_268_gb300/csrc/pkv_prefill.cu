// Prompt-side attention: a chunk of new tokens over the paged cache
// (pkv_paged_attn_chunk) and packed prompts (pkv_prompt_attn).  Contracts in
// include/pkv.h.
#include <cmath>

#include "pkv.h"
#include "pkv_prefill.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kReduceThreads = 256;

// Joins the partitions of the sequences that were cut: a warp a (token, query
// head) row, out = sum_p 2^(e_p - E) o_p / sum_p 2^(e_p - E) l_p with E the
// largest exponent, in the partitions' order.
template <bool BF, int D>
__global__ void __launch_bounds__(kReduceThreads) prefill_reduce_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int C = D / 32, BN = prefill_key_tile(D);
  pdl_wait();
  pdl_launch_dependents();
  if (a.plan[a.B].parts == 0) return;
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kReduceThreads / 32);
  const long long rows = static_cast<long long>(a.T) * a.Hq;
  for (long long row = blockIdx.x * (kReduceThreads / 32) + (threadIdx.x >> 5); row < rows; row += warps) {
    const int t = static_cast<int>(row / a.Hq);
    int lo = 0, hi = a.B;                    // the last sequence that starts at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.query_starts[mid] <= t) lo = mid; else hi = mid;
    }
    const PrefillPlan plan = a.plan[lo];
    const int q0 = a.query_starts[lo], q1 = a.query_starts[lo + 1];
    if (plan.parts < 2 || t < q0 || t >= q1) continue;
    const int L = a.key_starts != nullptr ? a.key_starts[lo + 1] - a.key_starts[lo] : a.context_lens[lo];
    const int lim = a.causal ? L - (q1 - t) : L - 1;           // last key that the row sees
    const int parts = lim < 0 ? 0 : min(plan.parts, lim / (plan.per * BN) + 1);
    const size_t from = static_cast<size_t>(plan.row) + (row - static_cast<long long>(q0) * a.Hq) * plan.parts;
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.part_ml[from + p].x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    float o[C] = {}, l = 0.f;
    for (int p = 0; p < parts; ++p) {
      const float2 ml = a.part_ml[from + p];
      if (ml.y == 0.f) continue;
      const float w = fast_exp2(ml.x - top);
      l = fmaf(w, ml.y, l);
      const float2* src = reinterpret_cast<const float2*>(a.part_o + (from + p) * D + lane * C);
#pragma unroll
      for (int c = 0; c < C / 2; ++c) {
        const float2 x = src[c];
        o[2 * c] = fmaf(w, x.x, o[2 * c]);
        o[2 * c + 1] = fmaf(w, x.y, o[2 * c + 1]);
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + lane * C);
#pragma unroll
    for (int c = 0; c < C / 2; ++c) dst[c] = pack2<BF>(o[2 * c] * inv, o[2 * c + 1] * inv);
  }
}

template <bool BF>
cudaError_t launch_reduce(const PrefillArgs& a, int D, unsigned grid, cudaStream_t stream) {
  auto kern = prefill_reduce_kernel<BF, 64>;
  if (D == 128) kern = prefill_reduce_kernel<BF, 128>;
  if (D == 256) kern = prefill_reduce_kernel<BF, 256>;
  return launch_pdl(kern, dim3(grid), kReduceThreads, 0, stream, a);
}

// Sizes of a call: whether sequences may be cut, the workspace for that, the grid.
struct CallSizes {
  int part_tiles;                // of a forced partition, else 0
  long long rows;                // partial rows at most
  size_t plan_bytes, bytes;
  unsigned grid;
};

CallSizes call_sizes(int B, int T, int Hq, int Hkv, int D, int max_keys, int split_tokens, int sms) {
  CallSizes c{};
  const int BN = prefill_key_tile(D), G = Hq / Hkv;
  const int per_item = 128 / G * prefill_row_tiles(D);
  c.part_tiles = (split_tokens + BN - 1) / BN;
  const long long smallest = c.part_tiles ? static_cast<long long>(c.part_tiles) * BN : kPrefillMinPart;
  const long long parts = (max_keys + smallest - 1) / smallest;    // of one sequence at most
  if (parts > 1) {
    c.rows = static_cast<long long>(T) * Hq * parts;
    if (!c.part_tiles) {
      // A sequence that is cut has at most twice the partitions that its key
      // tiles are units (prefill_parts), and the units of all are a few a CTA.
      const long long few = 2ll * kPrefillFewUnits * sms * kPrefillFewRows;
      const long long many = 2ll * kPrefillUnits * sms * 128 * prefill_row_tiles(D);
      if (c.rows > few + many) c.rows = few + many;
    }
    static_assert(sizeof(PrefillPlan) == 16, "what follows the plan is aligned");
    c.plan_bytes = (static_cast<size_t>(B) + 1) * sizeof(PrefillPlan);
    c.bytes = c.plan_bytes + static_cast<size_t>(c.rows) * (D * 4 + 8);
  }
  // every sequence's last item may be a small one
  const long long items = (static_cast<long long>(T) / per_item + B) * Hkv * (parts > 1 ? parts : 1);
  c.grid = static_cast<unsigned>(items < sms ? (items < 1 ? 1 : items) : sms);
  return c;
}

int launch(PrefillArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, bool bf, int D,
           float scale, int split_tokens, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  int sms = 0;
  int rc = device_sms(&sms);
  if (rc != PKV_OK) return rc;
  const CallSizes c = call_sizes(a.B, a.T, a.Hq, a.Hkv, D, a.max_keys, split_tokens, sms);
  if (c.bytes > 0) {
    if (!workspace) {
      rc = device_workspace(&workspace, &workspace_bytes);
      if (rc != PKV_OK) return rc;
    }
    if (!workspace || workspace_bytes < c.bytes || !aligned(workspace, 16)) return PKV_ERR_WORKSPACE;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    a.plan = reinterpret_cast<PrefillPlan*>(w);
    a.part_o = reinterpret_cast<float*>(w + c.plan_bytes);
    a.part_ml = reinterpret_cast<float2*>(w + c.plan_bytes + static_cast<size_t>(c.rows) * D * 4);
  }
  a.err = device_error_word();
  if (!a.err) return PKV_ERR_CUDA;
  a.part_tiles = c.part_tiles;
  a.ctas = sms;
  a.negative = scale < 0.f;
  // (a factor of zero would turn a hidden key's minus infinity into no number)
  a.scale_log2 = fmaxf(fabsf(scale) * 1.4426950408889634f, 0x1p-126f);
  cudaError_t e = bf ? launch_prefill_bf16(a, q, k, v, D, c.grid, stream)
                     : launch_prefill_f16(a, q, k, v, D, c.grid, stream);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launch();
  if (c.bytes > 0) {
    const long long rows = static_cast<long long>(a.T) * a.Hq, ctas = (rows + kReduceThreads / 32 - 1) / (kReduceThreads / 32);
    const unsigned grid = static_cast<unsigned>(ctas < 4ll * sms ? ctas : 4ll * sms);
    e = bf ? launch_reduce<true>(a, D, grid, stream) : launch_reduce<false>(a, D, grid, stream);
    if (e != cudaSuccess) return PKV_ERR_CUDA;
    count_launch();
  }
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
  int rc = check_chunk(s, 0, num_tokens);
  if (rc != PKV_OK) return rc;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc != PKV_OK) return rc;
  *bytes = call_sizes(s->num_seqs, num_tokens, s->num_q_heads, s->num_kv_heads, s->head_dim,
                      s->max_context_len, s->split_tokens, sms).bytes;
  return PKV_OK;
}

extern "C" int pkv_prompt_workspace_bytes(const pkv_prompt* p, size_t* bytes) {
  if (!bytes) return PKV_ERR_NULL;
  int rc = check_prompt(p);
  if (rc != PKV_OK) return rc;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc != PKV_OK) return rc;
  *bytes = call_sizes(p->num_seqs, p->num_tokens, p->num_q_heads, p->num_kv_heads, p->head_dim,
                      p->num_keys, p->split_tokens, sms).bytes;
  return PKV_OK;
}

extern "C" int pkv_paged_attn_chunk(const pkv_shape* s, const void* q, int64_t q_stride,
                                    int32_t num_tokens, const int32_t* query_starts,
                                    const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, const int32_t* context_lens,
                                    float scale, void* out, void* workspace, size_t workspace_bytes,
                                    pkv_stream_t stream) {
  int rc = check_chunk(s, q_stride, num_tokens);
  if (rc != PKV_OK) return rc;
  if (s->num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!q || !query_starts || !k_cache || !v_cache || !block_tables || !context_lens || !out)
    return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(query_starts, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) || q_stride % 8)
    return PKV_ERR_ALIGN;
  const bool bf = s->dtype == PKV_BF16;
  const int D = s->head_dim, G = s->num_q_heads / s->num_kv_heads;
  CUtensorMap tq, tk, tv;
  rc = rows_map(&tq, q, bf, D, s->num_q_heads, num_tokens,
                q_stride ? q_stride : static_cast<int64_t>(s->num_q_heads) * D, G, 128 / G);
  if (rc == PKV_OK) rc = block_map(&tk, k_cache, *s);
  if (rc == PKV_OK) rc = block_map(&tv, v_cache, *s);
  if (rc != PKV_OK) return rc;
  PrefillArgs a{};
  a.query_starts = query_starts;
  a.context_lens = context_lens;
  a.block_tables = block_tables;
  a.v = static_cast<const uint16_t*>(v_cache);
  a.out = static_cast<uint16_t*>(out);
  a.B = s->num_seqs;
  a.T = num_tokens;
  a.Hq = s->num_q_heads;
  a.Hkv = s->num_kv_heads;
  a.G = G;
  a.max_keys = s->max_context_len;
  a.MB = s->max_blocks_per_seq;
  a.NB = s->num_blocks;
  a.bs_log2 = s->block_size == 32 ? 5 : 4;
  a.causal = 1;
  return launch(a, tq, tk, tv, bf, D, scale, s->split_tokens, workspace, workspace_bytes,
                reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int pkv_prompt_attn(const pkv_prompt* p, const void* q, const void* k, const void* v,
                               const int32_t* query_starts, const int32_t* key_starts, float scale,
                               void* out, void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  int rc = check_prompt(p);
  if (rc != PKV_OK) return rc;
  if (p->num_seqs == 0 || p->num_tokens == 0) return PKV_OK;
  if (!q || !query_starts || !key_starts || !out || (p->num_keys > 0 && (!k || !v))) return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(query_starts, 4) || !aligned(key_starts, 4) || p->q_stride % 8 || p->k_stride % 8 ||
      p->v_stride % 8)
    return PKV_ERR_ALIGN;
  const bool bf = p->dtype == PKV_BF16;
  const int D = p->head_dim, G = p->num_q_heads / p->num_kv_heads, BN = prefill_key_tile(D);
  const int64_t kd = static_cast<int64_t>(p->num_kv_heads) * D;
  const int64_t ks = p->k_stride ? p->k_stride : kd, vs = p->v_stride ? p->v_stride : kd;
  CUtensorMap tq, tk, tv;
  rc = rows_map(&tq, q, bf, D, p->num_q_heads, p->num_tokens,
                p->q_stride ? p->q_stride : static_cast<int64_t>(p->num_q_heads) * D, G, 128 / G);
  if (rc != PKV_OK) return rc;
  tk = tv = tq;                            // (without keys none is loaded)
  if (p->num_keys > 0) {
    rc = rows_map(&tk, k, bf, D, p->num_kv_heads, p->num_keys, ks, 1, BN);
    if (rc == PKV_OK) rc = rows_map(&tv, v, bf, D, p->num_kv_heads, p->num_keys, vs, 1, BN);
    if (rc != PKV_OK) return rc;
  }
  PrefillArgs a{};
  a.query_starts = query_starts;
  a.key_starts = key_starts;
  a.v = static_cast<const uint16_t*>(v);
  a.v_stride = vs;
  a.out = static_cast<uint16_t*>(out);
  a.B = p->num_seqs;
  a.T = p->num_tokens;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = G;
  a.max_keys = p->num_keys;
  a.causal = p->causal != 0;
  return launch(a, tq, tk, tv, bf, D, scale, p->split_tokens, workspace, workspace_bytes,
                reinterpret_cast<cudaStream_t>(stream));
}
