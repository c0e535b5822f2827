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
constexpr int kReduceRows = 2;                        // of a warp, at once (one or four: 1-2% of a call more)
constexpr int kReduceCtaRows = kReduceThreads / 32 * kReduceRows;

// Joins the pieces of the items that were cut: out = sum_p 2^((m_p - M) c) o_p /
// sum_p 2^((m_p - M) c) l_p with M the largest reference, in the keys' order.  CTA
// (c, y) looks after the item whose second piece attention's CTA c had, if it
// had one, rows 16 y and up.  Bound by the latency of its few loads, so each step
// asks for all that it needs at once: the CTAs behind c, a lane each; the pieces'
// references and sums, a lane each, of two rows; these rows' outputs.
template <bool BF, int D>
__global__ void __launch_bounds__(kReduceThreads) prefill_reduce_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int C = D / 32, R = kReduceRows;
  pdl_wait();
  pdl_launch_dependents();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const PrefillCut cut = a.cuts[c0];
  const int rows = cut.ntok * a.G, row0 = blockIdx.y * kReduceCtaRows + (threadIdx.x >> 5) * R;
  if (cut.kind != 2 || row0 >= rows) return;
  float o[R][C] = {}, l[R] = {}, top[R];
#pragma unroll
  for (int r = 0; r < R; ++r) top[r] = -INFINITY;
  // 31 CTAs from c0 up at a time, and before the first of them the item's first piece
  bool more = true;
  for (int c = c0 - 1; more; c += 31) {
    const int mine = lane == 0 ? cut.first : c + lane;      // the CTA of the lane's piece
    int kind = 0, ends = 0;
    if (lane > 0 && mine < static_cast<int>(gridDim.x)) {
      kind = a.cuts[mine].kind;
      ends = a.cuts[mine].ends;
    }
    const uint32_t last = __ballot_sync(0xffffffffu, kind != 0 && ends);
    more = last == 0 && c + 32 < static_cast<int>(gridDim.x);
    const int until = last ? __ffs(last) - 1 : 31;          // the last lane with a piece of the item
    const bool have = lane == 0 ? c == c0 - 1 : kind != 0 && lane <= until;
    const size_t at = static_cast<size_t>(lane == 0 ? 2 * mine + 1 : 2 * mine) * a.rows + row0;
    float2 ml[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      ml[r] = have && row0 + r < rows ? a.part_ml[at + r] : make_float2(-INFINITY, 0.f);
    float w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float up = ml[r].y != 0.f ? fmaxf(top[r], ml[r].x) : top[r];
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, i));
      const float keep = top[r] == -INFINITY ? 0.f : fast_exp2((top[r] - up) * a.scale_log2);
      w[r] = ml[r].y != 0.f ? fast_exp2((ml[r].x - up) * a.scale_log2) : 0.f;
      float sum = w[r] * ml[r].y;
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
      l[r] = fmaf(l[r], keep, sum);
      top[r] = up;
#pragma unroll
      for (int e = 0; e < C; ++e) o[r][e] *= keep;
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, have); todo != 0; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const size_t src = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(at), from);
      float2 x[R][C / 2];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2* p = reinterpret_cast<const float2*>(a.part_o + (src + r) * D + lane * C);
#pragma unroll
        for (int e = 0; e < C / 2; ++e) x[r][e] = row0 + r < rows ? p[e] : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float wt = __shfl_sync(0xffffffffu, w[r], from);
        if (__shfl_sync(0xffffffffu, ml[r].y, from) == 0.f) continue;   // sees none of its keys
#pragma unroll
        for (int e = 0; e < C / 2; ++e) {
          o[r][2 * e] = fmaf(wt, x[r][e].x, o[r][2 * e]);
          o[r][2 * e + 1] = fmaf(wt, x[r][e].y, o[r][2 * e + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + r;
    if (row >= rows) return;
    const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
    const size_t out = static_cast<size_t>(cut.q_row + row / a.G) * a.Hq + cut.kvh * a.G + row % a.G;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + out * D + lane * C);
#pragma unroll
    for (int e = 0; e < C / 2; ++e) dst[e] = pack2<BF>(o[r][2 * e] * inv, o[r][2 * e + 1] * inv);
  }
}

template <bool BF>
cudaError_t launch_reduce(const PrefillArgs& a, int D, unsigned ctas, cudaStream_t stream) {
  auto kern = prefill_reduce_kernel<BF, 64>;
  if (D == 128) kern = prefill_reduce_kernel<BF, 128>;
  if (D == 256) kern = prefill_reduce_kernel<BF, 256>;
  return launch_pdl(kern, dim3(ctas, (a.rows + kReduceCtaRows - 1) / kReduceCtaRows), kReduceThreads, 0, stream, a);
}

// Sizes of a call: the grid, and the workspace where items may be cut.
struct CallSizes {
  int min_part;                  // key tiles of an item's first and last pieces at least
  int rows;                      // of an item at most
  size_t cut_bytes, bytes;
  unsigned grid;
  int small;                     // PrefillArgs
};

// The largest smallest part that split_tokens may ask for.  (A CTA's share may be
// more; what bounds an item's time is a sequence's length, kPrefillMostKeys.)
constexpr int kMostPart = 1 << 20;

CallSizes call_sizes(int B, int T, int Hq, int Hkv, int D, int max_keys, int split_tokens, int sms) {
  CallSizes c{};
  const int BN = prefill_key_tile(D), G = Hq / Hkv;
  const int per_item = 128 / G * prefill_row_tiles(D);
  const int part = split_tokens > 0 ? (split_tokens < kMostPart ? split_tokens : kMostPart) : kPrefillMinPart;
  c.min_part = (part - 1) / BN + 1;
  c.rows = (T < per_item ? T : per_item) * G;
  const int tiles = max_keys > 0 ? (max_keys - 1) / BN + 1 : 1;
  const bool cuts = tiles >= 2ll * c.min_part;
  // every sequence's last item may be a small one
  const long long items = (static_cast<long long>(T) / per_item + B) * Hkv;
  const long long pieces = items * (cuts ? tiles / c.min_part : 1);
  c.grid = static_cast<unsigned>(pieces < sms ? pieces : sms);
  const double longest = static_cast<double>(max_keys) * kPrefillKeyCost + kPrefillItemCost +
                         static_cast<double>(per_item) * kPrefillTokenCost;
  c.small = T / per_item < kPrefillSmallItems && max_keys <= kPrefillMostKeys &&
            static_cast<double>(items) * longest < 2147483648.0;
  if (cuts && c.grid > 1) {
    c.cut_bytes = (c.grid * sizeof(PrefillCut) + 31) / 32 * 32;
    c.bytes = 16 + c.cut_bytes + 2ull * c.grid * c.rows * (D * 4 + 8);   // 16: to a 32-byte boundary
  }
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
    uint8_t* w = static_cast<uint8_t*>(workspace) + (reinterpret_cast<uintptr_t>(workspace) & 16);
    a.cuts = reinterpret_cast<PrefillCut*>(w);
    a.part_o = reinterpret_cast<float*>(w + c.cut_bytes);
    a.part_ml = reinterpret_cast<float2*>(w + c.cut_bytes + 2ull * c.grid * c.rows * D * 4);
  }
  a.err = device_error_word();
  if (!a.err) return PKV_ERR_CUDA;
  a.rows = c.rows;
  a.min_part = c.min_part;
  a.small = c.small;
  a.negative = scale < 0.f;
  // (a factor of zero would turn a hidden key's minus infinity into no number)
  a.scale_log2 = fabsf(scale) * 1.4426950408889634f;
  if (a.scale_log2 < 0x1p-126f) a.scale_log2 = 0x1p-126f;
  cudaError_t e = bf ? launch_prefill_bf16(a, q, k, v, D, c.grid, stream)
                     : launch_prefill_f16(a, q, k, v, D, c.grid, stream);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launch();
  if (c.bytes > 0) {
    e = bf ? launch_reduce<true>(a, D, c.grid, stream) : launch_reduce<false>(a, D, c.grid, stream);
    if (e != cudaSuccess) return PKV_ERR_CUDA;
    count_launch();
  }
  return PKV_OK;
}

// A token stride (0: dense) of rows of `row` elements.
int check_stride(int64_t stride, int64_t row) {
  if (stride != 0 && stride < row) return PKV_ERR_INVALID;
  // what a tensor map holds, in bytes
  return stride >= (1ll << 39) ? PKV_ERR_UNSUPPORTED : PKV_OK;
}

// Rows and keys are counted in 32 bits, with room for the tiles' ends.
constexpr int kMostRows = 1 << 30;
// Every CTA looks at all sequences before its first load: 32 of them in about half
// a microsecond, a quarter of a second for so many.
constexpr int kMostSeqs = 1 << 24;

int check_prompt(const pkv_prompt* p) {
  if (!p) return PKV_ERR_NULL;
  if (p->num_seqs < 0 || p->num_q_heads < 1 || p->num_kv_heads < 1 || p->num_tokens < 0 ||
      p->num_keys < 0 || p->split_tokens < 0 || p->num_q_heads % p->num_kv_heads != 0)
    return PKV_ERR_INVALID;
  if (p->dtype != PKV_F16 && p->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return PKV_ERR_UNSUPPORTED;
  if (p->num_q_heads / p->num_kv_heads > 32 || p->num_tokens > kMostRows || p->num_keys > kMostRows ||
      p->num_seqs > kMostSeqs)
    return PKV_ERR_UNSUPPORTED;
  const int64_t kd = static_cast<int64_t>(p->num_kv_heads) * p->head_dim;
  int rc = check_stride(p->q_stride, static_cast<int64_t>(p->num_q_heads) * p->head_dim);
  if (rc == PKV_OK) rc = check_stride(p->k_stride, kd);
  return rc == PKV_OK ? check_stride(p->v_stride, kd) : rc;
}

int check_chunk(const pkv_shape* s, int64_t q_stride, int num_tokens) {
  const int rc = check_decode_shape(s);
  if (rc != PKV_OK) return rc;
  if (num_tokens < 0) return PKV_ERR_INVALID;
  if (s->kernel != 0 || num_tokens > kMostRows || s->max_context_len > kMostRows ||
      s->num_seqs > kMostSeqs)
    return PKV_ERR_UNSUPPORTED;
  return check_stride(q_stride, static_cast<int64_t>(s->num_q_heads) * s->head_dim);
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
  if (rc == PKV_OK) rc = block_map(&tk, k_cache, *s, false);
  if (rc == PKV_OK) rc = block_map(&tv, v_cache, *s, true);
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
