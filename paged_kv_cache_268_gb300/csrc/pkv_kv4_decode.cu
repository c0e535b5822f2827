// Paged single-token decode attention over the 4-bit cache
// (pkv_kv4_attn_decode, contract in include/pkv.h).
#include "pkv_kv4_decode.cuh"

namespace pkv {
namespace {

// CTAs that share the query heads of one kv head.
int kv4_chunks(const pkv_shape* s) {
  const int G = s->num_q_heads / s->num_kv_heads;
  const int heads = kv4_columns(s->head_dim, G) * kv4_tiles(s->head_dim, G);
  return (G + heads - 1) / heads;
}

// The sequences that are dispatched last and their partitions (Kv4Args).
struct Late {
  int first, P, S;
};

int kv4_plan(const pkv_shape* s, int sms, pkv_plan* plan, Late* late) {
  const int D = s->head_dim, bs = s->block_size;
  const int G = s->num_q_heads / s->num_kv_heads;
  *plan = pkv_plan{};
  plan->variant = 3;
  plan->warps_per_cta = kKv4Warps;
  plan->stages_per_warp = kv4_stages(D);
  const long long units =
      static_cast<long long>(s->num_seqs) * s->num_kv_heads * kv4_chunks(s);
  const int maxL = s->max_context_len;
  const int gran = kKv4Warps * kKv4Tokens;
  const int cap = kMaxBlocksPerCta * bs;
  long long P;
  if (s->split_tokens > 0) {
    P = (static_cast<long long>(s->split_tokens) + bs - 1) / bs * bs;
  } else {
    // Tokens per resident CTA if every sequence were of the largest length
    // (max_context_len, all that the host knows: a bound far above the lengths
    // costs empty CTAs and partitions of another size; 128 log-normal lengths
    // of up to 8192 56 us, 70 under a bound of 32768, 129 under 131072).
    // Measured on one GB300 over batches of 1 to 128 sequences (uniform and
    // log-normal lengths, 8 and 32 kv heads, head_dim 64 to 256), one size for
    // all sequences, before the last of them were cut finer (below):
    //  - from 6000 on, 2048-token partitions (64 x 512-4096 tokens, 32 heads:
    //    123 us, 126 at 1024), from 1000 on, 1024 (64 x 1-4096, 8 heads: 40 us,
    //    43 at 2048 or 512), below, half of it;
    //  - up to four sequences, whose lengths are mostly near the largest: one
    //    wave of equal partitions (4 x 32768 tokens: 36 us, 42-45 at 768-2048).
    //    Where that ends is not measured: 5 x 32768 tokens take 52 us, 8 take 75
    //    (floors 31 and 50);
    //  - at least 256 tokens, 128 where a sequence has at most 2048, since
    //    start-up and merge cost a CTA as much as about that many (1 x 8192: 8.1
    //    us at 256, 10.4 at 128; 1 x 500: 5.2 us at 128, 6.2 at 256); no split of
    //    up to 256 tokens (4.2 us, 4.5 in two).
    const long long slots =
        static_cast<long long>(sms) * kv4_ctas(D, kv4_columns(D, G), kv4_tiles(D, G));
    const long long per_slot = units * maxL / slots;
    P = per_slot >= 6000 ? 2048 : (per_slot >= 1000 ? 1024 : per_slot / 2);
    if (s->num_seqs <= 4 && units > 0 && units < slots) {
      const long long S = slots / units;
      P = (maxL + S - 1) / S;
    }
    const long long least = maxL <= 256 ? 256 : (maxL <= 2048 ? 128 : 256);
    if (P < least) P = least;
    P = (P + gran - 1) / gran * gran;
    // at most 1024 partitions per sequence
    const long long pmin = (static_cast<long long>(maxL) + 1023) / 1024;
    if (P < pmin) P = (pmin + gran - 1) / gran * gran;
  }
  if (P > cap) P = cap;
  if (P > maxL) P = (maxL + bs - 1) / bs * bs;
  if (P < bs) P = bs;
  const int S = static_cast<int>((maxL + P - 1) / P);
  plan->split_tokens = static_cast<int32_t>(P);
  plan->num_splits = S;
  *late = Late{s->num_seqs, static_cast<int>(P), S};
  if (s->split_tokens == 0 && P >= 1024 && s->num_seqs > 4) {
    // The CTAs that are dispatched last end at different times, and nothing is
    // left for the SMs that finish first: an eighth of the sequences is cut
    // finer, which evens the ends out.  Measured against one size for all:
    // 128 log-normal lengths, 8 kv heads, 55.9 us (61.6), 256 x 1-2048 69.4
    // (71.5), 64 x 512-4096 with 32 heads 116.8 (120.8), 64 x 1-4096 37.8
    // (39.7); equal lengths, which end together, lose: 128 x 8192 209 (206).
    // A quarter of the sequences: 56.7, 69.6, 119.9; 256 tokens: 59.1, 69.6,
    // 123.8.
    late->first = s->num_seqs - (s->num_seqs - 1) / 8 - 1;
    const long long pmin = (static_cast<long long>(maxL) + 1023) / 1024;
    long long P2 = pmin <= 512 ? 512 : (pmin + gran - 1) / gran * gran;
    if (P2 > P) P2 = P;
    late->P = static_cast<int>(P2);
    late->S = static_cast<int>((maxL + P2 - 1) / P2);
  }
  const long long per_split = static_cast<long long>(s->num_kv_heads) * kv4_chunks(s);
  const long long first = late->first, rest = s->num_seqs - late->first;
  const long long grid = per_split * (first * S + rest * late->S);
  if (grid > 0x7fffffffLL || static_cast<long long>(s->num_seqs) * s->num_q_heads > 0x7fffffffLL)
    return PKV_ERR_UNSUPPORTED;
  plan->grid_ctas = static_cast<int32_t>(grid);
  plan->workspace_bytes = static_cast<size_t>(s->num_q_heads) *
                          ((S > 1 ? first * S : 0) + (late->S > 1 ? rest * late->S : 0)) *
                          (static_cast<size_t>(D) * 4 + 8);
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
  Late late{};
  return kv4_plan(s, sms, plan, &late);
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
  Late late{};
  rc = kv4_plan(s, sms, &plan, &late);
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
  const int D = s->head_dim;
  a.chunks = kv4_chunks(s);
  a.late = late.first;
  a.P2 = late.P;
  a.S2 = late.S;
  a.early_ctas = static_cast<int>(static_cast<long long>(late.first) * s->num_kv_heads * a.chunks *
                                  plan.num_splits);
  const size_t Hq = s->num_q_heads;
  a.late_part = plan.num_splits > 1 ? late.first * Hq * plan.num_splits : 0;
  if (plan.workspace_bytes > 0) {
    const size_t rows = plan.workspace_bytes / (static_cast<size_t>(D) * 4 + 8);
    a.d.part_o = static_cast<float*>(workspace);
    a.d.part_ml = reinterpret_cast<float2*>(a.d.part_o + rows * D);
  }
  const bool bf = s->dtype == PKV_BF16;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = (bf ? launch_kv4_bf16 : launch_kv4_f16)(
      a, D, s->block_size, static_cast<unsigned>(plan.grid_ctas), plan.workspace_bytes > 0, st);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launch();
  if (plan.workspace_bytes > 0) count_launch();
  return PKV_OK;
}
