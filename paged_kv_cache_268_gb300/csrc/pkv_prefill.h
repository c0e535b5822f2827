// Arguments of the prompt-side attention kernels (pkv_paged_attn_chunk,
// pkv_prompt_attn), shared by the entry points and the kernel.
#pragma once

#include "pkv_internal.h"

namespace pkv {

struct PrefillArgs {
  const uint16_t* q;             // [T, Hq, D], token stride q_stride
  const uint16_t* k;             // packed: [S, Hkv, D]; paged: [NB, Hkv, bs, D]
  const uint16_t* v;
  const int32_t* query_starts;   // [B + 1]
  const int32_t* key_starts;     // packed: [B + 1]; paged: null
  const int32_t* context_lens;   // paged: [B]
  const int32_t* block_tables;   // paged: [B, MB]
  uint16_t* out;                 // [T, Hq, D]
  int* err;
  long long q_stride, k_stride, v_stride;   // elements between tokens
  int B, T, Hq, Hkv, G;
  int max_keys;                  // bound of a sequence's keys (paged), S (packed)
  int MB, NB, bs_log2;
  int causal;
  float scale;
};

// Queries and keys of sequence b: rows [q0, q0 + n) attend over L keys, whose
// first is key row k0 (packed).  False, and nothing to do, where the arrays
// hold no valid range; `code` then says what is wrong.
__device__ __forceinline__ bool prefill_seq(const PrefillArgs& a, int b, int& q0, int& n, int& k0,
                                            int& L, int& code) {
  q0 = a.query_starts[b];
  const int q1 = a.query_starts[b + 1];
  code = kDevBadStarts;
  n = L = k0 = 0;
  if (q0 < 0 || q1 < q0 || q1 > a.T) return false;
  if (a.key_starts != nullptr) {
    k0 = a.key_starts[b];
    const int k1 = a.key_starts[b + 1];
    if (k0 < 0 || k1 < k0 || k1 > a.max_keys) return false;
    L = k1 - k0;
  } else {
    L = a.context_lens[b];
    if (L < 0 || L > a.max_keys) {
      code = kDevBadContext;
      return false;
    }
  }
  n = q1 - q0;
  code = 0;
  return true;
}

}  // namespace pkv
