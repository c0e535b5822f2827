// Arguments of the prompt-side attention kernels (pkv_paged_attn_chunk,
// pkv_prompt_attn), shared by the entry points and the kernel.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// Sizes that the kernel and the planner agree on, by head_dim.
constexpr int prefill_row_tiles(int D) { return D == 256 ? 1 : 2; }   // of 128 rows, an item
constexpr int prefill_key_tile(int D) { return D == 256 ? 64 : 128; }

// Where a sequence's keys are cut into partitions (rule at prefill_parts).
constexpr int kPrefillMinPart = 512;      // keys at least
constexpr int kPrefillFewRows = 64;       // rows of a key head: cut finer up to here
constexpr int kPrefillFewUnits = 4;       // partitions a CTA's share of the work makes, few rows
constexpr int kPrefillUnits = 2;          // and many

// What the reduce has to know of a sequence; a last one says whether any was cut.
struct PrefillPlan {
  int parts;                     // partitions; below two: none were written
  int per;                       // key tiles of one
  long long row;                 // its first partial row
};

struct PrefillArgs {
  const int32_t* query_starts;   // [B + 1]
  const int32_t* key_starts;     // packed: [B + 1]; paged: null
  const int32_t* context_lens;   // paged: [B]
  const int32_t* block_tables;   // paged: [B, MB]
  const uint16_t* v;             // packed: [S, Hkv, D]; paged: [NB, Hkv, bs, D]
  uint16_t* out;                 // [T, Hq, D]
  PrefillPlan* plan;             // [B + 1], or null: no sequence is cut
  float2* part_ml;               // (exponent, sum) of a partial row
  float* part_o;                 // its un-normalised output [D]
  int* err;
  long long v_stride;            // packed: elements between tokens
  int B, T, Hq, Hkv, G;
  int max_keys;                  // bound of a sequence's keys (paged), S (packed)
  int MB, NB, bs_log2;
  int causal, negative;          // negative: the scale is
  int part_tiles;                // key tiles of a partition, 0: by the rule
  int ctas;                      // that share the work
  float scale_log2;              // |softmax scale| * log2(e)
};

cudaError_t launch_prefill_f16(const PrefillArgs&, const CUtensorMap& q, const CUtensorMap& k,
                               const CUtensorMap& v, int head_dim, unsigned grid, cudaStream_t);
cudaError_t launch_prefill_bf16(const PrefillArgs&, const CUtensorMap& q, const CUtensorMap& k,
                                const CUtensorMap& v, int head_dim, unsigned grid, cudaStream_t);

}  // namespace pkv
