// Arguments of the prompt-side attention kernels (pkv_paged_attn_chunk,
// pkv_prompt_attn), shared by the entry points and the kernel.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// Sizes that the kernel and the planner agree on, by head_dim.
constexpr int prefill_row_tiles(int D) { return D == 256 ? 1 : 2; }   // of 128 rows, an item
constexpr int prefill_key_tile(int D) { return D == 256 ? 64 : 128; }

// Keys of a sequence at most (checked on the device): the kernel's waits, some of
// which are as long as an item, give up after a few seconds.
constexpr int kPrefillMostKeys = 1 << 24;
// Keys of the smallest part of an item's keys that is left at one of its ends.
constexpr int kPrefillMinPart = 512;
// What an item costs a CTA: so much a key, and so much besides (a third of what
// a key of two row tiles takes is the unit), where it is causal more for its
// tokens, as key tiles that hide something take longer.  (Two thirds of it with
// one row tile, as its keys cost: mixed steps 1.2% slower, prompts the same.)
constexpr int kPrefillKeyCost = 3, kPrefillItemCost = 3 * 320, kPrefillTokenCost = 3;
constexpr int kPrefillKeyCost1 = 2, kPrefillItemCost1 = 3 * 320;   // with one row tile of two
// A reference score's exponent beyond which scores are taken relative to it before
// they are scaled (2^-16 of a weight is lost below).
constexpr float kPrefillFar = 256.f;
// Below so many items a key head, lines of less than 2^31 in all and no sequence
// longer than allowed, the scheduler counts in 32 bits.
constexpr int kPrefillSmallItems = 30000;

// What the reduce has to know of an item that CTA c goes on with where another
// CTA left off (kind 0: CTA c does no such thing).
struct PrefillCut {
  int kind;                      // 1: further pieces lie before it, 2: only the first one
  int first;                     // kind 2: the CTA that has the item's first piece
  int ends;                      // CTA c's piece is the item's last
  int kvh, q_row, ntok;
};

struct PrefillArgs {
  const int32_t* query_starts;   // [B + 1]
  const int32_t* key_starts;     // packed: [B + 1]; paged: null
  const int32_t* context_lens;   // paged: [B]
  const int32_t* block_tables;   // paged: [B, MB]
  const uint16_t* v;             // packed: [S, Hkv, D]; paged: [NB, Hkv, bs, D]
  uint16_t* out;                 // [T, Hq, D]
  PrefillCut* cuts;              // [CTAs], or null: no item is cut
  float2* part_ml;               // (reference score, sum) of a partial row, `rows` for a piece:
  float* part_o;                 //   piece 2c is CTA c's with keys before it, 2c + 1 its
                                 //   with only keys behind; the un-normalised output [D]
  int* err;
  long long v_stride;            // packed: elements between tokens
  int B, T, Hq, Hkv, G;
  int max_keys;                  // bound of a sequence's keys (paged), S (packed)
  int MB, NB, bs_log2;
  int causal, negative;          // negative: the scale is
  int rows;                      // of an item at most
  int min_part;                  // key tiles of an item's first and last pieces at least
  int small;                     // the scheduler may count in 32 bits
  float scale_log2;              // |softmax scale| * log2(e)
};

cudaError_t launch_prefill_f16(const PrefillArgs&, const CUtensorMap& q, const CUtensorMap& k,
                               const CUtensorMap& v, int head_dim, unsigned grid, cudaStream_t);
cudaError_t launch_prefill_bf16(const PrefillArgs&, const CUtensorMap& q, const CUtensorMap& k,
                                const CUtensorMap& v, int head_dim, unsigned grid, cudaStream_t);

}  // namespace pkv
