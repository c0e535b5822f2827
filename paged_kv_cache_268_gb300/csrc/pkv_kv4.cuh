// Layout and arithmetic of the 4-bit KV cache, shared by the kernels that
// write it, read it back and attend over it.  The format is stated in
// include/pkv.h.
//
// The layout is chosen for the attention kernel: the two 8-channel words that
// a tensor-core fragment wants lie in one 32-bit word, ldmatrix reads of eight
// rows hit eight different bank groups (the exclusive-or of the chunk number),
// and the value parameters of two neighbouring tokens lie side by side, as a
// fragment of probabilities holds them.  A token's codes stay one contiguous
// D/2 bytes, so that a single-token append touches few sectors.
#pragma once

#include <stdint.h>

namespace pkv {

constexpr int kGroup4 = 32;   // channels that share one scale and zero point

// Bytes of one (block, kv head) tile, K or V.
constexpr int kv4_tile_bytes(int D, int BS) { return BS * (D / 2 + D / 8); }

// Place of 16-byte chunk `g` (the codes of channel group g) within row `r`.
template <int D>
__host__ __device__ __forceinline__ int kv4_chunk(int r, int g) {
  return g ^ ((r * (D / 32) / 8) & (D / 32 - 1));
}

// Byte offset in a tile of the codes of group g of row r.
template <int D>
__host__ __device__ __forceinline__ int kv4_code_off(int r, int g) {
  return r * (D / 2) + kv4_chunk<D>(r, g) * 16;
}

// Byte offsets in a tile of the parameters of (row r, group g): keys keep
// (scale, zero) together; values keep the scales of rows 2u and 2u + 1
// together, then their zeros.
template <int D>
__host__ __device__ __forceinline__ int kv4_k_par_off(int BS, int r, int g) {
  return BS * (D / 2) + (r * (D / 32) + g) * 4;
}
template <int D>
__host__ __device__ __forceinline__ int kv4_v_par_off(int BS, int r, int g) {
  return BS * (D / 2) + ((r >> 1) * (D / 32) + g) * 8 + (r & 1) * 2;   // zero: 4 bytes on
}

}  // namespace pkv
