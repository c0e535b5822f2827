// Internal interface between the C-ABI front end (pkv_api.cu) and the decode
// kernel translation units (pkv_decode_inst.cu, compiled once per element
// type and kernel variant).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"

namespace pkv {

// Device error word codes (mirror PKV_DEV_* in include/pkv.h).
enum : int {
  kDevBadBlock = 1,
  kDevBadContext = 2,
  kDevBadSlot = 3,
  kDevTimeout = 4,
  kDevBadPosition = 5,
  kDevBadStarts = 6
};

// Largest number of KV blocks one CTA's partition may span.
constexpr int kMaxBlocksPerCta = 256;

struct DecodeArgs {
  const uint16_t* q;            // [B, Hq, D]
  const int32_t* block_tables;  // [B, MB]
  const int32_t* context_lens;  // [B]
  uint16_t* out;                // [B, Hq, D]
  float* part_o;                // un-normalised partial outputs [B, Hq, S, D]
  float2* part_ml;              // (running max in log2 units, sum) per partial row
  const uint16_t* k_new;        // fused append: this step's K/V rows [B, Hkv, D],
  const uint16_t* v_new;        //   or null for a plain decode
  uint16_t* k_cache;            // fused append: the caches the rows go to
  uint16_t* v_cache;
  int* err;                     // device error word
  int B, Hq, Hkv, G, MB, NB;
  int S;                        // splits per sequence (grid extent)
  int P;                        // tokens per split, multiple of the block size
  int max_ctx;                  // upper bound on every context length
  float scale_log2;             // softmax scale * log2(e)
};

// Per-(head_dim, block_size, variant) launch geometry.
struct KernelGeometry {
  int warps;        // warps per CTA, each with its own KV pipeline
  int stages;       // pipeline stages per warp (one K tile + one V tile each)
  int smem_bytes;   // dynamic shared memory per CTA
};

// Variant: 0 = CUDA-core kernel (group size 1 or 2), 1 = mma.sync tensor-core
// kernel (group size 1..32), 2 = tcgen05 kernel (its geometry is its own).
bool decode_geometry(int head_dim, int block_size, int variant, int group_size,
                     KernelGeometry* g);

// Launch the decode kernel over the grid B * Hkv * S of (sequence, kv head,
// partition) units.  Returns cudaErrorInvalidValue for an unbuilt combination.
cudaError_t launch_decode_f16_simt(const DecodeArgs&, const CUtensorMap&, const CUtensorMap&,
                                   int head_dim, int block_size, cudaStream_t);
cudaError_t launch_decode_bf16_simt(const DecodeArgs&, const CUtensorMap&, const CUtensorMap&,
                                    int head_dim, int block_size, cudaStream_t);
cudaError_t launch_decode_f16_mma(const DecodeArgs&, const CUtensorMap&, const CUtensorMap&,
                                  int head_dim, int block_size, cudaStream_t);
cudaError_t launch_decode_bf16_mma(const DecodeArgs&, const CUtensorMap&, const CUtensorMap&,
                                   int head_dim, int block_size, cudaStream_t);

// tcgen05 variant (head_dim 128, group size up to 32): same grid and
// partitions as the other variants; it walks a partition in 128-token groups
// (the last one may be ragged).
cudaError_t launch_decode_tc(const DecodeArgs&, const CUtensorMap&, const CUtensorMap&, bool bf16,
                             int head_dim, int block_size, cudaStream_t);
int tc_smem_bytes(int group_size);
int tc_ring_slots(int group_size);   // 32 KB K/V tile slots per CTA
int tc_warps(int group_size);        // warps per CTA (softmax, producer, MMA)

int* device_error_word();  // device address of the error word (current device)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Services of the front end (pkv_api.cu) to the other entry points.
int check_cache_shape(const pkv_shape*);     // PKV_OK or the PKV_ERR_* of a bad cache shape
int check_decode_shape(const pkv_shape*);    // the same for a decode batch
int device_sms(int* sms);                    // SM count of the current device
// Workspace set for the current device with pkv_set_workspace, or {nullptr, 0}.
int device_workspace(void** ptr, size_t* bytes);
// Tensor map of a cache in boxes of one block's rows, 128-byte swizzled: of 64
// channels (x channel, y row of [NB, Hkv, bs]), or all of them, 64 by 64 (whole:
// x channel of 64, y row, z which 64).
int block_map(CUtensorMap* out, const void* base, const pkv_shape& s, bool whole);
// Tensor map of packed rows [tokens, heads, head_dim], `stride` elements between
// tokens, in boxes of 64 channels x box_heads x box_tokens, 128-byte swizzled.
// What lies past the last token reads as zero.
int rows_map(CUtensorMap* out, const void* base, bool bf16, int head_dim, int heads, int64_t tokens,
             int64_t stride, int box_heads, int box_tokens);
void count_launch();                         // one more kernel for pkv_launch_count

// Launch with programmatic stream serialisation: the grid may become resident
// while the stream's previous kernel finishes, so the kernel calls pdl_wait()
// before its first access to memory.
template <class... KArgs, class... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, unsigned threads, size_t smem,
                       cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

}  // namespace pkv
