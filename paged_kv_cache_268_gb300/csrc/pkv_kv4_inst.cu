// Instantiates the 4-bit decode kernels for one element type; compiled once
// per PKV_INST_BF16.
#include <atomic>

#include "pkv_kv4_decode.cuh"

#ifndef PKV_INST_BF16
#error "define PKV_INST_BF16 (0 = binary16, 1 = bfloat16)"
#endif

namespace pkv {
namespace {

constexpr bool kBF = PKV_INST_BF16 != 0;

template <int D, int BS, int HC, int NT>
cudaError_t launch_one(const Kv4Args& a, unsigned grid, bool reduce, cudaStream_t stream) {
  constexpr int SMEM = kv4_smem(D, NT);
  auto kern = kv4_decode_kernel<kBF, D, BS, HC, NT>;
  // the shared-memory limit is raised once per device (threads that race here
  // set the same attribute)
  static std::atomic<unsigned> mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned bit = dev < 32 ? 1u << dev : 0u;
  if (bit == 0 || !(mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    mask.fetch_or(bit, std::memory_order_release);
  }
  e = launch_pdl(kern, dim3(grid), kKv4Warps * 32, SMEM, stream, a);
  if (e != cudaSuccess || !reduce) return e;
  const int row0 = a.d.S > 1 ? 0 : a.late * a.d.Hq;
  const unsigned rows = static_cast<unsigned>(a.d.B) * a.d.Hq - row0;
  return launch_pdl(kv4_reduce_kernel<kBF, D>, dim3((rows + 3) / 4), 128, 0, stream, a, row0);
}

template <int D, int BS>
cudaError_t launch_heads(const Kv4Args& a, unsigned grid, bool reduce, cudaStream_t stream) {
  if constexpr (D <= 128) {
    if (kv4_tiles(D, a.d.G) == 2) return launch_one<D, BS, 8, 2>(a, grid, reduce, stream);
  }
  if constexpr (D > 64) {
    if (kv4_columns(D, a.d.G) == 2) return launch_one<D, BS, 2, 1>(a, grid, reduce, stream);
  }
  return kv4_columns(D, a.d.G) == 4 ? launch_one<D, BS, 4, 1>(a, grid, reduce, stream)
                                    : launch_one<D, BS, 8, 1>(a, grid, reduce, stream);
}

template <int D>
cudaError_t launch_bs(const Kv4Args& a, int bs, unsigned grid, bool reduce, cudaStream_t stream) {
  return bs == 16 ? launch_heads<D, 16>(a, grid, reduce, stream) : launch_heads<D, 32>(a, grid, reduce, stream);
}

}  // namespace

#if PKV_INST_BF16
#define PKV_LAUNCH_NAME launch_kv4_bf16
#else
#define PKV_LAUNCH_NAME launch_kv4_f16
#endif

cudaError_t PKV_LAUNCH_NAME(const Kv4Args& a, int head_dim, int block_size, unsigned grid,
                            bool reduce, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_bs<64>(a, block_size, grid, reduce, stream);
    case 128: return launch_bs<128>(a, block_size, grid, reduce, stream);
    case 256: return launch_bs<256>(a, block_size, grid, reduce, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
