// Instantiates the prompt-side attention kernel for one element type
// (PKV_INST_BF16: 0 binary16, 1 bfloat16) and every head_dim.
#include <atomic>

#include "pkv_prefill.cuh"

namespace pkv {
namespace {

template <bool BF, int D>
cudaError_t launch(const PrefillArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   unsigned grid, cudaStream_t stream) {
  constexpr int SMEM = PrefillLayout<D>::BYTES;
  auto kern = prefill_kernel<BF, D>;
  // the shared-memory limit is raised once per device (every time past 32)
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
  return launch_pdl(kern, dim3(grid), PrefillLayout<D>::THREADS, SMEM, stream, a, q, k, v);
}

template <bool BF>
cudaError_t dispatch(const PrefillArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                     int D, unsigned grid, cudaStream_t stream) {
  switch (D) {
    case 64: return launch<BF, 64>(a, q, k, v, grid, stream);
    case 128: return launch<BF, 128>(a, q, k, v, grid, stream);
    case 256: return launch<BF, 256>(a, q, k, v, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

#if PKV_INST_BF16
cudaError_t launch_prefill_bf16(
#else
cudaError_t launch_prefill_f16(
#endif
    const PrefillArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, int head_dim,
    unsigned grid, cudaStream_t stream) {
  return dispatch<PKV_INST_BF16 != 0>(a, q, k, v, head_dim, grid, stream);
}

}  // namespace pkv
