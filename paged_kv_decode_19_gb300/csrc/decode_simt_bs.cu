// SIMT decode (decode_simt.cuh) of 8-bit caches with a scale per block of rows: every
// accepted shape that the tensor-core kernel of decode_bs.cuh does not take.
#include "decode_simt.cuh"

namespace pd {

template <typename KT>
static cudaError_t launch_simt_q(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                                 int* ctas) {
  if (q_dtype == kBF16) return launch_simt_t<KT, __nv_bfloat16, true>(p, grid, st, ctas);
  if (q_dtype == kF16) return launch_simt_t<KT, __half, true>(p, grid, st, ctas);
  if (q_dtype == kF32) return launch_simt_t<KT, float, true>(p, grid, st, ctas);
  return cudaErrorInvalidValue;
}

cudaError_t launch_decode_simt_bs(const DecodeParams& p, int q_dtype, int kv_dtype, dim3 grid,
                                  cudaStream_t st, int* ctas) {
  if (kv_dtype == kE4M3) return launch_simt_q<F8>(p, q_dtype, grid, st, ctas);
  if (kv_dtype == kI8) return launch_simt_q<I8>(p, q_dtype, grid, st, ctas);
  return cudaErrorInvalidValue;
}

}  // namespace pd
