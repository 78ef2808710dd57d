// SIMT decode (decode_simt.cuh) of 8-bit caches with a scale per block of rows: every
// accepted shape that the tensor-core kernel of decode_bs.cuh does not take (fp32 Q, D 256).
// Bound by its fp32 products, one block of 224 to 255 registers an SM (D 256 spills 24 bytes), far
// from the bytes.  Measured on one GB300, of the copy rate: D 256, 32 query heads on 8, 32 sequences of
// 512 to 4096 rows 343 us (11 %), 256 sequences 2.9 ms (12 %); fp32 Q at D 128, 32 sequences 127 us
// (15 %), where the tensor-core kernel takes 34 with a 16-bit Q.
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
