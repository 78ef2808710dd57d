// SIMT decode (decode_simt.cuh): the instantiations for fp32, f16, bf16 and per-tensor
// e4m3 caches, and which combinations exist.
#include "decode_simt.cuh"

namespace pd {

cudaError_t launch_decode_simt(const DecodeParams& p, int q_dtype, int kv_dtype, dim3 grid,
                               cudaStream_t st, int* ctas) {
  if (kv_dtype == kF32 && q_dtype == kF32) return launch_simt_t<float, float>(p, grid, st, ctas);
  if (kv_dtype == kBF16 && q_dtype == kBF16) return launch_simt_t<__nv_bfloat16, __nv_bfloat16>(p, grid, st, ctas);
  if (kv_dtype == kF16 && q_dtype == kF16) return launch_simt_t<__half, __half>(p, grid, st, ctas);
  if (kv_dtype == kE4M3 && q_dtype == kBF16) return launch_simt_t<F8, __nv_bfloat16>(p, grid, st, ctas);
  if (kv_dtype == kE4M3 && q_dtype == kF16) return launch_simt_t<F8, __half>(p, grid, st, ctas);
  if (kv_dtype == kE4M3 && q_dtype == kF32) return launch_simt_t<F8, float>(p, grid, st, ctas);
  return cudaErrorInvalidValue;
}

bool simt_supports(int q_dtype, int kv_dtype, int D) {
  if (D != 64 && D != 128 && D != 256) return false;
  if (kv_dtype == q_dtype && kv_dtype != kE4M3) return true;
  return kv_dtype == kE4M3 && (q_dtype == kBF16 || q_dtype == kF16 || q_dtype == kF32);
}

}  // namespace pd
