// Instantiations of the 4-bit tensor-core decode (decode_mx.cuh) for power-of-two scales, one per 32 dims:
// 16-bit Q, tiles gathered row by row.
#include "decode_mx.cuh"

namespace pd {

cudaError_t launch_mx_rows_e8m0(const DecodeParams& p, dim3 grid, cudaStream_t st, MmaConfig* cfg) {
  return launch_mx<32, false, true>(p, grid, st, cfg);
}

}  // namespace pd
