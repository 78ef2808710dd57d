// Instantiations of the 4-bit tensor-core decode (decode_mx.cuh) for e4m3 scales, one per 16 dims, tiles
// gathered row by row, F32 Q.
#include "decode_mx.cuh"

namespace pd {

cudaError_t launch_mx_f32_e4m3(const DecodeParams& p, dim3 grid, cudaStream_t st, MmaConfig* cfg) {
  return launch_mx_rows<16, true>(p, grid, st, cfg);
}

}  // namespace pd
