// Instantiations of the 4-bit tensor-core decode (decode_mx.cuh) for power-of-two scales, one per 32 dims:
// F32 Q, tiles copied whole.
#include "decode_mx.cuh"

namespace pd {

cudaError_t launch_mx_f32_e8m0(const DecodeParams& p, dim3 grid, cudaStream_t st, MmaConfig* cfg) {
  return launch_mx<32, true, false>(p, grid, st, cfg);
}

}  // namespace pd
