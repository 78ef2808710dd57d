// Instantiations of the 4-bit tensor-core decode (decode_mx.cuh) for e4m3 scales, one per 16 dims:
// 16-bit Q, tiles copied whole.
#include "decode_mx.cuh"

namespace pd {

cudaError_t launch_mx_e4m3(const DecodeParams& p, dim3 grid, cudaStream_t st, MmaConfig* cfg) {
  return launch_mx<16, false, false>(p, grid, st, cfg);
}

}  // namespace pd
