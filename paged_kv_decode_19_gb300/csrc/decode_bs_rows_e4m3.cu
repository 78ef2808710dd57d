// Instantiations of the block-scaled tensor-core decode (decode_bs.cuh) for e4m3 codes in tiles gathered row by
// row.
#include "decode_bs.cuh"

namespace pd {

cudaError_t launch_bs_rows_e4m3(const DecodeParams& p, const CUtensorMap& tm, int q_dtype, dim3 grid,
                                cudaStream_t st, MmaConfig* cfg) {
  return launch_bs_any<F8, true>(p, tm, q_dtype, grid, st, cfg);
}

}  // namespace pd
