// scaled_sliced.cu -- the sliced kernel (scaled_sliced.cuh) for 8-bit operands.
#include "scaled_sliced.cuh"

namespace dg {

int scaled_sliced_smem(int bn, int stages, int part_rows) { return sliced_smem<false>(bn, stages, part_rows); }

int scaled_sliced_clusters(int slices) { return resident_clusters<false>(slices); }

cudaError_t launch_scaled_sliced(const ScMaps& m, const ScParams& p, int grid, cudaStream_t s) {
  return launch<false>(m, p, grid, s);
}

}  // namespace dg
