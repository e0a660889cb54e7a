// mx4_sliced.cu -- the sliced kernel (scaled_sliced.cuh) for 4-bit operands.
#include "scaled_sliced.cuh"

namespace dg {

int mx4_sliced_smem(int bn, int stages, int part_rows) { return sliced_smem<true>(bn, stages, part_rows); }

int mx4_sliced_clusters(int slices) { return resident_clusters<true>(slices); }

cudaError_t launch_mx4_sliced(const ScMaps& m, const ScParams& p, int grid, cudaStream_t s) {
  return launch<true>(m, p, grid, s);
}

}  // namespace dg
