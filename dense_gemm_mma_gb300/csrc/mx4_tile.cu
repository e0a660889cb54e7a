// mx4_tile.cu -- the tile kernel (scaled_tile.cuh) for 4-bit operands.
#include "scaled_tile.cuh"

namespace dg {

cudaError_t launch_mx4_tile(bool pair, const ScMaps& m, const ScParams& p, int grid, cudaStream_t s) {
  return pair ? launch<true, true>(m, p, grid, s) : launch<false, true>(m, p, grid, s);
}

int mx4_tile_stages(bool pair) { return pair ? Cfg<true, true>::STAGES : Cfg<false, true>::STAGES; }

int mx4_tile_clusters() { return resident_pairs<true>(); }

}  // namespace dg
