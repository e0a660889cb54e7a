// scaled_tile.cu -- the tile kernel (scaled_tile.cuh) for 8-bit operands.
#include "scaled_tile.cuh"

namespace dg {

cudaError_t launch_scaled_tile(bool pair, const ScMaps& m, const ScParams& p, int grid, cudaStream_t s) {
  return pair ? launch<true, false>(m, p, grid, s) : launch<false, false>(m, p, grid, s);
}

int scaled_tile_stages(bool pair) { return pair ? Cfg<true, false, false>::STAGES : Cfg<false, false, false>::STAGES; }

int scaled_tile_clusters() { return resident_pairs<false>(); }

}  // namespace dg
