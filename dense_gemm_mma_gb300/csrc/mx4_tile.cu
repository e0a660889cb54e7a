// mx4_tile.cu -- the tile kernel (scaled_tile.cuh) for 4-bit operands.
#include "scaled_tile.cuh"

namespace dg {

namespace {
// Is a pair's call the six-stage kernel's: 16-bit results, and groups that its tables have room for.  Up to four k-blocks the
// five stages' rows of 128 bytes store faster, where little arithmetic is left behind the product (8192 x 8192 x 512 into
// fp16 35.4 us, six 40; x 1024 39.6 and 41.5; x 2048 60.8 and 53.5; with SiLU, x 512, 69 and 57).
bool six(const ScParams& p) {
  const bool simple = p.act != 3 && p.act != 4 && p.beta == 0.f;
  return p.out_kind != OUT_F32 && p.groups <= kSixGroups && (p.k_blocks > 4 || !simple);
}
}  // namespace

cudaError_t launch_mx4_tile(bool pair, const ScMaps& m, const ScParams& p, int grid, cudaStream_t s) {
  if (pair && six(p)) return launch<true, true, true>(m, p, grid, s);
  return pair ? launch<true, true>(m, p, grid, s) : launch<false, true>(m, p, grid, s);
}

int mx4_tile_stages(bool pair, const ScParams& p) {
  if (pair && six(p)) return Cfg<true, true, true>::STAGES;
  return pair ? Cfg<true, true, false>::STAGES : Cfg<false, true, false>::STAGES;
}

int mx4_tile_box_row(bool pair, const ScParams& p) { return pair && six(p) ? Cfg<true, true, true>::ROW : 128; }

int mx4_tile_clusters() {
  const int a = resident_pairs<true>(), b = resident_pairs<true, true>();
  return a < b ? a : b;
}

}  // namespace dg
