// The masked tile kernel with scores capped beyond kLargeCapLog2 and a distance bias.
#include "ps_masked_tile.cuh"

namespace ps {

cudaError_t launch_masked_tile_large_cap_bias(const MaskedAttnParams& p, bool bf16,
                                              const CUtensorMap& kmap, const CUtensorMap& vmap,
                                              const CUtensorMap& qmap, int ctas,
                                              cudaStream_t stream, bool direct) {
  return launch_masked_tile_kind<2, true>(p, bf16, kmap, vmap, qmap, ctas, stream, direct);
}

}  // namespace ps
