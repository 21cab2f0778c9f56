// The masked tile kernel for streams: the same with scores capped beyond kLargeCapLog2.
#include "ps_masked_tile.cuh"

namespace ps {

cudaError_t launch_stream_tile_large_cap(const StreamAttnParams& p, bool bf16,
                                         const CUtensorMap& kmap, const CUtensorMap& vmap,
                                         const CUtensorMap& qmap, int ctas, cudaStream_t stream,
                                         bool direct) {
  return launch_masked_tile_kind<2, false>(p, bf16, kmap, vmap, qmap, ctas, stream, direct);
}

}  // namespace ps
