// The masked tile kernel for streams: a window and the sequence's first keys.
#include "ps_masked_tile.cuh"

namespace ps {

cudaError_t launch_stream_tile_plain(const StreamAttnParams& p, bool bf16, const CUtensorMap& kmap,
                                   const CUtensorMap& vmap, const CUtensorMap& qmap, int ctas,
                                   cudaStream_t stream, bool direct) {
  return launch_masked_tile_kind<0, false>(p, bf16, kmap, vmap, qmap, ctas, stream, direct);
}

}  // namespace ps
