// The masked split kernel: masks that are an interval of keys per row.
#include "ps_masked_split.cuh"

namespace ps {

cudaError_t launch_masked_split(const MaskedAttnParams& p, bool bf16, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, int ctas, cudaStream_t stream,
                                bool pdl) {
  return launch_split_any(p, bf16, kmap, vmap, ctas, stream, pdl);
}

}  // namespace ps
