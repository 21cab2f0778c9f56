// Forking sequences of the paged cache: after beam search has chosen, for every child, the
// parent that it continues, the child's block table takes the parent's full blocks as they
// are (shared), and the rows of the parent's partly filled last block are copied into a
// block of the child's own, in every layer, since each child will write its next token
// there. All of it in one launch.
//
// Units, one warp each: per child its table row and length; per (child, layer, K or V) the
// tail rows, (L mod 16) * H_kv * D values that lie together in both blocks. A unit's
// indexes are a chain of three small loads, so the kernel is bound by bytes only with many
// layers, and by that chain's latency otherwise.
#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32) fork_kernel(const ForkParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t per_child = 1 + 2 * static_cast<int64_t>(p.layers);
  const int64_t units = per_child * p.groups * p.n_out;
  const int row_vecs = p.H_kv * p.D / 8;  // 16-byte chunks of a token's row
  const int64_t block_vecs = static_cast<int64_t>(kBlockSize) * row_vecs;
  const int64_t layer_vecs = block_vecs * p.num_blocks;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    // tables first: child c's table is unit c, then the tail units, layer by layer
    const int n = p.groups * p.n_out;
    const bool table = u < n;
    const int64_t v = table ? u : u - n;
    const int c = static_cast<int>(v % n), part = static_cast<int>(v / n);
    const int parent = p.parents[c];
    const int src = (c / p.n_out) * p.n_in + parent;
    const bool live = parent >= 0 && parent < p.n_in;
    if (!live && table && parent >= p.n_in && lane == 0) record_error(p.err, kDevBadSequence);
    const int L = live ? p.seq_lens[src] : 0;
    const int full = L / kBlockSize, rest = L - full * kBlockSize;
    const bool ok = L >= 0 && full + (rest > 0) <= p.max_blocks;
    if (!ok && table && lane == 0) record_error(p.err, kDevBadSequence);
    const int tail = ok && rest > 0 ? p.tails[c] : 0;
    if (table) {
      if (lane == 0) p.out_lens[c] = ok ? L : 0;
      if (!ok) continue;
      const int32_t* s = p.tables + static_cast<int64_t>(src) * p.max_blocks;
      int32_t* d = p.out_tables + static_cast<int64_t>(c) * p.max_blocks;
      for (int i = lane; i < full; i += 32) d[i] = s[i];
      if (rest > 0 && lane == 0) d[full] = tail;
    } else {
      if (!ok || rest == 0) continue;
      const int from = p.tables[static_cast<int64_t>(src) * p.max_blocks + full];
      if (from < 0 || from >= p.num_blocks || tail < 0 || tail >= p.num_blocks) {
        if (lane == 0 && part == 0) record_error(p.err, kDevBadBlockId);
        continue;
      }
      const int layer = part >> 1;
      uint4* pool = static_cast<uint4*>((part & 1) ? p.v_pool : p.k_pool) + layer * layer_vecs;
      const uint4* s = pool + from * block_vecs;
      uint4* d = pool + tail * block_vecs;
      const int vecs = rest * row_vecs;
      constexpr int kInFlight = 8;
      for (int i0 = lane; i0 < vecs; i0 += 32 * kInFlight) {
        uint4 r[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k)
          if (i0 + 32 * k < vecs) r[k] = s[i0 + 32 * k];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k)
          if (i0 + 32 * k < vecs) d[i0 + 32 * k] = r[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_fork(const ForkParams& p, int num_sms, cudaStream_t stream) {
  const int64_t units = (1 + 2 * static_cast<int64_t>(p.layers)) * p.groups * p.n_out;
  const int64_t want = (units + kWarps - 1) / kWarps, cap = static_cast<int64_t>(num_sms) * 8;
  return launch_kernel(fork_kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)),
                       dim3(kWarps * 32), 0, stream, true, p);
}

}  // namespace ps
