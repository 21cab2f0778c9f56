// Where the splits of a context begin, for the planner and (as plain C++) for the host.
#pragma once

#ifdef __CUDACC__
#define PS_BOTH __host__ __device__ __forceinline__
#else
#define PS_BOTH inline
#endif

namespace ps {

// First page of split k of ns, 0 <= k <= ns, of the pages [first, end): first + k span / ns. A
// context has up to 2^27 pages and is split up to 32 ways, so k span may pass 32 bits; with
// span = q ns + r no product does (r and k are at most ns).
PS_BOTH int split_start(int first, int end, int ns, int k) {
  const int span = end - first, q = span / ns, r = span - q * ns;
  return first + q * k + r * k / ns;
}

}  // namespace ps
