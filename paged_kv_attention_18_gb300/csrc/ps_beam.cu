// Beam search's selection over beams and vocabulary: of the W * V continuations of a
// prompt's beams, with score(w, v) = cum_w + x_wv - lse_w (lse_w the log-sum-exp of beam
// w's logits), the n best, ties to the lowest beam and then the lowest token.
//
// One pass over the logits. Within a beam the order of the scores is the order of the
// logits, so a chunk's n best candidates are chosen on the logits alone, before lse is
// known; the few that are left are scored and compared across chunks and beams in 64 bits.
//   scan    one CTA per (beam, chunk of kChunk logits). The chunk is held in registers:
//           16-byte loads, all in flight at once. Its maximum M and sum of exp(x - M) are
//           exact reductions of what is held; the candidates are the logits at or above a
//           bound tau: the n-th largest of a warp's 32 thread maxima is at most the n-th
//           largest logit of the chunk, and tau is the largest such bound of the CTA's
//           warps. A few dozen logits pass it; they are ranked among themselves.
//   merge   one CTA per prompt: lse of each beam from its chunks' (M, sum), then the same
//           bound on the chunks' candidates, and the ranks of those that pass.
// Bound by the bytes of the logits (read once). Sums: a chunk's 32 terms per thread are
// added in fp32, then across threads in fp32 pairs and across chunks in 64 bits.
#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = kBeamChunk;
constexpr int kPerThread = kChunk / kThreads;  // logits per thread
constexpr int kCap = 1024;                     // candidates ranked in shared memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.69314718055994530942;

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen<float>(float x) { return x; }
template <>
__device__ __forceinline__ float widen<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// NaN counts as -inf, -0 as +0 (so that it ties with it).
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : -INFINITY; }

// Unsigned integers in the order of the floats (no NaN).
__device__ __forceinline__ uint32_t order32(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ unsigned long long order64(double x) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
constexpr uint32_t kOrderNegInf = 0x007fffffu;  // order32(-inf)

// The largest and the n-th largest of the warp's 32 keys (n in 1..32).
__device__ __forceinline__ uint32_t warp_nth(uint32_t key, int n, uint32_t& top) {
  const int lane = threadIdx.x & 31;
  uint32_t m = __reduce_max_sync(0xffffffffu, key);
  top = m;
  for (int i = 1; i < n; ++i) {
    const int who = __ffs(__ballot_sync(0xffffffffu, key == m)) - 1;
    if (lane == who) key = 0;  // taken out (0 is below every key)
    m = __reduce_max_sync(0xffffffffu, key);
  }
  return m;
}

// Block-wide: the largest key, and a bound that at least n of the keys' owners reach.
__device__ __forceinline__ void block_bound(uint32_t key, int n, uint32_t* sh, uint32_t& top,
                                            uint32_t& tau) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t wt;
  const uint32_t wn = warp_nth(key, n, wt);
  if (lane == 0) {
    sh[warp] = wt;
    sh[kWarps + warp] = wn;
  }
  __syncthreads();
  top = tau = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    top = max(top, sh[w]);
    tau = max(tau, sh[kWarps + w]);
  }
}

__device__ __forceinline__ unsigned long long block_max(unsigned long long k,
                                                        unsigned long long* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(0xffffffffu, k, o);
    k = y > k ? y : k;
  }
  __syncthreads();  // the last round's values have been read
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = k;
  __syncthreads();
  k = sh[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) k = sh[w] > k ? sh[w] : k;
  return k;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(const BeamParams p) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  constexpr int kLoads = kPerThread / kVec;
  __shared__ uint32_t sh_key[2 * kWarps];
  __shared__ float sh_sum[kWarps];
  __shared__ unsigned long long sh_max[kWarps];
  __shared__ unsigned long long list[kCap];
  __shared__ int count;
  pdl_wait();
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;
  if (p.finished != nullptr && p.finished[row]) {
    pdl_launch_dependents();
    return;
  }
  if (threadIdx.x == 0) count = 0;
  const T* base = static_cast<const T*>(p.logits) + row * p.ld;
  // vectors start at the 16-byte boundary at or before the row's first logit
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / sizeof(T));
  const int first = chunk * kChunk - skew;  // token of the chunk's first place
  float x[kPerThread];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int t0 = first + (j * kThreads + threadIdx.x) * kVec;
    if (t0 >= 0 && t0 + kVec <= p.V) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(base + t0));
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[j * kVec + i] = clean(widen<T>(e[i]));
    } else {  // the row's ends: what lies outside the row is not read
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int t = t0 + i;
        x[j * kVec + i] = t >= 0 && t < p.V ? clean(widen<T>(base[t])) : -INFINITY;
      }
    }
  }
  auto token = [&](int i) {
    return first + ((i / kVec) * kThreads + static_cast<int>(threadIdx.x)) * kVec + i % kVec;
  };
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) m = fmaxf(m, x[i]);
  uint32_t top, tau;
  block_bound(order32(m), p.n, sh_key, top, tau);
  const float M = __uint_as_float(top ^ ((top >> 31) ? 0x80000000u : 0xffffffffu));
  // sum of exp(x - M), and the candidates
  float s0 = 0.f, s1 = 0.f;
  // (x - M first: rounding M log2(e) once for all terms would shift their sum)
  const float sub = M == -INFINITY ? 0.f : M;
  const uint32_t bound = tau > kOrderNegInf ? tau : kOrderNegInf + 1;
#pragma unroll
  for (int i = 0; i < kPerThread; i += 2) {
    s0 += fast_exp2((x[i] - sub) * kLog2e);
    s1 += fast_exp2((x[i + 1] - sub) * kLog2e);
  }
  if (order32(m) >= bound) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const uint32_t k = order32(x[i]);
      if (k >= bound) {
        const int at = atomicAdd(&count, 1);
        if (at < kCap)
          list[at] = (static_cast<unsigned long long>(k) << 32) |
                     (0xffffffffu - static_cast<uint32_t>(token(i)));
      }
    }
  }
  float s = s0 + s1;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) sh_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sh_sum[w];
    p.stat[blockIdx.x] = make_float2(M, s);
  }
  unsigned long long* out = p.cand + static_cast<int64_t>(blockIdx.x) * p.n;
  const int c = count;
  if (c <= kCap) {
    for (int i = threadIdx.x; i < c; i += kThreads) {
      const unsigned long long k = list[i];
      int rank = 0;
      for (int j = 0; j < c; ++j) rank += list[j] > k ? 1 : 0;
      if (rank < p.n) out[rank] = k;
    }
    for (int i = c + threadIdx.x; i < p.n; i += kThreads) out[i] = 0;  // none
  } else {
    // more equal logits than the list holds: n rounds of the block's largest key below
    // the one before
    unsigned long long last = ~0ull;
    for (int r = 0; r < p.n; ++r) {
      unsigned long long best = 0;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        const uint32_t k32 = order32(x[i]);
        const unsigned long long k = (static_cast<unsigned long long>(k32) << 32) |
                                     (0xffffffffu - static_cast<uint32_t>(token(i)));
        if (k32 >= bound && k < last && k > best) best = k;
      }
      last = block_max(best, sh_max);
      if (threadIdx.x == 0) out[r] = last;
    }
  }
}

// A candidate of the merge: its score's 64-bit order and its flat index (beam * V + token).
struct Best {
  unsigned long long score;
  int flat;
};
__device__ __forceinline__ bool better(const Best& a, const Best& b) {
  return a.score > b.score || (a.score == b.score && a.flat < b.flat);
}

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamParams p) {
  __shared__ uint32_t sh_key[2 * kWarps];
  __shared__ double sh_lse[kBeamMaxWidth];
  __shared__ double sh_cum[kBeamMaxWidth];
  __shared__ int sh_kind[kBeamMaxWidth];  // 0 no candidate, 1 scored, 2 finished
  __shared__ Best list[kCap];
  __shared__ Best sh_best[kWarps];
  __shared__ int count;
  pdl_wait();
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) count = 0;
  for (int w = warp; w < p.W; w += kWarps) {
    const int row = b * p.W + w;
    const float cum = p.scores[row];
    const bool fin = p.finished != nullptr && p.finished[row];
    int kind = cum > -INFINITY && cum < INFINITY ? (fin ? 2 : 1) : 0;
    double lse = 0.0;
    if (kind == 1) {
      const float2* st = p.stat + static_cast<int64_t>(row) * p.chunks;
      float M = -INFINITY;
      for (int c = lane; c < p.chunks; c += 32) M = fmaxf(M, st[c].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      if (!(M > -INFINITY && M < INFINITY)) {
        kind = 0;  // no finite logit, or an infinite one
      } else {
        double S = 0.0;
        for (int c = lane; c < p.chunks; c += 32)
          if (st[c].x > -INFINITY) S += static_cast<double>(st[c].y * expf(st[c].x - M));
#pragma unroll
        for (int o = 16; o; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
        // log S = k ln 2 + log(f), f in [1, 2): fp32 serves for log(f), whose rounding
        // is then below 2^-24 whatever the size of S
        const long long bits = __double_as_longlong(S);
        const int k = static_cast<int>(bits >> 52) - 1023;
        const double f =
            __longlong_as_double((bits & 0xfffffffffffffll) | 0x3ff0000000000000ll);
        lse = static_cast<double>(M) + k * kLn2 + static_cast<double>(logf(static_cast<float>(f)));
      }
    }
    if (lane == 0) {
      sh_kind[w] = kind;
      sh_lse[w] = lse;
      sh_cum[w] = cum;
    }
  }
  __syncthreads();
  const int per_beam = p.chunks * p.n, total = p.W * per_beam;
  // entry i of the prompt's lists; false where there is none
  auto entry = [&](int i, Best& e) -> bool {
    const int w = i / per_beam, r = i - w * per_beam;
    const int kind = sh_kind[w];
    double s;
    if (kind == 2) {
      if (r != 0) return false;
      s = sh_cum[w];
      e.flat = w * p.V + p.pad;
    } else {
      if (kind == 0) return false;
      const unsigned long long k = p.cand[(static_cast<int64_t>(b) * p.W + w) * per_beam + r];
      if (k == 0) return false;
      const uint32_t o = static_cast<uint32_t>(k >> 32);
      const float x = __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
      s = sh_cum[w] + (static_cast<double>(x) - sh_lse[w]);
      e.flat = w * p.V + static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
    }
    e.score = order64(s + 0.0);
    return true;
  };
  auto value = [](unsigned long long o) {
    return __longlong_as_double(
        static_cast<long long>(o ^ ((o >> 63) ? 0x8000000000000000ull : ~0ull)));
  };
  // the bound, on the scores rounded down to fp32 (which keeps their order)
  uint32_t mine = 0;
  for (int i = threadIdx.x; i < total; i += kThreads) {
    Best e;
    if (entry(i, e)) mine = max(mine, order32(__double2float_rd(value(e.score))));
  }
  uint32_t top, tau;
  block_bound(mine, p.n, sh_key, top, tau);
  const uint32_t bound = tau > 0 ? tau : 1;
  if (mine >= bound) {
    for (int i = threadIdx.x; i < total; i += kThreads) {
      Best e;
      if (entry(i, e) && order32(__double2float_rd(value(e.score))) >= bound) {
        const int at = atomicAdd(&count, 1);
        if (at < kCap) list[at] = e;
      }
    }
  }
  __syncthreads();
  const int64_t o = static_cast<int64_t>(b) * p.n;
  auto put = [&](int rank, const Best& e) {
    p.parents[o + rank] = e.flat / p.V;
    p.tokens[o + rank] = e.flat % p.V;
    p.out_scores[o + rank] = static_cast<float>(value(e.score));
  };
  auto none = [&](int rank) {
    p.parents[o + rank] = -1;
    p.tokens[o + rank] = -1;
    p.out_scores[o + rank] = -INFINITY;
  };
  const int c = count;
  if (c <= kCap) {
    for (int i = threadIdx.x; i < c; i += kThreads) {
      const Best e = list[i];
      int rank = 0;
      for (int j = 0; j < c; ++j) rank += better(list[j], e) ? 1 : 0;
      if (rank < p.n) put(rank, e);
    }
    for (int i = c + threadIdx.x; i < p.n; i += kThreads) none(i);
  } else {
    Best last{~0ull, -1};
    for (int r = 0; r < p.n; ++r) {
      Best best{0, 0x7fffffff};
      for (int i = threadIdx.x; i < total; i += kThreads) {
        Best e;
        if (entry(i, e) && better(last, e) && better(e, best)) best = e;
      }
#pragma unroll
      for (int s = 16; s; s >>= 1) {
        Best y;
        y.score = __shfl_xor_sync(0xffffffffu, best.score, s);
        y.flat = __shfl_xor_sync(0xffffffffu, best.flat, s);
        if (better(y, best)) best = y;
      }
      __syncthreads();
      if (lane == 0) sh_best[warp] = best;
      __syncthreads();
      best = sh_best[0];
      for (int w = 1; w < kWarps; ++w)
        if (better(sh_best[w], best)) best = sh_best[w];
      last = best;
      if (threadIdx.x == 0) put(r, best);
    }
  }
}

}  // namespace

int beam_chunks(int V) {
  // a row may start up to 15 bytes past a 16-byte boundary: 7 logits of 16 bits
  return static_cast<int>((static_cast<int64_t>(V) + 7 + kChunk - 1) / kChunk);
}

cudaError_t launch_beam_select(const BeamParams& p, int dtype, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(p.B) * p.W * p.chunks));
  cudaError_t e;
  if (dtype == 0) e = launch_kernel(beam_scan_kernel<__half>, grid, dim3(kThreads), 0, stream, true, p);
  else if (dtype == 1)
    e = launch_kernel(beam_scan_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, true, p);
  else
    e = launch_kernel(beam_scan_kernel<float>, grid, dim3(kThreads), 0, stream, true, p);
  if (e != cudaSuccess) return e;
  return launch_kernel(beam_merge_kernel, dim3(static_cast<unsigned>(p.B)), dim3(kThreads), 0,
                       stream, true, p);
}

}  // namespace ps
