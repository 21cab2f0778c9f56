// Beam search's selection over beams and vocabulary: of the W * V continuations of a
// prompt's beams, with score(w, v) = cum_w + x_wv - lse_w (lse_w the log-sum-exp of beam
// w's logits), the n best, ties to the lowest beam and then the lowest token.
//
// One pass over the logits. Within a beam the order of the scores is the order of the
// logits, so a chunk's n best candidates are chosen on the logits alone, before lse is
// known; the few that are left are scored and compared across chunks and beams in 64 bits.
//   scan    one CTA per (beam, chunk of logits), streamed in 16-byte loads: each thread keeps
//           its maximum m and the sum of exp(x - m). The candidates are the logits at or
//           above a bound tau: the n-th largest of a warp's 32 thread maxima is at most the
//           n-th largest logit of the chunk, and tau is the largest such bound of the CTA's
//           warps. Where a thread's maximum of a round reaches tau, its warp reads those 32
//           logits again (from the caches); a few dozen pass, and are ranked.
//   merge   one CTA per prompt: lse of each beam from its chunks' (M, sum), then the same
//           bound on the chunks' candidates, and the ranks of those that pass.
// Bound by the bytes of the logits (read once).
#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRound = 32 * kThreads;  // logits of a CTA per round of loads, two in flight
constexpr int kRounds = 4;             // rounds, at most
constexpr int kCap = 1024;             // candidates ranked in shared memory
constexpr int kEarly = 2;              // entries a merging thread holds in registers
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
__device__ __forceinline__ float from_order32(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
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

// The elements of one 16-byte word as floats, NaN as -inf.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float* x);
template <>
__device__ __forceinline__ void unpack<float>(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = fmaxf(__uint_as_float(u[i]), -INFINITY);
}
template <>
__device__ __forceinline__ void unpack<__half>(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __hmax2(*reinterpret_cast<const __half2*>(&u[i]),
                              __half2half2(__ushort_as_half(0xfc00)));
    const float2 f = __half22float2(h);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&u[i]),
                                     __bfloat162bfloat162(__ushort_as_bfloat16(0xff80)));
    const float2 f = __bfloat1622float2(h);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(const BeamParams p) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  constexpr int kWords = kRound / kVec / kThreads;  // words of a thread per round
  static_assert(kWords * kVec == 32, "a round is 32 logits per thread, one per lane");
  __shared__ uint32_t sh_key[2 * kWarps];
  __shared__ float sh_sum[kWarps];
  __shared__ unsigned long long sh_max[kWarps];
  __shared__ unsigned long long list[kCap];
  __shared__ int count;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;
  if (p.finished != nullptr && p.finished[row]) {
    pdl_launch_dependents();
    return;
  }
  if (threadIdx.x == 0) count = 0;
  const T* base = static_cast<const T*>(p.logits) + row * p.ld;
  // words start at the 16-byte boundary at or before the row's first logit; `lo` is the
  // token of the chunk's first place (below 0 by the row's offset from that boundary)
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / sizeof(T));
  const int lo = chunk * p.chunk - skew;
  const int end = min(lo + p.chunk, p.V);  // one past the chunk's last token
  // the word at token t (a multiple of kVec past lo); outside the chunk -inf, not read
  auto load = [&](int t) -> uint4 {
    if (t >= 0 && t + kVec <= end) return __ldg(reinterpret_cast<const uint4*>(base + t));
    union {
      uint4 w;
      T e[kVec];
    } u;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      u.e[i] = t + i >= 0 && t + i < end ? base[t + i] : static_cast<T>(-INFINITY);
    return u.w;
  };
  // token of thread `thread`'s word j of round r
  auto place = [&](int r, int j, int thread) { return lo + r * kRound + (j * kThreads + thread) * kVec; };
  // one pass: the thread's maximum m, each round's own maximum, and the thread's sum of
  // exp(x - sub), sub = m but for -inf; the next round's words are on their way meanwhile
  float m = -INFINITY, sub = 0.f, mr[kRounds];
  float2 sum = make_float2(0.f, 0.f);
  uint4 w[kWords];
#pragma unroll
  for (int j = 0; j < kWords; ++j) w[j] = load(place(0, j, threadIdx.x));
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    mr[r] = -INFINITY;
    if (lo + r * kRound >= end) continue;
    uint4 next[kWords];
    const bool more = r + 1 < kRounds && lo + (r + 1) * kRound < end;
    if (more) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) next[j] = load(place(r + 1, j, threadIdx.x));
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      float x[kVec];
      unpack<T>(w[j], x);
#pragma unroll
      for (int i = 0; i < kVec; i += 2) mr[r] = fmax3(mr[r], x[i], x[i + 1]);
      if (mr[r] > m) {
        const float a = sum.x + sum.y > 0.f ? fast_exp2((sub - mr[r]) * kLog2e) : 0.f;
        sum = fmul2(sum, make_float2(a, a));
        m = sub = mr[r];
      }
      // (x - sub first: rounding sub log2(e) once for all terms would shift their sum)
      const float2 one = make_float2(1.f, 1.f), ns = make_float2(-sub, -sub);
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        const float2 y = fmul2(ffma2(make_float2(x[i], x[i + 1]), one, ns),
                               make_float2(kLog2e, kLog2e));
        sum = ffma2(make_float2(fast_exp2(y.x), fast_exp2(y.y)), one, sum);
      }
    }
    if (more) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) w[j] = next[j];
    }
  }
  uint32_t top, tau;
  block_bound(order32(clean(m)), p.n, sh_key, top, tau);
  const float M = from_order32(top);
  float s = m > -INFINITY ? (sum.x + sum.y) * fast_exp2((m - M) * kLog2e) : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sh_sum[warp] = s;
  // The candidates. A round of a thread is 32 logits: where its maximum reaches the bound,
  // the warp reads them again (from the caches), one per lane. f(key) is called for every
  // logit at or above the bound.
  const uint32_t bound = tau > kOrderNegInf ? tau : kOrderNegInf + 1;
  auto each = [&](auto f) {
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      uint32_t who = __ballot_sync(0xffffffffu, order32(clean(mr[r])) >= bound);
      for (; who; who &= who - 1) {
        const int t = place(r, lane / kVec, warp * 32 + __ffs(who) - 1) + lane % kVec;
        if (t < 0 || t >= end) continue;
        const uint32_t k = order32(clean(widen<T>(base[t])));
        if (k >= bound)
          f((static_cast<unsigned long long>(k) << 32) | (0xffffffffu - static_cast<uint32_t>(t)));
      }
    }
  };
  each([&](unsigned long long k) {
    const int at = atomicAdd(&count, 1);
    if (at < kCap) list[at] = k;
  });
  __syncthreads();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += sh_sum[i];
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
    for (int i = 0; i < p.n; ++i) {
      unsigned long long best = 0;
      each([&](unsigned long long k) {
        if (k < last && k > best) best = k;
      });
      last = block_max(best, sh_max);
      if (threadIdx.x == 0) out[i] = last;
    }
  }
}

// Scores are pairs of floats hi + lo (|lo| at most half a step of hi): cum + (x - lse) with
// 2^-46 of the largest of the three lost at most, in fp32 adds alone (fp64 runs at a small
// fraction of their rate here). Equal values give equal pairs, and pairs in the order of
// (hi, lo) are in the order of their values.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

// A candidate of the merge: its score's order and its flat index (beam * V + token).
struct Best {
  unsigned long long score;
  int flat;
};
__device__ __forceinline__ bool better(const Best& a, const Best& b) {
  return a.score > b.score || (a.score == b.score && a.flat < b.flat);
}

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamParams p) {
  __shared__ uint32_t sh_key[2 * kWarps];
  __shared__ float2 sh_lse[kBeamMaxWidth];  // hi, lo
  __shared__ float sh_cum[kBeamMaxWidth];
  __shared__ int sh_kind[kBeamMaxWidth];  // 0 no candidate, 1 scored, 2 finished
  __shared__ Best list[kCap];
  __shared__ Best sh_best[kWarps];
  __shared__ int count;
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) count = 0;
  const int per_beam = p.chunks * p.n, total = p.W * per_beam;
  const unsigned long long* cand = p.cand + static_cast<int64_t>(b) * total;
  pdl_wait();
  // the thread's first entries, read beside the chunks' sums
  unsigned long long early[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const int i = threadIdx.x + k * kThreads;
    early[k] = i < total ? cand[i] : 0;
  }
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
      const float hi = static_cast<float>(lse);
      sh_lse[w] = make_float2(hi, static_cast<float>(lse - hi));
      sh_cum[w] = cum;
    }
  }
  __syncthreads();
  // entry i (logit and token k) of the prompt's lists; false where there is none
  auto entry = [&](int i, unsigned long long k, Best& e) -> bool {
    const int w = i / per_beam, r = i - w * per_beam;
    const int kind = sh_kind[w];
    float hi, lo = 0.f;
    if (kind == 2) {
      if (r != 0) return false;
      hi = sh_cum[w];
      e.flat = w * p.V + p.pad;
    } else {
      if (kind == 0) return false;
      if (k == 0) return false;
      const float x = from_order32(static_cast<uint32_t>(k >> 32));
      float d, e1, t, e2;
      two_sum(x, -sh_lse[w].x, d, e1);
      two_sum(sh_cum[w], d, t, e2);
      const float rest = __fadd_rn(e2, __fsub_rn(e1, sh_lse[w].y));
      two_sum(t, rest, hi, lo);
      e.flat = w * p.V + static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
    }
    e.score = (static_cast<unsigned long long>(order32(hi + 0.f)) << 32) | order32(lo + 0.f);
    return true;
  };
  // the bound, on the scores' high parts
  // f(entry) for each of the thread's entries
  auto each = [&](auto f) {
#pragma unroll
    for (int k = 0; k < kEarly; ++k) {
      const int i = threadIdx.x + k * kThreads;
      Best e;
      if (i < total && entry(i, early[k], e)) f(e);
    }
    for (int i = threadIdx.x + kEarly * kThreads; i < total; i += kThreads) {
      Best e;
      if (entry(i, cand[i], e)) f(e);
    }
  };
  uint32_t mine = 0;
  each([&](const Best& e) { mine = max(mine, static_cast<uint32_t>(e.score >> 32)); });
  uint32_t top, tau;
  block_bound(mine, p.n, sh_key, top, tau);
  const uint32_t bound = tau > 0 ? tau : 1;
  if (mine >= bound) {
    each([&](const Best& e) {
      if (static_cast<uint32_t>(e.score >> 32) >= bound) {
        const int at = atomicAdd(&count, 1);
        if (at < kCap) list[at] = e;
      }
    });
  }
  __syncthreads();
  const int64_t o = static_cast<int64_t>(b) * p.n;
  auto put = [&](int rank, const Best& e) {
    p.parents[o + rank] = e.flat / p.V;
    p.tokens[o + rank] = e.flat % p.V;
    p.out_scores[o + rank] = from_order32(static_cast<uint32_t>(e.score >> 32));
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
      each([&](const Best& e) {
        if (better(last, e) && better(e, best)) best = e;
      });
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

// Logits per CTA, a multiple of a round's share that fills the SMs a few times over: long
// chunks spread a CTA's fixed costs (the bound, the ranks, its launch) over more bytes, short
// ones keep a small batch's rows on many SMs.
int beam_chunk(int64_t rows, int V) {
  constexpr int64_t kStep = 2048, kTargetCtas = 1216;  // 8 a SM on 152 SMs
  int64_t c = (rows * V / kTargetCtas + kStep - 1) / kStep * kStep;
  c = c < kStep ? kStep : c > kRounds * kRound ? kRounds * kRound : c;
  return static_cast<int>(c);
}

int beam_chunks(int64_t rows, int V) {
  // a row may start up to 14 bytes past a 16-byte boundary: 7 logits of 16 bits
  const int c = beam_chunk(rows, V);
  return static_cast<int>((static_cast<int64_t>(V) + 7 + c - 1) / c);
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
