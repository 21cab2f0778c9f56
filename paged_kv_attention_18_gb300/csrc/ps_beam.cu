// Beam search's selection over beams and vocabulary: of the W * V continuations of a
// prompt's beams, with score(w, v) = cum_w + x_wv - lse_w (lse_w the log-sum-exp of beam
// w's logits), the n best, ties to the lowest beam and then the lowest token.
//
// One pass over the logits. Within a beam the order of the scores is the order of the
// logits, so a chunk's n best candidates are chosen on the logits alone, before lse is
// known; the few that are left are scored and compared across chunks and beams in 64 bits.
//   scan    one CTA per (beam, chunk of logits), streamed in 16-byte loads: each thread keeps
//           its maximum m and the sum of exp(x - m). The candidates are the logits at or
//           above a bound tau, the n-th largest of the threads' maxima: at most the n-th
//           largest logit of the chunk. Where a thread's maximum of a round reaches tau, a
//           warp reads those logits again (from the caches); little more than n pass, and
//           are ranked.
//   merge   one CTA per prompt: lse of each beam from its chunks' (M, sum), then the same
//           bound on the chunks' candidates, and the ranks of those that pass.
// Bound by the bytes of the logits (read once): 192 rows of 151936 bf16 logits (58 MB) scan in
// 17.5 us, of which 13 us are the stream (4.5 TB/s), 3 the bound and 1 the candidates; the
// merge of 48 prompts adds 3 to 4 us behind it. Listing candidates from the registers in the
// stream, against a bound from its first round, took 24 us: the few lanes that have one stop
// their warps every round.
#include <type_traits>

#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxChunk = 65536;       // logits of a CTA, at most
constexpr int kWords = 4;              // 16-byte words of a thread per round
constexpr int kDepth = 2;              // rounds in flight
constexpr int kRingBytes = kDepth * kWords * kThreads * 16;
constexpr int kCap = 512;              // candidates ranked in shared memory
constexpr int kPairs = 256;            // rounds of threads looked at again, at most
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

// Block-wide: the largest of the threads' keys (each above 0) and the n-th largest, n in
// 1 .. 32. Each warp sorts its keys; of the 8 n largest that leaves, those with fewer than n
// above them are the block's n largest (equal ones included). (A looser bound
// from two keys of each warp costs 2 us less, and 4 us more in candidates looked at.)
struct BoundSmem {
  alignas(16) uint32_t top[kWarps * kBeamMaxWidth];
  uint32_t tau;
};
__device__ __forceinline__ void block_bound(uint32_t key, int n, BoundSmem& sh, uint32_t& top,
                                            uint32_t& tau) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) sh.tau = 0xffffffffu;
  // the warp's keys in falling order (a bitonic network)
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j; j >>= 1) {
      const uint32_t y = __shfl_xor_sync(0xffffffffu, key, j);
      key = ((lane & j) == 0) == ((lane & k) == 0) ? max(key, y) : min(key, y);
    }
  if (lane < n) sh.top[warp * n + lane] = key;
  __syncthreads();
  top = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = max(top, sh.top[w * n]);
  if (threadIdx.x < kWarps * n) {
    const uint32_t k = sh.top[threadIdx.x];
    int above = 0;
#pragma unroll 4
    for (int i = 0; i < kWarps / 4 * n; ++i) {
      const uint4 t = reinterpret_cast<const uint4*>(sh.top)[i];
      above += (t.x > k) + (t.y > k) + (t.z > k) + (t.w > k);
    }
    if (above < n) atomicMin(&sh.tau, k);
  }
  __syncthreads();
  tau = sh.tau;
}

// done(i, rank) for each i < n, rank the number of j < n with above(i, j): eight threads an i.
template <class Above, class Done>
__device__ __forceinline__ void rank_list(int n, Above above, Done done) {
  const int part = threadIdx.x & 7;
  for (int i0 = 0; i0 < n; i0 += kThreads / 8) {
    const int i = i0 + (threadIdx.x >> 3);
    int rank = 0;
    if (i < n)
      for (int j = part; j < n; j += 8) rank += above(i, j) ? 1 : 0;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (part == 0 && i < n) done(i, rank);
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

// The elements of one 32-bit word as floats (one of fp32, two of a 16-bit type).
template <typename T>
__device__ __forceinline__ void unpack(uint32_t u, float* x);
template <>
__device__ __forceinline__ void unpack<float>(uint32_t u, float* x) { x[0] = __uint_as_float(u); }
template <>
__device__ __forceinline__ void unpack<__half>(uint32_t u, float* x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
  x[0] = f.x;
  x[1] = f.y;
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(uint32_t u, float* x) {
  x[0] = __uint_as_float(u << 16);
  x[1] = __uint_as_float(u & 0xffff0000u);
}

// The largest element of 16 such words; NaN only where all are.
template <typename T>
__device__ __forceinline__ float words_max(const uint32_t* w) {
  if constexpr (sizeof(T) == 4) {
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = fmax3(__uint_as_float(w[k]), __uint_as_float(w[4 + k]), __uint_as_float(w[8 + k]));
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], __uint_as_float(w[12 + k]));
    return fmax3(fmaxf(m[0], m[1]), m[2], m[3]);
  } else {
    using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    T2 m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = *reinterpret_cast<const T2*>(w + k);
#pragma unroll
    for (int i = 4; i < 16; i += 4)
#pragma unroll
      for (int k = 0; k < 4; ++k) m[k] = __hmax2(m[k], *reinterpret_cast<const T2*>(w + i + k));
    const T2 x = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
    return fmaxf(widen<T>(x.x), widen<T>(x.y));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(const BeamParams p) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  constexpr int kPer = kWords * kVec;  // logits of a thread per round
  constexpr int kRound = kPer * kThreads, kRounds = kMaxChunk / kRound;
  static_assert(kPer <= 32, "a warp looks at a thread's round again one logit per lane");
  __shared__ BoundSmem sh_key;
  __shared__ float sh_sum[kWarps], sh_round[kRounds][kThreads];
  __shared__ unsigned long long sh_max[kWarps];
  __shared__ unsigned long long list[kCap];
  __shared__ int count, pairs, pair[kPairs];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;
  if (p.finished != nullptr && p.finished[row]) {
    pdl_launch_dependents();
    return;
  }
  if (threadIdx.x == 0) {
    count = pairs = 0;
  }
  const T* base = static_cast<const T*>(p.logits) + row * p.ld;
  // words start at the 16-byte boundary at or before the row's first logit; `lo` is the
  // token of the chunk's first place (below 0 by the row's offset from that boundary)
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / sizeof(T));
  const int lo = chunk * p.chunk - skew;
  const int end = min(lo + p.chunk, p.V);  // one past the chunk's last token
  const int rounds = end > lo ? (end - lo + kRound - 1) / kRound : 0;
  // token of thread `thread`'s word j of round r
  auto place = [&](int r, int j, int thread) { return lo + r * kRound + (j * kThreads + thread) * kVec; };
  // Each thread's words go through its own slots of a ring in shared memory, kDepth rounds
  // deep, by asynchronous copies that it alone waits for and reads (no barrier). Outside the
  // chunk nothing is read and a slot holds -inf.
  extern __shared__ uint4 ring[];  // [kDepth][kWords][kThreads]
  auto fetch = [&](int r) {
    if (r < rounds) {
      uint4* slot = ring + (r % kDepth) * kWords * kThreads + threadIdx.x;
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        const int t = place(r, j, threadIdx.x);
        if (t >= 0 && t + kVec <= end) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           smem_u32(slot + j * kThreads)),
                       "l"(base + t)
                       : "memory");
        } else {
          T* e = reinterpret_cast<T*>(slot + j * kThreads);
#pragma unroll 1
          for (int i = 0; i < kVec; ++i)
            e[i] = t + i >= 0 && t + i < end ? base[t + i] : static_cast<T>(-INFINITY);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int r = 0; r < kDepth; ++r) fetch(r);
  // One pass. m: the thread's maximum; sum: of 2^((x + c) L), L = log2(e) in fp32, c = -m (0
  // before the first logit above -inf). The difference comes first: it is 0 at the maximum and
  // rounded by 2^-24 of itself elsewhere, whatever the logits' size, where x L - m L in one
  // fused operation is off by m L's rounding, 2^8 and more from |m| = 2^31 on, and overflows at
  // masks of the type's least value. (The rounds are not unrolled: straight-line code for all
  // of them ran at the rate of its instruction fetches. A round's maximum is kept in shared
  // memory.)
  float m = -INFINITY, c = 0.f;
  float2 sum = make_float2(0.f, 0.f);
  const float2 l2 = make_float2(kLog2e, kLog2e), one2 = make_float2(1.f, 1.f);
#pragma unroll 1
  for (int r = 0; r < rounds; ++r) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    uint4 w[kWords];
    const uint4* slot = ring + (r % kDepth) * kWords * kThreads + threadIdx.x;
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = slot[j * kThreads];
    fetch(r + kDepth);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(w);
    const float mr = fmaxf(words_max<T>(words), -INFINITY);
    sh_round[r][threadIdx.x] = mr;
    if (mr > m) {
      const float a = fast_exp2((m - mr) * kLog2e);  // (0 from -inf, whose sum is 0)
      sum = fmul2(sum, make_float2(a, a));
      m = mr;
      c = -m;
    }
    const float2 c2 = make_float2(c, c);
    float2 add[2] = {sum, make_float2(0.f, 0.f)};
    constexpr int kStep = sizeof(T) == 4 ? 2 : 1;  // words of a pair of logits
#pragma unroll
    for (int i = 0; i < 4 * kWords; i += kStep) {
      float x[2];
      if constexpr (sizeof(T) == 4) {
        x[0] = __uint_as_float(words[i]);
        x[1] = __uint_as_float(words[i + 1]);
      } else {
        unpack<T>(words[i], x);
      }
      const float2 y = fmul2(ffma2(make_float2(x[0], x[1]), one2, c2), l2);
      add[i / kStep % 2].x += fast_exp2(y.x);
      add[i / kStep % 2].y += fast_exp2(y.y);
    }
    sum = make_float2(add[0].x + add[1].x, add[0].y + add[1].y);
  }
  float total = sum.x + sum.y;
  if (total != total && m < INFINITY) {
    // a NaN among the thread's logits, which counts as -inf: the sum again without it
    total = 0.f;
    for (int r = 0; r < rounds; ++r)
      for (int j = 0; j < kWords; ++j)
        for (int i = 0; i < kVec; ++i) {
          const int t = place(r, j, threadIdx.x) + i;
          if (t >= 0 && t < end) total += fast_exp2((clean(widen<T>(base[t])) + c) * kLog2e);
        }
  }
  uint32_t top, tau;
  block_bound(order32(clean(m)), p.n, sh_key, top, tau);
  const float M = from_order32(top);
  float s = m > -INFINITY ? total * fast_exp2((m - M) * kLog2e) : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) sh_sum[warp] = s;
  // The candidates. The rounds of threads whose maximum reaches the bound are listed; a warp
  // reads a listed round's logits again (from the caches), one per lane, the rounds dealt to
  // the warps so that their reads are on the way together.
  const uint32_t bound = tau > kOrderNegInf ? tau : kOrderNegInf + 1;
  for (int r = 0; r < rounds; ++r)
    if (order32(clean(sh_round[r][threadIdx.x])) >= bound) {
      const int at = atomicAdd(&pairs, 1);
      if (at < kPairs) pair[at] = r * kThreads + threadIdx.x;
    }
  __syncthreads();
  const int n_pairs = pairs;
  // key of the lane's logit of pair x, 0 where there is none at or above the bound
  auto look = [&](int x) -> unsigned long long {
    const int t = place(x / kThreads, lane / kVec, x % kThreads) + lane % kVec;
    if (lane >= kPer || t < 0 || t >= end) return 0;
    const uint32_t k = order32(clean(widen<T>(base[t])));
    return k < bound ? 0
                     : (static_cast<unsigned long long>(k) << 32) |
                           (0xffffffffu - static_cast<uint32_t>(t));
  };
  auto put = [&](unsigned long long k) {
    if (k == 0) return;
    const int at = atomicAdd(&count, 1);
    if (at < kCap) list[at] = k;
  };
  constexpr int kLooks = 4;  // pairs of a warp on the way together
  for (int i = warp; i < n_pairs && n_pairs <= kPairs; i += kLooks * kWarps) {
    unsigned long long k[kLooks];
#pragma unroll
    for (int u = 0; u < kLooks; ++u)
      k[u] = i + u * kWarps < n_pairs ? look(pair[i + u * kWarps]) : 0;
#pragma unroll
    for (int u = 0; u < kLooks; ++u) put(k[u]);
  }
  __syncthreads();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += sh_sum[i];
    p.stat[blockIdx.x] = make_float2(M, s);
  }
  unsigned long long* out = p.cand + static_cast<int64_t>(blockIdx.x) * p.n;
  const int found = count;
  if (n_pairs <= kPairs && found <= kCap) {
    rank_list(found, [&](int i, int j) { return list[j] > list[i]; },
              [&](int i, int rank) {
                if (rank < p.n) out[rank] = list[i];
              });
    for (int i = found + threadIdx.x; i < p.n; i += kThreads) out[i] = 0;  // none
  } else {
    // more equal logits than the lists hold: n rounds of the block's largest key below the
    // one before
    unsigned long long last = ~0ull;
    for (int i = 0; i < p.n; ++i) {
      unsigned long long best = 0;
      for (int r = 0; r < rounds; ++r)
        for (int t = 0; t < 32; ++t) {
          if (order32(clean(sh_round[r][warp * 32 + t])) < bound) continue;  // (warp-uniform)
          const unsigned long long k = look(r * kThreads + warp * 32 + t);
          if (k < last && k > best) best = k;
        }
      last = block_max(best, sh_max);
      if (threadIdx.x == 0) out[i] = last;
    }
  }
}

// Scores are pairs of floats hi + lo (|lo| at most half a step of hi): cum + (x - M - log S),
// lse = M + log S, with 2^-46 of the largest of x - M, cum and log S lost at most, in fp32 adds
// alone (fp64 runs at a small fraction of their rate here). Equal values give equal pairs, and
// pairs in the order of (hi, lo) are in the order of their values. A sum below fp32's range (a
// masked logit of a beam that is masked itself) is -inf, behind every other.
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
  __shared__ BoundSmem sh_key;
  __shared__ float sh_M[kBeamMaxWidth];     // the beam's largest logit
  __shared__ float2 sh_cum[kBeamMaxWidth];  // cum - log S (a finished beam: cum): hi, lo
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
    float M = 0.f;
    float2 from = make_float2(cum, 0.f);
    if (kind == 1) {
      const float2* st = p.stat + static_cast<int64_t>(row) * p.chunks;
      M = -INFINITY;
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
        // is then below 2^-24 whatever the size of S (1 at least: the largest logit's term)
        const long long bits = __double_as_longlong(S);
        const int k = static_cast<int>(bits >> 52) - 1023;
        const double f =
            __longlong_as_double((bits & 0xfffffffffffffll) | 0x3ff0000000000000ll);
        const double log_s = k * kLn2 + static_cast<double>(logf(static_cast<float>(f)));
        const float hi = static_cast<float>(log_s);
        two_sum(cum, -hi, from.x, from.y);
        from.y = __fsub_rn(from.y, static_cast<float>(log_s - hi));
      }
    }
    if (lane == 0) {
      sh_kind[w] = kind;
      sh_M[w] = M;
      sh_cum[w] = from;
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
      hi = sh_cum[w].x;
      e.flat = w * p.V + p.pad;
    } else {
      if (kind == 0) return false;
      if (k == 0) return false;
      const float x = from_order32(static_cast<uint32_t>(k >> 32));
      float d, e1, t, e2;
      two_sum(x, -sh_M[w], d, e1);
      two_sum(sh_cum[w].x, d, t, e2);
      const float rest = __fadd_rn(e2, __fadd_rn(e1, sh_cum[w].y));
      two_sum(t, rest, hi, lo);
      if (!(hi > -INFINITY)) {
        hi = -INFINITY;
        lo = 0.f;
      }
      e.flat = w * p.V + static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
    }
    e.score = (static_cast<unsigned long long>(order32(hi + 0.f)) << 32) | order32(lo + 0.f);
    return true;
  };
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
  // few entries are ranked all of them; of many, those whose high part reaches a bound
  uint32_t mine = 0, bound = 1;
  if (total > kCap) {
    each([&](const Best& e) { mine = max(mine, static_cast<uint32_t>(e.score >> 32)); });
    uint32_t top, tau;
    block_bound(mine, p.n, sh_key, top, tau);
    bound = tau > 0 ? tau : 1;
  }
  if (mine >= bound || total <= kCap) {
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
    rank_list(c, [&](int i, int j) { return better(list[j], list[i]); },
              [&](int i, int rank) {
                if (rank < p.n) put(rank, list[i]);
              });
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

// Logits per CTA: a row's equal shares (multiples of kStep) in as many chunks as keep the CTAs
// to one wave (four an SM), but at least kStep and at most kMaxChunk logits. A CTA's fixed
// costs (launch, bound, ranks: some 4 us) are then paid once.
int beam_chunk(int64_t rows, int V) {
  constexpr int64_t kStep = 2048, kWave = 608;
  const int64_t places = static_cast<int64_t>(V) + 7;  // the row's offset from a boundary
  int64_t n = rows > 0 && rows < kWave ? kWave / rows : 1;
  const int64_t least = (places + kMaxChunk - 1) / kMaxChunk;
  if (n < least) n = least;
  return static_cast<int>(((places + n - 1) / n + kStep - 1) / kStep * kStep);
}

int beam_chunks(int64_t rows, int V) {
  // a row may start up to 14 bytes past a 16-byte boundary: 7 logits of 16 bits
  const int c = beam_chunk(rows, V);
  return static_cast<int>((static_cast<int64_t>(V) + 7 + c - 1) / c);
}

template <typename T>
static cudaError_t launch_scan(const BeamParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_smem_limit(beam_scan_kernel<T>, kRingBytes, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(p.B) * p.W * p.chunks));
  return launch_kernel(beam_scan_kernel<T>, grid, dim3(kThreads), kRingBytes, stream, true, p);
}

cudaError_t launch_beam_select(const BeamParams& p, int dtype, cudaStream_t stream) {
  const cudaError_t e = dtype == 0   ? launch_scan<__half>(p, stream)
                        : dtype == 1 ? launch_scan<__nv_bfloat16>(p, stream)
                                     : launch_scan<float>(p, stream);
  if (e != cudaSuccess) return e;
  return launch_kernel(beam_merge_kernel, dim3(static_cast<unsigned>(p.B)), dim3(kThreads), 0,
                       stream, true, p);
}

}  // namespace ps
