// Sampling: one token of every row of logits x, by temperature T, top-k, top-p and min-p, from
// a given random word R.
//
//     w_v = exp((x_v - max x) / T)          the order: x falling, then v rising
//     S_k: the first k.  nucleus: those of S_k whose predecessors' weights sum to less than
//     top_p times S_k's sum.  min-p: w_v >= min_p.  All three keep a prefix of the order.
//     Z = sum of the kept weights; the token is the first kept v, in the vocabulary's order,
//     whose running sum exceeds floor(R Z / 2^32).
//
// The token is a decision between neighbours whose borders lie as close as the smallest
// weight, so sums must not depend on an order and weights need more bits than fp32 has:
// with 2^17 tokens an error of 2^-24 in each border would change one draw in hundreds.
// A weight is a 64-bit fixed-point number (2^scale for the largest; scale leaves room for V of
// them), from exp2 in two floats: the difference x - max and its product with log2(e) / T are
// each kept as a sum of two floats, 2^(j/64) comes from a table, the rest (at most 2^(1/128))
// from three terms of its series, all within about 2^-30. Integer sums are exact in any order.
//
// A cluster takes a row, a slice of it in each CTA's shared memory, read from memory once; the
// first CTA decides, the others leave as soon as it has what it needs of them. By what the row
// asks for:
//   - the largest logit alone: its first place;
//   - top-k: the k-th largest of the threads' maxima bounds the k-th logit from below; the few
//     logits from the bound on are listed, and the list, sorted, decides everything;
//   - top-p without it: one pass takes the sum of all weights and counts the logits by weight
//     (32 bins a factor of two). The border's bin follows from the counts with each bin's middle
//     weight; a second pass sums the weights above that bin exactly and lists those around it.
//     The list, sorted, has the border, which the exact sums confirm, or a next bin is tried. A
//     nucleus that fits the list is listed whole;
//   - none of these: the sum of all weights (from min-p's border on), by warps; the word's point
//     lies in one warp's logits, which the first CTA reads again;
//   - what fits none (a list that overflows, as with equal logits everywhere; k beyond 1024; T
//     beyond 2^100): the border digit by digit, by histograms of places and exact weights.
#include <cooperative_groups.h>

#include <cfloat>

#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 2048;           // places that a row's list holds
constexpr int kShort = kThreads;      // places that sort in a fraction of the time
constexpr int kMaxTopK = 1024;        // k up to which the threads' maxima bound it
constexpr int kMaxCluster = 8;
constexpr int kSmemLimit = 232448;    // of a CTA
constexpr int kSmemTwo = 113 * 1024;  // of each of two on an SM
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: added, a float's low bits are its integer
constexpr int kMagicBits = 0x4b400000;
constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.9259629911266175e-08f;

// 2^31 * 2^(j / 64), rounded
__constant__ uint32_t kExp2Table[64] = {
    0x80000000u, 0x8164d1f4u, 0x82cd8699u, 0x843a28c4u, 0x85aac368u, 0x871f6197u,
    0x88980e81u, 0x8a14d575u, 0x8b95c1e4u, 0x8d1adf5bu, 0x8ea4398bu, 0x9031dc43u,
    0x91c3d374u, 0x935a2b2fu, 0x94f4efa9u, 0x96942d37u, 0x9837f052u, 0x99e04593u,
    0x9b8d39bau, 0x9d3ed9a7u, 0x9ef53261u, 0xa0b05110u, 0xa2704303u, 0xa43515aeu,
    0xa5fed6aau, 0xa7cd93b5u, 0xa9a15ab5u, 0xab7a39b6u, 0xad583eeau, 0xaf3b78adu,
    0xb123f582u, 0xb311c413u, 0xb504f334u, 0xb6fd91e3u, 0xb8fbaf47u, 0xbaff5ab2u,
    0xbd08a39fu, 0xbf1799b6u, 0xc12c4ccau, 0xc346ccdau, 0xc5672a11u, 0xc78d74c9u,
    0xc9b9bd86u, 0xcbec14ffu, 0xce248c15u, 0xd06333dbu, 0xd2a81d92u, 0xd4f35aacu,
    0xd744fccbu, 0xd99d15c2u, 0xdbfbb798u, 0xde60f482u, 0xe0ccdeecu, 0xe33f8973u,
    0xe5b906e7u, 0xe8396a50u, 0xeac0c6e8u, 0xed4f301fu, 0xefe4b99cu, 0xf281773cu,
    0xf5257d15u, 0xf7d0df73u, 0xfa83b2dbu, 0xfd3e0c0du};

// A token's place in the order, larger first: its logit's bits made to ascend, then the index
// made to descend.
constexpr int kIdxBits = 20;
constexpr uint32_t kIdxMask = (1u << kIdxBits) - 1;
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t place(uint32_t key, int v) {
  return static_cast<uint64_t>(key) << kIdxBits | (kIdxMask - v);
}
__device__ __forceinline__ float logit_at(uint64_t at) {
  return of_key(static_cast<uint32_t>(at >> kIdxBits));
}
__device__ __forceinline__ int token_at(uint64_t at) {
  return static_cast<int>(kIdxMask - (static_cast<uint32_t>(at) & kIdxMask));
}
constexpr uint32_t kLowestKey = 0x00800000u;  // the least finite float's (-inf, NaN: below)

template <int kType>  // 0 fp16, 1 bf16, 2 fp32
struct Elem {
  using Bits = uint16_t;
  static constexpr int kVec = 8;  // in 16 bytes
  static constexpr uint32_t kNone = kType == 1 ? 0xff80ff80u : 0xfc00fc00u;  // -inf
};
template <>
struct Elem<2> {
  using Bits = uint32_t;
  static constexpr int kVec = 4;
  static constexpr uint32_t kNone = 0xff800000u;
};

// Element e of a 16-byte vector; NaN counts as -inf, -0 as 0.
template <int kType>
__device__ __forceinline__ float element(const uint4& v, int e) {
  const uint32_t* w = &v.x;
  float x;
  if constexpr (kType == 2) x = __uint_as_float(w[e]);
  else if constexpr (kType == 1) x = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  else x = __half2float(__ushort_as_half(static_cast<unsigned short>(w[e / 2] >> (e & 1) * 16)));
  return fmaxf(x + 0.f, -INFINITY);
}

// Elements e and e + 1 as they are, for their weights (NaN and -inf weigh nothing, -0 as 0).
template <int kType>
__device__ __forceinline__ float2 pair(const uint4& v, int e) {
  const uint32_t* w = &v.x;
  if constexpr (kType == 2) return make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]));
  else if constexpr (kType == 1)
    return make_float2(__uint_as_float(w[e / 2] << 16), __uint_as_float(w[e / 2] & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w[e / 2]));
}

// The largest element of a vector (NaN counts as -inf).
template <int kType>
__device__ __forceinline__ float vector_max(const uint4& v) {
  if constexpr (kType == 2) {
    return fmaxf(fmax3(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z)),
                 fmaxf(__uint_as_float(v.w), -INFINITY));
  } else if constexpr (kType == 1) {
    auto h = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    const float2 f = __bfloat1622float2(__hmax2(__hmax2(h(v.x), h(v.y)), __hmax2(h(v.z), h(v.w))));
    return fmax3(f.x, f.y, -INFINITY);
  } else {
    auto h = [](uint32_t x) { return *reinterpret_cast<const __half2*>(&x); };
    const float2 f = __half22float2(__hmax2(__hmax2(h(v.x), h(v.y)), __hmax2(h(v.z), h(v.w))));
    return fmax3(f.x, f.y, -INFINITY);
  }
}

struct Row {
  float max;      // the row's largest logit (times s)
  float c, c_lo;  // log2(e) / T (over s) as two floats
  float s;        // 1, or 1/4 where differences would overflow beside T
  float limit;    // from this y on (scale + 2) a weight rounds to 0; the largest is 2^scale
  uint32_t down;  // 60 - scale, and what kMagicBits adds to an exponent
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Where two logits lie below the maximum: y = (max - x) log2(e) / T >= 0, as a float, and -64 y
// rounded to a whole number (as kMagic holds it; of no use from y = 2^16 on).
struct Below {
  float2 d, y, t;
};
__device__ __forceinline__ Below below(float2 x, const Row& r) {
  Below b;
  b.d = ffma2(x, both(-1.f), both(r.max));
  b.y = fmul2(b.d, both(r.c));
  b.t = ffma2(b.y, both(-64.f), both(kMagic));
  return b;
}
// Counting bin: 32 a factor of two, 64 factors; the last one takes the rest. Never falls as x does.
__device__ __forceinline__ int bin_of(float t) {  // y below 63.9
  return (kMagicBits - static_cast<int>(__float_as_uint(t))) >> 1;
}

// The weights of two logits.
template <int kType>
__device__ __forceinline__ void weights(float2 x, const Below& b, const Row& r,
                                        const uint32_t* table, uint64_t* w) {
  // -y = zh + zl: what the product and, in fp32, the difference were rounded by is kept. (The
  // differences of two 16-bit values are exact but for logits thousands of times smaller than
  // the maximum, whose error is 2^-24 of the difference and random.)
  float2 zl = ffma2(b.d, both(-r.c), b.y);
  zl = ffma2(b.d, both(-r.c_lo), zl);
  if constexpr (kType == 2) {
    const float2 q = ffma2(both(r.max), both(-1.f), b.d);
    const float2 e1 = ffma2(ffma2(q, both(-1.f), b.d), both(-1.f), both(r.max));
    const float2 err = ffma2(ffma2(x, both(1.f), q), both(-1.f), e1);
    zl = ffma2(err, both(-r.c), zl);
  }
  const float2 m = ffma2(both(kMagic), both(-1.f), b.t);
  const float2 s = ffma2(ffma2(m, both(1.f / 64.f), b.y), both(-1.f), zl);
  float2 q = ffma2(s, both(0.05550410866f), both(0.2402265070f));
  q = ffma2(s, q, both(0.6931471806f));
  q = fmul2(s, q);
  const float2 f = ffma2(q, both(536870912.f), both(kMagic));
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t bits = __float_as_uint(e ? b.t.y : b.t.x);  // (kMagicBits is a multiple of 64)
    uint32_t fi = __float_as_uint(e ? f.y : f.x) - (kMagicBits - (1u << 29));
    // from here on a weight rounds to 0 (and not a number: -inf, NaN): 0 whatever the shift
    if (!((e ? b.y.y : b.y.x) < r.limit)) fi = 0;
    const uint32_t down = r.down - (bits >> 6);  // 63 at most
    uint64_t half, p;
    asm("shl.b64 %0, %1, %2;" : "=l"(half) : "l"(1ull), "r"(down - 1));
    asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(p) : "r"(table[bits & 63]), "r"(fi), "l"(half));
    asm("shr.b64 %0, %1, %2;" : "=l"(w[e]) : "l"(p), "r"(down));
  }
}
template <int kType>
__device__ __forceinline__ uint64_t weight(float x, const Row& r, const uint32_t* table) {
  uint64_t w[2];
  const float2 xx = both(x * r.s);
  weights<kType>(xx, below(xx, r), r, table, w);
  return w[0];
}

// A copy of whole 16-byte words, global to shared, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// What the CTAs of a cluster show one another.
struct alignas(16) Shared {
  uint32_t count[kBins];
  unsigned long long list[kList];                  // places, in any order; or masses of bins
  unsigned long long sums[kMaxCluster * kWarps];   // (first CTA) every warp's kept weights
  unsigned long long warp[kWarps];
  unsigned long long total, found[2];
  uint32_t table[64];
  float max, edge[2];
  double fall;     // T ln(min_p)
  uint32_t least;  // the key of min-p's border
  int listed, state, at, guess[2];
  uint64_t arrived[kWarps];  // barriers of the warps' copies
};
static_assert(sizeof(Shared) % 16 == 0, "the slice behind it is read in 16-byte words");

// Inclusive sums over the block's threads, in their order.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, unsigned long long* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps - 1; ++w) v += w < warp ? sh[w] : 0;
  return v;
}
__device__ __forceinline__ uint64_t block_sum(uint64_t v, unsigned long long* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += sh[w];
  return v;
}

// The threads that settle a list: a warp, or the block. Element j * kSize + i in v[j] of thread i.
struct WarpGroup {
  static constexpr int kSize = 32;
  __device__ static int self() { return threadIdx.x & 31; }
  __device__ static void sync() { __syncwarp(); }
  __device__ static int count(bool x) { return __popc(__ballot_sync(0xffffffffu, x)); }
  __device__ static uint64_t scan(uint64_t v, unsigned long long*) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (self() >= o) v += y;
    }
    return v;
  }
};
struct BlockGroup {
  static constexpr int kSize = kThreads;
  __device__ static int self() { return threadIdx.x; }
  __device__ static void sync() { __syncthreads(); }
  __device__ static int count(bool x) { return __syncthreads_count(x); }
  __device__ static uint64_t scan(uint64_t v, unsigned long long* sh) { return block_scan(v, sh); }
};

// A bitonic sort, falling, of the first `size` values (a power of two, 32 at least).
template <class Group, int kPer>
__device__ __forceinline__ void sort_falling(uint64_t* v, int size, unsigned long long* sh) {
  constexpr int kSize = Group::kSize;
  const int me = Group::self();
#pragma unroll 1
  for (int k = 2; k <= size; k <<= 1) {
#pragma unroll 1
    for (int s = k >> 1; s > 0; s >>= 1) {
      if (s >= kSize) {
        const int js = s / kSize;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
#pragma unroll
          for (int o = j + 1; o < kPer; ++o) {
            if ((j ^ o) != js) continue;
            const bool up = ((j * kSize + me) & k) == 0;
            if ((v[j] < v[o]) == up) {
              const uint64_t y = v[j];
              v[j] = v[o];
              v[o] = y;
            }
          }
        }
        continue;
      }
      uint64_t other[kPer];
      if (s >= 32) {
        Group::sync();
#pragma unroll
        for (int j = 0; j < kPer; ++j) sh[j * kSize + me] = v[j];
        Group::sync();
#pragma unroll
        for (int j = 0; j < kPer; ++j) other[j] = sh[j * kSize + (me ^ s)];
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) other[j] = __shfl_xor_sync(0xffffffffu, v[j], s);
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = j * kSize + me;
        const bool larger = ((i & k) == 0) == ((i & s) == 0);
        if (larger == (v[j] < other[j])) v[j] = other[j];
      }
    }
  }
}

template <int kType>
struct Sampler {
  using E = Elem<kType>;
  using Bits = typename E::Bits;
  static constexpr int kVec = E::kVec, kTile = 32 * kVec;

  const SampleParams& p;
  Shared& sh;
  uint4* data;                  // the CTA's slice: 16-byte words as they lie in memory
  const Bits* x;                // the row
  cg::cluster_group cluster;
  int ctas, rank, row, tid, lane, warp;
  int first, t0, t1;            // token of the slice's first element; the warp's tiles
  float peak;                   // the row's largest logit
  Row r;
  float T, top_p, min_p;
  int k;
  bool greedy;

  struct Slice {
    int lo, hi, first, tiles, per_warp;
  };
  __device__ __forceinline__ Slice slice_of(int q) const {
    Slice s;
    s.lo = min(q * p.slice, p.V);
    s.hi = min(s.lo + p.slice, p.V);
    // (a slice is whole words, so all of them begin at the same place in one)
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(Bits));
    const int vecs = s.hi > s.lo ? (s.hi - s.lo + skew + kVec - 1) / kVec : 0;
    s.first = s.lo - skew;
    s.tiles = (vecs + 31) / 32;
    s.per_warp = (s.tiles + kWarps - 1) / kWarps;
    return s;
  }
  // the vector at token `at` of a slice, -inf outside it
  __device__ __forceinline__ uint4 load(int at, const Slice& s) const {
    if (at >= s.lo && at + kVec <= s.hi) return __ldg(reinterpret_cast<const uint4*>(x + at));
    Bits part[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      part[e] = at + e >= s.lo && at + e < s.hi ? x[at + e] : static_cast<Bits>(E::kNone);
    uint4 w;
    memcpy(&w, part, 16);
    return w;
  }
  template <class F>
  __device__ __forceinline__ void each_vector(F f) const {
    for (int t = t0; t < t1; ++t) f(data[t * 32 + lane], first + (t * 32 + lane) * kVec);
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    each_vector([&](const uint4& w, int at) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) f(element<kType>(w, e), at + e);
    });
  }
  template <class V>
  __device__ __forceinline__ V* at_first(V* v) const { return cluster.map_shared_rank(v, 0); }

  __device__ __forceinline__ void append(uint64_t at) const {
    const int i = atomicAdd(&sh.listed, 1);
    if (i < kList) sh.list[i] = at;
  }
  // Every logit from `edge` on, listed in the CTA.
  __device__ __forceinline__ void list_from(float edge) const {
    each_vector([&](const uint4& w, int at) {
      if (vector_max<kType>(w) >= edge) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float y = element<kType>(w, e);
          if (y >= edge) append(place(key_of(y), at + e));
        }
      }
    });
  }
  // The CTA's list joined to the first CTA's. (The cluster meets behind it.)
  __device__ __forceinline__ void send_list() const {
    if (rank == 0) return;
    __syncthreads();
    const int n = sh.listed;
    if (tid == 0) sh.at = n > 0 ? atomicAdd(at_first(&sh.listed), n) : 0;
    __syncthreads();
    unsigned long long* dst = at_first(sh.list);
    for (int i = tid; i < n && i < kList && sh.at + i < kList; i += kThreads)
      dst[sh.at + i] = sh.list[i];
  }

  __device__ __forceinline__ void finish(int token, float logit, uint64_t z) const {
    p.tokens[row] = token;
    const double lw = greedy ? 0.0 : (static_cast<double>(logit) - peak) / T;
    p.logprobs[row] = static_cast<float>(lw - log(ldexp(static_cast<double>(z), -p.scale)));
  }
  __device__ __forceinline__ uint64_t point(uint64_t z) const {
    return __umul64hi(static_cast<uint64_t>(p.random[row]) << 32, z);
  }
  // The first place that min-p keeps.
  __device__ __forceinline__ uint64_t min_place() const {
    return place(min_p > 0.f ? sh.least : kLowestKey, kIdxMask);
  }

  // The list of n places, all that may be kept, decides: top-k, top-p of the sum of those, min-p,
  // the draw. (First CTA; the warps of the group.)
  template <class Group, int kPer>
  __device__ __forceinline__ void decide(int n, uint64_t all, bool by_all) const {
    constexpr int kSize = Group::kSize;
    const int me = Group::self();
    uint64_t v[kPer], upto[kPer];
    int size = 32;
    while (size < n) size <<= 1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = j * kSize + me < n ? sh.list[j * kSize + me] : 0;
    sort_falling<Group, kPer>(v, size, sh.list);
    const int nk = k > 0 && k < n ? k : n;
    auto scan = [&](int m, auto weight_of) {
      uint64_t carry = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (j * kSize < m) {  // (uniform)
          upto[j] = carry + Group::scan(j * kSize + me < m ? weight_of(v[j]) : 0, sh.warp);
          if (kPer > 1) {
            Group::sync();
            if (me == kSize - 1) sh.total = upto[j];
            Group::sync();
            carry = sh.total;
          }
        }
      }
    };
    auto count = [&](int m, auto pred) {  // of the first m
      int c = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j * kSize < m) c += Group::count(j * kSize + me < m && pred(j));
      return c;
    };
    auto show = [&](int i) {  // the sum up to i, to every thread
      Group::sync();
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j * kSize + me == i) sh.total = upto[j];
      Group::sync();
      return static_cast<uint64_t>(sh.total);
    };
    scan(nk, [&](uint64_t at) { return weight<kType>(logit_at(at), r, sh.table); });
    int m = nk;
    if (top_p < 1.f) {
      const uint64_t target = share_of(by_all ? all : show(nk - 1));
      m = min(m, count(nk, [&](int j) { return upto[j] < target; }) + 1);
    }
    if (min_p > 0.f) {
      const uint64_t least = min_place();
      m = min(m, count(m, [&](int j) { return v[j] >= least; }));
    }
    const uint64_t z = show(m - 1), goal = point(z);
    // the kept ones in the vocabulary's order: the index (as a place has it) before the key
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      v[j] = j * kSize + me < m
                 ? (v[j] & kIdxMask) << 32 | static_cast<uint32_t>(v[j] >> kIdxBits)
                 : 0;
    int at = 0;
    if (m > 1) {
      size = 32;
      while (size < m) size <<= 1;
      sort_falling<Group, kPer>(v, size, sh.list);
      scan(m, [&](uint64_t u) {
        return weight<kType>(of_key(static_cast<uint32_t>(u)), r, sh.table);
      });
      at = count(m, [&](int j) { return upto[j] <= goal; });
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j * kSize + me == at)
        finish(static_cast<int>(kIdxMask - (v[j] >> 32)), of_key(static_cast<uint32_t>(v[j])), z);
  }
  __device__ void decide(int n, uint64_t all, bool by_all) const {
    if (n <= 128) {
      if (warp == 0) decide<WarpGroup, 4>(n, all, by_all);
    } else if (n <= kThreads) {
      decide<BlockGroup, 1>(n, all, by_all);
    } else {
      decide<BlockGroup, kList / kThreads>(n, all, by_all);
    }
  }

  // top_p's share of a sum, rounded up: a place is kept while the sum before it is less.
  // (top_p is 24 bits and a power of two: the product is exact.)
  __device__ __forceinline__ uint64_t share_of(uint64_t z) const {
    const uint32_t bits = __float_as_uint(top_p);
    const uint64_t m = (bits & 0x7fffffu) | 0x800000u;
    const int down = 150 - static_cast<int>(bits >> 23);  // 24 at least
    const uint64_t lo = z * m, hi = __umul64hi(z, m);
    if (down >= 64 + 24) return 1;
    if (down >= 64) {
      const uint64_t part = hi & ((1ull << (down - 64)) - 1);
      return (hi >> (down - 64)) + ((part | lo) != 0 ? 1 : 0);
    }
    return (hi << (64 - down) | lo >> down) + ((lo & ((1ull << down) - 1)) != 0 ? 1 : 0);
  }

  // Every warp's kept weights are in sh.sums: the draw among the places from `cut` on. The row's
  // logits of the warp that the point lies in are read again. (First CTA.)
  __device__ void draw(uint64_t cut) const {
    const int n = ctas * kWarps;
    const uint64_t upto = block_scan(tid < n ? sh.sums[tid] : 0, sh.warp);
    __syncthreads();
    if (tid == n - 1) sh.total = upto;
    __syncthreads();
    const uint64_t z = sh.total, goal = point(z);
    const uint64_t own = tid < n ? sh.sums[tid] : 0;
    if (tid < n && goal < upto && goal >= upto - own) {
      sh.at = tid;
      sh.found[0] = upto - own;
    }
    __syncthreads();
    const int q = sh.at / kWarps, w = sh.at % kWarps;
    uint64_t before = sh.found[0];
    const Slice s = slice_of(q);
    const int a = min(w * s.per_warp, s.tiles), b = min(a + s.per_warp, s.tiles);
    auto kept = [&](const uint4& v, int at, int e) -> uint64_t {
      const float y = element<kType>(v, e);
      return place(key_of(y), at + e) >= cut ? weight<kType>(y, r, sh.table) : 0;
    };
    for (int base = a; base < b; base += kWarps) {  // a tile a warp
      const int t = base + warp, at = s.first + (t * 32 + lane) * kVec;
      uint4 v = make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
      if (t < b) v = load(at, s);
      uint64_t some = 0;
#pragma unroll
      for (int e = 0; e < kVec; ++e) some += kept(v, at, e);
      const uint64_t end = before + block_scan(some, sh.warp);
      __syncthreads();
      if (tid == kThreads - 1) sh.total = end;
      __syncthreads();
      if (goal >= end - some && goal < end) {
        uint64_t y = end - some;
        for (int e = 0; e < kVec; ++e) {
          const uint64_t we = kept(v, at, e);
          if (goal < y + we) {
            finish(at + e, element<kType>(v, e), z);
            break;
          }
          y += we;
        }
      }
      before = sh.total;
      if (goal < before) break;  // (uniform)
    }
  }
  // A warp's sum to the first CTA. (The cluster meets behind it.)
  __device__ __forceinline__ void send_sum(uint64_t y) const {
#pragma unroll
    for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (lane == 0) at_first(sh.sums)[rank * kWarps + warp] = y;
  }

  // ---- the digit by digit search: places from `cut` on, up to which the sum (of 1 each, or of
  // the weights) is below `target` before them; the last one.
  __device__ uint64_t search(bool by_mass, uint64_t target, uint64_t cut) const {
    uint64_t prefix = 0;
    int shift = 32 + kIdxBits;
    while (shift > 0) {
      const int bits = shift > 31 ? 11 : 10, bins = 1 << bits, up = shift;
      shift -= bits;
      for (int i = tid; i < bins; i += kThreads) {
        sh.count[i] = 0;
        sh.list[i] = 0;
      }
      __syncthreads();
      each([&](float y, int v) {
        const uint64_t at = place(key_of(y), v);
        if (at < cut || at >> up != prefix) return;
        const int d = static_cast<int>(at >> shift) & (bins - 1);
        if (by_mass) atomicAdd(&sh.list[d], static_cast<unsigned long long>(weight<kType>(y, r, sh.table)));
        else atomicAdd(&sh.count[d], 1u);
      });
      cluster.sync();
      // four digits a thread, the highest first
      uint64_t sum[4], all = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = bins - 1 - (4 * tid + i);
        sum[i] = 0;
        for (int q = 0; d >= 0 && q < ctas; ++q)
          sum[i] += by_mass ? *cluster.map_shared_rank(&sh.list[d], q)
                            : *cluster.map_shared_rank(&sh.count[d], q);
        all += sum[i];
      }
      uint64_t before = block_scan(all, sh.warp) - all;
      if (before < target && before + all >= target) {
        for (int i = 0; i < 4; ++i) {
          if (before + sum[i] >= target) {
            sh.found[0] = bins - 1 - (4 * tid + i);
            sh.found[1] = before;
            break;
          }
          before += sum[i];
        }
      }
      cluster.sync();  // (the histograms have been read)
      prefix = prefix << bits | sh.found[0];
      target -= sh.found[1];
      __syncthreads();
    }
    return prefix;
  }
  // a sum over the cluster
  __device__ uint64_t cluster_sum(uint64_t y) const {
    y = block_sum(y, sh.warp);
    cluster.sync();
    if (tid == 0) sh.total = y;
    cluster.sync();
    y = 0;
    for (int q = 0; q < ctas; ++q) y += *cluster.map_shared_rank(&sh.total, q);
    return y;
  }
  __device__ void general() const {
    uint64_t cut = place(kLowestKey, kIdxMask);
    if (k > 0 && k < p.V) {
      uint64_t n = 0;
      each([&](float y, int) { n += key_of(y) >= kLowestKey; });
      if (cluster_sum(n) > static_cast<uint64_t>(k)) cut = search(false, k, cut);
    }
    if (top_p < 1.f) {
      uint64_t z = 0;
      each([&](float y, int v) {
        if (place(key_of(y), v) >= cut) z += weight<kType>(y, r, sh.table);
      });
      cut = search(true, share_of(cluster_sum(z)), cut);
    }
    const uint64_t least = min_place();
    cut = least > cut ? least : cut;
    cluster.sync();
    sum_and_draw(cut);
  }
  // The sum of the weights from `cut` on by warps, and the draw; the row is done.
  __device__ void sum_and_draw(uint64_t cut) const {
    uint64_t y = 0;
    if ((cut & kIdxMask) == 0 && r.s == 1.f) {  // (every token of the least logit)
      const float edge = logit_at(cut);
      const bool all = cut <= place(kLowestKey, kIdxMask);
      each_vector([&](const uint4& w, int) {
        if (!all && vector_max<kType>(w) < edge) return;
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          const float2 v = pair<kType>(w, e);
          uint64_t we[2];
          weights<kType>(v, below(v, r), r, sh.table, we);
          y += (all || v.x >= edge ? we[0] : 0) + (all || v.y >= edge ? we[1] : 0);
        }
      });
    } else {
      each([&](float v, int at) {
        if (place(key_of(v), at) >= cut) y += weight<kType>(v, r, sh.table);
      });
    }
    send_sum(y);
    cluster.sync();
    if (rank == 0) draw(cut);
  }

  // ---- the row's first largest logit
  __device__ void take_first() const {
    int at = 0x7fffffff;
    each_vector([&](const uint4& w, int v) {
      if (vector_max<kType>(w) >= peak) {
#pragma unroll
        for (int e = kVec - 1; e >= 0; --e)
          if (element<kType>(w, e) >= peak) at = min(at, v + e);
      }
    });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) at_first(sh.sums)[rank * kWarps + warp] = static_cast<unsigned>(at);
    cluster.sync();
    if (rank == 0 && warp == 0) {
      int v = 0x7fffffff;
      for (int i = lane; i < ctas * kWarps; i += 32) v = min(v, static_cast<int>(sh.sums[i]));
      v = __reduce_min_sync(0xffffffffu, v);
      if (lane == 0) {
        p.tokens[row] = v;
        p.logprobs[row] = 0.f;
      }
    }
  }

  // ---- top-k by the threads' maxima, counted in sh.count by their keys' first 11 bits
  __device__ float bound_of_k() const {
    if (warp == 0) {
      int top = static_cast<int>(key_of(peak + 0.f) >> 21), sum = 0, found = -1;
      for (; top >= 0 && found < 0; top -= 32) {
        const int bin = top - lane;
        int n = 0;
        for (int q = 0; bin >= 0 && q < ctas; ++q) n += *cluster.map_shared_rank(&sh.count[bin], q);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, n, o);
          if (lane >= o) n += y;
        }
        const unsigned has = __ballot_sync(0xffffffffu, sum + n >= k);
        if (has) found = top - (__ffs(has) - 1);
        sum += __shfl_sync(0xffffffffu, n, 31);
      }
      if (lane == 0) {
        const uint32_t key = found > 0 ? static_cast<uint32_t>(found) << 21 : 0u;
        sh.edge[0] = of_key(key > kLowestKey ? key : kLowestKey);
      }
    }
    __syncthreads();
    return sh.edge[0];
  }
  // The row by a list of all logits from `edge` on; false if they are too many.
  __device__ bool by_list(float edge, uint64_t all, bool by_all) const {
    list_from(edge);
    send_list();
    cluster.sync();
    const int n = *at_first(&sh.listed);
    if (n > kList) {
      cluster.sync();  // (the count has been read)
      return false;
    }
    if (rank == 0) decide(n, all, by_all);
    return true;
  }

  // The least logit whose bin is at most b (bins rise as logits fall). A warp does it.
  __device__ float edge_of(int b) const {
    uint32_t lo = kLowestKey, hi = key_of(peak + 0.f);  // hi: a key in a bin at most b
    while (hi > lo) {
      const uint32_t step = (hi - lo) / 32 + 1;
      const uint32_t key = lo + step * lane;
      bool in = key >= hi;
      if (!in) {
        const Below at = below(both(of_key(key)), r);
        in = at.y.x < 63.9f && bin_of(at.t.x) <= b;
      }
      const int f = __ffs(__ballot_sync(0xffffffffu, in)) - 1;  // the first key in (none: hi)
      const uint32_t was = lo;
      if (f >= 0) {
        hi = min(hi, was + step * static_cast<uint32_t>(f));
        if (f > 0) lo = was + step * static_cast<uint32_t>(f - 1) + 1;
      } else {
        lo = was + step * 31 + 1;
      }
    }
    return of_key(hi);
  }

  // ---- top-p without a small k
  __device__ bool by_nucleus() const {
    // The sum of all weights, and counts by bin; of the logits that may be kept: those under
    // (1 - top_p) / V of the largest weigh less than 1 - top_p of it together, so the border lies
    // above them.
    const float past = fminf(log2f(static_cast<float>(p.V)) - log2f(1.f - top_p) + 1.f, 63.9f);
    for (int i = tid; i < kBins; i += kThreads) sh.count[i] = 0;
    __syncthreads();
    uint64_t y = 0;
    each_vector([&](const uint4& w, int) {
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        const float2 v = pair<kType>(w, e);
        const Below b = below(v, r);
        uint64_t we[2];
        weights<kType>(v, b, r, sh.table, we);
        y += we[0] + we[1];
        if (b.y.x < past) atomicAdd(&sh.count[bin_of(b.t.x)], 1u);
        if (b.y.y < past) atomicAdd(&sh.count[bin_of(b.t.y)], 1u);
      }
    });
    y = block_sum(y, sh.warp);
    if (tid == 0) sh.total = y;
    cluster.sync();
    uint64_t all = 0;
    for (int q = 0; q < ctas; ++q) all += *cluster.map_shared_rank(&sh.total, q);
    const uint64_t target = share_of(all);
    // the bin of the border, each bin's logits counted with its middle weight; four bins a thread
    uint32_t n[4], sum_n = 0;
    float mass[4], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n[i] = 0;
      for (int q = 0; q < ctas; ++q) n[i] += *cluster.map_shared_rank(&sh.count[4 * tid + i], q);
      mass[i] = static_cast<float>(n[i]) * fast_exp2(-(2 * (4 * tid + i) + 0.5f) / 64.f);
      sum += mass[i];
      sum_n += n[i];
    }
    cluster.sync();  // (the sums and counts have been read)
    // (sums of masses in units of 2^-40: they take part in no decision)
    const uint64_t upto_n = block_scan(sum_n, sh.warp);
    const uint64_t own = __float2ull_rn(sum * 1099511627776.f);
    const uint64_t upto = block_scan(own, sh.warp);
    __syncthreads();
    if (tid == kThreads - 1) sh.total = upto;
    if (tid < 2) sh.guess[tid] = 0;
    __syncthreads();
    // The border by the counted masses, of their own sum (what a middle weight is off by cancels)
    // and of the exact one (some are left out): between the two, but for the bins' unevenness.
    const uint64_t goal = (target >> (p.scale - 40)) + 1;
    const uint64_t wants[2] = {share_of(sh.total), goal < sh.total ? goal : sh.total};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint64_t want = wants[g];
      if (upto - own < want && upto >= want) {
        float part = static_cast<float>(want - (upto - own)) * 0x1p-40f;
        int i = 0;
        for (; i < 3; ++i) {
          part -= mass[i];
          if (part <= 0.f) break;
        }
        sh.guess[g] = 4 * tid + i;
      }
    }
    __syncthreads();
    const int mid = min(sh.guess[0], kBins - 2);
    const int far = min(max(sh.guess[0], sh.guess[1]), kBins - 2);
    // merged counts up to each bin, for the window's choice
    {
      uint32_t c = static_cast<uint32_t>(upto_n) - sum_n;
#pragma unroll
      for (int i = 0; i < 4; ++i) sh.count[4 * tid + i] = c += n[i];
    }
    __syncthreads();
    auto upto_bin = [&](int b) { return b < 0 ? 0u : sh.count[min(b, kBins - 1)]; };
    // everything down to a bin past the border, or the bins around it
    int b1 = min(far + 1, kBins - 2), b0 = 0;
    if (upto_bin(b1) > kShort) {
      b1 = min(mid + 1, kBins - 2);
      b0 = max(mid - 1, 0);
      if (upto_bin(b1) - upto_bin(b0 - 1) > kShort) b0 = b1 = mid;
    }
    int least = 0, most = kBins - 2;  // the border's bin lies between
    while (least <= most) {
      if (upto_bin(b1) - upto_bin(b0 - 1) > kList) return false;
      if (warp == 0) {
        const float e = edge_of(b1);
        if (lane == 0) sh.edge[0] = e;
      } else if (warp == 1) {
        const float e = b0 > 0 ? edge_of(b0 - 1) : INFINITY;
        if (lane == 0) sh.edge[1] = e;
      }
      if (tid == 0 && rank != 0) sh.listed = 0;
      __syncthreads();
      const float low = sh.edge[0], high = sh.edge[1];
      if (b0 == 0) {
        if (by_list_round(low, all, target)) return true;
        least = b1 + 1;  // not all of the nucleus is in the list: on by what lacks
        b0 = step(least, 1, *at_first(&sh.found[0]));
      } else {
        y = 0;
        each_vector([&](const uint4& w, int at) {
          if (vector_max<kType>(w) >= low) {
#pragma unroll
            for (int e = 0; e < kVec; e += 2) {
              const float2 v = pair<kType>(w, e);
              uint64_t we[2];
              weights<kType>(v, below(v, r), r, sh.table, we);
              y += (v.x >= high ? we[0] : 0) + (v.y >= high ? we[1] : 0);
              if (v.x >= low && v.x < high) append(place(key_of(v.x + 0.f), at + e));
              if (v.y >= low && v.y < high) append(place(key_of(v.y + 0.f), at + e + 1));
            }
          }
        });
        send_sum(y);
        send_list();
        cluster.sync();
        if (rank == 0) border(target);
        cluster.sync();
        const int state = *at_first(&sh.state);
        if (state == 2) {  // min-p's border is the higher one
          cluster.sync();
          sum_and_draw(min_place());
          return true;
        }
        if (state == 0) {
          if (rank == 0) draw(sh.found[1]);
          return true;
        }
        // the border lies in another bin: so far on by the masses between
        if (state < 0) most = b0 - 1;
        else least = b1 + 1;
        b0 = step(state < 0 ? most : least, state < 0 ? -1 : 1, *at_first(&sh.found[0]));
      }
      b0 = b1 = min(max(b0, least), most);
      cluster.sync();  // (the state has been read, the list is empty again)
    }
    return false;
  }
  // The bin, from `bin` on by `by`, where the counted masses reach `gap` (of 2^scale). The merged
  // counts up to each bin are in sh.count.
  __device__ int step(int bin, int by, uint64_t gap) const {
    const float want = static_cast<float>(gap) * exp2f(-static_cast<float>(p.scale));
    float sum = 0.f;
    for (; bin >= 0 && bin <= kBins - 2; bin += 32 * by) {
      const int b = bin + by * lane;
      float m = 0.f;
      if (b >= 0 && b <= kBins - 2)
        m = static_cast<float>(sh.count[b] - (b > 0 ? sh.count[b - 1] : 0)) *
            fast_exp2(-(2 * b + 0.5f) / 64.f);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) m += y;
      }
      const unsigned has = __ballot_sync(0xffffffffu, sum + m >= want);
      if (has) return min(max(bin + by * (__ffs(has) - 1), 0), kBins - 2);
      sum += __shfl_sync(0xffffffffu, m, 31);
    }
    return bin;
  }
  // a window that begins at the maximum: the whole nucleus in the list
  __device__ bool by_list_round(float low, uint64_t all, uint64_t target) const {
    list_from(low);
    send_list();
    cluster.sync();
    if (rank == 0) {
      const int n = sh.listed;
      uint64_t y = 0;
      for (int i = tid; i < n; i += kThreads) y += weight<kType>(logit_at(sh.list[i]), r, sh.table);
      y = block_sum(y, sh.warp);
      const bool ok = y >= target;
      if (ok) decide(n, all, true);
      __syncthreads();
      if (tid == 0) {
        sh.state = ok ? 0 : 1;
        sh.found[0] = target - y;
        sh.listed = 0;
      }
    }
    cluster.sync();
    return *at_first(&sh.state) == 0;
  }
  // The border of `target` in the list, the weights above the list's in sh.sums: sh.state 0 if it
  // is there (the cut in sh.found[1], the kept of the list added to sh.sums), -1 above, 1 below;
  // 2 if min-p's is higher. (First CTA.)
  __device__ void border(uint64_t target) const {
    const int n = min(sh.listed, kList);
    const uint64_t above = block_sum(tid < ctas * kWarps ? sh.sums[tid] : 0, sh.warp);
    if (n <= 128) {
      if (warp == 0) border_t<WarpGroup, 4>(n, above, target);
    } else if (n <= kThreads) {
      border_t<BlockGroup, 1>(n, above, target);
    } else {
      border_t<BlockGroup, kList / kThreads>(n, above, target);
    }
    __syncthreads();
  }
  template <class Group, int kPer>
  __device__ __forceinline__ void border_t(int n, uint64_t above, uint64_t target) const {
    constexpr int kSize = Group::kSize;
    const int me = Group::self();
    uint64_t v[kPer];
    int size = 32;
    while (size < n) size <<= 1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = j * kSize + me < n ? sh.list[j * kSize + me] : 0;
    sort_falling<Group, kPer>(v, size, sh.list);
    uint64_t sum = above;
    int kept = 0;  // those whose sum with what is before them is below the target, and one more
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j * kSize >= n) continue;  // (uniform)
      const bool in = j * kSize + me < n;
      const uint64_t upto =
          sum + Group::scan(in ? weight<kType>(logit_at(v[j]), r, sh.table) : 0, sh.warp);
      Group::sync();
      if (me == kSize - 1) sh.total = upto;
      Group::sync();
      kept += Group::count(in && upto < target);
      sum = sh.total;
    }
    Group::sync();
    const bool ok = above < target && sum >= target;
    if (ok) {
      ++kept;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = j * kSize + me;
        if (i == kept - 1) sh.found[1] = v[j];
        if (i < kept) {
          const int token = token_at(v[j]), q = token / p.slice;
          const Slice s = slice_of(q);
          const int w = (token - s.first) / kTile / s.per_warp;
          atomicAdd(&sh.sums[q * kWarps + w],
                    static_cast<unsigned long long>(weight<kType>(logit_at(v[j]), r, sh.table)));
        }
      }
    }
    Group::sync();
    if (me == 0) {
      sh.state = !ok ? (above >= target ? -1 : 1) : min_place() > sh.found[1] ? 2 : 0;
      if (!ok) sh.found[0] = above >= target ? above - target : target - sum;
      sh.listed = 0;
    }
  }
};

template <int kType>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  using S = Sampler<kType>;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  S s{p, sh, reinterpret_cast<uint4*>(raw + sizeof(Shared)), nullptr, cg::this_cluster()};
  s.ctas = static_cast<int>(s.cluster.num_blocks());
  s.rank = static_cast<int>(s.cluster.block_rank());
  s.row = static_cast<int>(blockIdx.x) / s.ctas;
  s.tid = threadIdx.x;
  s.lane = s.tid & 31;
  s.warp = s.tid >> 5;
  s.x = static_cast<const typename S::Bits*>(p.logits) + s.row * p.ld;
  if (s.tid < 64) sh.table[s.tid] = kExp2Table[s.tid];
  for (int i = s.tid; i < kBins; i += kThreads) sh.count[i] = 0;
  if (s.tid == 0) sh.listed = 0;
  if (s.lane == 0) {
    mbar_init(&sh.arrived[s.warp], 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  s.T = p.temperature ? p.temperature[s.row] : 1.f;
  s.k = p.top_k ? p.top_k[s.row] : 0;
  s.top_p = p.top_p ? p.top_p[s.row] : 1.f;
  s.min_p = p.min_p ? p.min_p[s.row] : 0.f;
  s.greedy = !(s.T >= 0x1p-100f);
  if (s.k >= p.V || s.k < 0) s.k = 0;

  // min-p's border below the maximum: one thread's work while the others load
  const bool bordered = s.min_p > 0.f && !s.greedy;
  if (bordered && s.tid == kThreads - 1)
    sh.fall = s.min_p < 1.f ? static_cast<double>(s.T) * log(static_cast<double>(s.min_p)) : 0.0;

  // ---- the slice, and the maximum: a copy a warp of the words that lie in the slice whole, the
  // others word by word
  const typename S::Slice slice = s.slice_of(s.rank);
  s.first = slice.first;
  s.t0 = min(s.warp * slice.per_warp, slice.tiles);
  s.t1 = min(s.t0 + slice.per_warp, slice.tiles);
  const int whole0 = (slice.lo - slice.first + S::kVec - 1) / S::kVec;  // whole words
  const int whole1 = max((slice.hi - slice.first) / S::kVec, whole0);
  const int a = min(max(s.t0 * 32, whole0), whole1), b = max(min(s.t1 * 32, whole1), a);
  if (s.lane == 0 && b > a) {
    mbar_arrive_expect_tx(&sh.arrived[s.warp], 16 * (b - a));
    bulk_load(s.data + a, s.x + s.first + a * S::kVec, 16 * (b - a), &sh.arrived[s.warp]);
  }
  if (s.t1 * 32 > whole1 || s.t0 * 32 < whole0)
    for (int v = s.t0 * 32 + s.lane; v < s.t1 * 32; v += 32)
      if (v < whole0 || v >= whole1) s.data[v] = s.load(s.first + v * S::kVec, slice);
  float mx = -INFINITY;
  if (b > a && !mbar_wait(&sh.arrived[s.warp], 0)) record_error(p.err, kDevWaitTimeout);
  __syncwarp();
  for (int t = s.t0; t < s.t1; ++t)
    mx = fmaxf(mx, vector_max<kType>(s.data[t * 32 + s.lane]));
  mx += 0.f;
  if (s.k > 0 && mx > -INFINITY) atomicAdd(&sh.count[key_of(mx) >> 21], 1u);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (s.lane == 0) sh.warp[s.warp] = __float_as_uint(mx);
  __syncthreads();
  if (s.tid == 0) {
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, __uint_as_float(static_cast<uint32_t>(sh.warp[w])));
    sh.max = mx;
  }
  s.cluster.sync();
  s.peak = -INFINITY;
  for (int q = 0; q < s.ctas; ++q) s.peak = fmaxf(s.peak, *s.cluster.map_shared_rank(&sh.max, q));

  // ---- the row by what it asks for (the same in every thread of the cluster); the first CTA
  // stays until the others, which may look at its shared memory, have left
  if (!(fabsf(s.peak) < INFINITY)) {  // no token
    if (s.rank == 0 && s.tid == 0) {
      p.tokens[s.row] = -1;
      p.logprobs[s.row] = -INFINITY;
    }
    s.cluster.sync();
    return;
  }
  if (s.greedy || s.k == 1 || s.top_p <= 0.f) {
    s.take_first();
    return;
  }
  const bool far = s.T >= 0x1p100f;
  s.r.s = far ? 0.25f : 1.f;
  s.r.max = s.peak * s.r.s;
  // log2(e) / T to 2^-45 in two floats (fp64 by every thread costs microseconds here)
  const float Ts = s.T * s.r.s;
  s.r.c = kLog2eHi / Ts;
  s.r.c_lo = s.r.c > 0.f ? (fmaf(-s.r.c, Ts, kLog2eHi) + kLog2eLo) / Ts : 0.f;
  s.r.limit = static_cast<float>(p.scale + 2);
  s.r.down = 60 - p.scale + (kMagicBits >> 6);
  if (bordered) {
    if (s.tid == kThreads - 1) {
      const uint32_t key = key_of(__double2float_ru(s.peak + sh.fall) + 0.f);
      sh.least = key > kLowestKey ? key : kLowestKey;
    }
    __syncthreads();
  }
  bool done = false;
  if (!far) {
    if (s.k > 0 && s.k <= kMaxTopK) {
      done = s.by_list(s.bound_of_k(), 0, false);
    } else if (s.k == 0 && s.top_p < 1.f) {
      done = p.V <= kShort ? s.by_list(-FLT_MAX, 0, false) : s.by_nucleus();
    } else if (s.k == 0) {
      s.sum_and_draw(s.min_place());
      done = true;
    }
  }
  if (!done) {
    s.cluster.sync();
    s.general();
  }
  if (s.rank == 0) s.cluster.sync();  // (waits for the threads that have not left)
}

int smem_bytes(int slice, int size) {
  // (the slice may begin inside a word, and a tile is whole)
  const int vecs = slice * size / 16 + 1;
  return static_cast<int>(sizeof(Shared)) + (vecs + 31) / 32 * 512;
}

template <int kType>
cudaError_t launch_t(const SampleParams& p, int cluster, cudaStream_t stream) {
  constexpr int size = kType == 2 ? 4 : 2;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_smem_limit(sample_kernel<kType>, kSmemLimit, done);
  if (e != cudaSuccess) return e;
  return launch_cluster(sample_kernel<kType>, static_cast<unsigned>(p.B) * cluster, cluster,
                        kThreads, smem_bytes(p.slice, size), stream, p);
}

}  // namespace

cudaError_t launch_sample(SampleParams p, int dtype, int num_sms, cudaStream_t stream) {
  const int size = dtype == 2 ? 4 : 2, word = 16 / size;
  auto slice = [&](int ctas) { return ((p.V + ctas - 1) / ctas + word - 1) / word * word; };
  int cluster = 1;
  while (cluster < kMaxCluster && smem_bytes(slice(cluster), size) > kSmemTwo) cluster *= 2;
  // few rows: more CTAs for each, while a warp has a few tiles of its slice
  while (cluster < kMaxCluster && static_cast<int64_t>(p.B) * cluster * 2 <= num_sms &&
         slice(cluster * 2) >= 4 * kThreads * word)
    cluster *= 2;
  p.slice = slice(cluster);
  // the sum of V weights stays below 2^62
  p.scale = 62;
  while (p.scale > 0 && (static_cast<int64_t>(p.V) - 1) >> (62 - p.scale) != 0) --p.scale;
  if (p.scale > 58) p.scale = 58;  // (a weight is made with 60 bits)
  switch (dtype) {
    case 0: return launch_t<0>(p, cluster, stream);
    case 1: return launch_t<1>(p, cluster, stream);
    default: return launch_t<2>(p, cluster, stream);
  }
}

}  // namespace ps
