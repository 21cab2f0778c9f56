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
// A weight is a whole number of 2^-42 of the largest, from exp2 in two floats (see weights):
// within 2^-29 of itself before that rounding. Sums of whole numbers are exact in any order.
//
// A cluster takes a row, a slice of it in each CTA's shared memory, read from memory once; the
// first CTA decides, the others leave as soon as it has what it needs of them. By what the row
// asks for:
//   - the largest logit alone: its first place;
//   - a small top-k: the k-th largest of the maxima of parts of the row bounds the k-th logit from
//     below; the few logits from the bound on are listed, and the list decides everything;
//   - top-p without it: a first pass counts the logits by weight (80 bins or so a factor of two),
//     each bin with its middle weight, to guess the border's bin; a second one sums all weights and
//     those above that bin exactly, and lists the logits around it. The list, in order, has the
//     border if the sums say so; else a next bin is tried. A nucleus that fits the list is listed
//     whole. A large top-k the same way, its bin by the counts, top-p of it by another pass;
//   - none of these: the sum of all weights (from min-p's border on), by warps; the word's point
//     lies in one warp's logits, which the first CTA reads again;
//   - what fits none (a list that overflows, as with equal logits everywhere; T beyond 2^100): the
//     border digit by digit, by histograms of places and exact weights.
//
// Bound: not by bytes (256 rows of 151936 in bf16 are 78 MB, 12 us) but by the weights' arithmetic
// where all are summed (the FMA and ALU pipes at 0.3 each, 1.5 instructions a cycle) and, with
// two CTAs on an SM, by what a row does one thing behind another: load 3 us, maximum 1, list and
// decision 8 (top-k) or counts 8, merge and choice 5, exact pass 10, list in order 6, draw 4
// (top-p). 256 rows of 151936, bf16, us: greedy 25, unfiltered 69, min-p 48, top-k 50 54, top-p
// 0.9 167; one row 4.3, 12, -, 11.3, 29. 512 threads of 64 registers, or clusters of 8 at three CTAs
// an SM, gave nothing. What is left is this way's, not a limit: a row in its cluster's shared memory
// keeps other rows out, and a second read of it would come from the L2 for the most part.
#include <cooperative_groups.h>

#include <cfloat>
#include <utility>

#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kPerThread = kBins / kThreads;  // bins of a thread
constexpr int kFine = 128;            // second digit of the maxima's keys
constexpr int kList = 2048;           // places that a row's list holds
constexpr int kCounted = 256;         // places that are put in order by counting
constexpr int kShort = 512;           // places that sort in a fraction of the time
constexpr int kMaxTopK = 128;         // k up to which the parts' maxima bound it
constexpr int kFineTopK = 64;         // k from which they do so by two digits
constexpr int kMaxCluster = 8;
constexpr int kSums = kMaxCluster * kWarps;
constexpr int kMinWords = 4;          // of a thread's share of a slice, where CTAs are to spare
constexpr int kSmemLimit = 232448;    // of a CTA
constexpr int kSmemTwo = 113 * 1024;  // of each of two on an SM
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: added, a float's low bits are its integer
constexpr uint32_t kMagicBits = 0x4b400000u;
constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.9259629911266175e-08f;
constexpr float kFarthest = 62.f;     // y from which a weight counts as this one's, 0

// 2^(j / 64) / (1 + j / 64) as two floats, the first of 17 bits
__constant__ float2 kExp2Table[64] = {
    {1.0f, 0.000000000e+00f}, {0.9953384399414062f, -1.296752089e-06f},
    {0.9909286499023438f, 1.918489488e-06f}, {0.9867706298828125f, -5.961908869e-07f},
    {0.98284912109375f, -3.208220960e-06f}, {0.9791488647460938f, 2.861970358e-07f},
    {0.9756698608398438f, 1.362636112e-06f}, {0.9724044799804688f, -3.805937752e-07f},
    {0.9693374633789062f, 2.743434607e-06f}, {0.9664688110351562f, 3.590768983e-06f},
    {0.9637908935546875f, 3.045987796e-06f}, {0.9612960815429688f, 2.366336048e-06f},
    {0.9589767456054688f, 3.157347464e-06f}, {0.9568328857421875f, -2.790280291e-07f},
    {0.9548492431640625f, 1.923012405e-06f}, {0.953033447265625f, -2.973017217e-06f},
    {0.9513626098632812f, 3.082138846e-06f}, {0.9498519897460938f, 2.425128400e-07f},
    {0.948486328125f, -5.837500225e-07f}, {0.947265625f, -3.524869499e-06f},
    {0.9461746215820312f, 2.759045401e-06f}, {0.9452285766601562f, -7.125474326e-07f},
    {0.9444122314453125f, -2.216791017e-06f}, {0.9437179565429688f, 2.515055257e-06f},
    {0.9431533813476562f, 2.658398444e-06f}, {0.9427108764648438f, 2.803732741e-06f},
    {0.9423904418945312f, 5.990795415e-08f}, {0.9421844482421875f, -6.950618285e-07f},
    {0.9420928955078125f, -2.080247441e-06f}, {0.942108154296875f, 1.040008215e-06f},
    {0.9422378540039062f, -1.338624315e-06f}, {0.9424667358398438f, 3.780396582e-06f},
    {0.94281005859375f, -1.017011641e-06f}, {0.9432525634765625f, -2.525774562e-06f},
    {0.9437942504882812f, -2.703074642e-06f}, {0.9444351196289062f, -3.414299954e-06f},
    {0.9451675415039062f, 1.191897354e-06f}, {0.9459991455078125f, 1.791231171e-06f},
    {0.946929931640625f, -3.231974233e-06f}, {0.9479446411132812f, -1.590972545e-07f},
    {0.9490509033203125f, 1.912315383e-06f}, {0.9502487182617188f, 1.582835580e-06f},
    {0.9515380859375f, -2.481344154e-06f}, {0.9529037475585938f, 3.707449878e-06f},
    {0.9543609619140625f, 3.679240990e-06f}, {0.9559097290039062f, -3.719839924e-06f},
    {0.9575271606445312f, 3.299372338e-06f}, {0.9592361450195312f, 8.021958706e-07f},
    {0.9610214233398438f, 3.051235808e-06f}, {0.962890625f, 1.469141466e-06f},
    {0.9648361206054688f, 2.783603577e-06f}, {0.9668655395507812f, -1.492094157e-06f},
    {0.968963623046875f, 3.086124707e-06f}, {0.9711456298828125f, 4.856872238e-07f},
    {0.9734039306640625f, -2.398458946e-06f}, {0.9757308959960938f, 1.366457923e-06f},
    {0.9781341552734375f, 3.490811650e-06f}, {0.9806137084960938f, 3.349399321e-06f},
    {0.9831695556640625f, 3.507544477e-07f}, {0.9857940673828125f, 1.565312800e-06f},
    {0.988494873046875f, -1.163938691e-06f}, {0.9912643432617188f, -7.049936812e-07f},
    {0.9941024780273438f, 2.473934728e-06f}, {0.9970169067382812f, 3.034099905e-07f},
};

// 1 / (1 + (2 j + 1) / 64), rounded, and minus its logarithm as two floats
struct LogEntry {
  float c, hi, lo;
};
__constant__ LogEntry kLogTable[32] = {
    {9.846153855e-01f, 1.550418604e-02f, -4.370104834e-10f},
    {9.552238584e-01f, 4.580955952e-02f, -2.097004514e-10f},
    {9.275362492e-01f, 7.522340119e-02f, 1.422285845e-09f},
    {9.014084339e-01f, 1.037968099e-01f, 2.396367327e-09f},
    {8.767123222e-01f, 1.315763593e-01f, 5.967296879e-09f},
    {8.533333540e-01f, 1.586050093e-01f, -3.355146161e-09f},
    {8.311688304e-01f, 1.849223375e-01f, 1.893291079e-09f},
    {8.101266026e-01f, 2.105647475e-01f, -3.491095413e-09f},
    {7.901234627e-01f, 2.355660647e-01f, -8.531991225e-10f},
    {7.710843086e-01f, 2.599575520e-01f, 9.733652995e-09f},
    {7.529411912e-01f, 2.837681472e-01f, 6.342722347e-09f},
    {7.356321812e-01f, 3.070250452e-01f, -6.136276820e-09f},
    {7.191011310e-01f, 3.297532797e-01f, -3.558054518e-09f},
    {7.032967210e-01f, 3.519763947e-01f, 3.358148648e-09f},
    {6.881720424e-01f, 3.737164140e-01f, -3.249855274e-09f},
    {6.736842394e-01f, 3.949937522e-01f, 1.315889708e-08f},
    {6.597937942e-01f, 4.158279300e-01f, -4.096246009e-09f},
    {6.464646459e-01f, 4.362367690e-01f, -1.254712112e-09f},
    {6.336633563e-01f, 4.562374353e-01f, 1.397318972e-08f},
    {6.213592291e-01f, 4.758459032e-01f, -7.601449248e-09f},
    {6.095238328e-01f, 4.950772226e-01f, 6.027948363e-09f},
    {5.981308222e-01f, 5.139457583e-01f, 2.442445890e-08f},
    {5.871559381e-01f, 5.324648619e-01f, -2.015950074e-08f},
    {5.765765905e-01f, 5.506470799e-01f, 1.379366488e-08f},
    {5.663716793e-01f, 5.685047507e-01f, -1.165064845e-08f},
    {5.565217137e-01f, 5.860490799e-01f, 1.074336620e-08f},
    {5.470085740e-01f, 6.032907963e-01f, 5.798082015e-09f},
    {5.378151536e-01f, 6.202403307e-01f, 2.783301056e-08f},
    {5.289255977e-01f, 6.369075179e-01f, -1.376341796e-08f},
    {5.203251839e-01f, 6.533012986e-01f, 1.064733279e-08f},
    {5.120000243e-01f, 6.694306135e-01f, -7.072582076e-09f},
    {5.039370060e-01f, 6.853039861e-01f, 2.075166883e-08f},
};

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

// Elements e and e + 1 of a 16-byte vector as they are.
template <int kType>
__device__ __forceinline__ float2 pair(const uint4& v, int e) {
  const uint32_t* w = &v.x;
  if constexpr (kType == 2) return make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]));
  else if constexpr (kType == 1)
    return make_float2(__uint_as_float(w[e / 2] << 16), __uint_as_float(w[e / 2] & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w[e / 2]));
}
// Element e; NaN counts as -inf, -0 as 0.
template <int kType>
__device__ __forceinline__ float element(const uint4& v, int e) {
  const float2 x = pair<kType>(v, e & ~1);
  return fmaxf((e & 1 ? x.y : x.x) + 0.f, -INFINITY);
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

// Whether some element of a vector is in [low, high): two at a time for 16-bit types, against the
// bounds rounded up to the type (a value of it is no less than a bound if no less than that).
template <int kType>
struct Between {
  float low, high;
  uint32_t low2, high2;
  __device__ __forceinline__ Between(float a, float b) : low(a), high(b) {
    if constexpr (kType == 1) {
      const __nv_bfloat162 l = __bfloat162bfloat162(__float2bfloat16_ru(a)),
                           h = __bfloat162bfloat162(__float2bfloat16_ru(b));
      low2 = *reinterpret_cast<const uint32_t*>(&l);
      high2 = *reinterpret_cast<const uint32_t*>(&h);
    } else if constexpr (kType == 0) {
      const __half2 l = __half2half2(__float2half_ru(a)), h = __half2half2(__float2half_ru(b));
      low2 = *reinterpret_cast<const uint32_t*>(&l);
      high2 = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  __device__ __forceinline__ bool any(const uint4& v) const {
    const uint32_t* w = &v.x;
    uint32_t in = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kType == 2) {
        const float y = __uint_as_float(w[i]);
        in |= y >= low && y < high;
      } else if constexpr (kType == 1) {
        auto h = [](const uint32_t& x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
        in |= __hge2_mask(h(w[i]), h(low2)) & __hlt2_mask(h(w[i]), h(high2));
      } else {
        auto h = [](const uint32_t& x) { return *reinterpret_cast<const __half2*>(&x); };
        in |= __hge2_mask(h(w[i]), h(low2)) & __hlt2_mask(h(w[i]), h(high2));
      }
    }
    return in != 0;
  }
};

struct Row {
  float max;      // the row's largest logit (times s)
  float far;      // the difference whose y is kFarthest: larger ones count as it
  float c, c_lo;  // log2(e) / T (over s) as two floats
  float s;        // 1, or 2^-64 where T is so large that c_lo would lose its bits
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Where two logits (times s) lie below the maximum: y = (max - x) log2(e) / T >= 0 as a float, and
// -64 y rounded to a whole number (as kMagic holds it).
struct Below {
  float2 x, d0, d, y, t;
};
__device__ __forceinline__ Below below(float2 x, const Row& r) {
  Below b;
  b.x = x;
  b.d0 = ffma2(x, both(-1.f), both(r.max));
  b.d = make_float2(fminf(b.d0.x, r.far), fminf(b.d0.y, r.far));  // (NaN, -inf: the farthest)
  b.y = fmul2(b.d, both(r.c));
  b.t = ffma2(b.y, both(-64.f), both(kMagic));
  return b;
}
// Counting bin, `per` to a factor of two. Never falls as x does.
__device__ __forceinline__ int bin_of(float y, float per) {
  return static_cast<int>(__float_as_uint(fmaf(y, per, kMagic)) - kMagicBits);
}

// The weights of two logits, in two parts each: hi (units of 2^-20 of the largest) and lo (of
// 2^-42), as kMagic holds them.
struct Parts {
  uint32_t hi[2], lo[2];
};
template <int kType>
__device__ __forceinline__ Parts weights(const Below& b, const Row& r, const float2* table) {
  // -y = -64 y rounded / 64 + s; s keeps what the product and, in fp32, the difference were
  // rounded by. (The differences of two 16-bit values are exact but for logits thousands of times
  // smaller than the maximum, whose error is 2^-24 of the difference and random.)
  float2 zl = ffma2(b.d, both(-r.c), b.y);
  zl = ffma2(b.d, both(-r.c_lo), zl);
  if constexpr (kType == 2) {
    const float2 q = ffma2(both(r.max), both(-1.f), b.d0);
    const float2 e1 = ffma2(ffma2(q, both(-1.f), b.d0), both(-1.f), both(r.max));
    float2 err = ffma2(ffma2(b.x, both(1.f), q), both(-1.f), e1);
    err = make_float2(b.d0.x < r.far ? err.x : 0.f, b.d0.y < r.far ? err.y : 0.f);
    zl = ffma2(err, both(-r.c), zl);
  }
  const float2 m = ffma2(both(kMagic), both(-1.f), b.t);
  const float2 s = ffma2(ffma2(m, both(1.f / 64.f), b.y), both(-1.f), zl);
  // 2^s = 1 + q, |s| at most 1/128 and a little: the series' next term is under 2^-34
  float2 q = ffma2(s, both(0.05550410866f), both(0.2402265070f));
  q = fmul2(s, ffma2(s, q, both(0.6931471806f)));
  // 2^(-64 y rounded / 64) = f (hi + lo): f = 2^n (1 + j / 64) from the bits of t, hi and lo by
  // table; f hi is exact
  const uint32_t tx = __float_as_uint(b.t.x), ty = __float_as_uint(b.t.y);
  const float2 cx = table[tx & 63], cy = table[ty & 63];  // (kMagicBits is a multiple of 64)
  // (by one value each, where a packed operation would want its operands brought together)
  const float2 f = make_float2(__uint_as_float((tx << 17) + 0x3f800000u),
                               __uint_as_float((ty << 17) + 0x3f800000u));
  const float2 wh = make_float2(f.x * cx.x, f.y * cy.x);
  const float2 wl = fmul2(f, make_float2(fmaf(cx.x, q.x, cx.y), fmaf(cy.x, q.y, cy.y)));
  // their sum as two floats, and those as whole numbers: each remainder is exact
  const float2 hi = ffma2(wh, both(1.f), wl);
  const float2 lo = ffma2(ffma2(wh, both(-1.f), hi), both(-1.f), wl);
  const float2 a = ffma2(hi, both(0x1p20f), both(kMagic));
  const float2 am = ffma2(both(kMagic), both(-1.f), a);
  const float2 rest = ffma2(ffma2(am, both(-0x1p-20f), hi), both(1.f), lo);
  const float2 l = ffma2(rest, both(0x1p42f), both(kMagic));
  return {{__float_as_uint(a.x), __float_as_uint(a.y)},
          {__float_as_uint(l.x), __float_as_uint(l.y)}};
}
__device__ __forceinline__ uint64_t whole(uint32_t hi, uint32_t lo) {
  return static_cast<uint64_t>((static_cast<int64_t>(static_cast<int32_t>(hi)) << 22) +
                               static_cast<int32_t>(lo));
}
template <int kType>
__device__ __forceinline__ uint64_t weight(float x, const Row& r, const float2* table) {
  const Parts w = weights<kType>(below(both(x * r.s), r), r, table);
  return whole(w.hi[0] - kMagicBits, w.lo[0] - kMagicBits);
}

// A copy of whole 16-byte words, global to shared, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// What the CTAs of a cluster show one another.
struct alignas(16) Shared {
  uint32_t count[kBins];
  unsigned long long list[kList];          // places, in any order; or masses of bins
  uint32_t fine[kFine];
  unsigned long long kept[kSums], all[kSums];  // (first CTA) every warp's sums
  unsigned long long warp[kWarps];
  unsigned long long total, found[2], fold[kWarps][3];
  float2 table[64];
  double fall;     // T ln(min_p)
  float max, edge[2];
  uint32_t least;  // the key of min-p's border
  int listed, state, at, digit[2];
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

// A bitonic sort, falling, of the first `size` values (a power of two, 32 at least): element
// j * kThreads + tid in v[j] of thread tid.
template <int kPer>
__device__ __forceinline__ void sort_falling(uint64_t* v, int size, unsigned long long* sh) {
  const int me = threadIdx.x;
#pragma unroll 1
  for (int k = 2; k <= size; k <<= 1) {
#pragma unroll 1
    for (int s = k >> 1; s > 0; s >>= 1) {
      if (s >= kThreads) {
        const int js = s / kThreads;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
#pragma unroll
          for (int o = j + 1; o < kPer; ++o) {
            if ((j ^ o) != js) continue;
            const bool up = ((j * kThreads + me) & k) == 0;
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
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; ++j) sh[j * kThreads + me] = v[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; ++j) other[j] = sh[j * kThreads + (me ^ s)];
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) other[j] = __shfl_xor_sync(0xffffffffu, v[j], s);
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = j * kThreads + me;
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
  // (the next vector is on its way while f has one)
  template <class F>
  __device__ __forceinline__ void each_vector(F f) const {
    const uint4* v = data + t0 * 32 + lane;
    uint4 next = make_uint4(0, 0, 0, 0);
    if (t0 < t1) next = *v;
    int at = first + (t0 * 32 + lane) * kVec;
    for (int t = t0; t < t1; ++t, at += kTile) {
      const uint4 w = next;
      v += 32;
      if (t + 1 < t1) next = *v;
      f(w, at);
    }
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
  __device__ __forceinline__ uint64_t weight_at(uint64_t at) const {
    return weight<kType>(logit_at(at), r, sh.table);
  }

  __device__ __forceinline__ void append(uint64_t at) const {
    const int i = atomicAdd(&sh.listed, 1);
    if (i < kList) sh.list[i] = at;
  }
  // Every logit from `edge` on, listed in the CTA.
  __device__ __forceinline__ void list_from(float edge) const {
    constexpr int kAhead = 4;
    for (int t = t0; t < t1; t += kAhead) {
      float top[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        top[i] = t + i < t1 ? vector_max<kType>(data[(t + i) * 32 + lane]) : -INFINITY;
      if (fmax3(fmaxf(top[0], top[1]), top[2], top[3]) < edge) continue;
#pragma unroll 1
      for (int i = 0; i < kAhead; ++i) {
        if (t + i >= t1) break;
        const uint4 w = data[(t + i) * 32 + lane];
        if (vector_max<kType>(w) < edge) continue;
        const int at = first + ((t + i) * 32 + lane) * kVec;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float y = element<kType>(w, e);
          if (y >= edge) append(place(key_of(y), at + e));
        }
      }
    }
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

  // The row's results: -(peak - x) / T - ln(z / 2^42), by pairs of floats (one thread's fp64 would
  // cost a microsecond at the end of every row): within 2^-35, and rounded.
  __device__ __forceinline__ void finish(int token, float logit, uint64_t z) const {
    p.tokens[row] = token;
    if (r.s != 1.f) {  // (T beyond 2^100)
      p.logprobs[row] = static_cast<float>((static_cast<double>(logit) - peak) / T -
                                           log(static_cast<double>(z) * 0x1p-42));
      return;
    }
    auto two = [](float a, float b, float* err) {  // their sum, and what it was rounded by
      const float s = a + b, t = s - a;
      *err += (a - (s - t)) + (b - t);
      return s;
    };
    // (peak - x) / T: q and a remainder
    float lo = 0.f, de = 0.f;
    const float d = two(peak, -logit, &de), q = d / T;
    lo += (fmaf(-q, T, d) + de) / T;
    // ln z = e ln 2 - ln c + ln(m c), m in [1, 2) as 24 bits and the rest, c near 1 / m by table
    const int e = 63 - __clzll(static_cast<long long>(z));
    const uint64_t bits = z << (63 - e);
    const float mh = static_cast<float>(static_cast<uint32_t>(bits >> 40)) * 0x1p-23f;
    const float ml = static_cast<float>(static_cast<uint32_t>(bits >> 8)) * 0x1p-55f;
    const LogEntry g = kLogTable[(bits >> 58) & 31];
    const float pr = mh * g.c, pe = fmaf(mh, g.c, -pr) + ml * g.c;
    const float rh = pr - 1.f, s = rh + pe;  // |s| under 1 / 64: five terms of the series
    const float series = s * s * fmaf(s, fmaf(s, fmaf(s, 0.2f, -0.25f), 1.f / 3.f), -0.5f);
    const float n = static_cast<float>(e - 42);
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654299957767878e-09f;
    const float a = n * kLn2Hi;
    lo += fmaf(n, kLn2Hi, -a) + n * kLn2Lo + g.lo + pe + series;
    float sum = two(a, g.hi, &lo);
    sum = two(sum, rh, &lo);
    sum = two(sum, q, &lo);
    p.logprobs[row] = -(sum + lo);
  }
  __device__ __forceinline__ uint64_t point(uint64_t z) const {
    return __umul64hi(static_cast<uint64_t>(p.random[row]) << 32, z);
  }
  // The first place that min-p keeps.
  __device__ __forceinline__ uint64_t min_place() const {
    return place(min_p > 0.f ? sh.least : kLowestKey, kIdxMask);
  }
  // top_p's share of a sum, rounded up: a place is kept while the sum before it is less. (top_p is
  // 24 bits and a power of two: the product is exact.)
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

  // ---- the list of n places, all that may be kept, decides: top-k, top-p of the sum of those (or
  // of `all`), min-p, the draw. (First CTA.)

  // A few: each compares itself with the others, `parts` threads for a place, thread by thread a
  // part of the others. Sums of the weights in sh.list + kCounted over the places that `counts`,
  // and their number.
  struct Counted {
    uint64_t sum;
    int n;
  };
  template <class Counts>
  __device__ __forceinline__ Counted compare(int n, int i, int part, int parts,
                                             Counts counts) const {
    Counted c{0, 0};
    const unsigned long long *at = sh.list, *w = sh.list + kCounted;
    if (i < n) {
#pragma unroll 4
      for (int j = part; j < n; j += parts) {
        if (counts(at[j])) {
          c.sum += w[j];
          ++c.n;
        }
      }
    }
    for (int o = parts >> 1; o; o >>= 1) {
      c.sum += __shfl_xor_sync(0xffffffffu, c.sum, o);
      c.n += __shfl_xor_sync(0xffffffffu, c.n, o);
    }
    return c;
  }
  __device__ __forceinline__ int parts_of(int n) const {
    return n <= 32 ? 8 : n <= 64 ? 4 : n <= 128 ? 2 : 1;
  }
  __device__ __forceinline__ void weigh(int n) const {
    for (int i = tid; i < n; i += kThreads) sh.list[kCounted + i] = weight_at(sh.list[i]);
    __syncthreads();
  }
  __device__ __forceinline__ void decide_few(int n, uint64_t all, bool by_all) const {
    weigh(n);
    const int parts = parts_of(n), i = tid / parts, part = tid % parts;
    const uint64_t own = i < n ? sh.list[i] : 0, w = i < n ? sh.list[kCounted + i] : 0;
    const Counted before = compare(n, i, part, parts, [&](uint64_t at) { return at > own; });
    const int nk = k > 0 && k < n ? k : n;
    auto show = [&](int rank_of) {  // the sum up to the place of a rank, to every thread
      if (i < n && part == 0 && before.n == rank_of) sh.total = before.sum + w;
      __syncthreads();
      const uint64_t y = sh.total;
      __syncthreads();
      return y;
    };
    bool keep = i < n && before.n < nk;
    if (top_p < 1.f) {
      const uint64_t target = share_of(by_all ? all : show(nk - 1));
      keep = keep && before.sum < target;
    }
    if (min_p > 0.f) keep = keep && own >= min_place();
    const int m = __syncthreads_count(keep && part == 0);
    const uint64_t z = show(m - 1), goal = point(z);
    // in the vocabulary's order (a place's index falls): sums of the kept weights before
    if (i < n && part == 0 && !keep) sh.list[kCounted + i] = 0;
    __syncthreads();
    const Counted left = compare(n, i, part, parts, [&](uint64_t at) {
      return (at & kIdxMask) > (own & kIdxMask);
    });
    if (keep && part == 0 && left.sum <= goal && goal < left.sum + w)
      finish(token_at(own), logit_at(own), z);
  }
  // More: sorted by their places, then by their indexes.
  template <int kPer>
  __device__ __forceinline__ void decide_sorted(int n, uint64_t all, bool by_all) const {
    uint64_t v[kPer], upto[kPer];
    int size = 32;
    while (size < n) size <<= 1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = j * kThreads + tid < n ? sh.list[j * kThreads + tid] : 0;
    sort_falling<kPer>(v, size, sh.list);
    const int nk = k > 0 && k < n ? k : n;
    auto scan = [&](int m, auto weight_of) {
      uint64_t carry = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (j * kThreads < m) {  // (uniform)
          upto[j] = carry + block_scan(j * kThreads + tid < m ? weight_of(v[j]) : 0, sh.warp);
          __syncthreads();
          if (tid == kThreads - 1) sh.total = upto[j];
          __syncthreads();
          carry = sh.total;
        }
      }
    };
    auto count = [&](int m, auto pred) {  // of the first m
      int c = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j * kThreads < m) c += __syncthreads_count(j * kThreads + tid < m && pred(j));
      return c;
    };
    auto show = [&](int i) {  // the sum up to i, to every thread
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j * kThreads + tid == i) sh.total = upto[j];
      __syncthreads();
      return static_cast<uint64_t>(sh.total);
    };
    scan(nk, [&](uint64_t at) { return weight_at(at); });
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
      v[j] = j * kThreads + tid < m
                 ? (v[j] & kIdxMask) << 32 | static_cast<uint32_t>(v[j] >> kIdxBits)
                 : 0;
    size = 32;
    while (size < m) size <<= 1;
    sort_falling<kPer>(v, size, sh.list);
    scan(m, [&](uint64_t u) {
      return weight<kType>(of_key(static_cast<uint32_t>(u)), r, sh.table);
    });
    const int at = count(m, [&](int j) { return upto[j] <= goal; });
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j * kThreads + tid == at)
        finish(static_cast<int>(kIdxMask - (v[j] >> 32)), of_key(static_cast<uint32_t>(v[j])), z);
  }
  __device__ __forceinline__ void decide(int n, uint64_t all, bool by_all) const {
    if (n <= kCounted) decide_few(n, all, by_all);
    else if (n <= kShort) decide_sorted<kShort / kThreads>(n, all, by_all);
    else decide_sorted<kList / kThreads>(n, all, by_all);
  }

  // ---- Every warp's kept weights are in sh.kept: the draw among the places from `cut` on. The
  // row's logits of the warp that the point lies in are read again. (First CTA.)
  __device__ __forceinline__ void draw(uint64_t cut) const {
    const int n = ctas * kWarps;
    const uint64_t own = tid < n ? sh.kept[tid] : 0;
    const uint64_t upto = block_scan(own, sh.warp);
    __syncthreads();
    if (tid == n - 1) sh.total = upto;
    __syncthreads();
    const uint64_t z = sh.total, goal = point(z);
    if (tid < n && goal < upto && goal >= upto - own) {
      sh.at = tid;
      sh.found[0] = upto - own;
    }
    __syncthreads();
    const int q = sh.at / kWarps, w = sh.at % kWarps;
    uint64_t before = sh.found[0];
    const Slice s = slice_of(q);
    const int a = min(w * s.per_warp, s.tiles), b = min(a + s.per_warp, s.tiles);
    // elements e and e + 1 of a vector at token `at`
    auto kept = [&](const uint4& v, int at, int e, uint64_t* we) {
      const float2 y = make_float2(element<kType>(v, e), element<kType>(v, e + 1));
      we[0] = place(key_of(y.x), at + e) >= cut;
      we[1] = place(key_of(y.y), at + e + 1) >= cut;
      const Parts g = weights<kType>(below(make_float2(y.x * r.s, y.y * r.s), r), r, sh.table);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        we[i] = we[i] ? whole(g.hi[i] - kMagicBits, g.lo[i] - kMagicBits) : 0;
    };
    // some neighbouring tiles a warp, all on their way before the first is weighed
    constexpr int kAhead = 4;
    for (int base = a; base < b; base += kWarps * kAhead) {  // (once, but for the longest rows)
      const int each = min((b - base + kWarps - 1) / kWarps, kAhead);
      const int t0 = base + warp * each, t1 = min(t0 + each, b);
      uint4 v[kAhead];
      uint64_t some[kAhead], sum = 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        v[i] = make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
        if (t0 + i < t1) v[i] = load(s.first + ((t0 + i) * 32 + lane) * kVec, s);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        some[i] = 0;
        if (t0 + i < t1) {
#pragma unroll
          for (int e = 0; e < kVec; e += 2) {
            uint64_t we[2];
            kept(v[i], s.first + ((t0 + i) * 32 + lane) * kVec, e, we);
            some[i] += we[0] + we[1];
          }
        }
        sum += some[i];
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      __syncthreads();
      if (lane == 0) sh.warp[warp] = sum;
      __syncthreads();
      uint64_t at = before;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        at += i < warp ? sh.warp[i] : 0;
        before += sh.warp[i];
      }
      if (goal >= at && goal < at + sum) {  // one warp
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          uint64_t upto = some[i];
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          const uint64_t end = at + upto;
          if (goal >= end - some[i] && goal < end) {  // one lane of one tile
            const int token = s.first + ((t0 + i) * 32 + lane) * kVec;
            uint64_t y = end - some[i];
#pragma unroll
            for (int e = 0; e < kVec; e += 2) {
              uint64_t we[2];
              kept(v[i], token, e, we);
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                if (goal >= y && goal < y + we[f])
                  finish(token + e + f, element<kType>(v[i], e + f), z);
                y += we[f];
              }
            }
          }
          at += __shfl_sync(0xffffffffu, upto, 31);
        }
      }
      if (goal < before) break;  // (uniform)
    }
  }
  // A warp's sum to the first CTA. (The cluster meets behind it.)
  __device__ __forceinline__ void send_sum(uint64_t y, unsigned long long* sums) const {
#pragma unroll
    for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (lane == 0) at_first(sums)[rank * kWarps + warp] = y;
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
        if (by_mass)
          atomicAdd(&sh.list[d],
                    static_cast<unsigned long long>(weight<kType>(y, r, sh.table)));
        else
          atomicAdd(&sh.count[d], 1u);
      });
      cluster.sync();
      // some digits a thread, the highest first
      uint64_t sum[kPerThread], all = 0;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        const int d = bins - 1 - (kPerThread * tid + i);
        sum[i] = 0;
        for (int q = 0; d >= 0 && q < ctas; ++q)
          sum[i] += by_mass ? *cluster.map_shared_rank(&sh.list[d], q)
                            : *cluster.map_shared_rank(&sh.count[d], q);
        all += sum[i];
      }
      uint64_t before = block_scan(all, sh.warp) - all;
      if (before < target && before + all >= target) {
        for (int i = 0; i < kPerThread; ++i) {
          if (before + sum[i] >= target) {
            sh.found[0] = bins - 1 - (kPerThread * tid + i);
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
  __device__ __noinline__ uint64_t general() const {
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
    cluster.sync();
    return least > cut ? least : cut;
  }
  // The sum of the weights from `cut` on by warps, for the draw. (The cluster meets in it.)
  __device__ __forceinline__ void sum_from(uint64_t cut) const {
    uint64_t y = 0;
    if ((cut & kIdxMask) == 0 && r.s == 1.f) {  // (every token of the least logit)
      const float edge = logit_at(cut);
      uint32_t hi = 0, lo = 0, n = 0;
      if (cut <= place(kLowestKey, kIdxMask)) {  // (what is no token weighs nothing)
        each_vector([&](const uint4& w, int) {
#pragma unroll
          for (int e = 0; e < kVec; e += 2) {
            const Parts a = weights<kType>(below(pair<kType>(w, e), r), r, sh.table);
            hi += a.hi[0] + a.hi[1];
            lo += a.lo[0] + a.lo[1];
          }
          n += kVec;
        });
      } else {
        each_vector([&](const uint4& w, int) {
          if (vector_max<kType>(w) < edge) return;
#pragma unroll
          for (int e = 0; e < kVec; e += 2) {
            const float2 v = pair<kType>(w, e);
            const Parts a = weights<kType>(below(v, r), r, sh.table);
            if (v.x >= edge) {
              hi += a.hi[0];
              lo += a.lo[0];
              ++n;
            }
            if (v.y >= edge) {
              hi += a.hi[1];
              lo += a.lo[1];
              ++n;
            }
          }
        });
      }
      y = whole(hi - n * kMagicBits, lo - n * kMagicBits);
    } else {
      each([&](float v, int at) {
        if (place(key_of(v), at) >= cut) y += weight<kType>(v, r, sh.table);
      });
    }
    send_sum(y, sh.kept);
    cluster.sync();
  }

  // What a row still needs: nothing; the draw from `cut` on (the sums are there); the sums first;
  // the digit by digit search.
  static constexpr int kDone = 0, kDraw = 1, kSum = 2, kSearch = 3;

  // ---- the row's first largest logit
  __device__ __forceinline__ void take_first() const {
    int at = 0x7fffffff;
    each_vector([&](const uint4& w, int v) {
      if (vector_max<kType>(w) >= peak) {
#pragma unroll
        for (int e = kVec - 1; e >= 0; --e)
          if (element<kType>(w, e) >= peak) at = min(at, v + e);
      }
    });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) at_first(sh.kept)[rank * kWarps + warp] = static_cast<unsigned>(at);
    cluster.sync();
    if (rank == 0 && warp == 0) {
      int v = 0x7fffffff;
      for (int i = lane; i < ctas * kWarps; i += 32) v = min(v, static_cast<int>(sh.kept[i]));
      v = __reduce_min_sync(0xffffffffu, v);
      if (lane == 0) {
        p.tokens[row] = v;
        p.logprobs[row] = 0.f;
      }
    }
  }

  // ---- top-k by the maxima of parts of the row (two of each thread)

  // The digit, from `top` down, at which the counts of all CTAs reach `want`: in sh.digit[0], what
  // is still wanted of it in sh.digit[1]; -1 if they do not. (A warp, kEach digits a lane.)
  template <int kEach>
  __device__ __forceinline__ void digit_of(const uint32_t* counts, int top, int want) const {
    int found = -1;
    for (; top >= 0 && found < 0; top -= 32 * kEach) {
      int n[kEach], sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int bin = top - kEach * lane - i;
        n[i] = 0;
        if (bin >= 0) {
#pragma unroll
          for (int q = 0; q < kMaxCluster; ++q)
            if (q < ctas) n[i] += *cluster.map_shared_rank(&counts[bin], q);
        }
        sum += n[i];
      }
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned has = __ballot_sync(0xffffffffu, upto >= want);
      if (has) {
        const int l = __ffs(has) - 1;
        int at = top - kEach * lane, left = want - (upto - sum);
#pragma unroll
        for (int i = 0; i < kEach - 1; ++i) {
          if (left > n[i] && at == top - kEach * lane - i) {
            left -= n[i];
            --at;
          }
        }
        found = __shfl_sync(0xffffffffu, at, l);
        want = __shfl_sync(0xffffffffu, left, l);
      } else {
        want -= __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    if (lane == 0) {
      sh.digit[0] = found;
      sh.digit[1] = want;
    }
  }
  __device__ __forceinline__ float bound_of_k(const float* maxima) const {
    if (warp == 0) digit_of<1>(sh.count, static_cast<int>(key_of(peak + 0.f) >> 21), k);
    __syncthreads();
    const int d = sh.digit[0];
    uint32_t key = d > 0 ? static_cast<uint32_t>(d) << 21 : 0u;
    if (k >= kFineTopK && d > 0) {  // and by the next digit
      const int want = sh.digit[1];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t km = key_of(maxima[i]);
        if (km >> 21 == static_cast<uint32_t>(d)) atomicAdd(&sh.fine[(km >> 14) & (kFine - 1)], 1u);
      }
      cluster.sync();
      if (warp == 0) digit_of<kFine / 32>(sh.fine, kFine - 1, want);
      __syncthreads();
      key |= static_cast<uint32_t>(sh.digit[0]) << 14;  // (it is found: the first digit was)
    }
    return of_key(key > kLowestKey ? key : kLowestKey);
  }
  // The row by a list of all logits from `edge` on; false if they are too many.
  __device__ __forceinline__ bool by_list(float edge) const {
    list_from(edge);
    send_list();
    cluster.sync();
    const int n = *at_first(&sh.listed);
    if (n > kList) {
      cluster.sync();  // (the count has been read)
      return false;
    }
    // the first CTA stays until the others have read the count (its wait ends for those that have
    // left, too)
    auto read = cluster.barrier_arrive();
    if (rank == 0) {
      decide(n, 0, false);
      cluster.barrier_wait(std::move(read));
    }
    return true;
  }

  // The least logit whose bin is at most b (bins rise as logits fall). A warp does it.
  __device__ __forceinline__ float edge_of(int b, float per) const {
    uint32_t lo = kLowestKey, hi = key_of(peak + 0.f);  // hi: a key in a bin at most b
    while (hi > lo) {
      const uint32_t step = (hi - lo) / 32 + 1;
      const uint32_t key = lo + step * lane;
      const bool in = key >= hi || bin_of(below(both(of_key(key)), r).y.x, per) <= b;
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

  // ---- top-p without a small k, or a large k

  // A bin's counted mass, of the largest weight.
  __device__ __forceinline__ static float mass_of(uint32_t n, int b, float per) {
    return static_cast<float>(n) * fast_exp2(-static_cast<float>(b) / per);
  }
  // The counts up to bin b, in the first CTA.
  __device__ __forceinline__ uint32_t upto_bin(int b) const { return b < 0 ? 0u : sh.count[b]; }
  // The bin, from `bin` on by `by`, where the counted masses reach `gap`. (Every warp of the first
  // CTA.)
  __device__ __forceinline__ int step(int bin, int by, uint64_t gap, float per) const {
    const float want = static_cast<float>(gap) * 0x1p-42f;
    float sum = 0.f;
    for (; bin >= 0 && bin < kBins - 1; bin += 32 * by) {
      const int b = bin + by * lane;
      float m = 0.f;
      if (b >= 0 && b < kBins - 1) m = mass_of(upto_bin(b) - upto_bin(b - 1), b, per);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) m += y;
      }
      const unsigned has = __ballot_sync(0xffffffffu, sum + m >= want);
      if (has) return bin + by * (__ffs(has) - 1);
      sum += __shfl_sync(0xffffffffu, m, 31);
    }
    return bin;
  }
  // The first CTA's choice of a window, bins b0 .. b1, told to all: its bounds as logits.
  __device__ __forceinline__ void choose(int b0, int b1, float per) const {
    __syncthreads();
    if (warp == 0) {
      const float e = edge_of(b1, per);
      if (lane < ctas) cluster.map_shared_rank(sh.edge, lane)[0] = e;
    } else if (warp == 1) {
      const float e = b0 > 0 ? edge_of(b0 - 1, per) : INFINITY;
      if (lane < ctas) cluster.map_shared_rank(sh.edge, lane)[1] = e;
    }
  }

  // What the first CTA says: the row is done; the draw is next; min-p's border is the one; another
  // window; the row is for the digit search.
  static constexpr int kSettled = 0, kHere = 1, kMinP = 2, kAgain = 3, kFull = 4;
  static constexpr int kMass = 0, kCount = 1;
  __device__ __forceinline__ int by_border(uint64_t* cut) const {
    // Counts by bin, of the logits that may be kept: without a k those under (1 - top_p) / V of the
    // largest weigh less than 1 - top_p of it together, so the border lies above them.
    const float past =
        k > 0 ? kFarthest - 0.5f
              : fminf(log2f(static_cast<float>(p.V)) - log2f(1.f - top_p) + 1.f, kFarthest - 0.5f);
    const float per = (kBins - 2) / past;
    for (int i = tid; i < kBins; i += kThreads) sh.count[i] = 0;
    __syncthreads();
    each_vector([&](const uint4& w, int) {
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        // (as below has it, where it counts)
        const float2 y = fmul2(ffma2(pair<kType>(w, e), both(-1.f), both(r.max)), both(r.c));
        if (y.x < past) atomicAdd(&sh.count[bin_of(y.x, per)], 1u);
        if (y.y < past) atomicAdd(&sh.count[bin_of(y.y, per)], 1u);
      }
    });
    cluster.sync();  // (the first CTA's counts are all there)
    if (rank != 0) {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        const uint32_t n = sh.count[i * kThreads + tid];
        if (n != 0) atomicAdd(at_first(&sh.count[i * kThreads + tid]), n);
      }
    }
    cluster.sync();
    // The first CTA looks for the border's window; the others do as it says. By count: the k-th's
    // bin. By mass, with the target known or the share of all weights (0): everything down to a bin
    // past the border, or the bins around it; then where its sums say.
    int kind = kMass, least = 0, most = kBins - 2, b0 = 0, b1 = 0;
    uint64_t target = 0;
    auto around = [&](int from, int to) {
      from = min(max(from, least), most);
      to = min(max(to, from), most);
      b0 = max(from - 1, least);
      b1 = min(to + 1, most);
      if (least == 0 && k == 0 && upto_bin(b1) <= kCounted) b0 = 0;
      else if (upto_bin(b1) - upto_bin(b0 - 1) > kCounted / 2) {
        b0 = from;
        b1 = upto_bin(to) - upto_bin(from - 1) > kCounted ? (from + to) / 2 : to;
        if (upto_bin(b1) - upto_bin(b0 - 1) > kCounted) b0 = b1;
      }
    };
    int state = kAgain;
    if (rank == 0) {
      uint32_t n[kPerThread], sum_n = 0;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        n[i] = sh.count[kPerThread * tid + i];
        sum += mass_of(n[i], kPerThread * tid + i, per);
        sum_n += n[i];
      }
      // (masses in units of 2^-40 of the largest weight)
      const uint64_t own = __float2ull_rn(sum * 0x1p40f);
      const uint64_t upto = block_scan(own, sh.warp);
      const uint32_t upto_n = static_cast<uint32_t>(block_scan(sum_n, sh.warp));
      if (tid == kThreads - 1) {
        sh.total = upto;
        sh.at = static_cast<int>(upto_n);
      }
      if (tid < 2) sh.digit[tid] = 0;
      __syncthreads();
      const bool by_count = k > 0 && k < sh.at;
      uint32_t c = upto_n - sum_n;
      if (by_count) {
        kind = kCount;
        if (c < static_cast<uint32_t>(k) && upto_n >= static_cast<uint32_t>(k)) {
          int i = 0;
          for (uint32_t at = c; i < kPerThread - 1; ++i)
            if ((at += n[i]) >= static_cast<uint32_t>(k)) break;
          sh.digit[0] = kPerThread * tid + i;
        }
      } else if (top_p < 1.f) {
        // the share of the counted masses, and with as much as the others may weigh: the border
        // lies between the two but for the bins' unevenness
        const uint64_t rest = static_cast<uint64_t>(
            static_cast<float>(p.V - sh.at) * fast_exp2(40.f - past));
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const uint64_t share = share_of(sh.total + (f ? rest : 0));
          const uint64_t want = share < sh.total ? share : sh.total;
          if (upto - own < want && upto >= want) {
            float part = static_cast<float>(want - (upto - own)) * 0x1p-40f;
            int i = 0;
            for (; i < kPerThread - 1; ++i) {
              part -= mass_of(n[i], kPerThread * tid + i, per);
              if (part <= 0.f) break;
            }
            sh.digit[f] = kPerThread * tid + i;
          }
        }
      } else {
        state = kMinP;  // (what is behind the k-th weighs nothing)
      }
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) sh.count[kPerThread * tid + i] = c += n[i];
      __syncthreads();
      if (kind == kCount) b0 = b1 = sh.digit[0];
      else around(sh.digit[0], sh.digit[1]);
    }
    while (true) {
      if (rank == 0) {
        const uint32_t in = upto_bin(b1) - upto_bin(b0 - 1);
        if (state == kAgain && (least > most || in > kList)) state = kFull;
        if (state == kAgain) choose(b0, b1, per);
        if (tid < ctas) *cluster.map_shared_rank(&sh.state, tid) = state;
      }
      if (tid == 0) sh.listed = 0;
      cluster.sync();
      state = sh.state;
      if (state != kAgain) break;
      window();
      if (rank == 0) {
        uint64_t gap = 0;
        const int found = settle(kind, target, static_cast<uint32_t>(k) - upto_bin(b0 - 1),
                                 b0 == 0, &gap);
        if (found <= kMinP) {
          state = found;
        } else if (found == kNext) {  // top-p of the first k: its border lies above theirs
          kind = kMass;
          target = gap;
          const int mid = step(0, 1, gap, per);
          around(mid, mid);
        } else {  // the border lies in another bin: so far on by the masses between
          if (found == kAbove) most = b0 - 1;
          else least = b1 + 1;
          const int mid = step(found == kAbove ? most : least, found == kAbove ? -1 : 1, gap, per);
          b0 = b1 = min(max(mid, least), most);
        }
      }
    }
    if (state == kFull) return kSearch;
    if (state == kSettled) return kDone;
    *cut = state == kMinP ? min_place() : sh.found[1];  // (the latter the first CTA's)
    return state == kMinP ? kSum : kDraw;
  }
  // The pass over the row for a window: the sums of all weights and of those above it, the logits
  // inside listed, all for the first CTA.
  __device__ __forceinline__ void window() const {
    const float low = sh.edge[0], high = sh.edge[1];
    const Between<kType> inside(low, high);
    uint32_t hi = 0, lo = 0, num = 0, hi_up = 0, lo_up = 0;
    each_vector([&](const uint4& w, int at) {
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        const float2 v = pair<kType>(w, e);
        const Parts a = weights<kType>(below(v, r), r, sh.table);
        hi += a.hi[0] + a.hi[1];
        lo += a.lo[0] + a.lo[1];
        if (v.x >= high) {
          hi_up += a.hi[0] - kMagicBits;
          lo_up += a.lo[0] - kMagicBits;
        }
        if (v.y >= high) {
          hi_up += a.hi[1] - kMagicBits;
          lo_up += a.lo[1] - kMagicBits;
        }
      }
      num += kVec;
      if (inside.any(w)) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float y = element<kType>(w, e);
          if (y >= low && y < high) append(place(key_of(y), at + e));
        }
      }
    });
    send_sum(whole(hi - num * kMagicBits, lo - num * kMagicBits), sh.all);
    send_sum(whole(hi_up, lo_up), sh.kept);
    send_list();
    cluster.sync();
  }
  // What the first CTA finds of a window. By count: the list's first `need` places are kept; by
  // mass: the border of the target. The row is done; the border is here (the cut in sh.found[1],
  // the kept of the list added to sh.kept); min-p's is higher; it is above or below, by *gap; top-p of
  // the kept is next, its target in *gap.
  static constexpr int kAbove = 5, kBelow = 6, kNext = 7;
  __device__ __forceinline__ int settle(int kind, uint64_t target, uint32_t need, bool from_top,
                                        uint64_t* gap) const {
    const int n = min(sh.listed, kList), sums = ctas * kWarps;
    const bool few = n <= kCounted;
    uint64_t w = 0, inside = 0;  // (few: one place a thread at most)
    for (int i = tid; i < n; i += kThreads) {
      w = weight_at(sh.list[i]);
      inside += w;
      if (few) sh.list[kCounted + i] = w;
    }
    uint64_t all = tid < sums ? sh.all[tid] : 0, above = tid < sums ? sh.kept[tid] : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      above += __shfl_xor_sync(0xffffffffu, above, o);
      inside += __shfl_xor_sync(0xffffffffu, inside, o);
    }
    __syncthreads();
    if (lane == 0) {
      sh.fold[warp][0] = all;
      sh.fold[warp][1] = above;
      sh.fold[warp][2] = inside;
    }
    __syncthreads();
    all = above = inside = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      all += sh.fold[i][0];
      above += sh.fold[i][1];
      inside += sh.fold[i][2];
    }
    if (kind == kCount) {
      ordered(n, [&](uint64_t at, uint64_t w, uint32_t before_n, uint64_t before) {
        if (before_n < need) add_kept(at, w);
        if (before_n == need - 1) {
          sh.found[1] = at;
          sh.total = above + before + w;
        }
      });
      __syncthreads();
      if (top_p < 1.f) {
        *gap = share_of(sh.total);
        return kNext;
      }
    } else {
      const uint64_t upto = above + inside, goal = target ? target : share_of(all);
      if (above >= goal) {
        *gap = above - goal;
        return kAbove;
      }
      if (upto < goal) {
        *gap = goal - upto;
        return kBelow;
      }
      if (from_top && k == 0) {
        decide(n, all, true);
        return kSettled;
      }
      ordered(n, [&](uint64_t at, uint64_t w, uint32_t, uint64_t before) {
        before += above;
        if (before < goal) add_kept(at, w);
        if (before < goal && before + w >= goal) sh.found[1] = at;
      });
      __syncthreads();
    }
    return min_place() > sh.found[1] ? kMinP : kHere;
  }
  // A kept place of the list counts to the warp that its logit lies in.
  __device__ __forceinline__ void add_kept(uint64_t at, uint64_t w) const {
    const int token = token_at(at), q = token / p.slice;
    const Slice s = slice_of(q);
    const int t = (token - s.first) / kTile / s.per_warp;
    atomicAdd(&sh.kept[q * kWarps + t], static_cast<unsigned long long>(w));
  }
  // Every place of the list, its weight, how many are before it and what they weigh, to one thread.
  // (The first CTA; the weights of kCounted places or fewer behind them.)
  template <class F>
  __device__ __forceinline__ void ordered(int n, F f) const {
    if (n <= kCounted) {  // (weighed already)
      const int parts = parts_of(n), i = tid / parts, part = tid % parts;
      const uint64_t own = i < n ? sh.list[i] : 0, w = i < n ? sh.list[kCounted + i] : 0;
      const Counted c = compare(n, i, part, parts, [&](uint64_t at) { return at > own; });
      if (i < n && part == 0) f(own, w, static_cast<uint32_t>(c.n), c.sum);
    } else if (n <= kShort) {
      ordered_sorted<kShort / kThreads>(n, f);
    } else {
      ordered_sorted<kList / kThreads>(n, f);
    }
  }
  template <int kPer, class F>
  __device__ __forceinline__ void ordered_sorted(int n, F f) const {
    uint64_t v[kPer];
    int size = 32;
    while (size < n) size <<= 1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = j * kThreads + tid < n ? sh.list[j * kThreads + tid] : 0;
    sort_falling<kPer>(v, size, sh.list);
    uint64_t sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j * kThreads >= n) continue;  // (uniform)
      const bool in = j * kThreads + tid < n;
      const uint64_t w = in ? weight_at(v[j]) : 0, upto = sum + block_scan(w, sh.warp);
      __syncthreads();
      if (tid == kThreads - 1) sh.found[0] = upto;
      __syncthreads();
      sum = sh.found[0];
      if (in) f(v[j], w, static_cast<uint32_t>(j * kThreads + tid), upto - w);
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
  if (s.lane == 0) {
    mbar_init(&sh.arrived[s.warp], 1);
    fence_barrier_init();
  }
  __syncwarp();
  pdl_wait();

  // ---- the slice: a copy a warp of the words that lie in it whole, the others word by word
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
  // beside the copies: what the row asks for, and shared memory made ready
  s.T = p.temperature ? p.temperature[s.row] : 1.f;
  s.k = p.top_k ? p.top_k[s.row] : 0;
  s.top_p = p.top_p ? p.top_p[s.row] : 1.f;
  s.min_p = p.min_p ? p.min_p[s.row] : 0.f;
  s.greedy = !(s.T >= 0x1p-100f);
  if (s.k >= p.V || s.k < 0) s.k = 0;
  if (s.tid < 64) sh.table[s.tid] = kExp2Table[s.tid];
  if (s.k > 0) {
    for (int i = s.tid; i < kBins; i += kThreads) sh.count[i] = 0;
    for (int i = s.tid; i < kFine; i += kThreads) sh.fine[i] = 0;
  }
  if (s.tid == 0) sh.listed = 0;
  const bool bordered = s.min_p > 0.f && !s.greedy;
  if (bordered && s.tid == kThreads - 1)  // (fp64 by every thread would cost microseconds)
    sh.fall = s.min_p < 1.f ? static_cast<double>(s.T) * log(static_cast<double>(s.min_p)) : 0.0;
  __syncthreads();

  // ---- the maximum
  float mx[2] = {-INFINITY, -INFINITY};
  if (b > a && !mbar_wait(&sh.arrived[s.warp], 0)) record_error(p.err, kDevWaitTimeout);
  __syncwarp();
  for (int t = s.t0; t < s.t1; t += 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t + i < s.t1)
        mx[i & 1] = fmaxf(mx[i & 1], vector_max<kType>(s.data[(t + i) * 32 + s.lane]));
  }
  const float maxima[2] = {mx[0] + 0.f, mx[1] + 0.f};
  if (s.k > 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (maxima[i] > -INFINITY) atomicAdd(&sh.count[key_of(maxima[i]) >> 21], 1u);
  }
  float top = fmaxf(maxima[0], maxima[1]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (s.lane == 0) sh.warp[s.warp] = __float_as_uint(top);
  __syncthreads();
  if (s.tid == 0) {
    for (int w = 1; w < kWarps; ++w)
      top = fmaxf(top, __uint_as_float(static_cast<uint32_t>(sh.warp[w])));
    sh.max = top;
  }
  s.cluster.sync();
  s.peak = -INFINITY;
  for (int q = 0; q < s.ctas; ++q) s.peak = fmaxf(s.peak, *s.cluster.map_shared_rank(&sh.max, q));

  // ---- the row by what it asks for (the same in every thread of the cluster). A CTA leaves when
  // no other looks at its shared memory any more.
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
  // (from T = 2^104 or so the bits of c_lo that count would lie below the least float, 2^-149; those
  // that a logit below 2^-62 loses by the scale are under 2^-185 of T)
  s.r.s = far ? 0x1p-64f : 1.f;
  s.r.max = s.peak * s.r.s;
  // log2(e) / T to 2^-45 in two floats
  const float Ts = s.T * s.r.s;
  s.r.c = kLog2eHi / Ts;
  s.r.c_lo = s.r.c > 0.f ? (fmaf(-s.r.c, Ts, kLog2eHi) + kLog2eLo) / Ts : 0.f;
  s.r.far = fminf(kFarthest / s.r.c, FLT_MAX);
  if (bordered) {
    if (s.tid == kThreads - 1) {
      const uint32_t key = key_of(__double2float_ru(s.peak + sh.fall) + 0.f);
      sh.least = key > kLowestKey ? key : kLowestKey;
    }
    __syncthreads();
  }
  int todo = S::kSearch;
  uint64_t cut = 0;
  if (!far) {
    const bool filtered = s.k > 0 || s.top_p < 1.f, tiny = p.V <= kCounted;
    if (!filtered) {
      todo = S::kSum;
      cut = s.min_place();
    } else if (tiny || (s.k > 0 && s.k <= kMaxTopK)) {
      if (s.by_list(tiny ? -FLT_MAX : s.bound_of_k(maxima))) todo = S::kDone;
    }
    if (todo == S::kSearch) todo = s.by_border(&cut);
  }
  if (todo == S::kSearch) {
    s.cluster.sync();
    const S other = s;  // (that its address is taken there must not cost the rest its registers)
    cut = other.general();
    todo = S::kSum;
  }
  if (todo == S::kSum) s.sum_from(cut);
  if (todo != S::kDone && s.rank == 0) s.draw(cut);
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
  // (powers of two: others leave SMs of a GPC without a cluster; 100 rows of 50257 by threes took
  // 44 us with top-p, by twos 36)
  int cluster = 1;
  while (cluster < kMaxCluster && smem_bytes(slice(cluster), size) > kSmemTwo) cluster *= 2;
  // few rows: more CTAs for each while all of them run at once, two an SM, and a thread has a few
  // words of its slice
  const int64_t at_once = (smem_bytes(slice(cluster), size) <= kSmemTwo ? 2 : 1) * num_sms;
  while (cluster < kMaxCluster && static_cast<int64_t>(p.B) * cluster * 2 <= at_once &&
         slice(cluster * 2) >= kMinWords * kThreads * word)
    cluster *= 2;
  p.slice = slice(cluster);
  switch (dtype) {
    case 0: return launch_t<0>(p, cluster, stream);
    case 1: return launch_t<1>(p, cluster, stream);
    default: return launch_t<2>(p, cluster, stream);
  }
}

}  // namespace ps
