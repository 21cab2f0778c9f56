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
// A cluster takes a row, a slice of it in each CTA's shared memory, read from memory once.
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
constexpr int kMaxCluster = 8;
constexpr int kSmemLimit = 232448;      // of a CTA
static_assert(true);
constexpr int kSmemTwo = 113 * 1024;    // of each of two on an SM
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: added, a float's low bits are its integer
constexpr double kLog2eD = 1.4426950408889634073599246810018921;

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
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t place(uint32_t key, int v) {
  return static_cast<uint64_t>(key) << kIdxBits | ((1u << kIdxBits) - 1 - v);
}
constexpr uint32_t kLowestKey = 0x00800000u;  // the least finite float's (-inf, NaN: below)

template <int kType>  // 0 fp16, 1 bf16, 2 fp32
struct Elem {
  using Bits = uint16_t;
  static constexpr int kVec = 8;  // in 16 bytes
};
template <>
struct Elem<2> {
  using Bits = uint32_t;
  static constexpr int kVec = 4;
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

struct Row {
  float max;      // the row's largest logit
  float c, c_lo;  // log2(e) / T as two floats
  int scale;      // the largest weight is 2^scale
};

template <int kType>
__device__ __forceinline__ uint64_t weight(float x, const Row& r, const uint32_t* table) {
  // z = -(max - x) log2(e) / T as zh + zl. (The differences of two 16-bit values are exact but
  // for logits thousands of times smaller than the maximum, whose error is 2^-24 of the
  // difference and random.)
  const float d = fminf(r.max - x, FLT_MAX);
  const float zh = -(d * r.c);
  float zl = fmaf(d, -r.c, -zh) - d * r.c_lo;
  if constexpr (kType == 2) {
    const float b = d - r.max, err = (r.max - (d - b)) + (-x - b);
    zl = fmaf(err, -r.c, zl);
  }
  const float t = fmaf(zh, 64.f, kMagic);
  const int m = static_cast<int>(__float_as_uint(t)) - 0x4b400000;
  const float s = fmaf(t - kMagic, -1.f / 64.f, zh) + zl;
  const float q = s * fmaf(s, fmaf(s, 0.05550410866f, 0.2402265070f), 0.6931471806f);
  const uint32_t f =
      (1u << 29) + (__float_as_uint(fmaf(q, 536870912.f, kMagic)) - 0x4b400000u);
  const uint64_t w = static_cast<uint64_t>(table[m & 63]) * f;  // 2^60 times 2^(frac)
  const int down = 60 - r.scale - (m >> 6);
  // (zh past the range of the sum with kMagic, or not a number: nothing)
  return zh > -100.f && down < 63 ? (w + (1ull << (down - 1))) >> down : 0ull;
}

// What the CTAs of a cluster show one another.
struct alignas(16) Shared {
  uint32_t count[kBins];
  unsigned long long mass[kBins];
  unsigned long long total;       // this CTA's kept weights, or its largest place
  uint32_t table[64];
  unsigned long long warp[kWarps];
  unsigned long long found[2];    // a search's digit, and the sum above it
};
static_assert(sizeof(Shared) % 16 == 0, "the slice behind it is read in 16-byte words");

template <int kType>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
  using E = Elem<kType>;
  constexpr int kVec = E::kVec;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int row = static_cast<int>(blockIdx.x) / ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  uint4* data = reinterpret_cast<uint4*>(raw + sizeof(Shared));
  if (tid < 64) sh.table[tid] = kExp2Table[tid];
  pdl_wait();

  // ---- the CTA's slice of the row: whole 16-byte words as they lie in memory, those at its
  // ends filled up with -inf
  const typename E::Bits* x = static_cast<const typename E::Bits*>(p.logits) + row * p.ld;
  const int lo = min(rank * p.slice, p.V), hi = min(lo + p.slice, p.V);
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(x + lo) & 15) / sizeof(*x));
  const int vecs = hi > lo ? (hi - lo + skew + kVec - 1) / kVec : 0;
  const int tiles = (vecs + 31) / 32, per_warp = (tiles + kWarps - 1) / kWarps;
  const int t0 = min(warp * per_warp, tiles), t1 = min(t0 + per_warp, tiles);
  const int first = lo - skew;  // the token of the first vector's first element
  constexpr uint32_t kNone = kType == 2 ? 0xff800000u : kType == 1 ? 0xff80ff80u : 0xfc00fc00u;
  uint64_t best = 0;
  for (int t = t0; t < t1; ++t) {
    const int v = t * 32 + lane, at = first + v * kVec;
    uint4 w = make_uint4(kNone, kNone, kNone, kNone);
    if (at >= lo && at + kVec <= hi) {
      w = *reinterpret_cast<const uint4*>(x + at);
    } else {
      typename E::Bits part[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        part[e] = at + e >= lo && at + e < hi ? x[at + e] : static_cast<typename E::Bits>(kNone);
      memcpy(&w, part, 16);
    }
    data[v] = w;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const uint64_t at_e = place(key_of(element<kType>(w, e)), at + e);
      best = at_e > best ? at_e : best;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t y = __shfl_xor_sync(0xffffffffu, best, o);
    best = y > best ? y : best;
  }
  if (lane == 0) sh.warp[warp] = best;
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < kWarps; ++k) best = sh.warp[k] > best ? sh.warp[k] : best;
    sh.total = best;
  }
  cluster.sync();
  best = 0;
  for (int k = 0; k < ctas; ++k) {
    const uint64_t y = *cluster.map_shared_rank(&sh.total, k);
    best = y > best ? y : best;
  }

  const uint32_t top_key = static_cast<uint32_t>(best >> kIdxBits);
  Row r;
  r.max = of_key(top_key);
  if (top_key < kLowestKey || r.max == INFINITY) {  // no token (uniform over the cluster)
    if (rank == 0 && tid == 0) {
      p.tokens[row] = -1;
      p.logprobs[row] = -INFINITY;
    }
    cluster.sync();
    return;
  }
  const float T = p.temperature ? p.temperature[row] : 1.f;
  const int k = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f, min_p = p.min_p ? p.min_p[row] : 0.f;
  const bool greedy = !(T >= 0x1p-100f);
  const double c = greedy ? 0.0 : kLog2eD / T;
  r.c = static_cast<float>(c);
  r.c_lo = static_cast<float>(c - r.c);
  r.scale = p.scale;

  // every element of the CTA's slice, a warp's in the order of the vocabulary
  auto each = [&](auto f) {
    for (int t = t0; t < t1; ++t) {
      const int v = t * 32 + lane;
      const uint4 w = data[v];
#pragma unroll
      for (int e = 0; e < kVec; ++e) f(element<kType>(w, e), first + v * kVec + e);
    }
  };
  // sum over the CTA; every thread gets it
  auto cta_sum = [&](uint64_t y) {
#pragma unroll
    for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = y;
    __syncthreads();
    y = 0;
    for (int w = 0; w < kWarps; ++w) y += sh.warp[w];
    return y;
  };
  // and over the cluster
  auto cluster_sum = [&](uint64_t y) {
    y = cta_sum(y);
    cluster.sync();
    if (tid == 0) sh.total = y;
    cluster.sync();
    y = 0;
    for (int q = 0; q < ctas; ++q) y += *cluster.map_shared_rank(&sh.total, q);
    return y;
  };
  // The last place, from the top, of those from `cut` on, up to which the sum (of 1 each, or of
  // the weights) is below `target` before it: digit by digit, by histograms of the digits.
  auto search = [&](bool by_mass, uint64_t target, uint64_t cut) {
    uint64_t prefix = 0;
    int shift = 32 + kIdxBits;
    while (shift > 0) {
      const int bits = shift > 31 ? 11 : 10, bins = 1 << bits, up = shift;
      shift -= bits;
      for (int i = tid; i < bins; i += kThreads) {
        sh.count[i] = 0;
        sh.mass[i] = 0;
      }
      __syncthreads();
      each([&](float y, int v) {
        const uint64_t at = place(key_of(y), v);
        if (at < cut || at >> up != prefix) return;
        const int d = static_cast<int>(at >> shift) & (bins - 1);
        if (by_mass) atomicAdd(&sh.mass[d], static_cast<unsigned long long>(weight<kType>(y, r, sh.table)));
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
          sum[i] += by_mass ? *cluster.map_shared_rank(&sh.mass[d], q)
                            : *cluster.map_shared_rank(&sh.count[d], q);
        all += sum[i];
      }
      uint64_t upto = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) sh.warp[warp] = upto;
      __syncthreads();
      uint64_t before = upto - all;
      for (int w = 0; w < warp; ++w) before += sh.warp[w];
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
  };

  // ---- the last kept place
  uint64_t cut = place(kLowestKey, (1 << kIdxBits) - 1);
  if (greedy || k == 1 || top_p <= 0.f) {
    cut = best;
  } else {
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
      z = cluster_sum(z);
      const double goal = ceil(static_cast<double>(top_p) * static_cast<double>(z));
      const uint64_t target = goal < 1.0 ? 1 : static_cast<uint64_t>(goal);
      cut = search(true, target < z ? target : z, cut);
    }
    if (min_p > 0.f) {
      const double least = min_p < 1.f ? r.max + static_cast<double>(T) * log(static_cast<double>(min_p)) : r.max;
      const uint64_t at = place(key_of(__double2float_ru(least) + 0.f), (1 << kIdxBits) - 1);
      cut = at > cut ? at : cut;
    }
  }

  // ---- the draw
  uint64_t mine = 0;
  each([&](float y, int v) {
    if (place(key_of(y), v) >= cut) mine += weight<kType>(y, r, sh.table);
  });
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  __syncthreads();
  if (lane == 0) sh.warp[warp] = mine;
  __syncthreads();
  uint64_t before = 0, all = 0;  // of the CTA's warps
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? sh.warp[w] : 0;
    all += sh.warp[w];
  }
  cluster.sync();
  if (tid == 0) sh.total = all;
  cluster.sync();
  uint64_t z = 0;
  for (int q = 0; q < ctas; ++q) {
    const uint64_t y = *cluster.map_shared_rank(&sh.total, q);
    before += q < rank ? y : 0;
    z += y;
  }
  const uint64_t word = p.random[row];
  const uint64_t goal = __umul64hi(word << 32, z);
  if (before <= goal && goal < before + mine) {  // one warp of the cluster
    for (int t = t0; t < t1; ++t) {
      const int v = t * 32 + lane;
      const uint4 w = data[v];
      uint64_t some = 0;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float y = element<kType>(w, e);
        if (place(key_of(y), first + v * kVec + e) >= cut) some += weight<kType>(y, r, sh.table);
      }
      uint64_t upto = some;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const uint64_t end = before + __shfl_sync(0xffffffffu, upto, 31);
      if (goal < end) {
        uint64_t at = before + upto - some;
        if (at <= goal && goal < at + some) {
          for (int e = 0; e < kVec; ++e) {
            const float y = element<kType>(w, e);
            const int token = first + v * kVec + e;
            const uint64_t own = place(key_of(y), token) >= cut ? weight<kType>(y, r, sh.table) : 0;
            if (goal < at + own) {
              p.tokens[row] = token;
              const double lw = greedy ? 0.0 : (static_cast<double>(y) - r.max) / T;
              p.logprobs[row] = static_cast<float>(lw - log(ldexp(static_cast<double>(z), -p.scale)));
              break;
            }
            at += own;
          }
        }
        break;
      }
      before = end;
    }
  }
  cluster.sync();  // (the totals have been read)
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
