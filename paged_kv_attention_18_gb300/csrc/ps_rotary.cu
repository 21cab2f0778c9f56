// Rotary positions in their other forms, fused with the KV scatter: interleaved pairs
// (2i, 2i + 1) or half pairs (i, i + R/2) over the first R elements of a head, the rest
// passed through, with the frequencies given as a table (any scaling for long contexts is
// in the table) and a magnitude on the cosine and sine:
//     (x, y) -> (x c - y s, y c + x s),  c = m cos(pos f_i),  s = m sin(pos f_i).
//
// Angle: each frequency is held as a 64-bit fixed-point fraction of a turn; pos * F_i
// wrapping modulo 2^64 is the angle modulo one turn (exact but for F_i's own rounding, so
// far positions lose nothing to a product rounded in fp32); its top 32 bits, signed, give
// an fp32 angle in [-pi, pi). Products and sums are fp32, each output rounded once.
//
// Work: every row (query, key or value head of a token) is D/16 units of 32 bytes. A unit
// is the two 16-byte chunks that rotate together: chunks u and u + R/16 in the half
// layout, chunks 2u and 2u + 1 otherwise (interleaved, passed through, or a value row).
// Either way a rotating unit u uses frequencies 8u .. 8u + 7, so both layouts share one
// loop. Bytes bound the kernel: each input row is read once and each output row written
// once; a thread keeps kUnits units in flight while it computes the pass's cosines.
#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 3;
constexpr int kMaxPassTokens = 8;  // tokens whose cosines and sines a CTA holds at a time
constexpr int kUnits = 4;          // units in flight per thread
constexpr double kInvTwoPi = 0.15915494309189533576888376337251436203445964574046;
constexpr double kTwoTo64 = 18446744073709551616.0;
constexpr float kTurnToRad = 1.46291807926715968e-09f;  // 2 pi / 2^32

template <bool kBF16>
__device__ __forceinline__ float2 widen2(uint32_t u) {
  if constexpr (kBF16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// One pair turned in fp32, products and sums rounded separately (no contraction: both
// outputs of a pair then carry the same two roundings per product).
__device__ __forceinline__ float2 turn(float x, float y, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)),
                     __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s)));
}

// The eight pairs of a unit: chunks a and b, frequencies c[0..7], s[0..7].
template <bool kBF16, bool kInter>
__device__ __forceinline__ void turn_unit(uint4& a, uint4& b, const float* c, const float* s) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 x = widen2<kBF16>(wa[w]), y = widen2<kBF16>(wb[w]);
    if constexpr (kInter) {  // a word is one pair: chunk a holds pairs 0..3, b pairs 4..7
      const float2 u = turn(x.x, x.y, c[w], s[w]), v = turn(y.x, y.y, c[4 + w], s[4 + w]);
      wa[w] = pack2<kBF16>(u.x, u.y);
      wb[w] = pack2<kBF16>(v.x, v.y);
    } else {  // pair 2w: (x.x, y.x); pair 2w + 1: (x.y, y.y)
      const float2 u = turn(x.x, y.x, c[2 * w], s[2 * w]);
      const float2 v = turn(x.y, y.y, c[2 * w + 1], s[2 * w + 1]);
      wa[w] = pack2<kBF16>(u.x, v.x);
      wb[w] = pack2<kBF16>(u.y, v.y);
    }
  }
}

// A CTA takes an equal share of the tokens (one wave, to a token), in equal passes of at most
// kMaxPassTokens; a pass's rows are its tokens' H_q query, H_kv key and H_kv value rows, D/16
// units each. (Whole passes of 8 tokens dealt to the CTAs left some with half as many again:
// 8192 tokens of 32 + 8 + 8 heads took 36.6 us, equal
// shares take 34.2: 5.9 TB/s.)
template <bool kBF16, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    rotary_kernel(const RotaryParams p) {
  constexpr int kRowUnits = D / 16, kRowsPerRound = kThreads / kRowUnits;
  __shared__ unsigned long long turns[D / 2];
  __shared__ float cs[2][kMaxPassTokens][D / 2], sn[2][kMaxPassTokens][D / 2];
  const int half = p.rot / 2, rot_units = p.rot / 16;
  pdl_wait();
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double t = p.inv_freq[i] * kInvTwoPi;
    turns[i] = __double2ull_rn((t - floor(t)) * kTwoTo64);
  }
  const int heads = p.H_q + 2 * p.H_kv;
  const int un = threadIdx.x % kRowUnits, row0 = threadIdx.x / kRowUnits;
  const bool rotates = un < rot_units;
  const int ca = rotates && !kInter ? un : 2 * un;
  const int cb = rotates && !kInter ? un + rot_units : 2 * un + 1;
  const int t_lo = static_cast<int>(static_cast<int64_t>(p.T) * blockIdx.x / gridDim.x);
  const int t_hi = static_cast<int>(static_cast<int64_t>(p.T) * (blockIdx.x + 1) / gridDim.x);
  const int passes = (t_hi - t_lo + kMaxPassTokens - 1) / kMaxPassTokens;
  const int ppt = passes > 0 ? (t_hi - t_lo + passes - 1) / passes : 0;  // tokens of a pass
  const int rows = ppt * heads;
  const bool in_place = p.q_out == p.q;
  // (token of the pass, head) of the thread's first row, and what the next one adds to it
  const int u_first = row0 / heads, head_first = row0 - u_first * heads;
  const int u_step = kRowsPerRound / heads, head_step = kRowsPerRound - u_step * heads;
  __syncthreads();
  int buf = 0;
  for (int t0 = t_lo; t0 < t_hi; t0 += ppt, buf ^= 1) {
    int u = u_first, head = head_first;
    for (int r0 = 0; r0 < rows; r0 += kUnits * kRowsPerRound) {
      uint4 a[kUnits], b[kUnits];
      uint4* dst[kUnits];
      int kind[kUnits];  // -1: nothing to do; 0: copied as it is; 1 + token of the pass: turned
#pragma unroll
      for (int j = 0; j < kUnits; ++j, u += u_step, head += head_step) {
        if (head >= heads) {
          head -= heads;
          ++u;
        }
        const int t = t0 + u;
        kind[j] = -1;
        if (u >= ppt || t >= t_hi) continue;
        const uint4* src;
        if (head < p.H_q) {
          if (in_place && !rotates) continue;
          src = reinterpret_cast<const uint4*>(p.q + t * p.q_stride + head * D);
          dst[j] = reinterpret_cast<uint4*>(p.q_out + (static_cast<int64_t>(t) * p.qo_stride) +
                                            head * D);
          kind[j] = rotates ? 1 + u : 0;
        } else {
          const int h = head - p.H_q;
          const bool is_v = h >= p.H_kv;
          const int hk = is_v ? h - p.H_kv : h;
          const int slot = p.slots[t];
          if (slot >= p.num_slots && h == 0 && un == 0) record_error(p.err, kDevBadSlot);
          if (slot < 0 || slot >= p.num_slots) continue;
          src = reinterpret_cast<const uint4*>(is_v ? p.v + t * p.v_stride + hk * D
                                                    : p.k + t * p.k_stride + hk * D);
          dst[j] = reinterpret_cast<uint4*>(
              (is_v ? p.v_pool : p.k_pool) + (static_cast<int64_t>(slot) * p.H_kv + hk) * D);
          kind[j] = rotates && !is_v ? 1 + u : 0;
        }
        // a value row's units are adjacent chunks whatever the layout
        const bool adj = kind[j] == 0;
        a[j] = src[adj ? 2 * un : ca];
        b[j] = src[adj ? 2 * un + 1 : cb];
      }
      if (r0 == 0) {
        for (int x = threadIdx.x; x < ppt * half; x += kThreads) {
          const int ux = x / half, i = x - ux * half, t = t0 + ux;
          if (t >= t_hi) continue;
          const unsigned long long ph =
              static_cast<unsigned long long>(static_cast<long long>(p.pos[t])) * turns[i];
          float s, c;
          sincosf(static_cast<float>(static_cast<int32_t>(ph >> 32)) * kTurnToRad, &s, &c);
          cs[buf][ux][i] = c * p.magnitude;
          sn[buf][ux][i] = s * p.magnitude;
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        if (kind[j] < 0) continue;
        if (kind[j] > 0) {
          turn_unit<kBF16, kInter>(a[j], b[j], cs[buf][kind[j] - 1] + 8 * un,
                                   sn[buf][kind[j] - 1] + 8 * un);
          dst[j][ca] = a[j];
          dst[j][cb] = b[j];
        } else {
          dst[j][2 * un] = a[j];
          dst[j][2 * un + 1] = b[j];
        }
      }
    }
  }
}

template <bool kBF16, int D>
cudaError_t launch_t(const RotaryParams& p, bool inter, int num_sms, cudaStream_t stream) {
  const int ctas = num_sms * kCtasPerSm;
  const dim3 grid(static_cast<unsigned>(p.T < ctas ? p.T : ctas));
  return inter ? launch_kernel(rotary_kernel<kBF16, D, true>, grid, dim3(kThreads), 0, stream,
                               true, p)
               : launch_kernel(rotary_kernel<kBF16, D, false>, grid, dim3(kThreads), 0, stream,
                               true, p);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int D, bool interleaved, bool bf16, int num_sms,
                          cudaStream_t stream) {
  if (D == 128)
    return bf16 ? launch_t<true, 128>(p, interleaved, num_sms, stream)
                : launch_t<false, 128>(p, interleaved, num_sms, stream);
  return bf16 ? launch_t<true, 64>(p, interleaved, num_sms, stream)
              : launch_t<false, 64>(p, interleaved, num_sms, stream);
}

}  // namespace ps
