// Masked paged attention, decode and verify rows: the split kernel with a mask that is an
// interval of keys per row, scores capped by a tanh, and a bias that falls with the
// distance.
//
//     x_j = c tanh(scale q.K_j / c) - slope_h |p - j|,  lo <= j < hi   (see MaskedAttnParams)
//     out = sum_j softmax_j(x_j) V_j,  zeros for a row without keys
//
// in one pass over the keys with the running maximum and sum (log2 units). One warp streams
// one work item (16 packed rows of one KV head over one split of the context) through its
// own ring of TMA-filled pages, 8 warps an SM, like the causal split kernel; what the mask
// adds:
//   - the plan starts an item at the first page its rows see, so a sliding window costs
//     the window's bytes whatever the context, and pages before it are never read;
//   - a key that no row of the item sees has its V row zeroed in shared memory before the
//     product: 0 * V would keep a NaN of memory that was never written. Only the first and
//     last page can hold one, and with documents the pages of the item's own tokens (a row
//     that starts behind its own position sees nothing, nor does another see its key). Its
//     score is replaced, whatever it is;
//   - a row that has seen no key yet keeps its maximum at -inf and subtracts 0, so that
//     its weights are exactly 0.
// The cap is a polynomial in packed arithmetic where a warp's scores of a page lie within half
// of it, else a polynomial or one ex2 and one reciprocal by the score's size (ps_masked.cuh):
// within 2^-20 of the score, under 2^-14 on one at a cap of 50 (72 in log2 units), against the
// 2^-9 that P's rounding to bf16 costs. The kernel is bound by the bytes of K and V.
//
// Streams (StreamAttnParams) see an interval and the sequence's first keys, j < sinks: an item
// is two runs of pages, the sinks' before the window's, through the same ring one behind the
// other; on the turn from one to the other only the bounds of the rows' keys change. 128 decodes
// of 16 heads on 4, D 128, over a window of 4096 and 4 sinks: 174 us, 0.92 of the measured copy
// peak, as the window alone. Small batches, without a plan: a cluster of up to 8 CTAs for an
// item, whose warps share its pages out and send their joined rows to the row's CTA. One decode
// over a window of 4000, 12 heads on 2: 9.8 us with 8 CTAs, 22.4 with one, bound by each warp's
// chain of steps (about a microsecond a page: the copy's issue, two products, the softmax).
#pragma once

#include <cooperative_groups.h>

#include "ps_common.cuh"
#include "ps_launch.h"
#include "ps_masked.cuh"

namespace ps {

namespace {

// One CTA per SM. Items of 8 rows of 64 elements are light on registers: 16 warps with three
// pages each in flight hide their dependent steps better than 8 with six (contexts to 8191,
// 16 heads of 64 elements, each its own: 285 us with 8 warps, 272 with 16). Items of 128
// elements take 166 registers, and 12 warps with two pages each gained nothing.
template <int D, bool kNarrow, bool kStreamDirect>
struct MaskedSplit {
  static constexpr int kWarps =
      kStreamDirect ? stream_direct_warps(D, kNarrow) : masked_split_warps(D, kNarrow);
  static constexpr int kStages = (D == 128 ? 24 : 48) / kWarps;  // pages in flight per warp
  static constexpr int kRing = kStages + 2;           // item records
  static constexpr int kPage = kBlockSize * D * 2;    // one page of K (or V), one head
  static constexpr int kStage = 2 * kPage;
  static constexpr int kSmem =
      1024 + kWarps * (kStages * kStage + kStages * 8 + kRing * 64);
};

// 8 x 8 16-bit values transposed across the warp: lane 4 a + b holds (a, 2b), (a, 2b + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// kNarrow: items of at most 8 rows (one token of up to 8 query heads per KV head). The
// products are taken transposed, S^T = K Q^T and O^T = V^T P^T, with the 16 keys or 16 of
// the head's elements as the MMA's 16 rows and the item's 8 rows as its 8 columns: half the
// MMAs, scores and accumulators of a 16-row item whose upper half would be empty.
template <class Params, bool kBF16, int D, bool kDirect, bool kNarrow>
__global__ void __launch_bounds__(
    MaskedSplit<D, kNarrow, kDirect && Params::kSinks>::kWarps * 32, 1)
    masked_split_kernel(const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const Params p) {
  using C = MaskedSplit<D, kNarrow, kDirect && Params::kSinks>;
  constexpr int kWarps = C::kWarps;
  constexpr int S = C::kStages, kRing = C::kRing, kPage = C::kPage, kStage = C::kStage;
  constexpr int kBoxes = D / 64, kKSteps = D / 16;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* tiles = smem + warp * S * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kWarps * S * kStage) + warp * S;
  WorkItem* ring =
      reinterpret_cast<WorkItem*>(smem + kWarps * S * kStage + kWarps * S * 8) + warp * kRing;
  const uint32_t tiles_addr = smem_u32(tiles);

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  __syncwarp();
  pdl_wait();  // the plan (or, in direct mode, the work before this call) is complete
  pdl_launch_dependents();

  const int n_items = kDirect ? 0 : *reinterpret_cast<volatile int*>(p.hdr);
  bool first_fetch = true;
  [[maybe_unused]] bool first_scan = true;
  // Streams: p.direct CTAs, a cluster, share the pages of an item; row r is the r % p.direct'th's.
  constexpr bool kClusters = kDirect && Params::kSinks;
  [[maybe_unused]] const int ctas = kClusters ? p.direct : 1, rank = blockIdx.x % ctas;
  [[maybe_unused]] __shared__ int sh_stop;  // a CTA of the cluster has given up
  if constexpr (kClusters) {
    if (threadIdx.x == 0) sh_stop = 0;
    if (ctas > 1) cluster_arrive();
  }
  const bool tile_planned = !kDirect && *reinterpret_cast<volatile int*>(p.hdr + 4) > 0;
  const uint64_t policy = l2_policy_evict_first();

  // ---------------- issue side (runs ahead of compute by up to S pages) -------------
  int iss_page = 0, iss_end = 0, iss_seq = 0, iss_kv = 0;
  [[maybe_unused]] int iss_then = 0, iss_last = 0;  // the window's pages, behind the sinks'
  int bt_base = 0, bt_reg = -1;
  bool no_more = false;
  uint32_t g_issue = 0, ring_tail = 0;

  auto load_bt = [&](int first) {
    bt_base = first;
    const int pg = first + lane;
    bt_reg = pg < iss_end
                 ? __ldg(p.block_tables + static_cast<int64_t>(iss_seq) * p.max_blocks + pg)
                 : -1;
  };

  // Direct mode: the items are the groups of rows of each (sequence, KV head), in order; a CTA
  // takes its own and those a grid's width on. Each warp counts the groups of every sequence
  // (few: the launch has about an item a CTA) to find item idx. The item's record covers every
  // page its rows see; the CTA's warps share the pages out. Lane k returns field k.
  constexpr int kGroup = kNarrow ? 8 : 16;
  int dir_item = blockIdx.x / ctas, dir_items = 0;  // the CTA's item, items in all
  auto direct_item = [&](int idx) -> int {
    int b = -1, q0 = 0, n = 0, L = 0, nth = 0, groups = 0;  // the item's sequence, from its lane
    dir_items = 0;
    int q0a = 0, q1a = 0, La = 0;  // the next 32 sequences, one a lane, loaded ahead
    auto load = [&](int bl) {
      if (bl < p.B) {
        q0a = __ldg(p.qsl + bl);
        q1a = __ldg(p.qsl + bl + 1);
        La = __ldg(p.seq_lens + bl);
      }
    };
    load(lane);
    for (int base = 0; base < p.B; base += 32) {
      const int q0l = q0a, nl = q1a - q0a, Ll = La;
      const bool in = base + lane < p.B, ok = in && p.sequence_ok(q0a, q1a, La);
      load(base + 32 + lane);
      if (in && !ok && blockIdx.x == 0 && warp == 0 && first_scan)
        record_error(p.err, kDevBadSequence);
      const int gl = ok ? (nl * p.G + kGroup - 1) / kGroup : 0;
      int end = gl * p.H_kv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += y;
      }
      const int at = idx - dir_items;  // within these 32 sequences
      const unsigned past = __ballot_sync(0xffffffffu, end > at);
      if (b < 0 && past != 0) {
        const int src = __ffs(past) - 1;
        b = base + src;
        q0 = __shfl_sync(0xffffffffu, q0l, src);
        n = __shfl_sync(0xffffffffu, nl, src);
        L = __shfl_sync(0xffffffffu, Ll, src);
        groups = __shfl_sync(0xffffffffu, gl, src);
        nth = at - (__shfl_sync(0xffffffffu, end, src) - groups * p.H_kv);
      }
      dir_items += __shfl_sync(0xffffffffu, end, 31);
    }
    first_scan = false;
    if (b < 0) return 0;
    const int kv = nth / groups, j = nth - kv * groups;
    const int nrows = min(kGroup, n * p.G - kGroup * j);
    const int i0 = kGroup * j / p.G, i1 = (kGroup * j + nrows - 1) / p.G;
    int pre = 0, lo, s0 = 0, s1 = 0;
    if constexpr (Params::kSinks) {
      lo = p.window_lo(L - n + i0);
      s1 = (min(p.sinks, L - n + i1 + 1) + kBlockSize - 1) / kBlockSize;
    } else {
      pre = p.prefix_len(b, L);
      lo = p.row_lo(q0 + i0, L - n + i0);
    }
    const int hi = max(L - n + i1 + 1, pre);  // one past the last key (at most L)
    const int pe = (hi + kBlockSize - 1) / kBlockSize;
    // (one page at least, the sinks' included)
    const int pb = Params::kSinks ? min(lo / kBlockSize, pe) : min(lo / kBlockSize, pe - 1);
    const int warps = kWarps * ctas, nth_warp = rank * kWarps + warp;
    const int pages = s1 + pe - pb, share = (pages + warps - 1) / warps;
    // the warp's share of the pages, counted from the window's first with the sinks' before it
    const int from = pb - s1 + nth_warp * share, to = min(from + share, pe);
    int first = from, end = to;
    if constexpr (Params::kSinks) {
      s0 = min(nth_warp * share, s1);
      s1 = min(nth_warp * share + share, s1);
      first = max(from, pb);
      end = max(to, first);
    }
    int f = 0;
    f = lane == 0 ? b : f;
    f = lane == 1 ? kv : f;
    f = lane == 2 ? kGroup * j : f;
    f = lane == 3 ? nrows : f;
    f = lane == 4 ? first : f;                   // the warp's pages
    f = lane == 5 ? end : f;
    f = lane == 7 ? 1 : f;                       // one split (lane 6: split 0)
    f = lane == 8 ? L : f;
    f = lane == 9 ? n : f;
    f = lane == 10 ? q0 : f;
    f = lane == 12 ? lo : f;                     // pad[1..3], as the plan has them
    f = lane == 13 ? hi : f;
    f = lane == 14 ? (Params::kSinks ? s0 : pre) : f;
    if constexpr (Params::kSinks) f = lane == 15 ? s1 : f;
    return f;
  };
  int dir_rows = 0, dir_row0 = 0, dir_tok0 = 0, dir_kv = 0;  // the CTA's item, for the join

  // Issue the next page of work into stage g_issue % S; false when nothing is left.
  auto issue_one = [&]() -> bool {
    while (iss_page >= iss_end) {
      if constexpr (Params::kSinks) {
        if (iss_then < iss_last) {  // from the sinks to the window
          iss_page = iss_then;
          iss_end = iss_then = iss_last;
          load_bt(iss_page);
          continue;
        }
      }
      if (no_more) return false;
      int idx = 0;
      if constexpr (kDirect) {
        no_more = !first_fetch;  // one item at a time
        first_fetch = false;
        if (no_more) return false;
        idx = dir_item;
      } else if (first_fetch) {
        // each warp's first item is its own; with tile items planned a CTA's warps take
        // consecutive items, so that the other SMs are free for the tile kernel
        idx = tile_planned ? static_cast<int>(blockIdx.x) * kWarps + warp
                           : warp * static_cast<int>(gridDim.x) + blockIdx.x;
        first_fetch = false;
      } else {
        if (lane == 0) idx = atomicAdd(p.hdr + 1, 1) + static_cast<int>(gridDim.x) * kWarps;
        idx = __shfl_sync(0xffffffffu, idx, 0);
      }
      if (!kDirect && idx >= n_items) {
        no_more = true;
        return false;
      }
      int v;
      if constexpr (kDirect) {
        v = direct_item(idx);
        dir_kv = __shfl_sync(0xffffffffu, v, 1);
        dir_row0 = __shfl_sync(0xffffffffu, v, 2);
        dir_rows = __shfl_sync(0xffffffffu, v, 3);
        dir_tok0 = __shfl_sync(0xffffffffu, v, 10);
      } else v = lane < 16 ? __ldg(reinterpret_cast<const int*>(p.items + idx) + lane) : 0;
      const int pb = __shfl_sync(0xffffffffu, v, 4), pe = __shfl_sync(0xffffffffu, v, 5);
      int sb = 0, se = 0;
      if constexpr (Params::kSinks) {
        sb = __shfl_sync(0xffffffffu, v, 14);
        se = __shfl_sync(0xffffffffu, v, 15);
      }
      if (pe <= pb && se <= sb) continue;  // held by no row
      WorkItem* slot = ring + (ring_tail % kRing);
      if (lane < 16) reinterpret_cast<int*>(slot)[lane] = v;
      ++ring_tail;
      iss_seq = __shfl_sync(0xffffffffu, v, 0);
      iss_kv = __shfl_sync(0xffffffffu, v, 1);
      iss_page = pb;
      iss_end = pe;
      if constexpr (Params::kSinks) {
        iss_then = pb;
        iss_last = pe;
        iss_page = sb;
        iss_end = se;
        if (se <= sb) continue;
      }
      load_bt(iss_page);
    }
    if (iss_page - bt_base >= 32) load_bt(iss_page);
    const int blk = __shfl_sync(0xffffffffu, bt_reg, iss_page - bt_base);
    if (lane == 0) {
      int row = blk * kBlockSize;
      if (blk < 0 || blk >= p.num_blocks) {
        record_error(p.err, kDevBadBlockId);
        row = p.num_blocks * kBlockSize;  // past the tensor: the copy reads zeros
      }
      const uint32_t st = g_issue % S;
      uint8_t* dst = tiles + st * kStage;
      mbar_arrive_expect_tx(&full[st], kStage);
#pragma unroll
      for (int x = 0; x < kBoxes; ++x) {
        tma_load_2d_hint(dst + x * (kBlockSize * 128), &kmap, &full[st], iss_kv * D + x * 64,
                         row, policy);
        tma_load_2d_hint(dst + kPage + x * (kBlockSize * 128), &vmap, &full[st],
                         iss_kv * D + x * 64, row, policy);
      }
    }
    ++iss_page;
    ++g_issue;
    return true;
  };

  // ---------------- compute side ---------------------------------------------------
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t g_comp = 0, ring_head = 0;
  int comp_left = 0, comp_page = 0;
  // position from which a key may be seen by no row though others around it are: the item's
  // first token's, or the prefix's end behind it, where some row of the item sees nothing
  int own_key = 0;
  bool have_item = false;
  [[maybe_unused]] bool in_sinks = false;  // the current page is one of the sinks'
  [[maybe_unused]] int all_lo = 0, all_hi = 0;  // streams: the window's keys that every row sees
  WorkItem cur;
  // per-thread rows of the item: g and g + 8 (narrow: 2 t4 and 2 t4 + 1)
  int row_tok[2], row_h[2], row_pos[2], row_lo[2], row_hi[2];
  float m_run[2], l_run[2], slope[2];
  // wide: O of rows g, g + 8, columns 8 j + 2 t4 ..; narrow: O^T of elements 16 j + g, + 8
  // and rows 2 t4, 2 t4 + 1
  constexpr int kO = kNarrow ? D / 16 : D / 8;
  float o[kO][4];
  uint32_t qa[kKSteps][kNarrow ? 2 : 4];
  const uint16_t* qptr = static_cast<const uint16_t*>(p.q);

  auto start_item = [&]() {
    __syncwarp();  // the ring slot was written by lanes 0..15
    cur = ring[ring_head % kRing];
    ++ring_head;
    comp_page = cur.page_begin;
    comp_left = cur.page_end - cur.page_begin;
    if constexpr (Params::kSinks) {
      in_sinks = cur.pad[4] > cur.pad[3];
      if (in_sinks) {
        comp_page = cur.pad[3];
        comp_left += cur.pad[4] - cur.pad[3];
      }
    }
    have_item = true;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int rr = kNarrow ? 2 * t4 + r : g + 8 * r;
      row_tok[r] = -1;
      row_h[r] = row_pos[r] = row_lo[r] = row_hi[r] = 0;
      slope[r] = 0.f;
      if (rr < cur.nrows) {
        const int R = cur.row0 + rr;
        const int i = R / p.G;
        row_tok[r] = cur.tok0 + i;
        row_h[r] = cur.kv * p.G + (R - i * p.G);
        row_pos[r] = cur.ctx_len - cur.n_query + i;
        if constexpr (Params::kSinks) {
          row_lo[r] = p.window_lo(row_pos[r]);
          row_hi[r] = row_pos[r] + 1;
        } else {
          row_lo[r] = p.row_lo(row_tok[r], row_pos[r]);
          row_hi[r] = max(row_pos[r] + 1, cur.pad[3]);
        }
        if (p.slopes != nullptr) slope[r] = -kLog2e * __ldg(p.slopes + row_h[r]);
      }
      m_run[r] = -INFINITY;
      l_run[r] = 0.f;
    }
    if constexpr (Params::kSinks) {
      const int pos0 = cur.ctx_len - cur.n_query;
      all_lo = p.window_lo(pos0 + (cur.row0 + cur.nrows - 1) / p.G);
      all_hi = pos0 + cur.row0 / p.G + 1;
    }
    own_key = 0x7fffffff - kBlockSize;
    if constexpr (!Params::kSinks) {
      const bool empty = row_lo[0] > row_pos[0] || row_lo[1] > row_pos[1];
      const int pos0 = __shfl_sync(0xffffffffu, row_pos[0], 0);  // the item's first row's
      if (__any_sync(0xffffffffu, empty)) own_key = max(pos0, cur.pad[3]);
    }
#pragma unroll
    for (int j = 0; j < kO; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    // query fragments straight from global memory: rows g (and, wide, g + 8); columns 2 t4,
    // 2 t4 + 1 and 8 further on
#pragma unroll
    for (int r = 0; r < (kNarrow ? 1 : 2); ++r) {
      const int R = cur.row0 + g + 8 * r, i = R / p.G;
      const bool in = g + 8 * r < cur.nrows;
      const uint16_t* src = qptr + (static_cast<int64_t>(cur.tok0 + i) * p.H_q + cur.kv * p.G +
                                    (R - i * p.G)) * D + 2 * t4;
#pragma unroll
      for (int kk = 0; kk < kKSteps; ++kk) {
        const uint32_t lo = in ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16)) : 0;
        const uint32_t hi = in ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + 8)) : 0;
        if constexpr (kNarrow) {
          qa[kk][0] = lo;
          qa[kk][1] = hi;
        } else {
          qa[kk][r] = lo;
          qa[kk][2 + r] = hi;
        }
      }
    }
  };

  auto finish_item = [&]() {
#pragma unroll
    for (int r = 0; r < 2; ++r) {  // row sums across the lanes sharing a row
#pragma unroll
      for (int x = kNarrow ? 4 : 1; x < (kNarrow ? 32 : 4); x <<= 1)
        l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], x);
    }
    bool any[2], held[2];
    float inv[2];
    int64_t part[2];  // the row's partial entry, or -1: straight to the output
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      // a row without keys here gives zeros, whatever the products left in o
      any[r] = !(l_run[r] == 0.f);
      inv[r] = any[r] ? 1.f / l_run[r] : 0.f;
      part[r] = -1;
      const int ns_t = row_tok[r] < 0 ? 0 : __ldg(p.tok_ns + row_tok[r]);
      held[r] = cur.split < ns_t;  // else this split does not hold the row
      if (held[r] && ns_t > 1) {
        part[r] = static_cast<int64_t>(__ldg(p.tok_base + row_tok[r])) + cur.split * p.H_q + row_h[r];
        if (kNarrow ? g == 0 : t4 == 0)
          p.part_lse[part[r]] = any[r] ? m_run[r] + __log2f(l_run[r]) : -INFINITY;
      }
    }
    auto norm = [&](float x, int r) { return any[r] ? x * inv[r] : 0.f; };
    if constexpr (kNarrow) {
      // partials: eight lanes write a row's 8 consecutive elements
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (!held[r] || part[r] < 0) continue;
        float* dst = p.part_o + part[r] * D + g;
#pragma unroll
        for (int j = 0; j < kO; ++j) {
          dst[16 * j] = norm(o[j][r], r);
          dst[16 * j + 8] = norm(o[j][2 + r], r);
        }
      }
      // outputs: transposed back, lane 4 a + b then has row a's elements 2 b, 2 b + 1. The
      // rows of an item are of one token or of tokens split alike or not: row g's fate is
      // that of the lane that holds its sums.
      const bool direct0 = __shfl_sync(0xffffffffu, held[0] && part[0] < 0, g >> 1);
      const bool direct1 = __shfl_sync(0xffffffffu, held[1] && part[1] < 0, g >> 1);
      const int R = cur.row0 + g, i = R / p.G;
      uint32_t* dst = reinterpret_cast<uint32_t*>(
          static_cast<uint16_t*>(p.out) +
          (static_cast<int64_t>(cur.tok0 + i) * p.H_q + cur.kv * p.G + (R - i * p.G)) * D + 2 * t4);
      const bool mine = (g & 1) ? direct1 : direct0;
#pragma unroll
      for (int j = 0; j < kO; ++j) {
        const uint32_t lo = transpose8(pack2<kBF16>(norm(o[j][0], 0), norm(o[j][1], 1)));
        const uint32_t hi = transpose8(pack2<kBF16>(norm(o[j][2], 0), norm(o[j][3], 1)));
        if (mine) {
          dst[8 * j] = lo;
          dst[8 * j + 4] = hi;
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (!held[r]) continue;
        if (part[r] < 0) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(
              static_cast<uint16_t*>(p.out) +
              (static_cast<int64_t>(row_tok[r]) * p.H_q + row_h[r]) * D + 2 * t4);
#pragma unroll
          for (int j = 0; j < kO; ++j)
            dst[j * 4] = pack2<kBF16>(norm(o[j][2 * r], r), norm(o[j][2 * r + 1], r));
        } else {
          float2* dst = reinterpret_cast<float2*>(p.part_o + part[r] * D + 2 * t4);
#pragma unroll
          for (int j = 0; j < kO; ++j)
            dst[j * 4] = make_float2(norm(o[j][2 * r], r), norm(o[j][2 * r + 1], r));
        }
      }
    }
    have_item = false;
  };

  bool aborted = false;
[[maybe_unused]] next_item:  // (direct mode only)
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    m_run[r] = -INFINITY;
    l_run[r] = 0.f;
  }
  const uint32_t g_first = g_comp;
  for (int s = 0; s < S; ++s)  // fill the ring
    if (!issue_one()) break;

  while (true) {
    if (comp_left == 0) {
      if (!kDirect && have_item) finish_item();
      if (ring_head == ring_tail) break;  // everything issued has been computed
      start_item();
    }
    const uint32_t st = g_comp % S;
    if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (g_comp / S) & 1))) {
      if (lane == 0) record_error(p.err, kDevWaitTimeout);
      aborted = true;
      break;
    }
    const uint32_t kbase = tiles_addr + st * kStage;
    const uint32_t vbase = kbase + kPage;
    const int key_base = comp_page * kBlockSize;

    // the keys that some row of the item sees of this page, and each row
    int item_lo = cur.pad[1], item_hi = cur.pad[2];
    int see_lo[2] = {row_lo[0], row_lo[1]}, see_hi[2] = {row_hi[0], row_hi[1]};
    if constexpr (Params::kSinks) {
      if (in_sinks) {
        item_lo = see_lo[0] = see_lo[1] = 0;
        item_hi = min(item_hi, p.sinks);
        see_hi[0] = min(see_hi[0], p.sinks);
        see_hi[1] = min(see_hi[1], p.sinks);
      }
    }
    // V rows of keys that no row of the item sees: zero
    if (key_base < item_lo || key_base + kBlockSize > item_hi ||
        key_base + kBlockSize > own_key) {
      const int mine = key_base + (lane & 15);
      const unsigned dead = __ballot_sync(
          0xffffffffu, mine < item_lo || mine >= item_hi ||
                           (!Params::kSinks &&
                            p.key_unseen(mine, own_key, item_hi,
                                         cur.tok0 - (cur.ctx_len - cur.n_query))));
      uint8_t* v = tiles + st * kStage + kPage;
#pragma unroll
      for (int i = lane; i < kPage / 16; i += 32)
        if (dead >> (i % (kBlockSize * 8)) / 8 & 1u)
          reinterpret_cast<uint4*>(v)[i] = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }

    if constexpr (kNarrow) {
      // S^T = K Q^T for the page's 16 keys: lane holds keys g, g + 8 of rows 2 t4, 2 t4 + 1
      // (two accumulators, even and odd k steps, to halve the dependent mma chain)
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      {
        float s2[4] = {0.f, 0.f, 0.f, 0.f};
        const int mi = lane >> 3, key = (mi & 1) * 8 + (lane & 7);
#pragma unroll
        for (int kk = 0; kk < kKSteps; ++kk) {
          const int chunk = 2 * kk + (mi >> 1);
          const uint32_t addr = kbase + (chunk >> 3) * (kBlockSize * 128) + swz128(key, chunk & 7);
          uint32_t a[4];
          ldsm_x4(addr, a[0], a[1], a[2], a[3]);
          mma_16816<kBF16>((kk & 1) ? s2 : s, a, qa[kk][0], qa[kk][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += s2[e];
      }
      // the scores in log2 units: capped, biased, masked (element e: key g + 8 (e / 2), row e % 2)
      if (p.cap_log2 > 0.f) {
        cap_scores<4>(s, p);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] *= p.scale_log2;
      }
      bool up = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = e & 1, key = key_base + g + 8 * (e >> 1);
        float x = s[e];
        if constexpr (!Params::kSinks)
          x = fmaf(slope[r], fabsf(static_cast<float>(row_pos[r] - key)), x);
        s[e] = key >= see_lo[r] && key < see_hi[r] ? x : -INFINITY;
        up |= s[e] > m_run[r] + 8.f;
      }
      // The reference moves only when some score is more than 2^8 above it (P then stays
      // within 2^8, a sum of any length in fp32): the maxima across lanes and the rescaling
      // of O are paid a few times an item, not every page.
      if (__any_sync(0xffffffffu, up)) {
        float alpha[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = fmaxf(s[r], s[2 + r]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          const float m_new = fmaxf(m_run[r], mx);
          alpha[r] = m_run[r] == -INFINITY ? 1.f : fast_exp2(m_run[r] - m_new);
          m_run[r] = m_new;
          l_run[r] *= alpha[r];
        }
        const float2 a2 = make_float2(alpha[0], alpha[1]);
#pragma unroll
        for (int j = 0; j < kO; ++j) {
          const float2 u = fmul2(make_float2(o[j][0], o[j][1]), a2);
          const float2 v = fmul2(make_float2(o[j][2], o[j][3]), a2);
          o[j][0] = u.x;
          o[j][1] = u.y;
          o[j][2] = v.x;
          o[j][3] = v.y;
        }
      }
      uint32_t pt[2];  // P^T: keys g (g + 8), rows 2 t4, 2 t4 + 1
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
          x[r] = fast_exp2(s[2 * h + r] - (m_run[r] == -INFINITY ? 0.f : m_run[r]));
        pt[h] = pack2<kBF16>(x[0], x[1]);
        // the row sums use the rounded P the tensor core multiplies with
        float2 acc = make_float2(l_run[0], l_run[1]);
        add_pair_exact<kBF16>(acc, pt[h]);
        l_run[0] = acc.x;
        l_run[1] = acc.y;
      }
      const uint32_t b0 = transpose8(pt[0]), b1 = transpose8(pt[1]);
      {  // O^T += V^T P^T: the V page is [key][d], read transposed
        const int mi = lane >> 3, key = (mi >> 1) * 8 + (lane & 7);
#pragma unroll
        for (int j = 0; j < kO; ++j) {
          const int chunk = 2 * j + (mi & 1);
          const uint32_t addr = vbase + (chunk >> 3) * (kBlockSize * 128) + swz128(key, chunk & 7);
          uint32_t a[4];
          ldsm_x4_t(addr, a[0], a[1], a[2], a[3]);
          mma_16816<kBF16>(o[j], a, b0, b1);
        }
      }
    } else {
      // S = Q K^T for the page's 16 keys: two n8 tiles, two accumulators per tile (even and
      // odd k steps) to halve the dependent mma chain
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        float s2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int mi = lane >> 3, rr = lane & 7;
        const int key = (mi >> 1) * 8 + rr;
#pragma unroll
        for (int kk = 0; kk < kKSteps; ++kk) {
          const int chunk = 2 * kk + (mi & 1);
          const uint32_t addr = kbase + (chunk >> 3) * (kBlockSize * 128) + swz128(key, chunk & 7);
          uint32_t b0, b1, b2, b3;
          ldsm_x4(addr, b0, b1, b2, b3);
          float (*acc)[4] = (kk & 1) ? s2 : s;
          mma_16816<kBF16>(acc[0], qa[kk], b0, b1);
          mma_16816<kBF16>(acc[1], qa[kk], b2, b3);
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] += s2[nt][e];
      }
      // the scores in log2 units: capped, biased, masked
      if (p.cap_log2 > 0.f) {
        cap_scores<4>(s[0], p);
        cap_scores<4>(s[1], p);
      } else {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] *= p.scale_log2;
      }
      const int key0 = key_base + 2 * t4;
      float mx[2] = {-INFINITY, -INFINITY};
      // (streams: the reference moves only when some score is more than 2^8 above it, as above)
      bool up = !Params::kSinks;
      // (streams: no page is masked but the windows' first and last and the sinks'; 36 sequences of
      // 5 tokens over 1000 keys: 15.8 us with the test of every score, 14.8)
      if (!Params::kSinks || in_sinks || key_base < all_lo || key_base + kBlockSize > all_hi) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = e >> 1, key = key0 + nt * 8 + (e & 1);
            float x = s[nt][e];
            if constexpr (!Params::kSinks)
              x = fmaf(slope[r], fabsf(static_cast<float>(row_pos[r] - key)), x);
            s[nt][e] = key >= see_lo[r] && key < see_hi[r] ? x : -INFINITY;
          }
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[nt][e]);
      if constexpr (Params::kSinks)
        up = __any_sync(0xffffffffu, mx[0] > m_run[0] + 8.f || mx[1] > m_run[1] + 8.f);
      float m_use[2] = {m_run[0], m_run[1]};
      if (up) {
        float alpha[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
          const float m_new = fmaxf(m_run[r], mx[r]);
          m_use[r] = m_new == -INFINITY ? 0.f : m_new;
          alpha[r] = fast_exp2(m_run[r] - m_use[r]);
          m_run[r] = m_new;
          l_run[r] *= alpha[r];
        }
        const float2 a0 = make_float2(alpha[0], alpha[0]), a1 = make_float2(alpha[1], alpha[1]);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const float2 u = fmul2(make_float2(o[j][0], o[j][1]), a0);
          const float2 w = fmul2(make_float2(o[j][2], o[j][3]), a1);
          o[j][0] = u.x;
          o[j][1] = u.y;
          o[j][2] = w.x;
          o[j][3] = w.y;
        }
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r) m_use[r] = m_run[r] == -INFINITY ? 0.f : m_run[r];
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = fast_exp2(s[nt][e] - m_use[e >> 1]);
      uint32_t pa[4];
      pa[0] = pack2<kBF16>(s[0][0], s[0][1]);
      pa[1] = pack2<kBF16>(s[0][2], s[0][3]);
      pa[2] = pack2<kBF16>(s[1][0], s[1][1]);
      pa[3] = pack2<kBF16>(s[1][2], s[1][3]);
      // the row sums use the rounded P the tensor core multiplies with
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float2 acc = make_float2(l_run[r], 0.f);
        add_pair_exact<kBF16>(acc, pa[r]);
        add_pair_exact<kBF16>(acc, pa[2 + r]);
        l_run[r] = acc.x + acc.y;
      }
      {  // O += P V: the V page is [key][d], read transposed
        const int mi = lane >> 3, rr = lane & 7;
        const int key = (mi & 1) * 8 + rr;
#pragma unroll
        for (int np = 0; np < D / 16; ++np) {
          const int chunk = 2 * np + (mi >> 1);
          const uint32_t addr = vbase + (chunk >> 3) * (kBlockSize * 128) + swz128(key, chunk & 7);
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(addr, b0, b1, b2, b3);
          mma_16816<kBF16>(o[2 * np], pa, b0, b1);
          mma_16816<kBF16>(o[2 * np + 1], pa, b2, b3);
        }
      }
    }
    ++g_comp;
    ++comp_page;
    --comp_left;
    if constexpr (Params::kSinks) {
      if (in_sinks && comp_page == cur.pad[4]) {
        in_sinks = false;
        comp_page = cur.page_begin;
      }
    }
    __syncwarp();
    fence_proxy_async_smem();
    issue_one();
  }
  if (aborted) {
    // let the copies already issued land before the CTA's shared memory goes away
    for (uint32_t gg = g_comp; gg < g_issue; ++gg) mbar_wait(&full[gg % S], (gg / S) & 1, 1u << 20);
  }
  if constexpr (kDirect) {
    // The warps' shares of the item's pages joined: each leaves its O (not normalised) in its
    // own stages, which hold no page any more, and its rows' maxima and sums. (A row of O takes a
    // few columns more, so that the rows that a store's lanes write lie in other banks.)
    constexpr int kRowO = D + (kNarrow ? 4 : 8);
    static_assert(kGroup * kRowO * 4 <= S * kStage, "O of a warp");
    __shared__ float sh_m[kWarps][kGroup], sh_l[kWarps][kGroup];
    const bool worked = g_comp != g_first && !aborted;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int x = kNarrow ? 4 : 1; x < (kNarrow ? 32 : 4); x <<= 1)
        l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], x);
      const int row = kNarrow ? 2 * t4 + r : g + 8 * r;
      if (kNarrow ? g == 0 : t4 == 0) {
        sh_m[warp][row] = worked ? m_run[r] : -INFINITY;
        sh_l[warp][row] = worked ? l_run[r] : 0.f;
      }
      if (worked) {
        float* dst = reinterpret_cast<float*>(tiles) + row * kRowO;
#pragma unroll
        for (int j = 0; j < kO; ++j) {
          if constexpr (kNarrow) {
            dst[16 * j + g] = o[j][r];
            dst[16 * j + 8 + g] = o[j][2 + r];
          } else {
            *reinterpret_cast<float2*>(dst + j * 8 + 2 * t4) =
                make_float2(o[j][2 * r], o[j][2 * r + 1]);
          }
        }
      }
    }
    __syncthreads();
    // threads of a row, pairs of columns of each
    constexpr int kShare = kWarps * 32 / kGroup, kLanes = kShare >= 32 ? 32 : 16;
    constexpr int kPairs = D / 2 / kLanes;
    static_assert(kPairs * kLanes * 2 == D && kLanes * kGroup <= kWarps * 32, "join");
    const int row = threadIdx.x / kLanes, col = 2 * (threadIdx.x % kLanes);
    auto store_row = [&](int row, int col, const float2 (&acc)[kPairs], float sum) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int R = dir_row0 + row, i = R / p.G;
      uint32_t* dst = reinterpret_cast<uint32_t*>(
          static_cast<uint16_t*>(p.out) +
          (static_cast<int64_t>(dir_tok0 + i) * p.H_q + dir_kv * p.G + (R - i * p.G)) * D + col);
#pragma unroll
      for (int e = 0; e < kPairs; ++e)
        dst[kLanes * e] = pack2<kBF16>(acc[e].x * inv, acc[e].y * inv);
    };
    // (clusters: what the CTAs send of this one's rows: O, and maximum and sum)
    __shared__ float2 sh_o[kClusters ? kGroup * D / 2 : 1], sh_all[kClusters ? kGroup : 1];
    [[maybe_unused]] const auto cluster = cooperative_groups::this_cluster();
    if constexpr (kClusters)
      if (ctas > 1) cluster_wait();  // (every CTA has begun, or read what it was sent before)
    if (row < dir_rows) {
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) M = fmaxf(M, sh_m[k][row]);
      float2 acc[kPairs];
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < kPairs; ++e) acc[e] = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float m = sh_m[k][row];
        // (a warp whose share holds no key of the row is left out: its O may be anything)
        if (sh_l[k][row] == 0.f) continue;
        const float wgt = fast_exp2(m - M);
        sum += wgt * sh_l[k][row];
        const float* src =
            reinterpret_cast<const float*>(smem + k * S * kStage) + row * kRowO + col;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          const float2 o2 = *reinterpret_cast<const float2*>(src + 2 * kLanes * e);
          acc[e].x += wgt * o2.x;
          acc[e].y += wgt * o2.y;
        }
      }
      if (ctas == 1) {
        store_row(row, col, acc, sum);
      } else if constexpr (kClusters) {  // to the row's CTA
        const int at = rank * (kGroup / ctas) + row / ctas;
        float2* dst = cluster.map_shared_rank(sh_o, row % ctas) + (at * D + col) / 2;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) dst[kLanes * e] = acc[e];
        if (col == 0) cluster.map_shared_rank(sh_all, row % ctas)[at] = make_float2(M, sum);
      }
    }
    if constexpr (kClusters) {
      if (ctas > 1) {
        if (__syncthreads_or(aborted) && threadIdx.x < ctas)
          *cluster.map_shared_rank(&sh_stop, threadIdx.x) = 1;
        cluster_arrive();
        cluster_wait();
        if (row < dir_rows && row % ctas == rank) {
          const int at = row / ctas, step = kGroup / ctas;
          float M = -INFINITY;
          for (int c = 0; c < ctas; ++c) M = fmaxf(M, sh_all[at + c * step].x);
          float2 acc[kPairs];
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < kPairs; ++e) acc[e] = make_float2(0.f, 0.f);
          for (int c = 0; c < ctas; ++c) {
            const float2 ms = sh_all[at + c * step];
            if (ms.y == 0.f) continue;
            const float wgt = fast_exp2(ms.x - M);
            sum += wgt * ms.y;
            const float2* src = sh_o + ((at + c * step) * D + col) / 2;
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
              acc[e].x += wgt * src[kLanes * e].x;
              acc[e].y += wgt * src[kLanes * e].y;
            }
          }
          store_row(row, col, acc, sum);
        }
        dir_item += gridDim.x / ctas;
        if (dir_item >= dir_items || sh_stop != 0) return;  // (the same in every CTA)
        fence_proxy_async_smem();
        cluster_arrive();
        no_more = have_item = false;
        first_fetch = true;
        goto next_item;
      }
    }
    // the CTA's next item, once the stages that held O have been read
    dir_item += gridDim.x;
    fence_proxy_async_smem();
    if (__syncthreads_or(aborted) == 0 && dir_item < dir_items) {
      no_more = have_item = false;
      first_fetch = true;
      goto next_item;
    }
  }
}

template <bool kBF16, int D, bool kDirect, bool kNarrow, class Params>
cudaError_t launch_split_t(const Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                           int ctas, cudaStream_t stream, bool pdl) {
  using C = MaskedSplit<D, kNarrow, kDirect && Params::kSinks>;
  constexpr int smem = C::kSmem;
  auto kern = masked_split_kernel<Params, kBF16, D, kDirect, kNarrow>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_smem_limit(kern, smem, done);
  if (e != cudaSuccess) return e;
  if constexpr (kDirect && Params::kSinks) {
    if (p.direct > 1)
      return launch_cluster(kern, static_cast<unsigned>(ctas) * p.direct, p.direct, C::kWarps * 32,
                            smem, stream, kmap, vmap, p);
  }
  return launch_kernel(kern, dim3(ctas), dim3(C::kWarps * 32), smem, stream, pdl, kmap, vmap, p);
}

template <bool kDirect, bool kNarrow, class Params>
cudaError_t launch_split_d(const Params& p, bool bf16, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, int ctas, cudaStream_t stream, bool pdl) {
  if (p.D == 128)
    return bf16 ? launch_split_t<true, 128, kDirect, kNarrow>(p, kmap, vmap, ctas, stream, pdl)
                : launch_split_t<false, 128, kDirect, kNarrow>(p, kmap, vmap, ctas, stream, pdl);
  return bf16 ? launch_split_t<true, 64, kDirect, kNarrow>(p, kmap, vmap, ctas, stream, pdl)
              : launch_split_t<false, 64, kDirect, kNarrow>(p, kmap, vmap, ctas, stream, pdl);
}

template <class Params>
cudaError_t launch_split_any(const Params& p, bool bf16, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, int ctas, cudaStream_t stream, bool pdl) {
  if (p.direct)
    return p.group_rows == 8 ? launch_split_d<true, true>(p, bf16, kmap, vmap, ctas, stream, pdl)
                             : launch_split_d<true, false>(p, bf16, kmap, vmap, ctas, stream, pdl);
  return p.group_rows == 8 ? launch_split_d<false, true>(p, bf16, kmap, vmap, ctas, stream, pdl)
                           : launch_split_d<false, false>(p, bf16, kmap, vmap, ctas, stream, pdl);
}

}  // namespace

}  // namespace ps
