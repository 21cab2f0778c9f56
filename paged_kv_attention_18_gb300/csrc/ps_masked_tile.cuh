// Masked paged attention, chunks of new tokens: the tcgen05 tile kernel with a mask that is
// an interval of keys per row, scores capped by a tanh, and a bias that falls with the
// distance (see ps_masked_split.cuh for the formulas).
//
// One work item is a pair of query tiles A and B of one sequence and one KV head (up to 128
// packed rows each) over one split of the context; both share each tile of 128 keys:
//     S_g = Q_g K^T   (A = Q_g in shared memory, B = K)     -> TMEM
//     P_g = 2^(x(S_g) - m), online row maximum and sum      (softmax group g)
//     O_g += P_g V    (A = P_g in TMEM, B = V)              -> TMEM
// The warp roles are the causal tile kernel's: warp 0 items, Q and K; warp 2 V; warp 1 TMEM
// and every MMA; warp 3 the K/V watcher; from warp 4 the softmax groups of A and B, with one
// thread for a query row or two (kSoftmaxWarps).
// Bound: a group's chain S -> softmax -> PV -> next S (S overwrites P, so they cannot
// overlap), the two groups filling each other's gaps. 4 x 2048 tokens, each over 8192 keys, 32/8
// heads, D 128, 962 GFLOP: masks alone 670 us (1.44 PFLOP/s, 0.74 of the measured burst peak),
// capped 800 (bf16) and 877 (fp16), biased 777, both 997 (bf16) and 1020 (fp16).
// What the mask adds:
//   - an item's keys start at the first page its rows see and end with the last, so a
//     window or a packed document costs its own keys only;
//   - the watcher zeroes, before a V tile is handed to the tensor core, the V rows of keys
//     that no row of the item sees (on its first and last page, and with documents among the
//     item's own tokens): 0 * V would keep a NaN of memory that was never written;
//   - a key tile inside every row's interval skips the mask; in others a row drops the
//     columns outside [lo, hi);
//   - rows without keys get zeros, and -inf as the log-sum of a split that holds them.
// Streams (StreamAttnParams): the sinks' pages and the window's form one run of key tiles
// (ItemTiles), and a row drops the columns outside its window that are not its sinks'. As a tile
// of their own, of which 4 keys count, the sinks cost as much as 128 keys more: 4 x 2048 tokens
// over 8192 keys, 32/8 heads, D 128, bf16, 4 sinks: 239 against 225 us at a window of 2000, 92
// against 79 at 128. With masks by words (drop_unseen) these take 212 (206 GFLOP: 0.97 PFLOP/s,
// 0.49 of the measured burst peak) and 69. What is left is the items' own: 5 or 6 of an item's 30
// us are its first tile's, with the row's first maximum, and the epilogue.
#pragma once

#include <type_traits>

#include "ps_common.cuh"
#include "ps_launch.h"
#include "ps_masked.cuh"
#include "ps_tc05.cuh"

namespace ps {

namespace {

constexpr int kRows = 128;        // query rows per tile (MMA M)
constexpr int kKeys = 128;        // keys per KV tile (MMA N of S, K of PV) = 8 pages
constexpr int kPagesPerTile = kKeys / kBlockSize;
constexpr int kSub = kRows * 128; // bytes of one [128 rows x 64 elements] swizzled sub-tile
constexpr int kKStages = 3;       // K tile stages (freed once both products S have read them)
constexpr int kVStages = 2;       // V tile stages (freed once both products PV have read them)
constexpr int kItemRing = 4;     // item indices handed from the fetching warp to the others
// Softmax warps: one for every 32 query rows, or two (kDuo) with half of a key tile's columns
// each where a cap or a bias makes the softmax the longest part. (4 x 2048 tokens, contexts to
// 8192, 32/8 heads, D 128: capped 729 us with one, 580 with two; masks alone 486 and 495, and
// short documents, 1000 tokens of up to 300 each, 28 and 33: the two must agree on a row's
// reference.)
template <bool kDuo>
constexpr int kSoftmaxWarps = kDuo ? 16 : 8;
template <bool kDuo>
constexpr int kThreads = 128 + 32 * kSoftmaxWarps<kDuo>;
constexpr int kRescaleExp = 8;  // rescale O only when P sums to 2^8 or more
// A larger jump inside a tile moves the reference at once; below it P can reach 2^kMove,
// which must stay finite in the 16-bit type (fp16 tops out near 2^16, bf16 near 2^128).
template <bool kBF16>
constexpr float kMoveLog2 = kBF16 ? 64.f : 15.f;
// Exponent (biased, as in fp32) from which a half row's sum of P is too large: every P is
// below 2 to the power of it less 127 otherwise (bf16: 2^64, as above; fp16: 2^22, so none of
// 64 finite values overflowed). Such a sum (or an infinite one) sends the tile through the
// max and the reference move.
template <bool kBF16>
constexpr uint32_t kSumExp = kBF16 ? 127 + 64 : 127 + 22;
// The same bound for a 64-column half taken by one warp.
template <bool kBF16>
constexpr float kHalfSumMax = kBF16 ? 18446744073709551616.f : 4194304.f;
constexpr float kFixedCapLog2 = 73.f;  // caps up to 50.6 keep a fixed reference (bf16)
constexpr float kFixedLeastLog2 = -86.f;  // the least P against it (see `fixed`)
constexpr uint32_t kTmemCols = 512;

// TMEM columns of softmax group g: S (and P over it) at g*256, O at g*256 + 128
__host__ __device__ constexpr uint32_t col_s(int g) { return g * 256u; }
__host__ __device__ constexpr uint32_t col_o(int g) { return g * 256u + 128u; }

template <int D>
struct TileSmem {
  static constexpr int kQ = (D / 64) * kSub;  // one query tile
  static constexpr int kK = (D / 64) * kSub;  // one K or V tile (128 keys)
  static constexpr int kOffQ = 0;             // query tiles A, B
  static constexpr int kOffK = kOffQ + 2 * kQ;
  static constexpr int kOffV = kOffK + kKStages * kK;
  static constexpr int kOffBar = kOffV + kVStages * kK;
  static constexpr int kOffItems = kOffBar + 512;             // work items in flight
  static constexpr int kOffPair = kOffItems + 2 * kItemRing * 64;  // two warps' exchanges
  static constexpr int kBytes = kOffPair + 1024 + 1024;            // + alignment slack
};
static_assert(TileSmem<128>::kBytes <= 232448, "tile kernel shared memory");

struct TileBars {
  uint64_t q_full[2], q_empty[2];  // query tiles A and B, each freed after its last S
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t pair[8];  // the two warps that share the rows of a (group, quarter)
  uint64_t mma_final;
  uint64_t item_full[kItemRing], item_empty[kItemRing];
  int item_idx[kItemRing];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(TileBars) <= 512, "barrier block");

// An item fits this launch: a sequence and KV head of the batch, a page range inside the
// block table, and query rows inside the packed batch. Every role checks each item the
// same way and skips one that does not fit, so no role reads or writes outside its
// buffers on a plan it cannot use.
template <class Params>
__device__ __forceinline__ bool tile_item_ok(const WorkItem& w, const Params& p) {
  if (Params::kSinks && (w.pad[3] < 0 || w.pad[4] < w.pad[3] || w.pad[4] > p.max_blocks))
    return false;
  if (w.seq < 0 || w.seq >= p.B || w.kv < 0 || w.kv >= p.H_kv) return false;
  if (w.page_begin < 0 || w.page_end > p.max_blocks) return false;
  if (w.tok0 < 0 || w.row0 < 0 || w.nrows <= 0 || w.pad[0] < 0) return false;
  const int last_row = w.row0 + (w.pad[0] > 0 ? p.tpt * p.G + w.pad[0] : w.nrows) - 1;
  return w.tok0 + last_row / p.G < p.T;
}

// The key tiles of an item: its run of pages, or its two runs one behind the other, the sinks'
// first, eight pages a tile (the last one's rest is filled with zeros). Columns are counted from
// the window's first key, so those of the sinks' pages lie before it.
template <class Params>
struct ItemTiles {
  int pb, pe, nt;      // the window's pages (all of them without sinks); key tiles
  int sb = 0, sp = 0;  // the sinks' first page, their number
  __device__ __forceinline__ explicit ItemTiles(const WorkItem& w)
      : pb(w.page_begin), pe(w.page_end) {
    if constexpr (Params::kSinks) {
      sb = w.pad[3];
      sp = w.pad[4] - sb;
    }
    const int n = sp + pe - pb;
    nt = n > 0 ? (n + kPagesPerTile - 1) / kPagesPerTile : 0;
  }
  // key of tile j's first column, as if all of its pages were the window's
  __device__ __forceinline__ int key0(int j) const {
    return (pb - sp + j * kPagesPerTile) * kBlockSize;
  }
  // columns of tile j that hold sinks' pages (0 or less: none), and the key of its first
  __device__ __forceinline__ int sink_cols(int j) const {
    return Params::kSinks ? (sp - j * kPagesPerTile) * kBlockSize : 0;
  }
  __device__ __forceinline__ int sink_key0(int j) const {
    return (sb + j * kPagesPerTile) * kBlockSize;
  }
  // columns, from the item's first, of sinks that the row at position `pos` sees
  __device__ __forceinline__ int sunk(const Params& p, int pos) const {
    if constexpr (Params::kSinks)
      return min(sp * kBlockSize, min(p.sinks, pos + 1) - sb * kBlockSize);
    else
      return 0;
  }
  // page i of the item
  __device__ __forceinline__ int page(int i) const { return i < sp ? sb + i : pb + i - sp; }
};

// 32 columns of scores, those outside [low, lim] dropped (streams: but not those below `sunk`). One
// word has the columns that are kept, so that a column costs a test of a bit and a select in place
// of up to three comparisons. (6 chunks of 1000 in documents behind a prefix, 14/2 heads, D 64: 33.4
// us with those, 29.3.)
template <class Params>
__device__ __forceinline__ void drop_unseen(uint32_t* v, int lim, int low, int sunk) {
  auto from = [](int n) { return __funnelshift_lc(0u, ~0u, max(n, 0)); };  // columns n and on
  uint32_t kept = from(low) & ~from(lim + 1);
  if constexpr (Params::kSinks) kept |= ~from(sunk);
  if (__all_sync(0xffffffffu, kept == ~0u)) return;  // (a warp's rows are few tokens)
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(kept >> e & 1u)) v[e] = __float_as_uint(-INFINITY);
}

}  // namespace

// kDirect: no plan. Each CTA derives its items from seq_lens and qsl (every sequence
// unsplit, its query-tile pairs longest first).
// kCap: 0 none, 1 up to kLargeCapLog2, 2 beyond (the exact form of small scores in every tile; as
// a branch inside it made the kernel larger and its other caps 1.5 % slower).
template <class Params, bool kBF16, int D, bool kDirect, int kCap, bool kBias>
__global__ void __launch_bounds__(kThreads<(kCap > 0 || kBias)>, 1)
    masked_tile_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ CUtensorMap qmap, const Params p) {
  static_assert(!(Params::kSinks && kBias), "a stream's tiles go in order");
  using L = TileSmem<D>;
  constexpr int kHalves = D / 64;
  constexpr bool kDuo = kCap > 0 || kBias;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();

  // The set-up (barriers, TMEM, zeroed query rows, descriptor prefetch) touches only this
  // CTA's own state, so it runs while the kernels before this one finish.
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  TileBars* bars = reinterpret_cast<TileBars*>(smem + L::kOffBar);
  // Records of the items in flight: item it's record sits in slot it % (2 * kItemRing).
  // The fetching warp runs at most kItemRing items ahead of the slowest reader (the index
  // ring), so a slot is written again only after every reader has finished with it.
  WorkItem* items = reinterpret_cast<WorkItem*>(smem + L::kOffItems);
  const uint32_t sQ = smem_u32(smem + L::kOffQ);
  const uint32_t sK = smem_u32(smem + L::kOffK);
  const uint32_t sV = smem_u32(smem + L::kOffV);

  if (threadIdx.x == 0) {
    for (int q = 0; q < 2; ++q) {
      mbar_init(&bars->q_full[q], 1);
      mbar_init(&bars->q_empty[q], 1);
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&bars->s_full[g], 1);
      mbar_init(&bars->p_full[g], kSoftmaxWarps<kDuo> / 2 + (g == 0 ? 1 : 0));  // A's: + watcher
      mbar_init(&bars->o_done[g], 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&bars->pair[i], 2);
    mbar_init(&bars->mma_final, 1);
    for (int s = 0; s < kItemRing; ++s) {
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], 3 + kSoftmaxWarps<kDuo>);  // V producer, MMA, K/V watcher, softmax
    }
    bars->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    tma_prefetch_desc(&qmap);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  {
    // Rows past the G * tpt rows a query tile holds are never written by TMA: zero them
    // once, so that their S is 0 and they go through the softmax like any unmasked row.
    const int rows = p.G * p.tpt;
    const int words = (kRows - rows) * 128 / 16;  // 16-byte words per sub-tile
    for (int i = threadIdx.x; i < 2 * kHalves * words; i += kThreads<kDuo>) {
      const int sub = i / words, wd = i - sub * words;
      reinterpret_cast<uint4*>(smem + L::kOffQ + sub * kSub + rows * 128)[wd] = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();  // visible to the tensor core's reads
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort;

  int n_items = 0;
  if constexpr (!kDirect) {
    // the plan and the kernels before this one are complete; after the split kernel,
    // which let this kernel launch only once the plan was complete, the plan is read
    // without a wait and the wait for the split kernel comes at the end
    if (!p.after_split) pdl_wait();
    n_items = *reinterpret_cast<volatile const int*>(p.hdr + 4);
    if (n_items == 0) {  // nothing planned for this kernel (uniform across the grid)
      if (warp == 1) tmem_dealloc(tmem, kTmemCols);
      if (p.after_split && blockIdx.x == 0 && threadIdx.x == 0) pdl_wait();
      return;
    }
  } else {
    pdl_wait();  // the inputs may still be being written by the kernel before
  }

  // The key tile walked j-th of nt: with a bias the nearest first, so that the running
  // reference is set by the scores the bias lowers least and later tiles seldom move it.
  auto tile_at = [](int j, int nt) { return kBias ? nt - 1 - j : j; };
  // Bounded wait with a warp-uniform outcome: if any lane gives up (or another role has
  // given up), the whole warp leaves its loop together.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    bool ok = !*abort_flag && mbar_wait(bar, parity);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) {
      record_error(p.err, kDevWaitTimeout);
      *abort_flag = 1;
    }
    return ok;
  };
  // next work item from the ring (consumer side); -1 at the end or on a time-out
  auto next_item = [&](int it) -> int {
    const int slot = it % kItemRing;
    if (!wait(&bars->item_full[slot], (it / kItemRing) & 1)) return -1;
    const int idx = bars->item_idx[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
    return idx;
  };

  if (warp == 0 || warp == 2) {
    // ===================== producers: warp 0 (items, Q, K), warp 2 (V) ================
    const bool is_k = warp == 0;
    const int n_stages = is_k ? kKStages : kVStages;
    uint32_t g = 0, qa = 0, qb = 0;
    // Direct mode: lane b holds sequence b's query tokens n, context L, first token t0 and
    // items, each a pair of query tiles or one tile (p.tile_step; 0 for a sequence without
    // rows or an invalid one). Items go rank by rank (rank r: every sequence's r-th longest,
    // in batch order, each KV head), so csum(r) = H_kv * sum_b min(items_b, r) come before
    // rank r.
    int d_n = 0, d_L = 0, d_t0 = 0, d_pre = 0, d_pairs = 0, d_max = 0, d_total = 0;
    auto csum = [&](int r) -> int {
      int v = min(d_pairs, r);
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v * p.H_kv;
    };
    if constexpr (kDirect) {
      if (is_k && lane < p.B) {
        const int q0 = __ldg(p.qsl + lane), q1 = __ldg(p.qsl + lane + 1);
        const int L = __ldg(p.seq_lens + lane), n = q1 - q0;
        if (!p.sequence_ok(q0, q1, L)) {
          if (blockIdx.x == 0) record_error(p.err, kDevBadSequence);
        } else if (n > 0) {
          d_n = n;
          d_L = L;
          d_t0 = q0;
          if constexpr (!Params::kSinks) d_pre = p.prefix_len(lane, L);
          d_pairs = ((n + p.tpt - 1) / p.tpt + p.tile_step - 1) / p.tile_step;
        }
      }
      d_max = d_pairs;
#pragma unroll
      for (int o = 16; o; o >>= 1) d_max = max(d_max, __shfl_xor_sync(0xffffffffu, d_max, o));
      d_total = csum(d_max);
    }
    // field `lane` of direct item idx (< d_total)
    auto direct_field = [&](int idx) -> int {
      int lo = 0, hi = d_max - 1;  // rank: the last r with csum(r) <= idx
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (csum(mid) <= idx) lo = mid;
        else hi = mid - 1;
      }
      const int r = lo, k = idx - csum(r);
      const int nth = k / p.H_kv, kv = k - nth * p.H_kv;
      // the nth (from 0) sequence in batch order that has a pair of rank r
      const unsigned has = __ballot_sync(0xffffffffu, d_pairs > r);
      const bool hit = ((has >> lane) & 1u) && __popc(has & ((1u << lane) - 1u)) == nth;
      const int b = __ffs(__ballot_sync(0xffffffffu, hit)) - 1;
      const int n = __shfl_sync(0xffffffffu, d_n, b), L = __shfl_sync(0xffffffffu, d_L, b);
      const int t0 = __shfl_sync(0xffffffffu, d_t0, b);
      const int j = __shfl_sync(0xffffffffu, d_pairs, b) - 1 - r;  // rank 0: the last pair
      const int qa_ = p.tile_step * j * p.tpt, qb_ = qa_ + p.tpt;
      const int na = min(p.tpt, n - qa_);
      const int nb = p.tile_step == 2 && qb_ < n ? min(p.tpt, n - qb_) : 0;
      const int i_last = nb > 0 ? qb_ + nb - 1 : qa_ + na - 1;
      const int pre = __shfl_sync(0xffffffffu, d_pre, b);
      const int key_end = max(L - n + i_last + 1, pre);  // one past the last key (at most L)
      const int pe = (key_end + kBlockSize - 1) / kBlockSize;
      int key_lo;
      if constexpr (Params::kSinks) key_lo = p.window_lo(L - n + qa_);
      else key_lo = p.row_lo(t0 + qa_, L - n + qa_);
      int f = 0;  // seq, kv, row0, nrows, page_begin, page_end, split 0, nsplit 1, L, n, t0
      f = lane == 0 ? b : f;
      f = lane == 1 ? kv : f;
      f = lane == 2 ? qa_ * p.G : f;
      f = lane == 3 ? na * p.G : f;
      // (one page at least, the sinks' included)
      f = lane == 4 ? min(key_lo / kBlockSize, Params::kSinks ? pe : pe - 1) : f;
      f = lane == 5 ? pe : f;
      f = lane == 7 ? 1 : f;
      f = lane == 8 ? L : f;
      f = lane == 9 ? n : f;
      f = lane == 10 ? t0 : f;
      f = lane == 11 ? nb * p.G : f;  // rows of query tile B
      f = lane == 12 ? key_lo : f;    // pad[1..3], as the plan has them
      f = lane == 13 ? key_end : f;
      f = lane == 14 && !Params::kSinks ? pre : f;
      if constexpr (Params::kSinks)  // (lane 14: the sinks' first page, 0)
        f = lane == 15 ? (min(p.sinks, key_end) + kBlockSize - 1) / kBlockSize : f;
      return f;
    };
    for (int it = 0;; ++it) {
      int idx = 0;
      if (is_k && kDirect) {
        const int slot = it % kItemRing;
        if (!wait(&bars->item_empty[slot], ((it / kItemRing) & 1) ^ 1)) break;
        // (every other round in reverse, so that no CTA has the longest item of each)
        idx = it * static_cast<int>(gridDim.x) +
              static_cast<int>(it & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        if (idx >= d_total) idx = -1;
        if (idx >= 0) {
          const int f = direct_field(idx);
          if (lane < 16) reinterpret_cast<int*>(items + it % (2 * kItemRing))[lane] = f;
        }
        __syncwarp();
        if (lane == 0) {
          bars->item_idx[slot] = idx;
          mbar_arrive(&bars->item_full[slot]);
        }
      } else if (is_k) {
        const int slot = it % kItemRing;
        if (!wait(&bars->item_empty[slot], ((it / kItemRing) & 1) ^ 1)) break;
        if (lane < 4) {
          // lanes 0..3 copy the item's record into its shared-memory slot, lane 0 hands
          // out the index (its arrival orders the copy before every reader's wait)
          if (lane == 0) idx = atomicAdd(p.hdr + 5, 1);
          idx = __shfl_sync(0x0000000fu, idx, 0);
          if (idx >= n_items) idx = -1;
          if (idx >= 0)
            reinterpret_cast<uint4*>(items + it % (2 * kItemRing))[lane] =
                __ldg(reinterpret_cast<const uint4*>(p.tile_items + idx) + lane);
          __syncwarp(0x0000000fu);
          if (lane == 0) {
            bars->item_idx[slot] = idx;
            mbar_arrive(&bars->item_full[slot]);
          }
        }
        __syncwarp();
        idx = __shfl_sync(0xffffffffu, idx, 0);
      } else {
        idx = next_item(it);
      }
      if (idx < 0) break;
      const WorkItem& w = items[it % (2 * kItemRing)];
      const ItemTiles<Params> tiles(w);
      const int nt = tiles.nt;
      if (nt == 0 || !tile_item_ok(w, p)) continue;
      const int seq = w.seq, kv = w.kv, pages = tiles.sp + tiles.pe - tiles.pb;
      // query tiles (K warp): whole tokens x the G heads of this KV head. Each tile has its
      // own buffer, refilled as soon as that tile's last S of the previous item has read
      // it. They are loaded after the item's first K tile, whose stage frees earlier.
      auto load_q = [&]() -> bool {
        const bool has_b = w.pad[0] > 0;
        const int tok = w.tok0 + w.row0 / p.G;
        const uint32_t tile_bytes = kHalves * 64 * 2 * p.G * p.tpt;
        for (int q = 0; q < (has_b ? 2 : 1); ++q) {
          if (!wait(&bars->q_empty[q], ((q ? qb : qa) & 1) ^ 1)) return false;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars->q_full[q], tile_bytes);
            for (int h = 0; h < kHalves; ++h)
              tma_load_3d(smem + L::kOffQ + q * L::kQ + h * kSub, &qmap, &bars->q_full[q],
                          h * 64, kv * p.G, tok + q * p.tpt);
          }
        }
        ++qa;
        if (has_b) ++qb;
        return true;
      };
      // K (or V) tiles of 8 pages; pages past the split read the zero fill. One lane per
      // page copy: lane = page * kHalves + half (64-element half of the head).
      const int32_t* bt = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks;
      int bt_base = 1 << 28, bt_reg = -1;
      bool ok = true;
      const int pp = lane / kHalves, h = lane % kHalves;
      for (int j = 0; j < nt; ++j) {
        const int first = tile_at(j, nt) * kPagesPerTile;  // of the item's pages
        if (first < bt_base || first - bt_base + kPagesPerTile > 32) {
          bt_base = kBias ? max(first + kPagesPerTile - 32, 0) : first;
          bt_reg = bt_base + lane < pages ? __ldg(bt + tiles.page(bt_base + lane)) : -1;
        }
        const uint32_t st = g % n_stages;
        uint64_t* empty = is_k ? &bars->k_empty[st] : &bars->v_empty[st];
        uint64_t* full = is_k ? &bars->k_full[st] : &bars->v_full[st];
        if (!wait(empty, ((g / n_stages) & 1) ^ 1)) { ok = false; break; }
        const int blk = __shfl_sync(0xffffffffu, bt_reg, (first - bt_base + pp) & 31);
        uint8_t* dst = smem + (is_k ? L::kOffK : L::kOffV) + st * L::kK;
        if (lane == 0) mbar_arrive_expect_tx(full, L::kK);
        __syncwarp();
        if (lane < kPagesPerTile * kHalves) {
          int row;
          if (first + pp >= pages) {
            row = p.num_blocks * kBlockSize;  // past the pool: zero fill, no HBM read
          } else if (blk < 0 || blk >= p.num_blocks) {
            record_error(p.err, kDevBadBlockId);
            row = p.num_blocks * kBlockSize;
          } else {
            row = blk * kBlockSize;
          }
          tma_load_2d(dst + h * kSub + pp * (kBlockSize * 128), is_k ? &kmap : &vmap, full,
                      kv * D + h * 64, row);
        }
        ++g;
        if (is_k && j == 0 && !load_q()) { ok = false; break; }
      }
      if (!ok) break;
    }
  } else if (warp == 1) {
    // ============================ MMA issuer (one thread) ===========================
    // Issuing one tcgen05.mma occupies the thread for nearly as long as the tensor core
    // takes to run it (M128 N128 K16), so this loop is kept lean: lane 0 alone, with
    // descriptors formed as a base plus constant offsets and waits without warp votes.
    if (lane == 0) {
      constexpr uint32_t idS = idesc_f16(kBF16, kRows, kKeys, false);
      constexpr uint32_t idPV = idesc_f16(kBF16, kRows, D, true);
      // bounded single-thread wait; the abort flag is read only on the slow path
      auto wait1 = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        for (uint32_t i = 0; i < (1u << 24); ++i) {
          if (*abort_flag) return false;
          if (mbar_try_wait(bar, parity)) return true;
        }
        record_error(p.err, kDevWaitTimeout);
        *abort_flag = 1;
        return false;
      };
      // descriptor start addresses stay below 2^18 bytes, so offsets added to the 14-bit
      // start field (address / 16) never carry into the next field
      const uint64_t qdesc0 = sdesc_sw128(sQ, 16, 1024);
      const uint64_t qdesc1 = sdesc_sw128(sQ + L::kQ, 16, 1024);
      const uint64_t kdesc0 = sdesc_sw128(sK, 16, 1024);
      const uint64_t vdesc0 = sdesc_sw128(sV, kSub, 1024);
      uint32_t g = 0, qa = 0, qb = 0, pc[2] = {0, 0};
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int slot = it % kItemRing;
        if (!wait1(&bars->item_full[slot], (it / kItemRing) & 1)) break;
        const int idx = bars->item_idx[slot];
        mbar_arrive(&bars->item_empty[slot]);
        if (idx < 0) break;
        const WorkItem& w = items[it % (2 * kItemRing)];
        const int nt = ItemTiles<Params>(w).nt;
        if (!tile_item_ok(w, p)) {
          record_error(p.err, kDevPlanOverflow);  // a plan this launch cannot use
          continue;
        }
        if (nt == 0) continue;
        const bool has_b = w.pad[0] > 0;
        const int ng = has_b ? 2 : 1;
        if (!wait1(&bars->q_full[0], qa & 1)) break;
        const uint32_t g0 = g;
        // S of query tile `grp` against K tile j. Only the item's first K tile is waited
        // for here; P of query tile A for tile j - 1 implies K tile j (the K/V watcher).
        auto issue_s = [&](int grp, int j) -> bool {
          const uint32_t st = (g0 + j) % kKStages;
          if (j == 0 && grp == 0) {
            if (!wait1(&bars->k_full[st], ((g0 + j) / kKStages) & 1)) return false;
            tc_fence_after();
          }
          const uint64_t a0 = grp ? qdesc1 : qdesc0;
          const uint64_t b0 = kdesc0 + ((st * L::kK) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * kSub + (kk % 4) * 32) >> 4;
            umma_f16(tmem + col_s(grp), a0 + off, b0 + off, idS, kk > 0 ? 1u : 0u);
          }
          umma_commit(&bars->s_full[grp]);
          if (j == nt - 1) umma_commit(&bars->q_empty[grp]);  // last read of this Q tile
          if (grp == ng - 1) umma_commit(&bars->k_empty[st]);  // last reader of the K stage
          return true;
        };
        // O of query tile `grp` += P V of K/V tile j. P is the only wait: the softmax
        // warps arrive on it after their epilogue of the previous item has read O, and
        // the K/V watcher adds its arrival to query tile A's once V tile j (and K tile
        // j + 1) have landed.
        auto issue_pv = [&](int grp, int j) -> bool {
          if (!wait1(&bars->p_full[grp], pc[grp] & 1)) return false;
          ++pc[grp];
          const uint32_t st = (g0 + j) % kVStages;
          tc_fence_after();
          const uint64_t b0 = vdesc0 + ((st * L::kK) >> 4);
          const uint32_t acc0 = j > 0 ? 1u : 0u;
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            umma_f16_ts(tmem + col_o(grp),
                        tmem + col_s(grp) + (kDuo ? (kk / 4) * 64 + (kk % 4) * 8 : kk * 8),
                        b0 + ((kk * 2048) >> 4), idPV, kk > 0 ? 1u : acc0);
          if (grp == ng - 1) umma_commit(&bars->v_empty[st]);  // last reader of the V stage
          return true;
        };
        for (int q = 0; q < ng && ok; ++q) {
          if (q == 1 && !wait1(&bars->q_full[1], qb & 1)) {
            ok = false;
            break;
          }
          ok = issue_s(q, 0);
        }
        // per K/V tile: PV of A, next S of A, PV of B, next S of B. A query tile's next S
        // overwrites its P in TMEM, so it is issued after that tile's PV (in order).
        // A query tile's O is final after its last PV: its epilogue may start while the
        // other tile's last PV still waits for P.
        for (int j = 0; j < nt && ok; ++j)
          for (int q = 0; q < ng && ok; ++q) {
            ok = issue_pv(q, j);
            if (ok && j + 1 < nt) ok = issue_s(q, j + 1);
            if (ok && j + 1 == nt) umma_commit(&bars->o_done[q]);
          }
        if (!ok) break;
        g += nt;
        ++qa;
        if (ng > 1) ++qb;
      }
      // every MMA issued by this thread has completed before TMEM is released
      umma_commit(&bars->mma_final);
      mbar_wait(&bars->mma_final, 0, 1u << 22);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ============================ K/V watcher ==================================
    // P of query tile A also stands for V tile j and K tile j + 1 having landed: this
    // warp waits for them and adds its arrival to that P barrier, then waits for the
    // barrier's phase to complete so that it never runs a tile ahead. The MMA thread
    // then waits on P alone, and the softmax warps carry no extra waits.
    uint32_t gt = 0, pc = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int idx = next_item(it);
      if (idx < 0) break;
      const WorkItem& w = items[it % (2 * kItemRing)];
      const ItemTiles<Params> tiles(w);
      const int nt = tiles.nt;
      if (nt == 0 || !tile_item_ok(w, p)) continue;
      // Where some row of the item sees nothing, a key from the item's first token on (`own`,
      // behind the prefix) may be seen by none.
      const int pos0 = w.ctx_len - w.n_query, i0 = w.row0 / p.G;
      const int i1 = i0 + (w.pad[0] > 0 ? p.tpt + w.pad[0] / p.G : w.nrows / p.G);
      int own = 0x7fffffff;
      if (!Params::kSinks && p.starts != nullptr) {
        bool empty = false;
#pragma unroll 1
        for (int i = i0 + lane; i < i1; i += 32) empty |= __ldg(p.starts + w.tok0 + i) > pos0 + i;
        if (__any_sync(0xffffffffu, empty)) own = max(pos0 + i0, w.pad[3]);
      }
      for (int j = 0; j < nt && ok; ++j) {
        const uint32_t gv = gt + j, gk = gv + 1;
        ok = wait(&bars->v_full[gv % kVStages], (gv / kVStages) & 1) &&
             (j + 1 >= nt || wait(&bars->k_full[gk % kKStages], (gk / kKStages) & 1));
        if (!ok) break;
        // keys of this tile's pages that no row of the item sees (bits of `dead`): their V
        // rows are zeroed, four at a time (this code runs once or twice an item, so its size
        // counts: with loops unrolled, 6 chunks of documents took 31.1 us in place of 30.5, and
        // the 777 us with a bias above 788)
        const int at = tile_at(j, nt), kb = tiles.key0(at);
        const int ke = min(kb + kKeys, tiles.pe * kBlockSize);
        const int sink_cols = tiles.sink_cols(at);
        // (a tile's sinks, but for those of pages that hold sinks alone, end inside it)
        bool part = kb < w.pad[1] || ke > w.pad[2] || ke > own;
        if constexpr (Params::kSinks)
          part = sink_cols > 0
                     ? kb + max(sink_cols, 0) < w.pad[1] || ke > w.pad[2] ||
                           tiles.sink_key0(at) + min(sink_cols, kKeys) > min(p.sinks, w.pad[2])
                     : part;
        if (part) {
          uint8_t* v = smem + L::kOffV + (gv % kVStages) * L::kK + (lane & 7) * 16;
#pragma unroll 1
          for (int k = 0; k < kKeys; k += 32) {
            const int key = kb + k + lane;
            bool unseen = key < ke && (key < w.pad[1] || key >= w.pad[2] ||
                                       (!Params::kSinks &&
                                        p.key_unseen(key, own, w.pad[2], w.tok0 - pos0)));
            if constexpr (Params::kSinks)
              if (k + lane < sink_cols)
                unseen = tiles.sink_key0(at) + k + lane >= min(p.sinks, w.pad[2]);
            uint32_t dead = __ballot_sync(0xffffffffu, unseen);
            while (dead != 0) {
              const int four = (__ffs(dead) - 1) & ~3, r = four + (lane >> 3);
              if (dead >> r & 1u) {
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                  *reinterpret_cast<uint4*>(v + h * kSub + (k + r) * 128) = make_uint4(0, 0, 0, 0);
              }
              dead &= ~(15u << four);
            }
          }
          fence_proxy_async_smem();  // before the tensor core reads them
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&bars->p_full[0]);
        ok = wait(&bars->p_full[0], pc & 1);
        ++pc;
      }
      gt += nt;
    }
  } else if (warp >= 4) {
    // ============================ softmax groups + epilogue =========================
    if constexpr (!kDuo) {
      // ---- masks alone: one warp for 32 rows, a half of a tile's columns after the other
      const int grp = (warp - 4) >> 2;   // 0: query tile A, 1: query tile B
      const int quarter = warp & 3;      // TMEM lanes 32*quarter .. +31
      const int r = quarter * 32 + lane;
      const uint32_t trow = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      const uint32_t tS = trow + col_s(grp), tO = trow + col_o(grp);
      uint32_t sc = 0, act = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int idx = next_item(it);
        if (idx < 0) break;
        const WorkItem& w = items[it % (2 * kItemRing)];
        const ItemTiles<Params> tiles(w);
        const int pe = tiles.pe, nt = tiles.nt;
        if (nt == 0 || !tile_item_ok(w, p)) continue;
        const int nrows = grp == 0 ? w.nrows : w.pad[0];
        if (nrows == 0) continue;  // no query tile B in this item
        // this thread's query row
        const bool valid = r < nrows;
        const int R = w.row0 + grp * p.tpt * p.G + r;  // packed row within the sequence
        const int qtok = R / p.G;                        // query index within the sequence
        const int tok = w.tok0 + qtok;
        const int head = w.kv * p.G + R - qtok * p.G;
        const int pos = valid ? w.ctx_len - w.n_query + qtok : -1;
        // the row's keys: [key_lo, key_hi] within the item
        // (streams: [key_lo, key_hi] of the window's run)
        const int key_hi =
            min(Params::kSinks ? pos : max(pos, w.pad[3] - 1), pe * kBlockSize - 1);
        int key_lo = 0;
        if constexpr (Params::kSinks) key_lo = valid ? p.window_lo(pos) : 0;
        else key_lo = valid ? p.row_lo(tok, pos) : 0;
        // as columns of the item's tiles
        const int lim0 = key_hi - tiles.key0(0), low0 = key_lo - tiles.key0(0);
        const int sunk0 = Params::kSinks && valid ? tiles.sunk(p, pos) : 0;
        // the row's split count and partial base, fetched now so that the epilogue's
        // stores do not wait on them
        // (both loads are issued at once; nothing waits for them before the epilogue)
        const int ns_t = !valid ? 0 : kDirect ? 1 : __ldg(p.tok_ns + tok);
        const int tok_part = kDirect || !valid ? 0 : __ldg(p.tok_base + tok);
        // m_ref: the reference max (log2 units) that P, O and l are currently taken against;
        // m_next: a max more than 2^8 above it seen in the last tile, applied before the next
        float m_ref = -INFINITY, m_next = -INFINITY, l = 0.f;
        for (int j = 0; j < nt; ++j) {
          // visible columns: c <= lim (a row past the tile's rows is computed unmasked and
          // not written)
          // (streams: and those below `sunk`, of the sinks)
          const int lim = valid ? lim0 - j * kKeys : kKeys, low = valid ? low0 - j * kKeys : 0;
          [[maybe_unused]] const int sunk = sunk0 - j * kKeys;
          if (!wait(&bars->s_full[grp], sc & 1)) { ok = false; break; }
          ++sc;
          tc_fence_after();
          // This group's previous PV has completed (this S was issued after it): O is stable.
          auto rescale_o = [&](float alpha) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32];
              tmem_ld32(tO + c * 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
              tmem_st32(tO + c * 32, v);
            }
            tmem_st_wait();
          };
          if (__any_sync(0xffffffffu, m_next > m_ref)) {
            const bool need = m_next > m_ref;
            const float alpha = need ? fast_exp2(m_ref - m_next) : 1.f;
            if (j > 0) rescale_o(alpha);
            l *= alpha;
            if (need) m_ref = m_next;
          }
          // P = 2^(s*scale*log2e - m_ref) as 16-bit pairs written over S; half h of P lands
          // on columns 32h..32h+31, which the loads of halves <= h have already read
          const bool full =
              __all_sync(0xffffffffu, lim >= kKeys - 1 && low <= (Params::kSinks ? max(sunk, 0) : 0));
          // l holds the earlier tiles' sum; this tile's halves are summed apart, so that a
          // reference moved in half 1 can re-sum the half-0 P it re-rounds
          float l_half0 = 0.f, l_h = 0.f;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t v[64];
            tmem_ld32(tS + 64 * h, v);
            tmem_ld32(tS + 64 * h + 32, v + 32);
            tmem_ld_wait();
            if (!full) {
              drop_unseen<Params>(v, lim - 64 * h, low - 64 * h, sunk - 64 * h);
              drop_unseen<Params>(v + 32, lim - 64 * h - 32, low - 64 * h - 32,
                                  sunk - 64 * h - 32);
            }
            // P is taken against the row's reference without the half's max; the max (and a move
            // of the reference) is taken only when there is no reference yet, or when the half's
            // sum shows that P outgrew its bound, and P is then taken again
            bool with_max = __any_sync(0xffffffffu, m_ref == -INFINITY);
            uint32_t pk[32];
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
              if (with_max) {
                // four independent max chains
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 64; e += 8)
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    mq[k] = fmax3(mq[k], __uint_as_float(v[e + 2 * k]), __uint_as_float(v[e + 2 * k + 1]));
                const float mx = fmax3(fmaxf(mq[0], mq[1]), mq[2], mq[3]);
                const float m_half = mx == -INFINITY ? mx : mx * p.scale_log2;
                // no reference yet, or a jump P could overflow on: move the reference now,
                // rescaling what is already taken against the old one
                const bool move = m_half > m_ref + kMoveLog2<kBF16> ||
                                  (m_ref == -INFINITY && m_half != -INFINITY);
                if (__any_sync(0xffffffffu, move)) {
                  const float alpha = move && m_ref != -INFINITY ? fast_exp2(m_ref - m_half) : 1.f;
                  if (j > 0) rescale_o(alpha);
                  l *= alpha;
                  if (h == 1) {
                    // the half of P already written (columns 0..31) is scaled and rounded
                    // again; its sum is taken anew from the values the PV product will read
                    uint32_t q[32];
                    tmem_st_wait();
                    tmem_ld32(tS, q);
                    tmem_ld_wait();
                    float2 lq0[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                      q[e] = scale_pair<kBF16>(q[e], alpha);
                      add_pair_exact<kBF16>(lq0[e & 1], q[e]);
                    }
                    l_half0 = (lq0[0].x + lq0[0].y) + (lq0[1].x + lq0[1].y);
                    tmem_st32(tS, q);
                    tmem_st_wait();
                  }
                  if (move) m_ref = m_half;
                }
              }
              const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
              float2 lq[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // four sums
              // scale and subtract two scores per packed fma; the row sum adds the 16-bit P
              // values the MMA sees, widened exactly
              const float2 sl2x2 = make_float2(p.scale_log2, p.scale_log2);
              const float2 nm2 = make_float2(neg_m, neg_m);
#pragma unroll
              for (int e = 0; e < 64; e += 2) {
                const float2 x = ffma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                                       sl2x2, nm2);
                pk[e / 2] = pack2<kBF16>(fast_exp2(x.x), fast_exp2(x.y));
                add_pair_exact<kBF16>(lq[(e / 2) & 1], pk[e / 2]);
              }
              // P goes out before its sum is checked; a second pass writes it again
              if (pass > 0) tmem_st_wait();
              tmem_st16(tS + 32 * h, pk);
              tmem_st16(tS + 32 * h + 16, pk + 16);
              l_h = (lq[0].x + lq[0].y) + (lq[1].x + lq[1].y);
              if (with_max || __all_sync(0xffffffffu, l_h <= kHalfSumMax<kBF16>)) break;
              with_max = true;
            }
            if (h == 0) l_half0 = l_h;
            else l += l_half0 + l_h;
          }
          // O is rescaled lazily: when this tile's P summed to more than 2^8, the reference
          // moves up by log2 of that sum before the next tile (the new reference is at least
          // the row's max, so P stays at most 1 there)
          const float l_tile = l_half0 + l_h;
          m_next = l_tile > (1 << kRescaleExp) ? m_ref + __log2f(l_tile) : m_ref;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[grp]);
        }
        if (!ok) break;
        // epilogue: O / l of this group's rows to the output, or to the split partials
        if (!wait(&bars->o_done[grp], act & 1)) break;
        tc_fence_after();
        const bool write = valid && w.split < ns_t;
        const bool any = !(l == 0.f);  // a row without keys gives zeros, whatever O holds
        const float inv = any ? 1.f / l : 0.f;
        if (__all_sync(0xffffffffu, !write || ns_t == 1)) {
          // Direct output: each lane writes its own row, 64 columns (128 bytes) per TMEM
          // wait, as 32-byte stores when the output is 32-byte aligned (16-byte stores
          // otherwise), so every store instruction fills whole 32-byte sectors of 32 rows.
          uint16_t* dst = static_cast<uint16_t*>(p.out) + (static_cast<int64_t>(tok) * p.H_q + head) * D;
          const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
          const float2 inv2 = make_float2(inv, inv);
#pragma unroll 1
          for (int c4 = 0; c4 < D / 64; ++c4) {
            uint32_t v[64];
            tmem_ld32(tO + c4 * 64, v);
            tmem_ld32(tO + c4 * 64 + 32, v + 32);
            tmem_ld_wait();
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 x =
                  fmul2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), inv2);
              w[e] = any ? pack2<kBF16>(x.x, x.y) : 0u;
            }
            if (write) {
              if (wide) {
#pragma unroll
                for (int q = 0; q < 4; ++q) st_global_v8(dst + c4 * 64 + 16 * q, w + 8 * q);
              } else {
                uint4* d4 = reinterpret_cast<uint4*>(dst + c4 * 64);
#pragma unroll
                for (int q = 0; q < 8; ++q) d4[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
              }
            }
          }
        } else {
          // split partials (fp32), one row per lane
#pragma unroll 1
          for (int c2 = 0; c2 < D / 64; ++c2) {
            uint32_t v[64];
            tmem_ld32(tO + c2 * 64, v);
            tmem_ld32(tO + c2 * 64 + 32, v + 32);
            tmem_ld_wait();
            if (!write) continue;
            if (!any) {
#pragma unroll
              for (int e = 0; e < 64; ++e) v[e] = 0u;
            }
            if (ns_t == 1) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                                    (static_cast<int64_t>(tok) * p.H_q + head) * D +
                                                    c2 * 64);
#pragma unroll
              for (int q = 0; q < 8; ++q)
                dst[q] = make_uint4(
                    pack2<kBF16>(__uint_as_float(v[8 * q + 0]) * inv, __uint_as_float(v[8 * q + 1]) * inv),
                    pack2<kBF16>(__uint_as_float(v[8 * q + 2]) * inv, __uint_as_float(v[8 * q + 3]) * inv),
                    pack2<kBF16>(__uint_as_float(v[8 * q + 4]) * inv, __uint_as_float(v[8 * q + 5]) * inv),
                    pack2<kBF16>(__uint_as_float(v[8 * q + 6]) * inv, __uint_as_float(v[8 * q + 7]) * inv));
            } else {
              const int64_t pidx = static_cast<int64_t>(tok_part) + w.split * p.H_q + head;
              float4* dst = reinterpret_cast<float4*>(p.part_o + pidx * D + c2 * 64);
#pragma unroll
              for (int q = 0; q < 16; ++q)
                dst[q] = make_float4(__uint_as_float(v[4 * q]) * inv, __uint_as_float(v[4 * q + 1]) * inv,
                                     __uint_as_float(v[4 * q + 2]) * inv, __uint_as_float(v[4 * q + 3]) * inv);
              if (c2 == 0) p.part_lse[pidx] = any ? m_ref + __log2f(l) : -INFINITY;
            }
          }
        }
        ++act;
      }
    } else {
      // ---- a cap or a bias: two warps for 32 rows, a half of the columns each
      const int grp = (warp - 4) >> 3;        // 0: query tile A, 1: query tile B
      const int half = ((warp - 4) >> 2) & 1; // columns 64 * half .. + 63 of each key tile
      const int quarter = warp & 3;           // TMEM lanes 32*quarter .. +31
      const int r = quarter * 32 + lane;
      const uint32_t trow = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      const uint32_t tS = trow + col_s(grp) + 64 * half;            // P over its first 32 columns
      const uint32_t tO = trow + col_o(grp) + (D / 2) * half;       // the half of O it keeps
      // What the two warps of the same rows tell one another goes through 128 bytes of shared
      // memory and a barrier of the two (bounded, like every wait). A slot may be written once
      // the other warp has read what it held: before a tile's first exchange both warps' P of
      // the tile before has arrived, and with it their reads; otherwise a meeting lies between.
      uint64_t* pair_bar = &bars->pair[grp * 4 + quarter];
      uint8_t* slots = smem + L::kOffPair + (grp * 4 + quarter) * 128;
      const int own_slot = half * 32 + lane, other_slot = own_slot ^ 32;
      uint32_t px = 0;  // barrier phases so far
      auto meet = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(pair_bar);
        return wait(pair_bar, px++ & 1);
      };
      auto exchange8 = [&](uint32_t mine, uint32_t* theirs) -> bool {
        slots[own_slot] = static_cast<uint8_t>(mine);
        if (!meet()) return false;
        *theirs = slots[other_slot];
        return true;
      };
      auto exchange16 = [&](uint32_t mine, uint32_t* theirs) -> bool {
        slots[own_slot] = static_cast<uint8_t>(mine);
        slots[64 + own_slot] = static_cast<uint8_t>(mine >> 8);
        if (!meet()) return false;
        *theirs = slots[other_slot] | static_cast<uint32_t>(slots[64 + other_slot]) << 8;
        return meet();
      };
      // a float, in two halves
      auto exchange_float = [&](float mine, float* theirs) -> bool {
        uint32_t hi, lo;
        if (!exchange16(__float_as_uint(mine) >> 16, &hi) ||
            !exchange16(__float_as_uint(mine) & 0xffffu, &lo))
          return false;
        *theirs = __uint_as_float(hi << 16 | lo);
        return true;
      };
      // The larger of the row's two maxima, rounded up to a whole number of log2 units (as a
      // reference it need not be exact): 16 bits, or a float's exchange if some row's is out of
      // their range.
      auto row_max = [&](float* mx) -> bool {
        constexpr int kNone = -32768, kFar = 32767;
        const float up = ceilf(*mx);
        const int q = *mx == -INFINITY ? kNone : fabsf(up) < 32767.f ? static_cast<int>(up) : kFar;
        uint32_t got;
        if (!exchange16(static_cast<uint32_t>(q), &got)) return false;
        const int o = static_cast<int16_t>(got);
        if (__any_sync(0xffffffffu, q == kFar || o == kFar)) {
          float other;
          if (!exchange_float(*mx, &other)) return false;
          *mx = fmaxf(*mx, other);
          return true;
        }
        const int m = max(q, o);
        *mx = m == kNone ? -INFINITY : static_cast<float>(m);
        return true;
      };
      // Capped scores lie within c = cap_log2 of 0. Against a fixed reference of 86 - c (c at
      // most) every P is between 2^-86, so that products with |V| down to 2^-40 are normal in
      // fp32, and 2^(2 c - 86), 2^60 at kFixedCapLog2 (1 for caps up to 29), so that sums with
      // |V| up to 2^40 hold 2^28 keys. Then no maximum is taken, nothing moves, and the two warps
      // of a row have nothing to tell one another before the end.
      const bool fixed = kCap == 1 && !kBias && kBF16 && p.cap_log2 <= kFixedCapLog2;
      const float m_fixed = fixed ? fminf(p.cap_log2, -kFixedLeastLog2 - p.cap_log2) : -INFINITY;
      uint32_t sc = 0, act = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int idx = next_item(it);
        if (idx < 0) break;
        const WorkItem& w = items[it % (2 * kItemRing)];
        const ItemTiles<Params> tiles(w);
        const int pe = tiles.pe, nt = tiles.nt;
        if (nt == 0 || !tile_item_ok(w, p)) continue;
        const int nrows = grp == 0 ? w.nrows : w.pad[0];
        if (nrows == 0) continue;  // no query tile B in this item
        // this thread's query row
        const bool valid = r < nrows;
        const int R = w.row0 + grp * p.tpt * p.G + r;  // packed row within the sequence
        const int qtok = R / p.G;                        // query index within the sequence
        const int tok = w.tok0 + qtok;
        const int head = w.kv * p.G + R - qtok * p.G;
        const int pos = valid ? w.ctx_len - w.n_query + qtok : -1;
        // the row's keys within the item, [key_lo, key_hi], relative to the warp's columns (a
        // row past the tile's rows is computed unmasked and not written)
        const int col0 = tiles.key0(0) + 64 * half;
        const int key_hi =
            valid ? min(Params::kSinks ? pos : max(pos, w.pad[3] - 1), pe * kBlockSize - 1) - col0
                  : (1 << 30);
        int key_lo = -(1 << 30);
        if (valid) {
          if constexpr (Params::kSinks) key_lo = p.window_lo(pos) - col0;
          else key_lo = p.row_lo(tok, pos) - col0;
        }
        const int sunk0 = Params::kSinks && valid ? tiles.sunk(p, pos) - 64 * half : 0;
        const float slope = kBias && valid ? -kLog2e * __ldg(p.slopes + head) : 0.f;
        const float first_dist = static_cast<float>(pos - col0);  // of the item's first column
        // m_ref: the reference max (log2 units) that P, O and l are currently taken against;
        // m_next: the reference from the next tile on, when this one's P summed to over 2^8
        float m_ref = m_fixed, m_next = m_fixed, l = 0.f;
        for (int j = 0; j < nt; ++j) {
          const int t0 = tile_at(j, nt) * kKeys;  // the tile's first key, from the item's
          // visible: low <= c <= lim (streams: and those below `sunk`, of the sinks)
          const int lim = key_hi - t0, low = key_lo - t0;
          [[maybe_unused]] const int sunk = sunk0 - t0;
          if (!wait(&bars->s_full[grp], sc & 1)) { ok = false; break; }
          ++sc;
          tc_fence_after();
          // This group's previous PV has completed (this S was issued after it): O is stable.
          // Each of the two warps keeps a half of its columns.
          auto rescale_o = [&](float alpha) {
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              uint32_t v[32];
              tmem_ld32(tO + c * 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
              tmem_st32(tO + c * 32, v);
            }
            tmem_st_wait();
          };
          if (!fixed && __any_sync(0xffffffffu, m_next > m_ref)) {
            const float alpha = m_next > m_ref ? fast_exp2(m_ref - m_next) : 1.f;
            if (j > 0) rescale_o(alpha);
            l *= alpha;
            m_ref = fmaxf(m_ref, m_next);
          }
          const bool full =
              __all_sync(0xffffffffu, lim >= 63 && low <= (Params::kSinks ? max(sunk, 0) : 0));
          // every column visible, and (with a bias) none past the row's own position
          const bool one_sign =
              full && (!kBias || __all_sync(0xffffffffu, !valid || first_dist - t0 >= 63.f));
          uint32_t pk[32];
          float l_t = 0.f;
          // 32 columns of scores, raw
          auto load = [&](int h, uint32_t* v) {
            tmem_ld32(tS + 32 * h, v);
            tmem_ld_wait();
          };
          // brought to log2 units in place: any cap, any bias, masked
          auto to_log2 = [&](int h, uint32_t* v) {
            if constexpr (kCap > 0) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float raw = __uint_as_float(v[e]);
                v[e] = __float_as_uint(kCap == 1 ? capped_far(raw, p) : capped(raw, p));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                v[e] = __float_as_uint(__uint_as_float(v[e]) * p.scale_log2);
            }
            if constexpr (kBias) {
              const float d0 = first_dist - static_cast<float>(t0 + 32 * h);  // first column's
#pragma unroll
              for (int e = 0; e < 32; ++e)
                v[e] = __float_as_uint(
                    fmaf(slope, fabsf(d0 - static_cast<float>(e)), __uint_as_float(v[e])));
            }
            if constexpr (Params::kSinks) {
              if (!full) drop_unseen<Params>(v, lim - 32 * h, low - 32 * h, sunk - 32 * h);
            } else if (!full) {  // (by words: capped chunks of 2048 over 8192 593 us, so 585)
              const int hi = lim - 32 * h, lo = low - 32 * h;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e > hi || e < lo) v[e] = __float_as_uint(-INFINITY);
            }
          };
          // P of 32 columns against the reference, 16-bit pairs; the row sum adds the values the
          // MMA sees, widened exactly. Where every column is visible, the cap's argument small
          // and the distances of one sign, packed arithmetic takes the scores straight to the
          // exponent; otherwise to_log2 first.
          auto take = [&](int h) {
            uint32_t v[32];
            load(h, v);
            const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
            const float2 nm2 = make_float2(neg_m, neg_m);
            float2 lq[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // four sums
            auto raw = [&](int e) {
              return make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            };
            auto put = [&](int e, float2 x) {
              pk[16 * h + e / 2] = pack2<kBF16>(fast_exp2(x.x), fast_exp2(x.y));
              add_pair_exact<kBF16>(lq[(e / 2) & 1], pk[16 * h + e / 2]);
            };
            bool fast = one_sign;
            if constexpr (kCap > 0) {
              float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int e = 0; e < 32; e += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  a[k] = fmax3(a[k], fabsf(__uint_as_float(v[e + 2 * k])),
                               fabsf(__uint_as_float(v[e + 2 * k + 1])));
              const float y = fmax3(fmaxf(a[0], a[1]), a[2], a[3]) * p.cap_y;
              fast = fast && __all_sync(0xffffffffu, y <= 0.5f);
            }
            if (fast) {
              const float2 sl2x2 = make_float2(p.scale_log2, p.scale_log2);
              const float2 cap_y2 = make_float2(p.cap_y, p.cap_y);
              const float d0 = first_dist - static_cast<float>(t0 + 32 * h);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float2 c = nm2;
                if constexpr (kBias) {
                  const float x = fmaf(slope, d0 - static_cast<float>(e), neg_m);
                  c = make_float2(x, x - slope);
                }
                put(e, kCap > 0 ? capped_poly2(fmul2(raw(e), cap_y2), p.tanh4, c)
                            : ffma2(raw(e), sl2x2, c));
              }
            } else {
              to_log2(h, v);
#pragma unroll
              for (int e = 0; e < 32; e += 2) put(e, ffma2(raw(e), make_float2(1.f, 1.f), nm2));
            }
            l_t += (lq[0].x + lq[0].y) + (lq[1].x + lq[1].y);
          };
          // P is taken against the row's reference without the tile's max; the max (and a move
          // of the reference) is taken only when there is no reference yet, or when a half's
          // sum shows that P outgrew its bound (S is whole until then), and P is taken again.
          // Both warps see both sums and maxima, so they decide alike.
          uint32_t top = 0;  // exponent of the larger of the row's half sums
          // (a row without a reference asks for one only once it sees a key: lim and low are
          // those of the warp's half of the tile)
          const bool sees = (lim + 64 * half >= 0 && low + 64 * half <= kKeys - 1) ||
                            (Params::kSinks && sunk + 64 * half > 0);
          bool redo = !fixed && __any_sync(0xffffffffu, m_ref == -INFINITY && sees);
          if (fixed) {
            take(0);
            take(1);
          } else if (!redo) {
            take(0);
            take(1);
            const uint32_t mine = __float_as_uint(l_t) >> 23;
            if (!exchange8(mine, &top)) { ok = false; break; }
            top = max(top, mine);
            redo = __any_sync(0xffffffffu, top >= kSumExp<kBF16>);
            if (redo && !meet()) { ok = false; break; }  // the slots have been read
          }
          if (redo) {
            float mx = -INFINITY;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              uint32_t v[32];
              load(h, v);
              to_log2(h, v);
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                mx = fmax3(mx, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            }
            if (!row_max(&mx)) { ok = false; break; }
            // no reference yet, or a jump P could overflow on: move it now
            const bool move = mx > m_ref + kMoveLog2<kBF16> || (m_ref == -INFINITY && mx != -INFINITY);
            if (__any_sync(0xffffffffu, move)) {
              const float alpha = move && m_ref != -INFINITY ? fast_exp2(m_ref - mx) : 1.f;
              if (j > 0) rescale_o(alpha);
              l *= alpha;
              if (move) m_ref = mx;
            }
            l_t = 0.f;
            take(0);
            take(1);
            const uint32_t mine = __float_as_uint(l_t) >> 23;
            if (!exchange8(mine, &top)) { ok = false; break; }
            top = max(top, mine);
          }
          l += l_t;
          // O is rescaled lazily: when a half's P summed to 2^8 or more, the reference moves up
          // past log2 of that sum before the next tile (so that P stays at most 1 there)
          m_next = top >= 127 + kRescaleExp ? m_ref + static_cast<float>(static_cast<int>(top) - 126)
                                            : m_ref;
          tmem_st16(tS, pk);
          tmem_st16(tS + 16, pk + 16);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[grp]);
        }
        if (!ok) break;
        const int ns_t = !valid ? 0 : kDirect ? 1 : __ldg(p.tok_ns + tok);
        // epilogue: O / l of the warp's half of the columns to the output, or to the split
        // partials
        if (!wait(&bars->o_done[grp], act & 1)) break;
        tc_fence_after();
        // the row's sum, from both halves (in one order, so that both warps have the same)
        float other;
        if (!exchange_float(l, &other)) break;
        l = half ? other + l : l + other;
        const bool write = valid && w.split < ns_t;
        const bool any = !(l == 0.f);  // a row without keys gives zeros, whatever O holds
        const float inv = any ? 1.f / l : 0.f;
        const float2 inv2 = make_float2(inv, inv);
        uint16_t* dst = static_cast<uint16_t*>(p.out) +
                        (static_cast<int64_t>(tok) * p.H_q + head) * D + (D / 2) * half;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
        const int64_t pidx = kDirect || ns_t <= 1
                                 ? 0
                                 : static_cast<int64_t>(__ldg(p.tok_base + tok)) + w.split * p.H_q + head;
        if (write && ns_t > 1 && half == 0)
          p.part_lse[pidx] = any ? m_ref + __log2f(l) : -INFINITY;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t v[32];
          tmem_ld32(tO + c * 32, v);
          tmem_ld_wait();
          if (!write) continue;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x =
                fmul2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), inv2);
            v[e] = any ? __float_as_uint(x.x) : 0u;
            v[e + 1] = any ? __float_as_uint(x.y) : 0u;
          }
          if (ns_t == 1) {
            uint32_t o[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = pack2<kBF16>(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
            if (wide) {
#pragma unroll
              for (int q = 0; q < 2; ++q) st_global_v8(dst + c * 32 + 16 * q, o + 8 * q);
            } else {
              uint4* d4 = reinterpret_cast<uint4*>(dst + c * 32);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                d4[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
          } else {
            uint4* d4 = reinterpret_cast<uint4*>(p.part_o + pidx * D + (D / 2) * half + c * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              d4[q] = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
        }
        ++act;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (!kDirect && p.after_split && blockIdx.x == 0 && threadIdx.x == 0) pdl_wait();
}

template <bool kBF16, int D, bool kDirect, int kCap, bool kBias, class Params>
static cudaError_t launch_masked_tile_t(const Params& p, const CUtensorMap& kmap,
                                        const CUtensorMap& vmap, const CUtensorMap& qmap,
                                        int ctas, cudaStream_t stream) {
  constexpr int smem = TileSmem<D>::kBytes;
  auto kern = masked_tile_kernel<Params, kBF16, D, kDirect, kCap, kBias>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_smem_limit(kern, smem, done);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(ctas), dim3(kThreads<(kCap > 0 || kBias)>), smem, stream, true, kmap, vmap, qmap, p);
}

// The instantiations of one (cap, bias) pair: one per type, head size and mode.
template <int kCap, bool kBias, class Params>
static cudaError_t launch_masked_tile_kind(const Params& p, bool bf16,
                                           const CUtensorMap& kmap, const CUtensorMap& vmap,
                                           const CUtensorMap& qmap, int ctas,
                                           cudaStream_t stream, bool direct) {
  auto go = [&](auto b, auto d, auto m) {
    return launch_masked_tile_t<b.value, d.value, m.value, kCap, kBias>(p, kmap, vmap, qmap, ctas,
                                                                        stream);
  };
  using std::bool_constant;
  auto mode = [&](auto b, auto d) {
    return direct ? go(b, d, bool_constant<true>{}) : go(b, d, bool_constant<false>{});
  };
  auto size = [&](auto b) {
    return p.D == 128 ? mode(b, std::integral_constant<int, 128>{})
                      : mode(b, std::integral_constant<int, 64>{});
  };
  return bf16 ? size(bool_constant<true>{}) : size(bool_constant<false>{});
}

}  // namespace ps
