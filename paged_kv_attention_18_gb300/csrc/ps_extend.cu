// The blocks, slots, positions and packed offsets of a step, made on the device from every
// sequence's length and number of new tokens: pages past the tables' ends get blocks from a
// stack of free ones, and what a sliding window has left behind, or a sequence that ends
// holds, goes back onto it first.
//
//     need_b  = max(ceil((L_b + n_b) / 16) - H_b, 0)      blocks, in order of (sequence, page)
//     block i = free[count - 1 - i]                        (count: after the returns)
//     slot    = block(page) * 16 + position % 16
//
// H_b: the pages that the sequence holds, ceil(L_b / 16), or more where tokens were taken back
// (then counted by the caller's array, which the kernel keeps).
//
// One cluster: every CTA scans the whole batch (blocks given back, needed, tokens: sums over
// the sequences) into its own shared memory, all wait for one another, since lengths, count,
// tables and stack are changed in place, and then each writes its share of the sequences, the
// new blocks and the packed tokens, which find their sequence by bisection. A token on a new
// page takes its block from the stack, not from the table that another thread writes. Nothing
// here is work: a step is bound by the launch, the loads one behind another (lengths, table or
// stack) and the barriers. 256 decodes take 3.6 us (of which a call takes 3), 1000 sequences of
// up to 65 tokens 11.2: 4.9 and 15.5 with sums in 64 bits and a sequence a thread at a time; 1024
// threads a CTA took 8.9 and 13.8. Blocks that are given back cost more, twice a warp's look at each
// sequence's table, one behind the other: 256 decodes under a window of 1000 keys 13.4, 1000 of them
// 41; 16 sequences of 128 to 256 pages that end among 256, all of one warp, 55 more.
#include <cooperative_groups.h>

#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;            // of the cluster (the portable size)
constexpr int kPerCta = 4 * kThreads;  // tokens and sequences that ask for another CTA

// Tokens and blocks, as sums that stop at a cap each (one more than there is room for): 32 bits
// hold them whatever is asked for, and sums of sums are the same in any grouping.
struct Two {
  unsigned x, y;
};
__device__ __forceinline__ Two add(Two a, Two b, Two cap) {
  return Two{min(a.x + b.x, cap.x), min(a.y + b.y, cap.y)};
}

// Sums over the threads before this one, and over all.
__device__ __forceinline__ Two block_exscan(Two v, Two cap, Two* sh, Two& total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  auto up = [&](Two s, int o) {
    return Two{__shfl_up_sync(0xffffffffu, s.x, o), __shfl_up_sync(0xffffffffu, s.y, o)};
  };
  Two s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two y = up(s, o);
    if (lane >= o) s = add(s, y, cap);
  }
  Two before = up(s, 1);
  if (lane == 0) before = Two{0, 0};
  __syncthreads();
  if (lane == 31) sh[wid] = s;
  __syncthreads();
  Two w = lane < kWarps ? sh[lane] : Two{0, 0};
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const Two y = up(w, o);
    if (lane >= o) w = add(w, y, cap);
  }
  total = Two{__shfl_sync(0xffffffffu, w.x, kWarps - 1), __shfl_sync(0xffffffffu, w.y, kWarps - 1)};
  const Two base{__shfl_sync(0xffffffffu, w.x, (wid + 31) & 31),
                 __shfl_sync(0xffffffffu, w.y, (wid + 31) & 31)};
  return wid > 0 ? add(base, before, cap) : before;
}

// The largest b in [0, n) with at[b] <= x (at rises, at[0] <= x).
__device__ __forceinline__ int last_le(const int* at, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(int L) {
  return static_cast<int>((static_cast<unsigned>(L) + kBlockSize - 1) / kBlockSize);
}

// The entries that sequence b of length L with `had` pages gives back, visited by a warp:
// `take(page, id, nth)` for each, the highest page first. All of them for a sequence that ends; for
// a window, the pages that no later row sees, from the last one down to the first that is gone
// already. An entry that is no block of the pool is recorded and passed over. Returns how many.
template <class Take>
__device__ __forceinline__ int returned(const ExtendParams& p, int b, int L, int had, bool ends,
                                        Take take) {
  const int lane = threadIdx.x & 31;
  const int32_t* row = p.tables + static_cast<int64_t>(b) * p.max_blocks;
  int low = 0, high = had;  // [low, high)
  if (!ends) {
    if (p.window <= 0) return 0;
    low = pages_of(p.sinks);
    high = L - p.window + 1 > 0 ? (L - p.window + 1) / kBlockSize : 0;
  }
  int n = 0;
  for (int top = high - 1; top >= low; top -= 32) {
    const int page = top - lane;
    const int id = page >= low ? row[page] : -1;
    unsigned has = __ballot_sync(0xffffffffu, id >= 0);
    const bool gone = !ends && ~has != 0u;
    if (gone) has &= (1u << (__ffs(~has) - 1)) - 1u;  // up to the first gone
    if ((has >> lane) & 1u && id >= p.num_blocks) record_error(p.err, kDevBadBlockId);
    has &= __ballot_sync(0xffffffffu, id < p.num_blocks);
    if ((has >> lane) & 1u) take(page, id, n + __popc(has & ((1u << lane) - 1u)));
    n += __popc(has);
    if (gone) break;
  }
  return n;
}

// kHeld: p.held has the sequences' pages.
template <bool kHeld>
__global__ void __launch_bounds__(kThreads) extend_kernel(const ExtendParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int ctas = static_cast<int>(cluster.num_blocks());
  __shared__ Two sh[kWarps];
  extern __shared__ int arrays[];
  int* s_len = arrays;              // [B] context before the step
  int* s_tok = s_len + p.B + 1;     // [B + 1] first packed token
  int* s_blk = s_tok + p.B + 1;     // [B + 1] first new block
  int* s_ret = s_blk + p.B + 1;     // [B + 1] first block given back
  int* s_had = s_ret + p.B + 1;     // [B] pages held before the step (kHeld)
  // [B] 1: the sequence ends; 2: it is bad; 4: it goes without
  uint8_t* s_end = reinterpret_cast<uint8_t*>(s_had + (kHeld ? p.B : 0));
  auto had = [&](int b) {
    if constexpr (kHeld) return s_had[b];
    else return pages_of(s_len[b]);
  };
  const int tid = threadIdx.x, warp = tid >> 5;
  pdl_wait();

  int count = *p.free_count;
  if (count < 0 || count > p.free_capacity) {
    if (rank == 0 && tid == 0) record_error(p.err, kDevBadBlockId);
    count = 0;
  }
  // what each sequence asks for, and the blocks it gives back
  for (int b = tid; b < p.B; b += kThreads) {
    const int n = p.new_lens[b], L = p.seq_lens[b];
    const int64_t room = static_cast<int64_t>(p.max_blocks) * kBlockSize;
    bool ok = L >= 0 && L <= room && (n < 0 || static_cast<int64_t>(L) + n <= room) &&
              static_cast<int64_t>(L) + n <= 0x7fffffff - 1024;
    int pages = pages_of(L);
    if constexpr (kHeld) {
      const int held = p.held[b];
      ok = ok && held >= pages && held <= p.max_blocks;
      s_had[b] = pages = held;
    }
    if (!ok && rank == 0) record_error(p.err, kDevBadSequence);
    s_len[b] = L;
    s_end[b] = !ok ? 2 : n < 0 ? 1 : 0;
    s_tok[b] = ok && n > 0 ? n : 0;
    s_blk[b] = ok && n > 0 ? max(pages_of(L + n) - pages, 0) : 0;
    s_ret[b] = 0;
  }
  __syncthreads();
  // (a thread's sequences are neighbours)
  const int share = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * share, p.B), b_hi = min(b_lo + share, p.B);
  int gave = 0;
  {
    bool any = p.window > 0;
    for (int b = b_lo; !any && b < b_hi; ++b) any = s_end[b] == 1;
    if (__syncthreads_or(any)) {
      for (int b = warp; b < p.B; b += kWarps) {
        const int n =
            s_end[b] == 2
                ? 0
                : returned(p, b, s_len[b], had(b), s_end[b] == 1, [](int, int, int) {});
        if ((tid & 31) == 0) s_ret[b] = n;
      }
      __syncthreads();
      const Two cap{0x7fffffffu, 0};  // (at most every entry of the tables once)
      Two sum{0, 0}, total;
      for (int b = b_lo; b < b_hi; ++b) sum.x += s_ret[b];
      unsigned at = block_exscan(sum, cap, sh, total).x;
      for (int b = b_lo; b < b_hi; ++b) {
        const int n = s_ret[b];
        s_ret[b] = static_cast<int>(at);
        at += n;
      }
      gave = static_cast<int>(total.x);
    }
  }
  if (gave > p.free_capacity - count) {  // more than the stack holds: blocks given back twice
    if (rank == 0 && tid == 0) record_error(p.err, kDevBadBlockId);
  }
  const int have = min(gave, p.free_capacity - count) + count;
  // Who is served: what is asked for up to and with it is there. Blocks run out for every sequence
  // behind the first that goes without, but for those that need none; so do tokens. So a served
  // sequence's blocks lie behind those of all before it, and only its tokens' place wants a sum of
  // its own, if some sequence goes without.
  const Two cap{static_cast<unsigned>(p.T) + 1, static_cast<unsigned>(have) + 1};
  int tokens, blocks;
  {
    Two sum{0, 0}, total;
    for (int b = b_lo; b < b_hi; ++b)
      sum = add(sum, Two{static_cast<unsigned>(s_tok[b]), static_cast<unsigned>(s_blk[b])}, cap);
    Two at = block_exscan(sum, cap, sh, total);
    unsigned last = 0, kept = 0;  // blocks up to the thread's last served one; tokens
    bool all = true;
    for (int b = b_lo; b < b_hi; ++b) {
      const Two want{static_cast<unsigned>(s_tok[b]), static_cast<unsigned>(s_blk[b])};
      const Two end = add(at, want, cap);
      const bool room = end.x < cap.x, there = want.y == 0 || end.y < cap.y;
      const bool ok = (room && there) || (want.x == 0 && want.y == 0);
      if (ok) {
        if (want.y != 0) last = end.y;
        kept += want.x;
        s_tok[b] = static_cast<int>(at.x);
      } else {
        if (rank == 0) record_error(p.err, room ? kDevNoBlocks : kDevBadSequence);
        all = false;
        s_end[b] = 4;
      }
      s_blk[b] = static_cast<int>(at.y);
      at = end;
    }
    tokens = static_cast<int>(total.x);
    blocks = static_cast<int>(total.y);
    if (!__syncthreads_and(all)) {
      // tokens of the served; blocks up to the last of them
      Two sums;
      unsigned to = block_exscan(Two{kept, 0}, cap, sh, sums).x;
      tokens = static_cast<int>(sums.x);
      __syncthreads();
      last = __reduce_max_sync(0xffffffffu, last);
      if ((tid & 31) == 0) sh[warp].x = last;
      __syncthreads();
      blocks = 0;
      for (int w = 0; w < kWarps; ++w) blocks = max(blocks, static_cast<int>(sh[w].x));
      for (int b = b_lo; b < b_hi; ++b) {
        const int n = s_end[b] == 0 ? p.new_lens[b] : 0;
        s_tok[b] = static_cast<int>(to);
        to += n;
        s_blk[b] = min(s_blk[b], blocks);
      }
    }
  }
  if (tid == 0) {
    s_tok[p.B] = tokens;
    s_blk[p.B] = blocks;
    s_ret[p.B] = gave;
  }
  if (ctas > 1) cluster.sync();  // everything has been read that is written below
  else __syncthreads();

  if (gave > 0) {
    for (int b = rank * kWarps + warp; b < p.B; b += ctas * kWarps) {
      if (s_ret[b + 1] == s_ret[b]) continue;
      const int first = count + s_ret[b];
      int32_t* row = p.tables + static_cast<int64_t>(b) * p.max_blocks;
      returned(p, b, s_len[b], had(b), s_end[b] == 1, [&](int page, int id, int nth) {
        if (first + nth < p.free_capacity) p.free_blocks[first + nth] = id;
        row[page] = -1;
      });
    }
    if (ctas > 1) cluster.sync();  // the returned blocks can be taken again
    else __syncthreads();
  }
  const int stride = ctas * kThreads, me = rank * kThreads + tid;
  for (int b = me; b <= p.B; b += stride) {
    p.qsl[b] = s_tok[b];
    if (b == p.B) break;
    const int L = s_len[b] + (s_tok[b + 1] - s_tok[b]);
    p.out_lens[b] = s_end[b] == 1 ? 0 : L;
    if constexpr (kHeld) {
      if (s_end[b] <= 1) p.held[b] = s_end[b] == 1 ? 0 : max(s_had[b], pages_of(L));
    }
  }
  if (me == 0) *p.out_count = have - blocks;
  for (int i = me; i < blocks; i += stride) {
    const int b = last_le(s_blk, p.B, i);
    const int page = had(b) + i - s_blk[b];
    const int id = p.free_blocks[have - 1 - i];
    const bool ok = id >= 0 && id < p.num_blocks;
    if (!ok) record_error(p.err, kDevBadBlockId);
    p.tables[static_cast<int64_t>(b) * p.max_blocks + page] = ok ? id : -1;
  }
  // A thread's tokens lie a stride apart, a few at a time: it looks for the first one's sequence by
  // bisection, and their blocks' loads are all on their way before the first is used.
  constexpr int kAhead = 4;
  for (int base = me; base < p.T; base += kAhead * stride) {
    int pos[kAhead], slot[kAhead];
    const int32_t* from[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int t = base + u * stride;
      pos[u] = 0;
      from[u] = nullptr;
      if (t < tokens) {
        const int b = last_le(s_tok, p.B, t);
        pos[u] = s_len[b] + t - s_tok[b];
        const int page = pos[u] / kBlockSize, first = had(b);
        from[u] = page >= first ? p.free_blocks + have - 1 - (s_blk[b] + page - first)
                                : p.tables + static_cast<int64_t>(b) * p.max_blocks + page;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) slot[u] = from[u] != nullptr ? *from[u] : -1;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int t = base + u * stride;
      if (t >= p.T) break;
      const bool ok = slot[u] >= 0 && slot[u] < p.num_blocks;
      if (!ok && from[u] != nullptr) record_error(p.err, kDevBadBlockId);
      p.slots[t] = ok ? slot[u] * kBlockSize + pos[u] % kBlockSize : -1;
      p.positions[t] = pos[u];
    }
  }
}

}  // namespace

template <bool kHeld>
static cudaError_t launch_extend_t(const ExtendParams& p, cudaStream_t stream) {
  constexpr int kArrays = kHeld ? 5 : 4;
  const int smem = kArrays * (p.B + 1) * static_cast<int>(sizeof(int)) + p.B;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_smem_limit(extend_kernel<kHeld>,
                                          (4 * kArrays + 1) * (kExtendMaxSeqs + 1), done);
  if (e != cudaSuccess) return e;
  const int64_t want = (static_cast<int64_t>(p.T) + p.B + kPerCta - 1) / kPerCta;
  const int ctas = static_cast<int>(want < 1 ? 1 : want < kMaxCtas ? want : kMaxCtas);
  return launch_cluster(extend_kernel<kHeld>, ctas, ctas, kThreads, smem, stream, p);
}

cudaError_t launch_extend(const ExtendParams& p, cudaStream_t stream) {
  return p.held != nullptr ? launch_extend_t<true>(p, stream) : launch_extend_t<false>(p, stream);
}

}  // namespace ps
