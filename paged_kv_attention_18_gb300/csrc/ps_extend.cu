// The blocks, slots, positions and packed offsets of a step, made on the device from every
// sequence's length and number of new tokens: pages past the tables' ends get blocks from a
// stack of free ones, and what a sliding window has left behind, or a sequence that ends
// holds, goes back onto it first.
//
//     need_b  = ceil((L_b + n_b) / 16) - ceil(L_b / 16)   blocks, in order of (sequence, page)
//     block i = free[count - 1 - i]                        (count: after the returns)
//     slot    = block(page) * 16 + position % 16
//
// One cluster: every CTA scans the whole batch (blocks given back, needed, tokens: sums over
// the sequences) into its own shared memory, all wait for one another, since lengths, count,
// tables and stack are changed in place, and then each writes its share of the sequences, the
// new blocks and the packed tokens, which find their sequence by bisection. A token on a new
// page takes its block from the stack, not from the table that another thread writes. Nothing
// here is work: a step is bound by the launch, the loads one behind another (lengths, table or
// stack) and the barriers.
#include <cooperative_groups.h>

#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;            // of the cluster (the portable size)
constexpr int kPerCta = 4 * kThreads;  // tokens and sequences that ask for another CTA

struct Two {
  long long x, y;
};

// Exclusive sums over the block, and the totals.
__device__ Two block_exscan(Two v, Two* sh, Two& total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  Two s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, s.x, o), b = __shfl_up_sync(0xffffffffu, s.y, o);
    if (lane >= o) {
      s.x += a;
      s.y += b;
    }
  }
  if (lane == 31) sh[wid] = s;
  __syncthreads();
  Two before{0, 0}, all{0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const Two t = sh[w];
    if (w < wid) {
      before.x += t.x;
      before.y += t.y;
    }
    all.x += t.x;
    all.y += t.y;
  }
  __syncthreads();
  total = all;
  return Two{before.x + s.x - v.x, before.y + s.y - v.y};
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

// The entries that sequence b of length L gives back, visited by a warp: `take(page, id, nth)`
// for each, the highest page first. All of them for a sequence that ends; for a window, the pages
// that no later row sees, from the last one down to the first that is gone already. Returns how
// many.
template <class Take>
__device__ __forceinline__ int returned(const ExtendParams& p, int b, int L, bool ends, Take take) {
  const int lane = threadIdx.x & 31;
  const int32_t* row = p.tables + static_cast<int64_t>(b) * p.max_blocks;
  int low = 0, high = pages_of(L);  // [low, high)
  if (!ends) {
    if (p.window <= 0) return 0;
    low = pages_of(p.sinks);
    high = L - p.window + 1 > 0 ? (L - p.window + 1) / kBlockSize : 0;
  }
  int n = 0;
  for (int top = high - 1; top >= low; top -= 32) {
    const int page = top - lane;
    const int id = page >= low ? row[page] : -1;
    const bool held = id >= 0 && id < p.num_blocks;
    unsigned has = __ballot_sync(0xffffffffu, held);
    if (!ends && ~has != 0u) has &= (1u << (__ffs(~has) - 1)) - 1u;  // up to the first gone
    if ((has >> lane) & 1u) take(page, id, n + __popc(has & ((1u << lane) - 1u)));
    n += __popc(has);
    if (!ends && ~has != 0u) break;
  }
  return n;
}

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
  uint8_t* s_end = reinterpret_cast<uint8_t*>(s_ret + p.B + 1);  // [B] 1: ends; 2: left out
  const int tid = threadIdx.x, warp = tid >> 5;
  pdl_wait();

  int count = *p.free_count;
  if (count < 0 || count > p.free_capacity) {
    if (rank == 0 && tid == 0) record_error(p.err, kDevBadBlockId);
    count = 0;
  }
  // what each sequence asks for; the blocks given back
  for (int b = tid; b < p.B; b += kThreads) {
    const int n = p.new_lens[b], L = p.seq_lens[b];
    const int64_t room = static_cast<int64_t>(p.max_blocks) * kBlockSize;
    const bool ok = L >= 0 && L <= room && (n < 0 || static_cast<int64_t>(L) + n <= room) &&
                    static_cast<int64_t>(L) + n <= 0x7fffffff - 1024;
    if (!ok && rank == 0) record_error(p.err, kDevBadSequence);
    s_len[b] = L;
    s_end[b] = !ok ? 2 : n < 0 ? 1 : 0;
    s_tok[b] = ok && n > 0 ? n : 0;
    s_blk[b] = ok && n > 0 ? pages_of(L + n) - pages_of(L) : 0;
    s_ret[b] = 0;
  }
  __syncthreads();
  int gave = 0;
  {
    bool any = p.window > 0;
    for (int b = tid; !any && b < p.B; b += kThreads) any = s_end[b] == 1;
    if (__syncthreads_or(any)) {
      for (int b = warp; b < p.B; b += kWarps) {
        const int n =
            s_end[b] == 2 ? 0 : returned(p, b, s_len[b], s_end[b] == 1, [](int, int, int) {});
        if ((tid & 31) == 0) s_ret[b] = n;
      }
      __syncthreads();
      long long run = 0;
      for (int base = 0; base < p.B; base += kThreads) {
        const int b = base + tid;
        Two total;
        const Two e = block_exscan(Two{b < p.B ? s_ret[b] : 0, 0}, sh, total);
        if (b < p.B) s_ret[b] = static_cast<int>(run + e.x);
        run += total.x;
      }
      gave = static_cast<int>(run);  // (at most every entry of the tables once)
    }
  }
  if (gave > p.free_capacity - count) {  // more than the stack holds: blocks given back twice
    if (rank == 0 && tid == 0) record_error(p.err, kDevBadBlockId);
  }
  const int have = min(gave, p.free_capacity - count) + count;
  // who is served: what is asked for up to and with it is there
  long long run_tok = 0, run_blk = 0, at_tok = 0, at_blk = 0;
  for (int base = 0; base < p.B; base += kThreads) {
    const int b = base + tid;
    const Two want{b < p.B ? s_tok[b] : 0, b < p.B ? s_blk[b] : 0};
    Two total, given;
    const Two e = block_exscan(want, sh, total);
    const bool room = run_tok + e.x + want.x <= p.T;
    const bool blocks = want.y == 0 || run_blk + e.y + want.y <= have;
    const bool ok = room && blocks;
    if (!ok && rank == 0) record_error(p.err, room ? kDevNoBlocks : kDevBadSequence);
    const Two g = block_exscan(ok ? want : Two{0, 0}, sh, given);
    if (b < p.B) {
      s_tok[b] = static_cast<int>(at_tok + g.x);
      s_blk[b] = static_cast<int>(at_blk + g.y);
    }
    run_tok += total.x;
    run_blk += total.y;
    at_tok += given.x;
    at_blk += given.y;
  }
  const int tokens = static_cast<int>(at_tok), blocks = static_cast<int>(at_blk);
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
      returned(p, b, s_len[b], s_end[b] == 1, [&](int page, int id, int nth) {
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
    p.out_lens[b] = s_end[b] == 1 ? 0 : s_len[b] + (s_tok[b + 1] - s_tok[b]);
  }
  if (me == 0) *p.out_count = have - blocks;
  auto fresh = [&](int nth) {  // the nth new block, or -1
    const int id = p.free_blocks[have - 1 - nth];
    const bool ok = id >= 0 && id < p.num_blocks;
    if (!ok) record_error(p.err, kDevBadBlockId);
    return ok ? id : -1;
  };
  for (int i = me; i < blocks; i += stride) {
    const int b = last_le(s_blk, p.B, i);
    const int page = pages_of(s_len[b]) + i - s_blk[b];
    p.tables[static_cast<int64_t>(b) * p.max_blocks + page] = fresh(i);
  }
  for (int t = me; t < p.T; t += stride) {
    int slot = -1, pos = 0;
    if (t < tokens) {
      const int b = last_le(s_tok, p.B, t), L = s_len[b];
      pos = L + t - s_tok[b];
      const int page = pos / kBlockSize, had = pages_of(L);
      int id;
      if (page >= had) {
        id = fresh(s_blk[b] + page - had);
      } else {
        id = p.tables[static_cast<int64_t>(b) * p.max_blocks + page];
        if (id < 0 || id >= p.num_blocks) {
          record_error(p.err, kDevBadBlockId);
          id = -1;
        }
      }
      if (id >= 0) slot = id * kBlockSize + pos % kBlockSize;
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
}

}  // namespace

cudaError_t launch_extend(const ExtendParams& p, cudaStream_t stream) {
  const int smem = 4 * (p.B + 1) * static_cast<int>(sizeof(int)) + p.B;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e =
      ensure_smem_limit(extend_kernel, 17 * (kExtendMaxSeqs + 1), done);
  if (e != cudaSuccess) return e;
  const int64_t want = (static_cast<int64_t>(p.T) + p.B + kPerCta - 1) / kPerCta;
  const int ctas = static_cast<int>(want < 1 ? 1 : want < kMaxCtas ? want : kMaxCtas);
  return launch_cluster(extend_kernel, ctas, ctas, kThreads, smem, stream, p);
}

}  // namespace ps
