// Eviction from a paged cache by the weight that its keys received (sm_103a).
//
// For each sequence of more than `keep` tokens and each key head: the `first`
// and the `last` tokens stay, and of those between the keep - first - last
// with the largest weights (of equal ones the earlier).  A cluster of blocks
// takes a sequence and head; what is chosen is moved at once, so that one unit's
// choice (latency) runs beside others' moves (memory).
//
// Choice: weights as integers whose order is theirs, a part of the positions in
// each block's shared memory; the smallest that stays is found by its bytes
// from the top (four histograms, summed over the blocks), and the positions of
// what stays are written in order.
//
// Moving: token kept[i] goes to place i, in order, so i <= kept[i].  In place,
// the cluster goes through the kept tokens from the first on, a round at a time:
// all loads of a round complete (a barrier of the cluster) before its stores,
// which fill places below every source of the rounds that follow; so these are
// loading already, two rounds ahead, and the barrier's time is that of the
// last round's stores.  Rounds whose places lie below all sources that the last
// barrier has not covered need none: where a quarter stays that is all but a
// few (67608 tokens to 16384 in 24 heads: 126 -> 99 us; 64 sequences of 8704 to
// 4096 in 8 heads, E4M3: 274 -> 229).  Moves to other pages are a kernel of their
// own (113 -> 106 us for the first one below).
//
// Blocks a unit, the kernel and the shared memory for weights follow what the host
// knows, the sequences, heads and the table's width, not the lengths.  Where a
// block's part of the table's width is above 25600 tokens, the weights' memory leaves
// one block an SM: under a table of 4096 entries the long context below takes 143 us
// and the batch 125 (below, tables are as wide as the longest sequence).  Two
// sequences over the budget among 64 have one block a head all the same: 47 us, and
// 25 alone.
//
// Bound by memory; by latency where there are few tokens (and by the choice, 30 us
// of a long context's).  Measured:
//   64 sequences of 1024 to 8704, 8 heads, E4M3, 2048 stay, to other pages   106 us  4.9 TB/s (75.7 at a copy's rate)
//   one of 67608, 24 heads, BF16, 16384 stay, in place                       98 us  4.2      (60.8)
//                           E4M3                                             74 us  2.9      (31.4)
//   one of 1152, 2 heads, BF16, 1024 stay, in place                          11.9 us  (four histograms, one after another)
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMostBlocks = 8;  // of a unit
// Weights that a block keeps in shared memory; the rest of a longer part is
// read again (from the second-level cache).
constexpr int kSelCache = 48 * 1024;

// A weight as an integer: larger is larger, +0 and -0 alike, NaN above all.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t b = __float_as_uint(w);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if ((b & 0x7FFFFFFFu) == 0) return 0x80000000u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Tokens of sequence s, or -1 when its length or one of its pages (the
// destination's too) is out of range.  By the whole block.
__device__ __forceinline__ int checked_length(const PagedArgs& c, const EvictArgs& e, int s) {
  const int n = c.kv_len[s];
  const int stay = min(n, e.keep);
  bool bad = n < 0 || n > (static_cast<int64_t>(c.table_width) << c.page_shift) ||
             (e.to_table && stay > (static_cast<int64_t>(e.to_width) << c.page_shift));
  if (!bad) {
    const int pages = (n + c.page_size - 1) >> c.page_shift;
    for (int i = threadIdx.x; i < pages; i += blockDim.x) {
      const int page = __ldg(c.table + s * c.table_stride + i);
      bad |= page < 0 || page >= c.pages;
    }
    if (e.to_table) {
      const int to = (stay + c.page_size - 1) >> c.page_shift;
      for (int i = threadIdx.x; i < to; i += blockDim.x) {
        const int page = __ldg(e.to_table + s * e.to_stride + i);
        bad |= page < 0 || page >= c.pages;
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) paged_fail(c);
  return bad ? -1 : n;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same word of another block of the cluster.
__device__ __forceinline__ uint32_t cluster_word(const uint32_t* p, int block) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(block));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// The positions that stay, of unit (s, h) with n > keep tokens: each block of the
// cluster has a part of them, and each warp a part of that, in order.
template <bool kAlone>  // by one block
__device__ __forceinline__ void choose(const PagedArgs& c, const EvictArgs& e, int s, int h, int n, int rank, int cluster,
                                       int cache, uint32_t* s_keys, int32_t* kept) {
  const int blocks = kAlone ? 1 : cluster;
  __shared__ uint32_t s_hist[2][256];      // of every other pass
  __shared__ uint32_t s_all[256];          // of all blocks
  __shared__ uint32_t s_warp[2][kWarps];   // greater and equal, of each warp
  __shared__ uint32_t s_block[2];          // and of the block
  __shared__ uint32_t s_prefix, s_left;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int threads = kThreads;
  const int first_thread = rank * threads + threadIdx.x, all_threads = blocks * threads;
  const int m = n - e.first - e.last;                  // tokens to choose from
  const int want = e.keep - e.first - e.last;          // of them stay
  for (int i = first_thread; i < e.first; i += all_threads) kept[i] = i;
  for (int i = first_thread; i < e.last; i += all_threads) kept[e.keep - e.last + i] = n - e.last + i;
  if (want == 0) return;
  // the block's positions: [b0, b1), whole parts of 32 for each warp
  const int per_warp = (m + all_threads - 1) / all_threads * 32, per_block = per_warp * (threads / 32);
  const int b0 = min(static_cast<int64_t>(m), static_cast<int64_t>(rank) * per_block), b1 = min(static_cast<int64_t>(m), static_cast<int64_t>(b0) + per_block);
  // Weights past the shared memory are read in every pass.  Where another sequence's
  // moves change them meanwhile, on a page that the two must not share, more or fewer
  // may stay than there is room for: whatever comes of it, places hold positions.
  if (per_block > cache)
    for (int i = first_thread; i < want; i += all_threads) kept[e.first + i] = e.first + i;
  const int32_t* table = c.table + s * c.table_stride;
  auto weight_at = [&](int i) {
    const int pos = e.first + i, page = __ldg(table + (pos >> c.page_shift));
    return order_of(__ldg(e.weights + ((static_cast<int64_t>(page) * c.H + h) << c.page_shift) + (pos & (c.page_size - 1))));
  };
  auto key = [&](int i) { return i - b0 < cache ? s_keys[i - b0] : weight_at(i); };
#pragma unroll 8
  for (int i = b0 + threadIdx.x; i < min(b1, b0 + cache); i += threads) s_keys[i - b0] = weight_at(i);
  // the want-th largest key, byte by byte
  uint32_t prefix = 0, left = want;
  for (int shift = 24, pass = 0; shift >= 0; shift -= 8, pass ^= 1) {
    uint32_t* hist = s_hist[pass];
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = b0 + threadIdx.x; i < b1; i += threads) {
      const uint32_t k = key(i);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[k >> shift & 255], 1u);
    }
    if (blocks > 1) cluster_sync();
    else __syncthreads();
    if (blocks > 1) {
      if (threadIdx.x < 256) {
        uint32_t of[kMostBlocks], all = 0;
#pragma unroll
        for (int o = 0; o < kMostBlocks; ++o) of[o] = o < blocks ? cluster_word(&hist[threadIdx.x], o) : 0u;
#pragma unroll
        for (int o = 0; o < kMostBlocks; ++o) all += of[o];
        s_all[threadIdx.x] = all;
      }
      __syncthreads();
      hist = s_all;
    }
    if (warp == 0) {  // lane: bins 255 - 8 lane .. down
      uint32_t mine[8], sum = 0;
#pragma unroll
      for (int b = 0; b < 8; ++b) sum += mine[b] = hist[255 - 8 * lane - b];
      uint32_t upto = sum;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += y;
      }
      uint32_t before = upto - sum;
      if (before < left && upto >= left) {
        for (int b = 0; b < 8; ++b) {
          if (before + mine[b] >= left) {
            s_prefix = prefix << 8 | (255 - 8 * lane - b);
            s_left = left - before;
            break;
          }
          before += mine[b];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
    // (the next pass has the other histogram, and its barrier comes before this one is cleared)
  }
  const uint32_t least = prefix;
  const int equals = left;  // of those equal to the least this many stay
  // Counts of each warp's part first, then the places.
  const int i0 = min(b1, b0 + warp * per_warp), i1 = min(b1, i0 + per_warp);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t k = in ? key(i + lane) : 0u;
    gt += __popc(__ballot_sync(0xFFFFFFFFu, in && k > least));
    eq += __popc(__ballot_sync(0xFFFFFFFFu, in && k == least));
  }
  if (lane == 0) {
    s_warp[0][warp] = gt;
    s_warp[1][warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    const bool is = lane < threads / 32;
    const int a = is ? s_warp[0][lane] : 0, b = is ? s_warp[1][lane] : 0;
    int x = a, y = b;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, x, d), v = __shfl_up_sync(0xFFFFFFFFu, y, d);
      if (lane >= d) {
        x += u;
        y += v;
      }
    }
    if (is) {  // of the warps before
      s_warp[0][lane] = x - a;
      s_warp[1][lane] = y - b;
    }
    if (lane == 31) {
      s_block[0] = x;
      s_block[1] = y;
    }
  }
  if (blocks > 1) cluster_sync();
  else __syncthreads();
  int gt_before = s_warp[0][warp], eq_before = s_warp[1][warp];
  if (blocks > 1) {
    gt_before += __reduce_add_sync(0xFFFFFFFFu, lane < rank ? cluster_word(&s_block[0], lane) : 0u);
    eq_before += __reduce_add_sync(0xFFFFFFFFu, lane < rank ? cluster_word(&s_block[1], lane) : 0u);
  }
  // (read by others until the barrier behind the choice)
  int at = gt_before + min(eq_before, equals);
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t k = in ? key(i + lane) : 0u;
    const unsigned same = __ballot_sync(0xFFFFFFFFu, in && k == least), below = (1u << lane) - 1;
    const bool stays = in && (k > least || (k == least && eq_before + __popc(same & below) < equals));
    const unsigned mask = __ballot_sync(0xFFFFFFFFu, stays);
    const int to = at + __popc(mask & below);
    if (stays && to < want) kept[e.first + to] = e.first + i + lane;
    at += __popc(mask);
    eq_before += __popc(same);
  }
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

template <int kKind>
struct Move {
  static constexpr int kRow = kKind == 0 ? 256 : 128;            // bytes of a row of K or V
  static constexpr int kTokenBytes = 2 * kRow;
  static constexpr int kPerWarp = kKind == 0 ? 3 : 6;            // tokens of a warp and round
  static constexpr int kTokens = kPerWarp * kWarps;          // of a block and round
  static constexpr uint32_t kBuffer = kTokens * kTokenBytes;
  static constexpr int kBuffers = 4;
  static constexpr uint32_t kSmem = kBuffers * kBuffer + 8 * kThreads;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two blocks an SM");
};

template <int kKind, bool kAlone, bool kInPlace>  // kAlone: the cluster's first block chooses, else all
__global__ void __launch_bounds__(kThreads) evict_kernel(const PagedArgs c, const EvictArgs e, int blocks, int cache) {
  using M = Move<kKind>;
  extern __shared__ __align__(128) uint8_t s_rows[];  // weights, then rows
  const int unit = blockIdx.x / blocks, rank = blockIdx.x % blocks;
  const int s = unit / c.H, h = unit % c.H;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr bool in_place = kInPlace;
  int32_t* kept = e.kept + static_cast<int64_t>(unit) * e.keep;
  const int32_t* from_table = c.table + s * c.table_stride;
  const int32_t* to_table = in_place ? from_table : e.to_table + s * e.to_stride;
  // (the same for all blocks of a cluster)
  const int have = checked_length(c, e, s), n = min(have, e.keep);
  if (h == 0 && rank == 0 && threadIdx.x == 0) e.new_len[s] = have < 0 ? c.kv_len[s] : n;
  if (have <= e.keep) {  // (of a refused sequence nothing moves)
    for (int i = rank * kThreads + threadIdx.x; i < e.keep; i += blocks * kThreads) kept[i] = i < have ? i : -1;
    if (in_place || have <= 0) return;
  } else if (!kAlone || rank == 0) {
    choose<kAlone>(c, e, s, h, have, rank, blocks, cache, reinterpret_cast<uint32_t*>(s_rows), kept);
  }
  if (blocks > 1) cluster_sync();
  else __syncthreads();
  // A warp moves its tokens alone; only the rounds' barriers join the warps.
  const int step = M::kTokens * blocks;
  const int rounds = (n + step - 1) / step;  // (n <= 2^30)
  const uint32_t base = smem_u32(s_rows) + warp * M::kPerWarp * M::kTokenBytes;
  const uint32_t side = smem_u32(s_rows) + M::kBuffers * M::kBuffer + threadIdx.x * 8;
  struct Token {
    int64_t src, dst;  // rows; src < 0: nothing to move
    float w;
    uint8_t ke, ve;
  };
  // lane x < kPerWarp has token x of the warp and round.  A round's positions,
  // its pages, and its rows are loaded a round after another.
  const int mine = (rank * kWarps + warp) * M::kPerWarp + lane;
  auto place = [&](int round) { return round * step + mine; };
  auto position = [&](int round) {
    const int i = place(round);
    return round < rounds && lane < M::kPerWarp && i < n ? kept[i] : -1;
  };
  auto lookup = [&](int round, int pos) {
    Token t;
    t.src = t.dst = -1;
    t.w = 0.f;
    t.ke = t.ve = 0;
    const int i = place(round);
    if (pos >= 0 && !(in_place && pos == i)) {
      t.src = __ldg(from_table + (pos >> c.page_shift));
      t.dst = __ldg(to_table + (i >> c.page_shift));
      t.src = ((t.src * c.H + h) << c.page_shift) + (pos & (c.page_size - 1));
      t.dst = ((t.dst * c.H + h) << c.page_shift) + (i & (c.page_size - 1));
    }
    return t;
  };
  auto load = [&](int round, Token& t) {
    const uint32_t to = base + round % M::kBuffers * M::kBuffer;
    constexpr int kLanes = kKind == 0 ? 32 : 16, kAtOnce = 32 / kLanes;  // a token's lanes: half K, half V
    const int sub = lane % kLanes, chunk = sub % (kLanes / 2) * 16;
    const uint8_t* pages = sub < kLanes / 2 ? c.k_pages : c.v_pages;
#pragma unroll
    for (int x = 0; x < M::kPerWarp; x += kAtOnce) {
      const int y = x + lane / kLanes;
      const int64_t src = __shfl_sync(0xFFFFFFFFu, t.src, y);
      if (src >= 0) cp_async16(to + y * M::kTokenBytes + sub * 16, pages + src * M::kRow + chunk, true);
    }
    cp_commit();
    if (t.src >= 0) {
      t.w = e.weights[t.src];
      if (kKind != 0) {
        t.ke = c.k_exp[t.src];
        t.ve = c.v_exp[t.src];
      }
    }
  };
  auto finish = [&](int round, const Token& t) {
    const uint32_t from = base + round % M::kBuffers * M::kBuffer;
    constexpr int kLanes = kKind == 0 ? 32 : 16, kAtOnce = 32 / kLanes;
    const int sub = lane % kLanes, chunk = sub % (kLanes / 2) * 16;
    uint8_t* pages = sub < kLanes / 2 ? c.k_pages : c.v_pages;
#pragma unroll
    for (int x = 0; x < M::kPerWarp; x += kAtOnce) {
      const int y = x + lane / kLanes;
      const int64_t dst = __shfl_sync(0xFFFFFFFFu, t.dst, y);
      if (dst >= 0) {
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(from + y * M::kTokenBytes + sub * 16));
        *reinterpret_cast<uint4*>(pages + dst * M::kRow + chunk) = v;
      }
    }
    if (t.dst >= 0) {
      e.weights[t.dst] = t.w;
      if (kKind != 0) {
        c.k_exp[t.dst] = t.ke;
        c.v_exp[t.dst] = t.ve;
      }
    }
    __syncwarp();  // the buffer is free
  };
  // Places of round r lie below (r + 1) step.  Where the first token that the last
  // barrier has not covered comes from behind them, none of their sources is
  // still to be loaded, and the round's stores need no barrier of their own.
  auto uncovered = [&](int round) {
    const int64_t i = static_cast<int64_t>(round + 1) * step;
    return i < n ? kept[i] : 0x7FFFFFFF;
  };
  // (Of the first rounds they are in shared memory: a load in the loop would wait for
  // the rows before it.  Later ones have a barrier each.)
  __shared__ int s_limit[kThreads];
  int limit = in_place ? uncovered(threadIdx.x) : 0;
  // In iteration r the rows of round r have arrived, those of r + 1 and r + 2
  // are on their way, those of r - 1 go out while the cluster's blocks meet.
  Token before, now = lookup(0, position(0)), next = lookup(1, position(1)), after = lookup(2, position(2));
  int pos = position(3);
  load(0, now);
  load(1, next);
  if (in_place) {
    s_limit[threadIdx.x] = limit;
    limit = 0;
    __syncthreads();
  }
  // (BF16: in a loop of one the rounds' registers change places, which waits for
  // their loads: 134 against 124 us for what stays in place nearly as it is; E4M3:
  // four are 97 against 76 us for the long context)
#pragma unroll (kKind == 0 ? 4 : 1)
  for (int r = 0; r <= rounds; ++r) {
    Token last = lookup(r + 3, pos);
    pos = position(r + 4);
    bool meet = false;  // (the same for the whole cluster)
    if (r < rounds) {
      load(r + 2, after);
      cp_wait<2>();
      __syncwarp();
      if (in_place) {
        // What a lane loads into registers has to arrive before the barrier, too:
        // a store needs it.
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(side), "r"(__float_as_uint(now.w)),
                     "r"(static_cast<uint32_t>(now.ke) | static_cast<uint32_t>(now.ve) << 8)
                     : "memory");
        meet = __any_sync(0xFFFFFFFFu, limit < (r + 1) * step);  // (a vote: the compiler knows that a warp agrees)
        if (meet) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      }
    }
    if (r > 0) finish(r - 1, before);
    if (meet) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      limit = r < kThreads ? s_limit[r] : 0;
    }
    before = now;
    now = next;
    next = after;
    after = last;
  }
}

template <int kKind, bool kAlone, bool kInPlace>
cudaError_t launch_kernel(const PagedArgs& c, const EvictArgs& e, int64_t units, int blocks, int cache, cudaStream_t s) {
  using M = Move<kKind>;
  auto* kern = evict_kernel<kKind, kAlone, kInPlace>;
  static SmemOnce once;
  const uint32_t weights = static_cast<uint32_t>(cache) * 4, bytes = M::kSmem > weights ? M::kSmem : weights;
  constexpr uint32_t most = M::kSmem > kSelCache * 4 ? M::kSmem : kSelCache * 4;
  const cudaError_t err = once.set(reinterpret_cast<const void*>(kern), most);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, c, e, blocks, cache);
}

template <int kKind, bool kAlone>
cudaError_t launch(const PagedArgs& c, const EvictArgs& e, int64_t units, int blocks, int cache, cudaStream_t s) {
  return e.to_table ? launch_kernel<kKind, kAlone, false>(c, e, units, blocks, cache, s)
                    : launch_kernel<kKind, kAlone, true>(c, e, units, blocks, cache, s);
}

}  // namespace

cudaError_t launch_evict(const PagedArgs& c, const EvictArgs& e, int sms, cudaStream_t s) {
  const int64_t units = static_cast<int64_t>(c.seqs) * c.H;
  const int64_t longest = static_cast<int64_t>(c.table_width) << c.page_shift;
  // Two blocks an SM at most, of which a unit gets up to eight: 1152 tokens of 2
  // heads take 32 us with one, 21 with two, 16 with four and 12 with eight.
  int blocks = 1;
  while (blocks < kMostBlocks && units * blocks <= sms) blocks *= 2;
  // A choice by several blocks meets nine times: for 1152 tokens one block is
  // faster (12 us against 14), for 8704 eight are (28 against 31).
  const bool alone = blocks == 1 || longest <= 4096;
  const int choosers = alone ? 1 : blocks;
  const int64_t part = (longest + choosers * kThreads - 1) / (choosers * kThreads) * kThreads;
  const int cache = static_cast<int>(part < kSelCache ? part : kSelCache);
  if (c.kind == 0)
    return alone ? launch<0, true>(c, e, units, blocks, cache, s) : launch<0, false>(c, e, units, blocks, cache, s);
  return alone ? launch<1, true>(c, e, units, blocks, cache, s) : launch<1, false>(c, e, units, blocks, cache, s);
}

}  // namespace sa
