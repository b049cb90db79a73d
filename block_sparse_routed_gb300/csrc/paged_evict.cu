// Eviction from a paged cache by the weight that its keys received (sm_103a).
//
// For each sequence of more than `keep` tokens and each key head: the `first`
// and the `last` tokens stay, and of those between the keep - first - last
// with the largest weights (of equal ones the earlier).  Two kernels.
//
// Selection: a block a sequence and head.  Weights as integers whose order is
// theirs; the smallest that stays is found by its bytes from the top (four
// histograms), and the positions of what stays are written in order.
//
// Moving: token kept[i] goes to place i, in order, so i <= kept[i].  In place,
// a cluster takes a sequence and head and goes through the kept tokens from
// the first on, some at a time: all loads of one round complete (a barrier of
// the cluster) before its stores, which fill places below every source of the
// rounds that follow; so these may be loading already.
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
// Weights that the selection keeps in shared memory; longer sequences read
// them from memory (the second-level cache) each time.
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

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const PagedArgs c, const EvictArgs e) {
  extern __shared__ uint32_t s_keys[];
  __shared__ uint32_t s_hist[256];
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  __shared__ uint32_t s_prefix, s_left;
  const int s = blockIdx.x / c.H, h = blockIdx.x % c.H;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n = checked_length(c, e, s);
  int32_t* kept = e.kept + static_cast<int64_t>(blockIdx.x) * e.keep;
  if (h == 0 && threadIdx.x == 0) e.new_len[s] = n < 0 ? c.kv_len[s] : min(n, e.keep);
  if (n <= e.keep) {  // (a sequence that is refused moves nothing)
    for (int i = threadIdx.x; i < e.keep; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int m = n - e.first - e.last;                  // tokens to choose from
  const int want = e.keep - e.first - e.last;          // of them stay
  for (int i = threadIdx.x; i < e.first; i += kSelThreads) kept[i] = i;
  for (int i = threadIdx.x; i < e.last; i += kSelThreads) kept[e.keep - e.last + i] = n - e.last + i;
  if (want == 0) return;
  const int32_t* table = c.table + s * c.table_stride;
  auto weight_at = [&](int i) {
    const int pos = e.first + i, page = __ldg(table + (pos >> c.page_shift));
    return order_of(__ldg(e.weights + ((static_cast<int64_t>(page) * c.H + h) << c.page_shift) + (pos & (c.page_size - 1))));
  };
  const bool cached = m <= kSelCache;
  if (cached)
    for (int i = threadIdx.x; i < m; i += kSelThreads) s_keys[i] = weight_at(i);
  auto key = [&](int i) { return cached ? s_keys[i] : weight_at(i); };
  // the want-th largest key, byte by byte
  if (threadIdx.x == 0) {
    s_prefix = 0;
    s_left = want;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) s_hist[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int i = threadIdx.x; i < m; i += kSelThreads) {
      const uint32_t k = key(i);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&s_hist[k >> shift & 255], 1u);
    }
    __syncthreads();
    if (warp == 0) {  // lane: bins 255 - 8 lane .. down
      uint32_t mine[8], sum = 0;
#pragma unroll
      for (int b = 0; b < 8; ++b) sum += mine[b] = s_hist[255 - 8 * lane - b];
      uint32_t upto = sum;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += y;
      }
      const uint32_t left = s_left;
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
  }
  const uint32_t least = s_prefix;
  const int equals = s_left;  // of those equal to the least this many stay
  // Each warp has a part of the positions: counts first, then the places.
  const int part = (m + kSelThreads - 1) / kSelThreads * 32, i0 = min(m, warp * part), i1 = min(m, i0 + part);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key(i + lane) : 0u;
    const bool in = i + lane < i1;
    gt += __popc(__ballot_sync(0xFFFFFFFFu, in && k > least));
    eq += __popc(__ballot_sync(0xFFFFFFFFu, in && k == least));
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int gt_before = 0, eq_before = 0;
  for (int w = 0; w < warp; ++w) {
    gt_before += s_gt[w];
    eq_before += s_eq[w];
  }
  int at = gt_before + min(eq_before, equals);
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t k = in ? key(i + lane) : 0u;
    const unsigned same = __ballot_sync(0xFFFFFFFFu, in && k == least), below = (1u << lane) - 1;
    const bool stays = in && (k > least || (k == least && eq_before + __popc(same & below) < equals));
    const unsigned mask = __ballot_sync(0xFFFFFFFFu, stays);
    if (stays) kept[e.first + at + __popc(mask & below)] = e.first + i + lane;
    at += __popc(mask);
    eq_before += __popc(same);
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

constexpr int kMoveThreads = 256, kMoveWarps = kMoveThreads / 32;

template <int kKind>
struct Move {
  static constexpr int kRow = kKind == 0 ? 256 : 128;            // bytes of a row of K or V
  static constexpr int kTokenBytes = 2 * kRow;
  static constexpr int kPerWarp = kKind == 0 ? 12 : 24;          // tokens of a warp and round
  static constexpr int kTokens = kPerWarp * kMoveWarps;          // of a block and round
  static constexpr uint32_t kBuffer = kTokens * kTokenBytes;
  static constexpr uint32_t kSmem = 2 * kBuffer + 8 * kMoveThreads;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two blocks an SM");
};

// A warp moves its tokens alone; only the rounds' barriers join the warps.
template <int kKind>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const PagedArgs c, const EvictArgs e, int blocks) {
  using M = Move<kKind>;
  extern __shared__ __align__(128) uint8_t s_rows[];
  const int unit = blockIdx.x / blocks, rank = blockIdx.x % blocks;
  const int s = unit / c.H, h = unit % c.H;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool in_place = e.to_table == nullptr;
  const int32_t* kept = e.kept + static_cast<int64_t>(unit) * e.keep;
  const int32_t* from_table = c.table + s * c.table_stride;
  const int32_t* to_table = in_place ? from_table : e.to_table + s * e.to_stride;
  // (all entries of kept and the pages have been checked: a refused sequence has -1 throughout)
  const int n = kept[0] < 0 ? 0 : min(e.keep, c.kv_len[s]);
  const int step = M::kTokens * blocks;
  const int rounds = in_place && n == c.kv_len[s] ? 0 : (n + step - 1) / step;  // (n <= 2^30)
  const uint32_t base = smem_u32(s_rows) + warp * M::kPerWarp * M::kTokenBytes;
  const uint32_t side = smem_u32(s_rows) + 2 * M::kBuffer + threadIdx.x * 8;
  auto row_of = [&](const int32_t* table, int pos) -> int64_t {
    return ((static_cast<int64_t>(__ldg(table + (pos >> c.page_shift))) * c.H + h) << c.page_shift) + (pos & (c.page_size - 1));
  };
  struct Token {
    int64_t src, dst;  // rows; src < 0: nothing to move
    float w;
    uint8_t ke, ve;
  };
  // lane x < kPerWarp: token x of the warp and round
  auto begin = [&](int round) {
    Token t;
    t.src = t.dst = -1;
    t.w = 0.f;
    t.ke = t.ve = 0;
    const int i = round * step + (rank * kMoveWarps + warp) * M::kPerWarp + lane;
    if (lane < M::kPerWarp && i < n) {
      const int pos = kept[i];
      if (!in_place || pos != i) {
        t.src = row_of(from_table, pos);
        t.dst = row_of(to_table, i);
      }
    }
    const uint32_t to = base + (round & 1) * M::kBuffer;
    constexpr int kLanes = kKind == 0 ? 32 : 16, kAtOnce = 32 / kLanes;  // a token's lanes: half K, half V
    const int sub = lane % kLanes, chunk = sub % (kLanes / 2) * 16;
    const uint8_t* pages = sub < kLanes / 2 ? c.k_pages : c.v_pages;
#pragma unroll
    for (int x = 0; x < M::kPerWarp; x += kAtOnce) {
      const int mine = x + lane / kLanes;
      const int64_t src = __shfl_sync(0xFFFFFFFFu, t.src, mine);
      if (src >= 0) cp_async16(to + mine * M::kTokenBytes + sub * 16, pages + src * M::kRow + chunk, true);
    }
    cp_commit();
    if (t.src >= 0) {
      t.w = e.weights[t.src];
      if (kKind != 0) {
        t.ke = c.k_exp[t.src];
        t.ve = c.v_exp[t.src];
      }
    }
    return t;
  };
  auto finish = [&](int round, const Token& t) {
    const uint32_t from = base + (round & 1) * M::kBuffer;
    constexpr int kLanes = kKind == 0 ? 32 : 16, kAtOnce = 32 / kLanes;
    const int sub = lane % kLanes, chunk = sub % (kLanes / 2) * 16;
    uint8_t* pages = sub < kLanes / 2 ? c.k_pages : c.v_pages;
#pragma unroll
    for (int x = 0; x < M::kPerWarp; x += kAtOnce) {
      const int mine = x + lane / kLanes;
      const int64_t dst = __shfl_sync(0xFFFFFFFFu, t.dst, mine);
      if (dst >= 0) {
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(from + mine * M::kTokenBytes + sub * 16));
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
  if (rounds == 0) return;  // (alike in all blocks of a cluster)
  Token now = begin(0);
  for (int r = 0; r < rounds; ++r) {
    Token next;
    if (r + 1 < rounds) {
      next = begin(r + 1);
      cp_wait<1>();
    } else {
      cp_wait<0>();
    }
    __syncwarp();
    if (in_place) {
      // What a lane loads into registers has to arrive before the barrier, too:
      // a store needs it.
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(side), "r"(__float_as_uint(now.w)),
                   "r"(static_cast<uint32_t>(now.ke) | static_cast<uint32_t>(now.ve) << 8)
                   : "memory");
      cluster_sync();
    }
    finish(r, now);
    now = next;
  }
}

template <int kKind>
cudaError_t move(const PagedArgs& c, const EvictArgs& e, int blocks, cudaStream_t s) {
  using M = Move<kKind>;
  auto* kern = evict_move_kernel<kKind>;
  static SmemOnce once;
  cudaError_t err = once.set(reinterpret_cast<const void*>(kern), M::kSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(c.seqs) * c.H * blocks);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = M::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, c, e, blocks);
}

}  // namespace

cudaError_t launch_evict(const PagedArgs& c, const EvictArgs& e, int sms, cudaStream_t s) {
  static SmemOnce once;
  constexpr uint32_t bytes = kSelCache * 4;
  cudaError_t err = once.set(reinterpret_cast<const void*>(evict_select_kernel), bytes);
  if (err != cudaSuccess) return err;
  const int64_t longest = static_cast<int64_t>(c.table_width) << c.page_shift;
  const uint32_t need = static_cast<uint32_t>(longest < kSelCache ? longest : kSelCache) * 4;
  const int64_t units = static_cast<int64_t>(c.seqs) * c.H;
  evict_select_kernel<<<static_cast<unsigned>(units), kSelThreads, need, s>>>(c, e);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  // two blocks an SM, of which a sequence and head get up to eight
  int blocks = 8;
  while (blocks > 1 && units * blocks > 2 * sms) blocks /= 2;
  return c.kind == 0 ? move<0>(c, e, blocks, s) : move<1>(c, e, blocks, s);
}

}  // namespace sa
