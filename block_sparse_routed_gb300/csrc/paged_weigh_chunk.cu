// The attention weight that cached keys receive from chunks of rows (sm_103a):
// more than 16 packed rows a sequence and key head, on tcgen05 tensor cores.
//
//   w_j (+)= sum_r 2^(x_rj - L_r),   x_rj = scale log2(e) (q_r . k_j),  L_r = log2(e) lse_r
//
// The sum runs over rows, so keys are the products' M: a unit is 256 keys of
// one sequence and key head, two tiles of 128 that stay in tensor memory as
// the products' first operand while the rows that see some of them come by 96
// at a time.  A thread has a key: it reads the key's scores of 96 rows, and
// adds up their exponentials in registers.  Nothing passes between threads.
//
// Keys in tensor memory, because shared memory would not feed them: of a step
// (two tiles, 96 rows) products read Q there twice, 2 x 24 KB, and the copies
// write 24 KB, 560 cycles at 128 bytes a cycle, against 768 of the tensor
// pipe; with the keys in shared memory it would be 1060.
//
// The line of all steps of all units is cut into equal parts, one a CTA; a
// unit that a cut divides is joined from its parts in order by a second kernel.
//
// Warps: 0-2 gather Q (a group of any size, any strides), 32 rows each; 3
// walks the line and issues the products; 4-7 and 8-11 are the keys of tile 0
// and 1: they load the next unit's keys into registers while the present one's
// rows pass, widen codes, and write them to tensor memory.
//
// Tensor memory: K of tile t in columns [64 t, + 64); scores of tile t, every
// other step, in [128 + 96 (2 t + b), + 96).
#include <atomic>
#include <cstdint>

#include "internal.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sa {
namespace {

constexpr int kKeys = kWeighKeys;  // of a unit
constexpr int kRows = 96;          // packed rows of a step
constexpr int kStages = 4;
constexpr int kSegs = 3;
constexpr uint32_t kHalfBytes = kRows * 128;  // of a stage: 64 dimensions of its rows
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
// A unit's beginning and end, in steps.
constexpr int kOver = 3;
constexpr int kMinPlaces = 4;

constexpr int kThreads = 384;
// Registers after the split: their sum over warpgroups stays within the
// launch allocation (384 x 168).
constexpr uint32_t kRegsLaunch = 168, kRegsControl = 88, kRegsKeys = 208;
static_assert(kRegsControl + 2 * kRegsKeys <= 3 * kRegsLaunch, "");

// Shared memory, from a 1024-byte boundary.
constexpr uint32_t kOffNeg = kStages * kStageBytes;          // [stages][rows]: -L
constexpr uint32_t kOffPos = kOffNeg + kStages * kRows * 4;  // [stages][rows]: position
constexpr uint32_t kOffSeg = kOffPos + kStages * kRows * 4;
constexpr uint32_t kOffBar = kOffSeg + kSegs * 64;
constexpr uint32_t kOffMisc = kOffBar + 256;
constexpr uint32_t kSmem = kOffMisc + 64 + 1024;

enum {
  BAR_QFULL = 0,    // +stage (4): 96 lanes' copies and 3 warps
  BAR_QEMPTY = 4,   // +stage: the products and 8 warps of keys
  BAR_SFULL = 8,    // +2 tile, + every other step
  BAR_SEMPTY = 12,
  BAR_KREADY = 16,  // +tile
  BAR_SEGFULL = 18, // +segment (3)
  BAR_SEGEMPTY = 21,
  BAR_DRAIN = 24,
  NUM_BARS = 25
};

// One step of the walk: some steps of a unit.
struct Work {
  int valid;
  int row0, n, len, h, s;
  int key0;    // first key of the unit
  int lo, hi;  // its keys whose weight is written
  int rho0;    // first packed row
  int end;     // past the last
  int steps;
  int part;    // -1: the unit's weights; else the partial sums' slot (0 or 1)
};
static_assert(sizeof(Work) <= 64, "");

struct Unit {
  int lo, hi;      // keys whose weight is written
  int rho0, rows;  // packed rows that see some of them
  int steps, places;
};

// Keys of a sequence whose weights are written: [lo, hi).
__device__ __forceinline__ void seq_span(const WeighArgs& w, const PagedSeq& q, int& lo, int& hi) {
  lo = w.accumulate ? max(w.first, row_lo(w.a, q.len - q.n)) : w.first;
  hi = q.n > 0 ? q.len : 0;
}
__device__ __forceinline__ int blocks_of(int lo, int hi) {
  return hi > lo ? (hi + kKeys - 1) / kKeys - lo / kKeys : 0;
}

// Unit b of a sequence with the span [lo, hi).
__device__ __forceinline__ Unit unit_of(const WeighArgs& w, const PagedSeq& q, int lo, int hi, int b) {
  Unit u;
  const int key0 = (lo / kKeys + b) * kKeys;
  u.lo = max(lo, key0);
  u.hi = min(hi, key0 + kKeys);
  int i0 = 0, i1 = q.n;
  const int base = q.len - q.n;  // position of the first row
  if (w.a.causal) {
    i0 = min(max(u.lo - base, 0), q.n);
    if (w.a.window) i1 = static_cast<int>(min(int64_t(q.n), max(int64_t(i0), int64_t(u.hi) - 1 + w.a.window - base)));
  }
  u.rho0 = i0 * w.a.group;
  u.rows = (i1 - i0) * w.a.group;
  u.steps = max(1, (u.rows + kRows - 1) / kRows);
  u.places = u.steps + kOver;
  return u;
}

// Places of one head of the sequences base + lane, one a lane.  All keys that
// lie before the first row and inside the last row's window have all rows:
// only the units beside them are looked at one by one, many of them by the
// whole warp.
__device__ __forceinline__ int64_t lane_places(const WeighArgs& w, int base, int lane, bool& bad) {
  const int s = base + lane;
  PagedSeq q;
  q.n = q.len = q.row0 = 0;
  if (s < w.a.c.seqs) {
    bool b;
    q = paged_seq(w.a.c, s, b);
    bad |= b;
  }
  int lo, hi;
  seq_span(w, q, lo, hi);
  const int n = blocks_of(lo, hi);
  int from = 0, to = n;  // units with all rows: [from, to)
  if (w.a.causal) {
    const int first = lo / kKeys;
    to = min(n, max(0, (q.len - q.n) / kKeys + 1 - first));  // those that begin at or before the first row
    if (w.a.window) {  // those that end behind what the last row sees last
      const int64_t cut = int64_t(q.len) - w.a.window;
      while (from < to && int64_t(first + from + 1) * kKeys <= cut) ++from;
    }
    if (to > 0 && max(lo, (first + to - 1) * kKeys) > q.len - q.n) --to;
    to = max(to, from);
  }
  int64_t t = 0;
  if (to > from) t = static_cast<int64_t>(to - from) * unit_of(w, q, lo, hi, from).places;
  const int others = n - (to - from);
  if (others <= 4)
#pragma unroll 1
    for (int i = 0; i < others; ++i) t += unit_of(w, q, lo, hi, i < from ? i : i + to - from).places;
  unsigned many = __ballot_sync(0xFFFFFFFFu, others > 4);
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    PagedSeq r;
    r.row0 = 0;
    r.n = __shfl_sync(0xFFFFFFFFu, q.n, src);
    r.len = __shfl_sync(0xFFFFFFFFu, q.len, src);
    const int rlo = __shfl_sync(0xFFFFFFFFu, lo, src), rhi = __shfl_sync(0xFFFFFFFFu, hi, src);
    const int rfrom = __shfl_sync(0xFFFFFFFFu, from, src), rto = __shfl_sync(0xFFFFFFFFu, to, src);
    const int rothers = __shfl_sync(0xFFFFFFFFu, others, src);
    int64_t y = 0;
#pragma unroll 1
    for (int i = lane; i < rothers; i += 32) y += unit_of(w, r, rlo, rhi, i < rfrom ? i : i + rto - rfrom).places;
    y = warp_sum(y);
    if (lane == src) t += y;
  }
  return t;
}

struct Walk {
  int64_t at, end, total;
  int ctas;
  int s, h, b;
  int skip;  // places of the unit that earlier CTAs have
  PagedSeq q;
  int lo, hi, blocks;
};

__device__ __forceinline__ void walk_to(const WeighArgs& w, Walk& k) {
  bool bad;
  k.q = paged_seq(w.a.c, k.s, bad);
  seq_span(w, k.q, k.lo, k.hi);
  k.blocks = blocks_of(k.lo, k.hi);
}

__device__ __forceinline__ void walk_start(const WeighArgs& w, Walk& k, bool& bad) {
  const int lane = threadIdx.x % 32, cta = blockIdx.x;
  const PagedArgs& c = w.a.c;
  int64_t t = 0;
#pragma unroll 1
  for (int base = 0; base < c.seqs; base += 32) t += lane_places(w, base, lane, bad);
  k.total = warp_sum(t) * c.H;
  k.ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (k.total + kMinPlaces - 1) / kMinPlaces));
  k.at = k.end = 0;
  k.s = k.h = k.b = k.skip = 0;
  if (cta >= k.ctas) return;
  k.at = muldiv(cta, k.total, k.ctas);
  k.end = muldiv(cta + 1, k.total, k.ctas);
  int64_t left = k.at;
#pragma unroll 1
  for (int base = 0;; base += 32) {
    bool b;
    const int64_t mine = lane_places(w, base, lane, b) * c.H;
    const int64_t upto = warp_scan(mine, lane);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, upto > left);
    if (hit) {
      const int src = __ffs(hit) - 1;
      k.s = base + src;
      left = __shfl_sync(0xFFFFFFFFu, left - (upto - mine), src);
      t = __shfl_sync(0xFFFFFFFFu, mine, src);
      break;
    }
    left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  walk_to(w, k);
  t = muldiv(t, 1, c.H);
  k.h = static_cast<int>(muldiv(left, 1, t));
  left -= k.h * t;
  for (int b0 = 0;; b0 += 32) {
    const int64_t mine = b0 + lane < k.blocks ? unit_of(w, k.q, k.lo, k.hi, b0 + lane).places : 0;
    const int64_t upto = warp_scan(mine, lane);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, upto > left);
    if (hit) {
      const int src = __ffs(hit) - 1;
      k.b = b0 + src;
      k.skip = static_cast<int>(__shfl_sync(0xFFFFFFFFu, left - (upto - mine), src));
      return;
    }
    left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
}

__device__ __forceinline__ Work walk_step(const WeighArgs& w, Walk& k, WeighJoin& join) {
  Work g;
  g.valid = 0;
  while (k.at < k.end) {
    while (k.b >= k.blocks) {  // next head, next sequence with keys
      k.b = 0;
      if (k.blocks == 0 || ++k.h >= w.a.c.H) {
        k.h = 0;
        ++k.s;
        walk_to(w, k);
      }
    }
    const Unit u = unit_of(w, k.q, k.lo, k.hi, k.b);
    const int take = static_cast<int>(min(static_cast<int64_t>(u.places - k.skip), k.end - k.at));
    const int from = max(0, k.skip - kOver), to = max(0, k.skip + take - kOver);
    if (to > from) {
      g.valid = 1;
      g.row0 = k.q.row0;
      g.n = k.q.n;
      g.len = k.q.len;
      g.h = k.h;
      g.s = k.s;
      g.key0 = (k.lo / kKeys + k.b) * kKeys;
      g.lo = u.lo;
      g.hi = u.hi;
      g.rho0 = u.rho0 + from * kRows;
      g.end = u.rho0 + u.rows;
      g.steps = to - from;
      g.part = from == 0 ? (to == u.steps ? -1 : 1) : 0;
      if (g.part == 1) {  // the CTA that holds the unit's last place
        join.pieces = static_cast<int>(muldiv((k.at - k.skip + u.places) * k.ctas - 1, 1, k.total)) - static_cast<int>(blockIdx.x) + 1;
        join.s = g.s;
        join.h = g.h;
        join.key0 = g.key0;
        join.lo = g.lo;
        join.hi = g.hi;
        join.fresh = w.accumulate ? g.len - g.n : 0;
      }
    }
    k.at += take;
    k.skip = 0;
    ++k.b;
    if (g.valid) break;
  }
  return g;
}

__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void lds_f2x2(uint64_t& a, uint64_t& b, uint32_t addr) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}
__device__ __forceinline__ void lds_i4(int (&v)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}

// A key in registers: its row as it lies in the cache, and where its weight is.
template <int kKind>
struct Key {
  uint4 x[kKind == 0 ? 16 : 8];
  uint32_t exp;
  float old;
  int64_t at;  // of the weight; -1: none is written
};

template <int kKind>
__global__ void __launch_bounds__(kThreads, 1) weigh_chunk_kernel(const WeighArgs w, const WeighScratch ws) {
  const PagedAttnArgs& a = w.a;
  const PagedArgs& c = a.c;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(base);
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * i; };
  Work* segs = reinterpret_cast<Work*>(base + kOffSeg);
  volatile int32_t* s_abort = reinterpret_cast<volatile int32_t*>(base + kOffMisc);
  int32_t* s_bad = reinterpret_cast<int32_t*>(base + kOffMisc + 4);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(base + kOffMisc + 8);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    *s_abort = 0;
    *s_bad = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(BAR_QFULL + i), 3);
      mbar_init(bar(BAR_QEMPTY + i), 9);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(BAR_SFULL + i), 1);
      mbar_init(bar(BAR_SEMPTY + i), 4);
    }
    for (int t = 0; t < 2; ++t) mbar_init(bar(BAR_KREADY + t), 4);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(bar(BAR_SEGFULL + i), 1);
      mbar_init(bar(BAR_SEGEMPTY + i), 11);
    }
    mbar_init(bar(BAR_DRAIN), 1);
    fence_barrier_init();
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(tslot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tslot, 0);

  // By a whole warp; fails once another warp has given up, too.
  auto all_wait = [&](int b, int parity) {
    if (__all_sync(0xFFFFFFFFu, mbar_test_wait(bar(b), parity & 1))) return true;
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar(b), parity & 1, a.wait_limit) && *s_abort == 0) != 0;
  };
  auto next_seg = [&](int k, Work& g) -> bool {
    if (!all_wait(BAR_SEGFULL + k % kSegs, k / kSegs)) return false;
    g = segs[k % kSegs];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(BAR_SEGEMPTY + k % kSegs));
    return true;
  };
  bool ok = true;

  if (warp < 4) setmaxnreg_dec<kRegsControl>();
  if (warp < 3) {
    // ------------------------------------------------------------ rows of Q
    int x = 0;  // steps so far
    int pending = -1;  // the step whose copies are under way
    auto publish = [&](int step) {  // its copies have landed
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_QFULL + step % kStages));
    };
    for (int k = 0; ok; ++k) {
      Work g;
      ok = next_seg(k, g);
      if (!ok || !g.valid) break;
      for (int j = 0; j < g.steps; ++j, ++x) {
        const int st = x % kStages;
        ok = x < kStages || all_wait(BAR_QEMPTY + st, x / kStages - 1);
        if (!ok) break;
        const int r = 32 * warp + lane, rho = g.rho0 + j * kRows + r;
        const bool real = rho < g.end;
        const int i = div_group(a, rho), e = rho - i * a.group;
        const uint16_t* mine = a.q;
        float neg = -INFINITY;
        if (real) {
          mine += static_cast<int64_t>(g.row0 + i) * a.q_token + static_cast<int64_t>(g.h * a.group + e) * a.q_head;
          const float l = __ldg(w.lse + static_cast<int64_t>(g.row0 + i) * a.Hq + g.h * a.group + e);
          if (l != -INFINITY) neg = -l * 1.4426950408889634f;
        }
        const uint32_t to = sbase + st * kStageBytes + (lane % 16 / 8) * kHalfBytes;
#pragma unroll 8
        for (int y = 0; y < 32; y += 2) {
          const int row = y + lane / 16;
          const uint16_t* src = reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(mine), row));
          const bool is = g.rho0 + j * kRows + 32 * warp + row < g.end;
          cp_async16(to + (32 * warp + row) * 128 + ((lane ^ row) & 7) * 16, src + (is ? lane % 16 * 8 : 0), is);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        *reinterpret_cast<float*>(base + kOffNeg + (st * kRows + r) * 4) = neg;
        *reinterpret_cast<int*>(base + kOffPos + (st * kRows + r) * 4) = real ? g.len - g.n + i : -0x40000000;
        if (pending >= 0) {
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          publish(pending);
        }
        pending = x;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ok && pending >= 0) publish(pending);
    if (!ok) *s_abort = 1;
  } else if (warp == 3) {
    // ------------------------------------------------------------ the line, and the products
    Walk walk;
    bool bad = false;
    walk_start(w, walk, bad);
    WeighJoin join;
    join.pieces = 0;
    const uint32_t id = idesc_bf16(128, kRows, false, false);
    auto off = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4); };
    const uint32_t elect = elect_one();
    auto give = [&](int k, const Work& g) -> bool {
      if (k >= kSegs && !all_wait(BAR_SEGEMPTY + k % kSegs, k / kSegs - 1)) return false;
      if (lane == 0) {
        segs[k % kSegs] = g;
        mbar_arrive(bar(BAR_SEGFULL + k % kSegs));
      }
      __syncwarp();
      return true;
    };
    int x = 0;            // steps so far
    int y0 = 0, y1 = 0;   // of tile 0 and 1
    int u0 = 0, u1 = 0;   // units of them
    bool issued = false;
    Work g = walk_step(w, walk, join);
    ok = give(0, g);
    for (int k = 0; ok && g.valid; ++k) {
      const Work next = walk_step(w, walk, join);
      ok = give(k + 1, next);
      const int tiles = g.hi > g.key0 + 128 ? 2 : 1;
      ok = ok && all_wait(BAR_KREADY, u0) && (tiles < 2 || all_wait(BAR_KREADY + 1, u1));
      ++u0;
      if (tiles == 2) ++u1;
#pragma unroll 1
      for (int j = 0; j < g.steps && ok; ++j, ++x) {
        const int st = x % kStages;
        ok = all_wait(BAR_QFULL + st, x / kStages);
        if (!ok) break;
        const uint64_t qs = sdesc_sw128(sbase + st * kStageBytes, 16, 1024);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= tiles) break;
          const int y = t ? y1 : y0, s = 2 * t + (y & 1);
          ok = y < 2 || all_wait(BAR_SEMPTY + s, y / 2 - 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + 128 + kRows * s;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) umma_ts_elect(d, tmem + 64 * t + 8 * kk, qs + off(kk), id, kk > 0 ? 1u : 0u, elect);
          if (elect) {
            umma_commit(bar(BAR_SFULL + s));
            if (t + 1 == tiles) umma_commit(bar(BAR_QEMPTY + st));
          }
          __syncwarp();
          issued = true;
        }
        ++y0;
        if (tiles == 2) ++y1;
      }
      g = next;
    }
    if (!ok) *s_abort = 1;
    if (elect && issued) {  // products in flight complete before the CTA ends
      umma_commit(bar(BAR_DRAIN));
      mbar_wait(bar(BAR_DRAIN), 0, kWaitLimitNs);
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      ws.join[blockIdx.x] = join;
      if (bad) *s_bad = 1;
    }
  } else {
    // ------------------------------------------------------------ keys of tile t
    setmaxnreg_inc<kRegsKeys>();
    const int t = (warp - 4) / 4;
    const int row = (warp & 3) * 32 + lane;  // of the tile: a lane of tensor memory
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t k_col = tmem + lane_addr + 64 * t;
    const float c2 = a.scale * 1.4426950408889634f;
    const uint64_t c2x = f2(c2, c2);
    auto has = [&](const Work& g) { return g.valid && g.hi > g.key0 + 128 * t; };
    auto load = [&](const Work& g) {
      Key<kKind> key;
      key.at = -1;
      key.old = 0.f;
      key.exp = 0;
#pragma unroll
      for (auto& v : key.x) v = make_uint4(0, 0, 0, 0);
      const int j = g.key0 + 128 * t + row;
      if (!has(g) || j < g.lo || j >= g.hi) return key;
      const int page = __ldg(c.table + g.s * c.table_stride + (j >> c.page_shift));
      if (page < 0 || page >= c.pages) {
        *s_bad = 1;
        return key;
      }
      key.at = ((static_cast<int64_t>(page) * c.H + g.h) << c.page_shift) + (j & (c.page_size - 1));
      const uint8_t* src = c.k_pages + key.at * (kKind == 0 ? 256 : 128);
#pragma unroll
      for (int e = 0; e < (kKind == 0 ? 16 : 8); ++e) key.x[e] = ld_once(src + 16 * e);
      if constexpr (kKind != 0) key.exp = __ldg(c.k_exp + key.at);
      if (w.accumulate && j < g.len - g.n) key.old = w.weights[key.at];
      return key;
    };
    // The key's row in BF16 into tensor memory.
    auto store = [&](const Key<kKind>& key) {
      uint32_t z[2][32];
      if constexpr (kKind == 0) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          z[e / 8][e % 8 * 4] = key.x[e].x;
          z[e / 8][e % 8 * 4 + 1] = key.x[e].y;
          z[e / 8][e % 8 * 4 + 2] = key.x[e].z;
          z[e / 8][e % 8 * 4 + 3] = key.x[e].w;
        }
      } else {
        // codes land as the value times 2^-120; two factors, of 2^120 and the row's scale
        const uint32_t e1 = min(key.exp, 134u), two = key.exp == 255 ? 0x7FFF7FFFu : (e1 + 120) * 0x00800080u;
        const uint32_t more = (key.exp == 255 ? 127u : key.exp - e1 + 127) * 0x00800080u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t in[4] = {key.x[e].x, key.x[e].y, key.x[e].z, key.x[e].w};
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const uint32_t v = in[f];
            const uint32_t even = bf16x2_mul(bf16x2_mul(((v * 16) & 0x07F007F0u) | ((v * 256) & 0x80008000u), two), more);
            const uint32_t odd = bf16x2_mul(bf16x2_mul(((v >> 4) & 0x07F007F0u) | (v & 0x80008000u), two), more);
            z[e / 4][e % 4 * 8 + 2 * f] = __byte_perm(even, odd, 0x5410);
            z[e / 4][e % 4 * 8 + 2 * f + 1] = __byte_perm(even, odd, 0x7632);
          }
        }
      }
      tmem_st32(k_col, z[0]);
      tmem_st32(k_col + 32, z[1]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_KREADY + t));
    };
    int x = 0, y = 0;  // steps of the CTA, and of the tile
    Work g, next;
    ok = next_seg(0, g);
    Key<kKind> key;
    int64_t at = -1;
    float old = 0.f;
    if (ok) {
      key = load(g);
      if (has(g)) store(key);
      at = key.at;
      old = key.old;
    }
    for (int k = 0; ok && g.valid; ++k) {
      ok = next_seg(k + 1, next);
      if (!ok) break;
      key = load(next);
      const bool mine = has(g);
      float sum = 0.f;
      uint64_t acc[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[b] = f2(0.f, 0.f);
      const int j0 = g.key0 + 128 * t + row;
#pragma unroll 1
      for (int j = 0; j < g.steps; ++j, ++x) {
        const int st = x % kStages;
        ok = all_wait(BAR_QFULL + st, x / kStages);
        if (!ok) break;
        if (mine) {
          const int s = 2 * t + (y & 1);
          ok = all_wait(BAR_SFULL + s, y / 2);
          if (!ok) break;
          tc_fence_after();
          // the unit's last scores are there: the tile's K may be the next unit's
          if (j + 1 == g.steps && has(next)) store(key);
          ++y;
          // does some row of the step miss some key of the unit?
          bool edge = false;
          if (a.causal) {
            const int rho = g.rho0 + j * kRows, base_pos = g.len - g.n;
            edge = base_pos + div_group(a, rho) < g.hi - 1 ||
                   (a.window && static_cast<int64_t>(base_pos + div_group(a, min(rho + kRows, g.end) - 1)) - a.window >= g.lo);
          }
          const uint32_t col = tmem + lane_addr + 128 + kRows * s, negs = sbase + kOffNeg + st * kRows * 4,
                         poss = sbase + kOffPos + st * kRows * 4;
          uint32_t z[kRows / 32][32];
#pragma unroll
          for (int b = 0; b < kRows / 32; ++b) tmem_ld32(col + 32 * b, z[b]);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_SEMPTY + s));
          if (!edge) {
#pragma unroll
            for (int b = 0; b < kRows / 4; ++b) {
              uint64_t n0, n1;
              lds_f2x2(n0, n1, negs + 16 * b);
              const uint32_t* v = &z[b / 8][b % 8 * 4];
              float p0, p1, p2, p3;
              unf2(ffma2(f2(__uint_as_float(v[0]), __uint_as_float(v[1])), c2x, n0), p0, p1);
              unf2(ffma2(f2(__uint_as_float(v[2]), __uint_as_float(v[3])), c2x, n1), p2, p3);
              acc[2 * (b & 1)] = fadd2(acc[2 * (b & 1)], f2(ex2_approx(p0), ex2_approx(p1)));
              acc[2 * (b & 1) + 1] = fadd2(acc[2 * (b & 1) + 1], f2(ex2_approx(p2), ex2_approx(p3)));
            }
          } else {
#pragma unroll
            for (int b = 0; b < kRows / 4; ++b) {
              uint64_t n0, n1;
              int pos[4];
              lds_f2x2(n0, n1, negs + 16 * b);
              lds_i4(pos, poss + 16 * b);
              const uint32_t* v = &z[b / 8][b % 8 * 4];
              float p[4];
              unf2(ffma2(f2(__uint_as_float(v[0]), __uint_as_float(v[1])), c2x, n0), p[0], p[1]);
              unf2(ffma2(f2(__uint_as_float(v[2]), __uint_as_float(v[3])), c2x, n1), p[2], p[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                p[e] = j0 <= pos[e] && (!a.window || j0 > pos[e] - a.window) ? ex2_approx(p[e]) : 0.f;
              acc[0] = fadd2(acc[0], f2(p[0], p[1]));
              acc[1] = fadd2(acc[1], f2(p[2], p[3]));
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_QEMPTY + st));
      }
      if (!ok) break;
      if (mine) {
        float p, q;
        unf2(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), p, q);
        sum = p + q;
        if (g.part >= 0)
          ws.part[(static_cast<int64_t>(blockIdx.x) * 2 + g.part) * kKeys + 128 * t + row] = sum;
        else if (at >= 0)
          w.weights[at] = old + sum;
      } else if (has(next)) {
        store(key);
      }
      at = key.at;
      old = key.old;
      g = next;
    }
    if (!ok) {
      tmem_wait_st();
      *s_abort = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 3) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0) ws.cta_status[blockIdx.x] = *s_abort ? 5 /* SA_ETIMEOUT */ : (*s_bad ? kPagedInvalid : 0);
  griddep_launch_dependents();
}

// The units that a cut divided, their parts in order; and the call's status.
__global__ void __launch_bounds__(kKeys) weigh_join_kernel(const WeighArgs w, const WeighScratch ws) {
  griddep_wait();
  const PagedArgs& c = w.a.c;
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    int st = 0;
    for (int i = threadIdx.x; i < gridDim.x; i += 32) st = max(st, ws.cta_status[i]);
    st = __reduce_max_sync(0xFFFFFFFFu, st);
    if (threadIdx.x == 0) *c.status = st;
  }
  const WeighJoin d = ws.join[blockIdx.x];
  const int j = d.key0 + threadIdx.x;
  if (d.pieces == 0 || j < d.lo || j >= d.hi) return;
  const int page = c.table[d.s * c.table_stride + (j >> c.page_shift)];
  if (page < 0 || page >= c.pages) return;  // (reported)
  float sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < d.pieces; ++i)
    sum += ws.part[(static_cast<int64_t>(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * kKeys + threadIdx.x];
  float* to = w.weights + ((static_cast<int64_t>(page) * c.H + d.h) << c.page_shift) + (j & (c.page_size - 1));
  *to = (j < d.fresh ? *to : 0.f) + sum;
}

template <int kKind>
cudaError_t launch(const WeighArgs& w, const WeighScratch& ws, int ctas, cudaStream_t s) {
  auto* kern = weigh_chunk_kernel<kKind>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(kern), kSmem);
  if (e != cudaSuccess) return e;
  // The register split redistributes the launch allocation; a build with
  // fewer registers a thread would make setmaxnreg.inc wait forever.
  static std::atomic<int> known{0};
  int regs = known.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
    known.store(regs, std::memory_order_relaxed);
  }
  if (regs * 3 < static_cast<int>(kRegsControl + 2 * kRegsKeys)) return cudaErrorInvalidConfiguration;
  kern<<<ctas, kThreads, kSmem, s>>>(w, ws);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(weigh_join_kernel, dim3(ctas), dim3(kKeys), 0, s, w, ws);
}

}  // namespace

cudaError_t launch_weigh_chunk(const WeighArgs& w, const WeighScratch& ws, int ctas, cudaStream_t s) {
  return w.a.c.kind == 0 ? launch<0>(w, ws, ctas, s) : launch<1>(w, ws, ctas, s);
}

}  // namespace sa
